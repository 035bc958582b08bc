"""Ends of the ranges of the quantized linear layer's operators: tensor scales whose product leaves fp32's range
upwards, and norms of values so small that their share of the row is subnormal."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import linear_ref as ref
from calibration_free_weight_dualquant_b200 import binding, synth

pytestmark = pytest.mark.gpu

FMTS = ["nvfp4", "mxfp4", "mxfp8"]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    binding.load_library()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,rows,cols", [(5, 70, 256), (200, 300, 512), (2400, 2600, 512), (5, 70, 272)])
def test_matmul_tensor_scales_near_the_largest(dt, tokens, rows, cols):
    """The product of the tensor scales is beyond 2^255: an output whose sum is 0 is 0, every other one an infinity
    (the smallest nonzero sum is 2^-20)."""
    x = ref.random_quantized(tokens, cols, "nvfp4", 1)
    w = ref.random_quantized(rows, cols, "nvfp4", 2)
    x["codes"][3] = 0
    w["codes"][41] = 0
    x["tensor_scale"][0], w["tensor_scale"][0] = 3.3e38, -3.3e38
    y = binding.dq_matmul(ref.to(x, "cuda"), ref.to(w, "cuda"), "nvfp4", out_dtype=dt)
    want, _ = ref.matmul(x, w, "nvfp4")
    assert (want[3] == 0).all() and (want[:, 41] == 0).all()
    assert np.array_equal(ref.f64(y), np.where(want == 0, 0.0, np.copysign(np.inf, want)))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens,cols", [(40, 2048), (700, 1024), (3, 9216), (2, 40000)])
def test_norm_of_tiny_values_in_large_rows(fmt, tokens, cols):
    """h / rms(h) is subnormal in fp32 where g b brings it back into range: scales and codes are those of the fp64
    values all the same."""
    rng = torch.Generator().manual_seed(tokens + cols)
    x = 1000 * synth.make_activations(tokens, cols, seed=5).float()
    w = 1 + 0.3 * torch.randn(cols, generator=rng)
    b = torch.ones(cols)
    tiny = (torch.arange(cols) // ref.GROUP[fmt]) % 2 == 1
    k = torch.randint(-7, 8, (tokens, cols), generator=rng).double() * 2.0 ** -133
    x = torch.where(tiny, k, x.double()).to(torch.bfloat16)
    assert (x[:, tiny].double() == k[:, tiny]).all()  # bf16 subnormals
    w = torch.where(tiny, w.abs().clamp(0.5, 1.5) * 2.0 ** 120, w).to(torch.bfloat16)
    b = torch.where(tiny, torch.tensor(2.0 ** 5), b).to(torch.bfloat16)
    got = binding.dq_norm_quant(x.cuda(), w.cuda(), b.cuda(), fmt)
    want = ref.quantize(ref.norm(x, None, w, b, 1e-5)[1], fmt)
    if fmt == "nvfp4":
        assert np.float32(got["tensor_scale"].cpu()[0]) == want["tensor_scale"]
    for name in ("block_scales", "codes"):
        bad = got[name].cpu().numpy() != want[name]
        assert not bad.any(), "%s: %d of %d differ" % (name, bad.sum(), bad.size)
