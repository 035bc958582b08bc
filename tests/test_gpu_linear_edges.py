"""Ends of the ranges of the quantized linear layer's operators: tensor scales whose product leaves fp32's range
upwards."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import linear_ref as ref
from calibration_free_weight_dualquant_b200 import binding

pytestmark = pytest.mark.gpu


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
