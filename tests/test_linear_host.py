"""Refusals of dq_matmul, dq_norm_quant and dq_glu_quant: every bad argument is found on the host, before
anything is enqueued (no GPU needed)."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import linear_ref as ref
from calibration_free_weight_dualquant_b200 import binding, build

FAKE = 0x100000  # an aligned address; never dereferenced by a refused call


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def outs(codes=FAKE, scales=FAKE, sT=FAKE):
    return binding._Outputs(codes, scales, sT, None, None)


def matmul(lib, tokens=4, rows=8, cols=64, fmt=3, group=32, y=FAKE, dt=1, ws=FAKE, nbytes=256, X=None, W=None):
    x, w = X or outs(), W or outs()
    return lib.dq_matmul(ctypes.byref(x), tokens, ctypes.byref(w), rows, cols, fmt, group, y, dt, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=0), 1), (dict(rows=0), 1), (dict(cols=0), 1), (dict(tokens=-1), 1), (dict(cols=48), 1),
    (dict(fmt=-1), 1), (dict(fmt=6), 1), (dict(fmt=0, group=64), 2), (dict(fmt=1), 2), (dict(fmt=4), 2),
    (dict(fmt=2, group=32), 2), (dict(fmt=3, group=16), 2), (dict(dt=3), 1), (dict(y=None), 1), (dict(y=FAKE + 1), 1),
    (dict(dt=0, y=FAKE + 2), 1), (dict(ws=FAKE + 16), 1), (dict(nbytes=255), 3),
    (dict(X=outs(codes=None)), 1), (dict(W=outs(scales=None)), 1), (dict(fmt=2, group=16, X=outs(sT=None)), 1),
    (dict(fmt=2, group=16, W=outs(sT=FAKE + 2)), 1), (dict(tokens=2 ** 31), 2), (dict(tokens=2 ** 30, rows=2 ** 30), 2),
    (dict(cols=2 ** 27 + 32), 2),
])
def test_matmul_refusals(lib, kw, status):
    assert matmul(lib, **kw) == status


def norm(lib, X=FAKE, r=None, xdt=1, rows=2, cols=64, g=FAKE, eps=1e-5, b=FAKE, bdt=1, fmt=5, group=32, out=None, ro=None,
         ws=FAKE, nbytes=1024):
    o = out or outs()
    return lib.dq_norm_quant(X, r, xdt, rows, cols, g, eps, b, bdt, fmt, group, ctypes.byref(o), ro, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=0), 1), (dict(cols=0), 1), (dict(cols=40), 1), (dict(fmt=9), 1), (dict(fmt=0, group=64), 2),
    (dict(fmt=4), 2), (dict(fmt=2, group=32), 2), (dict(xdt=0), 2), (dict(bdt=0), 2), (dict(X=None), 1),
    (dict(X=FAKE + 8), 1), (dict(g=FAKE + 2), 1), (dict(b=FAKE + 1), 1), (dict(r=FAKE), 1), (dict(ro=FAKE), 1),
    (dict(r=FAKE, ro=FAKE + 4), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(out=outs(codes=FAKE + 4)), 1), (dict(out=outs(scales=None)), 1),
    (dict(fmt=2, group=16, out=outs(sT=None)), 1), (dict(fmt=2, group=16, ws=None), 1), (dict(ws=FAKE + 128), 1), (dict(nbytes=255), 3),
    (dict(fmt=2, group=16, nbytes=256), 3), (dict(rows=2 ** 40), 2), (dict(rows=1, cols=2 ** 31), 2),
])
def test_norm_refusals(lib, kw, status):
    assert norm(lib, **kw) == status


def test_norm_workspace_sizes(lib):
    assert lib.dq_norm_workspace_bytes(7, 64, 5, 32) == 256
    assert lib.dq_norm_workspace_bytes(7, 64, 2, 16) == 256 + 56
    for bad in ((0, 64, 5, 32), (7, 0, 5, 32), (7, 64, 4, 32), (7, 64, 5, 16), (7, 40, 5, 32), (2 ** 40, 64, 5, 32)):
        assert lib.dq_norm_workspace_bytes(*bad) == 0


def glu(lib, gate=FAKE, up=FAKE, xdt=1, rows=2, cols=64, ld=128, b=FAKE, bdt=1, fmt=5, group=32, out=None, ws=FAKE,
        nbytes=256):
    o = out or outs()
    return lib.dq_glu_quant(gate, up, xdt, rows, cols, ld, b, bdt, fmt, group, ctypes.byref(o), ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=0), 1), (dict(cols=72), 1), (dict(ld=56), 1), (dict(ld=132), 1), (dict(gate=None), 1), (dict(up=None), 1),
    (dict(gate=FAKE + 2), 1), (dict(up=FAKE + 8), 1), (dict(xdt=0), 2), (dict(fmt=1), 2), (dict(fmt=2), 2),
    (dict(b=FAKE + 1), 1), (dict(bdt=0), 2), (dict(out=outs(codes=None)), 1), (dict(ws=FAKE + 8), 1), (dict(nbytes=0), 3),
    (dict(fmt=2, group=16, out=outs(sT=None)), 1), (dict(rows=2 ** 32, ld=2 ** 20), 1), (dict(rows=1, cols=2 ** 31, ld=2 ** 31), 2),
])
def test_glu_refusals(lib, kw, status):
    assert glu(lib, **kw) == status


def test_binding_refuses_cpu_tensors_and_other_formats(lib):
    x = ref.random_quantized(2, 64, "mxfp4", 1)
    with pytest.raises(binding.DQError) as e:
        binding.dq_matmul(x, x, "mxfp4")
    assert e.value.status == 1
    for f in (lambda: binding.dq_matmul(x, x, "int4"), lambda: binding.dq_norm_quant(torch.zeros(2, 64), None, None, "mxint8"),
              lambda: binding.dq_glu_quant(torch.zeros(2, 128), None, "mxint4")):
        with pytest.raises(binding.DQError) as e:
            f()
        assert e.value.status == 2
    with pytest.raises(binding.DQError):
        binding.dq_norm_quant(torch.zeros(2, 64, dtype=torch.bfloat16), None, None, "mxfp8")
    with pytest.raises(binding.DQError):
        binding.dq_glu_quant(torch.zeros(2, 128, dtype=torch.bfloat16), None, "mxfp8")


def test_binding_refuses_another_devices_stream():
    class Stream:
        device_index, cuda_stream = 1, 0

    with pytest.raises(binding.DQError) as e:
        binding._call(torch.device("cuda", 0), Stream(), lambda *a: None)
    assert e.value.status == 1


def test_reference_quantizer_pins():
    """The tests' own definition on values whose answers are known."""
    x = np.zeros((1, 32))
    x[0, :8] = [448.0, 464.0, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, -1.0, -2.0 ** -11]
    q = ref.quantize(x, "mxfp8")
    assert q["block_scales"][0, 0] == 127
    v = ref.code_values("mxfp8", q["codes"])[0, :8]
    assert v.tolist() == [448.0, 448.0, 16.0, 20.0, 0.0, 2.0 ** -8, -1.0, 0.0]
    assert q["codes"][0, 7] == 0  # no negative zero
    x = np.zeros((1, 32))
    x[0, :8] = [6.0, 5.0, 2.5, 0.25, 0.75, 1.25, 1.75, -3.5]
    q = ref.quantize(x, "mxfp4")
    assert ref.code_values("mxfp4", q["codes"])[0, :8].tolist() == [6.0, 4.0, 2.0, 0.0, 1.0, 1.0, 2.0, -4.0]
    x[0, 0] = 9.0  # ratio 1.5: the scale goes up to 2
    assert ref.quantize(x, "mxfp4")["block_scales"][0, 0] == 128
    x[0, 0] = np.nan
    q = ref.quantize(x, "nvfp4")
    assert q["block_scales"][0].tolist() == [0x7F, 0x38] and not q["codes"][0, :8].any()
    one = {"codes": torch.tensor([[0x21] + [0] * 15], dtype=torch.uint8), "block_scales": torch.tensor([[128]], dtype=torch.uint8)}
    assert ref.decode(one, "mxfp4")[0, :3].tolist() == [1.0, 2.0, 0.0]
