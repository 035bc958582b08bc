"""Every kernel of dq_matmul and every way in which it divides the work, by cases that say which one they are for: a
change of the rule that chooses shows here as a failure, not as a kernel that no test runs.

Two comparisons a case.  Random operands against the fp64 product, with test_gpu_matmul's bound.  And operands whose
sums are known exactly: positive integers (codes of 8 to 15, or 3, 4 and 6) under one power-of-two scale a row.  All
partial sums, in any order, are integers below 2^24 times a power of two, so fp32 holds them without rounding and the
output has to be equal; sums of 16 to 22 bits leave no room for a partial result in fewer bits.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import linear_ref as ref
from calibration_free_weight_dualquant_b200 import binding

pytestmark = pytest.mark.gpu

FMTS = ["nvfp4", "mxfp4", "mxfp8"]
TYPES = [torch.float32, torch.bfloat16, torch.float16]
ALL, NV, MX = FMTS, ["nvfp4"], ["mxfp4", "mxfp8"]

# tokens, rows, cols, bytes by which the block scales are off a 32-byte boundary, formats,
# (kernel, tokens a tile, scales aligned, whole tiles, split tiles)
CASES = [
    # a CTA a tile: 16, 32, 64 and 128 tokens, whole and split
    (5, 128, 128, 0, ALL, ("tile", 16, False, True, False)),
    (9, 20001, 512, 0, ALL, ("tile", 16, True, True, False)),
    (3, 513, 4096, 0, ALL, ("tile", 16, True, False, True)),
    (16, 700, 2080, 0, ALL, ("tile", 16, False, False, True)),
    (20, 20000, 512, 0, ALL, ("tile", 32, True, True, False)),
    (31, 19001, 288, 0, ALL, ("tile", 32, False, True, False)),
    (17, 512, 4096, 16, ALL, ("tile", 32, True, False, True)),
    (32, 4096, 1056, 0, ALL, ("tile", 32, False, False, True)),
    (60, 20000, 1024, 0, ALL, ("tile", 64, True, True, False)),
    (60, 20000, 1056, 0, ALL, ("tile", 64, False, True, False)),
    (64, 640, 2048, 0, ALL, ("tile", 64, True, False, True)),
    (130, 300, 2080, 0, ALL, ("tile", 64, False, False, True)),
    (300, 6000, 512, 0, ALL, ("tile", 128, True, True, False)),
    (300, 6000, 288, 0, ALL, ("tile", 128, False, True, False)),
    (200, 2000, 12288, 0, ALL, ("tile", 128, True, False, True)),
    (200, 2000, 12064, 0, ALL, ("tile", 128, False, False, True)),
    # pairs: whole waves with a tail of columns and rows of Y at odd addresses, scales at every alignment
    (2100, 2305, 1056, 0, ALL, ("pair", 256, False, True, False)),
    (2100, 2560, 1056, 0, ALL, ("pair", 256, False, True, False)),
    (2300, 2501, 4096, 0, ALL, ("pair", 256, True, True, False)),
    (2300, 2500, 2048, 1, ALL, ("pair", 256, False, True, False)),
    (2300, 2500, 2048, 2, ALL, ("pair", 256, False, True, False)),
    (2300, 2504, 2048, 8, ALL, ("pair", 256, False, True, False)),
    (2300, 2504, 2048, 16, ALL, ("pair", 256, True, True, False)),
    # ... behind them tiles split over clusters, and split tiles alone
    (2304, 2560, 14336, 0, ALL, ("pair", 256, True, True, True)),
    (2100, 2201, 12064, 0, ALL, ("pair", 256, False, True, True)),
    (1500, 4096, 11008, 0, MX, ("pair", 256, False, True, True)),
    (512, 2048, 8192, 0, ALL, ("pair", 256, True, False, True)),
    (500, 2047, 8192, 0, ALL, ("pair", 256, True, False, True)),
    (300, 4096, 14336, 0, ALL, ("pair", 256, True, False, True)),
    (300, 4090, 14304, 0, ALL, ("pair", 256, False, False, True)),
    # codes that TMA cannot read
    (70, 130, 1040, 0, NV, ("any", 64, False, True, False)),
]
RUNS = [(c[:4], f, c[5]) for c in CASES for f in c[4]]
IDS = ["%s-%dx%dx%d+%d" % (f, *size) for size, f, _ in RUNS]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    binding.load_library()


def at_offset(t: torch.Tensor, by: int) -> torch.Tensor:
    buf = torch.empty(t.numel() * t.element_size() + 64, dtype=torch.uint8, device="cuda")
    v = buf[by:by + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
    v.copy_(t)
    return v


def on_device(q: dict, shift: int) -> dict:
    q = ref.to(q, "cuda")
    return dict(q, block_scales=at_offset(q["block_scales"], shift)) if shift else q


def which(x, w, fmt, out):
    k = binding.matmul_kernel(x, w, fmt, out)
    return k["kernel"], k["tile_tokens"], k["aligned_scales"], k["whole_tiles"] > 0, k["split_tiles"] > 0


def values(q: dict, fmt: str) -> torch.Tensor:
    """a q in fp64 on the device, without the tensor scale."""
    c, s = q["codes"].long(), q["block_scales"].long()
    if fmt == "mxfp8":
        table = torch.tensor(ref.code_values(fmt, np.arange(256, dtype=np.uint8)[None])[0], device="cuda")
        v = table[c]
    else:
        table = torch.tensor(np.concatenate([ref.E2M1, -ref.E2M1]), device="cuda")
        v = table[torch.stack([c & 15, c >> 4], dim=2).flatten(1)]
    a = torch.tensor(ref.block_values(fmt, np.arange(256)), device="cuda")[s]
    return (v.view(v.shape[0], a.shape[1], -1) * a[:, :, None]).flatten(1)


@pytest.mark.parametrize("size,fmt,kernel", RUNS, ids=IDS)
def test_random_operands(size, fmt, kernel):
    tokens, rows, cols, shift = size
    x = on_device(ref.random_quantized(tokens, cols, fmt, tokens + cols), shift)
    w = on_device(ref.random_quantized(rows, cols, fmt, rows + cols), shift)
    s = ref.tensor_scale(x, fmt) * ref.tensor_scale(w, fmt)
    xv, wv = values(x, fmt), values(w, fmt)
    want, sum_abs = (xv @ wv.T) * s, (xv.abs() @ wv.abs().T) * s
    for dt in TYPES[:2]:
        y = torch.empty(tokens, rows, dtype=dt, device="cuda")
        assert which(x, w, fmt, y) == kernel
        binding.dq_matmul(x, w, fmt, out=y)
        tol = (cols + 4) * 2.0 ** -24 * sum_abs
        tol = tol + torch.finfo(dt).eps / 2 * (want.abs() + tol)
        off = (y.double() - want).abs() > tol
        assert not off.any(), "%s: %d of %d" % (dt, off.sum().item(), off.numel())


LONG = [r for r in RUNS if r[0][2] >= 4096]


@pytest.mark.parametrize("size,fmt,kernel", LONG, ids=["%s-%dx%dx%d+%d" % (f, *size) for size, f, _ in LONG])
def test_rms_error_of_long_fp32_sums(size, fmt, kernel):
    """RMS error over sqrt(sum (x w)^2), the RMS of a sum of random signs.  The tensor core adds the products of 32
    (MXFP8) or 64 columns at a time to an fp32 sum; each addition is off by at most a unit of the last place, 2^-23 of a
    partial sum, whose RMS the whole one's bounds, and in the worst case all of them in one direction.  Two products
    with the tensor scales, and what is within an addition, one unit more, are 4 2^-24 together.  A partial sum in
    fp16 or bf16 would be off by about 2^-13 or 2^-10 of it: eight times
    the bound at 4096 columns and twice at 14336."""
    tokens, rows, cols, shift = size
    x = on_device(ref.random_quantized(tokens, cols, fmt, tokens + cols + 1), shift)
    w = on_device(ref.random_quantized(rows, cols, fmt, rows + cols + 1), shift)
    s = ref.tensor_scale(x, fmt) * ref.tensor_scale(w, fmt)
    xv, wv = values(x, fmt), values(w, fmt)
    y = binding.dq_matmul(x, w, fmt, out_dtype=torch.float32).double()
    error = (y - (xv @ wv.T) * s) / (((xv * xv) @ (wv * wv).T).sqrt() * s)
    additions = -(-cols // (32 if fmt == "mxfp8" else 64))
    assert error.square().mean().sqrt().item() <= additions * 2.0 ** -23 + 4 * 2.0 ** -24


def integers(rows: int, cols: int, fmt: str, seed: int, exps):
    """(quantized matrix, integer values, scale exponent of each row)."""
    rng = torch.Generator().manual_seed(seed)
    ints = torch.arange(8, 16) if fmt == "mxfp8" else torch.tensor([3, 4, 6])
    table = ints.float().to(torch.float8_e4m3fn).view(torch.uint8) if fmt == "mxfp8" else torch.tensor([5, 6, 7], dtype=torch.uint8)
    i = torch.randint(0, len(ints), (rows, cols), generator=rng)
    c = table[i] if fmt == "mxfp8" else table[i[:, 0::2]] | (table[i[:, 1::2]] << 4)
    e = torch.randint(*exps, (rows,), generator=rng)
    byte = (8 * (e + 7) if fmt == "nvfp4" else e + 127).to(torch.uint8)
    scales = byte[:, None].repeat(1, cols // ref.GROUP[fmt])
    return ({"codes": c.contiguous(), "block_scales": scales, "tensor_scale": torch.ones(1)}, ints[i].double().cuda(),
            e.double().cuda())


@pytest.mark.parametrize("size,fmt,kernel", RUNS, ids=IDS)
def test_exact_sums(size, fmt, kernel):
    """Equality in every output type, with Y at an odd address too, a NaN scale in one row of each operand, and (NVFP4)
    tensor scales whose product leaves fp32's normal range, so that it is applied in two factors."""
    tokens, rows, cols, shift = size
    exps = (-3, 4) if fmt == "nvfp4" else (-20, 20)
    x, xv, xe = integers(tokens, cols, fmt, 3 * tokens + cols, exps)
    w, wv, we = integers(rows, cols, fmt, 5 * rows + cols, exps)
    x["block_scales"][tokens - 2, -1] = w["block_scales"][rows - 2, 0] = 0x7F if fmt == "nvfp4" else 0xFF
    x, w = on_device(x, shift), on_device(w, shift)
    want = (xv @ wv.T) * torch.exp2(xe[:, None] + we[None, :])
    want[tokens - 2] = want[:, rows - 2] = float("nan")
    for sx, sw in ((1.0, 1.0), (2.0 ** -100, 2.0 ** -31)) if fmt == "nvfp4" else ((1.0, 1.0),):
        x["tensor_scale"].fill_(sx)
        w["tensor_scale"].fill_(sw)
        for dt in TYPES:
            expected = (want * (sx * sw)).float().to(dt)  # exact in fp32, so rounded once
            for odd in (0, 1):
                buf = torch.full((tokens * rows + 96,), -7.0, dtype=dt, device="cuda")
                y = buf[32 + odd:32 + odd + tokens * rows].view(tokens, rows)
                assert which(x, w, fmt, y) == kernel
                binding.dq_matmul(x, w, fmt, out=y)
                same = (y == expected) | (torch.isnan(y) & torch.isnan(expected))
                assert same.all(), "%s +%d: %d of %d differ" % (dt, odd, (~same).sum().item(), same.numel())
                assert (buf[:32 + odd] == -7).all() and (buf[32 + odd + tokens * rows:] == -7).all()


def test_the_cases_reach_every_kernel():
    reached = {(f, *k) for _, f, k in RUNS}
    for f in FMTS:
        for aligned in (True, False):
            for whole, split in ((True, False), (False, True)):
                for tokens in (16, 32, 64, 128):
                    assert (f, "tile", tokens, aligned, whole, split) in reached
                assert (f, "pair", 256, aligned, whole, split) in reached
            assert (f, "pair", 256, aligned, True, True) in reached
    assert ("nvfp4", "any", 64, False, True, False) in reached


def test_kernel_query_arguments():
    x = ref.to(ref.random_quantized(2, 64, "mxfp8", 1), "cuda")
    y = torch.empty(2, 2, device="cuda")
    assert binding.matmul_kernel(x, x, "mxfp8", y) == {
        "kernel": "tile", "tile_tokens": 16, "aligned_scales": False, "whole_tiles": 1, "split_tiles": 0, "split": 1}
    with pytest.raises(binding.DQError) as e:
        binding.matmul_kernel(x, x, "mxint8", y)
    assert e.value.status == 2
