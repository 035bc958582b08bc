"""dq_matmul against the fp64 product of the decoded operands.

Tolerance of an output y with S = sum |x| |w|: K fp32 additions in any order, each off by at most 2^-24 of a
partial sum that S bounds, then the tensor scales (two multiplications, 2^-24 each) and one rounding to the output
type (half a step, eps/2, of a value that already carries the rest).  The type's largest value m becomes an
infinity half a step further on, from m (1 + eps/4) at the latest: 65520 for f16, whose m is 65504.
"""
from __future__ import annotations

import threading

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


def check(y: torch.Tensor, x: dict, w: dict, fmt: str, label: str = ""):
    want, mags = ref.matmul(x, w, fmt)
    got = ref.f64(y)
    tol = (x_cols(x, fmt) + 4) * 2.0 ** -24 * mags
    half = torch.finfo(y.dtype).eps / 2
    top = torch.finfo(y.dtype).max
    over, under = np.abs(want) - tol > top * (1 + half), np.abs(want) + tol < top
    assert np.array_equal(got[over], np.copysign(np.inf, want[over])), label
    tol = tol + half * (np.abs(want) + tol) + torch.finfo(y.dtype).tiny * half
    fine = np.isfinite(want) & (under | (np.isfinite(got) & ~over))
    assert np.array_equal(np.isnan(want), np.isnan(got)), label
    off = np.abs(got - want)[fine] > tol[fine]
    assert not off.any(), "%s: %d of %d outputs off, worst %g times the tolerance" % (
        label, off.sum(), off.size, (np.abs(got - want)[fine] / tol[fine]).max())


def x_cols(x: dict, fmt: str) -> int:
    return x["codes"].shape[1] * (1 if fmt == "mxfp8" else 2)


def case(tokens, rows, cols, fmt, seed):
    return ref.random_quantized(tokens, cols, fmt, seed), ref.random_quantized(rows, cols, fmt, seed + 1)


SHAPES = [
    (1, 1, 32), (1, 128, 256), (2, 3, 64), (1, 4096, 4096), (7, 129, 96), (8, 1024, 4096), (9, 130, 512),
    (16, 4096, 14336), (17, 255, 288), (31, 128, 1024), (33, 257, 1056), (64, 640, 2048), (65, 64, 320),
    (100, 1001, 1056), (128, 128, 128), (129, 1024, 4096), (255, 384, 544), (256, 256, 256), (257, 513, 1120),
    (300, 96, 8192), (700, 1000, 1312), (1025, 2049, 160),
    # tiles of 256 x 256 left over after whole waves of the SM pairs, split in 2, 3 and 4, and a part of a wave
    (2300, 2500, 4096), (2500, 2300, 1024), (2000, 2600, 4096), (500, 2049, 4096), (300, 600, 4096),
    # tiles of 64 and 128 tokens, whole and split, and few pairs' tiles split in 4, 3 and 2
    (192, 4096, 1024), (130, 300, 2048), (128, 4096, 4096), (200, 2000, 12032), (180, 4090, 14336), (260, 3000, 14336),
    (300, 4096, 14336),
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens,rows,cols", SHAPES)
def test_matmul_parity(fmt, tokens, rows, cols):
    x, w = case(tokens, rows, cols, fmt, tokens + 7 * rows + cols)
    dt = (torch.float32, torch.bfloat16, torch.float16)[(tokens + rows) % 3]
    y = binding.dq_matmul(ref.to(x, "cuda"), ref.to(w, "cuda"), fmt, out_dtype=dt)
    assert y.shape == (tokens, rows) and y.dtype == dt
    check(y, x, w, fmt, "%s %s" % (fmt, dt))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,rows", [(5, 200), (200, 333), (600, 520)])
def test_matmul_output_types(fmt, dt, tokens, rows):
    x, w = case(tokens, rows, 768, fmt, 5)
    check(binding.dq_matmul(ref.to(x, "cuda"), ref.to(w, "cuda"), fmt, out_dtype=dt), x, w, fmt)


@pytest.mark.parametrize("tokens,rows,cols", [(1, 1, 16), (3, 200, 48), (70, 65, 1040), (1, 64, 16 * 63)])
def test_matmul_nvfp4_columns_of_half_alignment(tokens, rows, cols):
    """cols an odd multiple of 16: code rows that are not 16-byte aligned."""
    x, w = case(tokens, rows, cols, "nvfp4", cols)
    check(binding.dq_matmul(ref.to(x, "cuda"), ref.to(w, "cuda"), "nvfp4", out_dtype=torch.float32), x, w, "nvfp4")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("which", ["codes", "block_scales"])
def test_matmul_operands_at_odd_addresses(fmt, which):
    x, w = case(19, 150, 512, fmt, 9)
    xd, wd = ref.to(x, "cuda"), ref.to(w, "cuda")

    def shifted(t, by):
        buf = torch.empty(t.numel() + 64, dtype=torch.uint8, device="cuda")
        v = buf[by:by + t.numel()].view(t.shape)
        v.copy_(t)
        return v

    for by in (1, 2, 4, 8):
        a = dict(xd, **{which: shifted(xd[which], by)})
        b = dict(wd, **{which: shifted(wd[which], by)})
        check(binding.dq_matmul(a, b, fmt, out_dtype=torch.float32), x, w, fmt, "%s + %d" % (which, by))


@pytest.mark.parametrize("fmt", FMTS)
def test_matmul_single_products(fmt):
    """One nonzero element per operand row at every position of a group run: each code pair lands where it should."""
    cols = 512
    g = ref.GROUP[fmt]
    x, w = case(130, 140, cols, fmt, 21)
    one = 0x38 if fmt == "mxfp8" else 2
    xc = torch.zeros(130, cols, dtype=torch.uint8)
    wc = torch.zeros(140, cols, dtype=torch.uint8)
    xc[torch.arange(130), torch.arange(130) * 3 % cols] = one
    wc[torch.arange(140), torch.arange(140) * 3 % cols] = one
    wc[5] = one

    def pack(c):
        return c if fmt == "mxfp8" else c[:, 0::2] | (c[:, 1::2] << 4)

    x["codes"], w["codes"] = pack(xc).contiguous(), pack(wc).contiguous()
    y = binding.dq_matmul(ref.to(x, "cuda"), ref.to(w, "cuda"), fmt, out_dtype=torch.float32)
    want, _ = ref.matmul(x, w, fmt)
    # one product each, exact in fp32; the tensor scales' product and its multiplication round once each
    tol = (2 * 2.0 ** -24 + 2.0 ** -48) * np.abs(want) if fmt == "nvfp4" else 0.0
    assert (np.abs(ref.f64(y) - want) <= tol).all(), g


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens", [3, 150, 400])
def test_matmul_nan_scales_stay_in_their_rows(fmt, tokens):
    x, w = case(tokens, 200, 640, fmt, 31)
    x["block_scales"][1, 3] = 0x7F if fmt == "nvfp4" else 0xFF
    w["block_scales"][77, 0] = 0x7F if fmt == "nvfp4" else 0xFF
    y = binding.dq_matmul(ref.to(x, "cuda"), ref.to(w, "cuda"), fmt, out_dtype=torch.float32)
    bad = torch.isnan(y).cpu()
    assert bad[1].all() and bad[:, 77].all()
    keep = torch.ones_like(bad)
    keep[1] = False
    keep[:, 77] = False
    assert not bad[keep].any()


def test_matmul_tensor_scales_beyond_fp32_products():
    """Tensor scales whose product leaves fp32's range where the outputs do not."""
    x, w = case(4, 64, 256, "nvfp4", 41)
    x["tensor_scale"][0], w["tensor_scale"][0] = 2.0 ** -100, 2.0 ** -40
    check(binding.dq_matmul(ref.to(x, "cuda"), ref.to(w, "cuda"), "nvfp4", out_dtype=torch.float32), x, w, "nvfp4")
    x["tensor_scale"][0], w["tensor_scale"][0] = 2.0 ** 90, 2.0 ** -100
    check(binding.dq_matmul(ref.to(x, "cuda"), ref.to(w, "cuda"), "nvfp4", out_dtype=torch.float32), x, w, "nvfp4")


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_matmul_extreme_block_scales(fmt):
    """E8M0 bytes from 0 (2^-127) to 254 whose products stay in range."""
    x, w = case(6, 70, 256, fmt, 51)
    for lo, hi in ((0, 254), (254, 0), (1, 253), (60, 190)):
        x["block_scales"].fill_(lo)
        w["block_scales"].fill_(hi)
        check(binding.dq_matmul(ref.to(x, "cuda"), ref.to(w, "cuda"), fmt, out_dtype=torch.float32), x, w, fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_matmul_writes_its_output_only(fmt):
    for tokens, rows in ((1, 33), (5, 127), (129, 65), (300, 300)):
        x, w = case(tokens, rows, 256, fmt, 61)
        buf = torch.full((tokens * rows + 512,), -7.0, dtype=torch.bfloat16, device="cuda")
        out = buf[256:256 + tokens * rows].view(tokens, rows)
        binding.dq_matmul(ref.to(x, "cuda"), ref.to(w, "cuda"), fmt, out=out)
        assert (buf[:256] == -7).all() and (buf[256 + tokens * rows:] == -7).all()
        check(out, x, w, fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_matmul_repeats_bit_for_bit(fmt):
    for tokens, rows, cols in ((1, 512, 4096), (40, 256, 8192), (513, 300, 1024)):
        x, w = case(tokens, rows, cols, fmt, 71)
        xd, wd = ref.to(x, "cuda"), ref.to(w, "cuda")
        a = binding.dq_matmul(xd, wd, fmt, out_dtype=torch.float32)
        for _ in range(3):
            assert torch.equal(a, binding.dq_matmul(xd, wd, fmt, out_dtype=torch.float32))


def test_matmul_of_the_solvers_outputs():
    """dq_solve weights and dq_act_quant activations: X W^T up to the two quantizations' own errors, and the
    product of exactly what they stored."""
    wl = synth.WORKLOADS["nvfp4_g16_gateup_14336x4096"]
    W = synth.make_weight(wl, 256, 1024, seed=3).cuda()
    q = binding.dq_solve(W, "nvfp4", 16, 4)
    X = synth.make_activations(50, 1024, seed=4).cuda()
    a = binding.dq_act_quant(X, q["col_scales"], "nvfp4")
    y = binding.dq_matmul(a, q, "nvfp4")
    check(y, a, q, "nvfp4")
    full = X.double() @ W.double().t()
    assert (y.double() - full).norm() / full.norm() < 0.25


@pytest.mark.parametrize("fmt,wl", [("mxfp4", "mxfp4_g32_downproj_4096x14336"), ("mxfp8", "mxfp8_g32_downproj_4096x14336"),
                                    ("nvfp4", "nvfp4_g16_gateup_14336x4096")])
def test_mlp_block_of_solved_weights(fmt, wl):
    """norm, gate/up product, glu, down product on dq_solve's weights and column scales: each step against the fp64
    definition on what the one before stored."""
    tokens, cols, inter = 40, 512, 768
    wl = synth.WORKLOADS[wl]
    w1, w2 = synth.make_weight(wl, 2 * inter, cols, seed=1).cuda(), synth.make_weight(wl, cols, inter, seed=2).cuda()
    q1, q2 = (binding.dq_solve(w, fmt, wl.group, 4, wl.col_dtype) for w in (w1, w2))
    x = synth.make_activations(tokens, cols, seed=3).cuda()
    r = synth.make_activations(tokens, cols, seed=4).cuda()
    g = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    n = binding.dq_norm_quant(x, g, q1["col_scales"], fmt, residual=r)
    h, x64 = ref.norm(x, r, g, q1["col_scales"], 1e-5)
    assert torch.equal(n["residual"].cpu(), h)
    same_codes(n, ref.quantize(x64, fmt), fmt)
    gu = binding.dq_matmul(n, q1, fmt)
    check(gu, n, q1, fmt, "gate and up")
    a = binding.dq_glu_quant(gu, q2["col_scales"], fmt)
    same_codes(a, ref.quantize(ref.glu(gu[:, :inter], gu[:, inter:], q2["col_scales"]), fmt), fmt)
    y = binding.dq_matmul(a, q2, fmt, out_dtype=torch.float32)
    check(y, a, q2, fmt, "down")


def same_codes(got: dict, want: dict, fmt: str):
    for k in ("codes", "block_scales"):
        assert np.array_equal(got[k].cpu().numpy(), want[k]), k
    assert fmt != "nvfp4" or np.float32(got["tensor_scale"].cpu()[0]) == want["tensor_scale"]


def test_matmul_captured_and_replayed():
    x, w = case(3, 300, 1024, "nvfp4", 81)
    xd, wd = ref.to(x, "cuda"), ref.to(w, "cuda")
    out = torch.zeros(3, 300, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    binding.dq_matmul(xd, wd, "nvfp4", out=out, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.dq_matmul(xd, wd, "nvfp4", out=out, workspace=ws, check=False)
    x2 = ref.random_quantized(3, 1024, "nvfp4", 99)
    for k in xd:
        xd[k].copy_(x2[k])
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    check(out, x2, w, "nvfp4")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens,rows,cols", [(300, 1024, 4096), (2300, 2500, 4096), (40, 512, 2048)])
def test_matmul_of_many_tokens_captured_and_replayed(fmt, tokens, rows, cols):
    """Clusters, and whole waves followed by a launch over the rest, in a graph of two calls in a row."""
    x, w = case(tokens, rows, cols, fmt, 83)
    xd, wd = ref.to(x, "cuda"), ref.to(w, "cuda")
    outs = [torch.empty(tokens, rows, dtype=torch.float32, device="cuda") for _ in range(2)]
    binding.dq_matmul(xd, wd, fmt, out=outs[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for o in outs:
            binding.dq_matmul(xd, wd, fmt, out=o, check=False)
    x2 = ref.random_quantized(tokens, cols, fmt, 84)
    for k in xd:
        xd[k].copy_(x2[k])
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])
    check(outs[1], x2, w, fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_matmul_without_workspace_and_with_one(fmt):
    x, w = case(9, 300, 512, fmt, 85)
    xd, wd = ref.to(x, "cuda"), ref.to(w, "cuda")
    ws = torch.randint(0, 256, (256,), dtype=torch.uint8, device="cuda")  # its contents on entry do not matter
    a = binding.dq_matmul(xd, wd, fmt, out_dtype=torch.float32, workspace=ws)
    b = binding.dq_matmul(xd, wd, fmt, out_dtype=torch.float32, check=False)
    assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp8"])
def test_matmul_offsets_beyond_32_bits(fmt):
    """Weights of more than 2^32 bytes (MXFP8) or elements (NVFP4), outputs of more than 2^31 bytes: the last rows."""
    cols, rows = 4096, 2 ** 20 + 300
    codes = torch.zeros(rows, cols if fmt == "mxfp8" else cols // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(rows, cols // ref.GROUP[fmt], dtype=torch.uint8, device="cuda")
    x, tail = case(600, 300, cols, fmt, 87)
    codes[-300:] = tail["codes"].cuda()
    scales[-300:] = tail["block_scales"].cuda()
    big = {"codes": codes, "block_scales": scales, "tensor_scale": tail["tensor_scale"].cuda()}
    for tokens in (3, 600):
        part = {"codes": x["codes"][:tokens], "block_scales": x["block_scales"][:tokens], "tensor_scale": x["tensor_scale"]}
        y = binding.dq_matmul(ref.to(part, "cuda"), big, fmt, out_dtype=torch.float32)
        assert not y[:, :-300].any()
        check(y[:, -300:].contiguous(), part, tail, fmt)
        del y


def test_matmul_on_two_streams_at_once():
    cases = [case(2, 512, 2048, "mxfp4", 91), case(300, 512, 2048, "mxfp4", 93)]
    dev = [(ref.to(x, "cuda"), ref.to(w, "cuda")) for x, w in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    ys = [[], []]
    for _ in range(5):
        for i in range(2):
            ys[i].append(binding.dq_matmul(*dev[i], "mxfp4", stream=streams[i], check=False))
    torch.cuda.synchronize()
    for i in range(2):
        for y in ys[i]:
            check(y, *cases[i], "mxfp4")


def test_matmul_from_two_threads():
    """Calls of one kernel that take different amounts of shared memory, launched by two threads at once."""
    cases = [[ref.to(q, "cuda") for q in case(*size, "mxfp8", 51)] for size in ((1, 512, 16384), (1, 128 * 300, 128))]
    want = [binding.dq_matmul(x, w, "mxfp8") for x, w in cases]
    wrong = []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            ys = [binding.dq_matmul(*cases[i], "mxfp8", check=False, stream=stream) for _ in range(400)]
            stream.synchronize()
            wrong.extend(k for k, y in enumerate(ys) if not torch.equal(y, want[i]))
        except Exception as e:  # reported by the test's thread
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong[:3]
