"""dq_norm_quant and dq_glu_quant against their fp64 definitions: codes, block scales, the NVFP4 tensor scale and
the residual sum bit for bit.

The library decides in fp64 wherever fp32 cannot; its fp64 values and the definitions' differ by a few units of
2^-53, so a decision could differ only within about 2^-50 of a border, which these seeded inputs do not reach.
"""
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


def same(got: dict, x64: np.ndarray, fmt: str, label: str = ""):
    want = ref.quantize(x64, fmt)
    if fmt == "nvfp4":
        assert np.float32(got["tensor_scale"].cpu()[0]) == want["tensor_scale"], label
    for k in ("block_scales", "codes"):
        bad = np.argwhere(got[k].cpu().numpy() != want[k])
        assert bad.size == 0, "%s %s differ at %d places, first %s" % (label, k, len(bad), bad[:3].tolist())


def norm_case(tokens, cols, dtype, bdt, seed):
    rng = torch.Generator().manual_seed(seed)
    x = synth.make_activations(tokens, cols, seed=seed).to(dtype)
    r = (3 * torch.randn(tokens, cols, generator=rng)).to(dtype)
    w = (1 + 0.3 * torch.randn(cols, generator=rng)).to(dtype)
    return x, r, w, synth.make_col_scales(cols, seed + 1).to(bdt)


def cuda(t):
    return None if t is None else t.cuda()


def run_norm(x, r, w, b, fmt, eps=1e-5, label="", check=True, **kw):
    got = binding.dq_norm_quant(cuda(x), cuda(w), cuda(b), fmt, residual=cuda(r), eps=eps, check=check, **kw)
    torch.cuda.synchronize()
    h, x64 = ref.norm(x, r, w, b, eps)
    if r is not None:
        hg = got["residual"].cpu()  # a NaN's payload is not defined; everything else bit for bit
        assert torch.equal(torch.isnan(hg), torch.isnan(h)), label
        assert torch.equal(hg.nan_to_num(0.0).view(torch.int16), h.nan_to_num(0.0).view(torch.int16)), label
    same(got, x64, fmt, label)
    return got


SHAPES = [(1, 32), (1, 64), (3, 96), (2, 4096), (5, 1056), (37, 4096), (2, 4128), (3, 8192), (2, 14336), (2, 16384),
          (2, 16416), (1, 40000), (700, 256), (1500, 64)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens,cols", SHAPES)
def test_norm_parity(fmt, tokens, cols):
    dt = (torch.bfloat16, torch.float16)[(tokens + cols // 32) % 2]
    bdt = (torch.bfloat16, torch.float16)[tokens % 2]
    x, r, w, b = norm_case(tokens, cols, dt, bdt, tokens * 3 + cols)
    run_norm(x, r, w, b, fmt, label="with residual")
    run_norm(x, None, w, b, fmt, label="without residual")


@pytest.mark.parametrize("fmt", FMTS)
def test_norm_without_weight_or_column_scales(fmt):
    x, r, w, b = norm_case(9, 512, torch.bfloat16, torch.bfloat16, 7)
    run_norm(x, r, None, b, fmt)
    run_norm(x, r, w, None, fmt)
    run_norm(x, None, None, None, fmt, eps=0.0)


@pytest.mark.parametrize("fmt,tokens", [("mxfp8", 8192), ("nvfp4", 2048), ("mxfp4", 1000)])
def test_norm_full_size(fmt, tokens):
    x, r, w, b = norm_case(tokens, 4096, torch.bfloat16, torch.bfloat16, 17)
    run_norm(x, r, w, b, fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_norm_ties_and_zeros(fmt):
    """Rows of powers of two (1/rms exact, values on rounding borders), zero rows and zero groups."""
    cols = 256
    x = torch.zeros(6, cols)
    x[0] = 1.0
    x[1] = 2.0
    x[2, :128] = torch.tensor([2.0 ** 0.5]).to(torch.bfloat16).float()
    x[3, ::2] = 4.0
    x[5] = torch.linspace(-1, 1, cols)
    w = (torch.arange(cols) % 64 / 16.0 + 0.0625)
    for dt in (torch.bfloat16, torch.float16):
        run_norm(x.to(dt), None, w.to(dt), None, fmt, eps=1e-6)
        run_norm(x[:2].to(dt), None, w.to(dt), None, fmt, eps=0.0)
        run_norm(torch.zeros(3, cols).to(dt), None, w.to(dt), None, fmt, eps=1e-6)


@pytest.mark.parametrize("fmt", FMTS)
def test_norm_far_magnitudes(fmt):
    """Rows near the ends of bf16's range, tiny eps, and g b outside fp32's range."""
    cols = 128
    base = synth.make_activations(8, cols, seed=3).float()
    x = torch.stack([base[i] * s for i, s in enumerate((1e30, 1e36, 1e-30, 1e-37, 1.0, 1e-20, 1e20, 1e-3))])
    w = torch.ones(cols)
    w[::3] = 1e-25
    b = torch.ones(cols)
    b[::5] = 1e-25
    run_norm(x.to(torch.bfloat16), None, w.to(torch.bfloat16), b.to(torch.bfloat16), fmt, eps=0.0)
    run_norm(x.to(torch.bfloat16), None, (w * 1e-30).to(torch.bfloat16), b.to(torch.bfloat16), fmt, eps=1e-30)
    run_norm(x.to(torch.bfloat16), None, (w * 1e20).to(torch.bfloat16), (b * 1e15).to(torch.bfloat16), fmt, eps=0.0)
    tiny = (base * 1e-39).to(torch.bfloat16)  # subnormal inputs: 1/rms beyond fp32
    run_norm(tiny, None, w.to(torch.bfloat16), None, fmt, eps=0.0, check=False)


@pytest.mark.parametrize("fmt", FMTS)
def test_norm_non_finite_rows_stay_alone(fmt):
    x, r, w, b = norm_case(6, 512, torch.float16, torch.bfloat16, 23)
    x[1, 5] = float("inf")
    x[3, 500] = float("nan")
    r[4, 17] = 60000.0
    x[4, 17] = 60000.0  # the sum overflows fp16
    got = run_norm(x, r, w, b, fmt, check=False)
    nan = 0x7F if fmt == "nvfp4" else 0xFF
    s = got["block_scales"].cpu()
    assert (s[[1, 3, 4]] == nan).all() and (s[[0, 2, 5]] != nan).all()
    with pytest.raises(binding.DQError) as e:
        binding.dq_norm_quant(x.cuda(), w.cuda(), b.cuda(), fmt, residual=r.cuda())
    assert e.value.status == 4


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("where", ["x", "residual"])
def test_norm_in_place_residual(fmt, where):
    x, r, w, b = norm_case(11, 1024, torch.bfloat16, torch.bfloat16, 29)
    xd, rd = x.cuda(), r.cuda()
    dst = xd if where == "x" else rd
    got = binding.dq_norm_quant(xd, w.cuda(), b.cuda(), fmt, residual=rd, residual_out=dst)
    h, x64 = ref.norm(x, r, w, b, 1e-5)
    assert torch.equal(dst.cpu(), h)
    same(got, x64, fmt)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_rows_offsets_beyond_32_bits(fmt):
    """More than 2^31 elements: the last rows are what they are alone."""
    cols, rows = 4096, 2 ** 19 + 40
    x, r, w, b = norm_case(40, cols, torch.bfloat16, torch.bfloat16, 43)
    big = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    big[-40:] = x.cuda()
    got = binding.dq_norm_quant(big, w.cuda(), b.cuda(), fmt)
    alone = binding.dq_norm_quant(x.cuda(), w.cuda(), b.cuda(), fmt)
    for k in ("codes", "block_scales"):
        assert torch.equal(got[k][-40:], alone[k]), k
    assert not got["codes"][:-40].any() and (got["block_scales"][:-40] == 127).all()
    got = binding.dq_glu_quant((big, big), b.cuda(), fmt)
    alone = binding.dq_glu_quant((x.cuda(), x.cuda()), b.cuda(), fmt)
    for k in ("codes", "block_scales"):
        assert torch.equal(got[k][-40:], alone[k]), k


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens", [1, 2, 5, 8, 9, 40])
def test_rows_workspace_contents_do_not_matter(fmt, tokens):
    """One CTA, one cluster and a whole grid, each on a workspace full of anything, twice."""
    x, r, w, b = norm_case(tokens, 512, torch.bfloat16, torch.bfloat16, 47)
    gx, gb = glu_case(tokens, 1024, torch.bfloat16, 48)
    ws = torch.randint(0, 256, (256 + 8 * tokens,), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        run_norm(x, r, w, b, fmt, workspace=ws)
        ws.random_(0, 256)
        same(binding.dq_glu_quant(gx.cuda(), gb.cuda(), fmt, workspace=ws), ref.glu(gx[:, :1024], gx[:, 1024:], gb), fmt)


def glu_case(tokens, cols, dtype, seed):
    rng = torch.Generator().manual_seed(seed)
    x = (3 * torch.randn(tokens, 2 * cols, generator=rng)).to(dtype)
    return x, synth.make_col_scales(cols, seed)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens,cols", [(1, 32), (1, 14336), (3, 96), (5, 288), (16, 1056), (130, 512), (1000, 160)])
def test_glu_parity(fmt, tokens, cols):
    dt = (torch.bfloat16, torch.float16)[tokens % 2]
    x, b = glu_case(tokens, cols, dt, tokens + cols)
    same(binding.dq_glu_quant(x.cuda(), b.cuda(), fmt), ref.glu(x[:, :cols], x[:, cols:], b), fmt)
    same(binding.dq_glu_quant(x.cuda(), None, fmt), ref.glu(x[:, :cols], x[:, cols:], None), fmt)


@pytest.mark.parametrize("fmt,tokens", [("mxfp8", 1024), ("nvfp4", 512), ("mxfp4", 512)])
def test_glu_full_size(fmt, tokens):
    x, b = glu_case(tokens, 14336, torch.bfloat16, 3)
    same(binding.dq_glu_quant(x.cuda(), b.cuda(), fmt), ref.glu(x[:, :14336], x[:, 14336:], b), fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_glu_strided_pair(fmt):
    x, b = glu_case(33, 256, torch.bfloat16, 5)
    wide = torch.zeros(33, 1024, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:264] = x[:, :256].cuda()
    wide[:, 512:768] = x[:, 256:].cuda()
    got = binding.dq_glu_quant((wide[:, 8:264], wide[:, 512:768]), b.cuda(), fmt)
    same(got, ref.glu(x[:, :256], x[:, 256:], b), fmt)
    two = binding.dq_glu_quant((x[:, :256].contiguous().cuda(), x[:, 256:].contiguous().cuda()), b.cuda(), fmt)
    assert torch.equal(two["codes"], got["codes"]) and torch.equal(two["block_scales"], got["block_scales"])


@pytest.mark.parametrize("fmt", FMTS)
def test_glu_far_values(fmt):
    """Gates whose exponential leaves fp32, huge and tiny products, non-finite values."""
    cols = 64
    g = torch.tensor([-1e3, -200.0, -100.0, -90.0, -88.0, -80.5, -79.0, -1.0, 0.0, 1e-30, 1.0, 90.0, 200.0, 1e10, 1e25, 0.5])
    gate = g.repeat(8, cols // 16)
    up = torch.ones(8, cols)
    for i, s in enumerate((1.0, 1e30, 1e-30, 1e-38, 3e38, 1e12, -2.0, 0.0)):
        up[i] *= s
    b = torch.ones(cols)
    for bs in (1.0, 1e-20, 1e20):
        args = [t.to(torch.bfloat16) for t in (gate, up, b * bs)]
        x64 = ref.glu(*args)
        got = binding.dq_glu_quant((args[0].cuda(), args[1].cuda()), args[2].cuda(), fmt, check=False)
        torch.cuda.synchronize()
        same(got, x64, fmt, "b %g" % bs)
    gate = torch.randn(4, cols, generator=torch.Generator().manual_seed(1)).to(torch.float16)
    up = torch.ones(4, cols, dtype=torch.float16)
    gate[1, 3] = float("nan")
    gate[2, 40] = float("-inf")
    up[3, 0] = float("inf")
    got = binding.dq_glu_quant((gate.cuda(), up.cuda()), None, fmt, check=False)
    torch.cuda.synchronize()
    same(got, ref.glu(gate, up, None), fmt, "non-finite")
    with pytest.raises(binding.DQError) as e:
        binding.dq_glu_quant((gate.cuda(), up.cuda()), None, fmt)
    assert e.value.status == 4


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_write_their_outputs_only(fmt):
    tokens, cols = 5, 96
    x, r, w, b = norm_case(tokens, cols, torch.bfloat16, torch.bfloat16, 31)
    gx, gb = glu_case(tokens, cols, torch.bfloat16, 31)
    nc, ns = tokens * cols // (1 if fmt == "mxfp8" else 2), tokens * (cols // ref.GROUP[fmt])

    def bufs():
        c = torch.full((nc + 64,), 0xA5, dtype=torch.uint8, device="cuda")
        s = torch.full((ns + 64,), 0xA5, dtype=torch.uint8, device="cuda")
        out = {"codes": c[32:32 + nc].view(tokens, -1), "block_scales": s[32:32 + ns].view(tokens, -1),
               "tensor_scale": torch.zeros(1, device="cuda")}
        return c, s, out

    for f in (lambda o: binding.dq_norm_quant(x.cuda(), w.cuda(), b.cuda(), fmt, residual=r.cuda(), out=o),
              lambda o: binding.dq_glu_quant(gx.cuda(), gb.cuda(), fmt, out=o)):
        c, s, out = bufs()
        f(out)
        for t, n in ((c, nc), (s, ns)):
            assert (t[:32] == 0xA5).all() and (t[32 + n:] == 0xA5).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_captured_and_replayed(fmt):
    """One graph of the norm, both products and the glu, replayed on new inputs."""
    tokens, cols, inter = 6, 256, 384
    w1 = ref.to(ref.random_quantized(2 * inter, cols, fmt, 1, spread=0.3), "cuda")
    w2 = ref.to(ref.random_quantized(cols, inter, fmt, 2, spread=0.3), "cuda")
    x, r, w, b = (t.cuda() for t in norm_case(tokens, cols, torch.bfloat16, torch.bfloat16, 37))
    b2 = synth.make_col_scales(inter, 5).cuda()

    def block():
        q = binding.dq_norm_quant(x, w, b, fmt, residual=r, check=False)
        gu = binding.dq_matmul(q, w1, fmt, check=False)
        a = binding.dq_glu_quant(gu, b2, fmt, check=False)
        return q, gu, a, binding.dq_matmul(a, w2, fmt, check=False)

    block()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = block()
    x2, r2, _, _ = norm_case(tokens, cols, torch.bfloat16, torch.bfloat16, 41)
    x.copy_(x2)
    r.copy_(r2)
    g.replay()
    torch.cuda.synchronize()
    eager = block()
    torch.cuda.synchronize()
    assert torch.equal(held[3].view(torch.int16), eager[3].view(torch.int16))
    h, x64 = ref.norm(x2, r2, w, b, 1e-5)
    same(held[0], x64, fmt)
    want, mags = ref.matmul(held[0], w1, fmt)
    tol = (cols + 4) * 2.0 ** -24 * mags
    assert (np.abs(ref.f64(held[1]) - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol)).all()
    same(held[2], ref.glu(held[1][:, :inter], held[1][:, inter:], b2), fmt)
