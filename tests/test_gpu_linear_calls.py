"""Calls of the quantized linear layer that its documentation allows: several at once on streams and threads, a whole
block of many tokens captured and replayed, buffers at every alignment that is accepted, and very long rows."""
from __future__ import annotations

import threading

import numpy as np
import pytest
import torch

import linear_ref as ref
from calibration_free_weight_dualquant_b200 import binding, synth

pytestmark = pytest.mark.gpu

FMTS = ["nvfp4", "mxfp4", "mxfp8"]
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    binding.load_library()


def inputs(tokens, cols, seed, dtype=BF16):
    rng = torch.Generator().manual_seed(seed)
    x = synth.make_activations(tokens, cols, seed=seed).to(dtype)
    r = (3 * torch.randn(tokens, cols, generator=rng)).to(dtype)
    w = (1 + 0.3 * torch.randn(cols, generator=rng)).to(dtype)
    return x, r, w, synth.make_col_scales(cols, seed + 1).to(BF16)


def same(got: dict, x64: np.ndarray, fmt: str):
    want = ref.quantize(x64, fmt)
    if fmt == "nvfp4":
        assert np.float32(got["tensor_scale"].cpu()[0]) == want["tensor_scale"]
    for k in ("block_scales", "codes"):
        bad = got[k].cpu().numpy() != want[k]
        assert not bad.any(), "%s: %d of %d differ" % (k, bad.sum(), bad.size)


def equal(a: dict, b: dict) -> bool:
    return all(torch.equal(a[k], b[k]) for k in ("codes", "block_scales", "tensor_scale") if k in a)


class Block:
    """norm, gate and up product, glu, down product on weights of its own."""

    def __init__(self, fmt, tokens, cols, inter, seed):
        self.fmt = fmt
        self.w1 = ref.to(ref.random_quantized(2 * inter, cols, fmt, seed, spread=0.3), "cuda")
        self.w2 = ref.to(ref.random_quantized(cols, inter, fmt, seed + 1, spread=0.3), "cuda")
        self.x, self.r, self.w, self.b = (t.cuda() for t in inputs(tokens, cols, seed))
        self.b2 = synth.make_col_scales(inter, seed).to(BF16).cuda()

    def __call__(self, stream=None):
        kw = dict(check=False, stream=stream)
        q = binding.dq_norm_quant(self.x, self.w, self.b, self.fmt, residual=self.r, **kw)
        a = binding.dq_glu_quant(binding.dq_matmul(q, self.w1, self.fmt, **kw), self.b2, self.fmt, **kw)
        return q, a, binding.dq_matmul(a, self.w2, self.fmt, **kw)


def same_block(a, b):
    return equal(a[0], b[0]) and torch.equal(a[0]["residual"], b[0]["residual"]) and equal(a[1], b[1]) and torch.equal(
        a[2].view(torch.int16), b[2].view(torch.int16))


@pytest.mark.parametrize("fmt", FMTS)
def test_blocks_on_three_streams_at_once(fmt):
    blocks = [Block(fmt, t, 512, 768, 7 * t) for t in (1, 40, 1100)]
    want = [b() for b in blocks]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    got = [[] for _ in blocks]
    for _ in range(8):
        for i, b in enumerate(blocks):
            got[i].append(b(streams[i]))
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        for g in runs:
            assert same_block(g, w)


@pytest.mark.parametrize("fmt", FMTS)
def test_blocks_from_two_threads(fmt):
    blocks = [Block(fmt, t, 1024, 512, 11 * t) for t in (3, 700)]
    want = [b() for b in blocks]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            runs = [blocks[i](stream) for _ in range(40)]
            stream.synchronize()
            wrong.extend(k for k, g in enumerate(runs) if not same_block(g, want[i]))
        except Exception as e:  # reported by the test's thread
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong[:3]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens", [12, 333, 2300])
def test_a_block_of_many_tokens_captured_and_replayed(fmt, tokens):
    """Cooperative launches, memsets, clusters and pairs in one graph, replayed three times on other inputs."""
    block = Block(fmt, tokens, 1024, 1280, tokens)
    block()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = block()
    x, r, _, _ = inputs(tokens, 1024, tokens + 5)
    block.x.copy_(x)
    block.r.copy_(r)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert same_block(held, block())
    same(held[0], ref.norm(x, r, block.w, block.b, 1e-5)[1], fmt)


def placed(t: torch.Tensor, by: int) -> torch.Tensor:
    """A copy of t on the device, `by` bytes off a multiple of 256."""
    buf = torch.zeros(t.numel() * t.element_size() + 256, dtype=torch.uint8, device="cuda")
    v = buf[by:by + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
    v.copy_(t)
    return v


def outputs(tokens, cols, fmt, codes_by, scales_by):
    n = cols // (1 if fmt == "mxfp8" else 2)
    return {"codes": placed(torch.zeros(tokens, n, dtype=torch.uint8), codes_by),
            "block_scales": placed(torch.zeros(tokens, cols // ref.GROUP[fmt], dtype=torch.uint8), scales_by),
            "tensor_scale": placed(torch.zeros(1), 4)}


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens,cols", [(3, 1056), (700, 96), (2, 9216), (2, 40000)])
def test_rows_at_every_alignment(fmt, tokens, cols):
    """Inputs at 16 bytes, column scales at 2, codes at 8, block scales at 1, in every kind of kernel."""
    for dtype in (BF16, torch.float16):
        x, r, w, b = inputs(tokens, cols, 3 * cols, dtype)
        h, x64 = ref.norm(x, r, w, b, 1e-5)
        for xo, ro, ho, wo, bo, co, so in ((16, 0, 0, 16, 2, 8, 1), (0, 16, 48, 48, 6, 24, 3), (0, 0, 16, 0, 16, 16, 0)):
            out = outputs(tokens, cols, fmt, co, so)
            got = binding.dq_norm_quant(placed(x, xo), placed(w, wo), placed(b, bo), fmt, residual=placed(r, ro), out=out,
                                        residual_out=placed(torch.zeros_like(x), ho))
            assert torch.equal(got["residual"].cpu(), h)
            same(got, x64, fmt)
            out = outputs(tokens, cols, fmt, co, so)
            binding.dq_glu_quant((placed(x, xo), placed(r, ro)), placed(b, bo), fmt, out=out)
            same(out, ref.glu(x, r, b), fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_very_long_rows(fmt):
    cols = 2 ** 20 + 32
    x, r, w, b = inputs(2, cols, 5)
    same(binding.dq_norm_quant(x.cuda(), w.cuda(), b.cuda(), fmt, residual=r.cuda()), ref.norm(x, r, w, b, 1e-5)[1], fmt)
    same(binding.dq_glu_quant((x.cuda(), r.cuda()), b.cuda(), fmt), ref.glu(x, r, b), fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens,rows", [(1, 3), (200, 130), (600, 700)])
def test_very_long_products(fmt, tokens, rows):
    """2^20 + 32 columns against the fp64 product: test_gpu_matmul's bound."""
    cols = 2 ** 20 + 32 if tokens < 600 else 2 ** 17 + 32
    x, w = ref.random_quantized(tokens, cols, fmt, 1), ref.random_quantized(rows, cols, fmt, 2)
    y = ref.f64(binding.dq_matmul(ref.to(x, "cuda"), ref.to(w, "cuda"), fmt, out_dtype=torch.float32))
    want, sum_abs = ref.matmul(x, w, fmt)
    assert (np.abs(y - want) <= (cols + 4) * 2.0 ** -24 * sum_abs).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_a_batch_that_is_part_of_a_larger_one(fmt):
    """The first rows of a padded batch, and a product into the middle of a larger output: the rest stays."""
    x, r, w, b = inputs(64, 512, 9)
    xd = x.cuda()
    before = xd.clone()
    q = binding.dq_norm_quant(xd[8:29], w.cuda(), b.cuda(), fmt, residual=r.cuda()[8:29], residual_out=xd[8:29])
    h, x64 = ref.norm(x[8:29], r[8:29], w, b, 1e-5)
    same(q, x64, fmt)
    assert torch.equal(xd[8:29].cpu(), h) and torch.equal(xd[:8], before[:8]) and torch.equal(xd[29:], before[29:])
    wq = ref.to(ref.random_quantized(96, 512, fmt, 3), "cuda")
    y = torch.full((64, 96), -7.0, dtype=BF16, device="cuda")
    binding.dq_matmul(q, wq, fmt, out=y[5:26])
    assert torch.equal(y[5:26], binding.dq_matmul(q, wq, fmt)) and (y[:5] == -7).all() and (y[26:] == -7).all()
    one = {k: v[3:4] if v.dim() == 2 else v for k, v in q.items() if k in ("codes", "block_scales", "tensor_scale")}
    xv, wv = ref.decode(one, fmt), ref.decode(wq, fmt)
    s = ref.tensor_scale(q, fmt) * ref.tensor_scale(wq, fmt)
    got = ref.f64(binding.dq_matmul(one, wq, fmt, out_dtype=torch.float32))
    assert (np.abs(got - xv @ wv.T * s) <= 516 * 2.0 ** -24 * (np.abs(xv) @ np.abs(wv).T) * s).all()
