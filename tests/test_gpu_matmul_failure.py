"""dq_matmul's bounded waits on the GPU without a fault: dq_matmul_selftest lets one role of a CTA stop, the waits on
it run out after 2 ms, and the kernel ends with a status, with NaN where a sum was not finished and dq_matmul's own
bits everywhere else, and leaves the device usable."""
from __future__ import annotations

import pytest
import torch

import linear_ref as ref
from calibration_free_weight_dualquant_b200 import binding

pytestmark = pytest.mark.gpu

DQ_ECUDA = 5
NEVER = 2 ** 26 - 1


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    binding.load_library()


# tokens, rows, cols: one tile, tiles split over a cluster, three CTAs an SM, 64 and 128 tokens a tile, pairs of CTAs
# with several tiles each, split tiles of pairs alone and behind whole waves
SHAPES = [(1, 100, 512), (5, 512, 4096), (30, 300, 2048), (9, 60000, 256), (192, 4096, 1024), (128, 4096, 4096),
          (2304, 5000, 512), (512, 2048, 8192), (2300, 2500, 4096)]


def operands(tokens, rows, cols, fmt):
    x = ref.random_quantized(tokens, cols, fmt, tokens)
    w = ref.random_quantized(rows, cols, fmt, rows)
    return ref.to(x, "cuda"), ref.to(w, "cuda")


def bits(t):
    return t.view(torch.int32 if t.dtype == torch.float32 else torch.int16)


def run(x, w, fmt, want, rank, role, at):
    """Status and the mask of NaN outputs; all others are dq_matmul's, and nothing else is written."""
    tokens, rows = want.shape
    buf = torch.full((tokens * rows + 512,), -7.0, dtype=want.dtype, device="cuda")
    out = buf[256:256 + tokens * rows].view(tokens, rows)
    ws = torch.randint(0, 256, (256,), dtype=torch.uint8, device="cuda")
    status = binding.matmul_selftest(x, w, fmt, out, ws, rank, role, at)
    nan = torch.isnan(out)
    assert torch.equal(bits(out)[~nan], bits(want)[~nan])
    assert (buf[:256] == -7).all() and (buf[256 + tokens * rows:] == -7).all()
    return status, nan


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "mxfp8"])
@pytest.mark.parametrize("tokens,rows,cols", SHAPES)
def test_a_role_that_stops_ends_in_a_status_and_nan(fmt, tokens, rows, cols):
    x, w = operands(tokens, rows, cols, fmt)
    dt = torch.float32 if (tokens + rows) % 3 == 0 else torch.bfloat16
    want = binding.dq_matmul(x, w, fmt, out_dtype=dt)
    assert not torch.isnan(want).any()
    for rank in (0, 1):
        for role in (0, 1, 2):
            for at in (0, 1, 6):
                status, nan = run(x, w, fmt, want, rank, role, at)
                assert status in (0, DQ_ECUDA)
                assert bool(nan.any()) == (status == DQ_ECUDA), (rank, role, at)
                if rank == 0 and at == 0:  # every cluster has such a CTA, and it has work
                    assert nan.all(), (role, nan.float().mean().item())
    status, nan = run(x, w, fmt, want, 0, 0, NEVER)
    assert status == 0 and not nan.any()
    assert torch.equal(bits(want), bits(binding.dq_matmul(x, w, fmt, out_dtype=dt)))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp8"])
def test_split_pairs_give_whole_tiles_up(fmt):
    """One CTA of a cluster of several stops late: nothing that the others summed shows."""
    x, w = operands(256, 512, 16384, fmt)
    want = binding.dq_matmul(x, w, fmt, out_dtype=torch.float32)
    ranks = 0
    for rank in range(8):
        for at in (3, 9):
            status, nan = run(x, w, fmt, want, rank, 0, at)
            assert nan.all() if status == DQ_ECUDA else not nan.any()
            ranks += status == DQ_ECUDA
    assert ranks > 2
    assert torch.equal(want, binding.dq_matmul(x, w, fmt, out_dtype=torch.float32))


def test_selftest_arguments():
    x, w = operands(1, 64, 512, "mxfp8")
    out = torch.empty(1, 64, device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    for kw in (dict(rank=-1), dict(rank=8), dict(role=3), dict(at=2 ** 26), dict(wait_ns=1000), dict(wait_ns=2 * 10 ** 9)):
        with pytest.raises(binding.DQError) as e:
            binding.matmul_selftest(x, w, "mxfp8", out, ws, **{**dict(rank=0, role=0, at=0), **kw})
        assert e.value.status == 1
