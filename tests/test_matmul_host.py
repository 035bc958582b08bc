"""Refusals of dq_matmul_kernel and dq_matmul_selftest: found on the host, nothing is enqueued (no GPU needed)."""
from __future__ import annotations

import ctypes

import pytest

from calibration_free_weight_dualquant_b200 import binding, build

FAKE = 0x100000  # an aligned address; never dereferenced by a refused call


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def args(tokens=4, rows=8, cols=64, fmt=3, group=32, y=FAKE, dt=1):
    q = binding._Outputs(FAKE, FAKE, FAKE, None, None)
    return ctypes.byref(q), tokens, ctypes.byref(q), rows, cols, fmt, group, y, dt


@pytest.mark.parametrize("kw,status", [(dict(tokens=0), 1), (dict(cols=48), 1), (dict(fmt=1), 2), (dict(group=16), 2),
                                       (dict(y=None), 1), (dict(dt=3), 1), (dict(cols=2 ** 27 + 32), 2)])
def test_both_refuse_what_dq_matmul_refuses(lib, kw, status):
    info = binding._MatmulInfo()
    assert lib.dq_matmul_kernel(*args(**kw), ctypes.byref(info)) == status
    assert lib.dq_matmul_selftest(*args(**kw), FAKE, 256, 2_000_000, 0, 0, 0, None) == status


def test_kernel_needs_a_place_for_its_answer(lib):
    assert lib.dq_matmul_kernel(*args(), None) == 1


@pytest.mark.parametrize("kw,status", [
    (dict(ws=None), 1), (dict(ws=FAKE + 16), 1), (dict(nbytes=255), 3), (dict(wait=999_999), 1), (dict(wait=10 ** 9 + 1), 1),
    (dict(rank=-1), 1), (dict(rank=8), 1), (dict(role=-1), 1), (dict(role=3), 1), (dict(at=2 ** 26), 1),
])
def test_selftest_refusals(lib, kw, status):
    k = {**dict(ws=FAKE, nbytes=256, wait=2_000_000, rank=0, role=0, at=0), **kw}
    assert lib.dq_matmul_selftest(*args(), k["ws"], k["nbytes"], k["wait"], k["rank"], k["role"], k["at"], None) == status
