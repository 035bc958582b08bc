"""Errors of the linear layer's calls that torch raises: they are torch's own exceptions, as for the library's other
calls."""
from __future__ import annotations

import pytest
import torch

from calibration_free_weight_dualquant_b200 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    binding.load_library()


def test_an_allocation_that_fails_is_an_out_of_memory_error():
    """An output of 2^42 bytes over operands of 34 MB each."""
    def q(rows):
        return {"codes": torch.zeros(rows, 32, dtype=torch.uint8, device="cuda"),
                "block_scales": torch.full((rows, 1), 127, dtype=torch.uint8, device="cuda")}

    big = q(2 ** 20)
    with pytest.raises(torch.OutOfMemoryError):
        binding.dq_matmul(big, big, "mxfp8", out_dtype=torch.float32)
    y = binding.dq_matmul(q(3), big, "mxfp8", out_dtype=torch.float32)
    assert y.shape == (3, 2 ** 20) and not y.any()


def test_a_device_that_is_missing_or_other_is_an_error_of_the_call():
    x = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(binding.DQError) as e:
        binding.dq_norm_quant(x, torch.ones(64, dtype=torch.bfloat16), None, "mxfp8")  # a weight on the CPU
    assert e.value.status == 1
    with pytest.raises(KeyError):
        binding.dq_matmul({"codes": torch.zeros(1, 32, dtype=torch.uint8, device="cuda")},
                          {"codes": torch.zeros(1, 32, dtype=torch.uint8, device="cuda")}, "mxfp8")
