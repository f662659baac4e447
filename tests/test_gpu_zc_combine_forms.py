"""Combine and its gradients against 64 bits in every form that the gradient's
rule chooses: 16, 64 or 256 threads for a token's rows, all of them or one by
one, in one pass over the columns and in several (which case takes which form:
tests/test_step_forms_cpu.py)."""
import pytest

from tests import test_gpu_x_step as x

pytestmark = pytest.mark.gpu

# tokens, experts, topk, columns, rows a group is padded to, share of slots without a row, types of rows and sum
CASES = [
    (900, 20, 5, 136, 16, 0.3, "fp16", "bf16"),
    (8200, 24, 9, 136, 16, 0.2, "bf16", "bf16"),
    (8193, 6, 2, 256, 128, 0.0, "fp32", "fp32"),
    (8200, 9, 3, 264, 16, 0.4, "bf16", "fp32"),
    (700, 5, 4, 2048, 16, 0.1, "fp32", "bf16"),
    (4100, 16, 5, 776, 16, 0.3, "fp16", "fp16"),
    (4096, 7, 2, 2048, 1, 0.5, "bf16", "bf16"),
    (200, 12, 8, 4104, 16, 0.2, "bf16", "bf16"),
    (1023, 4, 1, 2056, 16, 0.0, "fp32", "fp16"),
    (128, 70, 64, 2056, 16, 0.5, "bf16", "bf16"),
    (128, 9, 3, 8712, 16, 0.3, "fp16", "fp32"),
    (1030, 20, 8, 2568, 16, 0.3, "bf16", "bf16"),
    (1024, 5, 3, 8712, 128, 0.1, "fp16", "fp16"),
    (1100, 70, 64, 2064, 1, 0.9, "fp32", "fp32"),
]


@pytest.mark.parametrize("T,E,topk,H,block,lost,dtype,out_dtype", CASES)
@pytest.mark.parametrize("weighted", [True, False])
def test_combine_in_every_form(T, E, topk, H, block, lost, dtype, out_dtype, weighted):
    x.test_combine(T, E, topk, H, block, lost, dtype, out_dtype, weighted)
