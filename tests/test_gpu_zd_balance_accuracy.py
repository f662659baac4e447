"""The balance loss's sums where FP32 could lose them: many rows of one sign."""
import pytest
import torch

from tests.gpu_util import log, require_gpu

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def M():
    require_gpu()
    import w4a16_int4_grouped_amd
    return w4a16_int4_grouped_amd


@pytest.mark.parametrize("E,dtype", [(13, "fp32"), (129, "bf16"), (2000, "bf16")])
def test_even_scores_of_the_most_tokens(E, dtype):
    """2^24 rows (2^23 of 2000) of equal logits: every p is 1 / E, so the loss is 1, the sum of the choices' shares."""
    m = M()
    T = 1 << 24 if E < 1000 else 1 << 23
    log(f"case balance of even scores T={T} E={E} {dtype}")
    x = torch.zeros(T, E, dtype=DT[dtype], device="cuda")
    ids = (torch.arange(T, device="cuda") % E).int()[:, None]
    loss, counts = m.router_balance(x, ids)
    del x
    assert torch.equal(counts[0].long(), torch.bincount(ids[:, 0].long(), minlength=E))
    # a step of half of 2^-23 for each addition in FP32, 128 in registers, up to 64 of those sums in LDS and 8 waves',
    # then FP64; 1 / E itself within 15 (of a sum of ones, a reciprocal and a product), the loss rounded once
    assert abs(float(loss) - 1) <= (128 + 64 + 8 + 15 + 1) * 2.0 ** -24
    torch.cuda.empty_cache()
