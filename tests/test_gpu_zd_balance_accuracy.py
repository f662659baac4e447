"""The balance loss where FP32 could lose it: many rows of one sign, logits far
from each other."""
import pytest
import torch

from tests import step_util as U
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
    log(f"  off by {abs(float(loss) - 1) * 2 ** 24:.1f} steps of 2^-24")
    assert abs(float(loss) - 1) <= (128 + 64 + 8 + 15 + 1) * 2.0 ** -24
    torch.cuda.empty_cache()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [8, 64, 100])
def test_scores_of_far_fp32_logits(E, score):
    """FP32 logits give scores and gradients to FP32, however far apart they are. Multiples of 2^-6, so that differences
    are exact; a token a sequence with one choice e, so that its loss is E p_e."""
    m = M()
    T = 3000
    log(f"case balance of far logits E={E} {score}")
    g = torch.Generator().manual_seed(E)
    x = torch.randint(-80 * 64, 1, (T, E), generator=g) / 64
    if score == "softmax":
        x += torch.randint(-40 * 64, 40 * 64, (T, 1), generator=g) / 64
    else:
        x[:, 0] = torch.randint(-20 * 64, 20 * 64, (T,), generator=g) / 64      # a sum of sigmoids above 2^-80
    ids = torch.randint(0, E, (T, 1), generator=g).int()
    off = torch.arange(T + 1, dtype=torch.int32)
    loss, n = m.router_balance(x.cuda(), ids.cuda(), score=score, offsets=off.cuda())
    p, rest = U.scores(x, score)
    want = E * p.gather(1, ids.long())[:, 0]
    # steps of 2^-24: e^x 4 (v_exp_f32 2, its correction 1, its input's last bits 1), 1 + x 1, its inverse 2, their product
    # 1; the sum of E terms 2 a lane and 6 of the lanes, besides its terms' own; its inverse 2, the product 1, the loss 1
    rel = (8 + 8 + 8 + 2 + 1 + 1) * 2.0 ** -24
    U.close(loss, want, want * rel + 2.0 ** -126 * E, "scores")
    d = m.router_balance_grad(x.cuda(), n, torch.ones(T).cuda(), 1, score=score, offsets=off.cuda()).cpu()
    # E p_i ([i = e] - p_e) (1 - s(l_i)): p twice, the difference 1, 1 - s 8, c 1, the wave's sum 6, products 4
    hit = torch.nn.functional.one_hot(ids[:, 0].long(), E).double()
    pe = p.gather(1, ids.long())
    exact = E * p * (hit - pe) * rest
    slack = E * p * rest * ((hit - pe).abs() * (28 + 8 + 6) + pe * (28 + 8)) * 2.0 ** -24
    U.close(d, exact, slack + 2.0 ** -126 * E, "gradient")
