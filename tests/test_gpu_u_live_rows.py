"""The operators in a row, forward and backward, checked row by row: every live
row's activations and gradients are finite and each row keeps to its own bound,
which a norm over all rows would hide; rows of no token are told apart by their
place, not by their value."""
import pytest
import torch

from tests.gpu_util import log, require_gpu
from tests.ops_util import check
from tests.test_gpu_n_operators import routed, tiny_handle

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,H,I,topk", [(1, 16, 256, 128, 4), (37, 16, 160, 96, 4), (300, 8, 256, 192, 2)])
def test_every_live_row(T, E, H, I, topk):
    require_gpu()
    import w4a16_int4_grouped_amd as M
    log(f"case live rows T={T} E={E} H={H} I={I}")
    h = tiny_handle(E, H, I)
    g = torch.Generator().manual_seed(T + 1)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, logits = r(T, H).bfloat16(), r(T, E)
    w1, w2 = (r(E, 2 * I, H) * H ** -0.5).bfloat16(), (r(E, H, I) * I ** -0.5).bfloat16()
    ids, _, a, off, slots = routed(M, h, x.cuda(), logits.cuda(), topk)
    lo, total, live = int(off[0]), int(off[-1]), slots.cpu()
    expert = ids.cpu().long().flatten()
    ends = off.cpu().long()
    assert ((ends[expert] <= live) & (live < ends[expert + 1])).all()      # a token's rows lie with its experts
    # the permuted rows: the token's, 0 in the padding of a group
    A = a.cpu()
    own = torch.zeros(a.shape[0], dtype=torch.bool)
    own[live] = True
    assert torch.equal(A[live], x.repeat_interleave(topk, 0))
    assert lo == 0 and (A[:total][~own[:total]] == 0).all()

    def product(name, got, q, p, C):
        """Each live row of `got` against q[row] . p[its expert]^T in 64 bits."""
        want = torch.stack([p[e].double() @ q[i].double() for e, i in zip(expert, live)])
        size = torch.stack([p[e].double().abs() @ q[i].double().abs() for e, i in zip(expert, live)])
        check(got[slots], want, size, C, name)

    hid = M.grouped_gemm(a, w1.cuda(), off)
    product("hidden", hid, A, w1, H)
    act = M.swiglu(hid)
    assert torch.isfinite(act[slots]).all()
    y = M.grouped_gemm(act, w2.cuda(), off)
    product("output", y, act.cpu(), w2, I)
    d_y = torch.zeros(a.shape[0], H, dtype=torch.bfloat16)
    d_y[live] = r(T * topk, H).bfloat16()
    d_act = M.grouped_gemm_dgrad(d_y.cuda(), w2.cuda(), off)
    product("gradient of the activation", d_act, d_y, w2.transpose(1, 2), H)
    hl = hid[slots].float().requires_grad_(True)
    (d,) = torch.autograd.grad(torch.nn.functional.silu(hl[:, :I]) * hl[:, I:], hl, d_act[slots].float())
    d_hid = torch.zeros_like(hid)
    d_hid[slots] = d.bfloat16()
    assert torch.isfinite(d_hid).all()
    product("gradient of the row", M.grouped_gemm_dgrad(d_hid, w1.cuda(), off), d_hid.cpu(), w1.transpose(1, 2), 2 * I)
    # weight gradients: the padding's rows are 0 in `a` and in the gradients, so they add nothing
    for name, dy, q in (("w1", d_hid, a), ("w2", d_y.cuda(), act)):
        got = M.grouped_gemm_wgrad(dy, q, off, out_dtype=torch.float32)
        DY, Q = dy.cpu().double(), q.cpu().double()
        rows = [live[expert == e] for e in range(E)]
        want = torch.stack([DY[i].T @ Q[i] for i in rows])
        size = torch.stack([DY[i].abs().T @ Q[i].abs() for i in rows])
        check(got, want, size, max(len(i) for i in rows) + 128, name)
