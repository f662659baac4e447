"""Router top-k and its gradient against 64-bit references: ids equal (ties
to the lowest index), weights and gradients within FP32 roundings, masked
experts, rows that leave fewer than k experts."""
import pytest
import torch

from tests.gpu_util import log, require_gpu

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def reference(logits, k, score, bias, renorm, scale):
    """(ids, weights, scores) in 64 bits on the CPU."""
    x = logits.double().cpu()
    x = torch.where(torch.isnan(x), -torch.inf, x).clamp(max=torch.finfo(torch.float32).max)
    if score == "softmax":
        top = x.amax(1, keepdim=True)
        p = torch.exp(x - torch.where(top == -torch.inf, 0.0, top))
        p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        p = torch.sigmoid(x)
    key = x if bias is None else p + bias.double().cpu()
    key = torch.where((x == -torch.inf) | torch.isnan(key), -torch.inf, key)
    val, ids = torch.sort(key, dim=1, descending=True, stable=True)
    ids, val = ids[:, :k], val[:, :k]
    got = val > -torch.inf
    if renorm:
        l = x.gather(1, ids)
        l = torch.where(got, l if score == "softmax" else torch.nn.functional.logsigmoid(l), -torch.inf)
        top = l.amax(1, keepdim=True)
        u = torch.exp(l - torch.where(top == -torch.inf, 0.0, top))
        w = u / u.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        w = p.gather(1, ids)
    return torch.where(got, ids, -1), torch.where(got, w * scale, 0.0), p


CASES = [
    # T, E, k, score, bias, renorm, dtype
    (1, 8, 2, "softmax", False, True, "bf16"),
    (1, 1, 1, "sigmoid", True, False, "fp32"),
    (5, 64, 64, "softmax", False, False, "fp32"),
    (7, 65, 6, "sigmoid", True, True, "bf16"),
    (33, 384, 8, "sigmoid", True, True, "fp32"),
    (130, 384, 8, "softmax", False, True, "bf16"),
    (64, 256, 4, "softmax", True, False, "fp16"),
    (9, 513, 16, "softmax", True, True, "fp32"),
    (3, 1025, 33, "sigmoid", False, False, "fp32"),
    (2, 4096, 64, "softmax", False, False, "bf16"),
    (2, 4096, 64, "sigmoid", True, True, "fp32"),
]


def inputs(T, E, dtype, bias, seed):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, E, generator=g) * 2).to(DT[dtype])
    b = (torch.randn(E, generator=g) * 0.1) if bias else None
    return x, b


@pytest.mark.parametrize("T,E,k,score,bias,renorm,dtype", CASES)
def test_topk(T, E, k, score, bias, renorm, dtype):
    require_gpu()
    import w4a16_int4_grouped_amd as M
    log(f"case router T={T} E={E} k={k} {score} bias={bias} renorm={renorm} {dtype}")
    x, b = inputs(T, E, dtype, bias, T * 7 + E)
    ids, w = M.router_topk(x.cuda(), k, score, None if b is None else b.cuda(), renorm, 2.5)
    rid, rw, _ = reference(x, k, score, b, renorm, 2.5)
    assert torch.equal(ids.cpu().long(), rid)
    # a score takes exp, a sum of up to E terms added in 64 lanes and a division: E/64 + 20 roundings, with
    # exp's own error of a few 2^-24 relative
    assert torch.allclose(w.double().cpu(), rw, rtol=(E / 64 + 20) * 2.0 ** -24, atol=1e-37)


@pytest.mark.parametrize("score,bias", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
@pytest.mark.parametrize("renorm", [False, True])
def test_masked_and_extreme_logits(score, bias, renorm):
    require_gpu()
    import w4a16_int4_grouped_amd as M
    E, k = 70, 4
    inf, nan, low = float("inf"), float("nan"), torch.finfo(torch.float32).min
    x, b = inputs(9, E, "fp32", bias, 5)
    x[0] = -inf                       # no expert left
    x[1] = nan
    x[2] = -inf
    x[2, 69] = 1.0                    # one left
    x[3] = low                        # the type's lowest value is a logit like any other
    x[4] = -inf
    x[4, [3, 66]] = low
    x[5, ::2] = nan
    x[6] = 0.0                        # all equal: the lowest indices
    x[7, 40] = inf
    x[8] = -300.0                     # sigmoid underflows FP32
    x[8, 11] = -299.0
    log(f"case router masks {score} bias={bias} renorm={renorm}")
    ids, w = M.router_topk(x.cuda(), k, score, None if b is None else b.cuda(), renorm)
    rid, rw, _ = reference(x, k, score, b, renorm, 1.0)
    assert torch.equal(ids.cpu().long(), rid)
    assert torch.isfinite(w).all()
    assert torch.allclose(w.double().cpu(), rw, rtol=22 * 2.0 ** -24, atol=2.0 ** -126)


def test_bias_masks_and_ties():
    require_gpu()
    import w4a16_int4_grouped_amd as M
    x = torch.zeros(2, 130)
    x[1] = torch.linspace(-1, 1, 130)
    b = torch.zeros(130)
    b[0], b[129] = -float("inf"), float("nan")
    ids, w = M.router_topk(x.cuda(), 3, "sigmoid", b.cuda(), False)
    assert ids.cpu().tolist() == [[1, 2, 3], [128, 127, 126]]
    # scores that FP32 cannot tell from each other: the bias decides in FP64
    x = torch.full((1, 64), 20.0)
    x[0, 50] = 20.5
    ids, _ = M.router_topk(x.cuda(), 1, "sigmoid", torch.zeros(64).cuda(), False)
    assert ids.item() == 50


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_order_of_every_kind_of_value(dtype):
    """Signed zeros are equal (the lower index first), subnormals are not; the largest finite value and infinity."""
    require_gpu()
    import w4a16_int4_grouped_amd as M
    f = torch.finfo(DT[dtype])
    tiny = f.smallest_normal * f.eps
    x = torch.tensor([[-0.0, 0.0, -tiny, tiny, 2 * tiny, -2 * tiny, f.max, float("inf"), f.min, -0.0, 1.0, f.max]],
                     dtype=torch.float64).to(DT[dtype])
    for shift in range(12):
        y = torch.roll(x, shift, 1)
        rid, rw, _ = reference(y, 12, "sigmoid", None, False, 1.0)
        ids, w = M.router_topk(y.cuda(), 12, "sigmoid")
        assert torch.equal(ids.cpu().long(), rid), shift
        assert torch.allclose(w.cpu().double(), rw, rtol=22 * 2.0 ** -24, atol=2.0 ** -126)


def test_strided_rows_out_stream_and_guards():
    require_gpu()
    import w4a16_int4_grouped_amd as M
    T, E, k = 21, 100, 5
    wide = torch.full((T, 137), 9.0, device="cuda")
    x, _ = inputs(T, E, "fp32", False, 3)
    view = wide[:, 3:3 + E]
    view.copy_(x)
    ids = torch.full((T + 1, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, k), 7.0, device="cuda")
    d_wide = torch.full((T + 1, 140), 5.0, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    M.router_topk(view, k, out=(ids[:T], w[:T]), stream=s)
    M.router_topk_grad(view, ids[:T], w[:T], out=d_wide[:T, :E], stream=s)
    s.synchronize()
    rid, rw, _ = reference(x, k, "softmax", None, False, 1.0)
    assert torch.equal(ids[:T].cpu().long(), rid)
    assert (ids[T] == -7).all() and (w[T] == 7.0).all()
    assert (d_wide[:T, E:] == 5.0).all() and (d_wide[T] == 5.0).all()
    assert torch.equal(d_wide[:T, :E], M.router_topk_grad(view, ids[:T], w[:T]))


def grad_reference(x, ids, dw, score, renorm, scale):
    """By autograd in 64 bits on the CPU."""
    l = torch.where(torch.isnan(x.double()), -torch.inf, x.double()).requires_grad_(True)
    p = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
    got = ids >= 0
    s = torch.where(got, p.gather(1, ids.clamp(min=0)), 0.0)
    w = s / s.sum(1, keepdim=True) if renorm else s
    (g,) = torch.autograd.grad((scale * w * torch.where(got, dw.double(), 0.0)).sum(), l)
    return g


@pytest.mark.parametrize("T,E,k,score,bias,renorm,dtype", CASES)
def test_gradient(T, E, k, score, bias, renorm, dtype):
    require_gpu()
    import w4a16_int4_grouped_amd as M
    log(f"case router gradient T={T} E={E} k={k} {score} renorm={renorm} {dtype}")
    x, b = inputs(T, E, dtype, bias, T * 7 + E)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(E))
    ids, w = M.router_topk(x.cuda(), k, score, None if b is None else b.cuda(), renorm, 2.5)
    d = M.router_topk_grad(x.cuda(), ids, dw.cuda(), score, renorm, 2.5)
    ref = grad_reference(x, ids.cpu().long(), dw, score, renorm, 2.5)
    # d = p (g - <g, p>): a difference of terms of at most |g| max, p with the roundings of test_topk
    f = torch.finfo(DT[dtype])
    top = 2.5 * float(dw.abs().max())
    tol = (E / 64 + k + 30) * 2.0 ** -24 * top + ref.abs() * f.eps / 2 + f.smallest_normal * f.eps
    err = (d.double().cpu() - ref).abs()
    log(f"  worst {float((err / tol).max()):.3g} of its bound")
    assert d.dtype == DT[dtype] and (err <= tol).all()


def test_gradient_against_differences():
    """(w(l + h) - w(l - h)) . dw / 2h for a sample of logits, with the reference's weights in 64 bits: h = 1e-4
    leaves a truncation of h^2 and nothing of FP32; the chosen ids stay (the gap at the border is larger)."""
    require_gpu()
    import w4a16_int4_grouped_amd as M
    E, k, h = 40, 4, 1e-4
    g = torch.Generator().manual_seed(3)
    x = torch.randperm(E, generator=g).float()[None] * 0.05
    dw = torch.randn(1, k, generator=g)
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            ids, _ = M.router_topk(x.cuda(), k, score, None, renorm, 1.5)
            d = M.router_topk_grad(x.cuda(), ids, dw.cuda(), score, renorm, 1.5).cpu().double()
            for e in list(range(0, E, 7)) + ids[0].tolist():
                up, dn = x.double().clone(), x.double().clone()
                up[0, e] += h
                dn[0, e] -= h
                num = [(reference(v, k, score, None, renorm, 1.5)[1] * dw.double()).sum() for v in (up, dn)]
                assert abs(float((num[0] - num[1]) / (2 * h)) - float(d[0, e])) < 1e-6, (score, renorm, e)


def test_gradient_of_masked_rows_and_repeated_ids():
    require_gpu()
    import w4a16_int4_grouped_amd as M
    x = torch.randn(4, 70, generator=torch.Generator().manual_seed(1))
    x[0] = -float("inf")
    x[1, 1:] = -float("inf")
    ids = torch.tensor([[-1, -1, -1], [0, -1, -1], [5, 99, -3], [7, 7, 9]], dtype=torch.int32)
    dw = torch.ones(4, 3)
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            d = M.router_topk_grad(x.cuda(), ids.cuda(), dw.cuda(), score, renorm).cpu()
            assert torch.isfinite(d).all()
            assert (d[0] == 0).all()
            if score == "softmax" or renorm:
                assert d[1].abs().max() < 1e-6       # one expert left: its weight is a constant
            assert (d[2] != 0).sum() <= (70 if score == "softmax" and not renorm else 1)
    one = M.router_topk_grad(x.cuda(), torch.tensor([[7, -1, 9]] * 4, dtype=torch.int32).cuda(),
                             torch.tensor([[2.0, 0.0, 1.0]] * 4).cuda(), "sigmoid", False).cpu()
    two = M.router_topk_grad(x.cuda(), ids[3:].expand(4, 3).contiguous().cuda(), dw.cuda(), "sigmoid", False).cpu()
    assert torch.allclose(one[3], two[3], rtol=1e-6)
