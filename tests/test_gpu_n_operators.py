"""The operators in a row, as a model runs them: router, alignment, permuted
rows, grouped products (BF16 and MXFP4) with SwiGLU between, against the
expert layer in 64 bits; and the router in front of the INT4 layer."""
import numpy as np
import pytest
import torch

import synth
from tests.gpu_util import bits_host, log, prepare, require_gpu
from tests.ops_util import mx_reference

pytestmark = pytest.mark.gpu


def routed(M, h, x, logits, topk):
    """Ids, weights and the permuted rows with their offsets."""
    T = x.shape[0]
    ids, w = M.router_topk(logits, topk, renorm=True)
    routing = h.align(ids)
    lay = h.routing_layout(T, topk)
    a, _, _ = h.permute(x, topk, routing)
    off = routing[lay.off_offsets: lay.off_offsets + h.E + 1]
    slots = routing[lay.off_slot_of: lay.off_slot_of + T * topk].long()
    return ids, w, a, off, slots


def tiny_handle(E, H, I):
    from tests.test_gpu_a_kernels import tiny_weights
    return prepare(tiny_weights(E, H, I, seed=5), "indexed")


@pytest.mark.parametrize("T,E,H,I,topk", [(1, 16, 256, 128, 4), (37, 16, 160, 96, 4), (300, 8, 256, 192, 2)])
def test_expert_layer_forward_and_backward(T, E, H, I, topk):
    require_gpu()
    import w4a16_int4_grouped_amd as M
    log(f"case operators T={T} E={E} H={H} I={I}")
    h = tiny_handle(E, H, I)
    g = torch.Generator().manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, logits = r(T, H).bfloat16(), r(T, E)
    w1, w2 = (r(E, 2 * I, H) * H ** -0.5).bfloat16(), (r(E, H, I) * I ** -0.5).bfloat16()
    ids, tw, a, off, slots = routed(M, h, x.cuda(), logits.cuda(), topk)
    hid = M.grouped_gemm(a, w1.cuda(), off)
    act = M.swiglu(hid)
    y = M.grouped_gemm(act, w2.cuda(), off)
    out = (y.float()[slots].view(T, topk, H) * tw[..., None]).sum(1).cpu().double()
    ref = torch.zeros(T, H, dtype=torch.float64)
    idc, twc = ids.cpu().long(), tw.cpu().double()
    for t in range(T):
        for j in range(topk):
            e = int(idc[t, j])
            u = w1[e].double() @ x[t].double()
            v = torch.nn.functional.silu(u[:I]) * u[I:]
            ref[t] += twc[t, j] * (w2[e].double() @ v)
    # three roundings to BF16 on the way, 2^-9 each in the norm over many values
    assert float((out - ref).norm() / ref.norm()) < 3 * 2.0 ** -8
    # backward: every gradient from the calls, fed to an autograd of the same function in 64 bits
    dout = r(T, H)
    d_y = torch.zeros(a.shape[0], H)
    d_y[slots.cpu()] = (dout[:, None, :] * tw.cpu()[..., None]).reshape(T * topk, H)
    d_y = d_y.bfloat16().cuda()
    d_act = M.grouped_gemm_dgrad(d_y, w2.cuda(), off)
    d_w2 = M.grouped_gemm_wgrad(d_y, act, off, out_dtype=torch.float32)
    d_tw = (y.float()[slots].view(T, topk, H) * dout.cuda()[:, None]).sum(-1)
    d_logits = M.router_topk_grad(logits.cuda(), ids, d_tw, renorm=True)
    hl = hid.float().requires_grad_(True)
    (d_hid,) = torch.autograd.grad(torch.nn.functional.silu(hl[:, :I]) * hl[:, I:], hl, d_act.float())
    d_hid = torch.where(torch.isfinite(d_hid), d_hid, 0.0).bfloat16()
    d_a = M.grouped_gemm_dgrad(d_hid, w1.cuda(), off)
    d_w1 = M.grouped_gemm_wgrad(d_hid, a, off, out_dtype=torch.float32)
    d_x = d_a.float()[slots].view(T, topk, H).sum(1)
    X, L = x.double().requires_grad_(True), logits.double().requires_grad_(True)
    W1, W2 = w1.double().requires_grad_(True), w2.double().requires_grad_(True)
    p = torch.softmax(L, 1).gather(1, idc)
    p = p / p.sum(1, keepdim=True)
    u = torch.einsum("tjnk,tk->tjn", W1[idc], X)
    v = torch.nn.functional.silu(u[..., :I]) * u[..., I:]
    o = (torch.einsum("tjhi,tji->tjh", W2[idc], v) * p[..., None]).sum(1)
    ref = torch.autograd.grad((o * dout.double()).sum(), (X, L, W1, W2))
    for name, got, want in zip(("x", "logits", "w1", "w2"), (d_x, d_logits, d_w1, d_w2), ref):
        rel = float((got.double().cpu() - want).norm() / want.norm())
        log(f"  gradient of {name}: {rel:.3g}")
        assert rel < 6 * 2.0 ** -8, name      # at most six BF16 roundings behind each other


def test_mxfp4_expert_layer():
    require_gpu()
    import w4a16_int4_grouped_amd as M
    T, E, H, I, topk = 65, 16, 256, 128, 4
    h = tiny_handle(E, H, I)
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, logits = r(T, H).bfloat16(), r(T, E)
    w1, w2 = r(E, 2 * I, H) * H ** -0.5, r(E, H, I) * I ** -0.5
    w1q, w2q = M.mx_quant(w1.cuda()), M.mx_quant(w2.cuda())
    ids, tw, a, off, slots = routed(M, h, x.cuda(), logits.cuda(), topk)
    hid = M.mx_grouped_gemm(*M.mx_quant(a), *w1q, off)
    act = M.swiglu(hid)
    y = M.mx_grouped_gemm(*M.mx_quant(act), *w2q, off).float()[slots].view(T, topk, H).cpu().double()
    # the same layer on the values the codes stand for, fed the kernel's own hand-offs
    W1, W2 = mx_reference(w1)[0], mx_reference(w2)[0]
    X, A = mx_reference(x)[0], mx_reference(act.cpu())[0]
    hc, idc = hid.cpu().double()[slots.cpu()].view(T, topk, 2 * I), ids.cpu().long()
    ref_h = torch.einsum("tjnk,tk->tjn", W1[idc], X)
    ref_y = torch.einsum("tjhi,tji->tjh", W2[idc], A[slots.cpu()].view(T, topk, I))
    for got, want in ((hc, ref_h), (y, ref_y)):
        # one rounding to BF16 (2^-8 of the value at most) and FP32 sums
        assert ((got - want).abs() <= want.abs() * 2.0 ** -8 + 1e-3 * want.abs().amax() * 2.0 ** -8).all()


def test_router_feeds_the_int4_layer():
    require_gpu()
    import w4a16_int4_grouped_amd as M
    T, E, H, I, topk = 40, 16, 256, 128, 4
    h = tiny_handle(E, H, I)
    x = torch.from_numpy(synth.activations(3, T, H).view(np.int16)).view(torch.bfloat16).cuda()
    logits = torch.randn(T, E, generator=torch.Generator().manual_seed(2))
    logits[5] = -float("inf")                      # a token no expert takes
    ids, w = M.router_topk(logits.cuda(), topk, score="sigmoid", bias=torch.zeros(E).cuda(), renorm=True, scale=2.5)
    out = h.indexed(x, ids, w)
    assert (out[5] == 0).all()
    order = torch.sort(logits.double(), dim=1, descending=True, stable=True)[1][:, :topk].int()
    s = torch.sigmoid(logits.double().gather(1, order.long()))
    keep = torch.arange(T) != 5
    assert torch.equal(ids.cpu()[keep], order[keep])
    again = h.indexed(x, ids.clone(), w.clone())
    assert np.array_equal(bits_host(out), bits_host(again))
    assert torch.allclose(w.cpu().double()[keep], (2.5 * s / s.sum(1, keepdim=True))[keep], rtol=1e-5)
