"""The operators of a training step as a program uses them: a whole expert layer
forward and backward against autograd in 64 bits, captured and replayed, on two
streams at once, on rows far apart, on data that breaks the documentation's
word; the same bits every time."""
import math

import pytest
import torch

from tests import step_util as U
from tests.gpu_util import log, require_gpu
from tests.ops_util import offsets_of, random_counts
from tests.test_gpu_n_operators import tiny_handle
from tests.test_gpu_p_reach import apart

pytestmark = pytest.mark.gpu


def M():
    require_gpu()
    import w4a16_int4_grouped_amd
    return w4a16_int4_grouped_amd


# ---- a layer ------------------------------------------------------------------------


class Layer:
    """One training step of a mixture of BF16 experts with biases, on the operators."""

    def __init__(self, T, E, H, I, topk, seed, ends):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.E, self.topk, self.I = E, topk, I
        self.h = tiny_handle(E, H, I)
        self.x, self.logits = r(T, H).bfloat16(), r(T, E)
        self.w1, self.w2 = (r(E, 2 * I, H) * H ** -0.5).bfloat16(), (r(E, H, I) * I ** -0.5).bfloat16()
        self.b1, self.b2 = (r(E, 2 * I) * 0.3).bfloat16(), (r(E, H) * 0.3).bfloat16()
        self.d_out, self.d_loss = r(T, H).bfloat16(), torch.tensor([30.0, -20.0, 10.0])
        self.ends = torch.tensor(ends, dtype=torch.int32)
        self.dev = {k: v.cuda() for k, v in vars(self).items() if isinstance(v, torch.Tensor)}

    def step(self, m):
        v, k, h = self.dev, self.topk, self.h
        T = self.x.shape[0]
        ids, w = m.router_topk(v["logits"], k, renorm=True)
        loss, counts = m.router_balance(v["logits"], ids, offsets=v["ends"])
        routing = h.align(ids)
        lay = h.routing_layout(T, k)
        part = lambda at, n: routing[at: at + n]  # noqa: E731
        off, src = part(lay.off_offsets, self.E + 1), part(lay.off_sorted, lay.cap)
        slots = part(lay.off_slot_of, T * k).view(T, k)
        xq = m.mx8_quant(v["x"])                                       # kept for the backward pass
        a, _, _ = h.permute(v["x"], k, routing)
        hid = m.grouped_linear(a, v["w1"], off, bias=v["b1"])
        act, hq, hs = m.swiglu_save(hid, offsets=off)                  # hq, hs kept
        y = m.grouped_linear(act, v["w2"], off, bias=v["b2"])          # y kept
        out = m.combine(y, slots, w)

        d_y, d_w = m.combine_grad(v["d_out"], slots, y=y, w=w, row_src=src, offsets=off)
        d_b2 = m.grouped_bias_grad(d_y, off, out_dtype=torch.float32)
        d_act = m.grouped_gemm_dgrad(d_y, v["w2"], off)
        d_hid, act2 = m.swiglu_grad(hq, d_act, scales=hs, offsets=off)
        d_w2 = m.grouped_gemm_wgrad(d_y, act2, off, out_dtype=torch.float32)
        d_b1 = m.grouped_bias_grad(d_hid, off, out_dtype=torch.float32)
        rows = m.mx8_dequant(*xq, row_src=src, topk=k, offsets=off)
        d_w1 = m.grouped_gemm_wgrad(d_hid, rows, off, out_dtype=torch.float32)
        d_x = m.combine(m.grouped_gemm_dgrad(d_hid, v["w1"], off), slots)
        d_logits = m.router_topk_grad(v["logits"], ids, d_w, renorm=True)
        m.router_balance_grad(v["logits"], counts, v["d_loss"], k, offsets=v["ends"], add=d_logits, out=d_logits)
        self.ids, self.counts = ids, counts
        return dict(out=out, loss=loss, x=d_x, logits=d_logits, w1=d_w1, w2=d_w2, b1=d_b1, b2=d_b2)

    def exact(self):
        ids, I, E, k = self.ids.cpu().long(), self.I, self.E, self.topk
        X, L, W1, W2, B1, B2 = (t.double().requires_grad_(True) for t in (self.x, self.logits, self.w1, self.w2, self.b1,
                                                                          self.b2))
        p = torch.softmax(L, 1)
        w = p.gather(1, ids)
        w = w / w.sum(1, keepdim=True)
        u = torch.einsum("tjnk,tk->tjn", W1[ids], X) + B1[ids]
        v = torch.nn.functional.silu(u[..., :I]) * u[..., I:]
        y = torch.einsum("tjhi,tji->tjh", W2[ids], v) + B2[ids]
        out = (y * w[..., None]).sum(1)
        loss = []
        for s, (lo, hi) in enumerate(U.sequences(len(ids), self.ends)):
            f = torch.bincount(ids[lo:hi].flatten(), minlength=E).double() / max((hi - lo) * k, 1)
            loss.append(E * (f * p[lo:hi].sum(0)).sum() / max(hi - lo, 1))
        loss = torch.stack(loss)
        grads = torch.autograd.grad((out * self.d_out.double()).sum() + (loss * self.d_loss.double()).sum(),
                                    (X, L, W1, W2, B1, B2))
        return dict(zip(("out", "loss", "x", "logits", "w1", "w2", "b1", "b2"), (out.detach(), loss.detach()) + grads))


@pytest.mark.parametrize("T,E,H,I,topk,ends", [(1, 16, 256, 128, 4, [0, 1, 1, 1]), (37, 16, 160, 96, 4, [0, 10, 10, 37]),
                                               (300, 8, 256, 192, 2, [0, 7, 180, 300])])
def test_expert_layer_forward_and_backward(T, E, H, I, topk, ends):
    m = M()
    log(f"case training step T={T} E={E} H={H} I={I}")
    layer = Layer(T, E, H, I, topk, T, ends)
    got = layer.step(m)
    want = layer.exact()
    # Of the norm over many values: a rounding to BF16 is 2^-9 at most; a value in 8 bits is off by up to a 64th of half
    # the power of two below its block's largest, 2^-7 / sqrt(3) of it in the mean, and the largest of 32 normal values
    # lies at 2.4 times their deviation on average: 1.1 %. Behind the checkpoint of h both g and u carry that, and the
    # derivatives of silu(g) u by them are within 1.1 times the values that they scale: 3.1 % at most, with the checkpoint
    # of x 4.2 %; up to six roundings to BF16 besides.
    six = 6 * 2.0 ** -8
    tol = dict(out=3 * 2.0 ** -8, loss=1e-5, logits=six, b2=six, w2=0.031 + six, x=0.031 + six, b1=0.031 + six, w1=0.042 + six)
    for name, t in tol.items():
        rel = float((got[name].double().cpu() - want[name]).norm() / want[name].norm())
        log(f"  {name}: {rel:.3g} (bound {t:.3g})")
        assert rel <= t, name
    again = layer.step(m)
    for name in got:
        assert torch.equal(got[name], again[name]), name


def test_whole_step_captured_and_replayed():
    """Every replay against the eager step on the same inputs, with eager work between."""
    m = M()
    layer = Layer(70, 16, 256, 128, 4, 3, [0, 20, 41, 70])
    eager = layer.step(m)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        layer.step(m)
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            held = layer.step(m)
    for i in range(4):
        g = torch.Generator().manual_seed(50 + i)
        for name in ("x", "d_out", "logits"):
            layer.dev[name].copy_(torch.randn(layer.dev[name].shape, generator=g).to(layer.dev[name].dtype))
        want = layer.step(m)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name in want:
            assert torch.equal(held[name], want[name]), (i, name)
        assert not torch.equal(held["x"], eager["x"])


# ---- calls of many kinds ----------------------------------------------------------------


def calls(m, big=False):
    """name -> call(stream), outputs of many sizes."""
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    T, E, k, H = (3000, 384, 8, 2560) if big else (300, 64, 4, 528)
    logits = r(T, E)
    ids, _ = m.router_topk(logits, k)
    ends = torch.tensor([0, T // 3, T // 2, T], dtype=torch.int32, device="cuda")
    _, counts = m.router_balance(logits, ids, offsets=ends)
    slots, src, off = (t.cuda() for t in U.routing(T, min(E, 48), k, 16, 5, 0.2))
    R = src.shape[0]
    y, w, d_out, d_loss = r(R, H).bfloat16(), r(T, k), r(T, H).bfloat16(), r(3)
    q, scales = m.mx8_quant(d_out)
    h, d_a = r(R, H).bfloat16(), r(R, H // 2).bfloat16()
    _, hq, hs = m.swiglu_save(h)
    wt, bias = (r(off.numel() - 1, 272, H) * H ** -0.5).bfloat16(), r(off.numel() - 1, 272)
    few = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    return {
        "router_balance": lambda s: m.router_balance(logits, ids, offsets=ends, stream=s),
        "router_balance of one": lambda s: m.router_balance(logits[:50], ids[:50], stream=s),
        "router_balance_grad": lambda s: m.router_balance_grad(logits, counts, d_loss, k, offsets=ends, stream=s),
        "combine": lambda s: m.combine(y, slots, w, stream=s),
        "combine_grad": lambda s: m.combine_grad(d_out, slots, y=y, w=w, row_src=src, stream=s),
        "mx8_quant": lambda s: m.mx8_quant(y, stream=s),
        "mx8_dequant": lambda s: m.mx8_dequant(q, scales, stream=s),
        "mx8_dequant of a routing": lambda s: m.mx8_dequant(q, scales, row_src=src, topk=k, stream=s),
        "swiglu_save": lambda s: m.swiglu_save(h, stream=s),
        "swiglu_grad": lambda s: m.swiglu_grad(hq, d_a, scales=hs, stream=s),
        "grouped_linear": lambda s: m.grouped_linear(y, wt, off, bias=bias, act="swiglu", stream=s),
        "grouped_bias_grad": lambda s: m.grouped_bias_grad(y, off, stream=s),
        "grouped_bias_grad in chunks": lambda s: m.grouped_bias_grad(y, few, stream=s),
    }


def tensors(out):
    return tuple(t for t in (out if isinstance(out, tuple) else (out,)) if t is not None)


def test_on_another_stream():
    """Outputs and workspaces are not of the current stream's memory, and hold what the current stream's calls give."""
    m = M()
    side = torch.cuda.Stream()
    for name, call in calls(m, big=True).items():
        log(f"case stream {name}")
        want = tensors(call(None))
        torch.cuda.synchronize()
        free = [torch.empty_like(t) for t in want]
        places = {t.data_ptr() for t in free if t.numel() * t.element_size() >= 1 << 20}
        del free
        got = tensors(call(side))
        side.synchronize()
        assert not places & {t.data_ptr() for t in got}, name
        for a, b in zip(got, want):
            assert torch.equal(a, b), name


def test_two_streams_at_once():
    m = M()
    made = calls(m)
    want = {n: tensors(c(None)) for n, c in made.items()}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(3):
        for n, c in made.items():
            for st in streams:
                got.append((n, tensors(c(st))))
    torch.cuda.synchronize()
    for n, out in got:
        for a, b in zip(out, want[n]):
            assert torch.equal(a, b), n


def test_each_call_captured_with_buffers_of_its_own():
    """Two graphs of the two-kernel calls that share a workspace, replayed in turn."""
    m = M()
    g = torch.Generator().manual_seed(1)
    x = [torch.randn(700, 100, generator=g).cuda() for _ in range(2)]
    ids = [t.topk(5, 1)[1].int() for t in x]
    dy = [torch.randn(6000, 72, generator=g).bfloat16().cuda() for _ in range(2)]
    off = torch.tensor([0, 6000], dtype=torch.int32, device="cuda")
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    st = torch.cuda.Stream()
    want, graphs, held = [], [], []
    for i in range(2):
        want.append(m.router_balance(x[i], ids[i]) + (m.grouped_bias_grad(dy[i], off),))
        gr = torch.cuda.CUDAGraph()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(gr, stream=st):
            held.append(m.router_balance(x[i], ids[i], ws=ws) + (m.grouped_bias_grad(dy[i], off, ws=ws),))
        graphs.append(gr)
    for _ in range(3):
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for i in range(2):
            for a, b in zip(held[i], want[i]):
                assert torch.equal(a, b)


def test_same_bits_every_time():
    m = M()
    for name, call in calls(m, big=True).items():
        want = tensors(call(None))
        for _ in range(4):
            for a, b in zip(tensors(call(None)), want):
                assert torch.equal(a, b), name


# ---- far apart --------------------------------------------------------------------------

FAR = 1 << 21


def test_rows_far_apart():
    m = M()
    slots, src, off = (t.cuda() for t in U.routing(400, 6, 3, 16, 1))
    R = src.shape[0]
    assert R > 1100
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    y, d, w = r(R, 72), r(400, 72), r(400, 3).float()
    far_y = apart(y, (FAR, 1))
    assert torch.equal(m.combine(far_y, slots, w), m.combine(y, slots, w))
    want, want_w = m.combine_grad(d, slots, y=y, w=w, row_src=src, offsets=off)
    out = apart(torch.full_like(y, 7), (FAR, 1))
    _, dw = m.combine_grad(d, slots, y=far_y, w=w, row_src=src, offsets=off, out=(out, None))
    assert torch.equal(out, want) and torch.equal(dw, want_w)
    q, s = m.mx8_quant(y)
    for a, b in zip(m.mx8_quant(far_y), (q, s)):
        assert torch.equal(a, b)
    m.mx8_dequant(q, s, row_src=src, topk=3, out=out)
    assert torch.equal(out, m.mx8_dequant(q, s, row_src=src, topk=3))
    h, d_a = r(R, 144), r(R, 72)
    far_h = apart(h, (FAR, 1))
    a, hq, hs = m.swiglu_save(h)
    got = m.swiglu_save(far_h, out=(out, torch.empty_like(hq), torch.empty_like(hs)))
    for p, v in zip(got, (a, hq, hs)):
        assert torch.equal(p, v)
    d_h, a2 = m.swiglu_grad(far_h, d_a)
    want = m.swiglu_grad(h, d_a)
    assert torch.equal(d_h, want[0]) and torch.equal(a2, want[1])
    m.swiglu_grad(hq, apart(d_a, (FAR, 1)), scales=hs, out=(far_h, out))
    want = m.swiglu_grad(hq, d_a, scales=hs)
    assert torch.equal(far_h, want[0]) and torch.equal(out, want[1])
    del far_h
    wt, bias = r(6, 144, 72), r(6, 144)
    res = apart(r(R, 72), (FAR, 1))
    want = m.grouped_linear(y, wt, off, bias=bias, act="swiglu", residual=res.contiguous(), out=torch.zeros_like(y))
    live = slice(0, int(off[-1]))
    got = m.grouped_linear(far_y, wt, off, bias=bias, act="swiglu", residual=res, out=res)
    assert torch.equal(got[live], want[live])
    assert torch.equal(m.grouped_bias_grad(far_y, off), m.grouped_bias_grad(y, off))


def test_weights_far_apart():
    """Gate and up halves 4.6 GB apart, rows of weights 4 MB."""
    m = M()
    g = torch.Generator(device="cuda").manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    a, w, bias = r(70, 72), r(1, 2224, 72), r(1, 2224)
    off = torch.tensor([0, 70], dtype=torch.int32, device="cuda")
    far = apart(w, (2224 * FAR, FAR, 1))
    for act in ("swiglu", "none"):
        assert torch.equal(m.grouped_linear(a, far, off, bias=bias, act=act), m.grouped_linear(a, w, off, bias=bias, act=act))
    a, off = r(3000, 72), torch.tensor([0, 3000], dtype=torch.int32, device="cuda")     # larger tiles
    assert torch.equal(m.grouped_linear(a, far, off, bias=bias, act="swiglu"),
                       m.grouped_linear(a, w, off, bias=bias, act="swiglu"))


def test_far_logits():
    m = M()
    x = torch.randn(600, 72, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    far = apart(x, (1 << 23, 1))
    ids = x.float().topk(5, 1)[1].int()
    want = m.router_balance(x, ids)
    for a, b in zip(m.router_balance(far, ids), want):
        assert torch.equal(a, b)
    d = torch.ones(1, device="cuda") * 1e5
    g = m.router_balance_grad(x, want[1], d, 5, add=x)
    m.router_balance_grad(x, want[1], d, 5, add=far, out=far)
    assert torch.equal(far, g)


def test_dense_rows_past_32_bits():
    """2^31 values and more: 8-bit rows of 8200, read back and as a routing; the rows at both ends are looked at."""
    m = M()
    rows, K = 262150, 8200
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    look = torch.tensor([0, 1, 131071, 262143, 262144, rows - 1])
    part = torch.randn(len(look), K, generator=torch.Generator().manual_seed(1)).bfloat16()
    x[look.cuda()] = part.cuda()
    q, s = m.mx8_quant(x)
    val = U.mx8(part)[0].bfloat16()
    assert torch.equal(m.mx8_dequant(q, s)[look.cuda()].cpu(), val)
    src = torch.arange(rows - 1, -1, -1, dtype=torch.int32, device="cuda")
    assert torch.equal(m.mx8_dequant(q, s, row_src=src, out=x)[(rows - 1 - look).cuda()].cpu(), val)


def test_more_routed_groups_than_32_bits_count():
    """8.4 million rows of 2056 read back from four: 2^31 groups of 8, of a width that fills its threads badly."""
    m = M()
    K, R = 2056, 8400003
    assert R * (K // 8) > 1 << 31
    x = torch.randn(4, K, generator=torch.Generator().manual_seed(3)).bfloat16()
    q, s = m.mx8_quant(x.cuda())
    val = U.mx8(x)[0].bfloat16().cuda()
    src = (torch.arange(R, device="cuda") * 7 % 5).int()                 # 4: no row
    out = torch.full((R, K), 3.0, dtype=torch.bfloat16, device="cuda")
    m.mx8_dequant(q, s, row_src=src, out=out)
    val = torch.cat([val, torch.zeros_like(val[:1])])
    for lo in (0, R // 4 - 20, R // 4 + 5, R // 2, R - 100):
        assert torch.equal(out[lo: lo + 100], val[src[lo: lo + 100].long()]), lo
    assert not (out[:, 0] == 3).any()


def test_many_sequences_and_many_tokens():
    """More sequences than a wave looks at in one step, most of them short or empty, and chunks of many rows."""
    m = M()
    T, E, k = 70001, 70, 3
    g = torch.Generator().manual_seed(7)
    for S in (65, 500, 5000):
        cuts = torch.randint(0, T + 1, (S - 1,), generator=g).sort()[0]
        cuts[S // 2: S // 2 + 20] = cuts[S // 2]
        off = torch.cat([torch.tensor([5]), cuts.clamp(5, T - 9).sort()[0], torch.tensor([T - 9])]).int()
        x = (torch.randn(T, E, generator=g) * 1.5).bfloat16()
        ids = x.float().topk(k, 1)[1].int()
        loss, counts = m.router_balance(x.cuda(), ids.cuda(), offsets=off.cuda())
        want, n = U.balance(x, ids, "softmax", off)
        assert torch.equal(counts.cpu(), n)
        U.close(loss, want, want.abs() * (float(U.score_error(x).max()) + 400 * 2.0 ** -24), f"loss of {S}")
        d_loss = torch.randn(S, generator=g) * E * T / S
        d = m.router_balance_grad(x.cuda(), counts, d_loss.cuda(), k, offsets=off.cuda())
        exact, slack = U.balance_grad(x, n, d_loss, k, "softmax", off)
        U.close(d, exact, slack, f"gradient of {S}")
        assert (d[:5] == 0).all() and (d[T - 9:] == 0).all()


def test_long_sums_of_the_largest_router():
    m = M()
    x = torch.randn(3000, 4096, generator=torch.Generator().manual_seed(2)).bfloat16()
    ids = x.float().topk(64, 1)[1].int()
    loss, counts = m.router_balance(x.cuda(), ids.cuda(), score="sigmoid")
    want, n = U.balance(x, ids, "sigmoid", None)
    assert torch.equal(counts.cpu(), n)
    U.close(loss, want, want.abs() * (float(U.score_error(x).max()) + 160 * 2.0 ** -24), "loss")


# ---- against the documentation's word ------------------------------------------------------


def guarded(shape, dtype, fill=7):
    """A tensor between two guards of 4 KB, and the check of both."""
    n = math.prod(shape)
    pad = 4096 // torch.empty(0, dtype=dtype).element_size()
    buf = torch.full((n + 2 * pad,), fill, dtype=dtype, device="cuda")
    return buf[pad: pad + n].view(shape), lambda: bool((buf[:pad] == fill).all() and (buf[pad + n:] == fill).all())


def test_bad_offsets_and_indices_touch_nothing_else():
    """Offsets that decrease, or lie outside the rows, and slots and sources of any value: outputs may hold anything,
    memory beside them stays as it was."""
    m = M()
    T, E, k, H, R = 90, 12, 3, 264, 200
    g = torch.Generator().manual_seed(3)
    big = 2 ** 31 - 1
    wild = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in
            ([0, 50, 20, 90], [-5, 30, 300, 90], [big, -big, big, -big], [60, 10, 80, 5], [-big, big, big, big], [90, 0, 0, 0])]
    x = torch.randn(T, E, generator=g).cuda()
    ids = torch.randint(-(2 ** 31), 2 ** 31 - 1, (T, k), generator=g).int().cuda()
    slots = torch.randint(-(2 ** 31), 2 ** 31 - 1, (T, k), generator=g).int().cuda()
    slots[::2] = torch.randint(0, R, (45, k), generator=g).int().cuda()          # rows named more than once among them
    src = torch.randint(-(2 ** 31), 2 ** 31 - 1, (R,), generator=g).int().cuda()
    y, d = torch.randn(R, H, generator=g).bfloat16().cuda(), torch.randn(T, H, generator=g).bfloat16().cuda()
    w = torch.randn(T, k, generator=g).cuda()
    wt = torch.randn(3, 2 * H, H, generator=g).bfloat16().cuda()
    q, s = m.mx8_quant(d)
    for off in wild:
        outs = dict(loss=guarded((3,), torch.float32), counts=guarded((3, E), torch.int32), d=guarded((T, E), torch.float32),
                    dy=guarded((R, H), torch.bfloat16), dw=guarded((T, k), torch.float32), a=guarded((R, H // 2 // 8 * 8), torch.bfloat16),
                    hq=guarded((R, 2, H // 2 // 8 * 8), torch.int8), hs=guarded((R, 2, 16), torch.uint8),
                    dh=guarded((R, H // 2 // 8 * 16), torch.bfloat16), lin=guarded((R, H), torch.bfloat16), db=guarded((3, H), torch.float32))
        o = {n: t for n, (t, _) in outs.items()}
        nbytes = m.lib().moe_router_balance_bytes(T, E, 3)
        ws, ws_ok = guarded((nbytes,), torch.uint8)
        o["counts"].zero_()
        m.router_balance(x, ids, offsets=off, out=(o["loss"], o["counts"]), ws=ws)
        m.router_balance_grad(x, o["counts"], torch.ones(3, device="cuda"), k, offsets=off, out=o["d"])
        m.combine_grad(d, slots, y=y, w=w, row_src=src, offsets=off, out=(o["dy"], o["dw"]))
        m.mx8_dequant(q, s, row_src=src, topk=k, offsets=off, out=o["lin"])
        I = H // 2 // 8 * 8
        h = y[:, : 2 * I]
        m.swiglu_save(h, offsets=off, out=(o["a"], o["hq"], o["hs"]))
        m.swiglu_grad(o["hq"], o["a"], scales=o["hs"], offsets=off, out=(o["dh"], None))
        m.grouped_linear(y, wt, off, act="swiglu", residual=y, out=o["lin"])
        m.grouped_bias_grad(y, off, out=o["db"])
        torch.cuda.synchronize()
        assert ws_ok()
        for n, (_, ok) in outs.items():
            assert ok(), n
    # a chunked bias gradient on such offsets
    dy = torch.randn(9000, 64, generator=g).bfloat16().cuda()
    for off in wild:
        off = off[:2].contiguous()
        nbytes = m.lib().moe_grouped_bias_grad_bytes(1, 9000, 64)
        assert nbytes > 0
        (ws, ws_ok), (db, ok) = guarded((nbytes,), torch.uint8), guarded((1, 64), torch.float32)
        m.grouped_bias_grad(dy, off, out=db, ws=ws)
        torch.cuda.synchronize()
        assert ws_ok() and ok()


def test_a_row_summed_more_than_once():
    m = M()
    y = torch.randn(3, 40, generator=torch.Generator().manual_seed(1))
    slots = torch.tensor([[0, 0, 2], [1, -1, 1], [2, 0, 1 << 30], [0, 0, 0]], dtype=torch.int32)
    w = torch.tensor([[1.0, 2, 3], [4, 5, 6], [0.5, -1, 9], [0, 0, 0]])
    out = m.combine(y.cuda(), slots.cuda(), w.cuda()).cpu()
    want = torch.stack([3 * y[0] + 3 * y[2], 10 * y[1], 0.5 * y[2] - y[0], 0 * y[0]])
    assert torch.allclose(out, want, rtol=0, atol=4 * 2.0 ** -23 * float(10 * y.abs().max()))


# ---- the ends of the ranges ------------------------------------------------------------------


def test_widest_rows():
    """2^20 columns (SwiGLU 2 x 2^19)."""
    m = M()
    W = 1 << 20
    g = torch.Generator().manual_seed(1)
    x = torch.randn(3, W, generator=g).bfloat16()
    q, s = m.mx8_quant(x.cuda())
    val, code, byte = U.mx8(x)
    assert torch.equal(q.cpu(), code) and torch.equal(s.cpu(), byte)
    assert torch.equal(m.mx8_dequant(q, s).cpu(), val.bfloat16())
    src = torch.tensor([5, 6, 0, 2, 1], dtype=torch.int32)       # of 3 x 2
    want = torch.stack([val[2], 0 * val[0], val[0], val[1], val[0]]).bfloat16()
    assert torch.equal(m.mx8_dequant(q, s, row_src=src.cuda(), topk=2).cpu(), want)
    a, hq, hs = m.swiglu_save(x.cuda())
    U.close(a, U.swiglu(x), U.swiglu_slack(x), "a")
    d_a = torch.randn(3, W // 2, generator=g).bfloat16()
    exact, slack = U.swiglu_grad(x, d_a)
    U.close(m.swiglu_grad(x.cuda(), d_a.cuda())[0], exact, slack, "d_h")
    slots = torch.tensor([[2, 0], [-1, 1]], dtype=torch.int32)
    w = torch.tensor([[0.5, 2.0], [3.0, -1.0]])
    out = m.combine(x.cuda(), slots.cuda(), w.cuda(), out_dtype=torch.float32).cpu().double()
    v = x.double()
    want = torch.stack([0.5 * v[2] + 2 * v[0], -v[1]])
    assert ((out - want).abs() <= (0.5 * v[2].abs() + 2 * v[0].abs() + v[1].abs()) * 2.0 ** -22).all()
    d_out = x[:2]
    dy, dw = m.combine_grad(d_out.cuda(), slots.cuda(), y=x.cuda(), w=w.cuda())
    d = d_out.double()
    assert torch.equal(dy.cpu(), torch.stack([2 * d[0], -d[1], 0.5 * d[0]]).bfloat16())
    want = torch.tensor([[float((d[0] * v[2]).sum()), float((d[0] * v[0]).sum())], [0.0, float((d[1] * v[1]).sum())]])
    size = torch.tensor([[float((d[0] * v[2]).abs().sum()), float((d[0] * v[0]).abs().sum())], [0.0, float((d[1] * v[1]).abs().sum())]])
    # a thread adds 2^20 / 256 products one after another, the rest are trees
    assert ((dw.cpu().double() - want).abs() <= size * (W / 256 + 12) * 2.0 ** -24).all()


def test_most_experts_and_sequences():
    m = M()
    g = torch.Generator().manual_seed(2)
    counts = [int(c) for c in torch.randint(0, 3, (4096,), generator=g)]
    rows = sum(counts)
    a, w = torch.randn(rows, 8, generator=g).bfloat16(), torch.randn(4096, 16, 8, generator=g).bfloat16()
    bias = torch.randn(4096, 16, generator=g)
    off = offsets_of(counts).cuda()
    for act in ("none", "swiglu"):
        exact, slack = U.linear(a, w, counts, bias, act, None)
        U.close(m.grouped_linear(a.cuda(), w.cuda(), off, bias=bias.cuda(), act=act), exact, slack, act)
    dy = torch.randn(rows, 16, generator=g).bfloat16()
    want = torch.stack([t.double().sum(0) for t in dy.split(counts)])
    U.close(m.grouped_bias_grad(dy.cuda(), off), want, 4 * 2.0 ** -24 * 10, "bias")
    # 2^20 sequences, nearly all empty
    S, T, E = 1 << 20, 500, 9
    cuts = torch.randint(0, S + 1, (T,), generator=g).sort()[0]
    ends = torch.bincount(cuts, minlength=S + 1).cumsum(0).int()         # of sequence s: the rows drawn up to it
    ends = torch.cat([torch.zeros(1, dtype=torch.int32), ends[:S]])
    x = torch.randn(T, E, generator=g)
    ids = x.topk(2, 1)[1].int()
    loss, n = m.router_balance(x.cuda(), ids.cuda(), offsets=ends.cuda())
    loss, n = loss.cpu(), n.cpu()
    last = int(ends[-1])
    assert int(n.sum()) == 2 * last and int((n.sum(1) > 0).sum()) == len(set(cuts[:last].tolist()))
    busy = (n.sum(1) > 0).nonzero()[:, 0]
    assert (loss[n.sum(1) == 0] == 0).all()
    p, _ = U.scores(x, "softmax")
    for s in busy[:40].tolist():
        lo, hi = int(ends[s]), int(ends[s + 1])
        want = E * (n[s].double() / (2 * (hi - lo)) * p[lo:hi].mean(0)).sum()
        assert abs(float(loss[s]) - float(want)) <= float(want) * 64 * 2.0 ** -23
