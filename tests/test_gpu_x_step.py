"""Operators of a training step against 64 bits: balance loss, a token's rows,
rows in 8 bits, SwiGLU with a checkpoint, and their gradients."""
import math

import pytest
import torch

from tests import step_util as U
from tests.gpu_util import log, require_gpu
from tests.ops_util import check

pytestmark = pytest.mark.gpu
DT = U.DT


def M():
    require_gpu()
    import w4a16_int4_grouped_amd
    return w4a16_int4_grouped_amd


def cuda(*ts):
    return tuple(None if t is None else t.cuda() for t in ts)


def logits_of(T, E, dtype, seed, masked=False, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, E, generator=g) * spread + torch.randn(E, generator=g) * 0.5).to(DT[dtype])
    if masked:
        x[torch.rand(T, E, generator=g) < 0.15] = -math.inf
        x[torch.rand(T, E, generator=g) < 0.02] = math.nan
        x[2::7] = -math.inf
        if T > 4:
            x[4, E // 2] = math.inf
    return x


def chosen(x, topk):
    v, i = U.clean(x).topk(topk, 1)
    return torch.where(v > -math.inf, i, -1).int()


def loss_close(got, want, logits, T):
    # each p is off by its relative error, and the sum over rows by at most a step a row of a wave (128) and a workgroup
    rel = float(U.score_error(logits).max()) + 160 * 2.0 ** -24 if T else 0.0
    U.close(got, want, want.abs() * rel, "loss")


@pytest.mark.parametrize("T,E,topk,offsets,score,dtype,masked", [
    (1, 1, 1, None, "softmax", "fp32", False),
    (1, 384, 8, None, "sigmoid", "bf16", False),
    (32, 8, 2, None, "softmax", "fp32", True),
    (64, 20, 3, [5, 61], "sigmoid", "bf16", True),
    (50, 20, 3, [7, 7], "softmax", "fp32", False),
    (65, 20, 3, None, "softmax", "fp16", False),
    (33, 64, 6, None, "sigmoid", "fp16", True),
    (31, 65, 3, [0, 31], "softmax", "bf16", True),
    (300, 100, 4, [0, 0, 1, 1, 33, 200, 300, 300], "sigmoid", "fp32", True),
    (1000, 256, 8, [3, 64, 64, 900], "softmax", "fp16", False),
    (777, 255, 5, None, "softmax", "bf16", False),
    (2050, 384, 8, [0, 1025, 2050], "sigmoid", "bf16", True),
    (500, 511, 16, [10, 20, 480], "softmax", "fp32", False),
    (129, 1000, 64, None, "sigmoid", "fp16", True),
    (70, 1024, 7, [0, 70], "softmax", "bf16", False),
    (50, 4096, 33, [0, 7, 50], "softmax", "fp32", True),
    (16, 2000, 9, None, "softmax", "bf16", True),
    (31, 700, 9, None, "sigmoid", "fp32", True),
    (700, 1500, 9, [3, 9, 9, 400, 690], "softmax", "bf16", True),
    (40, 1026, 8, None, "sigmoid", "bf16", False),
    (40000, 16, 2, [0, 39999, 40000], "softmax", "bf16", False),
])
def test_balance(T, E, topk, offsets, score, dtype, masked):
    m = M()
    log(f"case balance T={T} E={E} topk={topk} {offsets} {score} {dtype} masked={masked}")
    x = logits_of(T, E, dtype, T + E, masked)
    ids = chosen(x, topk)
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32)
    xc, ic, oc = cuda(x, ids, off)
    loss, counts = m.router_balance(xc, ic, score=score, offsets=oc)
    want, n = U.balance(x, ids, score, off)
    assert torch.equal(counts.cpu(), n)
    loss_close(loss, want, x, T)
    S = n.shape[0]
    d_loss = torch.randn(S, generator=torch.Generator().manual_seed(1)) * T * E / S
    for add in (None, torch.randn(T, E, generator=torch.Generator().manual_seed(2)).to(DT[dtype])):
        d = m.router_balance_grad(xc, counts, d_loss.cuda(), topk, score=score, offsets=oc,
                                  add=None if add is None else add.cuda())
        exact, slack = U.balance_grad(x, n, d_loss, topk, score, off, add)
        U.close(d, exact, slack, "gradient")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_gradient_against_differences(score):
    """Of the loss itself, in 64 bits, by central differences over some logits."""
    m = M()
    x, topk = logits_of(40, 24, "fp32", 3), 4
    ids = chosen(x, topk)
    off = torch.tensor([0, 17, 17, 40], dtype=torch.int32)
    d_loss = torch.tensor([0.7, 2.0, -1.3])
    _, n = U.balance(x, ids, score, off)
    d = m.router_balance_grad(*cuda(x, n, d_loss), topk, score=score, offsets=off.cuda()).cpu().double()
    h = 1e-5
    for t, e in [(0, 0), (3, 7), (16, 23), (17, 1), (39, 11)]:
        v = []
        for sign in (1, -1):
            y = x.double()
            y[t, e] += sign * h
            v.append(float((U.balance(y, ids, score, off)[0] * d_loss.double()).sum()))
        diff = (v[0] - v[1]) / (2 * h)
        # third derivatives of p are below 1, so h^2 / 6 times d_loss's factor; rounding of FP64 over h; FP32's own
        assert abs(float(d[t, e]) - diff) <= 1e-9 + 1e-10 / h * 1e-3 + 2e-6 * float(d.abs().max())


def test_balance_far_negative_sigmoids_and_large_logits():
    """Rows whose sigmoids all underflow, and logits at the ends of FP32."""
    m = M()
    x = torch.randn(8, 16, generator=torch.Generator().manual_seed(4)) * 2
    x[0] -= 100
    x[1] -= 300
    x[2] = -torch.finfo(torch.float32).max
    x[3, 5] = torch.finfo(torch.float32).max
    x[4] = -61 + torch.arange(16) / 10
    x[5] += 80
    ids = chosen(x, 2)
    for score in ("sigmoid", "softmax"):
        loss, counts = m.router_balance(*cuda(x, ids), score=score)
        want, n = U.balance(x, ids, score, None)
        assert torch.equal(counts.cpu(), n)
        loss_close(loss, want, x, 8)
        d = m.router_balance_grad(x.cuda(), counts, torch.ones(1).cuda(), 2, score=score)
        exact, slack = U.balance_grad(x, n, torch.ones(1), 2, score, None)
        U.close(d, exact, slack, score)


def test_balance_strides_in_place_and_foreign_ids():
    m = M()
    wide = logits_of(200, 130, "bf16", 9)
    x = wide[:, 1:98]                      # rows 130 values apart, not on 4 bytes
    ids = chosen(x, 3)
    ids[5] = torch.tensor([97, -7, 1 << 30])   # outside [0, 97)
    loss, counts = m.router_balance(wide.cuda()[:, 1:98], ids.cuda())
    want, n = U.balance(x, ids, "softmax", None)
    assert torch.equal(counts.cpu(), n)
    loss_close(loss, want, x, 200)
    d_loss = torch.tensor([500.0])
    add = torch.randn(200, 99, generator=torch.Generator().manual_seed(1)).bfloat16()
    buf = add.cuda()
    got = m.router_balance_grad(wide.cuda()[:, 1:98], counts, d_loss.cuda(), 3, add=buf[:, 1:98], out=buf[:, 1:98])
    exact, slack = U.balance_grad(x, n, d_loss, 3, "softmax", None, add[:, 1:98])
    U.close(got, exact, slack, "in place")
    assert torch.equal(buf[:, 0].cpu(), add[:, 0]) and torch.equal(buf[:, 98].cpu(), add[:, 98])


def test_balance_without_tokens():
    m = M()
    x, ids = torch.empty(0, 12).cuda(), torch.empty(0, 2, dtype=torch.int32).cuda()
    for off in (None, torch.zeros(4, dtype=torch.int32).cuda()):
        loss, counts = m.router_balance(x, ids, offsets=off)
        assert (loss == 0).all() and (counts == 0).all()
        assert m.router_balance_grad(x, counts, torch.ones_like(loss), 2, offsets=off).shape == (0, 12)


# ---- a token's rows ------------------------------------------------------------------


@pytest.mark.parametrize("T,E,topk,H,block,lost,dtype,out_dtype", [
    (1, 384, 8, 7168, 16, 0.0, "bf16", "bf16"),
    (1, 1, 1, 8, 1, 0.0, "fp32", "fp32"),
    (5, 4, 4, 24, 16, 0.5, "fp16", "fp32"),
    (67, 8, 2, 256, 16, 0.3, "bf16", "fp16"),
    (130, 16, 9, 520, 1, 0.9, "fp32", "bf16"),
    (33, 6, 3, 1032, 128, 0.0, "fp16", "fp16"),
    (40, 70, 64, 2056, 16, 0.2, "bf16", "bf16"),
    (1100, 12, 3, 1096, 16, 0.4, "bf16", "bf16"),
    (9, 5, 2, 16384, 16, 0.0, "fp32", "fp32"),
    (3, 4, 1, 8200, 1, 1.0, "bf16", "bf16"),
])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(T, E, topk, H, block, lost, dtype, out_dtype, weighted):
    m = M()
    log(f"case combine T={T} E={E} topk={topk} H={H} block={block} lost={lost} {dtype} -> {out_dtype} w={weighted}")
    slots, src, off = U.routing(T, E, topk, block, T + H, lost, spare=5)
    R = src.shape[0]
    g = torch.Generator().manual_seed(H)
    y = torch.randn(R, H, generator=g).to(DT[dtype])
    y[off[-1]:] = math.nan                         # rows of none are not read
    pad = (src >= T * topk).nonzero()[:, 0]
    y[pad] = math.nan
    w = torch.randn(T, topk, generator=g) if weighted else None
    d_out = torch.randn(T, H, generator=g).to(DT[dtype])
    yc, sc, wc, dc, rc, oc = cuda(y, slots, w, d_out, src, off)

    live = slots >= 0
    rows = torch.where(live[..., None], y[slots.long().clamp(min=0)].double(), 0.0) if R else torch.zeros(T, topk, H).double()
    w64 = torch.where(live, torch.ones(T, topk) if w is None else w, 0.0).double()[..., None]
    out = m.combine(yc, sc, wc, out_dtype=DT[out_dtype])
    check(out, (rows * w64).sum(1), (rows * w64).abs().sum(1), topk, "out")

    held = torch.full((R, H), 3.0, dtype=DT[dtype]).cuda()
    dw0 = torch.full((T, topk), math.nan).cuda()
    dy, dw = m.combine_grad(dc, sc, y=yc, w=wc, row_src=rc, offsets=oc, out=(held, dw0))
    assert dy is held and dw is dw0
    exact = torch.zeros(R, H, dtype=torch.float64)
    exact[slots[live].long()] = (w64 * d_out.double()[:, None, :])[live]
    exact[off[-1]:] = 3.0                          # behind the last group: as it was
    U.close(dy, exact, exact.abs() * 2.0 ** -24, "d_y")
    prod = rows * d_out.double()[:, None, :]
    U.close(dw, prod.sum(2), prod.abs().sum(2) * (H + 1) * 2.0 ** -24, "d_w")

    # without y: the rows alone; without row_src: the padding stays as it was
    only, none = m.combine_grad(dc, sc, w=wc, out=(torch.full_like(held, 3.0), None))
    assert none is None
    exact[pad] = 3.0
    U.close(only, exact, exact.abs() * 2.0 ** -24, "d_y alone")
    # without offsets: every row
    whole, _ = m.combine_grad(dc, sc, w=wc, row_src=rc)
    exact[pad] = 0.0
    U.close(whole, exact, exact.abs() * 2.0 ** -24, "all rows")


def test_combine_strides_and_guards():
    m = M()
    slots, src, off = U.routing(50, 6, 3, 16, 1)
    R, H = src.shape[0], 200
    g = torch.Generator().manual_seed(1)
    y = torch.randn(R, 256, generator=g).bfloat16().cuda()
    d = torch.randn(50, 208, generator=g).bfloat16().cuda()
    out = torch.full((50, 216), 7.0, dtype=torch.bfloat16, device="cuda")
    m.combine(y[:, 8:208], slots.cuda(), out=out[:, 8:208])
    want = m.combine(y[:, 8:208].contiguous(), slots.cuda())
    assert torch.equal(out[:, 8:208], want) and (out[:, :8] == 7).all() and (out[:, 208:] == 7).all()
    dy = torch.full((R, 216), 7.0, dtype=torch.bfloat16, device="cuda")
    _, dw = m.combine_grad(d[:, :200], slots.cuda(), y=y[:, 8:208], row_src=src.cuda(), offsets=off.cuda(),
                           out=(dy[:, 8:208], None))
    a, b = m.combine_grad(d[:, :200].contiguous(), slots.cuda(), y=y[:, 8:208].contiguous(), row_src=src.cuda(),
                          offsets=off.cuda())
    assert torch.equal(dy[:, 8:208], a) and torch.equal(dw, b)
    assert (dy[:, :8] == 7).all() and (dy[:, 208:] == 7).all()


def test_combine_of_nothing():
    m = M()
    y = torch.empty(0, 64, device="cuda")
    slots = torch.full((3, 2), 5, dtype=torch.int32, device="cuda")      # past R = 0
    assert (m.combine(y, slots, torch.ones(3, 2, device="cuda")) == 0).all()
    dy, dw = m.combine_grad(torch.ones(3, 64, device="cuda"), slots, y=y)
    assert dy.shape == (0, 64) and (dw == 0).all()
    none = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    assert m.combine(torch.ones(4, 64, device="cuda"), none).shape == (0, 64)
    dy, _ = m.combine_grad(torch.empty(0, 64, device="cuda"), none, row_src=torch.zeros(70, dtype=torch.int32, device="cuda"))
    assert (dy == 0).all()


# ---- rows in 8 bits --------------------------------------------------------------------


def rows_of(dtype, rows, K, seed):
    g = torch.Generator().manual_seed(seed)
    e = torch.randint(-10, 11, (rows, (K + 31) // 32), generator=g).float()
    return (torch.randn(rows, K, generator=g) * torch.exp2(e).repeat_interleave(32, 1)[:, :K] / 8).to(DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,K", [(1, 8), (1, 32), (3, 40), (7, 536), (65, 24), (130, 1032), (257, 7168), (1030, 16)])
def test_mx8(dtype, rows, K):
    m = M()
    log(f"case mx8 {dtype} rows={rows} K={K}")
    x = rows_of(dtype, rows, K, rows + K)
    q, s = m.mx8_quant(x.cuda())
    val, code, byte = U.mx8(x)
    n = (K + 31) // 32
    assert s.shape == (rows, m.mx8_scale_cols(K))
    assert torch.equal(s[:, :n].cpu(), byte) and (s[:, n:] == 0).all()
    assert torch.equal(q.cpu(), code)
    for out in ("bf16", "fp16", "fp32"):
        assert torch.equal(m.mx8_dequant(q, s, dtype=DT[out]).cpu(), val.to(DT[out]))
    # the block's largest loses at most a step of a 64th, the others half of it
    top = torch.nn.functional.pad(x.double(), (0, -K % 32)).view(rows, n, 32).abs().amax(2).repeat_interleave(32, 1)[:, :K]
    assert ((val - x.double()).abs() <= top / 64).all()


def test_mx8_borders_and_special_values():
    m = M()
    half = torch.arange(-128, 128).float() + 0.5
    x = torch.stack([torch.cat([t[:31], torch.tensor([64.0])]) * 2.0 ** e
                     for e in (0, -40, 40, -130, -138, 100, 120) for t in (half[:31], half[40:80], half[112:160], half[-40:])])
    x = torch.cat([x, torch.zeros(1, 32), torch.full((1, 32), -0.0), torch.full((1, 32), 2.0 ** -149),
                   torch.full((1, 32), torch.finfo(torch.float32).max), -torch.full((1, 32), 2.0 ** -126),
                   torch.full((1, 32), 2.0 ** -126 - 2.0 ** -149), torch.full((1, 32), 127.5), torch.full((1, 32), -127.99)])
    x[5, 31] = 127.9
    q, s = m.mx8_quant(x.cuda())
    val, code, byte = U.mx8(x)
    assert torch.equal(s[:, :1].cpu(), byte) and torch.equal(q.cpu(), code)
    assert torch.equal(m.mx8_dequant(q, s, dtype=torch.float32).cpu().double(), val)
    bad = rows_of("bf16", 4, 72, 3)
    bad[0, 40], bad[1, 0], bad[2, 71] = math.nan, math.inf, -math.inf
    q, s = m.mx8_quant(bad.cuda())
    val, code, byte = U.mx8(bad)
    assert torch.equal(s[:, :3].cpu(), byte) and torch.equal(q.cpu(), code)
    got = m.mx8_dequant(q, s, dtype=torch.float32).cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(val)) and torch.equal(got.nan_to_num(), val.nan_to_num())


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,topk,K", [(1, 8, 7168), (37, 3, 40), (200, 2, 1000)])
def test_mx8_as_the_rows_of_a_routing(dtype, T, topk, K):
    m = M()
    slots, src, off = U.routing(T, 9, topk, 16, T, 0.2, spare=7)
    src[0 if off[-1] == 0 else int(off[-1]) - 1] = -1           # as good as the sentinel
    x = rows_of(dtype, T, K, T + K)
    q, s = m.mx8_quant(x.cuda())
    val = U.mx8(x)[0].to(DT[dtype])
    out = torch.full((src.shape[0], K), 3.0, dtype=DT[dtype], device="cuda")
    m.mx8_dequant(q, s, row_src=src.cuda(), topk=topk, offsets=off.cuda(), out=out)
    want = torch.where(((src >= 0) & (src < T * topk))[:, None], val[(src.long() // topk).clamp(0, T - 1)],
                       torch.zeros((), dtype=DT[dtype]))
    want[off[-1]:] = 3.0
    assert torch.equal(out.cpu(), want)
    # the same row many times, all rows
    again = m.mx8_dequant(q, s, dtype=DT[dtype], row_src=torch.zeros(70, dtype=torch.int32, device="cuda"))
    assert torch.equal(again.cpu(), val[:1].expand(70, K))


def test_mx8_strides_and_guards():
    m = M()
    wide = rows_of("bf16", 40, 160, 1).cuda()
    x = wide[:, 8:152]
    q, s = m.mx8_quant(x)
    q2, s2 = m.mx8_quant(x.contiguous())
    assert torch.equal(q, q2) and torch.equal(s, s2)
    out = torch.full((40, 160), 3.0, dtype=torch.bfloat16, device="cuda")
    m.mx8_dequant(q, s, out=out[:, 8:152])
    assert torch.equal(out[:, 8:152], m.mx8_dequant(q, s)) and (out[:, :8] == 3).all() and (out[:, 152:] == 3).all()
    assert m.mx8_quant(torch.empty(0, 64, device="cuda"))[0].shape == (0, 64)


# ---- SwiGLU ----------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,I,live", [(1, 8, None), (3, 32, None), (70, 40, [5, 20, 61]), (33, 1024, [0, 33]),
                                         (129, 520, [0, 0]), (300, 256, [17, 17, 300])])
def test_swiglu(dtype, rows, I, live):
    m = M()
    log(f"case swiglu {dtype} rows={rows} I={I} live={live}")
    h = rows_of(dtype, rows, 2 * I, rows + I).clamp(-60, 60)
    d_a = torch.randn(rows, I, generator=torch.Generator().manual_seed(I)).to(DT[dtype])
    lo, hi = (0, rows) if live is None else (live[0], live[-1])
    off = None if live is None else torch.tensor(live, dtype=torch.int32).cuda()
    dead = torch.ones(rows, dtype=torch.bool)
    dead[lo:hi] = False
    hn = torch.where(dead[:, None], math.nan, h.float()).to(DT[dtype])           # not read
    cols = m.mx8_scale_cols(I)
    fresh = (torch.full((rows, I), 3.0, dtype=DT[dtype], device="cuda"),
             torch.full((rows, 2, I), 3, dtype=torch.int8, device="cuda"),
             torch.full((rows, 2, cols), 3, dtype=torch.uint8, device="cuda"))
    a, q, s = m.swiglu_save(hn.cuda(), offsets=off, out=fresh)
    U.close(a[lo:hi], U.swiglu(h)[lo:hi], U.swiglu_slack(h)[lo:hi], "a")
    q2, s2 = m.mx8_quant(h.cuda().view(2 * rows, I))
    assert torch.equal(q[lo:hi], q2.view(rows, 2, I)[lo:hi]) and torch.equal(s[lo:hi], s2.view(rows, 2, cols)[lo:hi])
    for t in (a, q, s):
        assert (t[:lo] == 3).all() and (t[hi:] == 3).all()

    kept = U.mx8(h.reshape(2 * rows, I))[0].reshape(rows, 2 * I)
    for values, args in ((kept, dict(h=q, scales=s)), (h.double(), dict(h=hn.cuda()))):
        out = (torch.full((rows, 2 * I), 3.0, dtype=DT[dtype], device="cuda"),
               torch.full((rows, I), 3.0, dtype=DT[dtype], device="cuda"))
        d_h, a2 = m.swiglu_grad(d_a=d_a.cuda(), offsets=off, out=out, **args)
        exact, slack = U.swiglu_grad(values, d_a)
        U.close(d_h[lo:hi], exact[lo:hi], slack[lo:hi], "d_h")
        U.close(a2[lo:hi], U.swiglu(values)[lo:hi], U.swiglu_slack(values)[lo:hi], "a again")
        for t in (d_h, a2):
            assert (t[:lo] == 3).all() and (t[hi:] == 3).all()
        alone, none = m.swiglu_grad(d_a=d_a.cuda(), offsets=off, need_a=False, **args)
        assert none is None and torch.equal(alone[lo:hi], d_h[lo:hi])


def test_swiglu_gradient_against_differences():
    m = M()
    g = torch.Generator().manual_seed(2)
    h, d_a = torch.randn(4, 32, generator=g) * 3, torch.randn(4, 16, generator=g)
    d = m.swiglu_grad(h.cuda(), d_a.cuda())[0].cpu().double()
    step = 1e-4
    for r, c in [(0, 0), (1, 5), (2, 15), (3, 16), (0, 31), (2, 20)]:
        v = []
        for sign in (1, -1):
            y = h.double()
            y[r, c] += sign * step
            v.append(float((U.swiglu(y) * d_a.double()).sum()))
        # central differences: step^2 / 6 times the third derivative (below 1 times |d u|), and FP32's own error
        size = float(d_a.abs().max() * h.abs().max())
        assert abs(float(d[r, c]) - (v[0] - v[1]) / (2 * step)) <= size * (step ** 2 + 60 * 2.0 ** -23)


def test_swiglu_far_gates():
    """Gates whose exponentials end FP32."""
    m = M()
    g = torch.tensor([-1e4, -200, -104, -89, -88, -20, -1e-30, 0.0, 1e-30, 20, 88, 104, 200, 1e4, 3e38, -3e38]).repeat(2)
    h = torch.cat([g, torch.linspace(-2, 2, 32)])[None]
    d_a = torch.linspace(1, 2, 32)[None]
    a, q, s = m.swiglu_save(h.cuda())
    d_h, a2 = m.swiglu_grad(h.cuda(), d_a.cuda())
    exact, slack = U.swiglu_grad(h, d_a)
    f = torch.isfinite(exact) & (exact.abs() < 3e38)
    U.close(d_h.cpu()[f], exact[f], slack[f], "d_h")
    want = U.swiglu(h)
    f = want.abs() < 3e38
    U.close(a.cpu()[f], want[f], U.swiglu_slack(h)[f], "a")
    assert torch.equal(a, a2)


def test_swiglu_strides():
    m = M()
    h = rows_of("bf16", 30, 240, 1).cuda()
    d_a = rows_of("bf16", 30, 112, 2).cuda()
    a, q, s = m.swiglu_save(h[:, 8:200])
    b = m.swiglu_save(h[:, 8:200].contiguous())
    assert all(torch.equal(x, y) for x, y in zip((a, q, s), b))
    out = torch.full((30, 208), 3.0, dtype=torch.bfloat16, device="cuda")
    d_h, a2 = m.swiglu_grad(h[:, 8:200], d_a[:, 8:104], out=(out[:, 8:200], None))
    want, _ = m.swiglu_grad(h[:, 8:200].contiguous(), d_a[:, 8:104].contiguous())
    assert a2 is None and torch.equal(d_h, want) and (out[:, :8] == 3).all() and (out[:, 200:] == 3).all()
