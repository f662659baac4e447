"""The operators where memory is far apart (offsets past 32 bits), captured in
a row and replayed, and run on two streams at once. Results are compared bit
for bit with the same operators on dense tensors, eager, one at a time."""
import pytest
import torch

from tests.gpu_util import log, require_gpu
from tests.ops_util import offsets_of
from tests.test_gpu_l_grouped import run
from tests.test_gpu_n_operators import routed, tiny_handle

pytestmark = pytest.mark.gpu

FAR = 1 << 21          # the largest distance of rows


def apart(t, stride):
    """t's values in rows (and experts) `stride` values apart."""
    size = 1 + sum((n - 1) * s for n, s in zip(t.shape, stride))
    v = torch.empty(size, dtype=t.dtype, device="cuda").as_strided(t.shape, stride)
    return v.copy_(t)


@pytest.mark.parametrize("way", ["fwd", "dgrad", "wgrad"])
def test_products_of_rows_far_apart(way):
    require_gpu()
    import w4a16_int4_grouped_amd as M
    log(f"case far apart {way}")
    counts, N, K = [700, 0, 500], 72, 136
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    dy, a, w = r(1200, N), r(1200, K), r(3, N, K)
    off = offsets_of(counts).cuda()
    want = run(M, way, dy, a, w, off)
    experts = ((1 << 31) + 8, FAR, 1)                   # the last expert begins 8 GiB on, the last row 4.7 GiB
    far = (apart(dy, (FAR, 1)) if way != "fwd" else dy, apart(a, (FAR, 1)) if way != "dgrad" else a,
           apart(w, experts) if way != "wgrad" else w)
    out = apart(torch.full_like(want, 7), experts if way == "wgrad" else (FAR, 1))
    run(M, way, *far, off, out=out)
    assert torch.equal(out, want)


def test_router_rows_far_apart():
    require_gpu()
    import w4a16_int4_grouped_amd as M
    logits = torch.randn(600, 72, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    far = apart(logits, (1 << 23, 1))
    ids, w = M.router_topk(logits, 5, renorm=True)
    for x, y in zip(M.router_topk(far, 5, renorm=True), (ids, w)):
        assert torch.equal(x, y)
    want = M.router_topk_grad(logits, ids, w, renorm=True)
    out = apart(torch.full_like(want, 7), (1 << 23, 1))
    M.router_topk_grad(far, ids, w, renorm=True, out=out)
    assert torch.equal(out, want)


def test_mxfp4_rows_past_32_bits():
    """1048581 x 8224: 17 GB of values, 4.3 GB of codes. Integers that FP4
    holds, so that every product is exact."""
    require_gpu()
    import w4a16_int4_grouped_amd as M
    rows, K, N = (1 << 20) + 5, 8224, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randint(-3, 4, s, generator=g, device="cuda", dtype=torch.int8).bfloat16()  # noqa: E731
    log("case MXFP4 past 32 bits")
    x, w = r(rows, K), r(2, N, K)
    q, scales = M.mx_quant(x)
    parts = [slice(0, 9), slice(rows // 2 - 4, rows // 2 + 5), slice(rows - 9, rows)]
    for p in parts:
        for got, want in zip((q[p], scales[p]), M.mx_quant(x[p])):
            assert torch.equal(got, want)
    back = M.mx_dequant(q, scales)
    for p in parts:
        assert torch.equal(back[p], x[p])
    del back
    wq = M.mx_quant(w)
    out = M.mx_grouped_gemm(q, scales, *wq, offsets_of([rows - 4, 4]).cuda(), out_dtype=torch.float32)
    wd = w.cpu().double()
    for p in parts:
        xd = x[p].cpu().double()
        e = (torch.arange(rows)[p] >= rows - 4).long()
        want = torch.stack([xd, xd], 0) @ wd.transpose(1, 2)
        assert torch.equal(out[p].cpu().double(), want[e, torch.arange(len(e))])


def layer(M, h, x, logits, w1, w2, w2q, topk, d_w):
    """Router to the last product, BF16 then MXFP4, and the router's gradient;
    what a token needs of each."""
    ids, tw, a, off, slots = routed(M, h, x, logits, topk)
    act = M.swiglu(M.grouped_gemm(a, w1, off))
    y = M.grouped_gemm(act, w2, off)
    ymx = M.mx_grouped_gemm(*M.mx_quant(act), *w2q, off)
    return ids, tw, y[slots], ymx[slots], M.router_topk_grad(logits, ids, d_w, renorm=True)


def case(M, seed, T=75, E=16, H=256, I=128, topk=4):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    w2 = (r(E, H, I) * I ** -0.5).bfloat16()
    return [r(T, H).bfloat16(), r(T, E), (r(E, 2 * I, H) * H ** -0.5).bfloat16(), w2, M.mx_quant(w2), topk, r(T, topk)]


def test_two_captured_rows_of_operators():
    require_gpu()
    import w4a16_int4_grouped_amd as M
    h = tiny_handle(16, 256, 128)
    cases = [case(M, 1), case(M, 2, T=9)]
    graphs, outs = [], []
    for c in cases:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            layer(M, h, *c)
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(layer(M, h, *c))
        graphs.append(g)
    for k in range(4):
        for c in cases:
            c[0].neg_()
            c[1].copy_(c[1].roll(k + 1, 1))
        torch.cuda.synchronize()
        for g in graphs if k % 2 else graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        for c, got in zip(cases, outs):
            for i, (x, y) in enumerate(zip(got, layer(M, h, *c))):
                assert torch.equal(x, y), (k, i)


def test_two_streams_at_once():
    require_gpu()
    import w4a16_int4_grouped_amd as M
    h = tiny_handle(16, 256, 128)
    cases = [case(M, 3, T=700), case(M, 4, T=130)]
    want = [layer(M, h, *c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for k in range(6):
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                got.append(layer(M, h, *c))
    torch.cuda.synchronize()
    for k, one in enumerate(got):
        for x, y in zip(one, want[k % 2]):
            assert torch.equal(x, y), k
