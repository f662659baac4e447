"""Grouped products over ragged rows and their gradients against 64-bit
references, at the sizes where tiles, steps and groups end."""
import pytest
import torch

from tests.gpu_util import log, require_gpu
from tests.ops_util import check, groups, offsets_of, random_counts

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}

SHAPES = [
    # E, N, K, counts
    (1, 8, 8, [1]),
    (3, 8, 16, [0, 5, 0]),
    (4, 136, 72, [1, 0, 127, 130]),
    (2, 264, 200, [128, 129]),
    (3, 256, 128, [256, 0, 64]),
    (5, 40, 1032, [15, 16, 17, 33, 64]),
    (2, 520, 320, [300, 513]),
    (70, 72, 88, "random"),
    (130, 264, 64, "random"),
]


def counts_of(E, counts):
    return random_counts(E, 3 * E + 7, E) if counts == "random" else counts


def reference(way, dy, a, w, counts, start=0):
    """The exact product and sum |q p|, in 64 bits on the CPU."""
    E = len(counts)
    if way == "wgrad":
        out = torch.zeros(E, dy.shape[1], a.shape[1], dtype=torch.float64)
    else:
        out = torch.zeros((a if way == "fwd" else dy).shape[0], w.shape[1] if way == "fwd" else w.shape[2],
                          dtype=torch.float64)
    mag = out.clone()
    for e, lo, hi in groups(counts, start):
        for dst, f in ((out, lambda t: t.double()), (mag, lambda t: t.double().abs())):
            if way == "fwd":
                dst[lo:hi] = f(a[lo:hi]) @ f(w[e]).T
            elif way == "dgrad":
                dst[lo:hi] = f(dy[lo:hi]) @ f(w[e])
            else:
                dst[e] = f(dy[lo:hi]).T @ f(a[lo:hi])
    return out, mag


def run(M, way, dy, a, w, off, **kw):
    if way == "fwd":
        return M.grouped_gemm(a, w, off, **kw)
    if way == "dgrad":
        return M.grouped_gemm_dgrad(dy, w, off, **kw)
    return M.grouped_gemm_wgrad(dy, a, off, **kw)


def inputs(E, N, K, rows, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(DT[dtype])  # noqa: E731
    return r(rows, N), r(rows, K), r(E, N, K)


@pytest.mark.parametrize("way", ["fwd", "dgrad", "wgrad"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("E,N,K,counts", SHAPES)
def test_products(way, dtype, E, N, K, counts):
    require_gpu()
    import w4a16_int4_grouped_amd as M
    counts = counts_of(E, counts)
    rows = sum(counts)
    log(f"case grouped {way} {dtype} E={E} N={N} K={K} rows={rows}")
    dy, a, w = inputs(E, N, K, rows, dtype, E + N + K)
    off = offsets_of(counts).cuda()
    ref, mag = reference(way, dy, a, w, counts)
    C = {"fwd": K, "dgrad": N, "wgrad": max(counts)}[way]
    for out_dtype in (DT[dtype], torch.float32):
        got = run(M, way, dy.cuda(), a.cuda(), w.cuda(), off, out_dtype=out_dtype)
        assert got.dtype == out_dtype
        check(got, ref, mag, C, f"{way} -> {out_dtype}")


@pytest.mark.parametrize("way", ["fwd", "dgrad", "wgrad"])
@pytest.mark.parametrize("E,N,K,counts", [(3, 392, 264, [130, 0, 300]), (40, 136, 584, "random"),
                                          (2, 776, 264, [700, 37]), (64, 520, 72, "random")])
def test_small_integers_are_exact(way, E, N, K, counts):
    """Integers of at most 3: every FP32 sum is exact, so any error is an indexing error."""
    require_gpu()
    import w4a16_int4_grouped_amd as M
    counts = counts_of(E, counts)
    rows = sum(counts)
    g = torch.Generator().manual_seed(N)
    r = lambda *s: torch.randint(-3, 4, s, generator=g).to(torch.bfloat16)  # noqa: E731
    dy, a, w = r(rows, N), r(rows, K), r(E, N, K)
    ref, _ = reference(way, dy, a, w, counts)
    got = run(M, way, dy.cuda(), a.cuda(), w.cuda(), offsets_of(counts).cuda(), out_dtype=torch.float32)
    assert torch.equal(got.double().cpu(), ref)


@pytest.mark.parametrize("way", ["fwd", "dgrad", "wgrad"])
@pytest.mark.parametrize("counts", [[3, 0, 20], [129, 1, 200], [40, 300, 0]])
def test_strides_guards_and_rows_of_no_group(way, counts):
    """Rows apart, NaN in every value that belongs to no product (columns between the rows, rows before the first
    group and behind the last, experts' gaps), canaries around the output."""
    require_gpu()
    import w4a16_int4_grouped_amd as M
    E, N, K, start, behind = 3, 136, 200, 5, 9
    rows = start + sum(counts) + behind
    nan = float("nan")

    def wide(x, pad):
        t = torch.full((x.shape[0], x.shape[1] + pad), nan, dtype=x.dtype, device="cuda")
        t[:, : x.shape[1]] = x.cuda()
        return t[:, : x.shape[1]]
    dy, a, w = inputs(E, N, K, rows, "bf16", 11)
    for t in (dy, a):
        t[:start] = nan
        t[rows - behind:] = nan
    wpad = torch.full((E, N + 3, K + 24), nan, dtype=w.dtype, device="cuda")
    wpad[:, :N, :K] = w.cuda()
    off = offsets_of(counts, start).cuda()
    ref, mag = reference(way, dy, a, w, counts, start)
    if way == "wgrad":
        whole = torch.full((E, N + 1, K + 8), 7.0, device="cuda")
        out = whole[:, :N, :K]
    else:
        whole = torch.full((rows, ref.shape[1] + 8), 7.0, device="cuda")
        out = whole[:, : ref.shape[1]]
    log(f"case grouped guards {way} {counts}")
    run(M, way, wide(dy, 16), wide(a, 8), wpad[:, :N, :K], off, out=out)
    torch.cuda.synchronize()
    C = max(K, N, *counts)
    if way == "wgrad":
        check(out, ref, mag, C, way)
        assert (whole[:, N:] == 7.0).all() and (whole[:, :, K:] == 7.0).all()
    else:
        live = slice(start, rows - behind)
        check(out[live], ref[live], mag[live], C, way)
        assert (whole[:start] == 7.0).all() and (whole[rows - behind:] == 7.0).all()
        assert (whole[:, ref.shape[1]:] == 7.0).all()


def test_nan_and_infinity_stay_in_their_rows():
    require_gpu()
    import w4a16_int4_grouped_amd as M
    counts = [20, 150]
    dy, a, w = inputs(2, 72, 136, 170, "bf16", 2)
    a[3, 7], a[30, 0] = float("nan"), float("inf")
    off = offsets_of(counts).cuda()
    y = M.grouped_gemm(a.cuda(), w.cuda(), off).cpu()
    bad = ~torch.isfinite(y).all(1)
    assert bad.nonzero().flatten().tolist() == [3, 30]
    d = M.grouped_gemm_wgrad(dy.cuda(), a.cuda(), off).cpu()
    assert (~torch.isfinite(d)).nonzero()[:, [0, 2]].unique(dim=0).tolist() == [[0, 7], [1, 0]]


def test_one_row_and_no_rows():
    require_gpu()
    import w4a16_int4_grouped_amd as M
    dy, a, w = (t.cuda() for t in inputs(4, 64, 64, 1, "fp16", 4))
    off = torch.tensor([0, 0, 0, 1, 1], dtype=torch.int32, device="cuda")
    assert torch.allclose(M.grouped_gemm(a, w, off).float(), a.float() @ w[2].float().T, rtol=2e-3, atol=2e-3)
    none = torch.zeros(5, dtype=torch.int32, device="cuda")
    out = torch.full((1, 64), 3.0, dtype=torch.float16, device="cuda")
    assert (M.grouped_gemm(a, w, none, out=out) == 3.0).all()
    assert (M.grouped_gemm_wgrad(dy, a, none) == 0).all()
    assert M.grouped_gemm(a[:0], w, none).shape == (0, 64)
    assert (M.grouped_gemm_wgrad(dy[:0], a[:0], none) == 0).all()


def test_one_weight_matrix_for_all_experts():
    """A broadcast weight (expert stride 0) in the product and its input gradient."""
    require_gpu()
    import w4a16_int4_grouped_amd as M
    dy, a, w = (t.cuda() for t in inputs(1, 72, 64, 50, "bf16", 6))
    off = offsets_of([10, 0, 40]).cuda()
    whole = torch.tensor([0, 50], dtype=torch.int32, device="cuda")
    assert torch.equal(M.grouped_gemm(a, w.expand(3, -1, -1), off), M.grouped_gemm(a, w, whole))
    assert torch.equal(M.grouped_gemm_dgrad(dy, w.expand(3, -1, -1), off), M.grouped_gemm_dgrad(dy, w, whole))


def test_offsets_outside_the_rows_are_clamped():
    require_gpu()
    import w4a16_int4_grouped_amd as M
    dy, a, w = (t.cuda() for t in inputs(2, 64, 64, 40, "bf16", 6))
    good = torch.tensor([0, 30, 40], dtype=torch.int32, device="cuda")
    bad = torch.tensor([-5, 30, 1 << 30], dtype=torch.int32, device="cuda")
    assert torch.equal(M.grouped_gemm(a, w, good), M.grouped_gemm(a, w, bad))
    assert torch.equal(M.grouped_gemm_wgrad(dy, a, good), M.grouped_gemm_wgrad(dy, a, bad))


def test_gradients_against_differences():
    """sum(dy . y) differs along one changed value by its gradient; products of small integers are exact, so the
    difference is too."""
    require_gpu()
    import w4a16_int4_grouped_amd as M
    g = torch.Generator().manual_seed(8)
    r = lambda *s: torch.randint(-3, 4, s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    counts = [7, 0, 21]
    dy, a, w = r(28, 40), r(28, 48), r(3, 40, 48)
    off = offsets_of(counts).cuda()
    f = lambda a, w: (M.grouped_gemm(a, w, off, out_dtype=torch.float32).double() * dy.double()).sum()  # noqa: E731
    da = M.grouped_gemm_dgrad(dy, w, off, out_dtype=torch.float32)
    dw = M.grouped_gemm_wgrad(dy, a, off, out_dtype=torch.float32)
    base = f(a, w)
    for r_, c in ((0, 0), (6, 47), (7, 3), (27, 31)):
        b = a.clone()
        b[r_, c] += 1
        assert float(f(b, w) - base) == float(da[r_, c])
    for e, n, k in ((0, 0, 0), (0, 39, 47), (1, 5, 5), (2, 17, 30)):
        b = w.clone()
        b[e, n, k] += 1
        assert float(f(a, b) - base) == float(dw[e, n, k])


def test_repeated_calls_streams_and_graph_replays():
    require_gpu()
    import w4a16_int4_grouped_amd as M
    counts = [5, 200, 0, 31]
    dy, a, w = (t.cuda() for t in inputs(4, 136, 264, sum(counts), "bf16", 9))
    off = offsets_of(counts).cuda()
    want = [run(M, way, dy, a, w, off) for way in ("fwd", "dgrad", "wgrad")]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = [run(M, way, dy, a, w, off, stream=s) for way in ("fwd", "dgrad", "wgrad")]
    s.synchronize()
    for x, y in zip(want, other):
        assert torch.equal(x, y)
    outs = [torch.empty_like(x) for x in want]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for way, o in zip(("fwd", "dgrad", "wgrad"), outs):
            run(M, way, dy, a, w, off, out=o)
    for k in range(4):
        moved = offsets_of(counts[k:] + counts[:k])
        off.copy_(moved)
        a.neg_()
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for way, o in zip(("fwd", "dgrad", "wgrad"), outs):
            assert torch.equal(o, run(M, way, dy, a, w, off)), (k, way)


@pytest.mark.parametrize("way,E,N,K,rows", [("fwd", 8, 512, 2048, 1500), ("dgrad", 8, 2048, 512, 1500),
                                            ("wgrad", 4, 512, 768, 3000), ("fwd", 48, 1024, 7168, 448),
                                            ("fwd", 6, 768, 1024, 4000), ("dgrad", 40, 640, 512, 300)])
def test_larger_products(way, E, N, K, rows):
    """Against FP64 products of the same inputs on the GPU."""
    require_gpu()
    import w4a16_int4_grouped_amd as M
    counts = random_counts(E, rows, 17)
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    dy, a, w = r(rows, N), r(rows, K), r(E, N, K)
    log(f"case grouped large {way} E={E} N={N} K={K} rows={rows}")
    got = run(M, way, dy, a, w, offsets_of(counts).cuda())
    ref, mag = reference(way, dy, a, w, counts)
    check(got, ref, mag, {"fwd": K, "dgrad": N, "wgrad": max(counts)}[way], way)
