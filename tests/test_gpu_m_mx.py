"""MXFP4: quantisation bit for bit against 64 bits, the scaled product
against 64 bits, blocks that hold NaN, infinities, zeros and subnormals."""
import pytest
import torch

from tests.gpu_util import log, require_gpu
from tests.ops_util import check, groups, mx_reference, mx_values, offsets_of, random_counts

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def rows_of(dtype, rows, K, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, K, generator=g) * torch.exp2(torch.randint(-10, 11, (rows, K // 32), generator=g).float()
                                                       ).repeat_interleave(32, 1)
    return x.to(DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 64), (7, 544), (65, 512), (130, 1056), (257, 7168)])
def test_quant_and_dequant(dtype, rows, K):
    require_gpu()
    import w4a16_int4_grouped_amd as M
    log(f"case mx quant {dtype} rows={rows} K={K}")
    x = rows_of(dtype, rows, K, rows + K)
    q, s = M.mx_quant(x.cuda())
    val, byte = mx_reference(x)
    assert q.shape == (rows, K // 2) and s.shape == (rows, M.mx_scale_cols(K))
    assert torch.equal(s[:, : K // 32].cpu(), byte)
    assert (s[:, K // 32:] == 0).all()
    assert torch.equal(mx_values(q.cpu(), s.cpu()), val)
    for out in ("bf16", "fp16", "fp32"):
        # e2m1 has 2 significant bits: exact in every type unless its exponents end (then rounded once)
        assert torch.equal(M.mx_dequant(q, s, dtype=DT[out]).cpu(), val.to(DT[out]))


def test_borders_and_ties():
    """Every tie and its neighbours, under scales from the smallest to the largest."""
    require_gpu()
    import w4a16_int4_grouped_amd as M
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0])
    near = torch.cat([ties, torch.nextafter(ties, ties * 0), torch.nextafter(ties, ties * 2)])
    near = torch.cat([near, -near[:4], torch.zeros(1)])
    assert near.numel() == 32
    near[torch.argmax(near.abs())] = 7.9
    x = torch.stack([near * 2.0 ** e for e in (0, -20, 40, -100, -120, -126, 120, 124, 125)])
    x = torch.cat([x, torch.zeros(1, 32), torch.full((1, 32), 2.0 ** -149), torch.full((1, 32), -0.0),
                   torch.full((1, 32), torch.finfo(torch.float32).max)])
    q, s = M.mx_quant(x.cuda())
    val, byte = mx_reference(x)
    assert torch.equal(s[:, :1].cpu(), byte)
    assert torch.equal(mx_values(q.cpu(), s.cpu()), val)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_nan_and_infinity_blocks(dtype):
    require_gpu()
    import w4a16_int4_grouped_amd as M
    x = rows_of(dtype, 4, 96, 3)
    x[0, 40], x[1, 0], x[2, 95] = float("nan"), float("inf"), -float("inf")
    q, s = M.mx_quant(x.cuda())
    _, byte = mx_reference(x)
    assert torch.equal(s[:, :3].cpu(), byte)
    v = M.mx_dequant(q, s, dtype=torch.float32).cpu()
    bad = torch.zeros(4, 3, dtype=torch.bool)
    bad[0, 1] = bad[1, 0] = bad[2, 2] = True
    assert torch.equal(torch.isnan(v), bad.repeat_interleave(32, 1))
    # and such a block makes its row of a product NaN, no other
    wq, ws = M.mx_quant(rows_of("bf16", 24, 96, 5).cuda())
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    y = M.mx_grouped_gemm(q, s, wq[None], ws[None], off)
    assert torch.equal(torch.isnan(y).all(1).cpu(), torch.tensor([True, True, True, False]))
    assert torch.isfinite(y[3]).all()


def test_strided_rows_guards_and_dimensions():
    require_gpu()
    import w4a16_int4_grouped_amd as M
    x = rows_of("bf16", 9, 160, 4)
    wide = torch.full((9, 200), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:168] = x.cuda()
    q = torch.full((10, 80), 99, dtype=torch.uint8, device="cuda")
    s = torch.full((10, 16), 99, dtype=torch.uint8, device="cuda")
    M.mx_quant(wide[:, 8:168], out=(q[:9], s[:9]))
    q2, s2 = M.mx_quant(x.cuda())
    assert torch.equal(q[:9], q2) and torch.equal(s[:9], s2)
    assert (q[9] == 99).all() and (s[9] == 99).all()
    out = torch.full((10, 176), 3.0, device="cuda")
    M.mx_dequant(q2, s2, out=out[:9, :160])
    assert torch.equal(out[:9, :160], M.mx_dequant(q2, s2, dtype=torch.float32))
    assert (out[9] == 3.0).all() and (out[:, 160:] == 3.0).all()
    q3, s3 = M.mx_quant(x.cuda().reshape(3, 3, 160))
    assert torch.equal(q3.reshape(9, 80), q2) and torch.equal(s3.reshape(9, 16), s2)
    e, t = M.mx_quant(x[:0].cuda())
    assert e.shape == (0, 80) and M.mx_dequant(e, t).shape == (0, 160)


SHAPES = [
    # E, N, K, counts
    (1, 8, 32, [1]),
    (3, 24, 96, [0, 5, 0]),
    (4, 136, 224, [1, 0, 127, 130]),
    (2, 264, 512, [128, 129]),
    (3, 256, 288, [256, 0, 64]),
    (5, 40, 1056, [15, 16, 17, 33, 64]),
    (2, 520, 736, [300, 513]),
    (70, 72, 352, "random"),
    (40, 1024, 2048, "random"),
]


def operands(E, N, K, rows, seed):
    """Random codes and scales of 2^-2 .. 2^1: products are multiples of 2^-6 of either sign and at most 144, whose FP32
    sums over these lengths stay exact (below 2^24 such steps)."""
    g = torch.Generator().manual_seed(seed)
    aq = torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, generator=g)
    wq = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, generator=g)
    cols = (K // 32 + 15) // 16 * 16
    a_s = torch.randint(125, 129, (rows, cols), dtype=torch.uint8, generator=g)
    w_s = torch.randint(125, 129, (E, N, cols), dtype=torch.uint8, generator=g)
    a_s[:, K // 32:], w_s[:, :, K // 32:] = 255, 255     # the padding is not read
    return aq, a_s, wq, w_s


def product(aq, a_s, wq, w_s, counts):
    a = mx_values(aq, a_s)
    y = torch.zeros(aq.shape[0], wq.shape[1], dtype=torch.float64)
    for e, lo, hi in groups(counts):
        if hi > lo:
            y[lo:hi] = a[lo:hi] @ mx_values(wq[e], w_s[e]).T
    return y


@pytest.mark.parametrize("E,N,K,counts", SHAPES)
def test_product_is_exact(E, N, K, counts):
    require_gpu()
    import w4a16_int4_grouped_amd as M
    counts = random_counts(E, 3 * E + 7, E) if counts == "random" else counts
    rows = sum(counts)
    log(f"case mx product E={E} N={N} K={K} rows={rows}")
    ops = operands(E, N, K, rows, N + K)
    ref = product(*ops, counts)
    got = M.mx_grouped_gemm(*(t.cuda() for t in ops), offsets_of(counts).cuda(), out_dtype=torch.float32)
    assert torch.equal(got.double().cpu(), ref)
    for dt in (torch.bfloat16, torch.float16):
        got = M.mx_grouped_gemm(*(t.cuda() for t in ops), offsets_of(counts).cuda(), out_dtype=dt)
        assert torch.equal(got.cpu(), ref.to(dt))


def test_product_of_wide_scales():
    require_gpu()
    import w4a16_int4_grouped_amd as M
    counts = [50, 3]
    aq, a_s, wq, w_s = operands(2, 72, 672, 53, 1)
    g = torch.Generator().manual_seed(2)
    a_s[:, :21] = torch.randint(90, 160, (53, 21), dtype=torch.uint8, generator=g)
    w_s[:, :, :21] = torch.randint(90, 150, (2, 72, 21), dtype=torch.uint8, generator=g)
    ref = product(aq, a_s, wq, w_s, counts)
    mag = product(aq & 0x77, a_s, wq & 0x77, w_s, counts)
    got = M.mx_grouped_gemm(aq.cuda(), a_s.cuda(), wq.cuda(), w_s.cuda(), offsets_of(counts).cuda(),
                            out_dtype=torch.float32)
    check(got, ref, mag, 672, "wide scales")


def test_rows_of_no_group_are_left():
    require_gpu()
    import w4a16_int4_grouped_amd as M
    for counts in ([7, 30], [150, 280]):
        n = sum(counts)
        ops = [t.cuda() for t in operands(2, 136, 96, n + 12, 3)]
        out = torch.full((n + 12, 144), 7.0, device="cuda")
        M.mx_grouped_gemm(*ops, offsets_of(counts, 4).cuda(), out=out[:, :136])
        assert (out[:4] == 7.0).all() and (out[n + 4:] == 7.0).all() and (out[:, 136:] == 7.0).all()
        inner = M.mx_grouped_gemm(ops[0][4:n + 4].contiguous(), ops[1][4:n + 4].contiguous(), ops[2], ops[3],
                                  offsets_of(counts).cuda(), out_dtype=torch.float32)
        assert torch.equal(out[4:n + 4, :136], inner)


def test_graph_replays():
    require_gpu()
    import w4a16_int4_grouped_amd as M
    counts = [40, 0, 9]
    x = rows_of("bf16", 49, 288, 8).cuda()
    _, _, wq, w_s = (t.cuda() for t in operands(3, 72, 288, 1, 6))
    off = offsets_of(counts).cuda()
    q, s = M.mx_quant(x)
    y = torch.empty(49, 72, dtype=torch.bfloat16, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.mx_quant(x, out=(q, s))
        M.mx_grouped_gemm(q, s, wq, w_s, off, out=y)
    for k in range(4):
        x.copy_(rows_of("bf16", 49, 288, 20 + k))
        off.copy_(offsets_of(counts[k % 3:] + counts[:k % 3]))
        y.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = M.mx_grouped_gemm(*M.mx_quant(x), wq, w_s, off)
        assert torch.equal(y, want)
