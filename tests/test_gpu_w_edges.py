"""The operators at the ends of their documented ranges: 4096 experts, rows and
columns of 2^20 values, subnormal operands, the smallest and largest scales.
Exact: small integers, or one product a sum."""
import pytest
import torch

from tests.gpu_util import log, require_gpu
from tests.ops_util import groups, mx_values, offsets_of, random_counts
from tests.test_gpu_l_grouped import reference, run

pytestmark = pytest.mark.gpu


def ints(*shape, seed, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-3, 4, shape, generator=g).to(dtype)


@pytest.mark.parametrize("way", ["fwd", "dgrad", "wgrad"])
@pytest.mark.parametrize("E", [64, 65, 4095, 4096])
def test_many_experts(way, E):
    require_gpu()
    import w4a16_int4_grouped_amd as M
    log(f"case many experts {way} E={E}")
    for counts in (random_counts(E, 700, E), [0] * (E - 1) + [300], [1] * E):
        n = sum(counts)
        dy, a, w = ints(n, 40, seed=1), ints(n, 24, seed=2), ints(E, 40, 24, seed=3)
        ref, _ = reference(way, dy, a, w, counts)
        got = run(M, way, dy.cuda(), a.cuda(), w.cuda(), offsets_of(counts).cuda(), out_dtype=torch.float32)
        assert torch.equal(got.double().cpu(), ref)


@pytest.mark.parametrize("way", ["fwd", "dgrad", "wgrad"])
@pytest.mark.parametrize("N,K", [(1 << 20, 8), (8, 1 << 20)])
def test_widest_matrices(way, N, K):
    require_gpu()
    import w4a16_int4_grouped_amd as M
    log(f"case widest {way} N={N} K={K}")
    counts = [3, 0, 2]
    dy, a, w = ints(5, N, seed=4), ints(5, K, seed=5), ints(3, N, K, seed=6)
    ref, _ = reference(way, dy, a, w, counts)
    got = run(M, way, dy.cuda(), a.cuda(), w.cuda(), offsets_of(counts).cuda(), out_dtype=torch.float32)
    assert torch.equal(got.double().cpu(), ref)


@pytest.mark.parametrize("N,K", [((1 << 20), 32), (8, 1 << 20)])
def test_widest_mxfp4(N, K):
    require_gpu()
    import w4a16_int4_grouped_amd as M
    log(f"case widest MXFP4 N={N} K={K}")
    x, w = ints(5, K, seed=7), ints(2, N, K, seed=8)
    q, wq = M.mx_quant(x.cuda()), M.mx_quant(w.cuda())
    got = M.mx_grouped_gemm(*q, *wq, offsets_of([3, 2]).cuda(), out_dtype=torch.float32)
    for e, lo, hi in groups([3, 2]):
        assert torch.equal(got[lo:hi].double().cpu(), x[lo:hi].double() @ w[e].double().T)
    assert torch.equal(M.mx_dequant(*q).cpu(), x)


@pytest.mark.parametrize("way", ["fwd", "dgrad", "wgrad"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_subnormal_operands(way, dtype):
    """One term a sum: a subnormal of the type times 1, or times 2^20 where the product would leave FP32's normal range."""
    require_gpu()
    import w4a16_int4_grouped_amd as M
    f = torch.finfo(dtype)
    tiny = f.smallest_normal * f.eps
    n = 32
    sub = (torch.arange(n * n).reshape(n, n) % 7 - 3).double() * tiny
    one = torch.eye(n, dtype=torch.float64) * (2.0 ** 20 if dtype == torch.bfloat16 else 1.0)
    off = offsets_of([n]).cuda()
    for dy, a, w in ((sub, sub, one), (one, one, sub)):
        if way == "wgrad":
            a = one if dy is sub else sub
        dy, a, w = (t.to(dtype) for t in (dy, a, w))
        ref, _ = reference(way, dy, a, w[None], [n])
        got = run(M, way, dy.cuda(), a.cuda(), w[None].cuda(), off, out_dtype=torch.float32)
        assert float(ref.abs().max()) > 0
        assert torch.equal(got.double().cpu(), ref)


@pytest.mark.parametrize("K", [32, 544, 2080])
@pytest.mark.parametrize("sa,sw", [(0, 254), (254, 0), (3, 250), (127, 127), (0, 127), (127, 0), (254, 100), (1, 100)])
def test_ends_of_the_scales(K, sa, sw):
    """Codes 1 and 0.5 times scales: where the products are values of FP32, sums of up to 2080 of them are exact. Where
    they are not (2^-155 and more, under FP32's smallest step 2^-149), each of at most K additions to a sum is off by at
    most that step."""
    require_gpu()
    import w4a16_int4_grouped_amd as M
    log(f"case scales K={K} {sa} {sw}")
    cols = M.mx_scale_cols(K)
    g = torch.Generator().manual_seed(K + sa)
    code = torch.tensor([0x11, 0x22, 0x12, 0x21], dtype=torch.uint8)
    aq, wq = code[torch.randint(0, 4, (70, K // 2), generator=g)], code[torch.randint(0, 4, (1, 72, K // 2), generator=g)]
    a_s, w_s = torch.full((70, cols), sa, dtype=torch.uint8), torch.full((1, 72, cols), sw, dtype=torch.uint8)
    ref = mx_values(aq, a_s) @ mx_values(wq[0], w_s[0]).T
    got = M.mx_grouped_gemm(aq.cuda(), a_s.cuda(), wq.cuda(), w_s.cuda(), offsets_of([70]).cuda(), out_dtype=torch.float32)
    if sa + sw - 254 - 2 >= -149:
        assert torch.equal(got.double().cpu(), ref.float().double())
    else:
        assert ((got.double().cpu() - ref).abs() <= K * 2.0 ** -149).all()


def test_nan_scales_of_weights():
    """A weight block of NaN makes its column NaN in the rows of its expert, no other."""
    require_gpu()
    import w4a16_int4_grouped_amd as M
    E, N, K = 2, 40, 160
    g = torch.Generator().manual_seed(3)
    x, w = torch.randn(50, K, generator=g), torch.randn(E, N, K, generator=g)
    w[1, 7, 33], w[0, 39, 159] = float("nan"), float("inf")
    y = M.mx_grouped_gemm(*M.mx_quant(x.cuda()), *M.mx_quant(w.cuda()), offsets_of([20, 30]).cuda())
    bad = torch.zeros(50, N, dtype=torch.bool)
    bad[20:, 7] = bad[:20, 39] = True
    assert torch.equal(torch.isnan(y).cpu(), bad)
    assert torch.isfinite(y.cpu()[~bad]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_outputs_past_the_types_range(dtype):
    """A sum past the output type's largest value is an infinity of its sign, one below its subnormals 0."""
    require_gpu()
    import w4a16_int4_grouped_amd as M
    big = torch.zeros(3, 64)
    big[0, 0], big[1, 0], big[2, 0] = 2.0 ** 100, -2.0 ** 100, 2.0 ** -100
    w = torch.zeros(1, 64, 64)
    w[0, 0, 0], w[0, 1, 0] = 2.0 ** 100, 2.0 ** -100
    y = M.grouped_gemm(big.bfloat16().cuda(), w.bfloat16().cuda(), offsets_of([3]).cuda(), out_dtype=dtype).cpu()
    want = (big.double() @ w[0].double().T).to(dtype)
    assert torch.equal(y, want)
