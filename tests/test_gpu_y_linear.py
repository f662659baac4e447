"""The experts' product with bias, SwiGLU and residual in its epilogue, and the
gradient of the biases, against 64 bits."""
import pytest
import torch

from tests import step_util as U
from tests.gpu_util import log, require_gpu
from tests.ops_util import groups, offsets_of, random_counts

pytestmark = pytest.mark.gpu
DT = U.DT


def M():
    require_gpu()
    import w4a16_int4_grouped_amd
    return w4a16_int4_grouped_amd


def inputs(E, rows, N, K, dtype, seed, act, bias=None, res=None):
    g = torch.Generator().manual_seed(seed)
    a = torch.randn(rows, K, generator=g).to(DT[dtype])
    w = (torch.randn(E, N, K, generator=g) * K ** -0.5).to(DT[dtype])
    b = None if bias is None else torch.randn(E, N, generator=g).to(DT[bias])
    cols = N // 2 if act == "swiglu" else N
    r = None if res is None else torch.randn(rows, cols, generator=g).to(DT[res])
    return a, w, b, r


def run(E, counts, N, K, dtype, act, bias, res, out_dtype, seed):
    """With 3 rows before the first group and 2 behind the last, which stay as they are."""
    m = M()
    rows = sum(counts) + 5
    a, w, b, r = inputs(E, rows, N, K, dtype, seed, act, bias, out_dtype if res else None)
    exact, slack = U.linear(a, w, counts, b, act, r, start=3)
    a[:3], a[-2:] = float("nan"), float("nan")
    cols = exact.shape[1]
    out = torch.full((rows, cols), 7.0, dtype=DT[out_dtype], device="cuda")
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    got = m.grouped_linear(c(a), c(w), offsets_of(counts, 3).cuda(), bias=c(b), act=act, residual=c(r), out=out)
    assert got is out
    U.close(out[3:-2], exact[3:-2], slack[3:-2], "out")
    assert (out[:3] == 7).all() and (out[-2:] == 7).all()


@pytest.mark.parametrize("E,counts,N,K", [
    (1, [1], 16, 8), (1, [0], 64, 64), (3, [5, 0, 33], 48, 72), (2, [64, 31], 144, 136), (4, [130, 1, 0, 257], 272, 200),
    (2, [300, 520], 528, 328), (1, [700], 1040, 264), (8, [40] * 8, 512, 1032), (3, [64, 64, 65], 4112, 64),
])
@pytest.mark.parametrize("dtype,act,bias,res,out_dtype", [
    ("bf16", "swiglu", None, False, "bf16"), ("bf16", "swiglu", "bf16", True, "bf16"),
    ("fp16", "swiglu", "fp32", False, "fp16"), ("bf16", "swiglu", "fp16", True, "fp32"),
    ("bf16", "none", "bf16", False, "bf16"), ("fp16", "none", "fp16", True, "fp16"),
    ("bf16", "none", None, True, "fp32"), ("fp16", "none", "fp32", False, "bf16"),
])
def test_linear(E, counts, N, K, dtype, act, bias, res, out_dtype):
    log(f"case linear E={E} rows={counts} N={N} K={K} {dtype} {act} bias={bias} res={res} -> {out_dtype}")
    run(E, counts, N, K, dtype, act, bias, res, out_dtype, N + K)


# E, rows, N, K whose form of tiles is each of the five (tests/test_step_cpu.py asserts it)
FORMS = [("few rows each", 64, 600, 2048, 4096), ("large", 16, 8192, 2048, 2048), ("two", 1, 1024, 4096, 512), ("four", 48, 4200, 2048, 128),
         ("split", 1, 250, 2432, 2048), ("thin", 1, 64, 512, 2048)]


@pytest.mark.parametrize("name,E,rows,N,K", FORMS)
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_every_form_of_tiles(name, E, rows, N, K, act):
    """Exact integers: every sum is below 2^24, so the product has one value; the epilogue rounds."""
    m = M()
    log(f"case linear form {name} E={E} rows={rows} N={N} K={K} {act}")
    counts = random_counts(E, rows, rows, empty=0.1)
    g = torch.Generator(device="cuda").manual_seed(rows)
    ints = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    a, w, bias = ints(rows, K), ints(E, N, K), ints(E, N)
    cols = N // 2 if act == "swiglu" else N
    res = ints(rows, cols).float()
    got = m.grouped_linear(a, w, offsets_of(counts).cuda(), bias=bias, act=act, residual=res, out_dtype=torch.float32)
    plain = m.grouped_linear(a, w, offsets_of(counts).cuda(), bias=bias, act=act, out_dtype=torch.float32)
    for e, lo, hi in groups(counts):
        z = a[lo:hi].float().double() @ w[e].double().T + bias[e].double()
        if act == "none":
            assert torch.equal(got[lo:hi].double(), z + res[lo:hi].double())
            assert torch.equal(plain[lo:hi].double(), z)
            continue
        gt, up = z[:, :cols], z[:, cols:]
        y = gt * torch.sigmoid(gt) * up
        slack = y.abs() * (2 * gt.abs() + 10) * 2.0 ** -23 + 2.0 ** -126 * (1 + (gt * up).abs())
        assert ((plain[lo:hi].double() - y).abs() <= slack).all()
        full = y + res[lo:hi].double()
        assert ((got[lo:hi].double() - full).abs() <= slack + (full.abs() + slack) * 2.0 ** -23).all()


def test_strides_residual_in_place_and_shared_weights():
    m = M()
    g = torch.Generator().manual_seed(3)
    E, counts, N, K = 3, [70, 0, 41], 96, 104
    rows = sum(counts)
    a = torch.randn(rows, 120, generator=g).bfloat16()[:, 8:112]
    w = torch.randn(1, N, K, generator=g).bfloat16().expand(E, N, K)          # one matrix for all experts
    bias = torch.randn(E, 112, generator=g).bfloat16()
    off = offsets_of(counts).cuda()
    for act, cols in (("none", N), ("swiglu", N // 2)):
        buf = torch.randn(rows, cols + 16, generator=g).bfloat16()
        exact, slack = U.linear(a, w, counts, bias[:, 8:104], act, buf[:, 8:-8])
        dev = buf.cuda()
        wc = w[:1].cuda().expand(E, N, K)
        full = torch.zeros(rows, 120, dtype=torch.bfloat16)
        full[:, 8:112] = a
        m.grouped_linear(full.cuda()[:, 8:112], wc, off, bias=bias.cuda()[:, 8:104], act=act, residual=dev[:, 8:-8],
                         out=dev[:, 8:-8])
        U.close(dev[:, 8:-8], exact, slack, act)
        assert torch.equal(dev[:, :8].cpu(), buf[:, :8]) and torch.equal(dev[:, -8:].cpu(), buf[:, -8:])


def test_linear_without_epilogue_is_the_grouped_product():
    m = M()
    a, w, _, _ = inputs(4, 300, 256, 192, "bf16", 1, "none")
    off = offsets_of(random_counts(4, 300, 2)).cuda()
    assert torch.equal(m.grouped_linear(a.cuda(), w.cuda(), off), m.grouped_gemm(a.cuda(), w.cuda(), off))


def test_nan_and_infinity_stay_in_their_rows():
    m = M()
    a, w, b, r = inputs(2, 40, 64, 64, "bf16", 1, "swiglu", "bf16", "bf16")
    a[3, 5], r[17, 2], b[1, 9] = float("inf"), float("nan"), float("nan")
    off = offsets_of([25, 15]).cuda()
    y = m.grouped_linear(a.cuda(), w.cuda(), off, bias=b.cuda(), act="swiglu", residual=r.cuda()).cpu()
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[17, 2] = True
    want[25:, 9] = True                      # gate column 9 of expert 1
    assert torch.equal(torch.cat([bad[:3], bad[4:]]), torch.cat([want[:3], want[4:]]))
    assert bad[3].any()


@pytest.mark.parametrize("dtype,out_dtype", [("bf16", "bf16"), ("fp16", "fp32"), ("bf16", "fp32"), ("fp16", "bf16")])
@pytest.mark.parametrize("E,counts,N", [
    (1, [1], 8), (1, [0], 72), (3, [0, 700, 3], 136), (48, None, 1024), (1, [5000], 64), (300, None, 520), (5, [64, 65, 63, 1, 0], 7168),
])
def test_bias_gradient(E, counts, N, dtype, out_dtype):
    m = M()
    counts = counts or random_counts(E, 40 * E, E)
    log(f"case bias gradient E={E} rows={sum(counts)} N={N} {dtype} -> {out_dtype}")
    rows = sum(counts) + 5
    dy = torch.randn(rows, N, generator=torch.Generator().manual_seed(N)).to(DT[dtype])
    exact = torch.stack([dy[lo:hi].double().sum(0) for _, lo, hi in groups(counts, 3)])
    size = torch.stack([dy[lo:hi].double().abs().sum(0) for _, lo, hi in groups(counts, 3)])
    steps = torch.tensor([n + 12 for n in counts]).double()[:, None]         # additions that a value passes, at most
    dy[:3], dy[-2:] = float("nan"), float("nan")
    db = m.grouped_bias_grad(dy.cuda(), offsets_of(counts, 3).cuda(), out_dtype=DT[out_dtype])
    U.close(db, exact, size * steps * 2.0 ** -24, "bias gradient")


def test_bias_gradient_strides_and_no_rows():
    m = M()
    dy = torch.randn(90, 88, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    off = offsets_of([30, 60]).cuda()
    out = torch.full((2, 96), 7.0, device="cuda")
    m.grouped_bias_grad(dy[:, 8:80], off, out=out[:, 8:80])
    assert torch.equal(out[:, 8:80], m.grouped_bias_grad(dy[:, 8:80].contiguous(), off, out_dtype=torch.float32))
    assert (out[:, :8] == 7).all() and (out[:, 80:] == 7).all()
    none = m.grouped_bias_grad(dy[:0, :64], torch.zeros(4, dtype=torch.int32, device="cuda"))
    assert none.shape == (3, 64) and (none == 0).all()
