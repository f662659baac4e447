"""The step's operators at sizes whose threads one launch does not take: HIP
refuses 2^32 of them along a dimension, sizes that the header allows have more."""
import pytest
import torch

from tests import step_util as U
from tests.gpu_util import log, require_gpu

pytestmark = pytest.mark.gpu


def M():
    require_gpu()
    import w4a16_int4_grouped_amd
    return w4a16_int4_grouped_amd


@pytest.fixture(autouse=True)
def memory():
    """Each test's tens of gigabytes go back before the next asks for its own."""
    yield
    torch.cuda.empty_cache()


def test_more_sequences_by_experts_than_a_launch_takes():
    """2^20 sequences of 200 experts: 2^22 workgroups of 1024 threads join the sums."""
    m = M()
    T, E, topk, S = 3000, 200, 4, 1 << 20
    log(f"case balance T={T} E={E} S={S}")
    g = torch.Generator().manual_seed(1)
    x = torch.randn(T, E, generator=g)
    ids = x.topk(topk, 1)[1].int()
    ends = torch.randint(0, T + 1, (S + 1,), generator=g).sort()[0].int()
    ends[0], ends[-1] = 0, T
    loss, counts = m.router_balance(x.cuda(), ids.cuda(), offsets=ends.cuda())
    full = (ends[1:] > ends[:-1]).nonzero()[:, 0]
    lens = torch.cat([ends[:1], ends[1:][full]])
    want, n = U.balance(x, ids, "softmax", lens)
    assert torch.equal(counts[full.cuda()].cpu(), n) and int(counts.sum()) == T * topk
    rel = float(U.score_error(x).max()) + 160 * 2.0 ** -24
    U.close(loss[full.cuda()], want, want.abs() * rel, "loss")
    assert int((loss != 0).sum()) == len(full)


def test_combine_of_more_tokens_than_a_launch_takes():
    """2^24 tokens of 1032 columns, a workgroup each."""
    m = M()
    T, H, R = 1 << 24, 1032, 5
    log(f"case combine T={T} H={H}")
    y = torch.randn(R, H, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    slots = (torch.arange(T, device="cuda") * 7 % (R + 1)).int()          # R: no row
    out = m.combine(y, slots[:, None])
    rows = torch.cat([y, torch.zeros_like(y[:1])])
    for lo in range(0, T, 1 << 21):
        hi = lo + (1 << 21)
        assert torch.equal(out[lo:hi], rows[slots[lo:hi].long()]), lo


def test_padding_of_more_rows_than_a_launch_takes():
    """2^28 rows, nearly all of them padding."""
    m = M()
    R, H, T = (1 << 28) + 5, 8, 3
    log(f"case combine_grad R={R} H={H}")
    d = torch.randn(T, H, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    slots = torch.tensor([[R - 1], [0], [1 << 27]], dtype=torch.int32, device="cuda")
    src = torch.full((R,), T, dtype=torch.int32, device="cuda")
    src[slots[:, 0].long()] = torch.arange(T, dtype=torch.int32, device="cuda")
    dy, _ = m.combine_grad(d, slots, row_src=src, out=(torch.full((R, H), 3.0, dtype=torch.bfloat16, device="cuda"), None))
    assert torch.equal(dy[slots[:, 0].long()], d)
    dy[slots[:, 0].long()] = 0
    for lo in range(0, R, 1 << 26):
        assert not dy[lo: lo + (1 << 26)].any(), lo


def test_gradients_of_more_tokens_than_a_launch_takes():
    """2^24 tokens of 16 rows, 16 threads a row; few of the rows are there."""
    m = M()
    T, topk, H, R = 1 << 24, 16, 264, 70
    log(f"case combine_grad T={T} topk={topk} H={H}")
    g = torch.Generator().manual_seed(4)
    row = torch.randn(3, H, generator=g).bfloat16().cuda()
    d = row[torch.arange(T, device="cuda") % 3]
    y = torch.randn(R, H, generator=g).bfloat16()
    slots = torch.full((T, topk), -1, dtype=torch.int32, device="cuda")
    t = torch.linspace(0, T - 1, R, dtype=torch.float64).long()
    j = torch.arange(R) % topk
    slots[t.cuda(), j.cuda()] = torch.arange(R, dtype=torch.int32, device="cuda")
    dy, dw = m.combine_grad(d, slots, y=y.cuda())
    want = row.cpu()[t % 3]
    assert torch.equal(dy.cpu(), want)
    prod = want.double() * y.double()
    U.close(dw[t.cuda(), j.cuda()], prod.sum(1), prod.abs().sum(1) * (H + 1) * 2.0 ** -24, "d_w")
    assert int((dw != 0).sum()) == R


def test_rows_to_8_bits_of_more_than_a_launch_takes():
    """2^24 rows of 2056, a workgroup each."""
    m = M()
    rows, K, n = 1 << 24, 2056, 1 << 12
    log(f"case mx8_quant rows={rows} K={K}")
    some = torch.randn(n, K, generator=torch.Generator().manual_seed(5)).bfloat16()
    x = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda")
    x.view(-1, n, K)[:] = some.cuda()
    q, s = m.mx8_quant(x)
    _, code, byte = U.mx8(some)
    code, byte = code.cuda(), byte.cuda()
    for lo in range(0, rows, n):
        assert torch.equal(q[lo: lo + n], code) and torch.equal(s[lo: lo + n, : byte.shape[1]], byte), lo


def test_rows_from_8_bits_of_more_than_a_launch_takes():
    """2^24 rows of 2056 of which the last are live: the others are not touched."""
    m = M()
    rows, K, n = 1 << 24, 2056, 1000
    log(f"case mx8_dequant rows={rows} K={K}")
    some = torch.randn(n, K, generator=torch.Generator().manual_seed(6)).bfloat16()
    q = torch.empty(rows, K, dtype=torch.int8, device="cuda")
    s = torch.empty(rows, m.mx8_scale_cols(K), dtype=torch.uint8, device="cuda")
    m.mx8_quant(some.cuda(), out=(q[-n:], s[-n:]))
    out = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda")
    out[-n - 5:] = 3
    live = torch.tensor([rows - n, rows], dtype=torch.int32, device="cuda")
    m.mx8_dequant(q, s, offsets=live, out=out)
    assert torch.equal(out[-n:].cpu(), U.mx8(some)[0].bfloat16()) and (out[-n - 5: -n] == 3).all()


def test_swiglu_of_more_rows_than_a_launch_takes():
    """2^30 rows of 8 of which the last are live, four threads each."""
    m = M()
    rows, I, n = 1 << 30, 8, 1000
    log(f"case swiglu_save rows={rows} I={I}")
    some = torch.randn(n, 2 * I, generator=torch.Generator().manual_seed(7)).bfloat16()
    h = torch.empty(rows, 2 * I, dtype=torch.bfloat16, device="cuda")
    h[-n:] = some.cuda()
    live = torch.tensor([rows - n, rows], dtype=torch.int32, device="cuda")
    a, q, s = m.swiglu_save(h, offsets=live)
    U.close(a[-n:], U.swiglu(some), U.swiglu_slack(some), "a")
    _, code, byte = U.mx8(some.view(2 * n, I))
    assert torch.equal(q[-n:].cpu(), code.reshape(n, 2, I)) and torch.equal(s[-n:, :, :1].cpu(), byte.reshape(n, 2, 1))


def test_swiglu_gradient_of_more_rows_than_a_launch_takes():
    """17 million rows of 1032 of which the last are live, a workgroup each."""
    m = M()
    rows, I, n = 17_000_003, 1032, 1000
    log(f"case swiglu_grad rows={rows} I={I}")
    g = torch.Generator().manual_seed(8)
    some = torch.randn(n, 2 * I, generator=g).bfloat16()
    d = torch.randn(n, I, generator=g).bfloat16()
    q = torch.empty(rows, 2, I, dtype=torch.int8, device="cuda")
    s = torch.empty(rows, 2, m.mx8_scale_cols(I), dtype=torch.uint8, device="cuda")
    code, byte = m.mx8_quant(some.cuda().view(2 * n, I))
    q[-n:], s[-n:] = code.view(n, 2, I), byte.view(n, 2, -1)
    d_a = torch.empty(rows, I, dtype=torch.bfloat16, device="cuda")
    d_a[-n:] = d.cuda()
    live = torch.tensor([rows - n, rows], dtype=torch.int32, device="cuda")
    d_h, _ = m.swiglu_grad(q, d_a, scales=s, offsets=live, need_a=False)
    exact, slack = U.swiglu_grad(U.mx8(some.view(2 * n, I))[0].reshape(n, 2 * I), d)
    U.close(d_h[-n:], exact, slack, "d_h")


def test_biases_of_more_experts_by_columns_than_a_launch_takes():
    """4096 experts of 2^17 columns: 2^23 workgroups of 512 threads."""
    m = M()
    E, N, rows = 4096, 1 << 17, 9
    log(f"case grouped_bias_grad E={E} N={N}")
    dy = torch.randn(rows, N, generator=torch.Generator().manual_seed(9)).bfloat16().cuda()
    at = torch.tensor([0, 1, 700, 2047, 2048, 3000, 4000, 4094, 4095])    # one row each
    counts = torch.zeros(E, dtype=torch.long)
    counts[at] = 1
    off = torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)]).int().cuda()
    db = m.grouped_bias_grad(dy, off, out=torch.full((E, N), 3.0, dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(db[at.cuda()], dy)
    db[at.cuda()] = 0
    assert not db.any()


def integers(*shape, seed):
    return torch.randint(-3, 4, shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


@pytest.mark.parametrize("way", ["forward", "input", "bias", "swiglu"])
def test_products_of_more_tiles_than_a_launch_takes(way):
    """4096 experts of a row each and 2^20 columns (of weights that all share): 2^25 tiles, exact on integers."""
    m = M()
    E, N, K = 4096, 1 << 20, 8
    log(f"case grouped {way} E={E} N={N} K={K}")
    off = torch.arange(E + 1, dtype=torch.int32, device="cuda")
    a = integers(E, K, seed=10)
    out = torch.full((E, N // 2 if way == "swiglu" else N), 777.0, dtype=torch.bfloat16, device="cuda")
    if way == "input":
        w = integers(1, K, N, seed=11)
        m.grouped_gemm_dgrad(a, w.expand(E, K, N), off, out=out)
        w = w[0]
    else:
        w = integers(1, N, K, seed=11)
        if way == "forward":
            m.grouped_gemm(a, w.expand(E, N, K), off, out=out)
        else:
            bias = integers(1, N, seed=14).expand(E, N).contiguous() if way == "bias" else None
            m.grouped_linear(a, w.expand(E, N, K), off, bias=bias, act="none" if bias is not None else way, out=out)
        w = w[0].t()
    for lo in range(0, E, 256):
        z = a[lo: lo + 256].float() @ w.float()
        if way == "bias":
            z += bias[0].float()
        got = out[lo: lo + 256]
        if way == "swiglu":
            gate, up = z[:, : N // 2], z[:, N // 2:]
            z = gate * torch.sigmoid(gate) * up
            # both FP32: the sigmoid within (2 |g| + 10) steps (|g| <= 72), rounded to half a step of BF16
            assert ((got.float() - z).abs() <= z.abs() * (2.0 ** -8 + 2 * 154 * 2.0 ** -23) + 2.0 ** -126).all(), lo
        else:
            assert torch.equal(got.float(), z), lo


def test_weight_gradients_of_more_tiles_than_a_launch_takes():
    """4096 experts of 8 by 2^20."""
    m = M()
    E, N, K, rows = 4096, 8, 1 << 20, 5
    log(f"case grouped wgrad E={E} N={N} K={K}")
    dy, a = integers(rows, N, seed=12), integers(rows, K, seed=13)
    at = torch.tensor([0, 2048, 4093, 4095])
    counts = torch.zeros(E, dtype=torch.long)
    counts[at] = torch.tensor([1, 2, 1, 1])
    off = torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)]).int().cuda()
    dw = torch.full((E, N, K), 7.0, dtype=torch.bfloat16, device="cuda")
    m.grouped_gemm_wgrad(dy, a, off, out=dw)
    for e, lo, hi in ((0, 0, 1), (2048, 1, 3), (4093, 3, 4), (4095, 4, 5)):
        assert torch.equal(dw[e].float(), dy[lo:hi].float().t() @ a[lo:hi].float()), e
        dw[e] = 0
    for lo in range(0, E, 256):
        assert not dw[lo: lo + 256].any(), lo
