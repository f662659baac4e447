"""Grouped products large enough for each of the tile forms, on small
integers: every FP32 sum is exact (at most 9 * 20000 < 2^24), so the outputs
have to equal FP64 products of the same inputs on the GPU. The groups' last
rows fall on every tile height, columns end inside a tile, contractions inside
a step."""
import pytest
import torch

from tests.gpu_util import log, require_gpu
from tests.ops_util import groups, offsets_of, random_counts
from tests.test_gpu_l_grouped import run

pytestmark = pytest.mark.gpu

UNEVEN = [2065, 1664, 3222, 2504, 0, 1, 2816, 1927, 3301]      # remainders 17, 128, 150, 200, -, 1, 0, 135, 229

CASES = [
    # way, E, N, K, counts (None: random, rows)
    ("fwd", 9, 2056, 584, UNEVEN),
    ("dgrad", 9, 584, 2056, UNEVEN),
    ("wgrad", 9, 2056, 1032, UNEVEN),
    ("wgrad", 12, 4104, 4104, 6000),
    ("fwd", 40, 4104, 72, 9000),
    ("fwd", 300, 1032, 1032, 30000),
    ("dgrad", 300, 1032, 264, 30000),
    ("wgrad", 70, 1032, 1032, 300),
    ("fwd", 5, 136, 7176, 300),
    ("dgrad", 4, 6088, 504, 564),
    ("wgrad", 2, 264, 520, 20000),
    ("fwd", 2, 264, 4104, [33, 0]),
]


def reference(way, dy, a, w, counts):
    E = len(counts)
    if way == "wgrad":
        out = torch.zeros(E, dy.shape[1], a.shape[1], dtype=torch.float64, device="cuda")
    else:
        out = torch.zeros(dy.shape[0], w.shape[1 if way == "fwd" else 2], dtype=torch.float64, device="cuda")
    for e, lo, hi in groups(counts):
        if way == "fwd":
            out[lo:hi] = a[lo:hi].double() @ w[e].double().T
        elif way == "dgrad":
            out[lo:hi] = dy[lo:hi].double() @ w[e].double()
        else:
            out[e] = dy[lo:hi].double().T @ a[lo:hi].double()
    return out


@pytest.mark.parametrize("way,E,N,K,counts", CASES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_every_tile_form_is_exact(way, E, N, K, counts, dtype):
    require_gpu()
    import w4a16_int4_grouped_amd as M
    counts = counts if isinstance(counts, list) else random_counts(E, counts, E)
    rows = sum(counts)
    log(f"case tiles {way} E={E} N={N} K={K} rows={rows} {dtype}")
    g = torch.Generator(device="cuda").manual_seed(N + K)
    r = lambda *s: torch.randint(-3, 4, s, generator=g, device="cuda").to(dtype)  # noqa: E731
    dy, a, w = r(rows, N), r(rows, K), r(E, N, K)
    off = offsets_of(counts).cuda()
    ref = reference(way, dy, a, w, counts)
    whole = torch.full((ref.shape[0] + 1,) + ref.shape[1:], 7.0, device="cuda")
    run(M, way, dy, a, w, off, out=whole[:-1])
    assert torch.equal(whole[:-1].double(), ref)
    assert (whole[-1] == 7.0).all()
    assert torch.equal(run(M, way, dy, a, w, off), ref.to(dtype))       # one rounding, to the type of the operands


@pytest.mark.parametrize("E,N,K,counts", [(9, 2056, 544, UNEVEN), (6, 4104, 2080, UNEVEN[:6]), (300, 1032, 1056, 30000),
                                          (40, 4104, 96, 9000), (5, 136, 7200, 300), (2, 264, 4128, [33, 0])])
def test_every_tile_form_of_mxfp4_is_exact(E, N, K, counts):
    """Scales of 2^-1 .. 2^1: products are multiples of 2^-4 of at most 144, 2304 such steps, and 7200 of them stay
    below 2^24 steps: every FP32 sum is exact."""
    require_gpu()
    import w4a16_int4_grouped_amd as M
    counts = counts if isinstance(counts, list) else random_counts(E, counts, E)
    rows = sum(counts)
    log(f"case mx tiles E={E} N={N} K={K} rows={rows}")
    g = torch.Generator(device="cuda").manual_seed(K)
    u8 = lambda lo, hi, *s: torch.randint(lo, hi, s, dtype=torch.uint8, generator=g, device="cuda")  # noqa: E731
    cols = M.mx_scale_cols(K)
    aq, wq = u8(0, 256, rows, K // 2), u8(0, 256, E, N, K // 2)
    a_s, w_s = u8(126, 129, rows, cols), u8(126, 129, E, N, cols)
    a_s[:, K // 32:], w_s[:, :, K // 32:] = 255, 255
    got = M.mx_grouped_gemm(aq, a_s, wq, w_s, offsets_of(counts).cuda(), out_dtype=torch.float32)
    a = M.mx_dequant(aq, a_s, dtype=torch.float32)
    for e, lo, hi in groups(counts):
        ref = a[lo:hi].double() @ M.mx_dequant(wq[e], w_s[e], dtype=torch.float32).double().T
        assert torch.equal(got[lo:hi].double(), ref), e


@pytest.mark.parametrize("offsets", [[0, 30, 10, 40, 40], [40, 0, 40, 0, 40], [5, 1 << 30, -7, 20, 39]])
def test_offsets_that_decrease_stay_inside(offsets):
    require_gpu()
    import w4a16_int4_grouped_amd as M
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    dy, a, w = r(40, 136), r(40, 72), r(4, 136, 72)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    for way, shape in (("fwd", (40, 136)), ("dgrad", (40, 72)), ("wgrad", (4, 136, 72))):
        whole = torch.full((shape[0] + 2,) + shape[1:], 7.0, device="cuda")
        run(M, way, dy, a, w, off, out=whole[1:-1])
        torch.cuda.synchronize()
        assert (whole[0] == 7.0).all() and (whole[-1] == 7.0).all()
