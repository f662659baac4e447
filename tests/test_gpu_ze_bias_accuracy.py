"""The biases' gradient where FP32 could lose it: many equal rows of one group."""
import pytest
import torch

from tests.gpu_util import log, require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,M,N", [
    (512, 1 << 22, 64),       # a workgroup for the group's 64 columns: 2^16 rows a lane
    (512, (1 << 22) + 77, 8),
    (1, 1 << 26, 8),          # in chunks: 2^15 of their sums a wave
    (2, (1 << 26) + 1000, 8),
])
def test_many_equal_rows(E, M, N):
    """2047 / 2048: in FP32 a long sum's every step would be rounded up."""
    require_gpu()
    import w4a16_int4_grouped_amd as m
    log(f"case grouped_bias_grad E={E} M={M} N={N}")
    dy = torch.full((M, N), 2047 / 2048, dtype=torch.float16, device="cuda")
    lo = 5 if E > 1 else 0
    off = torch.full((E + 1,), M, dtype=torch.int32)
    off[: E // 2 + 1] = lo
    off[0] = 0
    db = m.grouped_bias_grad(dy, off.cuda(), out_dtype=torch.float32).cpu()
    n = (off[1:] - off[:-1]).double()
    worst = ((db.double() - n[:, None] * 2047 / 2048).abs() / n.clamp(min=1)[:, None]).max()
    log(f"  off by {float(worst) * 2 ** 24:.1f} steps of 2^-24")
    # half a step of 2^-23 for each addition in FP32: 256 rows in a lane and 3 of a wave's 8 lanes and 8 waves of a group's
    # part, or 4, 3 and 8 of a chunk, then 256 chunks' sums and 8 waves; what FP64 joined is rounded once
    assert worst <= (256 + 3 + 8 + 4 + 3 + 8 + 1) * 2.0 ** -24
    torch.cuda.empty_cache()
