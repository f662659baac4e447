"""How far rows in 8 bits may be from their values: max(m / 128, 2^-134) for a
block's largest magnitude m."""
import pytest
import torch

from tests import step_util as U
from tests.gpu_util import log, require_gpu

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.mark.parametrize("dtype", DT)
def test_codes_are_as_near_as_documented(dtype):
    require_gpu()
    import w4a16_int4_grouped_amd as m
    g = torch.Generator().manual_seed(1)
    lowest = {"bf16": -133, "fp16": -24, "fp32": -149}[dtype]
    top = {"bf16": 127, "fp16": 15, "fp32": 127}[dtype]
    e = torch.arange(lowest, top + 1)
    log(f"case mx8 bound {dtype} 2^{lowest} .. 2^{top}")
    size = torch.cat([torch.ones(1, 32), torch.rand(1, 32, generator=g) + 0.5, torch.linspace(0.9, 1, 32)[None] * (2 - 2 ** -7),
                      torch.rand(5, 32, generator=g) * 2 * (1 - 2 ** -7)]).double()
    sign = torch.where(torch.rand(8, 32, generator=g) < 0.5, -1.0, 1.0).double()
    x = (size * sign * 2.0 ** e.double()[:, None, None]).reshape(-1, 32).to(DT[dtype])
    assert torch.isfinite(x).all()
    q, s = m.mx8_quant(x.cuda())
    got = m.mx8_dequant(q, s, dtype=torch.float32).cpu().double()
    most = (x.double().abs().amax(1, keepdim=True) / 128).clamp(min=2.0 ** -134)
    err = (got - x.double()).abs()
    log(f"  worst error {float((err / most).max()):.4f} of its bound")
    assert (err <= most).all()
    assert torch.equal(got, U.mx8(x)[0])
    # Where m is subnormal in FP32, a 128th of it is less than the least scale's half step, and an error may be more. BF16's
    # subnormals are whole steps of 2^-133, and exact.
    small = (x.double().abs().amax(1, keepdim=True) < 2.0 ** -126).expand(-1, 32)
    past = (err > x.double().abs().amax(1, keepdim=True) / 128) & small
    assert bool(past.any()) == (dtype == "fp32") and (dtype == "fp32" or (err[small] == 0).all())
