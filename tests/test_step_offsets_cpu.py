"""Offsets of more experts or sequences than the library's arguments hold are
refused; cut to 32 bits they would name fewer, or none."""
import pytest

import w4a16_int4_grouped_amd as M
from tests.test_step_cpu import F, I, Q, T, U, fake  # noqa: F401

FAR = (1 << 32) + 3        # 2 in 32 bits

CALLS = {
    "balance": lambda: M.router_balance(T(40, 8), T(40, 2, dtype=I), offsets=T(FAR, dtype=I)),
    "balance gradient": lambda: M.router_balance_grad(T(40, 8), T(FAR - 1, 8, dtype=I), T(FAR - 1, dtype=F), 2,
                                                      offsets=T(FAR, dtype=I)),
    "combine gradient": lambda: M.combine_grad(T(40, 64), T(40, 2, dtype=I), y=T(90, 64), row_src=T(90, dtype=I),
                                               offsets=T(FAR, dtype=I)),
    "dequant": lambda: M.mx8_dequant(T(40, 64, dtype=Q), T(40, 16, dtype=U), offsets=T(FAR, dtype=I)),
    "save": lambda: M.swiglu_save(T(40, 64), offsets=T(FAR, dtype=I)),
    "gradient": lambda: M.swiglu_grad(T(40, 64), T(40, 32), offsets=T(FAR, dtype=I)),
    "bias gradient": lambda: M.grouped_bias_grad(T(40, 64), T(FAR, dtype=I)),
}


@pytest.mark.parametrize("name", CALLS)
def test_offsets_past_31_bits(fake, name):  # noqa: F811
    with pytest.raises(M.MoeError, match="2\\^31") as e:
        CALLS[name]()
    assert e.value.status == M.MOE_ERR_INVALID_ARG
    assert not fake
