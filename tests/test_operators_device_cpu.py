"""A stream of another device than the tensors' is refused before any HIP call."""
import pytest
import torch

import w4a16_int4_grouped_amd as M
from tests.test_operators_streams_cpu import CALLS, Stream
from tests.test_operators_views_cpu import Standin


@pytest.mark.parametrize("name", CALLS)
def test_stream_of_another_device(monkeypatch, name):
    M._load()
    launched = []

    class Lib:
        def __getattr__(self, f):
            if f == "moe_mx_scale_cols":
                return lambda K: (K // 32 + 15) // 16 * 16
            return lambda *args: launched.append(f) or M.MOE_OK
    monkeypatch.setattr(M, "_lib", Lib())
    monkeypatch.setattr(M, "_new", lambda shape, dtype, device, stream: Standin(shape, dtype))
    monkeypatch.setattr(Standin, "device", torch.device("cuda", 0))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    M.mx_scale_cols.cache_clear()
    with pytest.raises(M.MoeError, match="stream") as e:
        CALLS[name](Stream(7, device_index=1))
    assert e.value.status == M.MOE_ERR_INVALID_ARG
    CALLS[name](Stream(7, device_index=0))
    M.mx_scale_cols.cache_clear()
    assert len(launched) == 1
