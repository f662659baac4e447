"""Which stream an output's memory comes from, with a stand-in for torch's
allocator: memory freed on the caller's stream may still be in use by kernels
queued there, so what a kernel on another stream writes has to come from that
stream's memory, and stays reserved for both."""
import contextlib
import types

import pytest
import torch

import w4a16_int4_grouped_amd as M
from tests.test_operators_views_cpu import Standin


class Stream:
    def __init__(self, number, device_index=0):
        self.cuda_stream, self.device_index = number, device_index
        self.device = torch.device("cuda", device_index)


CALLER, OTHER = Stream(0), Stream(7)


class Made(Standin):
    """An output: the stream it was made on, those it is kept for."""

    def __init__(self, shape, dtype, stream):
        super().__init__(shape, dtype)
        self.made_on, self.kept_for = stream, []

    def record_stream(self, s):
        self.kept_for.append(s)


@pytest.fixture
def made(monkeypatch):
    """The outputs that a call makes; its launches are recorded, not run."""
    now, outputs = [CALLER], []

    @contextlib.contextmanager
    def stream(s):
        now.append(s)
        yield
        now.pop()

    def empty(*shape, dtype, device):
        shape = shape[0] if len(shape) == 1 and not isinstance(shape[0], int) else shape
        outputs.append(Made(shape, dtype, now[-1]))
        return outputs[-1]

    fake = types.SimpleNamespace(
        empty=empty, cuda=types.SimpleNamespace(stream=stream, current_stream=lambda device=None: now[-1]),
        **{n: getattr(torch, n) for n in ("bfloat16", "float16", "float32", "int32", "uint8")})
    M._load()
    monkeypatch.setattr(M, "_torch", fake)
    monkeypatch.setattr(M, "_call", lambda fn, device, stream, *args: None)
    return outputs


B, F, I, U = torch.bfloat16, torch.float32, torch.int32, torch.uint8
CALLS = {
    "router_topk": lambda s: M.router_topk(Standin((6, 64), B), 4, stream=s),
    "router_topk_grad": lambda s: M.router_topk_grad(Standin((6, 64), B), Standin((6, 4), I), Standin((6, 4), F),
                                                     stream=s),
    "grouped_gemm": lambda s: M.grouped_gemm(Standin((6, 64), B), Standin((2, 32, 64), B), Standin((3,), I), stream=s),
    "grouped_gemm_dgrad": lambda s: M.grouped_gemm_dgrad(Standin((6, 32), B), Standin((2, 32, 64), B),
                                                         Standin((3,), I), stream=s),
    "grouped_gemm_wgrad": lambda s: M.grouped_gemm_wgrad(Standin((6, 32), B), Standin((6, 64), B), Standin((3,), I),
                                                         stream=s),
    "mx_quant": lambda s: M.mx_quant(Standin((6, 64), B), stream=s),
    "mx_dequant": lambda s: M.mx_dequant(Standin((6, 32), U), Standin((6, 16), U), stream=s),
    "mx_grouped_gemm": lambda s: M.mx_grouped_gemm(Standin((6, 32), U), Standin((6, 16), U), Standin((2, 8, 32), U),
                                                   Standin((2, 8, 16), U), Standin((3,), I), stream=s),
}


@pytest.mark.parametrize("name", CALLS)
def test_outputs_come_from_the_stream_that_writes_them(made, name):
    CALLS[name](OTHER)
    assert made
    for t in made:
        assert t.made_on is OTHER
        assert CALLER in t.kept_for


@pytest.mark.parametrize("name", CALLS)
def test_outputs_of_the_callers_own_stream(made, name):
    for stream in (None, CALLER):
        CALLS[name](stream)
    assert all(t.made_on is CALLER for t in made)
