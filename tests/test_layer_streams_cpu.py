"""Which stream the layer's buffers come from, its outputs and the workspaces
that it gives back on return, with a stand-in for torch's allocator."""
import contextlib
import ctypes
import os

import pytest
import torch

import w4a16_int4_grouped_amd as M
from tests.test_operators_streams_cpu import CALLER, OTHER, Made
from tests.test_operators_views_cpu import Standin

E, H, T, TOPK = 8, 256, 6, 2


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(M.LIB_PATH):
        from w4a16_int4_grouped_amd import build
        build.build()


def plan(mode):
    """A handle without weights."""
    h = M.PreparedWeights.__new__(M.PreparedWeights)
    d = M.make_desc(E, H, 512, mode)
    h.E, h.H, h.I, h.mode, h.device = E, H, 512, M.MODES[mode], torch.device("cuda", 0)
    h.handle = ctypes.c_void_p(M._lib.moe_plan_create(ctypes.byref(d)))
    return h


B, F, I = torch.bfloat16, torch.float32, torch.int32
X, IDS, W, ROUTING = Standin((T, H), B), Standin((T, TOPK), I), Standin((T, TOPK), F), Standin((4096,), I)
CALLS = {
    "align": lambda s: plan("indexed").align(IDS, stream=s),
    "align_ep": lambda s: plan("indexed").align_ep(IDS, Standin((16,), I), 16, stream=s),
    "permute": lambda s: plan("indexed").permute(X, TOPK, ROUTING, stream=s),
    "indexed": lambda s: plan("indexed").indexed(X, IDS, W, stream=s),
    "contiguous": lambda s: plan("contiguous").contiguous(Standin((128, H), B), Standin((128,), I), stream=s),
    "masked": lambda s: plan("masked").masked(Standin((E, 16, H), B), Standin((E,), I), 4, stream=s),
    "gate_up": lambda s: plan("indexed").gate_up(X, TOPK, ROUTING, stream=s),
    "down": lambda s: plan("indexed").down(Standin((64, 512), B), T, TOPK, ROUTING, stream=s),
    "dequant": lambda s: plan("indexed").dequant(13, 0, stream=s),
    "swiglu": lambda s: M.swiglu(Standin((T, 1024), B), stream=s),
    "weights": lambda s: M.PreparedWeights(Standin((E, 1024, H // 8), I), Standin((E, 1024, H // 32), B),
                                           Standin((E, H, 64), I), Standin((E, H, 16), B), stream=s),
}


class Buffer(Made):
    def element_size(self):
        return self.dtype.itemsize


@pytest.fixture
def no_launch(monkeypatch):
    """The buffers that a call makes; of the library, its host arithmetic only."""
    now, buffers = [CALLER], []

    @contextlib.contextmanager
    def stream(s):
        now.append(s)
        yield
        now.pop()

    def empty(*shape, dtype, device):
        shape = shape[0] if isinstance(shape[0], tuple) else shape
        buffers.append(Buffer(shape, dtype, now[-1]))
        return buffers[-1]

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[-1])
    L = M.lib()

    class Lib:
        def __getattr__(self, name):
            if name in ("moe_prepared_bytes", "moe_routing_bytes", "moe_routing_layout", "moe_workspace_bytes"):
                return getattr(L, name)
            return lambda *args: M.MOE_OK
    monkeypatch.setattr(M, "lib", Lib)
    return buffers


@pytest.mark.parametrize("name", CALLS)
def test_buffers_come_from_the_stream_that_uses_them(no_launch, name):
    CALLS[name](OTHER)
    assert no_launch
    for t in no_launch:
        assert t.made_on is OTHER
        assert CALLER in t.kept_for


@pytest.mark.parametrize("name", CALLS)
def test_buffers_of_the_callers_own_stream(no_launch, name):
    for stream in (None, CALLER):
        CALLS[name](stream)
    assert no_launch and all(t.made_on is CALLER for t in no_launch)
