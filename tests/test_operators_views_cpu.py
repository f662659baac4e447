"""Views and sizes that the operators' bindings have to refuse, with stand-ins
for GPU tensors: the library refuses them before any HIP call, or the binding
does."""
import math

import pytest
import torch

import w4a16_int4_grouped_amd as M


class Standin:
    """What the binding asks of a GPU tensor, without memory behind it."""
    is_cuda = True
    device = torch.device("cpu")

    def __init__(self, shape, dtype, stride=None):
        dense, n = [], 1
        for s in reversed(shape):
            dense.insert(0, n)
            n *= s
        self.shape, self.dtype, self._stride = torch.Size(shape), dtype, tuple(stride or dense)
        self._dense = self._stride == tuple(dense)

    def dim(self):
        return len(self.shape)

    def stride(self, d=None):
        return self._stride if d is None else self._stride[d]

    def is_contiguous(self):
        return self._dense

    def numel(self):
        return math.prod(self.shape)

    def data_ptr(self):
        return 1 << 20


@pytest.fixture(autouse=True)
def no_gpu(monkeypatch):
    import os
    if not os.path.exists(M.LIB_PATH):
        from w4a16_int4_grouped_amd import build
        build.build()

    def call(fn, device, stream, *args):
        M.check(fn(*args, None))
    monkeypatch.setattr(M, "_call", call)
    # outputs: none may be made for a size that is refused
    monkeypatch.setattr(M, "_new", lambda shape, dtype, device, stream: Standin(shape, dtype))


def refused(f, *a, **kw):
    with pytest.raises(M.MoeError) as e:
        f(*a, **kw)
    assert e.value.status == M.MOE_ERR_INVALID_ARG, e.value


B, F, I = torch.bfloat16, torch.float32, torch.int32


@pytest.mark.parametrize("stride", [(0, 1), (4, 1)])     # one row for all, rows that overlap
def test_rows_closer_than_their_width(stride):
    view = Standin((6, 64), B, stride)
    ids, w = Standin((6, 4), I), Standin((6, 4), F)
    refused(M.router_topk, view, 4)
    refused(M.router_topk_grad, view, ids, w)
    refused(M.router_topk_grad, Standin((6, 64), B), ids, w, out=view)
    off, w3 = Standin((3,), I), Standin((2, 32, 64), B)
    refused(M.grouped_gemm, view, w3, off)
    refused(M.grouped_gemm, Standin((6, 64), B), Standin((2, 64, 64), B), off, out=view)
    refused(M.grouped_gemm_dgrad, view, Standin((2, 64, 32), B), off)
    refused(M.grouped_gemm_wgrad, view, Standin((6, 32), B), off)
    refused(M.mx_quant, view)
    refused(M.mx_dequant, Standin((6, 32), torch.uint8), Standin((6, 16), torch.uint8), out=view)


BIG = (1 << 32) + 2     # 2 in 32 bits


def test_sizes_past_32_bits():
    ids, w = Standin((BIG, 1), I), Standin((BIG, 1), F)
    refused(M.router_topk, Standin((BIG, 8), B), 1)
    refused(M.router_topk, Standin((2, BIG), B), 1)
    refused(M.router_topk, Standin((2, 8), B), BIG)
    refused(M.router_topk_grad, Standin((BIG, 8), B), ids, w)
    refused(M.router_topk_grad, Standin((2, BIG), B), Standin((2, 1), I), Standin((2, 1), F))
    off, wide = Standin((3,), I), (1 << 32) + 64
    refused(M.grouped_gemm, Standin((BIG, 64), B), Standin((2, 32, 64), B), off)
    refused(M.grouped_gemm, Standin((2, wide), B, (64, 1)), Standin((2, 32, wide), B, (2048, 64, 1)), off)
    refused(M.grouped_gemm, Standin((2, 64), B), Standin((2, wide, 64), B), off, out=Standin((2, wide), B, (64, 1)))
    refused(M.grouped_gemm_dgrad, Standin((BIG, 64), B), Standin((2, 64, 32), B), off)
    refused(M.grouped_gemm_wgrad, Standin((BIG, 64), B), Standin((BIG, 32), B), off)
    refused(M.mx_scale_cols, (1 << 32) + 32)
    refused(M.mx_quant, Standin((2, (1 << 32) + 32), B, (32, 1)))
    u8 = torch.uint8
    refused(M.mx_grouped_gemm, Standin((BIG, 32), u8), Standin((BIG, 16), u8), Standin((2, 8, 32), u8),
            Standin((2, 8, 16), u8), off)
    refused(M.mx_grouped_gemm, Standin((2, 32), u8), Standin((2, 16), u8), Standin((2, BIG + 6, 32), u8),
            Standin((2, BIG + 6, 16), u8), off)
