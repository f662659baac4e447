"""Refusals of the operators of a training step, on the host before any HIP
call; what the binding checks of their tensors; where their outputs' memory
comes from."""
import contextlib
import ctypes
import os
import subprocess
import types

import pytest
import torch

import w4a16_int4_grouped_amd as M
from tests.test_operators_cpu import BAD_GEMM, ODD, OK, L, refused  # noqa: F401
from tests.test_operators_streams_cpu import CALLER, OTHER, Made, Stream
from tests.test_operators_views_cpu import Standin

HALF = ctypes.c_void_p((1 << 20) + 2)
B, F, H16, I, U, Q = torch.bfloat16, torch.float32, torch.float16, torch.int32, torch.uint8, torch.int8

BALANCE = dict(logits=OK, dtype=2, ld=64, T=4, E=64, ids=OK, topk=8, score=0, offsets=OK, S=3, loss=OK, counts=OK, ws=OK,
               ws_bytes=1 << 40)


@pytest.mark.parametrize("kw,word", [
    (dict(logits=None), "logits"), (dict(dtype=3), "dtype"), (dict(ld=63), "logits"), (dict(T=-1), "T ="),
    (dict(T=(1 << 24) + 1), "T ="), (dict(E=0), "E ="), (dict(E=4097, ld=4097), "E ="), (dict(topk=0), "topk"),
    (dict(topk=65, E=128, ld=128), "topk"), (dict(topk=9, E=8), "topk"), (dict(score=2), "score"),
    (dict(logits=HALF), "logits"), (dict(ids=None), "topk_ids"), (dict(ids=HALF), "topk_ids"), (dict(loss=None), "loss"),
    (dict(counts=HALF), "counts"), (dict(S=0), "S ="), (dict(S=(1 << 20) + 1), "S ="),
    (dict(S=1 << 19, E=4096, ld=4096), "S ="), (dict(offsets=None), "offsets"), (dict(offsets=HALF), "offsets"),
    (dict(ws=None), "workspace"), (dict(ws=ODD), "workspace"),
])
def test_balance_refusals(L, kw, word):  # noqa: F811
    refused(L.moe_router_balance(*dict(BALANCE, **kw).values(), None), word)


def test_balance_workspace(L):  # noqa: F811
    need = L.moe_router_balance_bytes(4, 64, 3)
    assert need > 0
    status = L.moe_router_balance(*dict(BALANCE, ws_bytes=need - 1).values(), None)
    assert status == M.MOE_ERR_WORKSPACE_TOO_SMALL and str(need) in M.last_error()
    for bad in ((-1, 64, 1), (1 << 25, 64, 1), (4, 0, 1), (4, 4097, 1), (4, 64, 0), (4, 4096, 1 << 19)):
        assert L.moe_router_balance_bytes(*bad) == -1
    for E, alone in ((8, 64), (512, 64), (513, 32), (1024, 32), (1025, 16), (4096, 16)):     # rows that need no workspace
        assert L.moe_router_balance_bytes(alone, E, 1) == 0 < L.moe_router_balance_bytes(alone + 1, E, 1)
    # of the largest calls: parts of 1024 chunks and each sequence
    assert L.moe_router_balance_bytes(1 << 24, 4096, 1) < 1 << 26


def test_balance_parts_never_meet():
    """Part c + s of chunk c and sequence s: distinct for the pairs that any offsets give, and within chunks + S."""
    import random
    rng = random.Random(1)
    for _ in range(300):
        T, S, chunk = rng.randint(0, 60), rng.randint(1, 12), rng.randint(1, 9)
        off = sorted(rng.randint(0, T) for _ in range(S + 1))
        chunks = (T + chunk - 1) // chunk
        pairs = [(c, s) for c in range(chunks) for s in range(S)
                 if max(off[s], c * chunk) < min(off[s + 1], (c + 1) * chunk, T)]
        parts = [c + s for c, s in pairs]
        assert len(set(parts)) == len(parts) and all(p < chunks + S for p in parts)


BALANCE_GRAD = dict(logits=OK, dtype=2, ld=64, T=4, E=64, topk=8, score=0, offsets=OK, S=3, counts=OK, d_loss=OK, add=None,
                    add_ld=0, d_logits=OK, d_ld=64)


@pytest.mark.parametrize("kw,word", [
    (dict(ld=63), "logits"), (dict(topk=0), "topk"), (dict(counts=None), "counts"), (dict(d_loss=HALF), "d_loss"),
    (dict(d_logits=None), "d_logits"), (dict(d_ld=63), "d_logits"), (dict(add=OK, add_ld=63), "add"),
    (dict(add=HALF, add_ld=64), "add"), (dict(S=0), "S ="), (dict(offsets=None), "offsets"), (dict(score=-1), "score"),
])
def test_balance_gradient_refusals(L, kw, word):  # noqa: F811
    refused(L.moe_router_balance_grad(*dict(BALANCE_GRAD, **kw).values(), None), word)


COMBINE = dict(y=OK, dtype=0, y_ld=64, R=10, H=64, slots=OK, T=4, topk=2, w=OK, out=OK, out_ld=64, out_dtype=0)
SIZES = [(dict(H=0), "H ="), (dict(H=60), "H ="), (dict(H=(1 << 20) + 8), "H ="), (dict(T=-1), "T ="),
         (dict(T=(1 << 24) + 1), "T ="), (dict(topk=0), "topk"), (dict(topk=65), "topk"), (dict(R=-1), "R ="),
         (dict(R=(1 << 30) + 1), "R ="), (dict(dtype=3), "dtype"), (dict(slots=None), "slots"), (dict(slots=HALF), "slots"),
         (dict(w=HALF), "weights"), (dict(y=ODD), "y NULL"), (dict(y_ld=56), "y:"), (dict(y_ld=68), "y:")]


@pytest.mark.parametrize("kw,word", SIZES + [
    (dict(y=None), "y NULL"), (dict(out=None), "out"), (dict(out_ld=60), "out"), (dict(out_dtype=5), "out_dtype"),
])
def test_combine_refusals(L, kw, word):  # noqa: F811
    refused(L.moe_combine(*dict(COMBINE, **kw).values(), None), word)


COMBINE_GRAD = dict(d_out=OK, dtype=0, d_ld=64, T=4, H=64, slots=OK, topk=2, w=OK, y=OK, y_ld=64, row_src=OK, offsets=OK,
                    E=3, d_y=OK, dy_ld=64, R=10, d_w=OK)


@pytest.mark.parametrize("kw,word", SIZES + [
    (dict(d_out=None), "d_out"), (dict(d_ld=60), "d_out"), (dict(d_y=None), "d_y"), (dict(dy_ld=1 << 22), "d_y"),
    (dict(row_src=None), "offsets without"), (dict(row_src=HALF), "row_src"), (dict(offsets=HALF), "offsets"),
    (dict(E=0), "E ="), (dict(E=4097), "E ="), (dict(y=None), "d_w without"), (dict(d_w=HALF), "d_w"),
])
def test_combine_gradient_refusals(L, kw, word):  # noqa: F811
    refused(L.moe_combine_grad(*dict(COMBINE_GRAD, **kw).values(), None), word)


QUANT = dict(x=OK, dtype=0, ld=64, rows=4, K=64, q=OK, scales=OK)


@pytest.mark.parametrize("kw,word", [
    (dict(x=None), "x NULL"), (dict(x=ODD), "x NULL"), (dict(dtype=3), "dtype"), (dict(ld=60), "x:"), (dict(ld=56), "x:"),
    (dict(rows=-1), "rows"), (dict(rows=(1 << 40) + 1, K=8), "rows"), (dict(rows=(1 << 22) + 1, K=1 << 20, ld=1 << 20), "rows"),
    (dict(K=0), "K ="), (dict(K=60), "K ="), (dict(K=(1 << 20) + 8), "K ="), (dict(q=None), "codes"),
    (dict(scales=ODD), "codes"),
])
def test_quant_refusals(L, kw, word):  # noqa: F811
    refused(L.moe_mx8_quant(*dict(QUANT, **kw).values(), None), word)


DEQUANT = dict(q=OK, scales=OK, rows=4, K=64, row_src=OK, topk=2, offsets=OK, E=3, out=OK, dtype=0, ld=64, out_rows=9)


@pytest.mark.parametrize("kw,word", [
    (dict(q=ODD), "codes"), (dict(scales=None), "codes"), (dict(K=60), "K ="), (dict(rows=-1), "rows"),
    (dict(out_rows=-1), "rows"), (dict(out_rows=(1 << 30) + 1), "row_src"), (dict(rows=(1 << 30) + 1), "row_src"),
    (dict(row_src=None), "out_rows"), (dict(row_src=HALF), "row_src"), (dict(topk=0), "topk"), (dict(offsets=HALF), "offsets"),
    (dict(E=0), "E ="), (dict(out=None), "out"), (dict(ld=60), "out"), (dict(dtype=-1), "dtype"),
])
def test_dequant_refusals(L, kw, word):  # noqa: F811
    refused(L.moe_mx8_dequant(*dict(DEQUANT, **kw).values(), None), word)


def test_scale_columns(L):  # noqa: F811
    for K, n in ((8, 16), (32, 16), (512, 16), (520, 32), (7168, 224), (1 << 20, 32768)):
        assert L.moe_mx8_scale_cols(K) == n
    for K in (0, -8, 12, (1 << 20) + 8):
        assert L.moe_mx8_scale_cols(K) == 0


SAVE = dict(h=OK, dtype=0, h_ld=64, rows=4, I=32, offsets=OK, E=3, a=OK, a_ld=32, q=OK, scales=OK)


@pytest.mark.parametrize("kw,word", [
    (dict(h=None), "h NULL"), (dict(h_ld=56), "h:"), (dict(dtype=3), "dtype"), (dict(rows=-1), "rows"),
    (dict(rows=(1 << 30) + 1), "rows"), (dict(I=0), "I ="), (dict(I=12), "I ="), (dict(I=(1 << 19) + 8), "I ="),
    (dict(offsets=HALF), "offsets"), (dict(E=4097), "E ="), (dict(a=ODD), "a NULL"), (dict(a_ld=24), "a:"),
    (dict(q=None), "codes"), (dict(scales=ODD), "codes"),
])
def test_swiglu_save_refusals(L, kw, word):  # noqa: F811
    refused(L.moe_swiglu_save(*dict(SAVE, **kw).values(), None), word)


GRAD = dict(h=OK, h_ld=64, q=None, scales=None, dtype=0, rows=4, I=32, d_a=OK, da_ld=32, offsets=OK, E=3, d_h=OK, dh_ld=64,
            a=OK, a_ld=32)


@pytest.mark.parametrize("kw,word", [
    (dict(h=None), "codes"), (dict(q=OK), "checkpoint"), (dict(h=None, q=OK), "codes"), (dict(h=ODD), "h NULL"),
    (dict(h_ld=56), "h:"), (dict(dtype=3), "dtype"), (dict(rows=-1), "rows"), (dict(I=12), "I ="), (dict(d_a=None), "d_a"),
    (dict(da_ld=24), "d_a"), (dict(d_h=None), "d_h"), (dict(dh_ld=56), "d_h"), (dict(a=ODD), "a NULL"), (dict(a_ld=24), "a:"),
    (dict(offsets=HALF), "offsets"), (dict(E=0), "E ="),
])
def test_swiglu_gradient_refusals(L, kw, word):  # noqa: F811
    refused(L.moe_swiglu_grad(*dict(GRAD, **kw).values(), None), word)


LINEAR = dict(a=OK, a_ld=64, w=OK, w_stride=64 * 64, w_ld=64, dtype=0, offsets=OK, E=4, M=16, N=64, K=64, bias=OK,
              bias_dtype=0, bias_ld=64, act=0, residual=OK, res_ld=64, out=OK, out_ld=64, out_dtype=0)


@pytest.mark.parametrize("kw,word", BAD_GEMM + [
    (dict(bias=ODD), "bias"), (dict(bias_ld=56), "bias"), (dict(bias_ld=68), "bias"), (dict(bias_dtype=3), "bias_dtype"),
    (dict(act=2), "act"), (dict(act=-1), "act"), (dict(act=1, N=56, w_stride=0), "N = 56"), (dict(residual=ODD), "residual"),
    (dict(res_ld=56), "residual"), (dict(act=1, out_ld=24), "out"), (dict(act=1, res_ld=24), "residual"),
])
def test_linear_refusals(L, kw, word):  # noqa: F811
    refused(L.moe_grouped_linear(*dict(LINEAR, **kw).values(), None), word)


BIAS = dict(dy=OK, dy_ld=64, dtype=0, offsets=OK, E=4, M=16, N=64, db=OK, db_ld=64, out_dtype=2, ws=OK, ws_bytes=1 << 30)


@pytest.mark.parametrize("kw,word", [
    (dict(dy=None), "dy"), (dict(dy=ODD), "dy"), (dict(dy_ld=56), "dy"), (dict(dtype=2), "BF16 or FP16"),
    (dict(offsets=None), "offsets"), (dict(E=0), "E ="), (dict(M=-1), "M ="), (dict(N=60), "multiples"), (dict(N=0), "N ="),
    (dict(db=None), "db"), (dict(db_ld=60), "db"), (dict(out_dtype=3), "out_dtype"),
    (dict(E=1, M=24576, ws=None), "workspace"), (dict(E=1, M=24576, ws=ODD), "workspace"),
])
def test_bias_gradient_refusals(L, kw, word):  # noqa: F811
    refused(L.moe_grouped_bias_grad(*dict(BIAS, **kw).values(), None), word)


def test_bias_gradient_workspace(L):  # noqa: F811
    size = L.moe_grouped_bias_grad_bytes
    for E, M_, N in ((48, 24576, 4096), (8, 448, 4096), (16, 8192, 1024), (2, 4096, 7168), (1, 0, 64), (4096, 1 << 30, 8)):
        assert size(E, M_, N) == 0 or M_ == 1 << 30
    for E, M_, N in ((1, 24576, 64), (1, 24576, 4096), (8, 24576, 64), (1, 4096, 512)):
        # a part for each chunk of 256 rows, and for each group one more
        assert size(E, M_, N) == (M_ // 256 + E) * N * 4
    need = size(1, 24576, 64)
    status = L.moe_grouped_bias_grad(*dict(BIAS, E=1, M=24576, ws_bytes=need - 1).values(), None)
    assert status == M.MOE_ERR_WORKSPACE_TOO_SMALL and str(need) in M.last_error()
    for bad in ((0, 1, 8), (4097, 1, 8), (1, -1, 8), (1, (1 << 30) + 1, 8), (1, 1, 4), (1, 1, (1 << 20) + 8)):
        assert size(*bad) == -1


FORM_MAIN = """
#include <cstdio>
#include "moe_ragged_form.h"
int main() {
  moe::FormCall p;
  while (std::scanf("%d %d %d %d", &p.E, &p.M, &p.I, &p.C) == 4) {
    p.mx = p.wgrad = false, p.J = 0, p.out_size = 4;
    std::printf("%d %d\\n", (int)moe::form_of(p), (int)moe::form_of_linear(p));
  }
}
"""


def test_forms_of_the_product_with_an_epilogue(tmp_path):
    """Each case of the GPU test of every form takes the form it is there for; few rows an expert and a long contraction
    take the split one where the plain product's rule would not, and nothing else changes."""
    from tests.test_gpu_y_linear import FORMS
    (tmp_path / "main.cpp").write_text(FORM_MAIN)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", os.path.join(M.PKG_DIR, "csrc"), str(tmp_path / "main.cpp"),
                    "-o", str(tmp_path / "forms")], check=True)

    def forms(calls):
        r = subprocess.run([str(tmp_path / "forms")], input="".join("%d %d %d %d\n" % c for c in calls), capture_output=True,
                           text=True, check=True)
        return [tuple(map(int, line.split())) for line in r.stdout.splitlines()]

    names = ["large", "two", "four", "split", "thin"]
    for (name, *call), (plain, got) in zip(FORMS, forms([tuple(c[1:]) for c in FORMS])):
        if name == "few rows each":
            assert (plain, got) == (0, 3)
        else:
            assert names[got] == name and plain == got, name
    few = [(48, 448, 4096, 7168), (8, 128, 14336, 4096), (384, 3584, 4096, 4096)]
    assert all(f == (0, 3) for f in forms(few))
    more = [(48, 1500, 4096, 7168), (48, 24576, 4096, 7168), (64, 600, 1024, 1024), (384, 4096, 7168, 256)]
    assert all(a == b for a, b in forms(more))


# ---- the binding ----------------------------------------------------------------------


def T(*shape, dtype=B, stride=None):
    return Standin(shape, dtype, stride)


CALLS = {
    "router_balance": lambda s=None: M.router_balance(T(40, 8, dtype=F), T(40, 2, dtype=I), offsets=T(3, dtype=I), stream=s),
    "router_balance_grad": lambda s=None: M.router_balance_grad(T(40, 8, dtype=F), T(2, 8, dtype=I), T(2, dtype=F), 2,
                                                                offsets=T(3, dtype=I), add=T(40, 8, dtype=F), stream=s),
    "combine": lambda s=None: M.combine(T(90, 64), T(40, 2, dtype=I), T(40, 2, dtype=F), stream=s),
    "combine_grad": lambda s=None: M.combine_grad(T(40, 64), T(40, 2, dtype=I), y=T(90, 64), w=T(40, 2, dtype=F),
                                                  row_src=T(90, dtype=I), offsets=T(4, dtype=I), stream=s),
    "mx8_quant": lambda s=None: M.mx8_quant(T(40, 64), stream=s),
    "mx8_dequant": lambda s=None: M.mx8_dequant(T(40, 64, dtype=Q), T(40, 16, dtype=U), row_src=T(80, dtype=I), topk=2,
                                                stream=s),
    "swiglu_save": lambda s=None: M.swiglu_save(T(40, 64), offsets=T(3, dtype=I), stream=s),
    "grouped_linear": lambda s=None: M.grouped_linear(T(40, 64), T(3, 32, 64), T(4, dtype=I), bias=T(3, 32), act="swiglu",
                                                      residual=T(40, 16), stream=s),
    "grouped_bias_grad": lambda s=None: M.grouped_bias_grad(T(40, 64), T(4, dtype=I), stream=s),
    "swiglu_grad": lambda s=None: M.swiglu_grad(T(40, 2, 32, dtype=Q), T(40, 32), scales=T(40, 2, 16, dtype=U), stream=s),
}


class Lib:
    """The library with its launches recorded, not run."""

    def __init__(self):
        self.launched = []

    def __getattr__(self, f):
        if f.endswith("scale_cols"):
            return lambda K: ((K + 31) // 32 + 15) // 16 * 16
        if f.endswith("balance_bytes") or f.endswith("bias_grad_bytes"):
            return lambda *sizes: 4096
        return lambda *args: self.launched.append((f, args)) or M.MOE_OK


@pytest.fixture
def fake(monkeypatch):
    M._load()
    fake_lib = Lib()
    monkeypatch.setattr(M, "_lib", fake_lib)
    monkeypatch.setattr(M, "lib", lambda: fake_lib)
    monkeypatch.setattr(M, "_new", lambda shape, dtype, device, stream: Standin(shape, dtype))
    monkeypatch.setattr(Standin, "device", torch.device("cuda", 0))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0, raising=False)
    caches = (M.mx8_scale_cols, M._balance_bytes, M._bias_grad_bytes)
    for c in caches:
        c.cache_clear()
    yield fake_lib.launched
    for c in caches:
        c.cache_clear()


@pytest.mark.parametrize("name", CALLS)
def test_stream_of_another_device(fake, name):
    with pytest.raises(M.MoeError, match="stream") as e:
        CALLS[name](Stream(7, device_index=1))
    assert e.value.status == M.MOE_ERR_INVALID_ARG
    assert not fake
    CALLS[name](Stream(7, device_index=0))
    assert [f for f, _ in fake] == ["moe_" + name]


BAD = [
    ("balance: ids of another length", lambda: M.router_balance(T(40, 8), T(39, 2, dtype=I))),
    ("balance: ids of another type", lambda: M.router_balance(T(40, 8), T(40, 2, dtype=torch.int64))),
    ("balance: score", lambda: M.router_balance(T(40, 8), T(40, 2, dtype=I), score="tanh")),
    ("balance: offsets of one", lambda: M.router_balance(T(40, 8), T(40, 2, dtype=I), offsets=T(1, dtype=I))),
    ("balance: offsets of another type", lambda: M.router_balance(T(40, 8), T(40, 2, dtype=I), offsets=T(3, dtype=F))),
    ("balance: outputs of another shape", lambda: M.router_balance(T(40, 8), T(40, 2, dtype=I), out=(T(2, dtype=F), T(1, 8, dtype=I)))),
    ("balance: workspace of another type", lambda: M.router_balance(T(40, 8), T(40, 2, dtype=I), ws=T(9999, dtype=Q))),
    ("balance: rows not adjacent", lambda: M.router_balance(T(40, 8, stride=(16, 2)), T(40, 2, dtype=I))),
    ("balance gradient: counts", lambda: M.router_balance_grad(T(40, 8), T(2, 8, dtype=I), T(1, dtype=F), 2)),
    ("balance gradient: d_loss", lambda: M.router_balance_grad(T(40, 8), T(1, 8, dtype=I), T(2, dtype=F), 2)),
    ("balance gradient: add of another type", lambda: M.router_balance_grad(T(40, 8), T(1, 8, dtype=I), T(1, dtype=F), 2,
                                                                           add=T(40, 8, dtype=F))),
    ("balance gradient: topk", lambda: M.router_balance_grad(T(40, 8), T(1, 8, dtype=I), T(1, dtype=F), 0)),
    ("combine: weights of another shape", lambda: M.combine(T(90, 64), T(40, 2, dtype=I), T(40, 3, dtype=F))),
    ("combine: weights of another type", lambda: M.combine(T(90, 64), T(40, 2, dtype=I), T(40, 2))),
    ("combine: output of another width", lambda: M.combine(T(90, 64), T(40, 2, dtype=I), out=T(40, 72))),
    ("combine: slots apart", lambda: M.combine(T(90, 64), T(40, 2, dtype=I, stride=(4, 1)))),
    ("combine gradient: no row count", lambda: M.combine_grad(T(40, 64), T(40, 2, dtype=I))),
    ("combine gradient: y of another width", lambda: M.combine_grad(T(40, 64), T(40, 2, dtype=I), y=T(90, 72))),
    ("combine gradient: y of another type", lambda: M.combine_grad(T(40, 64), T(40, 2, dtype=I), y=T(90, 64, dtype=F))),
    ("combine gradient: row_src of another length", lambda: M.combine_grad(T(40, 64), T(40, 2, dtype=I), y=T(90, 64),
                                                                          row_src=T(91, dtype=I))),
    ("combine gradient: offsets alone", lambda: M.combine_grad(T(40, 64), T(40, 2, dtype=I), y=T(90, 64), offsets=T(4, dtype=I))),
    ("combine gradient: d_w without y", lambda: M.combine_grad(T(40, 64), T(40, 2, dtype=I), out=(T(90, 64), T(40, 2, dtype=F)))),
    ("quant: three dimensions", lambda: M.mx8_quant(T(4, 4, 64))),
    ("quant: codes of another type", lambda: M.mx8_quant(T(40, 64), out=(T(40, 64, dtype=U), T(40, 16, dtype=U)))),
    ("quant: type", lambda: M.mx8_quant(T(40, 64, dtype=torch.float64))),
    ("dequant: scales of another width", lambda: M.mx8_dequant(T(40, 64, dtype=Q), T(40, 32, dtype=U))),
    ("dequant: out of another height", lambda: M.mx8_dequant(T(40, 64, dtype=Q), T(40, 16, dtype=U), row_src=T(80, dtype=I),
                                                             out=T(40, 64))),
    ("dequant: topk", lambda: M.mx8_dequant(T(40, 64, dtype=Q), T(40, 16, dtype=U), row_src=T(80, dtype=I), topk=0)),
    ("linear: act", lambda: M.grouped_linear(T(40, 64), T(3, 32, 64), T(4, dtype=I), act="gelu")),
    ("linear: bias of another width", lambda: M.grouped_linear(T(40, 64), T(3, 32, 64), T(4, dtype=I), bias=T(3, 16), act="swiglu")),
    ("linear: bias of another type", lambda: M.grouped_linear(T(40, 64), T(3, 32, 64), T(4, dtype=I), bias=T(3, 32, dtype=I))),
    ("linear: residual of another type", lambda: M.grouped_linear(T(40, 64), T(3, 32, 64), T(4, dtype=I), residual=T(40, 32, dtype=F))),
    ("linear: residual of another width", lambda: M.grouped_linear(T(40, 64), T(3, 32, 64), T(4, dtype=I), residual=T(40, 32), act="swiglu")),
    ("linear: out of another width", lambda: M.grouped_linear(T(40, 64), T(3, 32, 64), T(4, dtype=I), out=T(40, 32), act="swiglu")),
    ("linear: columns", lambda: M.grouped_linear(T(40, 72), T(3, 32, 64), T(4, dtype=I))),
    ("bias gradient: no offsets", lambda: M.grouped_bias_grad(T(40, 64), None)),
    ("bias gradient: out of another height", lambda: M.grouped_bias_grad(T(40, 64), T(4, dtype=I), out=T(4, 64))),
    ("bias gradient: workspace", lambda: M.grouped_bias_grad(T(40, 64), T(4, dtype=I), ws=T(9999, dtype=F))),
    ("save: odd width", lambda: M.swiglu_save(T(40, 63))),
    ("save: codes in two dimensions", lambda: M.swiglu_save(T(40, 64), out=(T(40, 32), T(40, 64, dtype=Q), T(40, 2, 16, dtype=U)))),
    ("gradient: h of another type", lambda: M.swiglu_grad(T(40, 64, dtype=H16), T(40, 32))),
    ("gradient: h of another width", lambda: M.swiglu_grad(T(40, 72), T(40, 32))),
    ("gradient: codes as values", lambda: M.swiglu_grad(T(40, 2, 32, dtype=Q), T(40, 32))),
    ("gradient: values with scales", lambda: M.swiglu_grad(T(40, 64), T(40, 32), scales=T(40, 2, 16, dtype=U))),
]


@pytest.mark.parametrize("call", [c for _, c in BAD], ids=[n for n, _ in BAD])
def test_binding_refusals(fake, call):
    with pytest.raises(M.MoeError) as e:
        call()
    assert e.value.status == M.MOE_ERR_INVALID_ARG
    assert not fake


def test_sizes_past_31_bits_are_refused(fake):
    big = 1 << 31
    for call in (lambda: M.router_balance(T(big, 8), T(big, 2, dtype=I)), lambda: M.combine(T(big, 64), T(40, 2, dtype=I)),
                 lambda: M.combine_grad(T(40, 64), T(40, 2, dtype=I), y=T(big, 64)), lambda: M.swiglu_save(T(big, 64)),
                 lambda: M.mx8_dequant(T(40, 64, dtype=Q), T(40, 16, dtype=U), row_src=T(big, dtype=I)),
                 lambda: M.swiglu_grad(T(big, 64), T(big, 32))):
        with pytest.raises(M.MoeError, match="2\\^31"):
            call()
    assert not fake


def test_outputs_come_from_the_launch_streams_memory(monkeypatch):
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

    stand_in = types.SimpleNamespace(
        empty=empty, cuda=types.SimpleNamespace(stream=stream, current_stream=lambda device=None: now[-1]),
        **{n: getattr(torch, n) for n in ("bfloat16", "float16", "float32", "int32", "uint8", "int8")})
    M._load()
    monkeypatch.setattr(M, "_torch", stand_in)
    monkeypatch.setattr(M, "_call", lambda fn, device, stream, *args: None)
    monkeypatch.setattr(M, "_lib", Lib())
    monkeypatch.setattr(M, "lib", lambda: M._lib)
    caches = (M.mx8_scale_cols, M._balance_bytes, M._bias_grad_bytes)
    for c in caches:
        c.cache_clear()
    for name, call in CALLS.items():
        outputs.clear()
        call(OTHER)
        assert outputs and all(t.made_on is OTHER and t.kept_for == [CALLER] for t in outputs), name
        outputs.clear()
        call(None)
        assert outputs and all(t.made_on is CALLER and not t.kept_for for t in outputs), name
    for c in caches:
        c.cache_clear()
