"""Refusals of the operators, on the host before any HIP call."""
import ctypes

import pytest
import torch

import w4a16_int4_grouped_amd as M

OK = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(M.LIB_PATH):
        from w4a16_int4_grouped_amd import build
        build.build()
    return M.lib()


def refused(status, word):
    assert status == M.MOE_ERR_INVALID_ARG
    assert word in M.last_error(), M.last_error()


ROUTER = dict(logits=OK, dtype=2, ld=64, T=4, E=64, topk=8, score=0, bias=None, renorm=1, scale=1.0, ids=OK, w=OK)


@pytest.mark.parametrize("kw,word", [
    (dict(logits=None), "logits"), (dict(dtype=3), "dtype"), (dict(ld=63), "logits"), (dict(T=-1), "T ="),
    (dict(E=0), "E ="), (dict(E=4097, ld=4097), "E ="), (dict(topk=0), "topk"), (dict(topk=65, E=128, ld=128), "topk"),
    (dict(topk=9, E=8), "topk"), (dict(score=2), "score"), (dict(ids=None), "topk_ids"), (dict(w=None), "topk_ids"),
    (dict(logits=ctypes.c_void_p((1 << 20) + 2)), "logits"), (dict(bias=ctypes.c_void_p(3)), "bias"),
])
def test_router_refusals(L, kw, word):
    a = dict(ROUTER, **kw)
    refused(L.moe_router_topk(*a.values(), None), word)


@pytest.mark.parametrize("kw,word", [
    (dict(ld=63), "logits"), (dict(topk=0), "topk"), (dict(ids=None), "topk_ids"), (dict(dw=None), "d_topk_w"),
    (dict(dl=None), "d_logits"), (dict(d_ld=63), "d_logits"), (dict(score=-1), "score"),
])
def test_router_gradient_refusals(L, kw, word):
    a = dict(logits=OK, dtype=2, ld=64, T=4, E=64, topk=8, score=0, renorm=1, scale=1.0, ids=OK, dw=OK, dl=OK, d_ld=64)
    a.update(kw)
    refused(L.moe_router_topk_grad(*a.values(), None), word)


GEMM = dict(a=OK, a_ld=64, w=OK, w_stride=64 * 64, w_ld=64, dtype=0, offsets=OK, E=4, M=16, N=64, K=64, out=OK,
            out_ld=64, out_dtype=0)
BAD_GEMM = [
    (dict(a=None), "NULL"), (dict(a=ODD), "aligned"), (dict(w=ODD), "w NULL"), (dict(out=None), "out"),
    (dict(a_ld=56), "values from row to row"), (dict(a_ld=68), "multiple of 8"), (dict(w_ld=1 << 22), "row to row"),
    (dict(w_stride=12), "experts"), (dict(w_stride=-8), "experts"), (dict(dtype=2), "BF16 or FP16"),
    (dict(out_dtype=3), "out_dtype"), (dict(offsets=None), "offsets"), (dict(E=0), "E ="), (dict(E=4097), "E ="),
    (dict(M=-1), "M ="), (dict(M=(1 << 30) + 1), "M ="), (dict(N=0), "N ="), (dict(N=60), "multiples"),
    (dict(K=4), "multiples"), (dict(out_ld=60), "out"),
]


@pytest.mark.parametrize("kw,word", BAD_GEMM)
def test_grouped_gemm_refusals(L, kw, word):
    refused(L.moe_grouped_gemm(*dict(GEMM, **kw).values(), None), word)
    if "a" not in kw and "a_ld" not in kw:      # the input gradient takes its arguments in the same order
        refused(L.moe_grouped_gemm_dgrad(*dict(GEMM, **kw).values(), None), "da" if word == "out" else word)


@pytest.mark.parametrize("kw,word", [
    (dict(dy=ODD), "dy"), (dict(a=None), "a NULL"), (dict(dw=None), "dw"), (dict(dw_ld=56), "dw"),
    (dict(dw_stride=64 * 63), "overlap"), (dict(dw_stride=64 * 64 + 4), "multiple of 8"), (dict(K=20), "multiples"),
    (dict(dtype=2), "BF16"), (dict(M=-3), "M ="),
])
def test_weight_gradient_refusals(L, kw, word):
    a = dict(dy=OK, dy_ld=64, a=OK, a_ld=64, dtype=0, offsets=OK, E=4, M=16, N=64, K=64, dw=OK, dw_stride=64 * 64,
             dw_ld=64, out_dtype=2)
    a.update(kw)
    refused(L.moe_grouped_gemm_wgrad(*a.values(), None), word)


@pytest.mark.parametrize("K,cols", [(32, 16), (512, 16), (544, 32), (7168, 224), (0, 0), (48, 0), (-32, 0),
                                    ((1 << 20) + 32, 0)])
def test_mx_scale_cols(L, K, cols):
    assert L.moe_mx_scale_cols(K) == cols


@pytest.mark.parametrize("kw,word", [
    (dict(x=ODD), "aligned"), (dict(dtype=5), "dtype"), (dict(ld=56), "values"), (dict(ld=68), "values"),
    (dict(rows=-1), "rows"), (dict(K=48), "K ="), (dict(q=None), "codes"), (dict(s=ODD), "codes"),
    (dict(rows=1 << 41), "rows"),
])
def test_mx_quant_refusals(L, kw, word):
    a = dict(x=OK, dtype=0, ld=64, rows=3, K=64, q=OK, s=OK)
    a.update(kw)
    refused(L.moe_mx_quant(*a.values(), None), word)
    refused(L.moe_mx_dequant(a["q"], a["s"], a["rows"], a["K"], a["x"], a["dtype"], a["ld"], None), word)


@pytest.mark.parametrize("kw,word", [
    (dict(aq=None), "a: codes"), (dict(a_s=ODD), "a: codes"), (dict(wq=ODD), "w: codes"), (dict(w_s=None), "w: codes"),
    (dict(K=48), "multiples"), (dict(N=12), "multiples"), (dict(out_ld=32), "out"), (dict(out_dtype=-1), "out_dtype"),
    (dict(offsets=None), "offsets"), (dict(E=0), "E ="), (dict(M=-1), "M ="),
])
def test_mx_gemm_refusals(L, kw, word):
    a = dict(aq=OK, a_s=OK, wq=OK, w_s=OK, offsets=OK, E=4, M=16, N=64, K=64, out=OK, out_ld=64, out_dtype=0)
    a.update(kw)
    refused(L.moe_mx_grouped_gemm(*a.values(), None), word)


def test_empty_calls_enqueue_nothing(L):
    assert L.moe_router_topk(*dict(ROUTER, T=0, logits=None, ids=None, w=None).values(), None) == M.MOE_OK
    assert L.moe_grouped_gemm(*dict(GEMM, M=0, a=None, out=None).values(), None) == M.MOE_OK
    assert L.moe_mx_quant(None, 0, 64, 0, 64, None, None, None) == M.MOE_OK


def test_binding_refuses_host_tensors_and_bad_shapes():
    a, w, off = torch.zeros(4, 64).bfloat16(), torch.zeros(2, 8, 64).bfloat16(), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(M.MoeError, match="not on a GPU"):
        M.grouped_gemm(a, w, off)
    with pytest.raises(M.MoeError, match="columns"):
        M.grouped_gemm(a[:, :32], w, off)
    with pytest.raises(M.MoeError, match="not on a GPU"):
        M.router_topk(torch.zeros(2, 8), 2)
    with pytest.raises(M.MoeError, match="not on a GPU"):
        M.mx_quant(a)
    with pytest.raises(M.MoeError, match="dy"):
        M.grouped_gemm_wgrad(a, a[:2], off)
    with pytest.raises(M.MoeError, match="K ="):
        M.mx_scale_cols(40)


def test_references_of_the_tests_agree_with_hand_worked_values():
    """The 64-bit quantiser used as reference, on values worked by hand."""
    from tests.ops_util import mx_reference, mx_values
    x = torch.zeros(1, 32)
    x[0, :8] = torch.tensor([6.0, 5.0, 3.5, 2.5, 0.25, 0.75, -7.0, 0.2])
    val, byte = mx_reference(x)
    assert byte.tolist() == [[127]]                 # floor(log2 7) - 2 = 0
    assert val[0, :8].tolist() == [6.0, 4.0, 4.0, 2.0, 0.0, 1.0, -6.0, 0.0]
    x = torch.full((1, 32), 1.0)
    assert mx_reference(x)[1].tolist() == [[125]]    # 1 = 4 * 2^-2
    assert mx_values(torch.full((1, 16), 0x66, dtype=torch.uint8), torch.tensor([[125]], dtype=torch.uint8)).eq(1).all()
