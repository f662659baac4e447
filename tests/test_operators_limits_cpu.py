"""The largest sizes that the header documents for the operators: one more is
refused on the host, before any HIP call."""
import os
import re

import pytest

import w4a16_int4_grouped_amd as M
from tests.test_operators_cpu import GEMM, OK, ROUTER, L, refused  # noqa: F401

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe_w4a16.h")


def comment_before(name):
    """The comment above a declaration (the group's comment above the first)."""
    text = open(HEADER).read()
    at = re.search(r"\b%s\(" % name, text).start()
    return re.sub(r"\n \* *", " ", re.findall(r"/\*.*?\*/", text[:at], flags=re.S)[-1])


@pytest.mark.parametrize("name,limit", [
    ("moe_router_topk", "T 0..2^24, E 1..4096, topk 1..min(E, 64)"), ("moe_router_topk_grad", "as moe_router_topk"),
    ("moe_grouped_gemm", "multiples of 8 up to 2^20, M at most 2^30, E 1..4096"),
    ("moe_mx_quant", "rows at most 2^40, rows * K at most 2^42"), ("moe_mx_dequant", "as moe_mx_quant"),
])
def test_the_header_names_them(name, limit):
    assert limit in comment_before(name)


def test_one_more_is_refused(L):  # noqa: F811
    refused(L.moe_router_topk(*dict(ROUTER, T=(1 << 24) + 1).values(), None), "T =")
    grad = dict(logits=OK, dtype=2, ld=64, T=(1 << 24) + 1, E=64, topk=8, score=0, renorm=1, scale=1.0, ids=OK, dw=OK,
                dl=OK, d_ld=64)
    refused(L.moe_router_topk_grad(*grad.values(), None), "T =")
    refused(L.moe_grouped_gemm(*dict(GEMM, M=(1 << 30) + 1).values(), None), "M =")
    refused(L.moe_grouped_gemm(*dict(GEMM, N=(1 << 20) + 8).values(), None), "multiples")
    refused(L.moe_grouped_gemm(*dict(GEMM, K=(1 << 20) + 8).values(), None), "multiples")
    for rows, K in (((1 << 40) + 1, 32), ((1 << 37) + 1, 32), ((1 << 22) + 1, 1 << 20)):
        refused(L.moe_mx_quant(OK, 0, K, rows, K, OK, OK, None), "rows")
        refused(L.moe_mx_dequant(OK, OK, rows, K, OK, 0, K, None), "rows")
    assert M.last_error()
