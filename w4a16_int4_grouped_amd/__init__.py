"""W4A16 mixture-of-experts expert layer for MI355X (gfx950).

Python binding of ``libmoe_w4a16.so`` (declared in include/moe_w4a16.h).
This module only marshals arguments: every step of the layer runs in the
library's HIP kernels. PyTorch supplies device memory and streams. There is
no CPU fallback: if the library is not built, every call raises.

Low-level names mirror the C ABI (``moe_prepare_weights``, ``moe_align``,
``moe_w4a16_indexed``, ...). ``PreparedWeights`` wraps a handle with
torch-tensor conveniences.
"""
from __future__ import annotations

import ctypes
import functools
import os

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
# the in-tree build of csrc/ (w4a16_int4_grouped_amd/build.py); no other library stands in for it
LIB_PATH = os.path.join(PKG_DIR, "libmoe_w4a16.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED_SCHEMA = 2
MOE_ERR_MODE_MISMATCH = 3
MOE_ERR_OVERRIDE_REJECTED = 4
MOE_ERR_WORKSPACE_TOO_SMALL = 5
MOE_ERR_HIP = 6
MOE_ERR_ROUTING_MISMATCH = 7

MOE_MODE_INDEXED = 0
MOE_MODE_CONTIGUOUS = 1
MOE_MODE_MASKED = 2
MODES = {"indexed": MOE_MODE_INDEXED, "contiguous": MOE_MODE_CONTIGUOUS, "masked": MOE_MODE_MASKED}

# bytes of the fixed device scratch array behind moe_w4a16_indexed_noalloc
NOALLOC_SCRATCH_BYTES = 128 << 20

MOE_SCALE_BF16 = 1
MOE_DTYPE_BF16, MOE_DTYPE_F16, MOE_DTYPE_F32 = 0, 1, 2
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_ACT_NONE, MOE_ACT_SWIGLU = 0, 1
ACTS = {"none": MOE_ACT_NONE, "swiglu": MOE_ACT_SWIGLU}
SCORES = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}
MOE_PACK_INT32_LOW_NIBBLE_FIRST_K = 1

EXPORTS = [
    "moe_abi_version", "moe_last_error", "moe_status_string", "moe_prepared_bytes",
    "moe_prepare_weights", "moe_release_weights", "moe_plan_create", "moe_routing_block", "moe_routing_bytes",
    "moe_routing_layout", "moe_align", "moe_align_ep", "moe_permute", "moe_workspace_bytes", "moe_w4a16_indexed",
    "moe_w4a16_indexed_noalloc", "moe_w4a16_contiguous", "moe_w4a16_masked", "moe_w4a16_gate_up", "moe_w4a16_down", "moe_swiglu",
    "moe_dequant_weights", "moe_describe",
    "moe_router_topk", "moe_router_topk_grad", "moe_grouped_gemm", "moe_grouped_gemm_dgrad", "moe_grouped_gemm_wgrad",
    "moe_mx_scale_cols", "moe_mx_quant", "moe_mx_dequant", "moe_mx_grouped_gemm",
    "moe_profile_enable", "moe_profile_reset", "moe_profile_read",
    "moe_router_balance_bytes", "moe_router_balance", "moe_router_balance_grad", "moe_combine", "moe_combine_grad",
    "moe_mx8_scale_cols", "moe_mx8_quant", "moe_mx8_dequant", "moe_swiglu_save", "moe_swiglu_grad",
    "moe_grouped_linear", "moe_grouped_bias_grad_bytes", "moe_grouped_bias_grad",
]


class WeightDesc(ctypes.Structure):
    _fields_ = [("num_experts", ctypes.c_int32), ("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("bits", ctypes.c_int32), ("group_size", ctypes.c_int32), ("zero_point", ctypes.c_int32),
                ("scale_dtype", ctypes.c_int32), ("pack_order", ctypes.c_int32), ("mode", ctypes.c_int32)]


def make_desc(E, H, I, mode="indexed", bits=4, group_size=32, zero_point=8,
              scale_dtype=MOE_SCALE_BF16, pack_order=MOE_PACK_INT32_LOW_NIBBLE_FIRST_K) -> WeightDesc:
    return WeightDesc(E, H, I, bits, group_size, zero_point, scale_dtype, pack_order,
                      MODES[mode] if isinstance(mode, str) else int(mode))


class Tuning(ctypes.Structure):
    _fields_ = [("block_m", ctypes.c_int32), ("schedule", ctypes.c_int32),
                ("dispatch", ctypes.c_int32), ("global_experts", ctypes.c_int32)]


class RoutingLayout(ctypes.Structure):
    _fields_ = [("block", ctypes.c_int32), ("cap", ctypes.c_int32), ("nblocks", ctypes.c_int32),
                ("sentinel", ctypes.c_int32), ("off_header", ctypes.c_int64),
                ("off_counts", ctypes.c_int64), ("off_offsets", ctypes.c_int64),
                ("off_sorted", ctypes.c_int64), ("off_block_expert", ctypes.c_int64),
                ("off_slot_of", ctypes.c_int64), ("off_scratch", ctypes.c_int64), ("total_ints", ctypes.c_int64)]


class MoeError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"{_STATUS.get(status, status)}: {msg}")
        self.status = status


_STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED_SCHEMA",
           3: "MOE_ERR_MODE_MISMATCH", 4: "MOE_ERR_OVERRIDE_REJECTED",
           5: "MOE_ERR_WORKSPACE_TOO_SMALL", 6: "MOE_ERR_HIP", 7: "MOE_ERR_ROUTING_MISMATCH"}

_lib = None


def lib() -> ctypes.CDLL:
    """Load the HIP library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m w4a16_int4_grouped_amd.build`"
                           " (there is no CPU fallback)")
    L = ctypes.CDLL(LIB_PATH)
    P, I32, I64, SZ, S = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
    F32 = ctypes.c_float
    sig = {
        "moe_abi_version": (S, []),
        "moe_last_error": (ctypes.c_char_p, []),
        "moe_status_string": (ctypes.c_char_p, [S]),
        "moe_prepared_bytes": (SZ, [ctypes.POINTER(WeightDesc)]),
        "moe_prepare_weights": (S, [ctypes.POINTER(WeightDesc), P, P, P, P, P, SZ, P, ctypes.POINTER(P)]),
        "moe_release_weights": (None, [P]),
        "moe_plan_create": (P, [ctypes.POINTER(WeightDesc)]),
        "moe_routing_block": (I32, [P, I32, I32, ctypes.POINTER(Tuning)]),
        "moe_routing_bytes": (SZ, [P, I32, I32, ctypes.POINTER(Tuning)]),
        "moe_routing_layout": (S, [P, I32, I32, ctypes.POINTER(Tuning), ctypes.POINTER(RoutingLayout)]),
        "moe_align": (S, [P, P, I32, I32, ctypes.POINTER(Tuning), P, SZ, P]),
        "moe_align_ep": (S, [P, P, I32, I32, P, I32, ctypes.POINTER(Tuning), P, SZ, P]),
        "moe_permute": (S, [P, P, I32, I32, ctypes.POINTER(Tuning), P, P, P, P, P]),
        "moe_workspace_bytes": (SZ, [P, I32, I32, I32, I32, ctypes.POINTER(Tuning)]),
        "moe_w4a16_indexed": (S, [P, P, I32, I32, P, P, P, P, P, SZ, ctypes.POINTER(Tuning), P]),
        "moe_w4a16_indexed_noalloc": (S, [P, P, I32, I32, P, P, P, ctypes.POINTER(Tuning), P]),
        "moe_w4a16_contiguous": (S, [P, P, I32, P, P, P, I32, I32, P, P, SZ, ctypes.POINTER(Tuning), P]),
        "moe_w4a16_masked": (S, [P, P, I32, P, I32, P, P, SZ, ctypes.POINTER(Tuning), P]),
        "moe_w4a16_gate_up": (S, [P, P, I32, I32, P, P, ctypes.POINTER(Tuning), P]),
        "moe_w4a16_down": (S, [P, P, I32, I32, P, P, ctypes.POINTER(Tuning), P]),
        "moe_swiglu": (S, [P, I64, I32, P, P]),
        "moe_dequant_weights": (S, [P, I32, I32, P, P]),
        "moe_describe": (S, [P, I32, I32, I32, I32, ctypes.POINTER(Tuning), ctypes.c_char_p, SZ]),
        "moe_router_topk": (S, [P, I32, I64, I32, I32, I32, I32, P, I32, F32, P, P, P]),
        "moe_router_topk_grad": (S, [P, I32, I64, I32, I32, I32, I32, I32, F32, P, P, P, I64, P]),
        "moe_grouped_gemm": (S, [P, I64, P, I64, I64, I32, P, I32, I32, I32, I32, P, I64, I32, P]),
        "moe_grouped_gemm_dgrad": (S, [P, I64, P, I64, I64, I32, P, I32, I32, I32, I32, P, I64, I32, P]),
        "moe_grouped_gemm_wgrad": (S, [P, I64, P, I64, I32, P, I32, I32, I32, I32, P, I64, I64, I32, P]),
        "moe_mx_scale_cols": (I32, [I32]),
        "moe_mx_quant": (S, [P, I32, I64, I64, I32, P, P, P]),
        "moe_mx_dequant": (S, [P, P, I64, I32, P, I32, I64, P]),
        "moe_mx_grouped_gemm": (S, [P, P, P, P, P, I32, I32, I32, I32, P, I64, I32, P]),
        "moe_router_balance_bytes": (I64, [I32, I32, I32]),
        "moe_router_balance": (S, [P, I32, I64, I32, I32, P, I32, I32, P, I32, P, P, P, SZ, P]),
        "moe_router_balance_grad": (S, [P, I32, I64, I32, I32, I32, I32, P, I32, P, P, P, I64, P, I64, P]),
        "moe_combine": (S, [P, I32, I64, I32, I32, P, I32, I32, P, P, I64, I32, P]),
        "moe_combine_grad": (S, [P, I32, I64, I32, I32, P, I32, P, P, I64, P, P, I32, P, I64, I32, P, P]),
        "moe_mx8_scale_cols": (I32, [I32]),
        "moe_mx8_quant": (S, [P, I32, I64, I64, I32, P, P, P]),
        "moe_mx8_dequant": (S, [P, P, I64, I32, P, I32, P, I32, P, I32, I64, I64, P]),
        "moe_swiglu_save": (S, [P, I32, I64, I32, I32, P, I32, P, I64, P, P, P]),
        "moe_grouped_linear": (S, [P, I64, P, I64, I64, I32, P, I32, I32, I32, I32, P, I32, I64, I32, P, I64, P, I64, I32,
                                   P]),
        "moe_grouped_bias_grad_bytes": (I64, [I32, I32, I32]),
        "moe_grouped_bias_grad": (S, [P, I64, I32, P, I32, I32, I32, P, I64, I32, P, SZ, P]),
        "moe_swiglu_grad": (S, [P, I64, P, P, I32, I32, I32, P, I64, P, I32, P, I64, P, I64, P]),
        "moe_profile_enable": (S, [S]),
        "moe_profile_reset": (None, []),
        "moe_profile_read": (S, [ctypes.c_char_p, SZ]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _lib = L
    return L


def last_error() -> str:
    return lib().moe_last_error().decode()


def check(status: int) -> None:
    if status != MOE_OK:
        raise MoeError(status, last_error())


# ---------------------------------------------------------------------------
# torch plumbing (device memory and streams only)
# ---------------------------------------------------------------------------

_torch = None
_CODES = None       # torch dtype -> MOE_DTYPE_*


def _load():
    global _torch, _CODES
    import torch
    _CODES = {torch.bfloat16: MOE_DTYPE_BF16, torch.float16: MOE_DTYPE_F16, torch.float32: MOE_DTYPE_F32}
    _torch = torch
    return torch


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else (_torch or _load()).cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _tuning(ovr):
    if ovr is None:
        return None
    if isinstance(ovr, Tuning):
        return ctypes.byref(ovr)
    return ctypes.byref(Tuning(int(ovr.get("block_m", 0)), int(ovr.get("schedule", 0)),
                               int(ovr.get("dispatch", 0)), int(ovr.get("global_experts", 0))))


def _new(shape, dtype, device, stream):
    """A buffer of a call. For a stream other than the current one it is made
    on that stream, because memory freed on the current one may still be in use
    by what is queued there, and kept from reuse until both are done with it."""
    torch = _torch or _load()
    if stream is not None:
        current = torch.cuda.current_stream(device)
        if stream.cuda_stream != current.cuda_stream:
            with torch.cuda.stream(stream):
                t = torch.empty(*shape, dtype=dtype, device=device)
            t.record_stream(current)
            return t
    return torch.empty(*shape, dtype=dtype, device=device)   # a tuple is read 0.1 us slower


def _empty(nbytes, device, stream):
    """A workspace."""
    return _new((max(int(nbytes), 1),), (_torch or _load()).uint8, device, stream)


class PreparedWeights:
    """A prepared-weight handle plus the device buffer it lives in.

    w13_q int32 [E, 2I, H/8], w13_s bf16 [E, 2I, H/32], w2_q int32 [E, H, I/8],
    w2_s bf16 [E, H, I/32], all on one GPU.
    """

    def __init__(self, w13_q, w13_s, w2_q, w2_s, mode="indexed", stream=None):
        import torch
        E, N13, _ = w13_q.shape
        H = w2_q.shape[1]
        I = N13 // 2
        self.E, self.H, self.I = E, H, I
        self.mode = MODES[mode] if isinstance(mode, str) else int(mode)
        self.device = w13_q.device
        desc = make_desc(E, H, I, self.mode)
        L = lib()
        nbytes = L.moe_prepared_bytes(ctypes.byref(desc))
        if nbytes == 0:
            raise MoeError(MOE_ERR_UNSUPPORTED_SCHEMA, last_error())
        self.buffer = _new((nbytes,), torch.uint8, self.device, stream)
        h = ctypes.c_void_p()
        check(L.moe_prepare_weights(ctypes.byref(desc), _ptr(w13_q), _ptr(w13_s), _ptr(w2_q), _ptr(w2_s),
                                    _ptr(self.buffer), nbytes, _stream(stream), ctypes.byref(h)))
        self.handle = h

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and _lib is not None:
            _lib.moe_release_weights(h)
            self.handle = None

    # -- routing ------------------------------------------------------------
    def routing_layout(self, T, topk, ovr=None) -> RoutingLayout:
        out = RoutingLayout()
        check(lib().moe_routing_layout(self.handle, T, topk, _tuning(ovr), ctypes.byref(out)))
        return out

    def align(self, topk_ids, ovr=None, routing=None, stream=None):
        import torch
        T, topk = topk_ids.shape
        nbytes = lib().moe_routing_bytes(self.handle, T, topk, _tuning(ovr))
        if nbytes == 0:
            check(MOE_ERR_INVALID_ARG)
        if routing is None:
            routing = _new((nbytes // 4,), torch.int32, self.device, stream)
        check(lib().moe_align(self.handle, _ptr(topk_ids), T, topk, _tuning(ovr), _ptr(routing),
                              routing.numel() * routing.element_size(), _stream(stream)))
        return routing

    def align_ep(self, topk_ids, expert_map, num_global_experts, ovr=None, routing=None, stream=None):
        """Routing of this handle's share of num_global_experts experts:
        expert_map[global id] = local expert or -1."""
        import torch
        T, topk = topk_ids.shape
        nbytes = lib().moe_routing_bytes(self.handle, T, topk, _tuning(ovr))
        if nbytes == 0:
            check(MOE_ERR_INVALID_ARG)
        if routing is None:
            routing = _new((nbytes // 4,), torch.int32, self.device, stream)
        check(lib().moe_align_ep(self.handle, _ptr(topk_ids), T, topk, _ptr(expert_map), num_global_experts,
                                 _tuning(ovr), _ptr(routing), routing.numel() * routing.element_size(),
                                 _stream(stream)))
        return routing

    def permute(self, x, topk, routing, ovr=None, stream=None, out=None):
        """Contiguous rows, m_indices and row_src of the routing; `out` may
        give the three buffers (routing capacity rows each)."""
        import torch
        T = x.shape[0]
        L = self.routing_layout(T, topk, ovr)
        if out is None:
            a = _new((L.cap, self.H), torch.bfloat16, self.device, stream)
            m = _new((L.cap,), torch.int32, self.device, stream)
            r = _new((L.cap,), torch.int32, self.device, stream)
        else:
            a, m, r = out
            if (a.dtype != torch.bfloat16 or m.dtype != torch.int32 or r.dtype != torch.int32
                    or not (a.is_contiguous() and m.is_contiguous() and r.is_contiguous())
                    or a.dim() != 2 or a.shape[0] < L.cap or a.shape[1] != self.H
                    or m.numel() < L.cap or r.numel() < L.cap):
                check(MOE_ERR_INVALID_ARG)
        check(lib().moe_permute(self.handle, _ptr(x), T, topk, _tuning(ovr), _ptr(routing), _ptr(a), _ptr(m),
                                _ptr(r), _stream(stream)))
        return a, m, r

    # -- the layer ------------------------------------------------------------
    def workspace_bytes(self, rows, topk=0, tokens=0, mode=None, ovr=None) -> int:
        m = self.mode if mode is None else mode
        return int(lib().moe_workspace_bytes(self.handle, m, rows, topk, tokens, _tuning(ovr)))

    def indexed(self, x, topk_ids, topk_w, routing=None, out=None, ws=None, ovr=None, stream=None):
        import torch
        T, topk = topk_ids.shape
        if out is None:
            out = _new((T, self.H), torch.bfloat16, self.device, stream)
        if ws is None:
            ws = _empty(self.workspace_bytes(T, topk, T, ovr=ovr), self.device, stream)
        check(lib().moe_w4a16_indexed(self.handle, _ptr(x), T, topk, _ptr(topk_ids), _ptr(topk_w),
                                      _ptr(routing), _ptr(out), _ptr(ws), ws.numel() * ws.element_size(),
                                      _tuning(ovr), _stream(stream)))
        return out

    def indexed_noalloc(self, x, topk_ids, topk_w, out, ovr=None, stream=None):
        """The indexed layer on the library's fixed scratch array: allocates
        nothing, so `out` must be given."""
        T, topk = topk_ids.shape
        check(lib().moe_w4a16_indexed_noalloc(self.handle, _ptr(x), T, topk, _ptr(topk_ids), _ptr(topk_w),
                                              _ptr(out), _tuning(ovr), _stream(stream)))
        return out

    def contiguous(self, a, m_indices, row_src=None, topk_w=None, T=0, topk=0, out=None, ws=None,
                   ovr=None, stream=None):
        import torch
        M_pad = a.shape[0]
        if out is None:
            rows = T if row_src is not None else M_pad
            out = _new((rows, self.H), torch.bfloat16, self.device, stream)
        if ws is None:
            ws = _empty(self.workspace_bytes(M_pad, topk if row_src is not None else 0, T), self.device, stream)
        check(lib().moe_w4a16_contiguous(self.handle, _ptr(a), M_pad, _ptr(m_indices), _ptr(row_src),
                                         _ptr(topk_w), T, topk, _ptr(out), _ptr(ws),
                                         ws.numel() * ws.element_size(), _tuning(ovr), _stream(stream)))
        return out

    def masked(self, a3, masked_m, expected_m, out=None, ws=None, ovr=None, stream=None):
        import torch
        E, max_m, H = a3.shape
        if out is None:
            out = _new((E * max_m, self.H), torch.bfloat16, self.device, stream)
        if ws is None:
            ws = _empty(self.workspace_bytes(max_m), self.device, stream)
        check(lib().moe_w4a16_masked(self.handle, _ptr(a3), max_m, _ptr(masked_m), expected_m, _ptr(out),
                                     _ptr(ws), ws.numel() * ws.element_size(), _tuning(ovr), _stream(stream)))
        return out

    # -- unfused steps (indexed) ------------------------------------------------
    def gate_up(self, x, topk, routing, out=None, ovr=None, stream=None):
        """BF16 [cap, 2I] gate | up rows at the routing's slots."""
        import torch
        T = x.shape[0]
        if out is None:
            cap = self.routing_layout(T, topk, ovr).cap
            out = _new((cap, 2 * self.I), torch.bfloat16, self.device, stream)
        check(lib().moe_w4a16_gate_up(self.handle, _ptr(x), T, topk, _ptr(routing), _ptr(out), _tuning(ovr),
                                      _stream(stream)))
        return out

    def down(self, a, T, topk, routing, out=None, ovr=None, stream=None):
        """BF16 [cap, H] rows of the second GEMM at the routing's slots."""
        import torch
        if out is None:
            out = _new((a.shape[0], self.H), torch.bfloat16, self.device, stream)
        check(lib().moe_w4a16_down(self.handle, _ptr(a), T, topk, _ptr(routing), _ptr(out), _tuning(ovr),
                                   _stream(stream)))
        return out

    def dequant(self, which, expert, stream=None):
        import torch
        shape = (2 * self.I, self.H) if which == 13 else (self.H, self.I)
        out = _new(shape, torch.bfloat16, self.device, stream)
        check(lib().moe_dequant_weights(self.handle, which, expert, _ptr(out), _stream(stream)))
        return out

    def describe(self, rows, topk=0, expected_m=0, ovr=None, mode=None) -> str:
        buf = ctypes.create_string_buffer(512)
        m = self.mode if mode is None else mode
        n = lib().moe_describe(self.handle, m, rows, topk, expected_m, _tuning(ovr), buf, 512)
        if n < 0:
            raise MoeError(MOE_ERR_INVALID_ARG, last_error())
        return buf.value.decode()


def swiglu(h, out=None, stream=None):
    """BF16 [rows, I] = silu(h[:, :I]) * h[:, I:] for BF16 h [rows, 2I]."""
    import torch
    rows, two_i = h.shape
    if out is None:
        out = _new((rows, two_i // 2), torch.bfloat16, h.device, stream)
    check(lib().moe_swiglu(_ptr(h), rows, two_i // 2, _ptr(out), _stream(stream)))
    return out


# ---------------------------------------------------------------------------
# Operators around the layer
# ---------------------------------------------------------------------------

# The smallest of these calls take a few microseconds on the GPU, less than the
# host needs for a call written carelessly: the helpers below look at every
# tensor once, pass plain integers to the library and ask torch for the raw
# stream.


def _dtype(t) -> int:
    """MOE_DTYPE_* of a torch dtype."""
    code = _CODES.get(t)
    if code is None:
        raise MoeError(MOE_ERR_INVALID_ARG, f"{t}: bfloat16, float16 or float32")
    return code


def _need(ok, msg):
    if not ok:
        raise MoeError(MOE_ERR_INVALID_ARG, msg)


def _fits(sizes):
    """Refuses sizes (joined by |) past 31 bits, which the library's arguments would cut off."""
    if sizes >> 31:
        raise MoeError(MOE_ERR_INVALID_ARG, "a size of 2^31 or more")


def _matrix(t, name, dtype=None, device=None, shape=None):
    """Checks a tensor's rows: on the GPU (the first operand's), of a dtype
    and shape, values of a row adjacent. Returns the row distance."""
    if not t.is_cuda:
        raise MoeError(MOE_ERR_INVALID_ARG, f"{name}: not on a GPU")
    if device is not None and t.device != device:
        raise MoeError(MOE_ERR_INVALID_ARG, f"{name}: on {t.device}, the first operand on {device}")
    if dtype is not None and t.dtype != dtype:
        raise MoeError(MOE_ERR_INVALID_ARG, f"{name}: {t.dtype}, expected {dtype}")
    s = t.shape
    if shape is not None and s != shape:
        raise MoeError(MOE_ERR_INVALID_ARG, f"{name}: shape {tuple(s)}, expected {shape}")
    st = t.stride()
    width = s[-1]
    # a dimension of one element has no meaningful stride
    if st[-1] != 1 and width > 1:
        raise MoeError(MOE_ERR_INVALID_ARG, f"{name}: the values of a row are not adjacent")
    return st[-2] if s[-2] > 1 else (width + 7) // 8 * 8


def _dense(t, name, dtype, device, shape):
    if not t.is_cuda or t.device != device:
        raise MoeError(MOE_ERR_INVALID_ARG, f"{name}: not on the first operand's GPU")
    if t.dtype != dtype or t.shape != shape:
        raise MoeError(MOE_ERR_INVALID_ARG, f"{name}: {t.dtype} {tuple(t.shape)}, expected {dtype} {shape}")
    if not t.is_contiguous():
        raise MoeError(MOE_ERR_INVALID_ARG, f"{name}: not contiguous")


def _call(fn, device, stream, *args):
    """fn(*args, stream) on `device`: on `stream`, or on its current stream."""
    torch = _torch
    if stream is not None and stream.device_index != device.index:
        raise MoeError(MOE_ERR_INVALID_ARG, f"stream: on device {stream.device_index}, the operands on {device}")
    if device.index != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            return _call(fn, device, stream, *args)
    status = fn(*args, torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream)
    if status != MOE_OK:
        check(status)


def router_topk(logits, topk, score="softmax", bias=None, renorm=False, scale=1.0, out=None, stream=None):
    """(ids int32, weights float32), both [T, topk]: each token's experts of
    largest logit (with `bias`, float32 [E]: of largest score + bias, in FP64),
    largest first, equal ones by index. Weight: scale * score, with `renorm`
    over the sum of the chosen scores. A logit of -inf or NaN takes its expert
    out for the token; places without an expert hold id -1 and weight 0, which
    the layer routes nowhere. logits [T, E] bf16, fp16 or fp32; `out` may give
    the two tensors."""
    torch = _torch or _load()
    _need(logits.dim() == 2, "logits: [T, E]")
    T, E = logits.shape
    ld = _matrix(logits, "logits")
    dev = logits.device
    if score not in SCORES:
        raise MoeError(MOE_ERR_INVALID_ARG, f"score {score!r}: softmax or sigmoid")
    _need(topk >= 1, "topk: at least 1")
    _fits(T | E | topk)
    if bias is not None:
        _dense(bias, "bias", torch.float32, dev, (E,))
    if out is None:
        ids = _new((T, topk), torch.int32, dev, stream)
        w = _new((T, topk), torch.float32, dev, stream)
    else:
        ids, w = out
        _dense(ids, "ids", torch.int32, dev, (T, topk))
        _dense(w, "weights", torch.float32, dev, (T, topk))
    _call((_lib or lib()).moe_router_topk, dev, stream,
          logits.data_ptr(), _dtype(logits.dtype), ld, T, E, topk, SCORES[score],
          None if bias is None else bias.data_ptr(), 1 if renorm else 0, scale, ids.data_ptr(), w.data_ptr())
    return ids, w


def router_topk_grad(logits, ids, d_w, score="softmax", renorm=False, scale=1.0, out=None, stream=None):
    """Gradient [T, E] of the logits (their dtype) for the ids that
    router_topk chose with the same score, renorm and scale, and the gradient
    d_w (float32 [T, topk]) of their weights."""
    torch = _torch or _load()
    _need(logits.dim() == 2 and ids.dim() == 2, "logits: [T, E], ids: [T, topk]")
    T, E = logits.shape
    ld = _matrix(logits, "logits")
    dev = logits.device
    topk = ids.shape[1]
    _fits(T | E | topk)
    if score not in SCORES:
        raise MoeError(MOE_ERR_INVALID_ARG, f"score {score!r}: softmax or sigmoid")
    _dense(ids, "ids", torch.int32, dev, (T, topk))
    _dense(d_w, "d_w", torch.float32, dev, (T, topk))
    if out is None:
        out = _new((T, E), logits.dtype, dev, stream)
        o_ld = E
    else:
        o_ld = _matrix(out, "out", logits.dtype, dev, (T, E))
    _call((_lib or lib()).moe_router_topk_grad, dev, stream,
          logits.data_ptr(), _dtype(logits.dtype), ld, T, E, topk, SCORES[score], 1 if renorm else 0, scale,
          ids.data_ptr(), d_w.data_ptr(), out.data_ptr(), o_ld)
    return out


def _weights(w, dtype, device):
    """Row and expert distances of w [E, N, K]."""
    ld = _matrix(w, "w", dtype, device)
    return ld, (w.stride(0) if w.shape[0] > 1 else 0)


def grouped_gemm(a, w, offsets, out=None, out_dtype=None, stream=None):
    """out[r] = a[r] . w[e]^T for the rows r in [offsets[e], offsets[e + 1]).

    a [M, K] and w [E, N, K] bf16 or fp16, offsets int32 [E + 1] on the GPU,
    not decreasing; out [M, N] of out_dtype (default a's; fp32 as well). Rows
    may be apart (strides of a multiple of 8). Rows of no expert are left as
    they are in `out`. N and K are multiples of 8."""
    if _torch is None:
        _load()
    _need(a.dim() == 2 and w.dim() == 3, "a: [M, K], w: [E, N, K]")
    M, K = a.shape
    E, N, Kw = w.shape
    if K != Kw:
        raise MoeError(MOE_ERR_INVALID_ARG, f"a has {K} columns, w {Kw}")
    _fits(M | N | K | E)
    dev = a.device
    a_ld = _matrix(a, "a")
    w_ld, w_stride = _weights(w, a.dtype, dev)
    _dense(offsets, "offsets", _torch.int32, dev, (E + 1,))
    if out is None:
        out = _new((M, N), out_dtype or a.dtype, dev, stream)
        o_ld = N
    else:
        o_ld = _matrix(out, "out", out_dtype, dev, (M, N))
    _call((_lib or lib()).moe_grouped_gemm, dev, stream,
          a.data_ptr(), a_ld, w.data_ptr(), w_stride, w_ld, _dtype(a.dtype), offsets.data_ptr(), E, M, N, K,
          out.data_ptr(), o_ld, _dtype(out.dtype))
    return out


def grouped_gemm_dgrad(dy, w, offsets, out=None, out_dtype=None, stream=None):
    """Gradient of grouped_gemm's `a`: out[r] = dy[r] . w[e], [M, K]."""
    if _torch is None:
        _load()
    _need(dy.dim() == 2 and w.dim() == 3, "dy: [M, N], w: [E, N, K]")
    M, N = dy.shape
    E, Nw, K = w.shape
    if N != Nw:
        raise MoeError(MOE_ERR_INVALID_ARG, f"dy has {N} columns, w {Nw} rows")
    _fits(M | N | K | E)
    dev = dy.device
    y_ld = _matrix(dy, "dy")
    w_ld, w_stride = _weights(w, dy.dtype, dev)
    _dense(offsets, "offsets", _torch.int32, dev, (E + 1,))
    if out is None:
        out = _new((M, K), out_dtype or dy.dtype, dev, stream)
        o_ld = K
    else:
        o_ld = _matrix(out, "out", out_dtype, dev, (M, K))
    _call((_lib or lib()).moe_grouped_gemm_dgrad, dev, stream,
          dy.data_ptr(), y_ld, w.data_ptr(), w_stride, w_ld, _dtype(dy.dtype), offsets.data_ptr(), E, M, N, K,
          out.data_ptr(), o_ld, _dtype(out.dtype))
    return out


def grouped_gemm_wgrad(dy, a, offsets, out=None, out_dtype=None, stream=None):
    """Gradient of grouped_gemm's `w`: out[e] = dy[rows of e]^T . a[rows of e],
    [E, N, K]; 0 for an expert without rows."""
    if _torch is None:
        _load()
    _need(dy.dim() == 2 and a.dim() == 2 and dy.shape[0] == a.shape[0], "dy: [M, N], a: [M, K]")
    M, N = dy.shape
    K = a.shape[1]
    dev = dy.device
    y_ld = _matrix(dy, "dy")
    a_ld = _matrix(a, "a", dy.dtype, dev)
    _need(offsets.dim() == 1 and offsets.shape[0] >= 2, "offsets: [E + 1]")
    E = offsets.shape[0] - 1
    _fits(M | N | K | E)
    _dense(offsets, "offsets", _torch.int32, dev, (E + 1,))
    if out is None:
        out = _new((E, N, K), out_dtype or dy.dtype, dev, stream)
    o_ld = _matrix(out, "out", out_dtype, dev, (E, N, K))
    stride = out.stride(0) if E > 1 else ((N - 1) * o_ld + K + 7) // 8 * 8
    _call((_lib or lib()).moe_grouped_gemm_wgrad, dev, stream,
          dy.data_ptr(), y_ld, a.data_ptr(), a_ld, _dtype(dy.dtype), offsets.data_ptr(), E, M, N, K,
          out.data_ptr(), stride, o_ld, _dtype(out.dtype))
    return out


def grouped_linear(a, w, offsets, bias=None, act="none", residual=None, out=None, out_dtype=None, stream=None):
    """grouped_gemm with an epilogue on its FP32 sums, rounded once: out[r] =
    [residual[r] +] act(a[r] . w[e]^T [+ bias[e]]). act "none", or "swiglu" for
    w[e] = gate | up (N a multiple of 16): silu(gate) * up, [M, N/2].

    bias [E, N] bf16, fp16 or fp32; residual of out's shape and dtype, may be
    `out` itself. Gradients: grouped_gemm_dgrad, grouped_gemm_wgrad and
    grouped_bias_grad for the gradient before act (swiglu_grad)."""
    if _torch is None:
        _load()
    _need(a.dim() == 2 and w.dim() == 3, "a: [M, K], w: [E, N, K]")
    M, K = a.shape
    E, N, Kw = w.shape
    if K != Kw:
        raise MoeError(MOE_ERR_INVALID_ARG, f"a has {K} columns, w {Kw}")
    code = ACTS.get(act)
    if code is None:
        raise MoeError(MOE_ERR_INVALID_ARG, f"act {act!r}: none or swiglu")
    _fits(M | N | K | E)
    dev = a.device
    a_ld = _matrix(a, "a")
    w_ld, w_stride = _weights(w, a.dtype, dev)
    _dense(offsets, "offsets", _torch.int32, dev, (E + 1,))
    cols = N // 2 if code else N
    if out is None:
        out = _new((M, cols), out_dtype or a.dtype, dev, stream)
        o_ld = cols
    else:
        o_ld = _matrix(out, "out", out_dtype, dev, (M, cols))
    b_at, b_type, b_ld = None, 0, 0
    if bias is not None:
        b_at, b_type, b_ld = bias.data_ptr(), _dtype(bias.dtype), _matrix(bias, "bias", None, dev, (E, N))
    r_ld = 0 if residual is None else _matrix(residual, "residual", out.dtype, dev, (M, cols))
    _call((_lib or lib()).moe_grouped_linear, dev, stream,
          a.data_ptr(), a_ld, w.data_ptr(), w_stride, w_ld, _dtype(a.dtype), offsets.data_ptr(), E, M, N, K,
          b_at, b_type, b_ld, code, None if residual is None else residual.data_ptr(), r_ld,
          out.data_ptr(), o_ld, _dtype(out.dtype))
    return out


@functools.lru_cache(maxsize=256)
def _bias_grad_bytes(E, M, N) -> int:
    n = lib().moe_grouped_bias_grad_bytes(E, M, N)
    if n < 0:
        check(MOE_ERR_INVALID_ARG)
    return n


def grouped_bias_grad(dy, offsets, out=None, out_dtype=None, ws=None, stream=None):
    """Gradient of grouped_linear's bias: out[e] = the sum of dy's rows of e,
    [E, N] of out_dtype (default dy's; fp32 as well); 0 for an expert without
    rows. dy [M, N] bf16 or fp16, N a multiple of 8. `ws` may give a uint8
    workspace."""
    if _torch is None:
        _load()
    _need(dy.dim() == 2, "dy: [M, N]")
    M, N = dy.shape
    dev = dy.device
    y_ld = _matrix(dy, "dy")
    _need(offsets is not None, "offsets: [E + 1]")
    off, E = _offsets(offsets, dev)
    _fits(M | N | E)
    if out is None:
        out = _new((E, N), out_dtype or dy.dtype, dev, stream)
        o_ld = N
    else:
        o_ld = _matrix(out, "out", out_dtype, dev, (E, N))
    nbytes = _bias_grad_bytes(E, M, N)
    if ws is not None:
        nbytes = ws.numel()
        _dense(ws, "ws", _torch.uint8, dev, (nbytes,))
    elif nbytes:
        ws = _empty(nbytes, dev, stream)
    _call((_lib or lib()).moe_grouped_bias_grad, dev, stream,
          dy.data_ptr(), y_ld, _dtype(dy.dtype), off, E, M, N, out.data_ptr(), o_ld, _dtype(out.dtype),
          None if ws is None else ws.data_ptr(), nbytes)
    return out


@functools.lru_cache(maxsize=None)
def mx_scale_cols(K) -> int:
    """Bytes of a row of MXFP4 scales: K / 32 rounded up to a multiple of 16."""
    _fits(K)
    n = lib().moe_mx_scale_cols(K)
    if n == 0:
        check(MOE_ERR_INVALID_ARG)
    return n


def mx_quant(x, out=None, stream=None):
    """MXFP4 rows of x [..., K] (bf16, fp16 or fp32, K a multiple of 32):
    (codes uint8 [..., K/2], the lower nibble first; scales uint8 [...,
    mx_scale_cols(K)], one E8M0 byte per 32 values). More than two dimensions
    must be dense; `out` may give the two tensors."""
    torch = _torch or _load()
    _need(x.dim() >= 2, "x: [..., K]")
    K = x.shape[-1]
    ld = _matrix(x, "x")
    _need(x.dim() == 2 or x.is_contiguous(), "x: more than two dimensions must be contiguous")
    rows = x.numel() // K if K else 0
    cols = mx_scale_cols(K)
    dev = x.device
    lead = tuple(x.shape[:-1])
    if out is None:
        q = _new(lead + (K // 2,), torch.uint8, dev, stream)
        scales = _new(lead + (cols,), torch.uint8, dev, stream)
    else:
        q, scales = out
        _dense(q, "codes", torch.uint8, dev, lead + (K // 2,))
        _dense(scales, "scales", torch.uint8, dev, lead + (cols,))
    _call((_lib or lib()).moe_mx_quant, dev, stream,
          x.data_ptr(), _dtype(x.dtype), ld if x.dim() == 2 else K, rows, K, q.data_ptr(), scales.data_ptr())
    return q, scales


def mx_dequant(q, scales, dtype=None, out=None, stream=None):
    """Values [..., K] of MXFP4 rows in `dtype` (default bf16)."""
    torch = _torch or _load()
    _need(q.dim() >= 2, "codes: [..., K/2]")
    K = 2 * q.shape[-1]
    lead = tuple(q.shape[:-1])
    dev = q.device
    _dense(q, "codes", torch.uint8, dev, tuple(q.shape))
    _dense(scales, "scales", torch.uint8, dev, lead + (mx_scale_cols(K),))
    if out is None:
        out = _new(lead + (K,), dtype or torch.bfloat16, dev, stream)
        ld = K
    else:
        ld = _matrix(out, "out", dtype, dev, lead + (K,))
        _need(out.dim() == 2 or out.is_contiguous(), "out: more than two dimensions must be contiguous")
    _call((_lib or lib()).moe_mx_dequant, dev, stream,
          q.data_ptr(), scales.data_ptr(), q.numel() * 2 // K, K, out.data_ptr(), _dtype(out.dtype),
          ld if out.dim() == 2 else K)
    return out


def mx_grouped_gemm(aq, a_scales, wq, w_scales, offsets, out=None, out_dtype=None, stream=None):
    """grouped_gemm on MXFP4 rows (aq uint8 [M, K/2]) and MXFP4 weights (wq
    uint8 [E, N, K/2]) with their scales as mx_quant writes them; out [M, N]
    of out_dtype (default bf16)."""
    torch = _torch or _load()
    _need(aq.dim() == 2 and wq.dim() == 3, "aq: [M, K/2], wq: [E, N, K/2]")
    M, E, N, K = aq.shape[0], wq.shape[0], wq.shape[1], 2 * aq.shape[1]
    dev = aq.device
    cols = mx_scale_cols(K)
    _fits(M | N | E)
    _dense(aq, "aq", torch.uint8, dev, (M, K // 2))
    _dense(a_scales, "a_scales", torch.uint8, dev, (M, cols))
    _dense(wq, "wq", torch.uint8, dev, (E, N, K // 2))
    _dense(w_scales, "w_scales", torch.uint8, dev, (E, N, cols))
    _dense(offsets, "offsets", _torch.int32, dev, (E + 1,))
    if out is None:
        out = _new((M, N), out_dtype or torch.bfloat16, dev, stream)
        o_ld = N
    else:
        o_ld = _matrix(out, "out", out_dtype, dev, (M, N))
    _call((_lib or lib()).moe_mx_grouped_gemm, dev, stream,
          aq.data_ptr(), a_scales.data_ptr(), wq.data_ptr(), w_scales.data_ptr(), offsets.data_ptr(), E, M, N, K,
          out.data_ptr(), o_ld, _dtype(out.dtype))
    return out


# ---------------------------------------------------------------------------
# Operators of a training step around the experts' products
# ---------------------------------------------------------------------------


def _score(score) -> int:
    code = SCORES.get(score)
    if code is None:
        raise MoeError(MOE_ERR_INVALID_ARG, f"score {score!r}: softmax or sigmoid")
    return code


def _offsets(t, device):
    """(pointer, count - 1) of int32 offsets, or (None, 0)."""
    if t is None:
        return None, 0
    _need(t.dim() == 1 and t.shape[0] >= 2, "offsets: [E + 1]")
    _fits(t.shape[0])
    _dense(t, "offsets", _torch.int32, device, tuple(t.shape))
    return t.data_ptr(), t.shape[0] - 1


@functools.lru_cache(maxsize=256)
def _balance_bytes(T, E, S) -> int:
    n = lib().moe_router_balance_bytes(T, E, S)
    if n < 0:
        check(MOE_ERR_INVALID_ARG)
    return n


def router_balance(logits, ids, score="softmax", offsets=None, out=None, ws=None, stream=None):
    """(loss float32 [S], counts int32 [S, E]) of S sequences of tokens, rows
    [offsets[s], offsets[s + 1]) of logits [T, E] (bf16, fp16 or fp32) and of
    their chosen experts ids (int32 [T, topk]); without offsets one sequence of
    all rows. counts: how often a sequence chose each expert. loss: E * sum_e
    f_e P_e with the shares f of the choices and the mean scores P (softmax, or
    sigmoids over their sum); 0 for an empty sequence. Ids outside [0, E) count
    nowhere, a logit of -inf or NaN has score 0. `out` may give the two tensors,
    `ws` a uint8 workspace."""
    torch = _torch or _load()
    _need(logits.dim() == 2 and ids.dim() == 2, "logits: [T, E], ids: [T, topk]")
    T, E = logits.shape
    topk = ids.shape[1]
    ld = _matrix(logits, "logits")
    dev = logits.device
    _fits(T | E | topk)
    _dense(ids, "ids", torch.int32, dev, (T, topk))
    off, S = (None, 1) if offsets is None else _offsets(offsets, dev)
    if out is None:
        loss = _new((S,), torch.float32, dev, stream)
        counts = _new((S, E), torch.int32, dev, stream)
    else:
        loss, counts = out
        _dense(loss, "loss", torch.float32, dev, (S,))
        _dense(counts, "counts", torch.int32, dev, (S, E))
    nbytes = _balance_bytes(T, E, S)
    if ws is not None:
        nbytes = ws.numel()
        _dense(ws, "ws", torch.uint8, dev, (nbytes,))
    elif nbytes:
        ws = _empty(nbytes, dev, stream)
    _call((_lib or lib()).moe_router_balance, dev, stream,
          logits.data_ptr(), _dtype(logits.dtype), ld, T, E, ids.data_ptr(), topk, _score(score), off, S,
          loss.data_ptr(), counts.data_ptr(), None if ws is None else ws.data_ptr(), nbytes)
    return loss, counts


def router_balance_grad(logits, counts, d_loss, topk, score="softmax", offsets=None, add=None, out=None, stream=None):
    """Gradient [T, E] of the logits (their dtype) for the gradient d_loss
    (float32 [S]) of router_balance's losses, with the counts that it returned;
    0 for rows of no sequence. `add` [T, E] (router_topk_grad's result, of the
    logits' dtype) is added before the one rounding; it may be `out` itself."""
    torch = _torch or _load()
    _need(logits.dim() == 2, "logits: [T, E]")
    T, E = logits.shape
    ld = _matrix(logits, "logits")
    dev = logits.device
    _need(topk >= 1, "topk: at least 1")
    _fits(T | E | topk)
    off, S = (None, 1) if offsets is None else _offsets(offsets, dev)
    _dense(counts, "counts", torch.int32, dev, (S, E))
    _dense(d_loss, "d_loss", torch.float32, dev, (S,))
    a_ld = 0 if add is None else _matrix(add, "add", logits.dtype, dev, (T, E))
    if out is None:
        out = _new((T, E), logits.dtype, dev, stream)
        o_ld = E
    else:
        o_ld = _matrix(out, "out", logits.dtype, dev, (T, E))
    _call((_lib or lib()).moe_router_balance_grad, dev, stream,
          logits.data_ptr(), _dtype(logits.dtype), ld, T, E, topk, _score(score), off, S, counts.data_ptr(),
          d_loss.data_ptr(), None if add is None else add.data_ptr(), a_ld, out.data_ptr(), o_ld)
    return out


def combine(y, slots, w=None, out=None, out_dtype=None, stream=None):
    """out[t] = sum_j w[t, j] * y[slots[t, j]] in FP32, j ascending, [T, H] of
    out_dtype (default y's): a token's routed rows. y [R, H] bf16, fp16 or fp32
    (H a multiple of 8), slots int32 [T, topk] (a slot outside [0, R), as -1,
    names no row), w float32 [T, topk] or None for 1: the gradient of a
    permutation's input. A routing buffer's slot_of section holds such slots."""
    torch = _torch or _load()
    _need(y.dim() == 2 and slots.dim() == 2, "y: [R, H], slots: [T, topk]")
    R, H = y.shape
    T, topk = slots.shape
    _fits(R | H | T | topk)
    y_ld = _matrix(y, "y")
    dev = y.device
    _dense(slots, "slots", torch.int32, dev, (T, topk))
    if w is not None:
        _dense(w, "w", torch.float32, dev, (T, topk))
    if out is None:
        out = _new((T, H), out_dtype or y.dtype, dev, stream)
        o_ld = H
    else:
        o_ld = _matrix(out, "out", out_dtype, dev, (T, H))
    _call((_lib or lib()).moe_combine, dev, stream,
          y.data_ptr(), _dtype(y.dtype), y_ld, R, H, slots.data_ptr(), T, topk, None if w is None else w.data_ptr(),
          out.data_ptr(), o_ld, _dtype(out.dtype))
    return out


def combine_grad(d_out, slots, y=None, w=None, row_src=None, offsets=None, out=None, stream=None):
    """(d_y [R, H], d_w float32 [T, topk]) for the gradient d_out [T, H] of
    combine's result: d_y[slots[t, j]] = w[t, j] * d_out[t], d_w[t, j] =
    <d_out[t], y[slots[t, j]]> (None without y). A row is named by one slot at
    most. R is y's, or row_src's, or that of the d_y in `out` = (d_y, d_w or
    None). Rows that no slot names stay as they are (unspecified in a new d_y),
    but with row_src (int32 [R], a routing buffer's sorted_ids section: t * topk
    + j of each row) the rows of [offsets[0], offsets[-1]) whose row_src lies
    outside [0, T * topk) become 0, which grouped products need in a group's
    padding; without offsets those of all R."""
    torch = _torch or _load()
    _need(d_out.dim() == 2 and slots.dim() == 2, "d_out: [T, H], slots: [T, topk]")
    T, H = d_out.shape
    topk = slots.shape[1]
    d_ld = _matrix(d_out, "d_out")
    dev = d_out.device
    _dense(slots, "slots", torch.int32, dev, (T, topk))
    if w is not None:
        _dense(w, "w", torch.float32, dev, (T, topk))
    d_y, d_w = (None, None) if out is None else out
    like = y if y is not None else row_src if row_src is not None else d_y
    _need(like is not None, "one of y, row_src and out gives the number of rows")
    R = like.shape[0]
    _fits(R | H | T | topk)
    y_ld = 0 if y is None else _matrix(y, "y", d_out.dtype, dev, (R, H))
    if row_src is not None:
        _dense(row_src, "row_src", torch.int32, dev, (R,))
    _need(offsets is None or row_src is not None, "offsets without row_src")
    off, E = _offsets(offsets, dev)
    if d_y is None:
        d_y = _new((R, H), d_out.dtype, dev, stream)
        dy_ld = H
    else:
        dy_ld = _matrix(d_y, "d_y", d_out.dtype, dev, (R, H))
    if d_w is not None:
        _need(y is not None, "d_w without y")
        _dense(d_w, "d_w", torch.float32, dev, (T, topk))
    elif y is not None:
        d_w = _new((T, topk), torch.float32, dev, stream)
    _call((_lib or lib()).moe_combine_grad, dev, stream,
          d_out.data_ptr(), _dtype(d_out.dtype), d_ld, T, H, slots.data_ptr(), topk, None if w is None else w.data_ptr(),
          None if y is None else y.data_ptr(), y_ld, None if row_src is None else row_src.data_ptr(), off, E,
          d_y.data_ptr(), dy_ld, R, None if d_w is None else d_w.data_ptr())
    return d_y, d_w


@functools.lru_cache(maxsize=None)
def mx8_scale_cols(K) -> int:
    """Bytes of a row of 8-bit rows' scales: K / 32 rounded up, then to a multiple of 16."""
    _fits(K)
    n = lib().moe_mx8_scale_cols(K)
    if n == 0:
        check(MOE_ERR_INVALID_ARG)
    return n


def mx8_quant(x, out=None, stream=None):
    """Rows of x [rows, K] (bf16, fp16 or fp32, K a multiple of 8) in 8 bits:
    (codes int8 [rows, K], scales uint8 [rows, mx8_scale_cols(K)], one E8M0 byte
    per 32 values). A value is code * 2^(byte - 133), within a 128th of its
    block's largest magnitude or, for the smallest magnitudes, within 2^-134
    (the least scale's half step), and exact in bf16; a block with a NaN or an
    infinity becomes NaN. `out` may give the two tensors."""
    torch = _torch or _load()
    _need(x.dim() == 2, "x: [rows, K]")
    rows, K = x.shape
    ld = _matrix(x, "x")
    cols = mx8_scale_cols(K)
    dev = x.device
    if out is None:
        q = _new((rows, K), torch.int8, dev, stream)
        scales = _new((rows, cols), torch.uint8, dev, stream)
    else:
        q, scales = out
        _dense(q, "codes", torch.int8, dev, (rows, K))
        _dense(scales, "scales", torch.uint8, dev, (rows, cols))
    _call((_lib or lib()).moe_mx8_quant, dev, stream,
          x.data_ptr(), _dtype(x.dtype), ld, rows, K, q.data_ptr(), scales.data_ptr())
    return q, scales


def mx8_dequant(q, scales, dtype=None, row_src=None, topk=1, offsets=None, out=None, stream=None):
    """Values of rows in 8 bits in `dtype` (default bf16): [rows, K], or with
    row_src (int32 [R]) [R, K] of rows row_src[r] // topk, 0 where row_src[r]
    lies outside [0, rows * topk). With a routing buffer's sorted_ids as row_src
    these are the rows that `permute` writes. With offsets (int32 [E + 1]) only
    rows [offsets[0], offsets[-1]) are written."""
    torch = _torch or _load()
    _need(q.dim() == 2, "codes: [rows, K]")
    rows, K = q.shape
    dev = q.device
    _dense(q, "codes", torch.int8, dev, (rows, K))
    _dense(scales, "scales", torch.uint8, dev, (rows, mx8_scale_cols(K)))
    R = rows
    if row_src is not None:
        _need(row_src.dim() == 1 and topk >= 1, "row_src: [R], topk: at least 1")
        R = row_src.shape[0]
        _dense(row_src, "row_src", torch.int32, dev, (R,))
        _fits(R | rows | topk)
    off, E = _offsets(offsets, dev)
    if out is None:
        out = _new((R, K), dtype or torch.bfloat16, dev, stream)
        ld = K
    else:
        ld = _matrix(out, "out", dtype, dev, (R, K))
    _call((_lib or lib()).moe_mx8_dequant, dev, stream,
          q.data_ptr(), scales.data_ptr(), rows, K, None if row_src is None else row_src.data_ptr(), topk, off, E,
          out.data_ptr(), _dtype(out.dtype), ld, R)
    return out


def swiglu_save(h, offsets=None, out=None, stream=None):
    """(a [rows, I], codes int8 [rows, 2, I], scales uint8 [rows, 2,
    mx8_scale_cols(I)]): a = silu(h[:, :I]) * h[:, I:] of h [rows, 2I] (bf16,
    fp16 or fp32, I a multiple of 8), and h in 8 bits for swiglu_grad, as
    mx8_quant writes the 2 * rows rows of I values. With offsets (int32 [E + 1])
    only rows [offsets[0], offsets[-1]) are read and written. `out` may give the
    three tensors."""
    torch = _torch or _load()
    _need(h.dim() == 2 and h.shape[1] % 2 == 0, "h: [rows, 2I]")
    rows, I = h.shape[0], h.shape[1] // 2
    _fits(rows | I)
    ld = _matrix(h, "h")
    cols = mx8_scale_cols(I)
    dev = h.device
    off, E = _offsets(offsets, dev)
    if out is None:
        a = _new((rows, I), h.dtype, dev, stream)
        q = _new((rows, 2, I), torch.int8, dev, stream)
        scales = _new((rows, 2, cols), torch.uint8, dev, stream)
        a_ld = I
    else:
        a, q, scales = out
        a_ld = _matrix(a, "a", h.dtype, dev, (rows, I))
        _dense(q, "codes", torch.int8, dev, (rows, 2, I))
        _dense(scales, "scales", torch.uint8, dev, (rows, 2, cols))
    _call((_lib or lib()).moe_swiglu_save, dev, stream,
          h.data_ptr(), _dtype(h.dtype), ld, rows, I, off, E, a.data_ptr(), a_ld, q.data_ptr(), scales.data_ptr())
    return a, q, scales


def swiglu_grad(h, d_a, scales=None, offsets=None, need_a=True, out=None, stream=None):
    """(d_h [rows, 2I], a [rows, I]) of d_a's dtype for the gradient d_a
    [rows, I] of a = silu(g) * u: the gradient of h = g | u, and a once more
    (None without need_a). h is [rows, 2I] of d_a's dtype, or with scales the
    codes int8 [rows, 2, I] that swiglu_save returned. With offsets (int32
    [E + 1]) only rows [offsets[0], offsets[-1]) are read and written. `out` may
    give the two tensors."""
    torch = _torch or _load()
    _need(d_a.dim() == 2, "d_a: [rows, I]")
    rows, I = d_a.shape
    _fits(rows | I)
    da_ld = _matrix(d_a, "d_a")
    dev = d_a.device
    off, E = _offsets(offsets, dev)
    if scales is None:
        h_at, h_ld, q_at, s_at = h.data_ptr(), _matrix(h, "h", d_a.dtype, dev, (rows, 2 * I)), None, None
    else:
        _dense(h, "codes", torch.int8, dev, (rows, 2, I))
        _dense(scales, "scales", torch.uint8, dev, (rows, 2, mx8_scale_cols(I)))
        h_at, h_ld, q_at, s_at = None, 0, h.data_ptr(), scales.data_ptr()
    if out is None:
        d_h = _new((rows, 2 * I), d_a.dtype, dev, stream)
        a = _new((rows, I), d_a.dtype, dev, stream) if need_a else None
        dh_ld, a_ld = 2 * I, I
    else:
        d_h, a = out
        dh_ld = _matrix(d_h, "d_h", d_a.dtype, dev, (rows, 2 * I))
        a_ld = 0 if a is None else _matrix(a, "a", d_a.dtype, dev, (rows, I))
    _call((_lib or lib()).moe_swiglu_grad, dev, stream,
          h_at, h_ld, q_at, s_at, _dtype(d_a.dtype), rows, I, d_a.data_ptr(), da_ld, off, E, d_h.data_ptr(), dh_ld,
          None if a is None else a.data_ptr(), a_ld)
    return d_h, a


def profile_enable(on=True):
    check(lib().moe_profile_enable(1 if on else 0))


def profile_reset():
    lib().moe_profile_reset()


def profile_read() -> dict:
    """{kernel name: (launches, total_ms)} since the last reset (synchronises)."""
    buf = ctypes.create_string_buffer(1 << 16)
    n = lib().moe_profile_read(buf, 1 << 16)
    out = {}
    for line in buf.value.decode().splitlines():
        name, cnt, ms = line.split()
        out[name] = (int(cnt), float(ms))
    return out
