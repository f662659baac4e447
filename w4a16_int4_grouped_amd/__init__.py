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
