"""ctypes binding of libtovl.so (include/tovl.h).

Argument marshalling only: every step of the hot path runs in the library's
CUDA kernels.  Functions keep the C names; tensors are passed as raw device
pointers taken from torch tensors, which serve only as device memory and
streams.  If the library is missing or cannot load, every call raises
``TovlError`` -- there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libtovl.so")

TOVL_OK = 0
TOVL_ERR_INVALID = 1
TOVL_ERR_UNSUPPORTED = 2
TOVL_ERR_CUDA = 3
TOVL_ERR_TIMEOUT = 4
TOVL_ERR_OOM = 5
TOVL_COPY_VECTOR = 0
TOVL_COPY_BULK = 1
TOVL_COPY_AUTO = 2

TOVL_BF16 = 0
TOVL_F32 = 1
TOVL_E4M3 = 2

OPT_PRODUCERS = 1
OPT_CONSUMERS = 2
OPT_COPY_MODE = 3
OPT_STATS = 4
OPT_TIMEOUT_NS = 5
OPT_COPY_CTAS = 6
OPT_COPY_WAITERS = 7
OPT_FAULT_GATE_OFFSET = 8
OPT_K_SLICES = 9
OPT_PAIRS = 10
OPT_MAX_PAIRS = 11
OPT_COOP_PAIRS = 12
OPT_COOPERATIVE = 13
OPT_PRODUCER_MODE = 14
OPT_PDL = 15
OPT_ROLE_SWITCH = 16
OPT_DISPATCH_ALIGN = 17
OPT_EMBEDDED = 18
OPT_RS_EPILOGUE = 19
OPT_L2_HINTS = 20
OPT_WIDE_TILES = 23


class TovlError(RuntimeError):
    def __init__(self, code: int, what: str, detail: str = ""):
        self.code = code
        msg = f"{what}: {error_string(code) if _lib else code}"
        if detail:
            msg += f" ({detail})"
        super().__init__(msg)


class tovl_config(ctypes.Structure):
    _fields_ = [
        ("device", ctypes.c_int),
        ("chunk_rows", ctypes.c_int),
        ("gate_rows", ctypes.c_int),
        ("producer_ctas", ctypes.c_int),
        ("consumer_ctas", ctypes.c_int),
        ("wait_timeout_ns", ctypes.c_longlong),
        ("copy_mode", ctypes.c_int),
        ("max_rows", ctypes.c_longlong),
        ("max_pairs", ctypes.c_int),
        ("max_experts", ctypes.c_int),
        ("k_slices", ctypes.c_int),
    ]


class tovl_kv_cache(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p),
        ("type", ctypes.c_int),
        ("pages", ctypes.c_int),
        ("page", ctypes.c_int),
        ("heads", ctypes.c_int),
        ("dim", ctypes.c_int),
        ("page_stride", ctypes.c_longlong),
        ("slot_stride", ctypes.c_longlong),
        ("head_stride", ctypes.c_longlong),
    ]


# every exported symbol of include/tovl.h with its ctypes signature
_P = ctypes.c_void_p
_I = ctypes.c_int
_LL = ctypes.c_longlong
_F = ctypes.c_float
_IP = ctypes.POINTER(ctypes.c_int)
_LLP = ctypes.POINTER(ctypes.c_longlong)
_ULLP = ctypes.POINTER(ctypes.c_ulonglong)
SIGNATURES = {
    "tovl_default_config": ([ctypes.POINTER(tovl_config), _I], None),
    "tovl_create": ([ctypes.POINTER(_P), ctypes.POINTER(tovl_config)], _I),
    "tovl_destroy": ([_P], _I),
    "tovl_gather_gemm": ([_P, ctypes.POINTER(_P), _I, _I, _I, _P, _I, _P, _P, _P], _I),
    "tovl_dispatch_rows": ([_I, _I, _I], _LL),
    "tovl_dispatch_rows_aligned": ([_I, _I, _I, _I], _LL),
    "tovl_dispatch_grouped_gemm": ([_P, _P, _I, _I, _P, _I, _I, _P, _I, _P, _P, _P, _P], _I),
    "tovl_combine": ([_P, _P, _I, _P, _P, _P, _P], _I),
    "tovl_gemm_reduce_scatter": ([_P, _P, _I, _I, _I, _P, _I, _P, _P, _P], _I),
    "tovl_add_rmsnorm": ([_P, _P, _LL, _P, _P, _I, _LL, _P, _F, _I, _I, _P, _LL, _P, _P, _I, _P], _I),
    "tovl_route_topk": ([_P, _P, _I, _LL, _I, _I, _I, _I, _P, _P, _P], _I),
    "tovl_moe_decode_workspace": ([_P, _I, _I, _I, _I], _LL),
    "tovl_moe_decode": ([_P, _P, _LL, _I, _I, _P, _P, _I, _I, _P, _P, _I, _P, _LL, _P, _LL, _P], _I),
    "tovl_moe_decode_q4": ([_P, _P, _LL, _I, _I, _P, _P, _I, _I, _P, _P, _P, _P, _P, _P, _I, _I, _P, _LL, _P, _LL,
                            _P], _I),
    "tovl_matvec_q4_workspace": ([_P, _I, _I], _LL),
    "tovl_matvec_q4": ([_P, _P, _I, _P, _LL, _I, _I, _P, _P, _P, _I, _I, _P, _LL, _P, _LL, _P], _I),
    "tovl_quantize_q4": ([_P, _P, _I, _I, _I, _I, _P, _P, _P, _P], _I),
    "tovl_page_plan": ([_P, _P, _P], _I),
    "tovl_rope_append": ([_P, _P, _P], _I),
    "tovl_attn_decode_workspace": ([_P, _I, _I, _I], _LL),
    "tovl_attn_decode": ([_P, _P, _P], _I),
    "tovl_gemm_only": ([_P, _P, _I, _I, _P, _I, _P, _P], _I),
    "tovl_copy_only": ([_P, ctypes.POINTER(_P), _I, _I, _I, _P, _P], _I),
    "tovl_gated_copy": ([_P, _P, _P, _LL, _I, _P, _I, _I, _P], _I),
    "tovl_sync_status": ([_P], _I),
    "tovl_ctrl_sizes": ([_P, _IP, _IP], _I),
    "tovl_read_ctrl": ([_P, _P, _P, _P, _LLP], _I),
    "tovl_read_plan": ([_P, _P, _P, _P, _P, _P, _IP], _I),
    "tovl_set_option": ([_P, _I, _LL], _I),
    "tovl_get_option": ([_P, _I, _LLP], _I),
    "tovl_read_stats": ([_P, _ULLP, _I], _I),
    "tovl_read_latency": ([_P, _P, _P, _I], _I),
    "tovl_read_trace": ([_P, _I, _P, _LL], _I),
    "tovl_dispatch_plan_noalloc": ([_P, _I, _I, _I, _P, _P, _P], _I),
    "tovl_num_sms": ([_P], _I),
    "tovl_error_string": ([_I], ctypes.c_char_p),
    "tovl_last_error": ([_P], ctypes.c_char_p),
}

# the structs of arguments, packed in the order of their fields (a third of the time of as many ctypes arguments)
_PLAN_ARGS = struct.Struct("@10Pq5i4x").pack
_ROPE_ARGS = struct.Struct("@8P4q5i4x").pack
_ATTN_ARGS = struct.Struct("@7P4q4if4x").pack

_lib = None
_lock = threading.Lock()


def load(path: str = LIB_PATH):
    """Load libtovl.so (built by ``build.py``); raise if it is absent."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise TovlError(TOVL_ERR_UNSUPPORTED, "libtovl.so not built",
                                "run consumer_movement_gemm_gb300.build")
            lib = ctypes.CDLL(path)
            for name, (args, res) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.argtypes = args
                fn.restype = res
            _lib = lib
    return _lib


def error_string(code: int) -> str:
    return load().tovl_error_string(code).decode()


def _check(h, rc: int, what: str):
    if rc != TOVL_OK:
        detail = load().tovl_last_error(h).decode() if h else ""
        raise TovlError(rc, what, detail)


def _ptr(t) -> int:
    """Device pointer of a torch tensor (or an int address)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# element types of the decode-step calls by torch dtype, filled in by the
# first such call (importing this module does not import torch)
_types = {}
_BF16 = _F32 = _E4M3 = _I32 = _U8 = None


def _load_types():
    global _BF16, _F32, _E4M3, _I32, _U8
    import torch
    _BF16, _F32, _E4M3, _I32, _U8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int32, torch.uint8
    _types.update({_BF16: TOVL_BF16, _F32: TOVL_F32, _E4M3: TOVL_E4M3})


def _type_of(name, t, allowed) -> int:
    code = _types.get(t.dtype)
    if code not in allowed:
        raise TypeError(f"{name} must not be {t.dtype}")
    return code


def _matrix(name, t, dtype, rows, cols) -> int:
    """Checks a [rows, cols] tensor whose rows are contiguous; returns the distance of its rows in elements."""
    if t is None or t.dtype is not dtype or t.shape != (rows, cols):
        raise TypeError(f"{name} must be {dtype} ({rows}, {cols})")
    s = t.stride()
    if s[1] != 1 and cols > 1:
        raise TypeError(f"{name} must have unit stride in its last dimension")
    return s[0] if rows > 1 else (cols + 15) // 16 * 16    # (one row: any distance will do)


def _dense(name, t, dtype, shape):
    """Checks a contiguous tensor; returns its address."""
    if t is None or t.dtype is not dtype or t.shape != shape:
        raise TypeError(f"{name} must be {dtype} {shape}")
    if not t.is_contiguous():
        raise TypeError(f"{name} must be contiguous")
    return t.data_ptr()


def _bytes(name, t) -> int:
    if not t.is_contiguous():
        raise TypeError(f"{name} must be contiguous")
    return t.nbytes


def _packed(name, w, lead, K, N, group):
    """Checks a packed matrix (words, scales, zeros or None), stacked where lead is (E,); returns its addresses."""
    if group not in (32, 64, 128) or K % group:
        raise TypeError(f"{name}: groups are 32, 64 or 128 rows and divide K")
    words, scales, zeros = w
    rows, groups = lead + (K // 8, N), lead + (K // group, N)
    if not (words is not None and words.dtype is _I32 and words.shape == rows and words.is_contiguous()):
        _dense(name + " words", words, _I32, rows)
    if not (scales is not None and scales.dtype is _BF16 and scales.shape == groups and scales.is_contiguous()):
        _dense(name + " scales", scales, _BF16, groups)
    if zeros is None:
        return words.data_ptr(), scales.data_ptr(), None
    return words.data_ptr(), scales.data_ptr(), _dense("zeros", zeros, _U8, groups)


def _heads(name, t, rows, heads, dim) -> int:
    """Checks a bf16 [rows, heads, dim] tensor whose rows are contiguous; returns the distance of its rows in elements."""
    if t is None or t.dtype is not _BF16 or t.shape != (rows, heads, dim):
        raise TypeError(f"{name} must be {_BF16} ({rows}, {heads}, {dim})")
    ld, h, d = t.stride()
    if (d != 1 and dim > 1) or (h != dim and heads > 1):
        raise TypeError(f"{name} must have contiguous heads")
    return ld if rows > 1 else (heads * dim + 7) // 8 * 8


class KVCache:
    """A paged cache: k and v [pages, page, heads, dim], bf16 or e4m3, of the same strides (any, e.g. transposed from
    [pages, heads, page, dim] or halves of one tensor; the last is 1); e4m3 with fp32 scales [pages, heads, page].  Keeps
    the tensors alive and the struct that the calls take."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if _BF16 is None:
            _load_types()
        code = _type_of("k", k, (TOVL_BF16, TOVL_E4M3))
        if k.dim() != 4 or v.dtype is not k.dtype or v.shape != k.shape:
            raise TypeError("k and v must be [pages, page, heads, dim] of one type and shape")
        shape = pages, page, heads, dim = tuple(k.shape)
        s = k.stride()
        if any(a != b for a, b, n in zip(s, v.stride(), shape) if n > 1) or (s[3] != 1 and dim > 1):
            raise TypeError("k and v must have the same strides, of 1 in the last dimension")
        if (code == TOVL_E4M3) != (k_scale is not None) or (code == TOVL_E4M3) != (v_scale is not None):
            raise TypeError("scales go with an e4m3 cache, and only with it")
        scales = [None if x is None else _dense(n, x, _F32, (pages, heads, page)) for n, x in (("k_scale", k_scale),
                                                                                             ("v_scale", v_scale))]
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.page, self.heads, self.dim = shape
        self.struct = tovl_kv_cache(k.data_ptr(), v.data_ptr(), *scales, code, *shape, s[0], s[1], s[2])
        self.ref = ctypes.addressof(self.struct)


def default_config(device: int = 0) -> tovl_config:
    cfg = tovl_config()
    load().tovl_default_config(ctypes.byref(cfg), device)
    return cfg


def dispatch_rows(T: int, k: int, E: int) -> int:
    return load().tovl_dispatch_rows(T, k, E)


def dispatch_rows_aligned(T: int, k: int, E: int, align: int) -> int:
    """Rows a dispatch buffer needs with expert segments aligned to ``align``."""
    return int(load().tovl_dispatch_rows_aligned(T, k, E, align))


def dispatch_plan_noalloc(topk, E: int, expert_offsets, dst_rows, stream=None) -> None:
    """Routing plan without allocating (library-owned fixed scratch)."""
    T, k = topk.shape
    rc = load().tovl_dispatch_plan_noalloc(_ptr(topk), T, k, E, _ptr(expert_offsets), _ptr(dst_rows),
                                           _stream(stream))
    _check(None, rc, "tovl_dispatch_plan_noalloc")


class Handle:
    """Owns one tovl handle (control plane + sequence number)."""

    def __init__(self, device: int = 0, **cfg_fields):
        cfg = default_config(device)
        for k, v in cfg_fields.items():
            setattr(cfg, k, v)
        h = ctypes.c_void_p()
        _check(None, load().tovl_create(ctypes.byref(h), ctypes.byref(cfg)), "tovl_create")
        self.h = h
        self.cfg = cfg

    def close(self):
        if getattr(self, "h", None):
            load().tovl_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.close()

    # ------------------------------------------------------------ hot path
    def gather_gemm(self, shards, W, gathered, out, stream=None):
        """shards: list of [R, K] bf16 device tensors (or one [S, R, K] tensor)."""
        ptrs, S, R, K = _shard_ptrs(shards)
        rc = load().tovl_gather_gemm(self.h, ptrs, S, R, K, _ptr(W), W.shape[1], _ptr(gathered), _ptr(out),
                                     _stream(stream))
        _check(self.h, rc, "tovl_gather_gemm")

    def dispatch_grouped_gemm(self, x, topk, W, dispatched, expert_offsets, out, stream=None):
        T, H = x.shape
        k = topk.shape[1]
        E, _, N = W.shape
        rc = load().tovl_dispatch_grouped_gemm(self.h, _ptr(x), T, H, _ptr(topk), k, E, _ptr(W), N,
                                               _ptr(dispatched), _ptr(expert_offsets), _ptr(out),
                                               _stream(stream))
        _check(self.h, rc, "tovl_dispatch_grouped_gemm")

    # ------------------------------------------------------------ controls
    def gemm_only(self, A, W, out, stream=None):
        M, K = A.shape
        rc = load().tovl_gemm_only(self.h, _ptr(A), M, K, _ptr(W), W.shape[1], _ptr(out), _stream(stream))
        _check(self.h, rc, "tovl_gemm_only")

    def copy_only(self, shards, gathered, stream=None):
        ptrs, S, R, K = _shard_ptrs(shards)
        rc = load().tovl_copy_only(self.h, ptrs, S, R, K, _ptr(gathered), _stream(stream))
        _check(self.h, rc, "tovl_copy_only")

    def gemm_reduce_scatter(self, X, W, partials, out, stream=None):
        """Row-parallel layer on logical shards: ``partials[s] = X[s] @ W[s]``
        and ``out = sum_s partials[s]``.  X [S, M, Ks], W [S, Ks, N]."""
        S, M, Ks = X.shape
        N = W.shape[2]
        rc = load().tovl_gemm_reduce_scatter(self.h, _ptr(X), S, M, Ks, _ptr(W), N, _ptr(partials), _ptr(out),
                                             _stream(stream))
        _check(self.h, rc, "tovl_gemm_reduce_scatter")

    def combine(self, y, gate_w, staging, combined, stream=None):
        """Combine of the last dispatch round: ``staging[t*k+j] = y[dst(t,j)]``
        and ``combined[t] = bf16(sum_j gate_w[t,j] * staging[t*k+j])``."""
        N = y.shape[1]
        import torch
        if gate_w.dtype != torch.float32:
            raise TypeError("gate weights must be float32")
        rc = load().tovl_combine(self.h, _ptr(y), N, _ptr(gate_w), _ptr(staging), _ptr(combined), _stream(stream))
        _check(self.h, rc, "tovl_combine")

    # ------------------------------------------------------------ decode step
    def add_rmsnorm(self, x, weight, eps, residual=None, residual_out=None, out=None, q=None, q_scale=None, group=128,
                    stream=None):
        """``r = x + residual``, ``y = r * rsqrt(mean(r^2) + eps) * weight``: ``residual_out`` = r, ``out`` = y in bf16,
        ``q`` = y in e4m3 with ``q_scale`` [T, ceil(H/group)] (one scale per row with ``group=0``).  Tensors may be
        slices with unit stride in the last dimension (``q`` and ``q_scale`` contiguous)."""
        if _BF16 is None:
            _load_types()
        T, H = x.shape
        ldx = _matrix("x", x, _BF16, T, H)
        res = res_out = q_ptr = s_ptr = out_ptr = None
        rt = ldr = ldo = 0
        if residual is not None:
            rt = _type_of("residual", residual, (TOVL_BF16, TOVL_F32))
            ldr = _matrix("residual", residual, residual.dtype, T, H)
            if _matrix("residual_out", residual_out, residual.dtype, T, H) != ldr:
                raise TypeError("residual_out must have the strides of residual")
            res, res_out = residual.data_ptr(), residual_out.data_ptr()
        if out is not None:
            ldo = _matrix("out", out, _BF16, T, H)
            out_ptr = out.data_ptr()
        if q is not None:
            q_ptr = _dense("q", q, _E4M3, (T, H))
            s_ptr = _dense("q_scale", q_scale, _F32, (T, -(-H // group) if group else 1))
        rc = (_lib or load()).tovl_add_rmsnorm(self.h, x.data_ptr(), ldx, res, res_out, rt, ldr,
                                               _dense("weight", weight, _BF16, (H,)), eps, T, H, out_ptr, ldo, q_ptr, s_ptr,
                                               group, _stream(stream))
        if rc:
            _check(self.h, rc, "tovl_add_rmsnorm")

    def route_topk(self, logits, topk, gate_w, renormalize=True, stream=None):
        """The k experts of each token (``topk`` int32 [T, k], -1 where none is left) and their softmax weights."""
        if _BF16 is None:
            _load_types()
        T, E = logits.shape
        k = topk.shape[1]
        rc = (_lib or load()).tovl_route_topk(self.h, logits.data_ptr(), _type_of("logits", logits, (TOVL_BF16, TOVL_F32)),
                                              _matrix("logits", logits, logits.dtype, T, E), T, E, k, 1 if renormalize else 0,
                                              _dense("topk", topk, _I32, (T, k)), _dense("gate_w", gate_w, _F32, (T, k)),
                                              _stream(stream))
        if rc:
            _check(self.h, rc, "tovl_route_topk")

    def moe_decode_workspace(self, T: int, k: int, H: int, I: int) -> int:
        """Bytes of workspace of ``moe_decode`` and ``moe_decode_q4``."""
        n = load().tovl_moe_decode_workspace(self.h, T, k, H, I)
        if n < 0:
            raise TovlError(TOVL_ERR_UNSUPPORTED, "tovl_moe_decode_workspace")
        return n

    def moe_decode(self, x, topk, gate_w, W13, W2, out, workspace, stream=None):
        """The gated expert layer for up to 64 tokens: W13 [E, H, 2I] (gate columns, then up columns), W2 [E, I, H]."""
        if _BF16 is None:
            _load_types()
        T, H = x.shape
        k = topk.shape[1]
        E, I = W2.shape[:2]
        rc = (_lib or load()).tovl_moe_decode(
            self.h, x.data_ptr(), _matrix("x", x, _BF16, T, H), T, H, _dense("topk", topk, _I32, (T, k)),
            _dense("gate_w", gate_w, _F32, (T, k)), k, E, _dense("W13", W13, _BF16, (E, H, 2 * I)),
            _dense("W2", W2, _BF16, (E, I, H)), I, out.data_ptr(), _matrix("out", out, _BF16, T, H), workspace.data_ptr(),
            _bytes("workspace", workspace), _stream(stream))
        if rc:
            _check(self.h, rc, "tovl_moe_decode")

    def moe_decode_q4(self, x, topk, gate_w, W13, W2, group, out, workspace, stream=None):
        """``moe_decode`` with packed experts: W13 and W2 are (words, scales, zeros or None) as ``quantize_q4`` makes."""
        if _BF16 is None:
            _load_types()
        T, H = x.shape
        k = topk.shape[1]
        E, I8 = W2[0].shape[:2]
        I = I8 * 8
        rc = (_lib or load()).tovl_moe_decode_q4(
            self.h, x.data_ptr(), _matrix("x", x, _BF16, T, H), T, H, _dense("topk", topk, _I32, (T, k)),
            _dense("gate_w", gate_w, _F32, (T, k)), k, E, *_packed("W13", W13, (E,), H, 2 * I, group),
            *_packed("W2", W2, (E,), I, H, group), group, I, out.data_ptr(), _matrix("out", out, _BF16, T, H),
            workspace.data_ptr(), _bytes("workspace", workspace), _stream(stream))
        if rc:
            _check(self.h, rc, "tovl_moe_decode_q4")

    def matvec_q4_workspace(self, T: int, N: int) -> int:
        """Bytes of workspace of ``matvec_q4``."""
        n = load().tovl_matvec_q4_workspace(self.h, T, N)
        if n < 0:
            raise TovlError(TOVL_ERR_UNSUPPORTED, "tovl_matvec_q4_workspace")
        return n

    def matvec_q4(self, x, wq, w_scale, group, out, workspace, zero=None, x_scale=None, stream=None):
        """``out = x @ W`` for up to 64 rows and a packed matrix W [K, N]; x bf16, or e4m3 with ``x_scale``
        [T, ceil(K/128)]."""
        if _BF16 is None:
            _load_types()
        T, K = x.shape
        N = wq.shape[1]
        xt = _type_of("x", x, (TOVL_BF16, TOVL_E4M3))
        if (xt == TOVL_E4M3) != (x_scale is not None):
            raise TypeError("x_scale goes with e4m3 rows, and only with them")
        rc = (_lib or load()).tovl_matvec_q4(
            self.h, x.data_ptr(), xt, None if x_scale is None else _dense("x_scale", x_scale, _F32, (T, -(-K // 128))),
            _matrix("x", x, x.dtype, T, K), T, K, *_packed("wq", (wq, w_scale, zero), (), K, N, group), group, N,
            out.data_ptr(), _matrix("out", out, _BF16, T, N), workspace.data_ptr(), _bytes("workspace", workspace),
            _stream(stream))
        if rc:
            _check(self.h, rc, "tovl_matvec_q4")

    def quantize_q4(self, W, group=128, zeros=False, stream=None):
        """Packs bf16 W [E, K, N] or [K, N]: (words int32 [.., K/8, N], scales bf16 [.., K/group, N], zeros uint8 or
        None)."""
        import torch
        if W.dtype != torch.bfloat16 or W.dim() not in (2, 3) or not W.is_contiguous():
            raise TypeError("W must be a contiguous bfloat16 matrix or a stack of them")
        lead, (K, N) = tuple(W.shape[:-2]), W.shape[-2:]
        words = torch.empty(*lead, K // 8, N, dtype=torch.int32, device=W.device)
        scale = torch.empty(*lead, K // group, N, dtype=torch.bfloat16, device=W.device)
        zero = torch.empty(*lead, K // group, N, dtype=torch.uint8, device=W.device) if zeros else None
        rc = load().tovl_quantize_q4(self.h, _ptr(W), lead[0] if lead else 1, K, N, group, _ptr(words), _ptr(scale),
                                     _ptr(zero), _stream(stream))
        _check(self.h, rc, "tovl_quantize_q4")
        return words, scale, zero

    # ------------------------------------------------------------ paged attention step
    def page_plan(self, length, add, table, ring, state, page, length_out, state_out, slots, positions, starts, stream=None):
        """Pages, cache slots and positions of ``add`` [B] new tokens (-1: the request has ended) of requests that hold
        ``length`` tokens: takes pages from ``ring`` into ``table`` [B, width] and gives ended requests' back;
        ``length_out`` and ``state_out`` may be ``length`` and ``state``.  All int32."""
        if _BF16 is None:
            _load_types()
        i32 = _I32
        B, width = table.shape
        cap, pages = slots.numel(), ring.numel()
        ldt, last = table.stride()
        if not (length.dtype is i32 and add.dtype is i32 and table.dtype is i32 and ring.dtype is i32 and state.dtype is i32 and
                length_out.dtype is i32 and state_out.dtype is i32 and slots.dtype is i32 and positions.dtype is i32 and
                starts.dtype is i32):
            raise TypeError(f"tensors must be {i32}")
        if not (length.numel() == add.numel() == length_out.numel() == B and state.numel() == state_out.numel() == 4 and
                positions.numel() == cap and starts.numel() == B + 1):
            raise TypeError("length, add and length_out have B elements, starts one more, state and state_out 4, positions as "
                            "many as slots")
        if not (length.is_contiguous() and add.is_contiguous() and ring.is_contiguous() and state.is_contiguous() and
                length_out.is_contiguous() and state_out.is_contiguous() and slots.is_contiguous() and
                positions.is_contiguous() and starts.is_contiguous() and (last == 1 or width == 1)):
            raise TypeError("tensors must be contiguous, but for the distance of the table's rows")
        rc = (_lib or load()).tovl_page_plan(
            self.h, _PLAN_ARGS(length.data_ptr(), add.data_ptr(), table.data_ptr(), ring.data_ptr(), state.data_ptr(),
                               length_out.data_ptr(), state_out.data_ptr(), slots.data_ptr(), positions.data_ptr(),
                               starts.data_ptr(), ldt if B > 1 else width, B, width, pages, page, cap),
            stream if stream.__class__ is int else _stream(stream))
        if rc:
            _check(self.h, rc, "tovl_page_plan")

    def rope_append(self, q, k, v, positions, slots, cos_sin, cache, q_out, interleaved=False, stream=None):
        """Rotary embedding of q [T, Hq, dim] into ``q_out`` and of k [T, heads, dim], k and v to their ``slots`` of a
        ``KVCache`` (-1: not written); ``cos_sin`` fp32 [positions, rot] (None: no rotation).  Tensors may be slices of one
        projection's rows."""
        if _BF16 is None:
            _load_types()
        T, Hq, D = q.shape
        if D != cache.dim:
            raise TypeError(f"q must have {cache.dim} columns")
        far = rot = table = 0
        if cos_sin is not None:
            far, rot = cos_sin.shape
            if cos_sin.dtype is not _F32 or not cos_sin.is_contiguous():
                raise TypeError(f"cos_sin must be contiguous {_F32}")
            table = cos_sin.data_ptr()
        if not (positions.dtype is _I32 and slots.dtype is _I32 and positions.numel() == slots.numel() == T and
                positions.is_contiguous() and slots.is_contiguous()):
            raise TypeError(f"positions and slots must be contiguous {_I32} ({T},)")
        heads = cache.heads
        of_k = (T, heads, D)
        lq, hq, dq = q.stride()
        lk, hk, dk = k.stride()
        lv, hv, dv = v.stride()
        lo, ho, do = q_out.stride()
        if not (dq == dk == dv == do == 1 and hq == hk == hv == ho == D and q.dtype is k.dtype is v.dtype is q_out.dtype
                is _BF16 and q_out.shape == (T, Hq, D) and k.shape == of_k and v.shape == of_k):
            # (one by one: what is wrong, or a dimension of 1 with any stride)
            lq, lk, lv, lo = _heads("q", q, T, Hq, D), _heads("k", k, T, heads, D), _heads("v", v, T, heads, D), _heads(
                "q_out", q_out, T, Hq, D)
        elif T == 1:
            lq = lo = (Hq * D + 7) // 8 * 8
            lk = lv = (heads * D + 7) // 8 * 8
        rc = (_lib or load()).tovl_rope_append(
            self.h, _ROPE_ARGS(q.data_ptr(), k.data_ptr(), v.data_ptr(), q_out.data_ptr(), positions.data_ptr(),
                               slots.data_ptr(), table, cache.ref, lq, lk, lv, lo, T, Hq, far, rot, 1 if interleaved else 0),
            stream if stream.__class__ is int else _stream(stream))
        if rc:
            _check(self.h, rc, "tovl_rope_append")

    def attn_decode_workspace(self, Hq: int, heads: int, dim: int) -> int:
        """Bytes of workspace of ``attn_decode``, any batch and lengths."""
        n = load().tovl_attn_decode_workspace(self.h, Hq, heads, dim)
        if n < 0:
            raise TovlError(TOVL_ERR_UNSUPPORTED, "tovl_attn_decode_workspace")
        return n

    def attn_decode(self, q, cache, table, length, scale, out, workspace, window=0, lse=None, stream=None):
        """Attention of one new token per request: q [B, Hq, dim] over the ``length`` [B] cached tokens (the last
        ``window`` of them) in the pages of ``table`` [B, width]; ``lse`` fp32 [B, Hq]."""
        if _BF16 is None:
            _load_types()
        B, Hq, D = q.shape
        if D != cache.dim:
            raise TypeError(f"q must have {cache.dim} columns")
        rows, width = table.shape
        ldt, last = table.stride()
        if not (table.dtype is _I32 and length.dtype is _I32 and rows == length.numel() == B and length.is_contiguous() and
                (last == 1 or width == 1) and (lse is None or (lse.dtype is _F32 and lse.shape == (B, Hq) and lse.is_contiguous()))):
            raise TypeError(f"table must be {_I32} ({B}, width) with contiguous rows, length contiguous {_I32} ({B},), lse "
                            f"contiguous {_F32} ({B}, {Hq})")
        rc = (_lib or load()).tovl_attn_decode(
            self.h, _ATTN_ARGS(q.data_ptr(), out.data_ptr(), 0 if lse is None else lse.data_ptr(), table.data_ptr(),
                               length.data_ptr(), cache.ref, workspace.data_ptr(), _heads("q", q, B, Hq, D),
                               _heads("out", out, B, Hq, D), ldt if B > 1 else width, _bytes("workspace", workspace), B, Hq,
                               width, window, scale),
            stream if stream.__class__ is int else _stream(stream))
        if rc:
            _check(self.h, rc, "tovl_attn_decode")

    def gated_copy(self, src, dst, perm, gated=True, stamps=False, stream=None):
        n, rb = src.shape
        rc = load().tovl_gated_copy(self.h, _ptr(src), _ptr(dst), n, rb * src.element_size(), _ptr(perm),
                                    1 if gated else 0, 1 if stamps else 0, _stream(stream))
        _check(self.h, rc, "tovl_gated_copy")

    # ------------------------------------------------------------ diagnostics
    def sync_status(self) -> int:
        return load().tovl_sync_status(self.h)

    def ctrl_sizes(self):
        a, b = ctypes.c_int(), ctypes.c_int()
        _check(self.h, load().tovl_ctrl_sizes(self.h, ctypes.byref(a), ctypes.byref(b)), "tovl_ctrl_sizes")
        return a.value, b.value

    def read_ctrl(self):
        import numpy as np
        nc, nb = self.ctrl_sizes()
        slots = np.zeros(nc, np.int32)
        cnts = np.zeros(nc, np.int32)
        rb = np.zeros(nb, np.int32)
        seq = ctypes.c_longlong()
        rc = load().tovl_read_ctrl(self.h, slots.ctypes.data, cnts.ctypes.data, rb.ctypes.data, ctypes.byref(seq))
        _check(self.h, rc, "tovl_read_ctrl")
        return slots, cnts, rb, seq.value

    def read_plan(self, T: int, k: int, E: int):
        import numpy as np
        rows = dispatch_rows_aligned(T, k, E, self.get_option(OPT_DISPATCH_ALIGN))
        counts = np.zeros(E, np.int32)
        dst = np.zeros(T * k, np.int32)
        src = np.zeros(max(rows, 1), np.int32)
        pad = np.zeros(max(rows // 128, 1), np.int32)
        blk = np.zeros(max(rows // 128, 1), np.int32)
        m_pad = ctypes.c_int()
        rc = load().tovl_read_plan(self.h, counts.ctypes.data, dst.ctypes.data, src.ctypes.data, pad.ctypes.data,
                                   blk.ctypes.data, ctypes.byref(m_pad))
        _check(self.h, rc, "tovl_read_plan")
        m = m_pad.value
        return counts, dst, src[:m].copy(), pad[:m // 128].copy(), blk[:m // 128].copy(), m

    def set_option(self, option: int, value: int):
        _check(self.h, load().tovl_set_option(self.h, option, int(value)), "tovl_set_option")

    def get_option(self, option: int) -> int:
        v = ctypes.c_longlong()
        _check(self.h, load().tovl_get_option(self.h, option, ctypes.byref(v)), "tovl_get_option")
        return v.value

    def read_stats(self):
        arr = (ctypes.c_ulonglong * 8)()
        _check(self.h, load().tovl_read_stats(self.h, arr, 8), "tovl_read_stats")
        return list(arr)

    def read_latency(self, n: int):
        import numpy as np
        pub = np.zeros(n, np.int64)
        obs = np.zeros(n, np.int64)
        rc = load().tovl_read_latency(self.h, pub.ctypes.data, obs.ctypes.data, n)
        _check(self.h, rc, "tovl_read_latency")
        return pub, obs

    def read_trace(self, what: int, n: int):
        import numpy as np
        out = np.zeros(n, np.int64)
        _check(self.h, load().tovl_read_trace(self.h, what, out.ctypes.data, n), "tovl_read_trace")
        return out

    @property
    def num_sms(self) -> int:
        return load().tovl_num_sms(self.h)


def _shard_ptrs(shards):
    if hasattr(shards, "dim") and shards.dim() == 3:
        shards = [shards[s] for s in range(shards.shape[0])]
    S = len(shards)
    R, K = shards[0].shape
    arr = (ctypes.c_void_p * S)(*[_ptr(s) for s in shards])
    return arr, S, R, K
