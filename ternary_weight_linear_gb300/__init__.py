"""Ternary-weight linear layer for GB300 (sm_103a).

A thin ctypes binding over the C ABI in ``include/tern.h`` (``libtern.so``,
built in-tree by ``ternary_weight_linear_gb300.build``).  The functions here
only marshal arguments: they check dtypes, shapes and devices of torch
tensors, pass raw device pointers and the current CUDA stream, and raise on a
non-zero status.  Every step of the layer runs in the library's CUDA kernels;
there is no CPU path.  If the library has not been built, importing works but
every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
import threading

import torch

from .build import LIB_PATH, build  # noqa: F401  (re-exported for convenience)

__all__ = [
    "tern_pack", "tern_quant_act_s8", "tern_linear", "tern_linear_workspace_bytes",
    "tern_select_rung", "tern_rung_name", "tern_last_rung", "tern_last_rung_id",
    "tern_last_launches",
    "tern_reload_env", "tern_device_status", "tern_status_string", "TernError", "load",
    "tern_linear_small_t_noalloc", "tern_repack_t5", "tern_rotate_bf16",
    "tern_linear_s8", "tern_add_rmsnorm_s8", "tern_kv8_append", "tern_kv8_attention",
    "tern_kv8_attention_workspace_bytes", "KV8_BLOCK",
    "tern_norm_add_norm_s8", "tern_rope_frequencies", "tern_rope", "tern_kv8_append_rope",
    "ROPE_SCALINGS", "tern_kv8_attention_shared", "tern_kv8_attention_shared_workspace_bytes",
    "tern_selftest_wait_timeout", "RUNGS",
    "EXPORTED_SYMBOLS", "NOALLOC_SCRATCH_BYTES", "SYNC_BYTES", "T5_GROUP_BYTES", "ROTATION_BLOCK",
]

RUNGS = {0: "gemv", 1: "small_t", 2: "small_t_tiled", 3: "s8", 4: "bf16"}

# Every symbol include/tern.h declares.
EXPORTED_SYMBOLS = (
    "tern_pack", "tern_quant_act_s8", "tern_linear_workspace_bytes", "tern_linear",
    "tern_select_rung", "tern_rung_name", "tern_last_rung_id", "tern_last_rung",
    "tern_last_launches", "tern_status_string", "tern_reload_env", "tern_device_status",
    "tern_linear_small_t_noalloc", "tern_repack_t5", "tern_rotate_bf16",
    "tern_selftest_wait_timeout", "tern_linear_s8", "tern_add_rmsnorm_s8", "tern_kv8_append",
    "tern_kv8_attention", "tern_kv8_attention_workspace_bytes", "tern_norm_add_norm_s8",
    "tern_rope_frequencies", "tern_rope", "tern_kv8_append_rope", "tern_kv8_attention_shared",
    "tern_kv8_attention_shared_workspace_bytes",
)

# Size of the library's fixed scratch for tern_linear_small_t_noalloc.
NOALLOC_SCRATCH_BYTES = 8 << 20
# Leading bytes of every workspace owned by the library (TERN_SYNC_BYTES):
# zero before first use, then left alone.
SYNC_BYTES = 4096
# Base-3 bytes per 128-weight group (five weights per byte, rounded up).
T5_GROUP_BYTES = 26
# Width of the Hadamard rotation's blocks along K.
ROTATION_BLOCK = 1024
# Tokens of a page of the int8 cache, which is the block that shares a scale.
KV8_BLOCK = 64
# tern_rope_scaling
ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "bands": 3, "ramp": 4}

# tern_type
_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


class _KV8Cache(ctypes.Structure):
    """tern_kv8_cache."""
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("codes", "scales", "page_table", "seq_lens", "row_start")] + [
                    (n, ctypes.c_int) for n in
                    ("pages", "seqs", "table_width", "kv_heads", "head_dim")]


class _Rotation(ctypes.Structure):
    """tern_rotation."""
    _fields_ = [("freq", ctypes.c_void_p), ("rotary_dim", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("magnitude", ctypes.c_float)]


_lock = threading.Lock()
_lib = None


class TernError(RuntimeError):
    def __init__(self, func: str, status: int):
        self.status = status
        super().__init__(f"{func} failed: {status_text(status)} ({status})")


def load() -> ctypes.CDLL:
    """Load libtern.so.  Raises if it has not been built (no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -c \"import __graft_entry__ as g; "
                f"g.build()\"` (or ternary_weight_linear_gb300.build.build())")
        lib = ctypes.CDLL(LIB_PATH)
        P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        lib.tern_pack.argtypes = [P, P, I, I, P, P]
        lib.tern_pack.restype = I
        lib.tern_quant_act_s8.argtypes = [P, P, P, I, I, P]
        lib.tern_quant_act_s8.restype = I
        lib.tern_linear_workspace_bytes.argtypes = [I, I, I]
        lib.tern_linear_workspace_bytes.restype = Z
        lib.tern_linear.argtypes = [P, P, P, P, I, I, I, P, Z, P]
        lib.tern_linear.restype = I
        lib.tern_select_rung.argtypes = [I]
        lib.tern_select_rung.restype = I
        lib.tern_rung_name.argtypes = [I]
        lib.tern_rung_name.restype = ctypes.c_char_p
        lib.tern_last_rung_id.argtypes = []
        lib.tern_last_rung_id.restype = I
        lib.tern_last_rung.argtypes = []
        lib.tern_last_rung.restype = ctypes.c_char_p
        lib.tern_last_launches.argtypes = []
        lib.tern_last_launches.restype = I
        lib.tern_status_string.argtypes = [I]
        lib.tern_status_string.restype = ctypes.c_char_p
        lib.tern_reload_env.argtypes = []
        lib.tern_reload_env.restype = None
        lib.tern_device_status.argtypes = [P]
        lib.tern_device_status.restype = I
        lib.tern_linear_small_t_noalloc.argtypes = [P, P, P, P, I, I, I, P]
        lib.tern_linear_small_t_noalloc.restype = I
        lib.tern_repack_t5.argtypes = [P, P, I, I, P, P]
        lib.tern_repack_t5.restype = I
        lib.tern_rotate_bf16.argtypes = [P, P, I, I, P]
        lib.tern_rotate_bf16.restype = I
        L, F = ctypes.c_longlong, ctypes.c_float
        C = ctypes.POINTER(_KV8Cache)
        lib.tern_linear_s8.argtypes = [P, P, P, P, P, I, I, I, P, Z, P]
        lib.tern_linear_s8.restype = I
        lib.tern_add_rmsnorm_s8.argtypes = [P, I, L, P, P, I, P, I, F, P, P, P, I, I, P]
        lib.tern_add_rmsnorm_s8.restype = I
        lib.tern_kv8_append.argtypes = [C, P, P, I, L, L, I, I, P]
        lib.tern_kv8_append.restype = I
        lib.tern_kv8_attention_workspace_bytes.argtypes = [I, I, I, I, I]
        lib.tern_kv8_attention_workspace_bytes.restype = Z
        lib.tern_kv8_attention.argtypes = [C, P, I, L, L, I, I, I, I, I, F, P, P, P, Z, P]
        lib.tern_kv8_attention.restype = I
        R, Dbl = ctypes.POINTER(_Rotation), ctypes.c_double
        lib.tern_norm_add_norm_s8.argtypes = [P, I, L, P, I, P, I, L, F, P, P, I, F, P, I, F, P, P,
                                              P, I, I, P]
        lib.tern_norm_add_norm_s8.restype = I
        lib.tern_rope_frequencies.argtypes = [I, Dbl, I, Dbl, Dbl, Dbl, Dbl, P, P]
        lib.tern_rope_frequencies.restype = I
        lib.tern_rope.argtypes = [P, I, L, L, P, I, L, L, P, R, I, I, I, P]
        lib.tern_rope.restype = I
        lib.tern_kv8_append_rope.argtypes = [C, P, P, P, I, L, L, I, L, L, P, R, P, I, I, I, P]
        lib.tern_kv8_append_rope.restype = I
        lib.tern_kv8_attention_shared_workspace_bytes.argtypes = [I, I, I, I, I]
        lib.tern_kv8_attention_shared_workspace_bytes.restype = Z
        lib.tern_kv8_attention_shared.argtypes = [C, P, I, L, L, I, I, I, I, I, I, F, P, P, P, Z, P]
        lib.tern_kv8_attention_shared.restype = I
        lib.tern_selftest_wait_timeout.argtypes = [I, P]
        lib.tern_selftest_wait_timeout.restype = I
        _lib = lib
        return lib


def status_text(status: int) -> str:
    try:
        return load().tern_status_string(int(status)).decode()
    except Exception:  # pragma: no cover
        return "status"


def tern_status_string(status: int) -> str:
    return load().tern_status_string(int(status)).decode()


def _check(func: str, rc: int) -> None:
    if rc != 0:
        raise TernError(func, rc)


# torch's own way to the current stream's handle without building a Stream
# object (0.2 us against 3 us, of calls that take ten)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None and _raw_device is not None:
            return _raw_stream(_raw_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dev(t: torch.Tensor, name: str, dtype, shape=None) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _strided(t: torch.Tensor, name: str, dtypes, ndim: int) -> int:
    """A CUDA tensor whose last dimension is contiguous; the others may be strided."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be one of {tuple(dtypes)}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {t.dim()}")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return t.data_ptr()


def _heads(t: torch.Tensor, name: str, dtypes):
    """The same for a [rows, heads, dim] operand: pointer, shape, (row, head) strides;
    where there is one row or head its stride does not matter.  Each of its properties
    is read once (they cost 0.1 us, of calls that take three)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be one of {tuple(dtypes)}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must have 3 dimensions, got {len(shape)}")
    rows, heads, dim = shape
    ld, hd, step = t.stride()
    if step != 1 and dim > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return t.data_ptr(), shape, (ld if rows > 1 else heads * dim, hd if heads > 1 else dim)


def _most(n) -> int:
    """An upper bound as a C int, which holds every size that there can be
    (ctypes would keep the low bits of a larger one)."""
    n = int(n)
    return n if -1 <= n < 2 ** 31 else -1 if n < 0 else 2 ** 31 - 1


_CURRENT = contextlib.nullcontext()


def _allocating(stream):
    """What a call allocates for itself belongs to the stream that it runs on."""
    if stream is None:
        return _CURRENT
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream)


# ------------------------------------------------------------------ entry points

def tern_pack(W: torch.Tensor, Wpacked: torch.Tensor | None = None,
              bad_count: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """int8 [N, K] ternary weights -> packed int32 [N, K/16] (uint32 bit patterns)."""
    N, K = W.shape
    if Wpacked is None:
        Wpacked = torch.empty((N, K // 16), dtype=torch.int32, device=W.device)
    pw = _dev(W, "W", torch.int8)
    pp = _dev(Wpacked, "Wpacked", torch.int32, (N, K // 16))
    pb = _dev(bad_count, "bad_count", torch.int32) if bad_count is not None else None
    _check("tern_pack", load().tern_pack(pw, pp, K, N, pb, _stream(stream)))
    return Wpacked


def tern_repack_t5(Pt5: torch.Tensor, K: int, Wpacked: torch.Tensor | None = None,
                   bad_count: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """base-3 packed weights uint8 [N, K/128*26] (five weights per byte) ->
    packed int32 [N, K/16] (uint32 bit patterns of the 2-bit layout)."""
    N = Pt5.shape[0]
    if Wpacked is None:
        Wpacked = torch.empty((N, K // 16), dtype=torch.int32, device=Pt5.device)
    pp = _dev(Pt5, "Pt5", torch.uint8, (N, K // 128 * T5_GROUP_BYTES))
    pw = _dev(Wpacked, "Wpacked", torch.int32, (N, K // 16))
    pb = _dev(bad_count, "bad_count", torch.int32) if bad_count is not None else None
    _check("tern_repack_t5", load().tern_repack_t5(pp, pw, int(K), N, pb, _stream(stream)))
    return Wpacked


def tern_rotate_bf16(x: torch.Tensor, xr: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Blockwise (1024) Hadamard rotation of bf16 activations [T, K]; xr may be x."""
    T, K = x.shape
    if xr is None:
        xr = torch.empty_like(x)
    _check("tern_rotate_bf16", load().tern_rotate_bf16(
        _dev(x, "x", torch.bfloat16), _dev(xr, "xr", torch.bfloat16, (T, K)), T, K,
        _stream(stream)))
    return xr


def tern_quant_act_s8(x: torch.Tensor, q: torch.Tensor | None = None,
                      x_scale: torch.Tensor | None = None, stream=None):
    """bf16 [T, K] -> (int8 codes [T, K], fp32 x_scale [T])."""
    T, K = x.shape
    if q is None:
        q = torch.empty((T, K), dtype=torch.int8, device=x.device)
    if x_scale is None:
        x_scale = torch.empty((T,), dtype=torch.float32, device=x.device)
    _check("tern_quant_act_s8", load().tern_quant_act_s8(
        _dev(x, "x", torch.bfloat16), _dev(q, "q", torch.int8, (T, K)),
        _dev(x_scale, "x_scale", torch.float32, (T,)), T, K, _stream(stream)))
    return q, x_scale


def tern_linear_workspace_bytes(T: int, K: int, N: int) -> int:
    return int(load().tern_linear_workspace_bytes(int(T), int(K), int(N)))


def tern_linear(Wpacked: torch.Tensor, scales: torch.Tensor, x: torch.Tensor,
                y: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """y [T, N] fp32 = ternary linear of bf16 x [T, K] with packed weights [N, K/16]
    and fp16 group scales [N, K/128].

    `workspace` (uint8, at least tern_linear_workspace_bytes(T, K, N) bytes) is
    allocated zeroed per call when omitted.  A workspace kept across calls
    must start with SYNC_BYTES zero bytes before its first use and then be
    left alone (the library keeps that area valid); zero it again after
    tern_device_status reports a timeout."""
    T, K = x.shape
    N = Wpacked.shape[0]
    if y is None:
        y = torch.empty((T, N), dtype=torch.float32, device=x.device)
    need = tern_linear_workspace_bytes(T, K, N)
    if workspace is None and need:
        # zeros: the leading synchronisation area must start zeroed
        workspace = torch.zeros(need, dtype=torch.uint8, device=x.device)
    pws = _dev(workspace, "workspace", torch.uint8) if workspace is not None else None
    nws = workspace.numel() if workspace is not None else 0
    rc = load().tern_linear(
        _dev(Wpacked, "Wpacked", torch.int32, (N, K // 16)),
        _dev(scales, "scales", torch.float16, (N, K // 128)),
        _dev(x, "x", torch.bfloat16), _dev(y, "y", torch.float32, (T, N)),
        T, K, N, pws, nws, _stream(stream))
    _check("tern_linear", rc)
    return y


def tern_linear_s8(Wpacked: torch.Tensor, scales: torch.Tensor, q: torch.Tensor,
                   x_scale: torch.Tensor, y: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y [T, N] fp32 = the ternary linear layer on int8 codes q [T, K] with
    token scales x_scale [T] (tern_quant_act_s8's or tern_add_rmsnorm_s8's):
    y[t, n] = x_scale[t] * sum_g scales[n, g] * (exact integer sum of group g).

    The workspace is tern_linear's, with the same rules.  Refused where
    TERN_ROTATE is set: codes cannot be rotated any more."""
    T, K = q.shape
    N = Wpacked.shape[0]
    need = tern_linear_workspace_bytes(T, K, N)
    with _allocating(stream):
        if y is None:
            y = torch.empty((T, N), dtype=torch.float32, device=q.device)
        if workspace is None and need:
            workspace = torch.zeros(need, dtype=torch.uint8, device=q.device)
    pws = _dev(workspace, "workspace", torch.uint8) if workspace is not None else None
    nws = workspace.numel() if workspace is not None else 0
    rc = load().tern_linear_s8(
        _dev(Wpacked, "Wpacked", torch.int32, (N, K // 16)),
        _dev(scales, "scales", torch.float16, (N, K // 128)),
        _dev(q, "q", torch.int8), _dev(x_scale, "x_scale", torch.float32, (T,)),
        _dev(y, "y", torch.float32, (T, N)), T, K, N, pws, nws, _stream(stream))
    _check("tern_linear_s8", rc)
    return y


def tern_add_rmsnorm_s8(x: torch.Tensor, weight: torch.Tensor,
                        residual: torch.Tensor | None = None, eps: float = 1e-6, *,
                        residual_out: torch.Tensor | None = None, q: torch.Tensor | None = None,
                        x_scale: torch.Tensor | None = None, y: torch.Tensor | None = None,
                        quantise: bool = True, stream=None):
    """Residual addition, root-mean-square norm and int8 codes of token rows.

    r = x + residual, rounded to the residual's type (r = x without one);
    y = r * weight / sqrt(mean(r^2) + eps); x_scale[t] = max|y[t]| / 127;
    q = rint(y / x_scale) in [-127, 127].  x [T, K] is fp32 (as tern_linear
    gives it) or bf16, its rows may be strided; residual bf16 or fp32; weight
    [K] bf16 or fp32.  `residual_out` (allocated when omitted) may be
    `residual` itself.  `y`, if given, is written with the bf16 norm output,
    which the bf16-activation rungs take; with quantise=False there are no
    codes beside it.  Returns (q, x_scale, r), None for what is not written
    (r without a residual)."""
    T, K = x.shape
    px = _strided(x, "x", (torch.float32, torch.bfloat16), 2)
    ld = x.stride(0) if T > 1 else K
    with _allocating(stream):
        if quantise:
            if q is None:
                q = torch.empty((T, K), dtype=torch.int8, device=x.device)
            if x_scale is None:
                x_scale = torch.empty((T,), dtype=torch.float32, device=x.device)
        elif q is not None or x_scale is not None or y is None:
            raise ValueError("quantise=False writes y alone")
        if residual is not None and residual_out is None:
            residual_out = torch.empty_like(residual)
    pr = pro = None
    rt = 0
    if residual is not None:
        if residual.dtype not in (torch.float32, torch.bfloat16):
            raise ValueError(f"residual must be float32 or bfloat16, got {residual.dtype}")
        rt = _TYPES[residual.dtype]
        pr = _dev(residual, "residual", residual.dtype, (T, K))
        pro = _dev(residual_out, "residual_out", residual.dtype, (T, K))
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    if weight.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"weight must be float32 or bfloat16, got {weight.dtype}")
    rc = load().tern_add_rmsnorm_s8(
        px, _TYPES[x.dtype], ld, pr, pro, rt, _dev(weight, "weight", weight.dtype, (K,)),
        _TYPES[weight.dtype], eps, _dev(q, "q", torch.int8, (T, K)) if quantise else None,
        _dev(x_scale, "x_scale", torch.float32, (T,)) if quantise else None,
        _dev(y, "y", torch.bfloat16, (T, K)) if y is not None else None, T, K, _stream(stream))
    _check("tern_add_rmsnorm_s8", rc)
    return q, x_scale, residual_out


def tern_norm_add_norm_s8(x: torch.Tensor, post_weight: torch.Tensor | None,
                          residual: torch.Tensor, weight: torch.Tensor,
                          gate: torch.Tensor | None = None, residual_scale: float = 1.0,
                          branch_scale: float = 1.0, eps: float = 1e-6, *,
                          residual_out: torch.Tensor | None = None,
                          q: torch.Tensor | None = None, x_scale: torch.Tensor | None = None,
                          y: torch.Tensor | None = None, quantise: bool = True, stream=None):
    """The norm after a block, its gate, the residual's addition, and the norm
    before the next block with its int8 codes.

    n = x * post_weight / sqrt(mean(x^2) + eps) (n = x where post_weight is
    None); r = residual_scale * residual + branch_scale * gate * n, rounded to
    the residual's type; y, x_scale and q of r and `weight` as in
    tern_add_rmsnorm_s8.  x [T, K] fp32 or bf16, its rows may be strided; gate
    [K] (the same for every token) or [T, K] (rows may be strided or expanded);
    residual [T, K]; all of fp32 or bf16.  `residual_out` (allocated when
    omitted) may be `residual` itself.  `y`, `quantise` as there.  Returns (q,
    x_scale, r), None for codes that are not written."""
    T, K = x.shape
    floats = (torch.float32, torch.bfloat16)
    px = _strided(x, "x", floats, 2)
    ld = x.stride(0) if T > 1 else K
    for t, name in ((residual, "residual"), (weight, "weight"), (post_weight, "post_weight")):
        if t is not None and t.dtype not in floats:
            raise ValueError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    pg, gt, gld = None, 0, 0
    if gate is not None:
        pg = _strided(gate, "gate", floats, gate.dim())
        if tuple(gate.shape) not in ((K,), (T, K)):
            raise ValueError(f"gate must have shape ({K},) or ({T}, {K}), got {tuple(gate.shape)}")
        gt = _TYPES[gate.dtype]
        gld = gate.stride(0) if gate.dim() == 2 and T > 1 else 0
    with _allocating(stream):
        if quantise:
            if q is None:
                q = torch.empty((T, K), dtype=torch.int8, device=x.device)
            if x_scale is None:
                x_scale = torch.empty((T,), dtype=torch.float32, device=x.device)
        elif q is not None or x_scale is not None or y is None:
            raise ValueError("quantise=False writes y alone")
        if residual_out is None:
            residual_out = torch.empty((T, K), dtype=residual.dtype, device=x.device)
    rc = load().tern_norm_add_norm_s8(
        px, _TYPES[x.dtype], ld,
        _dev(post_weight, "post_weight", post_weight.dtype, (K,)) if post_weight is not None
        else None, _TYPES[post_weight.dtype] if post_weight is not None else 0,
        pg, gt, gld, branch_scale, _dev(residual, "residual", residual.dtype, (T, K)),
        _dev(residual_out, "residual_out", residual.dtype, (T, K)), _TYPES[residual.dtype],
        residual_scale, _dev(weight, "weight", weight.dtype, (K,)), _TYPES[weight.dtype], eps,
        _dev(q, "q", torch.int8, (T, K)) if quantise else None,
        _dev(x_scale, "x_scale", torch.float32, (T,)) if quantise else None,
        _dev(y, "y", torch.bfloat16, (T, K)) if y is not None else None, T, K, _stream(stream))
    _check("tern_norm_add_norm_s8", rc)
    return q, x_scale, residual_out


def tern_rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str = "none",
                          factor: float = 1.0, trained: float = 0.0, low: float = 1.0,
                          high: float | None = None, device="cuda"):
    """The table of a rotation and its magnitude: (freq, magnitude).

    freq int64 [rotary_dim / 2] on `device`: turns a token in units of 2^-64 of
    theta_i = base^(-2 i / rotary_dim), scaled for a context `factor` times the
    `trained` one: "linear" (theta / factor), "base" (a larger base), "bands"
    (pairs that turn `high` = 4 times and more in the trained context stay,
    those that turn `low` = 1 times and less are slowed, linear in their turns
    between) or "ramp" (the same between `high` = 32 and `low` = 1 turns, linear
    in the pair's number, with a magnitude of 0.1 ln(factor) + 1)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {tuple(ROPE_SCALINGS)}, got {scaling!r}")
    if high is None:
        high = 4.0 if scaling == "bands" else 32.0
    rotary_dim = int(rotary_dim)
    freq = torch.zeros(max(1, rotary_dim // 2), dtype=torch.int64)
    magnitude = ctypes.c_float()
    _check("tern_rope_frequencies", load().tern_rope_frequencies(
        rotary_dim, base, ROPE_SCALINGS[scaling], factor, trained, low, high, freq.data_ptr(),
        ctypes.addressof(magnitude)))
    return freq.to(device), magnitude.value


def _rotation(freq, interleaved, magnitude) -> _Rotation:
    n = freq.numel()
    return _Rotation(_dev(freq, "freq", torch.int64, (n,)), 2 * n, bool(interleaved), magnitude)


def tern_rope(x: torch.Tensor, positions: torch.Tensor, freq: torch.Tensor, *,
              interleaved: bool = False, magnitude: float = 1.0,
              out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Rotary positions of rows x [T, heads, dim] (fp32, bf16 or fp16; rows and
    heads may be strided) at int32 positions [T].

    The first 2 * len(freq) elements of a head are pairs: the two halves, or
    neighbours where `interleaved`; freq and magnitude are those of
    tern_rope_frequencies.  `out` may be x itself, or of another of the three
    types; it is allocated like a dense x when omitted.  Negated positions turn
    backwards, which is also the gradient."""
    px, shape, xs = _heads(x, "x", _TYPES)
    T, heads, dim = shape
    if out is None:
        with _allocating(stream):
            out = torch.empty(shape, dtype=x.dtype, device=x.device)
    po, out_shape, os = _heads(out, "out", _TYPES)
    if out_shape != shape:
        raise ValueError(f"out must have shape {tuple(shape)}, got {tuple(out_shape)}")
    if T == 0 or heads == 0:
        return out
    rot = _rotation(freq, interleaved, magnitude)
    rc = load().tern_rope(
        px, _TYPES[x.dtype], *xs, po, _TYPES[out.dtype], *os,
        _dev(positions, "positions", torch.int32, (T,)), ctypes.byref(rot), T, heads, dim,
        _stream(stream))
    _check("tern_rope", rc)
    return out


def _kv8_cache(codes, scales, page_table, row_start, seq_lens) -> _KV8Cache:
    shape = codes.shape
    if len(shape) != 5 or shape[1] != 2 or shape[3] != KV8_BLOCK:
        raise ValueError(f"codes must be [pages, 2, kv_heads, {KV8_BLOCK}, head_dim], "
                         f"got {tuple(shape)}")
    pages, _, heads, _, dim = shape
    table = page_table.shape
    if len(table) != 2:
        raise ValueError("page_table must be [seqs, pages of a sequence]")
    seqs, width = table
    return _KV8Cache(
        _dev(codes, "codes", torch.int8), _dev(scales, "scales", torch.float32, (pages, 2, heads)),
        _dev(page_table, "page_table", torch.int32),
        _dev(seq_lens, "seq_lens", torch.int32, (seqs,)),
        _dev(row_start, "row_start", torch.int32, (seqs + 1,)), pages, seqs, width, heads, dim)


def tern_kv8_append(k: torch.Tensor, v: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                    page_table: torch.Tensor, row_start: torch.Tensor, seq_lens: torch.Tensor,
                    max_new: int | None = None, stream=None) -> None:
    """Write the new keys and values of every sequence into the paged int8 cache.

    k, v [rows, kv_heads, head_dim] (fp32, bf16 or fp16; rows and heads may be
    strided, both alike): the rows of sequence b are [row_start[b],
    row_start[b + 1]), its last tokens of seq_lens[b].  codes int8 [pages, 2,
    kv_heads, 64, head_dim] and scales fp32 [pages, 2, kv_heads] are updated;
    page_table int32 [seqs, width].  `max_new` bounds the new tokens of a
    sequence (the rows of the call when omitted: right, but with CTAs for as
    many pages of every sequence).  tern_device_status tells of inconsistent
    index arrays, whose sequences or pages are skipped."""
    cache = _kv8_cache(codes, scales, page_table, row_start, seq_lens)
    pk, shape, ks = _heads(k, "k", _TYPES)
    pv, v_shape, vs = _heads(v, "v", (k.dtype,))
    rows, kv_heads, dim = shape
    if shape != v_shape or ks != vs or kv_heads != cache.kv_heads or dim != cache.head_dim:
        raise ValueError("k and v must be [rows, kv_heads, head_dim] with the same strides")
    rc = load().tern_kv8_append(
        ctypes.byref(cache), pk, pv, _TYPES[k.dtype], *ks, rows,
        max(1, rows) if max_new is None else _most(max_new), _stream(stream))
    _check("tern_kv8_append", rc)


def tern_kv8_append_rope(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor,
                         codes: torch.Tensor, scales: torch.Tensor, page_table: torch.Tensor,
                         row_start: torch.Tensor, seq_lens: torch.Tensor, freq: torch.Tensor, *,
                         interleaved: bool = False, magnitude: float = 1.0,
                         positions: torch.Tensor | None = None, max_new: int | None = None,
                         q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
    """tern_kv8_append with the keys turned on the way, and the same rows'
    queries turned into q_out, in one launch.

    q [rows, heads, head_dim] of k's type (rows and heads may be strided), or
    None; q_out bf16 (allocated when omitted) or fp16 [rows, heads, head_dim].
    The rotation as in tern_rope, at the tokens' positions in the cache or at
    int32 `positions` [rows].  Returns q_out."""
    cache = _kv8_cache(codes, scales, page_table, row_start, seq_lens)
    pk, shape, ks = _heads(k, "k", _TYPES)
    dtype = k.dtype
    pv, v_shape, vs = _heads(v, "v", (dtype,))
    rows, kv_heads, dim = shape
    if shape != v_shape or ks != vs or kv_heads != cache.kv_heads or dim != cache.head_dim:
        raise ValueError("k and v must be [rows, kv_heads, head_dim] with the same strides")
    pq = po = None
    qs, heads, qt = (0, 0), 0, 0
    if q is not None:
        pq, q_shape, qs = _heads(q, "q", (dtype,))
        heads = q_shape[1]
        if q_shape != (rows, heads, dim):
            raise ValueError(f"q must be [{rows}, heads, {dim}], got {tuple(q_shape)}")
        if q_out is None:
            with _allocating(stream):
                q_out = torch.empty((rows, heads, dim), dtype=torch.bfloat16, device=q.device)
        q_type = q_out.dtype
        if q_type not in (torch.bfloat16, torch.float16):
            raise ValueError(f"q_out must be bfloat16 or float16, got {q_type}")
        po, qt = _dev(q_out, "q_out", q_type, q_shape), _TYPES[q_type]
    elif q_out is not None:
        raise ValueError("q_out without q")
    rot = _rotation(freq, interleaved, magnitude)
    rc = load().tern_kv8_append_rope(
        ctypes.byref(cache), pq, pk, pv, _TYPES[dtype], *qs, heads, *ks,
        _dev(positions, "positions", torch.int32, (rows,)) if positions is not None else None,
        ctypes.byref(rot), po, qt, rows, max(1, rows) if max_new is None else _most(max_new),
        _stream(stream))
    _check("tern_kv8_append_rope", rc)
    return q_out


def tern_kv8_attention_workspace_bytes(seqs: int, rows: int, heads: int, kv_heads: int,
                                       head_dim: int) -> int:
    return int(load().tern_kv8_attention_workspace_bytes(int(seqs), int(rows), int(heads),
                                                         int(kv_heads), int(head_dim)))


def tern_kv8_attention(q: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                       page_table: torch.Tensor, row_start: torch.Tensor, seq_lens: torch.Tensor,
                       max_new: int | None = None, window: int = 0, sinks: int = 0,
                       softmax_scale: float | None = None, out: torch.Tensor | None = None,
                       lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """Causal attention of the newest tokens of every sequence over the paged
    int8 cache (which already holds them).

    q [rows, heads, head_dim] (bf16 or fp16, rows and heads may be strided),
    rows of sequence b at [row_start[b], row_start[b + 1]).  window > 0: a
    token sees the last `window` tokens, itself included, and the first
    `sinks`.  softmax_scale defaults to head_dim ** -0.5.  Returns `out`
    [rows, heads, head_dim] of q's type; `lse` fp32 [rows, heads], if given,
    is written with the logarithm of the softmax's sum.

    Give `max_new`, the most new tokens of a sequence: without it the call's
    rows are taken, and a decode step of several sequences runs the prompt
    kernel for nothing and wider tiles.  page_table's width also chooses the
    kernels of 17 to 24 rows a head: a tight one is best.

    `workspace` (uint8, tern_kv8_attention_workspace_bytes bytes) is allocated
    zeroed per call when omitted; one kept across calls starts with SYNC_BYTES
    zero bytes and is then left alone."""
    return _attention("tern_kv8_attention", (), q, codes, scales, page_table, row_start, seq_lens,
                      max_new, window, sinks, softmax_scale, out, lse, workspace, stream)


def _attention(name, shared, q, codes, scales, page_table, row_start, seq_lens, max_new, window,
               sinks, softmax_scale, out, lse, workspace, stream):
    """The entry `name`; shared: its arguments that the ordinary one lacks."""
    cache = _kv8_cache(codes, scales, page_table, row_start, seq_lens)
    pq, shape, qs = _heads(q, "q", (torch.bfloat16, torch.float16))
    rows, heads, dim = shape
    dtype = q.dtype
    if dim != cache.head_dim:
        raise ValueError(f"q's head_dim {dim} is not the cache's {cache.head_dim}")
    with _allocating(stream):
        if out is None:
            out = torch.empty(shape, dtype=dtype, device=q.device)
        if workspace is None:
            need = (tern_kv8_attention_shared_workspace_bytes
                    if shared and shared[0] and cache.seqs > 1
                    else tern_kv8_attention_workspace_bytes)
            workspace = torch.empty(need(cache.seqs, max(1, rows), heads, cache.kv_heads, dim),
                                    dtype=torch.uint8, device=q.device)
            workspace[:SYNC_BYTES].zero_()  # the rest is scratch
    rc = getattr(load(), name)(
        ctypes.byref(cache), pq, _TYPES[dtype], *qs, rows, heads, *shared,
        max(1, rows) if max_new is None else _most(max_new), _most(window), _most(sinks),
        1 / math.sqrt(dim) if softmax_scale is None else float(softmax_scale),
        _dev(out, "out", dtype, shape),
        _dev(lse, "lse", torch.float32, (rows, heads)) if lse is not None else None,
        _dev(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream))
    _check(name, rc)
    return out


def tern_kv8_attention_shared_workspace_bytes(seqs: int, rows: int, heads: int, kv_heads: int,
                                              head_dim: int) -> int:
    return int(load().tern_kv8_attention_shared_workspace_bytes(int(seqs), int(rows), int(heads),
                                                                int(kv_heads), int(head_dim)))


def tern_kv8_attention_shared(q: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                              page_table: torch.Tensor, row_start: torch.Tensor,
                              seq_lens: torch.Tensor, shared: int, max_new: int | None = None,
                              window: int = 0, sinks: int = 0,
                              softmax_scale: float | None = None,
                              out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                              workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """tern_kv8_attention for a batch whose sequences begin with the same pages.

    The first `shared` tokens (a multiple of 64) of every sequence lie in the
    same pages: the first shared / 64 entries of the rows of page_table are
    alike.  They are read once for all rows of the batch where that gains by the
    table's width (a tight table is best).  New tokens lie behind them.  The result
    is tern_kv8_attention's; the other arguments are as there, the workspace of
    tern_kv8_attention_shared_workspace_bytes bytes (of tern_kv8_attention's where
    `shared` is 0 or there is one sequence)."""
    return _attention("tern_kv8_attention_shared", (_most(shared),), q, codes, scales, page_table,
                      row_start, seq_lens, max_new, window, sinks, softmax_scale, out, lse,
                      workspace, stream)


def tern_linear_small_t_noalloc(Wpacked: torch.Tensor, scales: torch.Tensor, x: torch.Tensor,
                                y: torch.Tensor, stream=None) -> torch.Tensor:
    """tern_linear for T = 1..16 that takes no workspace and allocates nothing.

    For callers that cannot allocate device memory (plug-in interfaces that
    pass only inputs and outputs, engines that forbid allocation after
    start-up, latency-critical code where cudaMalloc/cudaFree would
    synchronise the device).  The library's fixed 4 MiB device scratch is
    shared by every call on a device, so calls must not overlap on the GPU.
    The first call on a device does per-device set-up and should come before
    any stream capture.  `y` must be given (fp32 [T, N])."""
    T, K = x.shape
    N = Wpacked.shape[0]
    rc = load().tern_linear_small_t_noalloc(
        _dev(Wpacked, "Wpacked", torch.int32, (N, K // 16)),
        _dev(scales, "scales", torch.float16, (N, K // 128)),
        _dev(x, "x", torch.bfloat16), _dev(y, "y", torch.float32, (T, N)),
        T, K, N, _stream(stream))
    _check("tern_linear_small_t_noalloc", rc)
    return y


def tern_select_rung(T: int) -> int:
    return int(load().tern_select_rung(int(T)))


def tern_rung_name(rung: int) -> str:
    return load().tern_rung_name(int(rung)).decode()


def tern_last_rung() -> str:
    return load().tern_last_rung().decode()


def tern_last_rung_id() -> int:
    return int(load().tern_last_rung_id())


def tern_last_launches() -> int:
    """Kernels this thread's last successful tern_linear launched."""
    return int(load().tern_last_launches())


def tern_reload_env() -> None:
    load().tern_reload_env()


def tern_selftest_wait_timeout(which: int, stream=None) -> None:
    """Launch the failure-path diagnostic: a kernel whose bounded wait (0: an
    mbarrier, 1: a device counter) runs out after 2 s and records the timeout;
    tern_device_status then returns TERN_ETIMEOUT (-6)."""
    _check("tern_selftest_wait_timeout",
           load().tern_selftest_wait_timeout(int(which), _stream(stream)))


def tern_device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error word."""
    return int(load().tern_device_status(_stream(stream)))
