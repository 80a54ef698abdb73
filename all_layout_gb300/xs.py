"""ctypes binding of libxs (include/xs.h): argument marshalling only.

Every step of the hot path runs in the library's CUDA kernels; this module
turns torch CUDA tensors into device pointers and a stream handle and raises
``XsError`` on a non-OK status. Importing it loads ``libxs.so`` and fails
loudly if the library has not been built; there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
import struct
from typing import NamedTuple

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libxs.so")
_HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       "include", "xs.h")

OK, ERR_INVALID, ERR_UNSUPPORTED, ERR_ALIGN, ERR_CUDA, ERR_TIMEOUT = range(6)
FLAG_COMPLETION_COUPLED = 1
MAX_SHARDS = 8


ROPE_ADJACENT = 1
_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


class XsError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


if not os.path.exists(_LIB_PATH):
    raise ImportError(f"libxs.so is not built ({_LIB_PATH}); run __graft_entry__.build()")
_lib = ctypes.CDLL(_LIB_PATH)

_vp, _i = ctypes.c_void_p, ctypes.c_int
_PP = ctypes.POINTER(ctypes.c_void_p)
_lib.xs_attn_fused.argtypes = [_vp, _vp, _vp, _PP, _i, _i, _i, _i, _i, _i, _vp]
_lib.xs_attn_fused_ex.argtypes = [_vp, _vp, _vp, _PP, _i, _i, _i, _i, _i, _i, _i, _vp, _vp]
_lib.xs_attn.argtypes = [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp]
_lib.xs_scatter.argtypes = [_vp, _PP, _i, _i, _i, _i, _i, _vp]
_lib.xs_attn_serial.argtypes = [_vp, _vp, _vp, _vp, _PP, _i, _i, _i, _i, _i, _vp]
_lib.xs_attn_ulysses.argtypes = [_PP, _PP, _PP, _PP] + [_i] * 8 + [_vp]
_lib.xs_store_burst_probe.argtypes = [_vp, ctypes.c_ulonglong, _i, ctypes.c_ulonglong, _i,
                                      ctypes.c_ulonglong, _i, _vp, _vp]
_lib.xs_attn_serial_noalloc.argtypes = [_vp, _vp, _vp, _PP, _i, _i, _i, _i, _i, _vp]
for _f in ("xs_attn_fused", "xs_attn_fused_ex", "xs_attn", "xs_scatter", "xs_attn_serial", "xs_attn_serial_noalloc",
           "xs_attn_ulysses", "xs_store_burst_probe",
           "xs_last_device_status", "xs_selftest_bounded_wait"):
    getattr(_lib, _f).restype = _i
_lib.xs_status_string.argtypes = [_i]
_lib.xs_status_string.restype = ctypes.c_char_p
_lib.xs_last_device_status.argtypes = [_vp]
_lib.xs_selftest_bounded_wait.argtypes = [_vp]
_lib.xs_set_wait_limit_ns.argtypes = [ctypes.c_ulonglong]
_lib.xs_set_wait_limit_ns.restype = ctypes.c_ulonglong
_lib.xs_abi_version.restype = _i
_lib.xs_selftest_exp2.argtypes = [_vp, _vp, _vp, _i, _vp]
_lib.xs_selftest_exp2.restype = _i
_lib.xs_set_workspace.argtypes = [_vp, ctypes.c_ulonglong, _vp]
_lib.xs_set_workspace.restype = _i
_lib.xs_workspace_bytes.argtypes = [_i, _i, _i, _i, ctypes.POINTER(ctypes.c_ulonglong),
                                    ctypes.POINTER(ctypes.c_int)]
_lib.xs_workspace_bytes.restype = _i


# struct xs_rope_tensor: x, y, weight, x_stride[3], y_stride[3], heads, rotate.
_ROPE_TENSOR = struct.Struct("@3P6q2i")
_lib.xs_rope.argtypes = [_vp, _i, _vp, ctypes.c_longlong, _vp, _i, _vp, _i, _i, _i, ctypes.c_float,
                         _i, _i, _i, _vp]
_lib.xs_rope.restype = _i

# struct xs_diff_args: q, k, v, their strides, lambda, norm_weight, kv_len, scale, eps, out_scale,
# B, H, H_kv, Nq, Nk, d.
_DIFF_ARGS = struct.Struct("@3P9q3P3f6i0q")
_lib.xs_diff_attn.argtypes = [_vp, _vp, _vp, _vp, ctypes.c_ulonglong, _vp]
_lib.xs_diff_attn_fused.argtypes = [_vp, _vp, _i, _vp, ctypes.c_ulonglong, _vp]
_lib.xs_diff_workspace_bytes.argtypes = [_i, _i, _i, _i, _i, _i, ctypes.POINTER(ctypes.c_ulonglong)]
for _f in ("xs_diff_attn", "xs_diff_attn_fused", "xs_diff_workspace_bytes"):
    getattr(_lib, _f).restype = _i
_STRIDES = struct.Struct("@3q")

# struct xs_pages: pages, stride, count. struct xs_cache: k, v, k_scale, v_scale, n_pages, H_kv,
# page_size, d. struct xs_prefix_args: q, prefix_k, prefix_v, k, v, kv_len, the strides of q (3),
# prefix_k, prefix_v (2 each), k, v (3 each), prefix_pages, pages, cache, scale, B, H, H_kv, Nq, Np,
# Nk, d.
_PAGES = struct.Struct("@Pqi0q")
_CACHE = struct.Struct("@4P4i0q")
_PREFIX_ARGS = struct.Struct("@6P13qPqi0qPqi0q4P4if7i0q")
_lib.xs_cache_write.argtypes = [_vp] * 8 + [_i, _i, _i, _vp]
_lib.xs_cache_read.argtypes = [_vp] * 8 + [_i, _i, _i, _vp]
_lib.xs_prefix_attn.argtypes = [_vp, _vp, _vp, _vp, ctypes.c_ulonglong, _vp]
_lib.xs_prefix_attn_fused.argtypes = [_vp, _vp, _i, _vp, ctypes.c_ulonglong, _vp]
_lib.xs_prefix_workspace_bytes.argtypes = [_i] * 8 + [ctypes.POINTER(ctypes.c_ulonglong)]
for _f in ("xs_cache_write", "xs_cache_read", "xs_prefix_attn", "xs_prefix_attn_fused", "xs_prefix_workspace_bytes"):
    getattr(_lib, _f).restype = _i


def library():
    """The loaded ctypes library (for direct C-ABI calls)."""
    return _lib


def library_path() -> str:
    return _LIB_PATH


def declared_symbols():
    """Function names declared in include/xs.h."""
    text = open(_HEADER).read()
    return sorted(set(re.findall(r"\b(xs_[a-z_]+)\s*\(", text)))


def status_string(status: int) -> str:
    return _lib.xs_status_string(int(status)).decode()


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return ctypes.c_void_p(t)
    return ctypes.c_void_p(t.data_ptr())


def _shard_array(shards):
    arr = (ctypes.c_void_p * max(1, len(shards)))()
    for i, s in enumerate(shards):
        arr[i] = s if isinstance(s, int) else (s.data_ptr() if s is not None else None)
    return ctypes.cast(arr, _PP), arr


def _check(status, what):
    if status != OK:
        raise XsError(status, what)


def _dims(q):
    B, H, N, d = q.shape
    return int(B), int(N), int(H), int(d)


def attn_fused(q, k, v, shards, store_tile: int = 8, stream=None):
    """Fused attention + shard layout. q, k, v: [B, H, N, d] bf16 CUDA tensors;
    shards: P tensors [B, N/P, H, d] bf16."""
    B, N, H, d = _dims(q)
    pp, keep = _shard_array(shards)
    _check(_lib.xs_attn_fused(_ptr(q), _ptr(k), _ptr(v), pp, B, N, H, d, len(shards),
                              int(store_tile), _stream(stream)), "xs_attn_fused")


def attn_fused_ex(q, k, v, shards, store_tile: int = 8, flags: int = 0, spans=None,
                  stream=None):
    """xs_attn_fused_ex: optional completion-coupled stores and per-tile store
    spans (spans: an int64 CUDA tensor of 2*B*H*(N/128) entries, or None)."""
    B, N, H, d = _dims(q)
    pp, keep = _shard_array(shards)
    _check(_lib.xs_attn_fused_ex(_ptr(q), _ptr(k), _ptr(v), pp, B, N, H, d, len(shards),
                                 int(store_tile), int(flags), _ptr(spans), _stream(stream)),
           "xs_attn_fused_ex")


def attn(q, k, v, o, stream=None):
    """Attention alone into o [B, H, N, d] bf16."""
    B, N, H, d = _dims(q)
    _check(_lib.xs_attn(_ptr(q), _ptr(k), _ptr(v), _ptr(o), B, N, H, d, _stream(stream)),
           "xs_attn")


def scatter(o, shards, stream=None):
    """Layout alone: o [B, H, N, d] -> shards."""
    B, N, H, d = _dims(o)
    pp, keep = _shard_array(shards)
    _check(_lib.xs_scatter(_ptr(o), pp, B, N, H, d, len(shards), _stream(stream)), "xs_scatter")


def attn_serial(q, k, v, o_scratch, shards, stream=None):
    """Serial execution: attention into o_scratch, then the layout kernel."""
    B, N, H, d = _dims(q)
    pp, keep = _shard_array(shards)
    _check(_lib.xs_attn_serial(_ptr(q), _ptr(k), _ptr(v), _ptr(o_scratch), pp, B, N, H, d,
                               len(shards), _stream(stream)), "xs_attn_serial")


def attn_ulysses(q_shards, k_shards, v_shards, out_shards, h0, H, store_tile: int = 8,
                 stream=None):
    """Both Ulysses All-to-Alls fused: q/k/v_shards are P sequence shards
    [B, N/P, H_total, d]; computes heads [h0, h0 + H) and stores them into
    out_shards [B, N/P, H_total, d]."""
    B, R, H_total, d = (int(x) for x in q_shards[0].shape)
    P = len(q_shards)
    qp, kq = _shard_array(q_shards)
    kp, kk = _shard_array(k_shards)
    vp, kv = _shard_array(v_shards)
    op, ko = _shard_array(out_shards)
    _check(_lib.xs_attn_ulysses(qp, kp, vp, op, B, R * P, H_total, int(h0), int(H), d, P,
                                int(store_tile), _stream(stream)), "xs_attn_ulysses")


def attn_serial_noalloc(q, k, v, shards, stream=None):
    """Serial execution with the intermediate o kept in the library's fixed
    scratch array (no device allocation; see xs_attn_serial_noalloc in xs.h)."""
    B, N, H, d = _dims(q)
    pp, keep = _shard_array(shards)
    _check(_lib.xs_attn_serial_noalloc(_ptr(q), _ptr(k), _ptr(v), pp, B, N, H, d, len(shards),
                                       _stream(stream)), "xs_attn_serial_noalloc")


def _require(ok, what):
    if not ok:
        raise ValueError(what)


def _on(index, stream, call, *args):
    """call(*args, stream) with device `index` current; the default stream is its current one.
    (The raw handle: building a Stream object takes longer than a small launch.)"""
    if torch.cuda.current_device() != index:
        with torch.cuda.device(index):
            return _on(index, stream, call, *args)
    handle = torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream(stream)
    return call(*args, handle)


def _operand(name, t, dtype, shape, index):
    """Checks an operand's type, place and shape; its strides."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != index or t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)} on cuda:{index}, not "
                         f"{t.dtype} of shape {tuple(t.shape)} on {t.device}")
    return t.stride()


def _vector(name, t, dtype, size, index):
    """Checks an optional vector operand; its address or 0."""
    if t is None:
        return 0
    if _operand(name, t, dtype, (size,), index)[0] != 1 and size > 1:
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


@functools.lru_cache(maxsize=64)
def _rope_axes(axis_dims, theta, freqs):
    """Host arrays of the C call (axis_dims; radians per position step of every pair) and the
    number of axes."""
    axis_dims = tuple(int(a) for a in axis_dims)
    n_axes, rot = len(axis_dims), sum(axis_dims)
    _require(1 <= n_axes <= 4 and all(a >= 2 and a % 2 == 0 for a in axis_dims),
             "axis_dims must name 1 to 4 axes of an even number of columns each")
    if freqs is None:
        freqs = [float(theta) ** (-2.0 * i / a) for a in axis_dims for i in range(a // 2)]
    _require(len(freqs) == rot // 2, f"freqs must have {rot // 2} entries")
    return (_i * n_axes)(*axis_dims), (ctypes.c_double * len(freqs))(*freqs), n_axes


def qkv_rope(q_in, k_in, v_in, q, k, v, pos, axis_dims, *, theta: float = 10000.0, freqs=None,
             q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = True,
             stream=None):
    """Rotary positions with several axes, with the RMS norm of q and k (see xs_rope in xs.h).

    q_in, k_in, v_in: [B, N, heads, d] views of the projection's output (any strides, d
    contiguous; bf16, fp16 or fp32); q, k, v: the outputs [B, heads, N, d], views of any strides
    too (an input's own .transpose(1, 2) updates it in place), of the same type or bf16. k and v
    may be None, in pairs with their inputs; v is moved without a rotation. pos: int32 [N, axes]
    or [B, N, axes]. axis_dims: columns of each axis (their sum is rotated); pair i of an axis
    of a columns turns by theta**(-2i/a) radians a step, or by freqs, one value a pair.
    interleaved: columns (2i, 2i + 1) are a pair; otherwise (i, i + rotated/2).
    q_weight, k_weight: fp32 [d], or None for no norm."""
    _require(isinstance(q_in, torch.Tensor) and q_in.is_cuda and q_in.dim() == 4,
             "q_in must be a CUDA tensor [B, N, heads, d]")
    B, N, _, d = q_in.shape
    dev, src = q_in.get_device(), q_in.dtype
    dst = q.dtype if isinstance(q, torch.Tensor) else None
    _require(src in _TYPES and dst in _TYPES, "q_in and q must be bf16, fp16 or fp32")
    dims, table, n_axes = _rope_axes(tuple(axis_dims), theta, None if freqs is None else tuple(map(float, freqs)))
    _require(isinstance(pos, torch.Tensor), "pos must be [N, axes] or [B, N, axes]")
    shared = pos.dim() == 2
    ps = _operand("pos", pos, torch.int32, (N, n_axes) if shared else (B, N, n_axes), dev)
    _require(pos.is_contiguous(), "pos must be contiguous")
    packed, n, rows = b"", 0, 0
    for name, x, y, weight, rotate in (("q", q_in, q, q_weight, 1), ("k", k_in, k, k_weight, 1),
                                       ("v", v_in, v, None, 0)):
        if x is None or y is None:
            _require(x is y, f"{name}_in and {name} must both be given, or neither")
            continue
        _require(isinstance(x, torch.Tensor) and x.dim() == 4, f"{name}_in must be [B, N, heads, d]")
        h = x.shape[2]
        a = _operand(name + "_in", x, src, (B, N, h, d), dev)
        b = _operand(name, y, dst, (B, h, N, d), dev)
        if (a[3] != 1 or b[3] != 1) and d > 1:
            raise ValueError(f"the last dimension of {name}_in and {name} must be contiguous")
        packed += _ROPE_TENSOR.pack(x.data_ptr(), y.data_ptr(), _vector(name + "_weight", weight, torch.float32, d, dev),
                                    a[0], a[1], a[2], b[0], b[2], b[1], h, rotate)
        n += 1
        rows += B * h * N
    if rows == 0:
        return
    _check(_on(dev, stream, _lib.xs_rope, packed, n, pos.data_ptr(), 0 if shared or B == 1 else ps[0], dims,
               n_axes, table, B, N, d, eps, ROPE_ADJACENT if interleaved else 0, _TYPES[src], _TYPES[dst]),
           "xs_rope")


def _diff_args(q, k, v, lam, kv_len, norm_weight, eps, out_scale, scale):
    """(struct xs_diff_args, B, H, Nq, d, device index) of checked operands."""
    _require(isinstance(q, torch.Tensor) and q.is_cuda and q.dim() == 4, "q must be a CUDA tensor [B, H, Nq, d]")
    _require(isinstance(k, torch.Tensor) and k.dim() == 4, "k must be a CUDA tensor [B, H_kv, Nk, d]")
    B, H, Nq, d = q.shape
    Hk, Nk = k.shape[1], k.shape[2]
    dev, bf16 = q.get_device(), torch.bfloat16
    qs = _operand("q", q, bf16, q.shape, dev)
    ks = _operand("k", k, bf16, (B, Hk, Nk, d), dev)
    vs = _operand("v", v, bf16, (B, Hk, Nk, d), dev)
    if (qs[3] != 1 or ks[3] != 1 or vs[3] != 1) and d > 1:
        raise ValueError("the last dimension of q, k and v must be contiguous")
    packed = _DIFF_ARGS.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), *qs[:3], *ks[:3], *vs[:3],
                             _vector("lam", lam, torch.float32, H, dev),
                             _vector("norm_weight", norm_weight, torch.float32, d, dev),
                             _vector("kv_len", kv_len, torch.int32, B, dev),
                             (max(d, 1) / 2) ** -0.5 if scale is None else scale, eps, out_scale, B, H, Hk, Nq, Nk, d)
    return packed, B, H, Nq, d, dev


def _diff_workspace(ws, index):
    if ws is None:
        return 0, 0
    if not isinstance(ws, torch.Tensor) or ws.get_device() != index or not ws.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{index}")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _diff_check(status, what, q, norm_weight, ws_bytes):
    if status == ERR_INVALID and q.shape[3] == 256 and norm_weight is not None:
        rows = min(128, (q.shape[2] + 7) // 8 * 8)
        if ws_bytes < 16384 + 1024 * rows:
            what += " (a norm at d = 256 needs a workspace: alloc_diff_workspace)"
    _check(status, what)


def diff_attn(q, k, v, o, lam, *, kv_len=None, norm_weight=None, eps: float = 1e-5,
              out_scale: float = 1.0, scale=None, workspace=None, stream=None):
    """Differential attention into o (see xs_diff_attn in xs.h). q: [B, H, Nq, d]; k, v:
    [B, H_kv, Nk, d]; o: [B, H, Nq, d]; bf16 views of any strides, d contiguous. The first d/2
    columns of q and k are the first map's. lam: fp32 [H]; norm_weight: fp32 [d] or None; kv_len:
    int32 [B] (keys that count) or None; scale: of the scores, 1/sqrt(d/2) if None; workspace:
    from alloc_diff_workspace, or None (at d = 256 a norm needs one). o must not overlap an input."""
    packed, B, H, Nq, d, dev = _diff_args(q, k, v, lam, kv_len, norm_weight, eps, out_scale, scale)
    os_ = _operand("o", o, torch.bfloat16, q.shape, dev)
    if os_[3] != 1 and d > 1:
        raise ValueError("the last dimension of o must be contiguous")
    if o.numel() == 0:
        return
    ws, n = _diff_workspace(workspace, dev)
    _diff_check(_on(dev, stream, _lib.xs_diff_attn, packed, o.data_ptr(), _STRIDES.pack(*os_[:3]), ws, n),
                "xs_diff_attn", q, norm_weight, n)


def diff_attn_fused(q, k, v, shards, lam, *, kv_len=None, norm_weight=None, eps: float = 1e-5,
                    out_scale: float = 1.0, scale=None, workspace=None, stream=None):
    """diff_attn with the fused shard layout: shards are P tensors [B, Nq/P, H, d] bf16
    (alloc_shards), as in attn_fused."""
    packed, B, H, Nq, d, dev = _diff_args(q, k, v, lam, kv_len, norm_weight, eps, out_scale, scale)
    P = len(shards)
    _require(1 <= P <= MAX_SHARDS and Nq % P == 0, f"1 to {MAX_SHARDS} shards that divide Nq = {Nq} are needed, not {P}")
    pointers = []
    for s in shards:
        _operand("shards", s, torch.bfloat16, (B, Nq // P, H, d), dev)
        _require(s.is_contiguous(), "shards must be contiguous")
        pointers.append(s.data_ptr())
    if q.numel() == 0:
        return
    ws, n = _diff_workspace(workspace, dev)
    _diff_check(_on(dev, stream, _lib.xs_diff_attn_fused, packed, (ctypes.c_void_p * P)(*pointers), P, ws, n),
                "xs_diff_attn_fused", q, norm_weight, n)


def alloc_diff_workspace(B: int, H: int, Nq: int, Nk: int, d: int, norm: bool = False, device="cuda"):
    """A zeroed workspace (through torch) with which diff_attn and diff_attn_fused of this shape can
    take every schedule; larger shapes' workspaces serve smaller ones."""
    n = ctypes.c_ulonglong(0)
    with torch.cuda.device(device):
        _check(_lib.xs_diff_workspace_bytes(B, H, Nq, Nk, d, 1 if norm else 0, ctypes.byref(n)),
               "xs_diff_workspace_bytes")
        return torch.zeros(int(n.value), dtype=torch.uint8, device=device)


class KVCache(NamedTuple):
    """A quantised key/value cache (see xs_cache in xs.h): k, v float8_e4m3fn [n_pages, H_kv,
    page_size, d]; k_scale, v_scale uint8 [n_pages, H_kv, page_size], a row's scale being
    2**(byte - 127). All contiguous, on one device."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor


def alloc_cache(n_pages: int, H_kv: int, page_size: int, d: int, device="cuda") -> KVCache:
    """A cache of zeros (through torch). page_size: a power of two from 16 to 1024."""
    codes = [torch.zeros((n_pages, H_kv, page_size, d), dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
             for _ in range(2)]
    return KVCache(*codes, *(torch.full((n_pages, H_kv, page_size), 127, dtype=torch.uint8, device=device)
                             for _ in range(2)))


def _cache_fields(cache, index):
    """Fields of struct xs_cache of a checked cache."""
    k, v, ks, vs = cache
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("cache.k must be a CUDA tensor [n_pages, H_kv, page_size, d]")
    shape = k.shape
    for name, t, dtype, want in (("k", k, torch.float8_e4m3fn, shape), ("v", v, torch.float8_e4m3fn, shape),
                                 ("k_scale", ks, torch.uint8, shape[:3]), ("v_scale", vs, torch.uint8, shape[:3])):
        _operand("cache." + name, t, dtype, want, index)
        if not t.is_contiguous():
            raise ValueError(f"cache.{name} must be contiguous")
    return (k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), *shape)


def _page_list(name, pages, B, index):
    """Fields of struct xs_pages: [n] (one list for all) or [B, n] int32."""
    if not isinstance(pages, torch.Tensor) or pages.dim() not in (1, 2):
        raise ValueError(f"{name} must be [n] or [B, n]")
    n = pages.shape[-1]
    st = _operand(name, pages, torch.int32, (n,) if pages.dim() == 1 else (B, n), index)
    if st[-1] != 1 and n > 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return pages.data_ptr() if pages.numel() else 0, st[0] if pages.dim() == 2 and B > 1 else 0, n


def _cache_rows(call, what, k, v, cache, pages, start, lens, stream):
    _require(isinstance(k, torch.Tensor) and k.is_cuda and k.dim() == 4, "k must be a CUDA tensor [B, H_kv, N, d]")
    B, H, N, d = k.shape
    dev, dtype = k.get_device(), k.dtype
    _require(dtype in _TYPES, "k and v must be bf16, fp16 or fp32")
    ks, vs = k.stride(), _operand("v", v, dtype, k.shape, dev)
    if (ks[3] != 1 or vs[3] != 1) and d > 1:
        raise ValueError("the last dimension of k and v must be contiguous")
    fields = _cache_fields(cache, dev)
    if fields[5] != H or fields[7] != d:
        raise ValueError(f"the cache holds {fields[5]} heads of {fields[7]} columns, k {H} of {d}")
    packed, lists = _CACHE.pack(*fields), _PAGES.pack(*_page_list("pages", pages, B, dev))
    start, lens = _vector("start", start, torch.int32, B, dev), _vector("lens", lens, torch.int32, B, dev)
    if k.numel() == 0:
        return
    _check(_on(dev, stream, call, packed, k.data_ptr(), v.data_ptr(), _STRIDES.pack(*ks[:3]), _STRIDES.pack(*vs[:3]),
               lists, start, lens, B, N, _TYPES[dtype]), what)


def cache_write(k, v, cache, pages, *, start=None, lens=None, stream=None):
    """Quantises rows into a cache (see xs_cache_write in xs.h). k, v: [B, H_kv, N, d] views of any
    strides, d contiguous (bf16, fp16 or fp32; a projection's [B, N, H_kv, d] transposed, too).
    Token n of request b goes to place start[b] + n of its pages: place i is row i % page_size of
    page pages[b, i // page_size]. pages: int32 [B, n], or [n] for one list; start, lens: int32 [B]
    or None (0; every token). Tokens from lens[b] on, and those without a page, are not stored."""
    _cache_rows(_lib.xs_cache_write, "xs_cache_write", k, v, cache, pages, start, lens, stream)


def cache_read(cache, pages, k, v, *, start=None, lens=None, stream=None):
    """The values that places start[b] + n of a cache stand for, into k and v [B, H_kv, N, d] (see
    xs_cache_read in xs.h; arguments as in cache_write). Tokens from lens[b] on are left as they
    were, those without a page become NaN."""
    _cache_rows(_lib.xs_cache_read, "xs_cache_read", k, v, cache, pages, start, lens, stream)


def _prefix_args(q, prefix_k, prefix_v, k, v, kv_len, cache, prefix_pages, prefix_len, pages, max_len, scale):
    """(struct xs_prefix_args, B, H, Nq, d, device index) of checked operands."""
    _require(isinstance(q, torch.Tensor) and q.is_cuda and q.dim() == 4, "q must be a CUDA tensor [B, H, Nq, d]")
    B, H, Nq, d = q.shape
    dev, bf16 = q.get_device(), torch.bfloat16
    qs = _operand("q", q, bf16, q.shape, dev)
    Hk = Np = Nk = 0
    fields, lists, own_lists = (0,) * 8, (0, 0, 0), (0, 0, 0)
    pointers, ps, ks = [0, 0, 0, 0], (0, 0, 0, 0), (0,) * 6
    contiguous = qs[3] == 1
    if cache is not None:
        fields = _cache_fields(cache, dev)
        Hk = fields[5]
    if prefix_k is not None:
        _require(isinstance(prefix_k, torch.Tensor) and prefix_k.dim() == 3, "prefix_k must be [H_kv, Np, d]")
        _require(prefix_pages is None and prefix_len is None, "the prefix lies in prefix_k and prefix_v or in prefix_pages")
        Hk, Np = Hk or prefix_k.shape[0], prefix_k.shape[1]
        a, b = (_operand(n, t, bf16, (Hk, Np, d), dev) for n, t in (("prefix_k", prefix_k), ("prefix_v", prefix_v)))
        pointers[:2] = prefix_k.data_ptr(), prefix_v.data_ptr()
        ps, contiguous = a[:2] + b[:2], contiguous and a[2] == 1 and b[2] == 1
    elif prefix_pages is not None:
        _require(cache is not None, "prefix_pages needs a cache")
        _require(prefix_v is None, "prefix_v needs prefix_k")
        _require(isinstance(prefix_pages, torch.Tensor) and prefix_pages.dim() == 1, "prefix_pages must be [n]")
        lists = _page_list("prefix_pages", prefix_pages, 1, dev)
        Np = lists[2] * fields[6] if prefix_len is None else prefix_len
        _require(0 <= Np <= lists[2] * fields[6], f"prefix_pages hold {lists[2] * fields[6]} keys, not {prefix_len}")
    else:
        _require(prefix_v is None and prefix_len is None, "prefix_v needs prefix_k, prefix_len prefix_pages")
    if k is not None:
        _require(isinstance(k, torch.Tensor) and k.dim() == 4, "k must be a CUDA tensor [B, H_kv, Nk, d]")
        _require(pages is None and max_len is None, "the own keys lie in k and v or in pages")
        Hk, Nk = Hk or k.shape[1], k.shape[2]
        a, b = (_operand(n, t, bf16, (B, Hk, Nk, d), dev) for n, t in (("k", k), ("v", v)))
        pointers[2:] = k.data_ptr(), v.data_ptr()
        ks, contiguous = a[:3] + b[:3], contiguous and a[3] == 1 and b[3] == 1
    elif pages is not None:
        _require(cache is not None, "pages needs a cache")
        _require(v is None, "v needs k")
        own_lists = _page_list("pages", pages, B, dev)
        Nk = own_lists[2] * fields[6] if max_len is None else max_len
        _require(0 <= Nk <= own_lists[2] * fields[6], f"pages hold {own_lists[2] * fields[6]} keys, not {max_len}")
    else:
        _require(v is None and max_len is None, "v needs k, max_len pages")
    if not contiguous and d > 1:
        raise ValueError("the last dimension of q, prefix_k, prefix_v, k and v must be contiguous")
    packed = _PREFIX_ARGS.pack(q.data_ptr(), *(p if n else 0 for p, n in zip(pointers, (Np, Np, Nk, Nk))),
                               _vector("kv_len", kv_len, torch.int32, B, dev), *qs[:3], *ps, *ks, *lists, *own_lists,
                               *fields, max(d, 1) ** -0.5 if scale is None else scale, B, H, Hk or H, Nq, Np, Nk, d)
    return packed, B, H, Nq, d, dev


def prefix_attn(q, o, *, prefix_k=None, prefix_v=None, k=None, v=None, kv_len=None, cache=None, prefix_pages=None,
                prefix_len=None, pages=None, max_len=None, scale=None, workspace=None, stream=None):
    """Attention of a batch of requests that share a prefix, into o (see xs_prefix_attn in xs.h).
    q, o: [B, H, Nq, d]. The prefix's keys and values: prefix_k, prefix_v [H_kv, Np, d], or the first
    prefix_len places of prefix_pages (int32 [n]) of `cache`. The requests' own ones: k, v
    [B, H_kv, Nk, d], or the first max_len places of pages (int32 [B, n]) of `cache`; of both the
    first kv_len[b] count (int32 [B], or None: all). Tensors are bf16 views of any strides, d
    contiguous (64 or 128). scale: of the scores, 1/sqrt(d) if None; workspace: from
    alloc_prefix_workspace, or None. o must not overlap an input."""
    packed, B, H, Nq, d, dev = _prefix_args(q, prefix_k, prefix_v, k, v, kv_len, cache, prefix_pages, prefix_len,
                                            pages, max_len, scale)
    os_ = _operand("o", o, torch.bfloat16, q.shape, dev)
    if os_[3] != 1 and d > 1:
        raise ValueError("the last dimension of o must be contiguous")
    if o.numel() == 0:
        return
    ws, n = _diff_workspace(workspace, dev)
    _check(_on(dev, stream, _lib.xs_prefix_attn, packed, o.data_ptr(), _STRIDES.pack(*os_[:3]), ws, n), "xs_prefix_attn")


def prefix_attn_fused(q, shards, *, prefix_k=None, prefix_v=None, k=None, v=None, kv_len=None, cache=None,
                      prefix_pages=None, prefix_len=None, pages=None, max_len=None, scale=None, workspace=None,
                      stream=None):
    """prefix_attn with the fused shard layout: shards are P tensors [B, Nq/P, H, d] bf16
    (alloc_shards), as in attn_fused."""
    packed, B, H, Nq, d, dev = _prefix_args(q, prefix_k, prefix_v, k, v, kv_len, cache, prefix_pages, prefix_len,
                                            pages, max_len, scale)
    P = len(shards)
    _require(1 <= P <= MAX_SHARDS and Nq % P == 0, f"1 to {MAX_SHARDS} shards that divide Nq = {Nq} are needed, not {P}")
    pointers = []
    for s in shards:
        _operand("shards", s, torch.bfloat16, (B, Nq // P, H, d), dev)
        _require(s.is_contiguous(), "shards must be contiguous")
        pointers.append(s.data_ptr())
    if q.numel() == 0:
        return
    ws, n = _diff_workspace(workspace, dev)
    _check(_on(dev, stream, _lib.xs_prefix_attn_fused, packed, (ctypes.c_void_p * P)(*pointers), P, ws, n),
           "xs_prefix_attn_fused")


def alloc_prefix_workspace(B: int, H: int, H_kv: int, Nq: int, Np: int, Nk: int, d: int, prefix_cached: bool = False,
                           own_cached: bool = False, device="cuda"):
    """A workspace (through torch) with which prefix_attn and prefix_attn_fused of this shape can take
    every schedule; larger shapes' workspaces serve smaller ones. prefix_cached, own_cached: which
    keys and values lie in a cache."""
    n = ctypes.c_ulonglong(0)
    with torch.cuda.device(device):
        _check(_lib.xs_prefix_workspace_bytes(B, H, H_kv, Nq, Np, Nk, d, (1 if prefix_cached else 0) | (2 if own_cached else 0),
                                              ctypes.byref(n)), "xs_prefix_workspace_bytes")
        return torch.empty(int(n.value), dtype=torch.uint8, device=device)


def store_burst_probe(dst, K, burst_bytes, n_bursts, gap_ns, mode, times, stream=None):
    """Store-burst probe (see xs_store_burst_probe): dst a uint8 CUDA tensor,
    times an int64 CUDA tensor of 2*K*n_bursts entries."""
    _check(_lib.xs_store_burst_probe(_ptr(dst), dst.numel() * dst.element_size(), int(K),
                                     int(burst_bytes), int(n_bursts), int(gap_ns), int(mode),
                                     _ptr(times), _stream(stream)), "xs_store_burst_probe")


def last_device_status(stream=None) -> int:
    return int(_lib.xs_last_device_status(_stream(stream)))


def set_wait_limit_ns(limit_ns: int) -> int:
    return int(_lib.xs_set_wait_limit_ns(int(limit_ns)))


def selftest_bounded_wait(stream=None):
    _check(_lib.xs_selftest_bounded_wait(_stream(stream)), "xs_selftest_bounded_wait")


def selftest_exp2(x, stream=None):
    """(polynomial 2^x, MUFU 2^x) for a float32 CUDA tensor x (see xs_selftest_exp2)."""
    x = x.contiguous()
    poly, mufu = torch.empty_like(x), torch.empty_like(x)
    _check(_lib.xs_selftest_exp2(_ptr(x), _ptr(poly), _ptr(mufu), x.numel(), _stream(stream)),
           "xs_selftest_exp2")
    return poly, mufu


def alloc_shards(B, N, H, d, P, device="cuda"):
    """P separate destination buffers [B, N/P, H, d] bf16 (one allocation each)."""
    return [torch.empty((B, N // P, H, d), dtype=torch.bfloat16, device=device)
            for _ in range(P)]


def set_workspace(ws=None, stream=None):
    """Registers a caller-owned uint8 CUDA tensor as the workspace of the
    balanced (stream-K) schedule on its device (None removes it). Keep the
    tensor alive while registered."""
    if ws is None:
        _check(_lib.xs_set_workspace(None, 0, _stream(stream)), "xs_set_workspace")
        return
    if not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    _check(_lib.xs_set_workspace(ws.data_ptr(), ws.numel() * ws.element_size(), _stream(stream)),
           "xs_set_workspace")


def workspace_bytes(B: int, N: int, H: int, d: int):
    """(bytes, cut): the workspace a launch of this shape would use with ample
    workspace, and 1 if it would take the balanced schedule (else 0)."""
    b, sp = ctypes.c_ulonglong(0), ctypes.c_int(0)
    _check(_lib.xs_workspace_bytes(B, N, H, d, ctypes.byref(b), ctypes.byref(sp)),
           "xs_workspace_bytes")
    return int(b.value), int(sp.value)


def alloc_workspace(B: int, N: int, H: int, d: int, device="cuda"):
    """Allocates (through torch) and registers the workspace a shape needs;
    returns the tensor (None when that shape keeps whole units)."""
    n, _ = workspace_bytes(B, N, H, d)
    if n == 0:
        return None
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    set_workspace(ws)
    return ws
