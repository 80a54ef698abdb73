"""Differential attention without a GPU: the refusals of its C entry points and of its binding."""
import ctypes
import math

import pytest
import torch

A = 0x10000   # a 256-byte aligned fake device address; never dereferenced


@pytest.fixture(scope="module")
def xs():
    import __graft_entry__
    __graft_entry__.build()
    from all_layout_gb300 import xs as _xs
    return _xs


def _call(xs, q=A, k=A, v=A, lam=A, w=0, kv_len=0, scale=0.125, eps=1e-5, out_scale=1.0, B=0, H=4, Hk=2, Nq=256,
          Nk=100, d=64, qs=None, ks=None, vs=None, os_=None, o=A, shards=None, P=None, ws=None, ws_bytes=0, args=True):
    """B = 0 by default: a call that passes every check then ends as an empty problem."""
    qs = qs or (H * Nq * d, Nq * d, d)
    ks = ks or (Hk * Nk * d, Nk * d, d)
    packed = xs._DIFF_ARGS.pack(q or 0, k or 0, v or 0, *qs, *ks, *(vs or ks), lam or 0, w, kv_len, scale, eps,
                                out_scale, B, H, Hk, Nq, Nk, d)
    lib, packed = xs.library(), packed if args else None
    if shards is not None:
        arr = (ctypes.c_void_p * max(1, len(shards)))(*shards)
        return lib.xs_diff_attn_fused(packed, arr, len(shards) if P is None else P, ws, ws_bytes, None)
    return lib.xs_diff_attn(packed, o, xs._STRIDES.pack(*(os_ or qs)), ws, ws_bytes, None)


def test_argument_struct_size(xs):
    """3 pointers, 9 strides, 3 pointers, 3 floats, 6 ints, padded to 8 bytes."""
    assert xs._DIFF_ARGS.size == 24 + 72 + 24 + 12 + 24 + 4


@pytest.mark.parametrize("kw,code", [
    (dict(args=False), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(lam=None), 1),
    (dict(o=None), 1), (dict(B=-1), 1), (dict(H=-1), 1), (dict(Hk=-1), 1), (dict(Nq=-1), 1), (dict(Nk=-1), 1),
    (dict(Hk=0), 1), (dict(Hk=3), 1), (dict(Hk=8), 1),
    (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=math.inf), 1), (dict(scale=math.nan), 1),
    (dict(eps=-1e-9), 1), (dict(eps=math.nan), 1), (dict(out_scale=math.inf), 1), (dict(out_scale=math.nan), 1),
    (dict(shards=(A, None)), 1), (dict(shards=(A,) * 9, Nq=288), 1), (dict(shards=(A,) * 3), 1), (dict(shards=(A,), P=0), 1),
    (dict(ws=None, ws_bytes=64), 1),
    (dict(B=2, qs=(0, 64 * 256, 64)), 1), (dict(B=2, qs=(65536, 0, 64)), 1), (dict(B=2, ks=(12800, 6400, 32)), 1),
    (dict(B=2, vs=(12800, -6400, 64)), 1), (dict(B=2, os_=(65536, 16384, 8)), 1),
    (dict(B=2, d=256, w=A, shards=(A,)), 1), (dict(B=2, d=256, w=A, shards=(A,), ws=A, ws_bytes=16384 + 100), 1),
    (dict(d=96), 2), (dict(d=32), 2), (dict(d=512), 2), (dict(B=1 << 20, H=1 << 12, Hk=1, qs=(1 << 36, 1 << 20, 64)), 2),
    (dict(q=A + 8), 3), (dict(k=A + 2), 3), (dict(v=A + 4), 3), (dict(o=A + 8), 3), (dict(w=A + 8), 3), (dict(lam=A + 2), 3),
    (dict(kv_len=A + 1), 3), (dict(ws=A + 16, ws_bytes=1 << 20), 3), (dict(shards=(A, A + 8)), 3),
    (dict(B=2, qs=(65536, 16384, 68)), 3), (dict(B=2, ks=(12800, 6401, 64)), 3), (dict(B=2, os_=(65540, 16384, 64)), 3),
    (dict(), 0), (dict(B=2, H=0), 0), (dict(B=2, Nq=0), 0), (dict(k=None, v=None, Nk=0), 0), (dict(shards=(A,) * 8), 0),
    (dict(ws=A, ws_bytes=1 << 20), 0),
])
def test_refusals(xs, kw, code):
    assert _call(xs, **kw) == code


def test_null_shards_and_strides(xs):
    lib = xs.library()
    packed = xs._DIFF_ARGS.pack(A, A, A, *(64,) * 9, A, 0, 0, 0.1, 0.0, 1.0, 0, 1, 1, 8, 8, 64)
    assert lib.xs_diff_attn_fused(packed, None, 1, None, 0, None) == xs.ERR_INVALID
    assert lib.xs_diff_attn(packed, A, None, None, 0, None) == xs.ERR_INVALID


def test_workspace_bytes_refusals(xs):
    lib, n = xs.library(), ctypes.c_ulonglong(7)
    assert lib.xs_diff_workspace_bytes(1, 1, 1, 1, 64, 0, None) == xs.ERR_INVALID
    assert lib.xs_diff_workspace_bytes(1, 1, -1, 1, 64, 0, ctypes.byref(n)) == xs.ERR_INVALID
    assert lib.xs_diff_workspace_bytes(1, 1, 1, 1, 96, 0, ctypes.byref(n)) == xs.ERR_UNSUPPORTED
    assert lib.xs_diff_workspace_bytes(1, 1, 0, 1, 64, 0, ctypes.byref(n)) == xs.OK and n.value == 0


def test_binding_refuses_cpu_tensors(xs):
    t = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        xs.diff_attn(t, t, t, t, torch.zeros(2))
    with pytest.raises(ValueError, match="CUDA"):
        xs.diff_attn_fused(t, t, t, [t], torch.zeros(2))
