"""Shared-prefix attention without a GPU: refusals of the C entry points (before any device work) and of the binding."""
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


def _call(xs, q=A, pk=A, pv=A, k=A, v=A, kv_len=None, qst=None, pst=None, kst=None, ppages=0, pcount=0, pages=0, count=0,
          cache=(0,) * 8, scale=0.125, B=2, H=4, Hk=2, Nq=8, Np=40, Nk=24, d=64, o=2 * A, ost=None, ws=None, ws_bytes=0,
          shards=None, P=None, args=True, o_stride=True):
    z = lambda x: x or 0   # noqa: E731
    ps = pst or (Np * d, d)
    ks = kst or (Hk * Nk * d, Nk * d, d)
    packed = xs._PREFIX_ARGS.pack(z(q), z(pk), z(pv), z(k), z(v), z(kv_len), *(qst or (H * Nq * d, Nq * d, d)), *ps, *ps,
                                  *ks, *ks, z(ppages), 0, pcount, z(pages), count, count, *cache, scale, B, H, Hk, Nq,
                                  Np, Nk, d)
    lib = xs.library()
    if shards is not None:
        arr = (ctypes.c_void_p * max(1, len(shards)))(*shards)
        return lib.xs_prefix_attn_fused(packed if args else None, arr, len(shards) if P is None else P, ws, ws_bytes, None)
    st = xs._STRIDES.pack(*(ost or (H * Nq * d, Nq * d, d)))
    return lib.xs_prefix_attn(packed if args else None, o, st if o_stride else None, ws, ws_bytes, None)


CACHE = (A, A, A, A, 8, 2, 64, 64)
CACHED = dict(pk=None, pv=None, k=None, v=None, ppages=A, pcount=1, pages=A, count=1, cache=CACHE)


@pytest.mark.parametrize("kw,code", [
    (dict(args=False), 1), (dict(q=None), 1), (dict(o=None), 1), (dict(o_stride=False), 1), (dict(pv=None), 1),
    (dict(v=None), 1), (dict(pk=None), 1), (dict(k=None), 1),                  # cached, and no cache
    (dict(B=-1), 1), (dict(H=-4), 1), (dict(Hk=0), 1), (dict(H=3), 1), (dict(Nq=-1), 1), (dict(Np=-1), 1), (dict(Nk=-1), 1),
    (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=math.nan), 1), (dict(scale=math.inf), 1),
    (dict(shards=(A, None)), 1), (dict(shards=(A,) * 9), 1), (dict(shards=(A,) * 3), 1), (dict(shards=(A,), P=0), 1),
    (dict(ws_bytes=4096), 1), (dict(qst=(2048, 32, 64)), 1), (dict(ost=(2048, 512, 0)), 1), (dict(pst=(0, 64)), 1),
    (dict(kst=(1536, 768, 32)), 1),
    (dict(CACHED, cache=(A, A, A, A, 8, 3, 64, 64)), 1), (dict(CACHED, cache=(A, A, A, A, 8, 2, 64, 128)), 1),
    (dict(CACHED, cache=(A, 0, A, A, 8, 2, 64, 64)), 1), (dict(CACHED, ppages=None), 1), (dict(CACHED, pages=None), 1),
    (dict(CACHED, pcount=-1), 1),
    (dict(d=32), 2), (dict(d=256), 2), (dict(d=96), 2), (dict(CACHED, cache=(A, A, A, A, 8, 2, 48, 64)), 2),
    (dict(Np=(1 << 29) + 1), 2), (dict(H=1 << 24, Hk=1, Nq=1 << 20, qst=(1 << 38, 1 << 34, 64), ost=(1 << 38, 1 << 34, 64)), 2),
    (dict(q=A + 8), 3), (dict(pk=A + 2), 3), (dict(v=A + 4), 3), (dict(o=A + 8), 3), (dict(kv_len=A + 2), 3),
    (dict(ws=A + 16, ws_bytes=1 << 20), 3), (dict(shards=(A, A + 8)), 3), (dict(qst=(2048, 516, 64)), 3),
    (dict(pst=(2564, 64)), 3), (dict(kst=(3084, 1536, 64)), 3), (dict(ost=(2048, 512, 68)), 3),
    (dict(CACHED, cache=(A + 8, A, A, A, 8, 2, 64, 64)), 3), (dict(CACHED, pages=A + 2), 3),
    (dict(B=0), 0), (dict(H=0), 0), (dict(Nq=0), 0), (dict(Nq=0, Np=0, Nk=0, pk=None, pv=None, k=None, v=None), 0),
])
def test_refusals(xs, kw, code):
    assert _call(xs, **kw) == code


def test_null_shard_array(xs):
    assert xs.library().xs_prefix_attn_fused(A, None, 2, None, 0, None) == xs.ERR_INVALID


def test_workspace_refusals(xs):
    n = ctypes.c_ulonglong(7)
    call = lambda *a: xs.library().xs_prefix_workspace_bytes(*a, ctypes.byref(n))   # noqa: E731
    assert xs.library().xs_prefix_workspace_bytes(1, 2, 2, 1, 8, 8, 64, 0, None) == xs.ERR_INVALID
    assert call(-1, 2, 2, 1, 8, 8, 64, 0) == xs.ERR_INVALID
    assert call(1, 3, 2, 1, 8, 8, 64, 0) == xs.ERR_INVALID
    assert call(1, 2, 2, 1, 8, 8, 64, 4) == xs.ERR_INVALID
    assert call(1, 2, 2, 1, 8, 8, 256, 0) == xs.ERR_UNSUPPORTED
    assert call(0, 2, 2, 1, 8, 8, 64, 3) == xs.OK and n.value == 0


def test_binding_refuses(xs):
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        xs.prefix_attn(x, x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        xs.prefix_attn_fused(x, [x])
