"""xs_rope and qkv_rope without a GPU: refusals of the C entry point (before any device work) and
of the binding, and the 64-bit turn arithmetic that the kernel uses, against exact rationals."""
import ctypes
import math
import os
import random
import subprocess
from fractions import Fraction

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x10000   # a 16-byte aligned fake device address; never dereferenced


@pytest.fixture(scope="module")
def xs():
    import __graft_entry__
    __graft_entry__.build()
    from all_layout_gb300 import xs as _xs
    return _xs


def _call(xs, x=A, y=2 * A, w=None, xst=None, yst=None, heads=4, n=1, pos=A, pos_b=0, axes=(16, 24, 24),
          n_axes=None, freqs="default", B=2, N=8, d=64, eps=1e-6, flags=1, it=0, ot=0, tensors=True):
    one = xs._ROPE_TENSOR.pack(x or 0, y or 0, w or 0, *(xst or (N * 4 * 64, 4 * 64, 64)),
                               *(yst or (N * 4 * 64, 64, N * 64)), heads, 1)
    arr = one * 3
    dims = (ctypes.c_int * max(1, len(axes)))(*axes)
    f = [0.5] * 128 if freqs == "default" else freqs
    table = None if f is None else (ctypes.c_double * len(f))(*f)
    return xs.library().xs_rope(arr if tensors else None, n, pos, pos_b, dims, len(axes) if n_axes is None else n_axes,
                                table, B, N, d, eps, flags, it, ot, None)


@pytest.mark.parametrize("kw,code", [
    (dict(tensors=False), 1), (dict(x=None), 1), (dict(y=None), 1), (dict(pos=None), 1), (dict(freqs=None), 1),
    (dict(n=0), 1), (dict(n=4), 1), (dict(B=-1), 1), (dict(N=-1), 1), (dict(d=-8), 1), (dict(heads=-1), 1),
    (dict(axes=(16, 24, 23)), 1), (dict(axes=(16, 24, 26)), 1), (dict(axes=(0, 16)), 1), (dict(axes=(-16, 16)), 1),
    (dict(n_axes=0), 1), (dict(axes=(2,) * 5), 1), (dict(eps=-1.0), 1), (dict(eps=math.nan), 1), (dict(eps=math.inf), 1),
    (dict(flags=2), 1), (dict(it=3), 1), (dict(ot=-1), 1), (dict(pos_b=-3), 1), (dict(freqs=[math.inf] * 128), 1),
    (dict(xst=(-64, 256, 64)), 1), (dict(yst=(2048, 32, 512)), 1), (dict(yst=(2048, 0, 512)), 1),
    (dict(y=A), 1),                                                  # in place with other strides
    (dict(y=A, yst=(2048, 256, 64), it=1, ot=0), 1),                 # in place with another type
    (dict(d=60, axes=(16,)), 2), (dict(d=264, axes=(16,), yst=(8448, 264, 2112)), 2), (dict(d=4, axes=(2,)), 2),
    (dict(flags=0, axes=(16, 26)), 2),                               # 42 columns in halves of 21
    (dict(it=0, ot=1), 2), (dict(it=0, ot=2), 2), (dict(it=1, ot=2), 2),
    (dict(B=1 << 16, N=1 << 16), 2), (dict(heads=40000, n=3), 2),
    (dict(x=A + 8), 3), (dict(y=2 * A + 2), 3), (dict(w=A + 4), 3), (dict(pos=A + 2), 3),
    (dict(xst=(2048, 260, 64)), 3), (dict(yst=(2048, 68, 512)), 3), (dict(it=2, ot=2, xst=(2048, 258, 64)), 3),
    (dict(B=0), 0), (dict(N=0), 0), (dict(heads=0), 0),
])
def test_refusals(xs, kw, code):
    assert _call(xs, **kw) == code


def test_strides_of_single_rows_do_not_matter(xs):
    """B = N = 0 after the checks of strides: extents of one may carry any stride."""
    assert _call(xs, B=1, N=0, xst=(3, 260, 64), yst=(1, 64, 512)) == 0


def test_tensors_without_heads(xs):
    assert _call(xs, heads=0, xst=(2048, 260, 64)) == 0
    assert _call(xs, heads=0, yst=(2048, 3, 512)) == 0
    assert _call(xs, heads=0, x=None, y=None) == 0


def test_binding_refuses_before_the_library(xs):
    t = torch.zeros(2, 8, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        xs.qkv_rope(t, None, None, t.transpose(1, 2), None, None, torch.zeros(8, 3, dtype=torch.int32), (16, 24, 24))
    with pytest.raises(ValueError, match="CUDA"):
        xs.qkv_rope(None, None, None, None, None, None, None, (16,))


def test_default_frequencies(xs):
    dims, table, n_axes = xs._rope_axes((4, 6), 10000.0, None)
    assert list(dims) == [4, 6] and n_axes == 2
    want = [1.0, 1e4 ** -0.5, 1.0, 1e4 ** (-1 / 3), 1e4 ** (-2 / 3)]
    assert list(table) == pytest.approx(want, rel=1e-15)


@pytest.mark.parametrize("freq", [1.0, 1e4 ** -0.25, 1e4 ** (-62 / 64), 7.5, -0.3])
@pytest.mark.parametrize("pos", [0, 1, -1, 4095, 1 << 20, (1 << 31) - 1, -(1 << 31)])
def test_turn_arithmetic(freq, pos):
    """pos * f modulo a turn as the wrapping product of pos and a 64-bit fraction of a turn. The
    fraction is off by the division by 2 pi in 64-bit floats (2^-53 relative, and 2^-53 of the
    rounded 2 pi) and by the cut at 2^-64; over |pos| <= 2^31 steps of at most 1.2 turns that is
    below 2^31 * (1.2 * 2^-52 + 2^-53 + 2^-64) < 2^-20 of a turn, the worst case at the far end."""
    two_pi = Fraction(math.pi) * 2 + Fraction(2.4492935982947064e-16)     # pi to 107 bits: math.pi + its error
    turns = freq / 6.283185307179586476925
    turns -= math.floor(turns)
    fixed = int(turns * 2.0 ** 64) if turns < 1 else 0
    got = Fraction((pos * fixed) % (1 << 64), 1 << 64)
    want = Fraction(freq) * pos / two_pi
    diff = (got - want) % 1
    diff = min(diff, 1 - diff)
    assert diff < Fraction(max(1, abs(pos)), 1 << 31) * Fraction(1, 1 << 20) + Fraction(1, 1 << 60)


def two_pi():
    """2 pi to 400 bits and more, from Machin's pi / 4 = 4 arctan(1/5) - arctan(1/239)."""
    one = 1 << 440

    def arctan_inverse(n):
        term, total, k = one // n, 0, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= n * n
            k += 2
        return total
    return Fraction(8 * (4 * arctan_inverse(5) - arctan_inverse(239)), one)


@pytest.fixture(scope="module")
def turns(tmp_path_factory):
    """turns_per_step of the library's header, built as host code."""
    folder = tmp_path_factory.mktemp("turns")
    (folder / "t.cpp").write_text(f'#include "{ROOT}/all_layout_gb300/csrc/turns.h"\n'
                                  'extern "C" unsigned long long f(double x) { return xs::turns_per_step(x); }\n'
                                  'extern "C" int fits(double x) { return xs::turns_fit(x); }\n')
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-o", folder / "t.so", folder / "t.cpp"], check=True)
    lib = ctypes.CDLL(str(folder / "t.so"))
    lib.f.restype, lib.f.argtypes = ctypes.c_ulonglong, [ctypes.c_double]
    lib.fits.argtypes = [ctypes.c_double]
    return lib


def test_fraction_of_a_turn(turns):
    """The 64-bit fraction of every frequency below 2^64 is the exact one, rounded to nearest (half a unit,
    and 2^-60 of one for the 192 bits of 1 / (2 pi)): 2^-34 of a turn over 2^31 steps."""
    rng, whole = random.Random(5), two_pi()
    freqs = [1.0, 0.3, 7.25, 100.0, 1e4, 1e6, 2.0 ** 52, 2.0 ** 63, math.nextafter(2.0 ** 64, 0), 0.0, 5e-324, 2.0 ** -61, 2.0 ** -62,
             2.0 ** -63, 2.0 ** -64, math.tau, 2 * math.tau, math.nextafter(math.tau, 7), 1e4 ** -0.25, 1e4 ** (-62 / 64)]
    freqs += [rng.uniform(1, 2) * 2.0 ** rng.randint(-80, 63) for _ in range(3000)]
    for f in freqs + [-f for f in freqs]:
        want = Fraction(f) / whole * (1 << 64)
        diff = (turns.f(f) - want) % (1 << 64)
        assert min(diff, (1 << 64) - diff) <= Fraction(1, 2) + Fraction(1, 1 << 60), f


def test_frequencies_out_of_range(turns, xs):
    for f in (2.0 ** 64, -2.0 ** 64, 1e300):
        assert not turns.fits(f)
        assert _call(xs, freqs=[f] * 128) == xs.ERR_UNSUPPORTED
    assert turns.fits(math.nextafter(2.0 ** 64, 0)) and turns.fits(0.0) and turns.fits(-1.0)
    assert _call(xs, B=0, freqs=[math.nextafter(2.0 ** 64, 0)] * 128) == xs.OK
