"""xs_cache_write, xs_cache_read and their bindings without a GPU: refusals before any device work, the layout of
the structs, and the plain form's codes against torch's own conversion."""
import ctypes

import pytest
import torch

from cache_ref import to_codes, values

A = 0x10000   # a 16-byte aligned fake device address; never dereferenced


@pytest.fixture(scope="module")
def xs():
    import __graft_entry__
    __graft_entry__.build()
    from all_layout_gb300 import xs as _xs
    return _xs


def _call(xs, write=True, k=A, v=2 * A, cache=(A, A, A, A), n_pages=4, H=2, page=64, d=64, kst=None, vst=None, pages=A,
          stride=4, count=4, start=None, lens=None, B=2, N=8, type=0, no=()):
    c = xs._CACHE.pack(*(x or 0 for x in cache), n_pages, H, page, d)
    lists = xs._PAGES.pack(pages or 0, stride, count)
    ks = xs._STRIDES.pack(*(kst or (H * N * d, N * d, d)))
    vs = xs._STRIDES.pack(*(vst or (H * N * d, N * d, d)))
    call = xs.library().xs_cache_write if write else xs.library().xs_cache_read
    return call(None if "cache" in no else c, k, v, None if "kst" in no else ks, None if "vst" in no else vs,
                None if "lists" in no else lists, start, lens, B, N, type, None)


@pytest.mark.parametrize("write", [True, False])
@pytest.mark.parametrize("kw,code", [
    (dict(no=("cache",)), 1), (dict(no=("lists",)), 1), (dict(no=("kst",)), 1), (dict(no=("vst",)), 1),
    (dict(k=None), 1), (dict(v=None), 1), (dict(pages=None), 1), (dict(cache=(None, A, A, A)), 1),
    (dict(cache=(A, A, A, None)), 1), (dict(B=-1), 1), (dict(N=-1), 1), (dict(H=-1), 1), (dict(n_pages=-1), 1),
    (dict(page=0), 1), (dict(page=-16), 1), (dict(count=-1), 1), (dict(stride=-4), 1), (dict(type=3), 1),
    (dict(type=-1), 1), (dict(kst=(-1024, 512, 64)), 1), (dict(d=-16), 1),
    (dict(d=72), 2), (dict(d=8), 2), (dict(d=272), 2), (dict(page=48), 2), (dict(page=8), 2), (dict(page=2048), 2),
    (dict(N=1 << 30, H=2, kst=(1 << 40, 1 << 37, 64), vst=(1 << 40, 1 << 37, 64)), 2),
    (dict(k=A + 8), 3), (dict(v=A + 2), 3), (dict(cache=(A + 8, A, A, A)), 3), (dict(cache=(A, A, A + 4, A)), 3),
    (dict(start=A + 2), 3), (dict(lens=A + 1), 3), (dict(pages=A + 2), 3), (dict(vst=(1024, 512, 68)), 3),
    (dict(type=2, kst=(1024, 512, 66)), 3),
    (dict(B=0), 0), (dict(N=0), 0), (dict(H=0, d=64), 0),
])
def test_refusals(xs, write, kw, code):
    assert _call(xs, write, **kw) == code


def test_outputs_that_overlap(xs):
    """A read's rows must not overlap; a write may read one row often."""
    assert _call(xs, False, kst=(1024, 0, 64)) == 1
    assert _call(xs, False, vst=(1024, 512, 32)) == 1
    assert _call(xs, True, N=0, kst=(0, 0, 0)) == 0


def test_struct_sizes(xs, tmp_path):
    import subprocess
    src = tmp_path / "s.cpp"
    src.write_text('#include "include/xs.h"\n#include <cstdio>\nint main() { printf("%zu %zu %zu", sizeof(xs_cache), '
                   'sizeof(xs_pages), sizeof(xs_prefix_args)); }\n')
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run(["g++", "-I", root, str(src), "-o", str(tmp_path / "s")], check=True)
    got = subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout
    assert got == f"{xs._CACHE.size} {xs._PAGES.size} {xs._PREFIX_ARGS.size}"


def test_bindings_refuse(xs):
    x = torch.zeros(1, 2, 4, 64)
    for call in (lambda: xs.cache_write(x, x, None, None), lambda: xs.cache_read(None, None, x, x)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_plain_form_against_torch():
    """The reference's codes are torch's e4m3 of the scaled rows, and its values those of torch's codes."""
    x = torch.randn(500, 64, generator=torch.Generator().manual_seed(1)) * torch.exp(4 * torch.randn(500, 1, generator=torch.Generator().manual_seed(2)))
    code, byte = to_codes(x)
    scaled = (x.double() * torch.pow(2.0, 127 - byte.double())[:, None]).float()
    assert torch.equal(code, scaled.to(torch.float8_e4m3fn).view(torch.uint8))
    assert torch.equal(values(code, byte), code.view(torch.float8_e4m3fn).double() * torch.pow(2.0, byte.double() - 127)[:, None])
    top = scaled.abs().amax(-1)
    assert (top <= 448).all() and (top > 224).all()


def test_rows_of_a_thread(tmp_path):
    """The second row of a thread, where heads have few tokens and where tokens number nearly 2^31: one head's last rows
    lead past the end, never to a token in front of the first."""
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "t.cpp"
    src.write_text(r"""
#include "all_layout_gb300/csrc/cache.h"
#include <initializer_list>
#include <cstdio>
int main() {
  const long long sizes[][2] = {{1, 1}, {24, 1}, {7, 3}, {3, 255}, {5, 257}, {1, 0x7fffffff}, {1, 0x7fffffff - 255}, {1, 0x7fffff00},
                                {2, 0x3fffffff}, {0x7fffffff, 1}, {46341, 46340}, {1, 1 << 30}};
  long long bad = 0;
  for (const auto &s : sizes)
    for (unsigned by = 16; by <= 256; by *= 2) {
      const long long H = s[0], N = s[1], rows = H * N;
      for (long long k = 0; k < 4096; ++k)
        for (const long long row : {k, rows / 2 + k, rows - k}) {
          if (row < 0 || row > rows) continue;
          xs::TokenAt t = xs::token_at(static_cast<unsigned>(row), static_cast<unsigned>(N));
          for (int u = 0; u < 2; ++u) {
            const long long want = row + u * by;
            bad += want < rows ? t.h != want / N || t.n != want % N : t.h < H;
            xs::step_token(t, by, static_cast<unsigned>(N), static_cast<int>(H));
          }
        }
    }
  std::printf("%lld", bad);
}
""")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", root, str(src), "-o", str(tmp_path / "t")], check=True)
    assert subprocess.run([str(tmp_path / "t")], capture_output=True, text=True, check=True).stdout == "0"
