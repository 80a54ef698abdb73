"""cache_write and cache_read against the definition in 64 bits on the CPU. Everything but the rounding of
fp16 outputs is exact, so codes, scale bytes and values have to be equal."""
import math

import pytest
import torch

from cache_ref import to_codes, values

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def xs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    from all_layout_gb300 import xs as _xs
    torch.cuda.set_device(0)
    return _xs


def rows(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * torch.exp(3 * torch.randn(shape[:-1] + (1,), generator=g))).to(dtype)


def lists(B, each, seed, spare=3):
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(B * each + spare, generator=g)[:B * each].view(B, each).to(torch.int32), B * each + spare


def place(pages, page, b, pos):
    """(page, row) of a place of request b; None where no page holds it."""
    if pos < 0 or pos // page >= pages.shape[-1]:
        return None
    return int(pages[b, pos // page]), pos % page


def bits(t):
    return t.cpu().view(torch.uint8)


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("B,H,N,d,page,start,lens", [
    (1, 1, 1, 16, 16, [0], None),
    (8, 8, 1, 128, 64, [5, 63, 64, 65, 0, 127, 1, 100], None),
    (3, 5, 237, 80, 32, [77, 0, 31], [237, 0, 101]),
    (2, 3, 130, 64, 128, [1, 120], [400, -7]),
    (2, 2, 77, 256, 16, [3, 0], None),
    (1, 24, 300, 96, 1024, [900], [299]),
])
def test_write(xs, dtype, B, H, N, d, page, start, lens):
    x = rows((B, N, 2 * H, d), dtype, 1)
    pages, n_pages = lists(B, -(-(max(start) + N) // page), 2)
    cache = xs.alloc_cache(n_pages, H, page, d)
    for t in cache:
        t.view(torch.uint8).fill_(0x55)
    want = [bits(t).clone() for t in cache]
    xd = x.cuda().transpose(1, 2)
    xs.cache_write(xd[:, :H], xd[:, H:], cache, pages.cuda(), start=torch.tensor(start, dtype=torch.int32).cuda(),
                   lens=None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda())
    for i in range(2):
        code, byte = to_codes(x[:, :, i * H:(i + 1) * H])
        for b in range(B):
            for n in range(N if lens is None else min(max(lens[b], 0), N)):
                pg, r = place(pages, page, b, start[b] + n)
                want[i][pg, :, r], want[2 + i][pg, :, r] = code[b, n], byte[b, n]
    for got, ref, name in zip(cache, want, cache._fields):
        assert torch.equal(bits(got), ref), name


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("B,H,N,d,page,lens", [
    (1, 1, 1, 16, 16, None), (8, 8, 1, 128, 64, None), (3, 5, 237, 80, 32, [237, 0, 101]),
    (2, 3, 130, 64, 128, [1000, -1]), (2, 2, 77, 256, 16, None)])
def test_read(xs, dtype, B, H, N, d, page, lens):
    g = torch.Generator().manual_seed(3)
    start = [7 * b for b in range(B)]
    pages, n_pages = lists(B, -(-(max(start) + N) // page), 4)
    codes = [torch.randint(0, 256, (n_pages, H, page, d), generator=g, dtype=torch.uint8) for _ in range(2)]
    scale = [torch.randint(120, 135, (n_pages, H, page), generator=g, dtype=torch.uint8) for _ in range(2)]
    cache = xs.KVCache(*(t.cuda().view(torch.float8_e4m3fn) for t in codes), *(t.cuda() for t in scale))
    out = [torch.full((B, N, H, d), 7.0, dtype=dtype, device="cuda").transpose(1, 2) for _ in range(2)]
    xs.cache_read(cache, pages.cuda(), *out, start=torch.tensor(start, dtype=torch.int32).cuda(),
                  lens=None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda())
    for i in range(2):
        want = torch.full((B, H, N, d), 7.0, dtype=torch.float64)
        for b in range(B):
            for n in range(N if lens is None else min(max(lens[b], 0), N)):
                pg, r = place(pages, page, b, start[b] + n)
                want[b, :, n] = values(codes[i][pg, :, r], scale[i][pg, :, r])
        assert torch.equal(out[i].cpu().double().nan_to_num(12345.0), want.to(dtype).double().nan_to_num(12345.0))


def test_rows_that_are_not_ordinary(xs):
    """Zeros, the border 448 * 2^e, the smallest and largest magnitudes, ties, infinities and NaN."""
    inf, nan, big = math.inf, math.nan, torch.finfo(FP).max
    r = torch.zeros(16, 16)
    r[1, 0], r[2, 0] = 448.0, torch.nextafter(torch.tensor(448.0), torch.tensor(1e9))
    r[3, :4] = torch.tensor([1.0, 1 / 16 + 1, 3 / 16 + 1, -1 / 16 - 1])
    r[4, 0], r[5, 0], r[6, 0] = 2.0 ** -149, 2.0 ** -126, big
    r[7, :3] = torch.tensor([1.0, inf, 2.0])
    r[8, :3] = torch.tensor([nan, 1.0, 2.0])
    r[9, :2] = torch.tensor([-0.0, -2.0 ** -30])
    r[10, :3] = torch.tensor([448.0, 2.0 ** -9, 2.0 ** -10])
    r[11, :3] = torch.tensor([448.0, 3 * 2.0 ** -10, -(2.0 ** -11)])
    r[12, 0] = 448 * 2.0 ** 119
    r[13, 0] = 448 * 2.0 ** -120
    r[14] = torch.tensor([464.0, 432.0, 416.0, 400.0] * 4)
    r[15, 15] = -inf
    x = r.view(1, 1, 16, 16)
    cache = xs.alloc_cache(1, 1, 16, 16)
    pages = torch.zeros(1, dtype=torch.int32, device="cuda")
    xs.cache_write(x.cuda(), x.neg().cuda(), cache, pages)
    for i, y in enumerate((x, -x)):
        code, byte = to_codes(y[0, 0])
        assert torch.equal(bits(cache[i])[0, 0], code) and torch.equal(bits(cache[2 + i])[0, 0], byte)
        back = [torch.empty(1, 1, 16, 16, device="cuda") for _ in range(2)]
        xs.cache_read(cache, pages, *back)
        want = values(code, byte).float()
        assert torch.equal(back[i].cpu()[0, 0].nan_to_num(9.0), want.nan_to_num(9.0))
        assert back[i].cpu()[0, 0][[7, 8, 15]].isnan().all()


def test_places_without_a_page(xs):
    """Nothing is stored there, and they read as NaN: negative places, past the list, page numbers out of range."""
    B, H, N, d, page = 3, 2, 40, 64, 16
    pages = torch.tensor([[0, 1], [2, -1], [99, 3]], dtype=torch.int32)
    start = torch.tensor([-5, 0, 0], dtype=torch.int32)
    cache = xs.alloc_cache(4, H, page, d)
    x = rows((B, H, N, d), BF, 5)
    xs.cache_write(x.cuda(), x.cuda(), cache, pages.cuda(), start=start.cuda())
    k, v = (torch.zeros(B, H, N, d, device="cuda") for _ in range(2))
    xs.cache_read(cache, pages.cuda(), k, v, start=start.cuda())
    for b in range(B):
        for n in range(N):
            at = place(pages, page, b, int(start[b]) + n)
            got = k[b, :, n].cpu()
            if at is None or not 0 <= at[0] < 4:
                assert got.isnan().all(), (b, n)
            else:
                assert torch.equal(got.double(), values(*to_codes(x[b, :, n]))), (b, n)
    assert torch.equal(k.nan_to_num(1.0), v.nan_to_num(1.0))


def test_other_stream_and_graph(xs):
    B, H, N, d, page = 2, 3, 50, 128, 32
    pages, n = lists(B, 2, 6)
    pages, x = pages.cuda(), rows((B, H, N, d), BF, 7).cuda()
    a, b = xs.alloc_cache(n, H, page, d), xs.alloc_cache(n, H, page, d)
    out = [torch.zeros_like(x) for _ in range(4)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        xs.cache_write(x, x, a, pages)
        xs.cache_read(a, pages, out[0], out[1])
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        xs.cache_write(x, x, b, pages)
        xs.cache_read(b, pages, out[2], out[3])
    x.neg_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], out[1]) and torch.equal(out[2], out[3]) and torch.equal(out[2], -out[0])


def test_offsets_past_32_bits(xs):
    """A cache of 2^32 codes and more: the last page's rows land there."""
    H, page, d = 8, 1024, 256
    n = (1 << 32) // (H * page * d) + 2
    cache = xs.alloc_cache(n, H, page, d)
    x = rows((1, H, 100, d), BF, 8)
    pages = torch.tensor([n - 1], dtype=torch.int32, device="cuda")
    xs.cache_write(x.cuda(), (-x).cuda(), cache, pages)
    code, byte = to_codes(x[0])
    assert torch.equal(bits(cache.k[n - 1, :, :100]), code) and torch.equal(bits(cache.k_scale[n - 1, :, :100]), byte)
    k, v = torch.empty(1, H, 100, d, device="cuda"), torch.empty(1, H, 100, d, device="cuda")
    xs.cache_read(cache, pages, k, v)
    assert torch.equal(k[0].cpu().double(), values(code, byte)) and torch.equal(k, -v)
    assert not bits(cache.k[:n - 1:97]).any()
