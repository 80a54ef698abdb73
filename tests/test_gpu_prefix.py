"""prefix_attn and prefix_attn_fused against the formula in 64 bits.

Tolerance of an element, from the arithmetic: the output's rounding, at most 2^-8 of the value; the
weights' rounding to bf16, at most 2^-8 of each, so 2^-8 of the weights' mean of |v|; and the fp32 work
before it (scores of up to 128 products, their scaling, 2^x to 2 ulp, sums over the keys in the order of
the tiles, the pieces' factors), all relative to the same mean and under 2^-11 for scores below 2^9."""
import math

import pytest
import torch

from cache_ref import prefix_formula, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def xs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    from all_layout_gb300 import xs as _xs
    torch.cuda.set_device(0)
    return _xs


def check(got, want, what=""):
    ref, size = want
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -11) * size + 2.0 ** -133
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / tol).max()):.2f} of the tolerance"


class Problem:
    """Operands of one call. kinds: 'bf16' or 'cache' for the prefix's and the own keys."""

    def __init__(self, xs, B, H, Hk, d, Nq, Np, Nk, lens=None, prefix="bf16", own="bf16", page=32, seed=0, scale=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *s: torch.randn(s, generator=g, device="cuda")   # noqa: E731
        self.xs, self.shape, self.scale = xs, (B, H, Hk, d, Nq, Np, Nk), scale
        self.q = (2 * normal(B, H, Nq, d)).bfloat16()
        self.lens = [Nk] * B if lens is None else [min(max(n, 0), Nk) for n in lens]
        self.kw = {"scale": scale}
        if lens is not None:
            self.kw["kv_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        n_prefix = -(-Np // page) if prefix == "cache" else 0
        n_own = -(-Nk // page) if own == "cache" else 0
        total = n_prefix + B * n_own + 2
        order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        codes = [torch.randint(0, 256, (total, Hk, page, d), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
        for c in codes:   # ordinary values: exponents 4 to 10, no NaN
            c.copy_((c & 0x87) | ((c >> 3 & 15) % 7 + 4) << 3)
        scales = [torch.randint(121, 128, (total, Hk, page), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
        self.codes, self.scales = codes, scales
        if "cache" in (prefix, own):
            self.kw["cache"] = xs.KVCache(*(c.view(torch.float8_e4m3fn) for c in codes), *scales)
        every = [values(codes[i], scales[i]) for i in range(2)]                    # [total, Hk, page, d]
        flat = lambda i, p, n: every[i][p.long()].transpose(0, 1).flatten(1, 2)[:, :n]   # noqa: E731
        if prefix == "cache":
            self.kw.update(prefix_pages=order[:n_prefix].contiguous(), prefix_len=Np)
            self.prefix = [flat(i, order[:n_prefix], Np) if Np else normal(Hk, 0, d).double() for i in range(2)]
        else:
            t = [normal(Hk, Np, d).bfloat16() for _ in range(2)]
            self.kw.update(prefix_k=t[0], prefix_v=t[1])
            self.prefix = [x.double() for x in t]
        if own == "cache":
            pages = order[n_prefix:n_prefix + B * n_own].view(B, n_own).contiguous()
            self.kw.update(pages=pages, max_len=Nk)
            self.own = [torch.stack([flat(i, pages[b], Nk) if Nk else normal(Hk, 0, d).double() for b in range(B)]) for i in range(2)]
        else:
            t = [normal(B, Hk, Nk, d).bfloat16() for _ in range(2)]
            self.kw.update(k=t[0], v=t[1])
            self.own = [x.double() for x in t]

    def workspace(self):
        B, H, Hk, d, Nq, Np, Nk = self.shape
        ws = self.xs.alloc_prefix_workspace(B, H, Hk, Nq, Np, Nk, d, prefix_cached="prefix_pages" in self.kw, own_cached="pages" in self.kw)
        return ws.fill_(0xff)   # any content will do

    def want(self):
        return prefix_formula(self.q.double(), self.prefix, self.own, self.lens, self.shape[3] ** -0.5 if self.scale is None else self.scale)

    def run(self, workspace=None, P=0):
        B, H, _, d, Nq, _, _ = self.shape
        if P:
            out = self.xs.alloc_shards(B, Nq, H, d, P)
            for t in out:
                t.fill_(math.nan)
            self.xs.prefix_attn_fused(self.q, out, workspace=workspace, **self.kw)
            return torch.cat(out, 1).transpose(1, 2)
        out = torch.full((B, H, Nq, d), math.nan, dtype=torch.bfloat16, device="cuda")
        self.xs.prefix_attn(self.q, out, workspace=workspace, **self.kw)
        return out

    def test(self, P=0):
        want = self.want()
        check(self.run(P=P), want, "whole units")
        check(self.run(self.workspace(), P=P), want, "workspace")
        assert self.xs.last_device_status() == self.xs.OK


KINDS = [("bf16", "bf16"), ("cache", "bf16"), ("bf16", "cache"), ("cache", "cache")]


@pytest.mark.parametrize("prefix,own", KINDS)
@pytest.mark.parametrize("B,H,Hk,d,Nq,Np,Nk,lens", [
    (1, 1, 1, 128, 1, 1, 1, None),
    (1, 1, 1, 64, 1, 128, 0, None),
    (2, 2, 1, 128, 1, 0, 1, None),
    (8, 6, 2, 128, 1, 1000, 100, [100, 0, 1, 15, 16, 17, 99, 33]),        # 24 rows: four copies
    (8, 4, 1, 64, 2, 700, 130, [130, 129, 128, 127, 0, 0, 1, 64]),         # 64 rows: two copies
    (5, 3, 3, 128, 13, 257, 40, [40, 0, 39, 1, 40]),                       # 65 rows: one
    (3, 4, 2, 64, 77, 130, 300, [300, 0, 111]),                            # tiles over several requests
    (2, 2, 2, 128, 300, 0, 500, [500, 7]),
    (3, 2, 1, 128, 129, 300, 0, None),
    (40, 2, 2, 128, 1, 200, 60, [(7 * b) % 61 for b in range(40)]),
    # Many rows: pairs of tiles, over several requests and heads, with requests between that have no keys.
    (2, 4, 2, 128, 640, 700, 900, [900, 333]),
    (3, 2, 1, 64, 500, 1000, 300, [1, 0, 300]),
    (7, 4, 2, 128, 100, 300, 200, [200, 0, 0, 128, 129, 0, 1]),
    (4, 3, 3, 64, 257, 0, 513, [0, 513, 512, 0]),
    (2, 8, 1, 128, 321, 129, 0, None),
])
def test_formula(xs, prefix, own, B, H, Hk, d, Nq, Np, Nk, lens):
    Problem(xs, B, H, Hk, d, Nq, Np, Nk, lens, prefix, own, seed=B + Nq).test()


@pytest.mark.parametrize("page", [16, 64, 128, 256, 1024])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq", [1, 40])
def test_pages(xs, page, d, Nq):
    """Pages smaller and larger than a tile, ends inside a tile."""
    Problem(xs, 3, 4, 2, d, Nq, 1500, 333, [333, 16, 0], "cache", "cache", page=page, seed=page).test()


@pytest.mark.parametrize("P", [1, 2, 5, 8])
@pytest.mark.parametrize("Nq", [40, 400])
def test_shards(xs, P, Nq):
    Problem(xs, 3, 4, 2, 128, Nq, 300, 100, [100, 0, 57], "cache", "bf16").test(P=P)


def test_many_requests(xs):
    """More requests than one launch takes, own keys in tensors and in pages."""
    lens = [(5 * b) % 23 for b in range(600)]
    for own in ("bf16", "cache"):
        Problem(xs, 600, 2, 1, 64, 1, 100, 22, lens, "cache", own, page=16).test()


@pytest.mark.parametrize("Nq", [1, 200])
@pytest.mark.parametrize("own", ["bf16", "cache"])
def test_what_lies_behind_the_lengths(xs, Nq, own):
    """NaN and infinities behind a request's last key, in the pages' unused rows too, change nothing."""
    B, H, Hk, d, Np, Nk, page = 3, 4, 2, 128, 200, 150, 64
    p = Problem(xs, B, H, Hk, d, Nq, Np, Nk, [150, 37, 0], "cache", own, page=page, seed=3)
    before = p.run(p.workspace()).clone(), p.run().clone()
    if own == "bf16":
        for b, n in enumerate(p.lens):
            p.kw["k"][b, :, n:] = math.nan
            p.kw["v"][b, :, n:] = math.inf
    used = torch.zeros(p.codes[0].shape[0], page, dtype=torch.bool, device="cuda")
    for i, pg in enumerate(p.kw["prefix_pages"].tolist()):
        used[pg, :max(0, min(page, Np - i * page))] = True
    if own == "cache":
        for b, n in enumerate(p.lens):
            for i, pg in enumerate(p.kw["pages"][b].tolist()):
                used[pg, :max(0, min(page, n - i * page))] = True
    for codes, scales in zip(p.codes, p.scales):
        codes.masked_fill_(~used[:, None, :, None], 0x7f)
        scales.masked_fill_(~used[:, None], 255)
    assert torch.equal(p.run(p.workspace()), before[0]) and torch.equal(p.run(), before[1])
    check(before[0], p.want())


def test_keys_without_a_page(xs):
    """They count as NaN: rows that see one are NaN, the others are as ever; nothing else is read."""
    for Nq in (1, 150):
        p = Problem(xs, 3, 4, 2, 64, Nq, 128, 100, [100, 40, 0], "cache", "cache", page=32, seed=4)
        want = p.want()
        p.kw["pages"][0, 3] = 10 ** 6
        p.kw["pages"][1, 2:] = -5          # behind the second request's last key
        for ws in (None, p.workspace()):
            got = p.run(ws)
            assert got[0].isnan().all()
            check(got[1:], (want[0][1:], want[1][1:]))
        p.kw["prefix_pages"][0] = -1
        assert p.run(p.workspace()).isnan().all()


@pytest.mark.parametrize("Nq", [1, 20, 200])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_requests_do_not_touch_each_other(xs, Nq, value):
    """A value or key of one request that is not a number changes that request's rows alone (of the k/v head)."""
    p = Problem(xs, 4, 4, 2, 128, Nq, 100, 60, [60, 3, 60, 17], "bf16", "bf16", seed=17)
    ws = p.workspace()
    before = p.run(ws).clone(), p.run().clone()
    for name in ("v", "k"):
        keep = p.kw[name].clone()
        p.kw[name][2, 0, 5, 7] = value
        for got, ref in zip((p.run(ws), p.run()), before):
            assert not torch.isfinite(got[2, :2, :, 7]).any() if name == "v" else got[2, :2].isnan().any()
            assert torch.equal(got[[0, 1, 3]], ref[[0, 1, 3]]) and torch.equal(got[2, 2:], ref[2, 2:])
        p.kw[name].copy_(keep)


@pytest.mark.parametrize("Nq", [1, 33, 300])
def test_scales_over_their_range(xs, Nq):
    """Rows of keys and values of very different magnitudes, in a cache and out of it: scales from 2^-60 to 2^40."""
    p = Problem(xs, 2, 2, 1, 128, Nq, 260, 140, None, "cache", "bf16", page=16, seed=5, scale=0.01)
    g = torch.Generator(device="cuda").manual_seed(6)
    for i, t in enumerate(p.scales):
        t.copy_(torch.randint(67, 168 if i else 128, t.shape, generator=g, device="cuda", dtype=torch.uint8))
    p.q.mul_(torch.exp(3 * torch.randn(p.q.shape[:3] + (1,), generator=g, device="cuda")).bfloat16())
    every = [values(p.codes[i], p.scales[i]) for i in range(2)]
    n = p.kw["prefix_pages"].long()
    p.prefix = [every[i][n].transpose(0, 1).flatten(1, 2)[:, :260] for i in range(2)]
    p.test()


def test_queries_over_their_range(xs):
    """Rows of queries from 2^-100 to 2^60, columns that stand out by 2^20, zeros: each row meets cached keys times a power of two."""
    p = Problem(xs, 1, 1, 1, 64, 64, 300, 0, None, "cache", "bf16", page=16, seed=7)
    e = torch.linspace(-100, 20, 64, device="cuda").round()
    p.q.copy_((p.q.float() * torch.exp2(e)[None, None, :, None]).bfloat16())
    p.q[0, 0, 40, 3] *= 2.0 ** 20
    p.codes[0][..., 3] = 0             # (K has nothing there)
    p.q[0, 0, 50] = 0
    p.kw["scale"] = p.scale = 2.0 ** -6
    small = (e[:, None] < 12).expand(64, 64)
    every = [values(p.codes[i], p.scales[i]) for i in range(2)]
    n = p.kw["prefix_pages"].long()
    p.prefix = [every[i][n].transpose(0, 1).flatten(1, 2)[:, :300] for i in range(2)]
    want = p.want()
    for ws in (None, p.workspace()):
        got = p.run(ws)
        check(got[0, 0][small[:, 0]], (want[0][0, 0][small[:, 0]], want[1][0, 0][small[:, 0]]))
        assert torch.isfinite(got).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq", [1, 100])
def test_queries_with_a_column_that_stands_out(xs, d, Nq):
    """A column 2^12 times the others that the keys have nothing in: the parts of a query that meet cached keys still
    hold the others in full (to 2^-13 of a row's largest)."""
    p = Problem(xs, 1, 1, 1, d, Nq, 300, 0, None, "cache", "bf16", page=128, seed=11, scale=d ** -0.5)
    p.q.copy_((torch.rand_like(p.q, dtype=torch.float32) + 1).bfloat16() * torch.randn_like(p.q).sign())
    p.q[p.q >= 2] = 1
    p.q[p.q <= -2] = -1
    p.q[..., 5] = 4096
    p.codes[0][..., 5] = 0
    p.prefix[0][..., 5] = 0
    for ws in (None, p.workspace()):
        check(p.run(ws), p.want())


@pytest.mark.parametrize("d", [64, 128])
def test_sums_of_codes(xs, d):
    """Two keys whose scores differ by 2^-24 of what cancels in them: the sums hold fp32's bits."""
    cache = xs.alloc_cache(1, 1, 16, d)
    rows = torch.zeros(2, d, device="cuda")
    rows[:, 0:d - 2:2], rows[:, 1:d - 2:2] = 448.0, -448.0
    rows[0, d - 1] = 2.0 ** -9
    cache.k[0, 0, :2] = rows.to(torch.float8_e4m3fn)
    cache.v[0, 0, :1] = torch.ones(1, d, device="cuda").to(torch.float8_e4m3fn)
    q = torch.ones(1, 1, 1, d, device="cuda", dtype=torch.bfloat16)
    o = torch.empty_like(q)
    pages = torch.zeros(1, dtype=torch.int32, device="cuda")
    xs.prefix_attn(q, o, cache=cache, prefix_pages=pages, prefix_len=2, scale=2.0 ** 9)   # scores 1 and 0
    want = 1 / (1 + math.exp(-1))
    assert (o.double() - want).abs().max() <= (2.0 ** -8 + 2.0 ** -8 + 2.0 ** -11) * want   # as in check


@pytest.mark.parametrize("kind", ["bf16", "cache"])
@pytest.mark.parametrize("Nq", [20, 300])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_queries_that_are_not_numbers(xs, kind, Nq, value):
    """A query with a NaN or an infinity: its row is NaN, the others are as without it."""
    p = Problem(xs, 2, 2, 1, 64, Nq, 200, 100, [100, 30], kind, kind, seed=12)
    p.q[1, 0, 7] = 1.0                    # (the formula's own row, put aside)
    want = p.want()
    p.q[1, 0, 7, 3] = value
    for ws in (None, p.workspace()):
        got = p.run(ws)
        assert torch.isnan(got[1, 0, 7]).all()
        rest = torch.ones(2, 2, Nq, dtype=torch.bool, device="cuda")
        rest[1, 0, 7] = False
        check(got[rest], (want[0][rest], want[1][rest]))


def test_identical_values(xs):
    """Equal rows of V come back exactly but for the output's rounding: 2^-8 and the weights' sum against their rounding."""
    p = Problem(xs, 2, 2, 2, 128, 5, 300, 100, [100, 3], "bf16", "bf16", seed=8)
    row = torch.randn(128, device="cuda").bfloat16()
    p.kw["prefix_v"][:] = row
    p.kw["v"][:] = row
    p.prefix[1][:], p.own[1][:] = row.double(), row.double()
    p.test()


def test_views(xs):
    """Token-major q and o, keys and values out of one projection, a page list out of a larger table, strides of one row."""
    B, H, Hk, d, Nq, Np, Nk = 2, 4, 2, 128, 50, 200, 90
    p = Problem(xs, B, H, Hk, d, Nq, Np, Nk, [90, 11], "bf16", "bf16", seed=9)
    want = p.want()
    x = torch.empty(B, Nk, 2 * Hk, d, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    x[:, :Hk], x[:, Hk:] = p.kw["k"], p.kw["v"]
    pk = torch.empty(Np, 2, Hk, d, dtype=torch.bfloat16, device="cuda")
    pk[:, 0], pk[:, 1] = p.kw["prefix_k"].transpose(0, 1), p.kw["prefix_v"].transpose(0, 1)
    q = torch.empty(B, Nq, H + 3, d, dtype=torch.bfloat16, device="cuda")[:, :, 1:H + 1].transpose(1, 2)
    q.copy_(p.q)
    for ws in (None, p.workspace()):
        o = torch.full((B, Nq, H, d), math.nan, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
        xs.prefix_attn(q, o, k=x[:, :Hk], v=x[:, Hk:], kv_len=p.kw["kv_len"], prefix_k=pk[:, 0].transpose(0, 1),
                       prefix_v=pk[:, 1].transpose(0, 1), workspace=ws)
        check(o, want)
    c = Problem(xs, B, H, Hk, 64, 3, 100, 90, [90, 11], "cache", "cache", page=16, seed=10)
    table = torch.full((B, 20), -1, dtype=torch.int32, device="cuda")
    table[:, 4:10] = c.kw["pages"]
    c.kw["pages"] = table[:, 4:10]
    c.test()


def test_small_workspaces(xs):
    """Less than everything: whole units, then parts, then cached keys read as they are."""
    p = Problem(xs, 2, 2, 1, 128, 300, 4000, 100, [100, 1], "cache", "cache", seed=11)
    want, ws = p.want(), p.workspace()
    for n in (0, 4096, 8192, 1 << 20, 8 << 20, ws.numel() // 2, ws.numel()):
        check(p.run(ws[:n] if n else None), want, f"{n} bytes")


def test_streams_and_graphs(xs):
    """Two captured calls that share a workspace, replayed with other inputs and among eager calls; another stream."""
    a = Problem(xs, 4, 4, 2, 128, 1, 3000, 64, [64, 0, 5, 33], "cache", "cache", seed=12)
    b = Problem(xs, 2, 4, 2, 128, 300, 500, 200, [200, 31], "cache", "bf16", seed=13)
    ws = b.workspace()
    ws = ws if ws.numel() > a.workspace().numel() else a.workspace()
    outs = [torch.zeros_like(p.q) for p in (a, b)]
    g = torch.cuda.CUDAGraph()
    a.run(ws), b.run(ws)
    with torch.cuda.graph(g):
        for p, o in zip((a, b), outs):
            xs.prefix_attn(p.q, o, workspace=ws, **p.kw)
    side = torch.cuda.Stream()
    for turn in range(3):
        a.q.neg_(), b.q.mul_(0.5)
        a.kw["kv_len"].copy_(torch.tensor([turn, 64, 7, 0], dtype=torch.int32))
        a.lens = [turn, 64, 7, 0]
        g.replay()
        eager = b.run(ws)
        check(outs[0], a.want(), "graph")
        check(outs[1], b.want(), "graph")
        assert torch.equal(eager, outs[1])
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = a.run(ws)
        side.synchronize()
        assert torch.equal(other, outs[0])


def test_same_from_launch_to_launch(xs):
    p = Problem(xs, 6, 6, 2, 128, 3, 5000, 100, [100, 0, 31, 99, 5, 64], "cache", "bf16", seed=14)
    ws = p.workspace()
    first = p.run(ws).clone()
    for _ in range(20):
        assert torch.equal(p.run(ws), first)


def test_empty(xs):
    """No request, head or query: nothing happens. No key at all: zeros."""
    for B, H, Nq in ((0, 2, 3), (2, 2, 0)):
        q = torch.zeros(B, H, Nq, 64, dtype=torch.bfloat16, device="cuda")
        xs.prefix_attn(q, torch.empty_like(q), prefix_k=q.new_zeros(2, 5, 64), prefix_v=q.new_zeros(2, 5, 64))
    for Nq in (1, 300):
        q = torch.randn(3, 2, Nq, 64, device="cuda").bfloat16()
        o = torch.full_like(q, math.nan)
        xs.prefix_attn(q, o)
        assert not o.any()
        k = torch.full((3, 2, 9, 64), math.nan, dtype=torch.bfloat16, device="cuda")
        o.fill_(math.nan)
        xs.prefix_attn(q, o, k=k, v=k, kv_len=torch.tensor([0, -3, 0], dtype=torch.int32, device="cuda"))
        assert not o.any()


def test_long_cache(xs):
    """Places past 2^32 bytes of codes: the last pages of a cache of 2^32 codes."""
    H, page, d = 8, 1024, 128
    n = (1 << 32) // (H * page * d) + 4
    cache = xs.alloc_cache(n, H, page, d)
    g = torch.Generator(device="cuda").manual_seed(15)
    k, v = (torch.randn(1, H, 2000, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    pages = torch.tensor([n - 1, n - 3], dtype=torch.int32, device="cuda")
    xs.cache_write(k, v, cache, pages)
    back = [torch.empty(1, H, 2000, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    xs.cache_read(cache, pages, *back)
    for Nq in (1, 200):
        q = torch.randn(2, H, Nq, d, generator=g, device="cuda").bfloat16()
        o = torch.empty_like(q)
        xs.prefix_attn(q, o, cache=cache, prefix_pages=pages, prefix_len=2000,
                       workspace=xs.alloc_prefix_workspace(2, H, H, Nq, 2000, 0, d, prefix_cached=True))
        none = [q.new_zeros(2, H, 0, d).double() for _ in range(2)]
        check(o, prefix_formula(q.double(), [b[0].double() for b in back], none, [0, 0], d ** -0.5))


def test_layer_from_projection_to_shards(xs):
    """As a program uses them together: rotary positions and norms, the new tokens into the cache, attention over the
    shared history and the requests' own tokens, into sequence shards; then one more token a request."""
    B, H, Hk, d, page, P = 2, 8, 4, 128, 32, 4
    g = torch.Generator(device="cuda").manual_seed(16)
    normal = lambda *s: torch.randn(s, generator=g, device="cuda")   # noqa: E731
    n_hist, n_new = 500, 96
    cache = xs.alloc_cache(64, Hk, page, d)
    order = torch.randperm(64, generator=g, device="cuda").to(torch.int32)
    hist, own = order[:16].contiguous(), order[16:16 + 2 * 4].view(2, 4).contiguous()
    one = torch.ones(d, device="cuda")

    def project(b, n, first):
        x = normal(b, n, H + 2 * Hk, d).bfloat16()
        q, k, v = (torch.empty(b, h, n, d, dtype=torch.bfloat16, device="cuda") for h in (H, Hk, Hk))
        pos = (first + torch.arange(n, device="cuda"))[:, None].to(torch.int32).contiguous()
        xs.qkv_rope(x[:, :, :H], x[:, :, H:H + Hk], x[:, :, H + Hk:], q, k, v, pos, (d,), q_weight=one, k_weight=one)
        return q, k, v

    def read(pages, n, b):
        k, v = (torch.empty(b, Hk, n, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        xs.cache_read(cache, pages, k, v)
        return k.double(), v.double()

    _, k, v = project(1, n_hist, 0)
    xs.cache_write(k, v, cache, hist)
    prefix = [t[0] for t in read(hist, n_hist, 1)]
    assert (prefix[0] - k[0].double()).abs().max() <= 2.0 ** -4 * k.abs().max()
    q, k, v = project(B, n_new, n_hist)
    shards = xs.alloc_shards(B, n_new, H, d, P)
    ws = xs.alloc_prefix_workspace(B, H, Hk, n_new, n_hist, n_new, d, prefix_cached=True)
    xs.prefix_attn_fused(q, shards, k=k, v=v, cache=cache, prefix_pages=hist, prefix_len=n_hist, workspace=ws)
    check(torch.cat(shards, 1).transpose(1, 2),
          prefix_formula(q.double(), prefix, [k.double(), v.double()], [n_new] * B, d ** -0.5), "the frame")
    xs.cache_write(k, v, cache, own)
    start = torch.full((B,), n_new, dtype=torch.int32, device="cuda")
    for step in range(3):
        q, k, v = project(B, 1, n_hist + n_new + step)
        xs.cache_write(k, v, cache, own, start=start)
        start += 1
        o = torch.empty_like(q)
        xs.prefix_attn(q, o, cache=cache, prefix_pages=hist, prefix_len=n_hist, pages=own, max_len=4 * page, kv_len=start,
                       workspace=ws)
        mine = read(own, n_new + step + 1, B)
        check(o, prefix_formula(q.double(), prefix, mine, [n_new + step + 1] * B, d ** -0.5), f"token {step}")
    assert xs.last_device_status() == xs.OK


def test_binding_refuses(xs):
    """Operands that do not belong together, on the host, before any launch."""
    q = torch.zeros(2, 4, 8, 64, dtype=torch.bfloat16, device="cuda")
    o = torch.full_like(q, 3.0)
    kv, pre = torch.zeros(2, 2, 20, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 20, 64, dtype=torch.bfloat16, device="cuda")
    cache = xs.alloc_cache(4, 2, 16, 64)
    one, two = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    for kw in (dict(k=kv), dict(v=kv), dict(prefix_v=pre), dict(prefix_k=pre), dict(prefix_len=3), dict(max_len=3),
               dict(prefix_pages=one), dict(pages=two), dict(cache=cache, prefix_pages=two), dict(cache=cache, prefix_pages=[0]),
               dict(cache=cache, prefix_pages=one, prefix_len=49), dict(cache=cache, prefix_pages=one, prefix_len=-1),
               dict(cache=cache, pages=two, max_len=49), dict(cache=cache, pages=two, v=kv),
               dict(cache=cache, prefix_pages=one, prefix_v=pre), dict(cache=cache, prefix_pages=one, prefix_k=pre, prefix_v=pre),
               dict(cache=cache, pages=two[:1]), dict(cache=cache, pages=two.long()), dict(k=kv, v=kv[:, :1]),
               dict(k=kv, v=kv.float()), dict(k=kv.transpose(2, 3), v=kv), dict(k=kv, v=kv, kv_len=one),
               dict(k=kv.cpu(), v=kv.cpu()), dict(k=kv, v=kv, workspace=torch.zeros(8))):
        with pytest.raises(ValueError):
            xs.prefix_attn(q, o, **kw)
            pytest.fail(f"took {sorted(kw)}")
    with pytest.raises(ValueError):
        xs.prefix_attn_fused(q, xs.alloc_shards(2, 8, 4, 64, 2)[:1], k=kv, v=kv)
    with pytest.raises(ValueError):   # other heads than k's
        xs.prefix_attn(q, o, cache=xs.alloc_cache(4, 4, 16, 64), prefix_pages=one, k=kv, v=kv)
    with pytest.raises(xs.XsError):   # other columns than q's
        xs.prefix_attn(q, o, cache=xs.alloc_cache(4, 2, 16, 128), prefix_pages=one, k=kv, v=kv)
    assert (o == 3).all()
