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
