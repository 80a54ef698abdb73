"""prefix_attn where a CTA takes many items one after the other, and cached values that are not numbers."""
import pytest
import torch

from cache_ref import values
from test_gpu_prefix import Problem, check, xs   # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def row_of(p, pages, i):
    """(page, row in it) of place i of a list."""
    size = p.codes[0].shape[2]
    return int(pages[i // size]), i % size


@pytest.mark.parametrize("Np", [0, 300])          # one tile, and several
@pytest.mark.parametrize("Nq", [1, 33, 200])
def test_cached_values_without_a_scale(xs, Nq, Np):
    """A value row with the scale byte 255 beside a finite key makes NaN of the rows that see it and of no others."""
    p = Problem(xs, 4, 4, 2, 128, Nq, Np, 60, [60, 3, 60, 17], "cache", "cache", seed=21)
    ws = p.workspace()
    before = p.run(ws).clone(), p.run().clone()
    scale = p.scales[1]
    page, row = row_of(p, p.kw["pages"][2], 5)
    keep = int(scale[page, 0, row])
    scale[page, 0, row] = 255
    for got, ref in zip((p.run(ws), p.run()), before):
        assert got[2, :2].isnan().all()
        assert torch.equal(got[[0, 1, 3]], ref[[0, 1, 3]]) and torch.equal(got[2, 2:], ref[2, 2:])
    scale[page, 0, row] = keep
    if Np:
        page, row = row_of(p, p.kw["prefix_pages"], 131)
        scale[page, 1, row] = 255
        for got, ref in zip((p.run(ws), p.run()), before):
            assert got[:, 2:].isnan().all() and torch.equal(got[:, :2], ref[:, :2])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq", [1, 20, 50])
@pytest.mark.parametrize("Np,Nk,own", [(100, 0, "bf16"), (0, 90, "cache"), (0, 90, "bf16"), (100, 90, "cache"), (300, 40, "bf16")])
def test_items_in_turn(xs, d, Nq, Np, Nk, own):
    """Five and more items a CTA, of one tile (a group of warps then has none of them) and of several; what one item
    finds among its values is not another's."""
    Hk = 5 * sms() + 3
    p = Problem(xs, 2, Hk, Hk, d, Nq, Np, Nk, [Nk, Nk // 2], "cache", own, page=16, seed=22)
    want = p.want()
    check(p.run(), want)
    g = torch.Generator(device="cuda").manual_seed(23)
    bad = torch.rand(Hk, generator=g, device="cuda") < 0.3
    if Np:
        page, row = row_of(p, p.kw["prefix_pages"], 7)
        p.scales[1][page, bad, row] = 255
    elif own == "cache":
        for b in range(2):
            page, row = row_of(p, p.kw["pages"][b], 7)
            p.scales[1][page, bad, row] = 255
    else:
        p.kw["v"][:, bad, 7, 3] = float("nan")
    first = p.run().clone()
    assert (first[:, bad].isnan().all() if Np or own == "cache" else first[:, bad][..., 3].isnan().all())
    check(first[:, ~bad], (want[0][:, ~bad], want[1][:, ~bad]))
    for _ in range(10):
        again = p.run()
        assert torch.equal(again[:, ~bad], first[:, ~bad]) and torch.equal(again.isnan(), first.isnan())
    assert xs.last_device_status() == xs.OK


def run_both(p, ws):
    """The call with cached parts read as they are, and with a workspace (for many rows: read back first)."""
    return p.run().clone(), p.run(ws).clone()


@pytest.mark.parametrize("code,byte", [(0x7f, 127), (0xff, 3), (0x7e, 254), (0xfe, 247), (0x7f, 140)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq", [1, 33, 200])
def test_cached_values_that_are_not_numbers(xs, Nq, d, code, byte):
    """A NaN's code under an ordinary scale byte, or a value past the largest bf16: the rows that see it have no finite
    number in its column, the others are as they were."""
    p = Problem(xs, 4, 4, 2, d, Nq, 300, 60, [60, 3, 60, 17], "cache", "cache", seed=24)
    ws = p.workspace()
    before = run_both(p, ws)
    page, row = row_of(p, p.kw["pages"][2], 5)
    keep = p.codes[1][page, 0, row].clone(), int(p.scales[1][page, 0, row])
    p.codes[1][page, 0, row, 37] = code
    p.scales[1][page, 0, row] = byte
    for got, ref in zip(run_both(p, ws), before):
        assert not torch.isfinite(got[2, :2, :, 37]).any()
        assert torch.equal(got[[0, 1, 3]], ref[[0, 1, 3]]) and torch.equal(got[2, 2:], ref[2, 2:])
    p.codes[1][page, 0, row], p.scales[1][page, 0, row] = keep
    for i in (131, 299):   # a whole tile of the prefix, and its last one
        page, row = row_of(p, p.kw["prefix_pages"], i)
        keep = p.codes[1][page, 1, row].clone(), int(p.scales[1][page, 1, row])
        p.codes[1][page, 1, row, 40] = code
        p.scales[1][page, 1, row] = byte
        for got, ref in zip(run_both(p, ws), before):
            assert not torch.isfinite(got[:, 2:, :, 40]).any() and torch.equal(got[:, :2], ref[:, :2])
        p.codes[1][page, 1, row], p.scales[1][page, 1, row] = keep
    for got, ref in zip(run_both(p, ws), before):
        assert torch.equal(got, ref)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq", [1, 33, 300])
@pytest.mark.parametrize("e", [100, 113, 116, -112, -120])
def test_scores_of_scales_far_from_queries(xs, Nq, d, e):
    """Keys of some 2^e against queries of 2^-e: their products are ordinary scores. Other keys in the same tiles are far
    smaller (at -120 all are alike, and queries reach 2^120); rows of queries of zeros see weights that are all the same."""
    B, H, Hk, Np, Nk = 2, 2, 1, 260, 140
    p = Problem(xs, B, H, Hk, d, Nq, Np, Nk, [140, 0], "cache", "cache", page=16, seed=25)
    g = torch.Generator(device="cuda").manual_seed(26)
    t = p.scales[0]
    far = torch.rand(t.shape, generator=g, device="cuda") < 0.5
    lower = torch.randint(-120, e - 30 if e > 0 else max(e - 3, -119), t.shape, generator=g, device="cuda")
    t.copy_((torch.where(far, torch.full_like(lower, e), lower) + 127).to(torch.uint8))
    p.q.copy_((p.q.double() * 2.0 ** (-e - 2)).bfloat16())
    p.q[0, 1, 0] = 0
    n = p.kw["prefix_pages"].long()
    k = values(p.codes[0], t)
    p.prefix[0] = k[n].transpose(0, 1).flatten(1, 2)[:, :Np]
    p.own[0] = torch.stack([k[p.kw["pages"][b].long()].transpose(0, 1).flatten(1, 2)[:, :Nk] for b in range(B)])
    used = torch.zeros(t.shape[0], 16, dtype=torch.bool, device="cuda")
    for pages, count in ((p.kw["prefix_pages"], Np), (p.kw["pages"][0], Nk)):
        for i in range(count):
            used[row_of(p, pages, i)] = True
    for behind in (0, 127, 246, 254, 255):     # scale bytes of rows that no request sees
        t.masked_fill_(~used[:, None], behind)
        p.test()


@pytest.mark.parametrize("d", [64, 128])
def test_requests_of_different_scales_in_one_tile(xs, d):
    """One request's keys are large and its queries small, the other's the reverse."""
    p = Problem(xs, 2, 2, 1, d, 1, 0, 48, [48, 48], "cache", "cache", page=16, seed=27)
    t = p.scales[0]
    for b, e in enumerate((116, -114)):
        t[p.kw["pages"][b].long()] = e + 127
        p.q[b] = (p.q[b].double() * 2.0 ** (-e - 2)).bfloat16()
    k = values(p.codes[0], t)
    p.own[0] = torch.stack([k[p.kw["pages"][b].long()].transpose(0, 1).flatten(1, 2)[:, :48] for b in range(2)])
    p.test()


@pytest.mark.parametrize("prefix,own", [("cache", "cache"), ("cache", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("d,B,Nq", [(128, 2, 1), (64, 3, 17), (128, 2, 50), (64, 1, 128)])      # 4, 2, 1 and 1 copies of the rows
@pytest.mark.parametrize("full", [1, 2, 3])
def test_units_past_full_waves(xs, full, d, B, Nq, prefix, own):
    """A few units more than fill all SMs once, twice, three times, one tile of rows each: with a workspace the last ones
    (more than SMs) are cut after none, one and two whole units a CTA, without one a CTA takes up to four."""
    H = full * sms() + 9
    p = Problem(xs, B, H, H, d, Nq, 1500, 140, [140, 0, 33][:B], prefix, own, page=64, seed=30 + full)
    want, ws = p.want(), p.workspace()
    whole, cut = p.run(), p.run(ws)
    check(whole, want, "whole units")
    check(cut, want, "cut units")
    assert not torch.equal(whole, cut)     # (other sums: some were cut)
    for _ in range(5):
        assert torch.equal(p.run(ws.fill_(0xff)), cut) and torch.equal(p.run(), whole)
    assert xs.last_device_status() == xs.OK


@pytest.mark.parametrize("own", ["cache", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("full", [1, 2, 3])
def test_pairs_of_tiles_past_full_waves(xs, full, d, own):
    """The same with many rows: five units of two row tiles a head, requests whose ends lie inside one."""
    Hk = (full * sms() + 9 + 4) // 5
    p = Problem(xs, 3, Hk, Hk, d, 300, 2500, 400, [400, 0, 129], "bf16", own, page=64, seed=40 + full)
    want, ws = p.want(), p.workspace()
    got = p.run(ws)
    check(got, want, "cut units")
    for _ in range(5):
        assert torch.equal(p.run(ws.fill_(0xff)), got)
    check(p.run(), want, "whole units")
    assert xs.last_device_status() == xs.OK


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq", [1, 20, 50, 200])
def test_every_code(xs, Nq, d):
    """All finite codes of keys and values, zeros and the format's subnormals among them, under scales down to 2^-120 (values)."""
    p = Problem(xs, 2, 2, 1, d, Nq, 300, 70, [70, 13], "cache", "cache", page=32, seed=28, scale=2.0 ** -7)
    g = torch.Generator(device="cuda").manual_seed(29)
    for c in p.codes:
        size = torch.randint(0, 127, c.shape, generator=g, device="cuda", dtype=torch.uint8)
        c.copy_(size | (c & 0x80))
    p.scales[0].copy_(torch.randint(112, 119, p.scales[0].shape, generator=g, device="cuda", dtype=torch.uint8))
    p.scales[1].copy_(torch.where(torch.rand(p.scales[1].shape, generator=g, device="cuda") < 0.5, 7, 150).to(torch.uint8))
    k, v = (values(p.codes[i], p.scales[i]) for i in range(2))
    n = p.kw["prefix_pages"].long()
    for i, x in enumerate((k, v)):
        p.prefix[i] = x[n].transpose(0, 1).flatten(1, 2)[:, :300]
        p.own[i] = torch.stack([x[p.kw["pages"][b].long()].transpose(0, 1).flatten(1, 2)[:, :70] for b in range(2)])
    p.test()
    p.scales[1].fill_(7)       # (values below bf16's normal ones, in tiles of the short loop too)
    v = values(p.codes[1], p.scales[1])
    p.prefix[1] = v[n].transpose(0, 1).flatten(1, 2)[:, :300]
    p.own[1] = torch.stack([v[p.kw["pages"][b].long()].transpose(0, 1).flatten(1, 2)[:, :70] for b in range(2)])
    want, ws = p.want(), p.workspace()
    for got in (p.run(), p.run(ws)):
        # as in check, with a subnormal result's rounding, 2^-134, and fp32's own at most 2^-149 a key in the sums
        assert ((got.double() - want[0]).abs() <= 2.0 ** -8 * want[0].abs() + (2.0 ** -8 + 2.0 ** -11) * want[1] + 2.0 ** -133).all()
