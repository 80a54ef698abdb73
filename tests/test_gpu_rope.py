"""qkv_rope against the formula in 64 bits on the CPU.

Tolerance of an element, from the arithmetic: the output rounding, at most half a step of the type
(u = 2^-8 bf16, 2^-11 fp16, 2^-24 fp32, relative to the value), plus the fp32 work before it, which
is relative to the pair's length r: the norm (a sum of up to 256 squares over 8 per thread and 5
shuffles: 13 roundings, halved by the root, a division, an addition, rsqrt to 2 ulp, two products:
under 16 * 2^-24), sine and cosine (sincospif within 2 ulp of values up to 1, its argument rounded
to 2^-24 of a turn's half and cut at 2^-32 of a turn: pi * 2^-24 + 2^-30 in the angle) and three
roundings of the rotation: 32 * 2^-24 * r in all. For far positions the table of exact angles
itself is off by 2^-52 relative, at most 2^-21 of a radian at 2^31: added where |pos| is large."""
import math
from fractions import Fraction

import pytest
import torch

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}


@pytest.fixture(scope="module")
def xs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    from all_layout_gb300 import xs as _xs
    torch.cuda.set_device(0)
    return _xs


def formula(x, pos, axes, freqs, weight, eps, adjacent, rotate):
    """x [B, N, H, d] -> ([B, H, N, d] in 64 bits, length of each element's pair)."""
    x = x.double()
    if weight is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()
    size = x.abs()
    if rotate:
        rot = sum(axes)
        axis = torch.tensor([a for a, n in enumerate(axes) for _ in range(n // 2)])
        ang = pos.double()[..., axis] * torch.tensor(freqs, dtype=torch.float64)
        ang = ang if ang.dim() == 3 else ang[None]
        cos, sin = ang.cos()[:, :, None], ang.sin()[:, :, None]
        lo = torch.arange(0, rot, 2) if adjacent else torch.arange(rot // 2)
        hi = lo + 1 if adjacent else lo + rot // 2
        a, b = x[..., lo], x[..., hi]
        x, size = x.clone(), size.clone()
        x[..., lo], x[..., hi] = a * cos - b * sin, b * cos + a * sin
        size[..., lo] = size[..., hi] = torch.hypot(a, b)
    return x.transpose(1, 2), size.transpose(1, 2)


def check(got, want, what, far=0.0):
    ref, size = want
    got = got.cpu()
    tol = U[got.dtype] * ref.abs() + (32 * 2.0 ** -24 * (1 + U[got.dtype]) + far) * size + TINY[got.dtype]
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} off, worst {float((err / tol.clamp_min(1e-300)).max()):.2f} of the tolerance"


def freqs_of(axes, theta=10000.0):
    return [theta ** (-2.0 * i / a) for a in axes for i in range(a // 2)]


def case(B, N, H, Hk, d, axes, src, dst, norm, seed, hi=5000, shared=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, N, H + 2 * Hk, d, generator=g).to(src)
    pos = torch.randint(-hi, hi + 1, ((N, len(axes)) if shared else (B, N, len(axes))), generator=g, dtype=torch.int32)
    w = [1 + 0.2 * torch.randn(d, generator=g) if norm else None for _ in range(2)]
    out = [torch.full((B, h, N, d), math.nan, dtype=dst, device="cuda") for h in (H, Hk, Hk)]
    return x, pos, w, out


BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("adjacent", [True, False])
@pytest.mark.parametrize("B,N,H,Hk,d,axes,src,dst,norm", [
    (1, 1, 1, 1, 16, (16,), BF, BF, True),
    (1, 1, 24, 24, 128, (16, 56, 56), BF, BF, True),
    (8, 1, 3, 1, 64, (32, 32), BF, BF, False),
    (2, 3, 5, 5, 80, (16, 32, 32), FP, BF, True),
    (3, 129, 6, 2, 72, (16, 8, 8), HF, BF, True),
    (2, 257, 4, 4, 96, (32, 32, 32), HF, HF, False),
    (1, 1000, 2, 1, 256, (64, 96, 96), BF, BF, True),
    (1, 33, 7, 7, 256, (16, 16, 16, 16), FP, FP, True),
    (2, 77, 9, 3, 16, (16,), FP, FP, False),
    (1, 2049, 1, 1, 128, (32, 48, 48), BF, BF, False),
    (2, 50, 13, 13, 24, (16,), BF, BF, True),
])
def test_formula(xs, adjacent, B, N, H, Hk, d, axes, src, dst, norm):
    x, pos, w, (q, k, v) = case(B, N, H, Hk, d, axes, src, dst, norm, seed=N + d)
    xd = x.cuda()
    wd = [t.cuda() if t is not None else None for t in w]
    xs.qkv_rope(xd[:, :, :H], xd[:, :, H:H + Hk], xd[:, :, H + Hk:], q, k, v, pos.cuda(), axes,
                q_weight=wd[0], k_weight=wd[1], interleaved=adjacent)
    fr = freqs_of(axes)
    check(q, formula(x[:, :, :H], pos, axes, fr, w[0], 1e-6, adjacent, True), "q")
    check(k, formula(x[:, :, H:H + Hk], pos, axes, fr, w[1], 1e-6, adjacent, True), "k")
    check(v, formula(x[:, :, H + Hk:], pos, axes, fr, None, 1e-6, adjacent, False), "v")


def test_axis_widths_that_cut_a_vector(xs):
    """Adjacent pairs of axes of 44, 42 and 42 columns (eight columns straddle two axes), and 10
    rotated columns of 64 (the rotated part ends inside a vector)."""
    for axes, d in (((44, 42, 42), 128), ((4, 6), 64), ((2,), 8)):
        x, pos, w, (q, k, v) = case(2, 70, 3, 2, d, axes, BF, BF, True, seed=5, shared=True)
        xd = x.cuda()
        xs.qkv_rope(xd[:, :, :3], xd[:, :, 3:5], xd[:, :, 5:], q, k, v, pos.cuda(), axes,
                    q_weight=w[0].cuda(), k_weight=w[1].cuda())
        check(q, formula(x[:, :, :3], pos, axes, freqs_of(axes), w[0], 1e-6, True, True), "q")
        check(k, formula(x[:, :, 3:5], pos, axes, freqs_of(axes), w[1], 1e-6, True, True), "k")


def test_far_and_negative_positions(xs):
    axes, d, N = (64, 64), 128, 64
    x, _, _, (q, k, v) = case(1, N, 2, 1, d, axes, FP, FP, False, seed=9)
    g = torch.Generator().manual_seed(3)
    pos = torch.randint(-(1 << 31), (1 << 31) - 1, (N, 2), generator=g, dtype=torch.int64).to(torch.int32)
    pos[0] = torch.tensor([(1 << 31) - 1, -(1 << 31)], dtype=torch.int32)
    xs.qkv_rope(x[:, :, :2].cuda(), None, None, q, None, None, pos.cuda(), axes)
    check(q, formula(x[:, :, :2], pos, axes, freqs_of(axes), None, 0, True, True), "q", far=2.0 ** -20)


def test_custom_frequencies_above_a_turn(xs):
    axes = (8,)
    fr = [7.25, -0.5, 0.0, 1e-7]
    x, pos, _, (q, _, _) = case(1, 40, 2, 1, 64, axes, FP, FP, False, seed=2, hi=300)
    xs.qkv_rope(x[:, :, :2].cuda(), None, None, q, None, None, pos.cuda(), axes, freqs=fr)
    check(q, formula(x[:, :, :2], pos, axes, fr, None, 0, True, True), "q")


@pytest.mark.parametrize("freq", [0.3, 1.0, 7.25, -100.0, 1e4, 1e6, -2.5e15, 1.7e19])
def test_angles_of_every_position_and_frequency(xs, freq):
    """pos * freq modulo a turn from exact rationals, over the whole range of 32-bit positions: no allowance
    for far positions or high frequencies beside the rounding of the angle's fraction of a turn."""
    from test_rope_host import two_pi
    g = torch.Generator().manual_seed(3)
    pos = torch.randint(-(1 << 31), (1 << 31) - 1, (97, 1), generator=g, dtype=torch.int64).to(torch.int32)
    pos[:6, 0] = torch.tensor([(1 << 31) - 1, -(1 << 31), -1, 1, 0, (1 << 31) - 2], dtype=torch.int32)
    x = torch.randn(1, 97, 2, 8, generator=g)
    q = torch.empty(1, 2, 97, 8, device="cuda")
    xs.qkv_rope(x.cuda(), None, None, q, None, None, pos.cuda(), (2,), freqs=[freq])
    turns = [float(Fraction(freq) * int(p) / two_pi() % 1) for p in pos[:, 0]]   # off by 2^-53 at most
    ang = 2 * math.pi * torch.tensor(turns, dtype=torch.float64)[None, :, None]
    a, b = x[..., 0].double(), x[..., 1].double()
    want, size = x.double().clone(), x.double().abs()
    want[..., 0], want[..., 1] = a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()
    size[..., :2] = torch.hypot(a, b)[..., None]
    check(q, (want.transpose(1, 2), size.transpose(1, 2)), f"freq {freq}")


@pytest.mark.parametrize("adjacent", [True, False])
def test_in_place_on_token_major_and_back(xs, adjacent):
    """In place on [B, N, H, d] (a sequence shard), then undone by negated positions."""
    axes = (16, 24, 24) if adjacent else (32, 16, 16)
    x, pos, _, _ = case(2, 31, 5, 1, 64, axes, FP, FP, False, seed=6)
    x = x[:, :, :5].contiguous()
    y = x.cuda()
    xs.qkv_rope(y, None, None, y.transpose(1, 2), None, None, pos.cuda(), axes, interleaved=adjacent)
    want = formula(x, pos, axes, freqs_of(axes), None, 0, adjacent, True)
    check(y.transpose(1, 2), want, "in place")
    xs.qkv_rope(y, None, None, y.transpose(1, 2), None, None, (-pos).cuda(), axes, interleaved=adjacent)
    size = want[1]
    assert ((y.cpu().double() - x.double()).abs().transpose(1, 2) <= 64 * 2.0 ** -24 * size * 2).all()


def test_strides_offsets_and_untouched_neighbours(xs):
    """Rows inside larger buffers on both sides; nothing else is written."""
    B, N, H, d, axes = 2, 19, 3, 64, (32, 32)
    g = torch.Generator().manual_seed(8)
    big = torch.randn(B + 1, N + 3, H + 2, d + 24, generator=g).to(BF).cuda()
    src = big[1:, 2:2 + N, 1:1 + H, 8:8 + d]
    pos = torch.randint(0, 99, (N, 2), generator=g, dtype=torch.int32)
    buf = torch.full((B, H + 1, N + 5, d + 16), 7.0, dtype=BF, device="cuda")
    dst = buf[:, 1:, 3:3 + N, 8:8 + d]
    xs.qkv_rope(src, None, None, dst, None, None, pos.cuda(), axes, interleaved=False)
    check(dst, formula(src.cpu(), pos, axes, freqs_of(axes), None, 0, False, True), "dst")
    dst.fill_(7.0)
    assert bool((buf == 7.0).all())


def test_broadcast_input(xs):
    """A batch stride of 0: one row of tokens for every batch entry, at its own positions."""
    x, pos, _, (q, _, _) = case(3, 21, 2, 1, 64, (64,), BF, BF, False, seed=4)
    one = x[:1, :, :2].cuda()
    xs.qkv_rope(one.expand(3, -1, -1, -1), None, None, q, None, None, pos.cuda(), (64,))
    check(q, formula(x[:1, :, :2].expand(3, -1, -1, -1), pos, (64,), freqs_of((64,)), None, 0, True, True), "q")


@pytest.mark.parametrize("adjacent", [True, False])
def test_infinities_and_nan_stay_where_they_are(xs, adjacent):
    """Special values in v, and in the columns of q past the rotated part, pass; a row's NaN stays in it."""
    x = torch.randn(1, 9, 3, 64).to(BF)
    x[0, 3, 0, 40], x[0, 4, 0, 63], x[0, 5, 2, 1] = math.inf, math.nan, -math.inf
    xd = x.cuda()
    out = [torch.zeros(1, 1, 9, 64, dtype=BF, device="cuda") for _ in range(3)]
    pos = torch.arange(9, dtype=torch.int32)[:, None].contiguous()
    xs.qkv_rope(xd[:, :, :1], xd[:, :, 1:2], xd[:, :, 2:], *out, pos.cuda(), (32,), interleaved=adjacent)
    q, k, v = (t.cpu() for t in out)
    assert torch.equal(v[0, 0], x[0, :, 2])
    assert torch.equal(q[0, 0, :, 32:].nan_to_num(nan=5.0), x[0, :, 0, 32:].nan_to_num(nan=5.0))
    assert torch.isfinite(q[0, 0, :, :32]).all() and torch.isfinite(k).all()


def test_large_and_tiny_rows_under_the_norm(xs):
    """Squares near the end of fp32's range and rows of zeros: x / sqrt(mean + eps)."""
    x = torch.randn(1, 6, 2, 128).to(BF)
    x[0, 0] = x[0, 0] * 1e17
    x[0, 1] = 0
    x[0, 2] = x[0, 2] * 1e-10
    w = torch.ones(128)
    q = torch.empty(1, 2, 6, 128, dtype=BF, device="cuda")
    pos = torch.zeros(6, 1, dtype=torch.int32)
    xs.qkv_rope(x.cuda(), None, None, q, None, None, pos.cuda(), (64,), q_weight=w.cuda())
    check(q, formula(x, pos, (64,), freqs_of((64,)), w, 1e-6, True, True), "q")


@pytest.mark.parametrize("adjacent", [True, False])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-30])
@pytest.mark.parametrize("H,d,src,dst", [(3, 8, FP, FP), (70, 80, BF, BF), (3, 128, BF, BF), (34, 256, FP, FP), (3, 128, FP, BF), (3, 64, HF, HF)])
def test_norm_over_the_whole_range_of_the_type(xs, H, d, src, dst, eps, adjacent):
    """Rows whose squares leave fp32's range, both ways, beside ordinary ones; a row of zeros stays one, also
    with eps = 0; a NaN stays in its row, and an infinity leaves zeros beside NaN. (Rows of subnormal numbers
    are left out where the result would be one too.)"""
    g = torch.Generator().manual_seed(d)
    sizes = [1.0, 0.0, 1e-4, 1e4] if src is HF else [1.0, 0.0, 1e-25, 1e20, 1e-37, 3e37, 1e-20, 1e18, 1e-12, 1e10]
    rows = torch.randn(len(sizes), H, d, generator=g).clamp(-4, 4) * torch.tensor(sizes)[:, None, None]
    rows[:, H // 2, 1:] *= 2.0 ** -30   # one column far above the others
    x = torch.cat([rows, torch.ones(2, H, d)])[None].to(src)
    x[0, -2, :, 3], x[0, -1, :, 5] = math.nan, math.inf
    N = x.shape[1]
    w = 1 + 0.2 * torch.randn(d, generator=g)
    pos = torch.zeros(N, 1, dtype=torch.int32)
    q = torch.full((1, H, N, d), 7.0, dtype=dst, device="cuda")
    xd = x.cuda()
    xs.qkv_rope(xd, None, None, q, None, None, pos.cuda(), (8,), q_weight=w.cuda(), eps=eps, interleaved=adjacent)
    want, size = formula(x[:, :-2], pos[:-2], (8,), freqs_of((8,)), w, eps, adjacent, True)
    check(q[:, :, :-2], (want.nan_to_num(nan=0.0), size.nan_to_num(nan=0.0)), "q")   # 0 / 0: the row of zeros
    assert not q[0, :, 1].any()
    assert q[0, :, -2].isnan().all()
    last = q[0, :, -1]
    pair = [4, 5] if adjacent else [1, 5]
    assert last[:, pair].isnan().any() and not last[:, [i for i in range(d) if i not in pair]].any()
    if src is dst:
        xs.qkv_rope(xd, None, None, xd.transpose(1, 2), None, None, pos.cuda(), (8,), q_weight=w.cuda(), eps=eps, interleaved=adjacent)
        assert torch.equal(xd.transpose(1, 2).nan_to_num(nan=9.0), q.nan_to_num(nan=9.0))


def test_norm_in_place_with_tiny_weights(xs):
    """Rows that are tiny after the norm are not normed twice."""
    x = torch.randn(1, 40, 37, 64, generator=torch.Generator().manual_seed(1))
    x[:, ::3, ::2] *= 1e-25
    w = torch.full((64,), 1e-27)
    pos, xd = torch.arange(40, dtype=torch.int32)[:, None].contiguous(), x.cuda()
    xs.qkv_rope(xd, None, None, xd.transpose(1, 2), None, None, pos.cuda(), (64,), q_weight=w.cuda(), eps=0.0)
    check(xd.transpose(1, 2), formula(x, pos, (64,), freqs_of((64,)), w, 0.0, True, True), "in place")


def test_offsets_past_32_bits(xs):
    """A head stride that puts the last rows more than 2^32 elements behind the first."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    stride = (1 << 32) + 4096
    buf = torch.empty(stride + 64 * 128, dtype=BF, device="cuda")
    x = buf.as_strided((1, 100, 2, 64), (stride * 2, 64, stride, 1))
    y = torch.empty(stride + 64 * 128, dtype=BF, device="cuda").as_strided((1, 2, 100, 64), (stride * 2, stride, 64, 1))
    src = torch.randn(1, 100, 2, 64).to(BF)
    x.copy_(src)
    pos = torch.arange(100, dtype=torch.int32)[:, None].contiguous()
    xs.qkv_rope(x, None, None, y, None, None, pos.cuda(), (64,))
    check(y, formula(src, pos, (64,), freqs_of((64,)), None, 0, True, True), "q")


def test_stream_and_graph(xs):
    x, pos, w, (q, k, v) = case(1, 200, 4, 4, 128, (32, 48, 48), BF, BF, True, seed=3)
    xd, pd, wd = x.cuda(), pos.cuda(), w[0].cuda()
    args = (xd[:, :, :4], xd[:, :, 4:8], xd[:, :, 8:], q, k, v, pd, (32, 48, 48))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    xs.qkv_rope(*args, q_weight=wd, k_weight=wd, stream=s)
    s.synchronize()
    first = [t.clone() for t in (q, k, v)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        xs.qkv_rope(*args, q_weight=wd, k_weight=wd)
    x2 = torch.randn_like(x.float()).to(BF)
    for data, want in ((x2, None), (x, first)):
        xd.copy_(data)
        for t in (q, k, v):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        if want:
            assert all(torch.equal(a, b) for a, b in zip((q, k, v), want))
        else:
            check(q, formula(x2[:, :, :4], pos, (32, 48, 48), freqs_of((32, 48, 48)), w[0], 1e-6, True, True), "q")


def test_tensors_without_heads(xs):
    """k and v of no heads (no rows to write) leave the others as they are."""
    x, pos, _, (q, k, v) = case(2, 9, 3, 0, 64, (64,), BF, BF, False, seed=1)
    xd = x.cuda()
    xs.qkv_rope(xd[:, :, :3], xd[:, :, 3:], xd[:, :, 3:], q, k, v, pos.cuda(), (64,))
    check(q, formula(x, pos, (64,), freqs_of((64,)), None, 0, True, True), "q")
    xs.qkv_rope(xd[:, :, 3:], xd[:, :, :3], None, k, q, None, pos.cuda(), (64,))
    check(q, formula(x, pos, (64,), freqs_of((64,)), None, 0, True, True), "q as k")


def test_empty(xs):
    z = torch.empty(1, 0, 4, 64, dtype=BF, device="cuda")
    xs.qkv_rope(z, None, None, z.transpose(1, 2), None, None, torch.empty(0, 1, dtype=torch.int32, device="cuda"), (64,))


def test_binding_refusals(xs):
    x = torch.zeros(1, 4, 2, 64, dtype=BF, device="cuda")
    y = torch.zeros(1, 2, 4, 64, dtype=BF, device="cuda")
    pos = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    ok = dict(q_in=x, k_in=None, v_in=None, q=y, k=None, v=None, pos=pos, axis_dims=(64,))
    xs.qkv_rope(**ok)
    for bad in (dict(pos=pos.long()), dict(pos=pos[:3]), dict(q=y[:, :1]), dict(q=y.double()), dict(k_in=x),
                dict(pos=pos.cpu()), dict(axis_dims=()), dict(freqs=[1.0]), dict(q_weight=torch.ones(64, device="cuda", dtype=BF)),
                dict(q_weight=torch.ones(32, device="cuda")), dict(q=torch.zeros(1, 2, 64, 4, dtype=BF, device="cuda").transpose(2, 3))):
        with pytest.raises(ValueError):
            xs.qkv_rope(**{**ok, **bad})
    with pytest.raises(xs.XsError):
        xs.qkv_rope(**{**ok, "axis_dims": (128,)})
    torch.cuda.synchronize()
