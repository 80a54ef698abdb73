"""Differential attention against its definition in 64 bits.

Tolerances, from the arithmetic. u = 2^-8 is half a bf16 step relative to a value. The weights of a
map, a_j (1 + e_j) with |e_j| <= u after their rounding to bf16, are divided by their own sum: a map's
x_t = sum_j a_j v_j becomes x_t + sum_j a_j e_j (v_j - x_t) to first order, off by at most u (A_t + |x_t|)
with A_t = sum_j a_j |v_j|; x by the sum over the maps, the second times |lambda|. Everything else
before the output is fp32: a score of d/2 products accumulated at up to 2^-23 each (128 * 2^-23 *
sum|q k| * scale < 2^-12 for the scores here, below 16), the exponential (2^-22), sums over the keys and the pieces (2^-24 a term, of positive terms): together
below u/4, taken as u/4 of the same sum. The norm multiplies by r = 1/sqrt(mean x^2 + eps): the row's own
error moves r by at most rms(error of x) * r relative. The output rounding adds u |o|.
Beside this bound of every element, the error as a whole: rounding errors are independent and uniform, of
standard deviation at most u/sqrt(3) of what is rounded, so the root of the summed squares is compared with
that of u^2/3 (sum_j a1_j^2 (v_j - x_1)^2 + lambda^2 a2_j^2 (v_j - x_2)^2, times the norm's factor squared,
+ o^2), times 1.5."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
BF = torch.bfloat16


@pytest.fixture(scope="module")
def xs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    from all_layout_gb300 import xs as _xs
    torch.cuda.set_device(0)
    return _xs


def reference(q, k, v, lam, lens=None, weight=None, eps=1e-5, out_scale=1.0, scale=None, rows=None):
    """(o, bound of |error|, expected variance) [B, H, rows, d] in 64 bits, head by head on the GPU."""
    B, H, Nq, d = q.shape
    Hk, Nk = k.shape[1], k.shape[2]
    half = d // 2
    scale = half ** -0.5 if scale is None else scale
    rows = torch.arange(Nq, device=q.device) if rows is None else rows
    out, tol, var = (torch.zeros(B, H, len(rows), d, dtype=torch.float64, device=q.device) for _ in range(3))
    for b in range(B):
        n = Nk if lens is None else max(0, min(Nk, int(lens[b])))
        if n == 0:
            continue
        for h in range(H):
            kk, vv = k[b, h * Hk // H, :n].double(), v[b, h * Hk // H, :n].double()
            for i in range(0, len(rows), 2048):
                qq = q[b, h, rows[i:i + 2048]].double()
                for part, f in ((slice(0, half), 1.0), (slice(half, d), -float(lam[h]))):
                    a = torch.softmax(qq[:, part] @ kk[:, part].T * scale, 1)
                    x, a2 = a @ vv, a.square()
                    out[b, h, i:i + 2048] += f * x
                    tol[b, h, i:i + 2048] += abs(f) * (a @ vv.abs() + x.abs())
                    var[b, h, i:i + 2048] += f * f * (a2 @ vv.square() - 2 * x * (a2 @ vv) + x.square() * a2.sum(1, keepdim=True)).clamp(min=0)
    tol *= U * 1.25
    factor = torch.full((1,), float(out_scale), dtype=torch.float64, device=q.device)
    extra = 0.0
    if weight is not None:
        r = 1 / (out.square().mean(-1, keepdim=True) + eps).sqrt()
        extra = tol.square().mean(-1, keepdim=True).sqrt() * r
        factor = r * weight.double() * out_scale
    o = out * factor
    tol = factor.abs() * tol + o.abs() * (extra + U + 2.0 ** -20) + 2.0 ** -134
    var = (var * factor.square() + o.square()) * U * U / 3
    return o, tol, var


def check(got, ref, what):
    o, tol, var = ref
    err = (got.double() - o).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off; first at "
                           f"{[int(i) for i in bad.nonzero()[0]]}, worst {float((err / tol).nan_to_num(nan=1e9).max()):.2f} of the bound")
    have, may = float(err.square().sum().sqrt()), 1.5 * float(var.sum().sqrt())
    assert have <= may or have < 1e-30, f"{what}: error {have:.3e} as a whole, {may:.3e} expected at most"


def inputs(B, H, Hk, Nq, Nk, d, seed, q_scale=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF)  # noqa: E731
    lam = 0.2 + 0.6 * torch.rand(H, generator=g, device="cuda")
    w = 1 + 0.2 * torch.randn(d, generator=g, device="cuda")
    return rnd(B, H, Nq, d) * q_scale, rnd(B, Hk, Nk, d), rnd(B, Hk, Nk, d), lam, w


def workspace(nbytes=96 << 20):
    return torch.zeros(nbytes, dtype=torch.uint8, device="cuda")


def done(xs, ws=None):
    torch.cuda.synchronize()
    assert xs.last_device_status() == xs.OK
    if ws is not None:
        assert not ws[:16384].any(), "the workspace's counters are not zero after the call"


SHAPES = [
    (1, 1, 1, 1, 1), (2, 3, 3, 1, 128), (1, 2, 1, 1, 129), (1, 1, 1, 128, 127), (1, 1, 1, 129, 128), (1, 2, 2, 127, 255),
    (2, 4, 2, 3, 700), (1, 2, 1, 300, 1), (3, 2, 2, 257, 385), (1, 6, 3, 640, 1025), (1, 1, 1, 9, 20000), (2, 24, 24, 1, 3000),
    (1, 3, 1, 8, 9001), (1, 40, 40, 500, 640), (1, 2, 2, 200, 9000), (700, 2, 1, 1, 5),
]


@pytest.mark.parametrize("use_ws", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("B,H,Hk,Nq,Nk", SHAPES)
def test_shapes(xs, B, H, Hk, Nq, Nk, d, use_ws):
    q, k, v, lam, w = inputs(B, H, Hk, Nq, Nk, d, seed=Nq + Nk + d)
    ws = workspace() if use_ws else None
    norm = w if (use_ws or d != 256) and (Nq + Nk) % 2 else None
    o = torch.full_like(q, math.nan)
    xs.diff_attn(q, k, v, o, lam, norm_weight=norm, out_scale=0.7, workspace=ws)
    done(xs, ws)
    check(o, reference(q, k, v, lam, weight=norm, out_scale=0.7), "o")


@pytest.mark.parametrize("use_ws", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("B,H,Hk,Nq,Nk,lens", [
    (3, 2, 1, 150, 300, (300, 131, 0)), (4, 3, 3, 1, 5000, (4999, 1, 0, 128)), (2, 2, 2, 260, 129, (500, -3)),
    (70, 1, 1, 5, 400, tuple((37 * i) % 401 for i in range(70))), (40, 8, 4, 130, 520, tuple((129 * i) % 521 for i in range(40))),
    (3, 2, 2, 200, 6000, (6000, 100, 0)), (60, 1, 1, 5, 3000, tuple((911 * i) % 3001 if i % 3 else i // 40 for i in range(60))),
])
def test_lengths_and_what_lies_behind_them(xs, B, H, Hk, Nq, Nk, lens, d, use_ws):
    """Keys past an entry's length hold NaN and infinities in k and v; entries without keys give zeros."""
    q, k, v, lam, w = inputs(B, H, Hk, Nq, Nk, d, seed=B + Nk + d)
    for b, n in enumerate(lens):
        n = max(0, min(Nk, n))
        k[b, :, n:], v[b, :, n:] = math.nan, math.inf
        v[b, :, n:, ::2] = -math.inf
        v[b, :, n:, ::3] = math.nan
    ws = workspace() if use_ws else None
    norm = w if use_ws or d != 256 else None
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o = torch.full_like(q, math.nan)
    xs.diff_attn(q, k, v, o, lam, kv_len=kv_len, norm_weight=norm, workspace=ws)
    done(xs, ws)
    check(o, reference(q, k, v, lam, lens=lens, weight=norm), "o")
    for b, n in enumerate(lens):
        if n <= 0:
            assert not o[b].any()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_all_lengths_zero_and_no_keys(xs, d):
    q, k, v, lam, w = inputs(2, 2, 2, 140, 50, d, seed=d)
    ws = workspace()
    for kk, vv, kv_len in ((k, v, torch.zeros(2, dtype=torch.int32, device="cuda")), (k[:, :, :0], v[:, :, :0], None)):
        for eps in (1e-5, 0.0):
            o = torch.full_like(q, math.nan)
            xs.diff_attn(q, kk, vv, o, lam, kv_len=kv_len, norm_weight=w, eps=eps, workspace=ws)
            done(xs, ws)
            assert not o.any()


@pytest.mark.parametrize("use_ws", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("B,H,Nq,Nk,P", [(1, 4, 256, 256, 2), (2, 3, 7 * 41, 500, 7), (1, 24, 1024, 1024, 8), (2, 2, 8, 1300, 8), (1, 5, 200, 64, 1)])
def test_shards(xs, B, H, Nq, Nk, P, d, use_ws):
    """Into P shards carved from one allocation with canaries between them."""
    q, k, v, lam, w = inputs(B, H, H, Nq, Nk, d, seed=Nq + P)
    ws = workspace() if use_ws else None
    norm = w if use_ws or d != 256 else None
    size, gap = B * (Nq // P) * H * d, 1024
    buf = torch.full(((size + gap) * P + gap,), 3.0, dtype=BF, device="cuda")
    shards = [buf[gap + p * (size + gap):][:size].view(B, Nq // P, H, d) for p in range(P)]
    for s in shards:
        s.fill_(math.nan)
    xs.diff_attn_fused(q, k, v, shards, lam, norm_weight=norm, workspace=ws)
    done(xs, ws)
    got = torch.cat(shards, 1).transpose(1, 2)
    check(got, reference(q, k, v, lam, weight=norm), "shards")
    for s in shards:
        s.fill_(3.0)
    assert bool((buf == 3.0).all())


@pytest.mark.parametrize("d", [64, 128, 256])
def test_strides(xs, d):
    """Token-major operands inside larger buffers, a token-major output; nothing else is written."""
    B, H, Hk, Nq, Nk = 2, 4, 2, 200, 333
    q0, k0, v0, lam, w = inputs(B, H, Hk, Nq, Nk, d, seed=d + 1)
    qkv = torch.full((B, Nk, H + 2 * Hk + 1, d + 8), math.nan, dtype=BF, device="cuda")
    q = qkv[:, :Nq, :H, :d].transpose(1, 2)
    k, v = qkv[:, :, H:H + Hk, :d].transpose(1, 2), qkv[:, :, H + Hk:H + 2 * Hk, 8:].transpose(1, 2)
    q.copy_(q0), k.copy_(k0), v.copy_(v0)
    buf = torch.full((B + 1, Nq + 2, H + 3, d + 16), 5.0, dtype=BF, device="cuda")
    o = buf[1:, 1:1 + Nq, 2:2 + H, 8:8 + d].transpose(1, 2)
    xs.diff_attn(q, k, v, o, lam, workspace=workspace())
    done(xs)
    check(o, reference(q, k, v, lam), "o")
    o.fill_(5.0)
    assert bool((buf == 5.0).all())


def test_offsets_past_32_bits(xs):
    """A head stride of more than 2^32 elements in k, v and o."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    d, Nq, Nk, stride = 128, 70, 200, (1 << 32) + 8192
    q, k0, v0, lam, w = inputs(1, 2, 2, Nq, Nk, d, seed=4)
    view = lambda n: torch.empty(stride + n * d, dtype=BF, device="cuda").as_strided((1, 2, n, d), (2 * stride, stride, d, 1))  # noqa: E731
    k, v, o = view(Nk), view(Nk), view(Nq)
    k.copy_(k0), v.copy_(v0)
    xs.diff_attn(q, k, v, o, lam, norm_weight=w)
    done(xs)
    check(o, reference(q, k, v, lam, weight=w), "o")


@pytest.mark.parametrize("use_ws", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_peaked_and_growing_scores(xs, d, use_ws):
    """Scores that grow along the keys (the running maximum is rescaled again and again), and rows
    that one key takes whole."""
    B, H, Nq, Nk = 1, 2, 130, 1400
    q, k, v, lam, w = inputs(B, H, H, Nq, Nk, d, seed=7, q_scale=4.0)
    ramp = torch.linspace(0.05, 1.6, Nk, device="cuda")
    k = (k.float() * ramp[:, None]).to(BF)
    o = torch.full_like(q, math.nan)
    xs.diff_attn(q, k, v, o, lam, norm_weight=w if use_ws else None, workspace=workspace() if use_ws else None)
    done(xs)
    check(o, reference(q, k, v, lam, weight=w if use_ws else None), "o")


@pytest.mark.parametrize("use_ws", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("grow", ["up", "down", "steps"])
def test_scores_that_grow_past_every_range(xs, d, use_ws, grow):
    """Whole-numbered q and k, whose products are exact, with scores from 0 to tens of thousands: a row's
    weights would overflow or vanish if their reference did not move with them (or moved with the smallest)."""
    g = torch.Generator(device="cuda").manual_seed(d)
    H, Nq, Nk = 2, 140, 1500
    size = {"up": torch.linspace(0, 120, Nk), "down": torch.linspace(120, 0, Nk),
            "steps": torch.tensor([0.0, 100.0, 1.0, 120.0, 3.0, 60.0]).repeat_interleave(Nk // 6)}[grow].cuda()
    q = torch.randint(-4, 5, (1, H, Nq, d), generator=g, device="cuda").to(BF)
    k = (torch.randint(-2, 3, (1, H, Nk, d), generator=g, device="cuda") * size[:, None]).round().to(BF)
    v = torch.randn(1, H, Nk, d, generator=g, device="cuda").to(BF)
    lam = torch.rand(H, generator=g, device="cuda")
    o = torch.full_like(q, math.nan)
    xs.diff_attn(q, k, v, o, lam, workspace=workspace() if use_ws else None)
    done(xs)
    check(o, reference(q, k, v, lam), "o")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("below", [0, 6])
def test_scores_of_minus_infinity(xs, d, below):
    """The first keys' scores overflow to -inf (weight 0); those behind them are ordinary, or all low."""
    q, k, v, lam, _ = inputs(1, 2, 2, 150, 900, d, seed=d)
    q = (q.float().abs() + 0.5).to(BF).float() * 2.0 ** 64
    kk = k.float()
    kk[:, :, :200] = -(kk[:, :, :200].abs() + 0.5) * 2.0 ** 64 * 4.0
    kk[:, :, 200:] = (kk[:, :, 200:] * 0.25 - below) * 2.0 ** -64
    q, k = q.to(BF), kk.to(BF)
    for ws in (None, workspace()):
        o = torch.full_like(q, math.nan)
        xs.diff_attn(q, k, v, o, lam, workspace=ws)
        done(xs)
        # The oracle leaves the keys of weight 0 out; scores of some hundreds add 2^-23 of their size.
        check(o, reference(q, k[:, :, 200:].contiguous(), v[:, :, 200:].contiguous(), lam), "o")


@pytest.mark.parametrize("use_ws", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Nq", [3, 20, 150])
def test_maps_without_a_finite_score(xs, Nq, d, use_ws):
    """Every score of one map overflows to -inf: that map gives 0, the other its mean, in whole units and
    in pieces; with both maps so the rows are zeros, under a norm too."""
    H, Nk, half = 2, 6000, d // 2
    ws = workspace() if use_ws else None
    for gone in ((0,), (1,), (0, 1)):
        q, k, v, lam, w = inputs(1, H, H, Nq, Nk, d, seed=Nq + d)
        for t in gone:
            part = slice(t * half, (t + 1) * half)
            q[..., part] = (q[..., part].float().abs() + 0.5) * 2.0 ** 64
            k[..., part] = -(k[..., part].float().abs() + 0.5) * 2.0 ** 66
        o = torch.full_like(q, math.nan)
        xs.diff_attn(q, k, v, o, lam, norm_weight=w if len(gone) == 2 and (use_ws or d != 256) else None, workspace=ws)
        done(xs, ws)
        if len(gone) == 2:
            assert not o.any()
            continue
        # The map that is left, as a first map whose second has lambda 0; times -lambda where it is the second.
        qq, kk = (q, k) if gone == (1,) else (x.roll(half, -1) for x in (q, k))
        qq, kk = qq.clone(), kk.clone()
        qq[..., half:] = 0
        ref, tol, var = reference(qq, kk, v, torch.zeros_like(lam))
        if gone == (0,):
            f = -lam.double()[None, :, None, None]
            ref, tol, var = ref * f, tol * f.abs(), var * f.square()
        check(o, (ref, tol, var), f"map {gone[0]} gone")


@pytest.mark.parametrize("d,use_ws", [(64, False), (64, True), (128, False), (128, True), (256, True)])
@pytest.mark.parametrize("Nq,Nk", [(3, 6000), (12, 6000), (40, 6000), (150, 6000), (150, 40)])
@pytest.mark.parametrize("size,eps", [(1e-25, 0.0), (1e20, 1e-5), (1e-20, 1e-38), (1.0, 0.0)])
def test_norm_of_rows_whose_squares_leave_the_range(xs, Nq, Nk, d, size, eps, use_ws):
    """x / sqrt(mean x^2 + eps) of rows that fp32 holds but not their squares; one head has its values in one
    half of the columns only, one in a single column."""
    q, k, v, lam, w = inputs(1, 3, 3, Nq, Nk, d, seed=Nq + Nk + d)
    v = (v.float() * size).to(BF)
    v[:, 1, :, :d // 2] = 0
    v[:, 2, :, 1:] = 0
    ws = workspace() if use_ws else None
    o = torch.full_like(q, math.nan)
    xs.diff_attn(q, k, v, o, lam, norm_weight=w, eps=eps, workspace=ws)
    done(xs, ws)
    check(o, reference(q, k, v, lam, weight=w, eps=eps), "o")


@pytest.mark.parametrize("lam_value", [0.0, 1.0, -0.5, 3.0])
def test_lambda_and_scale(xs, lam_value):
    q, k, v, _, _ = inputs(1, 3, 3, 200, 300, 128, seed=11)
    lam = torch.full((3,), lam_value, device="cuda")
    o = torch.empty_like(q)
    xs.diff_attn(q, k, v, o, lam, scale=0.05, out_scale=-2.0)
    done(xs)
    check(o, reference(q, k, v, lam, scale=0.05, out_scale=-2.0), "o")


def test_identical_values_give_them_back(xs):
    """Every key has the same v: both maps give it whatever their weights, x = (1 - lambda) v, off by the
    output's rounding and fp32's."""
    for d in (64, 128, 256):
        q, k, v, lam, _ = inputs(1, 2, 2, 150, 700, d, seed=d)
        v = v[:, :, :1].expand(-1, -1, 700, -1).contiguous()
        o = torch.empty_like(q)
        xs.diff_attn(q, k, v, o, lam, workspace=workspace())
        done(xs)
        want = (1 - lam.double())[None, :, None, None] * v[:, :, :150].double()
        assert ((o.double() - want).abs() <= U * want.abs() + 2.0 ** -12 * (1 + lam.double())[None, :, None, None] * v[:, :, :150].double().abs()).all()


@pytest.mark.parametrize("B,H,Nq,Nk,d", [(1, 24, 2048, 2048, 128), (1, 12, 1024, 2048, 256), (1, 48, 1024, 1500, 64), (4, 24, 1, 16384, 128), (1, 1, 1, 40000, 128)])
def test_repeatable_with_a_workspace(xs, B, H, Nq, Nk, d):
    """Bit for bit the same from launch to launch, and within the bound of the reference on sampled rows."""
    q, k, v, lam, w = inputs(B, H, H, Nq, Nk, d, seed=5)
    ws = workspace()
    outs = []
    for _ in range(6):
        o = torch.full_like(q, math.nan)
        xs.diff_attn(q, k, v, o, lam, norm_weight=w, workspace=ws)
        outs.append(o)
    done(xs, ws)
    assert all(torch.equal(outs[0], o) for o in outs[1:])
    rows = torch.unique(torch.tensor([0, Nq // 3, Nq // 2, Nq - 1], device="cuda"))
    check(outs[0][:, :, rows], reference(q, k, v, lam, weight=w, rows=rows), "rows")


def test_workspace_that_is_just_enough_and_one_that_is_not(xs):
    """A canary behind exactly the reported bytes stays; a smaller workspace falls back to whole units."""
    for d in (64, 128, 256):
        q, k, v, lam, w = inputs(1, 6, 6, 900, 1100, d, seed=3)
        full = xs.alloc_diff_workspace(1, 6, 900, 1100, d, norm=True)
        buf = torch.zeros(full.numel() + 4096, dtype=torch.uint8, device="cuda")
        buf[full.numel():] = 77
        place = 128 * 256 * 4 if d == 256 else 0   # of a CTA: one, some, and almost a second one
        for n in (full.numel(), 16384 + place, 16384 + 2 * place - 256 * (d == 256), 16384 + 42 * place):
            o = torch.full_like(q, math.nan)
            xs.diff_attn(q, k, v, o, lam, norm_weight=w, workspace=buf[:n])
            done(xs, buf)
            check(o, reference(q, k, v, lam, weight=w), f"o with {n} bytes")
        assert bool((buf[full.numel():] == 77).all())


def test_a_small_workspace_does_not_slow_a_call_without_a_norm(xs):
    """d = 256, no norm: with places for a few SMs the call runs as without a workspace (bit for bit the same
    result), with a place for every unit as with the whole workspace."""
    B, H, Nq, Nk, d = 1, 12, 1024, 1024, 256
    q, k, v, lam, w = inputs(B, H, H, Nq, Nk, d, seed=3)
    full = xs.alloc_diff_workspace(B, H, Nq, Nk, d)
    buf = torch.zeros(full.numel() + 4096, dtype=torch.uint8, device="cuda")
    buf[full.numel():] = 77
    ref, outs = reference(q, k, v, lam), {}
    for places in (0, 1, 2, 40, 47, 96, "all"):
        n = full.numel() if places == "all" else 16384 + places * 128 * 256 * 4
        o = torch.full_like(q, math.nan)
        xs.diff_attn(q, k, v, o, lam, workspace=buf[:n] if places else None)
        done(xs, buf)
        check(o, ref, f"{places} places")
        outs[places] = o
    for places in (1, 2, 40, 47):
        assert torch.equal(outs[places], outs[0]), places
    assert torch.equal(outs[96], outs["all"]) and not torch.equal(outs["all"], outs[0])
    assert bool((buf[full.numel():] == 77).all())


@pytest.mark.parametrize("d1,d2", [(128, 64), (256, 256)])
def test_two_graphs_one_workspace_and_streams(xs, d1, d2):
    """Two captured calls of different shapes share a workspace, replayed one after the other; two
    streams with a workspace each run at once."""
    cases = [inputs(1, 3, 3, 300, 2000, d1, seed=1), inputs(2, 2, 2, 1, 5000, d2, seed=2)]
    ws = [workspace(), workspace()]
    outs = [torch.empty_like(c[0]) for c in cases]
    refs = [reference(*c[:4], weight=c[4]) for c in cases]
    for c, o in zip(cases, outs):
        xs.diff_attn(*c[:3], o, c[3], norm_weight=c[4], workspace=ws[0])   # loads the code before the capture
    torch.cuda.synchronize()
    graphs = []
    for c, o in zip(cases, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            xs.diff_attn(*c[:3], o, c[3], norm_weight=c[4], workspace=ws[0])
        graphs.append(g)
    for _ in range(3):
        for o in outs:
            o.fill_(math.nan)
        for g in graphs:
            g.replay()
        done(xs, ws[0])
        for o, r in zip(outs, refs):
            check(o, r, "replay")
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for o in outs:
        o.fill_(math.nan)
    torch.cuda.synchronize()
    for _ in range(5):
        for i, (c, o) in enumerate(zip(cases, outs)):
            xs.diff_attn(*c[:3], o, c[3], norm_weight=c[4], workspace=ws[i], stream=streams[i])
    done(xs, ws[1])
    for o, r in zip(outs, refs):
        check(o, r, "streams")


@pytest.mark.parametrize("d", [64, 128, 256])
def test_rope_then_attention_into_shards(xs, d):
    """The two operators as a layer uses them: a projection's output to rotated, normalised q and k,
    then attention over them into the shards (padded batch), captured as one graph."""
    B, N, H, Hk, P = 2, 296, 4, 2, 8
    g = torch.Generator(device="cuda").manual_seed(d)
    x = torch.randn(B, N, H + 2 * Hk, d, generator=g, device="cuda").to(BF)
    wq, wk, wo = (1 + 0.1 * torch.randn(d, generator=g, device="cuda") for _ in range(3))
    lam = torch.rand(H, generator=g, device="cuda")
    n = torch.arange(N, device="cuda")
    pos = torch.stack([n // 64, n // 8 % 8, n % 8], 1).to(torch.int32)
    axes = (d // 4, 3 * d // 8, 3 * d // 8)
    lens = (N, 170)
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q, k, v = (torch.empty(B, h, N, d, dtype=BF, device="cuda") for h in (H, Hk, Hk))
    shards = xs.alloc_shards(B, N, H, d, P)
    ws = xs.alloc_diff_workspace(B, H, N, N, d, norm=True)

    def layer():
        xs.qkv_rope(x[:, :, :H], x[:, :, H:H + Hk], x[:, :, H + Hk:], q, k, v, pos, axes, q_weight=wq, k_weight=wk)
        xs.diff_attn_fused(q, k, v, shards, lam, kv_len=kv_len, norm_weight=wo, workspace=ws)

    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    x.copy_(torch.randn(x.shape, generator=g, device="cuda").to(BF))
    graph.replay()
    done(xs, ws)
    # q, k and v as the formula gives them, rounded to bf16 as the layer does: one step of a bf16 apart at most.
    y = x.double()
    ang = pos.double()[:, torch.repeat_interleave(torch.arange(3, device="cuda"), torch.tensor([a // 2 for a in axes], device="cuda"))]
    ang = ang * torch.tensor([1e4 ** (-2 * i / a) for a in axes for i in range(a // 2)], device="cuda", dtype=torch.float64)
    for got, part, weight in ((q, y[:, :, :H], wq), (k, y[:, :, H:H + Hk], wk)):
        part = part / (part.square().mean(-1, keepdim=True) + 1e-6).sqrt() * weight.double()
        z = torch.view_as_complex(part.unflatten(-1, (-1, 2)).contiguous()) * torch.polar(torch.ones_like(ang), ang)[None, :, None]
        want = torch.view_as_real(z).flatten(-2).transpose(1, 2)
        assert ((got.double() - want).abs() <= U * want.abs() + 2.0 ** -18 * z.abs().repeat_interleave(2, -1).transpose(1, 2)).all()
    assert torch.equal(v, x[:, :, H + Hk:].transpose(1, 2))
    check(torch.cat(shards, 1).transpose(1, 2), reference(q, k, v, lam, lens=lens, weight=wo), "shards")


def test_binding_refusals(xs):
    q, k, v, lam, w = inputs(1, 4, 2, 16, 20, 64, seed=0)
    o = torch.empty_like(q)
    ok = dict(q=q, k=k, v=v, o=o, lam=lam)
    xs.diff_attn(**ok)
    for bad in (dict(k=k.float()), dict(v=v[:, :, :3]), dict(lam=lam[:2]), dict(lam=lam.double()), dict(o=o[:, :, :4]),
                dict(q=q.transpose(2, 3).contiguous().transpose(2, 3)), dict(norm_weight=w.to(BF)), dict(norm_weight=w[:32]),
                dict(kv_len=torch.zeros(2, dtype=torch.int32, device="cuda")), dict(kv_len=torch.zeros(1, dtype=torch.int64, device="cuda")),
                dict(workspace=torch.zeros(1 << 20, dtype=torch.uint8)), dict(lam=lam.cpu())):
        with pytest.raises(ValueError):
            xs.diff_attn(**{**ok, **bad})
    for bad in (dict(scale=-1.0), dict(out_scale=math.inf), dict(k=k[:, :1].expand(-1, 3, -1, -1).contiguous(), v=v[:, :1].expand(-1, 3, -1, -1).contiguous()),
                dict(k=k[:, :, :1].expand(-1, -1, 20, -1))):
        with pytest.raises(xs.XsError):
            xs.diff_attn(**{**ok, **bad})
    with pytest.raises(ValueError):
        xs.diff_attn_fused(q, k, v, xs.alloc_shards(1, 16, 4, 64, 2)[:1], lam)
    with pytest.raises(ValueError):
        xs.diff_attn_fused(q, k, v, xs.alloc_shards(1, 16, 4, 64, 2) * 4 + [o], lam)
    done(xs)


def test_refusal_of_a_norm_without_a_workspace(xs):
    """At d = 256 the refusal names the workspace; other invalid arguments do not."""
    q, k, v, lam, w = inputs(1, 2, 2, 20, 30, 256, seed=0)
    o, shards = torch.empty_like(q), xs.alloc_shards(1, 20, 2, 256, 2)
    small = workspace(16384 + 24 * 1024 - 256)
    for ws in (None, small):
        with pytest.raises(xs.XsError, match="needs a workspace") as e:
            xs.diff_attn(q, k, v, o, lam, norm_weight=w, workspace=ws)
        assert e.value.status == xs.ERR_INVALID
        with pytest.raises(xs.XsError, match="needs a workspace"):
            xs.diff_attn_fused(q, k, v, shards, lam, norm_weight=w, workspace=ws)
    for bad in (dict(norm_weight=w, workspace=workspace(16384 + 24 * 1024)), dict()):
        with pytest.raises(xs.XsError) as e:
            xs.diff_attn(q, k, v, o, lam, scale=-1.0, **bad)
        assert "workspace" not in str(e.value)
    done(xs)
