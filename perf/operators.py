"""Cases of the rotary-position and the differential-attention operators, with their plain forms.

rope  q, k and v of a projection, token-major [B, N, heads, d], become the head-major tensors
      [B, heads, N, d] that attention reads: q and k RMS-normalised per head (optional) and rotated
      by the token's position along several axes (time, height, width), v moved as it is.
diff  o = norm((softmax(q1 k1^T / sqrt(d/2)) - lambda softmax(q2 k2^T / sqrt(d/2))) v) * out_scale,
      where q = [q1 | q2] and k = [k1 | k2] share the d columns of a head; written head-major or
      into P sequence shards; keys behind a batch entry's length do not count.
"""
import math

import torch

own = False

#: Elements of one block of scores in the plain form (4 GB of fp32): longer ones go block by block.
BLOCK = 1 << 30
#: Flops that exact() does in 64 bits within about 20 seconds.
EXACT_FLOPS = 1.1e13


def listed():
    return [
        # The smallest workload of this repository: launch latency is all of it.
        _rope("rope small", B=1, N=256, H=4, d=64, axes="16,24,24"),
        # One new token for each of 8 requests, head dimension 128: the single-token form.
        _rope("rope one token", B=8, N=1, H=24, d=128, axes="16,56,56", norm=True),
        # Image-DiT with normalised q and k, adjacent pairs.
        _rope("rope image", B=1, N=4096, H=24, d=128, axes="16,56,56", norm=True),
        # A ragged batch out of an fp32 projection; fewer k/v heads; first half pairs with second half.
        _rope("rope ragged fp32", B=3, N=1237, H=15, Hk=5, d=80, axes="16,32,32", src="fp32", adjacent=False),
        # Head dimension 256 in fp16, half of the columns rotated, the others passed on.
        _rope("rope wide fp16", B=1, N=16384, H=12, d=256, axes="32,48,48", src="fp16", dst="fp16", adjacent=False, norm=True),
        # Video-DiT, the largest sequence here: HBM traffic is all of it.
        _rope("rope video", B=1, N=65536, H=24, d=128, axes="44,42,42", norm=True),
        # One query token against a long sequence of keys, 4 requests.
        _diff("diff one token", B=4, H=24, d=128, Nq=1, Nk=16384, norm=True),
        # Padded conditioning of three requests, the last one with none; odd sizes, shared k/v heads.
        _diff("diff padded d64", B=3, H=8, Hk=4, d=64, Nq=777, Nk=1101, ragged=True, norm=True),
        # Image-DiT, stored into its 8 sequence shards.
        _diff("diff image", B=1, H=24, d=128, Nq=4096, Nk=4096, P=8, norm=True),
        # Head dimension 256 (two maps of 128).
        _diff("diff wide", B=1, H=12, d=256, Nq=4096, Nk=4096, norm=True),
        # A 16K sequence, every head, head-major output.
        _diff("diff 16k", B=1, H=24, d=128, Nq=16384, Nk=16384),
        # One of eight ranks' share of the heads of video-DiT, stored into 8 shards: the largest.
        _diff("diff video share", B=1, H=3, d=128, Nq=65536, Nk=65536, P=8, norm=True),
    ]


def _rope(name, **kw):
    c = {"name": name, "op": "rope", "Hk": kw.get("H"), "src": "bf16", "dst": "bf16", "adjacent": True, "norm": False}
    c.update(kw)
    return c


def _diff(name, **kw):
    c = {"name": name, "op": "diff", "Hk": kw.get("H"), "P": 0, "ragged": False, "norm": False}
    c.update(kw)
    return c


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    B = rng.randint(1, 4)
    Hk = rng.randint(1, 8)
    H = Hk * rng.randint(1, 3)
    if rng.random() < 0.45:
        d = rng.choice([64, 80, 96, 128, 256])
        while True:
            N = _log_int(rng, 1, 65536)
            if B * N * (H + 2 * Hk) * d <= 65536 * 72 * 128:
                break
        part = rng.choice([d, d, 48])
        first = rng.choice([8, 16])
        second = (part - first) // 4 * 2
        src = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        c = _rope("", B=B, N=N, H=H, Hk=Hk, d=d, axes="%d,%d,%d" % (first, second, part - first - second), src=src,
                  dst=rng.choice(["bf16", src]), adjacent=rng.random() < 0.5, norm=rng.random() < 0.5)
    else:
        d = rng.choice([64, 128, 128, 256])
        while True:
            Nq, Nk = _log_int(rng, 1, 16384), _log_int(rng, 1, 65536)
            if 6 * B * H * Nq * Nk * d <= 5e12:
                break
        P = rng.choice([0, 0, 2, 5, 8])
        if P:
            Nq = (Nq + P - 1) // P * P
        c = _diff("", B=B, H=H, Hk=Hk, d=d, Nq=Nq, Nk=Nk, P=P, ragged=rng.random() < 0.4, norm=rng.random() < 0.6)
    del c["name"]
    return c


DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
THETA = 10000.0
ROPE_EPS, DIFF_EPS = 1e-6, 1e-5
OUT_SCALE = 0.2   # 1 - lambda_init of a deep layer


def _axes(c):
    return tuple(int(x) for x in c["axes"].split(","))


def _lens(c):
    """Keys of each batch entry: a padded batch whose last entry (of several) has none."""
    if not c["ragged"]:
        return [c["Nk"]] * c["B"]
    return [max(0, c["Nk"] - b * c["Nk"] // max(1, c["B"] - 1)) if c["B"] > 1 else (c["Nk"] + 1) // 2 for b in range(c["B"])]


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    B, H, Hk, d = c["B"], c["H"], c["Hk"], c["d"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    if c["op"] == "rope":
        N = c["N"]
        x = normal(B, N, H + 2 * Hk, d).to(DTYPES[c["src"]])   # one projection's output: q, k and v heads of a token
        wide = max(1, math.isqrt(max(1, N // 16)))             # a grid of frames of wide x wide tokens
        n = torch.arange(N, device=dev)
        pos = torch.stack([n // (wide * wide), n // wide % wide, n % wide], 1).to(torch.int32)
        start = torch.randint(0, 4096, (B, 1, 1), generator=g, device=dev, dtype=torch.int32)   # frames before these
        pos = pos[None] + start * torch.tensor([1, 0, 0], device=dev, dtype=torch.int32)
        weights = [(1 + 0.1 * normal(d)) if c["norm"] else None for _ in range(2)]
        out = [torch.empty((B, h, N, d), device=dev, dtype=DTYPES[c["dst"]]) for h in (H, Hk, Hk)]
        return {"case": c, "x": x, "pos": pos.contiguous(), "weights": weights, "out": out}
    Nq, Nk = c["Nq"], c["Nk"]
    q, k, v = normal(B, H, Nq, d).bfloat16(), normal(B, Hk, Nk, d).bfloat16(), normal(B, Hk, Nk, d).bfloat16()
    s = {"case": c, "q": q * 2, "k": k, "v": v, "lam": 0.2 + 0.6 * torch.rand(H, generator=g, device=dev),
         "weight": 1 + 0.1 * normal(d) if c["norm"] else None,
         "len": torch.tensor(_lens(c), device=dev, dtype=torch.int32) if c["ragged"] else None}
    if c["P"]:
        s["out"] = [torch.empty((B, Nq // c["P"], H, d), device=dev, dtype=torch.bfloat16) for _ in range(c["P"])]
    else:
        s["out"] = torch.empty((B, H, Nq, d), device=dev, dtype=torch.bfloat16)
    # The workspace a serving program keeps: zeroed once, enough for any call of this size.
    stage = B * H * Nq * d * 4 if d == 256 and c["norm"] else 0
    s["workspace"] = torch.zeros((64 << 20) + stage, device=dev, dtype=torch.uint8)
    return s


def run(state):
    c = state["case"]
    if c["op"] == "rope":
        return _rope_own(state) if own else _rope_plain(state)
    return _diff_own(state) if own else _diff_plain(state)


def _rope_own(s):
    from all_layout_gb300 import xs
    c, x, (q, k, v) = s["case"], s["x"], s["out"]
    H, Hk = c["H"], c["Hk"]
    xs.qkv_rope(x[:, :, :H], x[:, :, H:H + Hk], x[:, :, H + Hk:], q, k, v, s["pos"], _axes(c), theta=THETA,
                q_weight=s["weights"][0], k_weight=s["weights"][1], eps=ROPE_EPS, interleaved=c["adjacent"])
    return q, k, v


def _diff_own(s):
    from all_layout_gb300 import xs
    c = s["case"]
    call = xs.diff_attn_fused if c["P"] else xs.diff_attn
    call(s["q"], s["k"], s["v"], s["out"], s["lam"], kv_len=s["len"], norm_weight=s["weight"], eps=DIFF_EPS,
         out_scale=OUT_SCALE, workspace=s["workspace"])
    return s["out"]


def _rope_plain(s):
    c, x = s["case"], s["x"]
    H, Hk, axes = c["H"], c["Hk"], _axes(c)
    rot = sum(axes)
    # Angles in 64 bits: a far position times a frequency loses its fraction of a turn in 32.
    freq = torch.cat([THETA ** (-torch.arange(0, a, 2, device=x.device, dtype=torch.float64) / a) for a in axes])
    axis = torch.repeat_interleave(torch.arange(len(axes), device=x.device), torch.tensor([a // 2 for a in axes], device=x.device), output_size=rot // 2)
    angle = s["pos"].double()[..., axis] * freq                        # [B, N, rot / 2]
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]
    out = []
    parts = ((x[:, :, :H], s["weights"][0], True), (x[:, :, H:H + Hk], s["weights"][1], True), (x[:, :, H + Hk:], None, False))
    for y, weight, turned in parts:
        y = y.float()
        if weight is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + ROPE_EPS) * weight
        if turned:
            if c["adjacent"]:
                a, b = y[..., 0:rot:2], y[..., 1:rot:2]
                turn = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
            else:
                a, b = y[..., : rot // 2], y[..., rot // 2: rot]
                turn = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
            y = torch.cat([turn, y[..., rot:]], -1)
        out.append(y.transpose(1, 2).to(DTYPES[c["dst"]]).contiguous())
    return tuple(out)


def _softmax(s, dead):
    if dead is not None:
        s = s.masked_fill_(dead, -math.inf)
    m = s.amax(-1, keepdim=True)
    if dead is not None:
        m = m.masked_fill(m == -math.inf, 0.0)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    if dead is not None:
        total = total.masked_fill(total == 0, 1.0)
    return p.div_(total)


def _diff_plain(s):
    c = s["case"]
    B, H, Hk, d, Nq, Nk = (c[x] for x in ("B", "H", "Hk", "d", "Nq", "Nk"))
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    dead = None
    if s["len"] is not None:
        gone = torch.arange(Nk, device=q.device) >= s["len"][:, None]               # [B, Nk]
        dead = gone[:, None, None]
        v = v.masked_fill(gone[:, None, :, None], 0.0)
    if Hk != H:
        k, v = k.repeat_interleave(H // Hk, 1), v.repeat_interleave(H // Hk, 1)
    half, lam = d // 2, s["lam"][:, None, None]
    k1, k2 = k[..., :half].transpose(2, 3), k[..., half:].transpose(2, 3)
    scale = half ** -0.5
    out = torch.empty((B, H, Nq, d), device=q.device)
    step = max(1, BLOCK // (B * H * Nk))
    for i in range(0, Nq, step):   # blocks of queries, so that the scores fit the memory
        rows = q[:, :, i:i + step]
        a = _softmax((rows[..., :half] * scale) @ k1, dead)
        b = _softmax((rows[..., half:] * scale) @ k2, dead)
        out[:, :, i:i + step] = a.sub_(b.mul_(lam)) @ v
        del a, b
    if s["weight"] is not None:
        out = out * torch.rsqrt(out.square().mean(-1, keepdim=True) + DIFF_EPS) * s["weight"]
    out = (out * OUT_SCALE).bfloat16()
    if c["P"]:
        return [t.contiguous() for t in out.transpose(1, 2).chunk(c["P"], 1)]
    return out


def work(case):
    c = case
    B, H, Hk, d = c["B"], c["H"], c["Hk"], c["d"]
    if c["op"] == "rope":
        size = {"bf16": 2, "fp16": 2, "fp32": 4}
        values = B * c["N"] * (H + 2 * Hk) * d
        return {"bytes": values * (size[c["src"]] + size[c["dst"]]) + 12 * B * c["N"], "flops": 6 * values}
    lens = _lens(c)
    pairs = c["Nq"] * sum(lens) * H
    # Two score maps of d / 2 columns and two products with v of d columns, two flops each.
    return {"bytes": 2 * d * (2 * B * H * c["Nq"] + 2 * Hk * sum(lens)), "flops": 6 * pairs * d}


def exact(case, seed):
    c = case
    if c["op"] == "diff" and work(c)["flops"] > EXACT_FLOPS:
        return None
    s = prepare(case, seed)
    return _rope_exact(s) if c["op"] == "rope" else _diff_exact(s)


def _rope_exact(s):
    """Every pair of columns as a complex number, times exp(i angle), in 64 bits."""
    c, dev = s["case"], s["x"].device
    B, N, H, Hk, d = (c[x] for x in ("B", "N", "H", "Hk", "d"))
    lo, hi, angle, at = [], [], [], 0
    rot = sum(_axes(c))
    for n, a in enumerate(_axes(c)):
        for i in range(a // 2):
            pair = at // 2 + i
            lo.append(2 * pair if c["adjacent"] else pair)
            hi.append(2 * pair + 1 if c["adjacent"] else pair + rot // 2)
            angle.append(s["pos"][:, :, n].double() / THETA ** (2 * i / a))
        at += a
    turn = torch.polar(torch.ones((B, N, rot // 2), device=dev, dtype=torch.float64), torch.stack(angle, -1))
    lo, hi = torch.tensor(lo, device=dev), torch.tensor(hi, device=dev)
    out = []
    for first, heads, weight, turned in ((0, H, s["weights"][0], True), (H, Hk, s["weights"][1], True), (H + Hk, Hk, None, False)):
        y = torch.empty((B, heads, N, d), device=dev, dtype=torch.float64)
        for h in range(heads):
            x = s["x"][:, :, first + h].double()
            if weight is not None:
                x = x / (x.pow(2).sum(-1, keepdim=True) / d + ROPE_EPS).sqrt() * weight.double()
            if turned:
                z = torch.complex(x[..., lo], x[..., hi]) * turn
                x = x.clone()
                x[..., lo], x[..., hi] = z.real, z.imag
            y[:, h] = x
        out.append(y.float() if y.numel() > 1 << 28 else y)
    return tuple(out)


def _diff_exact(s):
    """Head by head over the keys that count, weights from the logarithm of their sum, in 64 bits."""
    c = s["case"]
    B, H, Hk, d, Nq = (c[x] for x in ("B", "H", "Hk", "d", "Nq"))
    half = d // 2
    y = torch.zeros((B, Nq, H, d), device=s["q"].device, dtype=torch.float64)
    for b, n in enumerate(_lens(c)):
        for h in range(H):
            if not n:
                continue
            k, v = (s[x][b, h * Hk // H, :n].double() for x in ("k", "v"))
            for i in range(0, Nq, 4096):
                q = s["q"][b, h, i:i + 4096].double()
                for sign, part in ((1.0, slice(0, half)), (-s["lam"][h].double(), slice(half, d))):
                    t = q[:, part] @ k[:, part].T / math.sqrt(half)
                    t -= torch.logsumexp(t, 1, keepdim=True)
                    y[b, i:i + 4096, h] += sign * (t.exp_() @ v)
    if s["weight"] is not None:
        y = y / (y.pow(2).sum(-1, keepdim=True) / d + DIFF_EPS).sqrt() * s["weight"].double()
    y *= OUT_SCALE
    if c["P"]:
        R = Nq // c["P"]
        return [y[:, p * R:(p + 1) * R].contiguous() for p in range(c["P"])]
    return y.transpose(1, 2).contiguous()
