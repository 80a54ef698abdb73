"""Cases of the quantised key/value cache and of attention over a shared prefix, with their plain forms.

write   keys and values [B, H_kv, N, d] go into the pages of a cache in e4m3, every row of d values
        with a power of two as its scale: 2^e with the least e for which the row's largest magnitude
        is at most 448 * 2^e. Token n of request b stands at place start[b] + n of the request's pages;
        tokens from lens[b] on are not stored.
read    the values that the cache stands for, code * 2^e, of consecutive places of the requests' pages.
attn    softmax(q [prefix | own]^T / sqrt(d)) [prefix | own] for a batch of requests: the keys and
        values of the prefix are the same for all of them, the own ones are each request's, of which
        the first kv_len[b] count. Both parts lie in bf16 tensors or in pages of one cache.
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
        # The new token of each of 8 requests, as a single-token step stores it.
        _rows("write one token", "write", B=8, N=1, Hk=8, d=128, page=64, past=1000),
        # A ragged batch out of an fp32 projection, heads of 80 columns.
        _rows("write ragged fp32", "write", B=3, N=1237, Hk=5, d=80, page=32, past=77, ragged=True, type="fp32"),
        # An image's tokens, every head.
        _rows("write image", "write", B=1, N=4096, Hk=24, d=128, page=128),
        # The history of three requests of different lengths, back in fp32.
        _rows("read ragged fp32", "read", B=3, N=1101, Hk=4, d=64, page=16, past=40, ragged=True, type="fp32"),
        # 16K tokens at head dimension 256, in fp16.
        _rows("read wide fp16", "read", B=1, N=16384, Hk=12, d=256, page=64, type="fp16"),
        # The keys and values of a 64K sequence: HBM traffic is all of it.
        _rows("read video", "read", B=1, N=65536, Hk=24, d=128, page=128),
        # The smallest workload of this repository, two requests behind a short common text.
        _attn("attn small", B=2, H=4, d=64, Nq=256, Np=77, Nk=256),
        # One new token for each of 8 requests, the prompt and their own tokens in the cache; shared k/v heads.
        _attn("attn one token", B=8, H=24, Hk=8, d=128, Nq=1, Np=16384, Nk=1024, prefix="cache", owned="cache", page=64, ragged=True),
        # One new token for each of 16 requests behind a 64K history, every head its own keys.
        _attn("attn long history", B=16, H=24, d=128, Nq=1, Np=65536, Nk=256, prefix="cache", owned="cache", page=128, ragged=True),
        # Padded requests behind common conditioning, the last one with no keys of its own; odd sizes.
        _attn("attn padded d64", B=3, H=8, Hk=4, d=64, Nq=777, Np=1101, Nk=777, ragged=True),
        # Four candidates of an image behind a reference image in the cache, stored into 8 sequence shards.
        _attn("attn image", B=4, H=24, d=128, Nq=4096, Np=4096, Nk=4096, prefix="cache", page=128, P=8),
        # Two continuations of a video: a frame's tokens against 32K tokens of history and their own: the largest.
        _attn("attn video", B=2, H=24, d=128, Nq=4096, Np=32768, Nk=4096, prefix="cache", page=128),
    ]


def _rows(name, op, **kw):
    return {"name": name, "op": op, "past": 0, "ragged": False, "type": "bf16", **kw}


def _attn(name, **kw):
    c = {"name": name, "op": "attn", "Hk": kw.get("H"), "prefix": "bf16", "owned": "bf16", "page": 64, "ragged": False, "P": 0}
    c.update(kw)
    return c


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    page = rng.choice([16, 32, 64, 128])
    if rng.random() < 0.4:
        d = rng.choice([64, 80, 96, 128, 128, 256])
        B, Hk = rng.randint(1, 8), rng.randint(1, 24)
        while True:
            N = _log_int(rng, 1, 65536)
            if B * N * Hk * d <= 65536 * 24 * 128:
                break
        c = _rows("", rng.choice(["write", "read"]), B=B, N=N, Hk=Hk, d=d, page=page, past=rng.choice([0, rng.randint(1, 4096)]),
                  ragged=rng.random() < 0.4, type=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    else:
        d = rng.choice([64, 128, 128])
        B, Hk = rng.choice([1, 2, 3, 4, 8, 16, 32]), rng.randint(1, 8)
        H = Hk * rng.randint(1, 4)
        while True:
            Nq = _log_int(rng, 1, 4096) if rng.random() < 0.6 else rng.randint(1, 4)
            Np, Nk = _log_int(rng, 1, 65536), _log_int(rng, 1, 4096)
            if 4 * B * H * Nq * (Np + Nk) * d <= 2.5e12 and Hk * (Np + B * Nk) * d <= 65536 * 24 * 128:
                break
        P = rng.choice([0, 0, 0, 2, 5, 8])
        if P:
            Nq = (Nq + P - 1) // P * P
        c = _attn("", B=B, H=H, Hk=Hk, d=d, Nq=Nq, Np=Np, Nk=Nk, prefix=rng.choice(["bf16", "cache", "cache"]),
                  owned=rng.choice(["bf16", "cache"]), page=page, ragged=rng.random() < 0.5, P=P)
    del c["name"]
    return c


DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _lens(c):
    """Tokens (or own keys) of each request: of a ragged batch of several the last one has none."""
    n, B = c["N"] if "N" in c else c["Nk"], c["B"]
    if not c["ragged"]:
        return [n] * B
    return [max(0, n - b * n // max(1, B - 1)) if B > 1 else (n + 1) // 2 for b in range(B)]


def _to_rows(x):
    """(codes in e4m3, exponents + 127 in 8 bits) of rows x."""
    big = x.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(big)                                   # big = m 2^e with m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(big == 0, torch.zeros_like(e), e - 9 + (m > 0.875).to(e.dtype))
    return (x * _power(127 - e)).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8).squeeze(-1)


def _power(e):
    """2^(e - 127) in fp32, for e in [1, 254]."""
    return (e.int() << 23).view(torch.float32)


def _from_pages(codes, scales, pages, at, n):
    """Rows of places [at, at + n) of a list of pages [m], fp32 [H_kv, n, d]."""
    x = codes.view(torch.uint8)[pages].view(torch.float8_e4m3fn).float()             # [m, H_kv, page, d]
    x = x * _power(scales[pages])[..., None]
    return x.transpose(0, 1).flatten(1, 2)[:, at:at + n]


def _empty_cache(n_pages, c, dev):
    shape = (n_pages, c["Hk"], c["page"], c["d"])
    codes = [torch.zeros(shape, device=dev, dtype=torch.uint8).view(torch.float8_e4m3fn) for _ in range(2)]
    return codes + [torch.full(shape[:3], 127, device=dev, dtype=torch.uint8) for _ in range(2)]


def _full_cache(n_pages, c, normal):
    """A cache whose every page holds normal values, in the order (k, v, k_scale, v_scale)."""
    got = [_to_rows(normal(n_pages, c["Hk"], c["page"], c["d"]).mul_(1 + i)) for i in range(2)]
    return [got[0][0], got[1][0], got[0][1], got[1][1]]


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    B, Hk, d, page = c["B"], c["Hk"], c["d"], c["page"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    def ints(v):
        return torch.tensor(v, device=dev, dtype=torch.int32)

    def page_lists(*counts):
        """Lists of so many pages each, all different, scattered over the cache."""
        every = torch.randperm(sum(counts) + 3, generator=g, device=dev).to(torch.int32)
        return every[:sum(counts)].split(list(counts)), sum(counts) + 3

    s = {"case": c}
    if c["op"] != "attn":
        N, type_ = c["N"], DTYPES[c["type"]]
        each = (c["past"] + N + page - 1) // page
        lists, n_pages = page_lists(*[each] * B)
        s["pages"] = torch.stack(lists)
        s["start"] = ints([max(0, c["past"] - 3 * b) for b in range(B)])     # tokens that stand before these
        s["lens"] = ints(_lens(c)) if c["ragged"] else None
        if c["op"] == "write":
            s["x"] = (normal(B, N, 2 * Hk, d) * torch.exp(normal(B, N, 2 * Hk, 1))).to(type_)   # a projection's k and v heads
            s["cache"] = _empty_cache(n_pages, c, dev)
        else:
            s["cache"] = _full_cache(n_pages, c, normal)
            s["out"] = [torch.zeros((B, Hk, N, d), device=dev, dtype=type_) for _ in range(2)]
        return s
    H, Nq, Np, Nk = c["H"], c["Nq"], c["Np"], c["Nk"]
    s["q"] = (normal(B, H, Nq, d) * 2).bfloat16()
    s["len"] = ints(_lens(c)) if c["ragged"] else None
    counts = [-(-Np // page) if c["prefix"] == "cache" else 0] + [-(-Nk // page) if c["owned"] == "cache" else 0] * B
    if sum(counts):
        lists, n_pages = page_lists(*counts)
        s["cache"] = _full_cache(n_pages, c, normal)
    if c["prefix"] == "cache":
        s["prefix_pages"] = lists[0].contiguous()
    else:
        s["prefix"] = [normal(Hk, Np, d).bfloat16() for _ in range(2)]
    if c["owned"] == "cache":
        s["pages"] = torch.stack(lists[1:])
    else:
        s["own"] = [normal(B, Hk, Nk, d).bfloat16() for _ in range(2)]
    if c["P"]:
        s["out"] = [torch.empty((B, Nq // c["P"], H, d), device=dev, dtype=torch.bfloat16) for _ in range(c["P"])]
    else:
        s["out"] = torch.empty((B, H, Nq, d), device=dev, dtype=torch.bfloat16)
    # The workspace that a serving program keeps for all its layers: partial results, and the keys and values in bf16.
    s["workspace"] = torch.zeros((128 << 20) + 4 * Hk * d * (Np + 256 + B * (Nk + 256)), device=dev, dtype=torch.uint8)
    return s


def run(state):
    c = state["case"]
    if own:
        return {"write": _write_own, "read": _read_own, "attn": _attn_own}[c["op"]](state)
    return {"write": _write_plain, "read": _read_plain, "attn": _attn_plain}[c["op"]](state)


def _kv(s):
    """k and v [B, H_kv, N, d] of the projection's output."""
    x, Hk = s["x"].transpose(1, 2), s["case"]["Hk"]
    return x[:, :Hk], x[:, Hk:]


def _write_own(s):
    from all_layout_gb300 import xs
    k, v = _kv(s)
    xs.cache_write(k, v, xs.KVCache(*s["cache"]), s["pages"], start=s["start"], lens=s["lens"])
    return s["cache"]


def _read_own(s):
    from all_layout_gb300 import xs
    k, v = s["out"]
    xs.cache_read(xs.KVCache(*s["cache"]), s["pages"], k, v, start=s["start"], lens=s["lens"])
    return k, v


def _attn_own(s):
    from all_layout_gb300 import xs
    c = s["case"]
    kw = {"kv_len": s["len"], "workspace": s["workspace"]}
    if "cache" in s:
        kw["cache"] = xs.KVCache(*s["cache"])
    if c["prefix"] == "cache":
        kw.update(prefix_pages=s["prefix_pages"], prefix_len=c["Np"])
    else:
        kw.update(prefix_k=s["prefix"][0], prefix_v=s["prefix"][1])
    if c["owned"] == "cache":
        kw.update(pages=s["pages"], max_len=c["Nk"])
    else:
        kw.update(k=s["own"][0], v=s["own"][1])
    (xs.prefix_attn_fused if c["P"] else xs.prefix_attn)(s["q"], s["out"], **kw)
    return s["out"]


def _places(s):
    """(page, row in the page, whether it counts) of every token, [B, N] each."""
    c, dev = s["case"], s["pages"].device
    n = torch.arange(c["N"], device=dev)
    at = s["start"].long()[:, None] + n
    live = n < (s["lens"].long()[:, None] if s["lens"] is not None else c["N"] + 0 * at)
    return s["pages"].long().gather(1, at // c["page"]), at % c["page"], live


def _write_plain(s):
    page, row, live = _places(s)
    page, row = page[live], row[live]
    k, v, k_scale, v_scale = s["cache"]
    for x, codes, scales in zip(_kv(s), (k, v), (k_scale, v_scale)):
        got, e = _to_rows(x.float().transpose(1, 2)[live])     # [tokens, H_kv, d]
        codes.view(torch.uint8)[page, :, row] = got.view(torch.uint8)
        scales[page, :, row] = e
    return s["cache"]


def _read_plain(s):
    page, row, live = _places(s)
    k, v, k_scale, v_scale = s["cache"]
    for out, codes, scales in zip(s["out"], (k, v), (k_scale, v_scale)):
        x = codes.view(torch.uint8)[page, :, row].view(torch.float8_e4m3fn).float()           # [B, N, H_kv, d]
        x = x * _power(scales[page, :, row])[..., None]
        out.copy_(torch.where(live[:, None, :, None], x.transpose(1, 2).to(out.dtype), out))
    return tuple(s["out"])


def _parts(s):
    """Prefix keys and values [H_kv, Np, d] and own ones [B, H_kv, Nk, d], fp32."""
    c = s["case"]
    if c["prefix"] == "cache":
        prefix = [_from_pages(s["cache"][i], s["cache"][2 + i], s["prefix_pages"], 0, c["Np"]) for i in range(2)]
    else:
        prefix = [x.float() for x in s["prefix"]]
    if c["owned"] == "cache":
        mine = [_from_pages(s["cache"][i], s["cache"][2 + i], s["pages"].flatten(), 0, s["pages"].numel() * c["page"])
                .unflatten(1, (c["B"], -1))[:, :, :c["Nk"]].transpose(0, 1) for i in range(2)]
    else:
        mine = [x.float() for x in s["own"]]
    return prefix, mine


def _attn_plain(s):
    c = s["case"]
    B, H, Hk, d, Nq, Np, Nk = (c[x] for x in ("B", "H", "Hk", "d", "Nq", "Np", "Nk"))
    (pk, pv), (k, v) = _parts(s)
    dead = None
    if s["len"] is not None:
        gone = torch.arange(Nk, device=k.device) >= s["len"][:, None]               # [B, Nk]
        dead = gone[:, None, None, None]
        v = v.masked_fill(gone[:, None, :, None], 0.0)
    q = s["q"].float().unflatten(1, (Hk, H // Hk)) * d ** -0.5                      # [B, H_kv, group, Nq, d]
    out = torch.empty((B, Hk, H // Hk, Nq, d), device=q.device)
    step = max(1, BLOCK // (B * H * (Np + Nk)))
    for i in range(0, Nq, step):   # blocks of queries, so that the scores fit the memory
        rows = q[:, :, :, i:i + step]
        flat = rows.transpose(0, 1).flatten(1, 3)                                   # [H_kv, all rows, d]
        a = (flat @ pk.transpose(1, 2)).view(Hk, B, H // Hk, -1, Np).transpose(0, 1)
        b = (rows.flatten(2, 3) @ k.transpose(2, 3)).view(B, Hk, H // Hk, -1, Nk)
        if dead is not None:
            b = b.masked_fill_(dead, -math.inf)
        m = torch.maximum(a.amax(-1, keepdim=True), b.amax(-1, keepdim=True))
        a, b = a.sub_(m).exp_(), b.sub_(m).exp_()
        total = a.sum(-1, keepdim=True) + b.sum(-1, keepdim=True)
        x = (a.transpose(0, 1).flatten(1, 3) @ pv).view(Hk, B, H // Hk, -1, d).transpose(0, 1)
        out[:, :, :, i:i + step] = (x + (b.flatten(2, 3) @ v).view(B, Hk, H // Hk, -1, d)) / total
        del a, b, x
    out = out.flatten(1, 2).bfloat16()
    if c["P"]:
        return [t.contiguous() for t in out.transpose(1, 2).chunk(c["P"], 1)]
    return out


def work(case):
    c = case
    B, Hk, d = c["B"], c["Hk"], c["d"]
    if c["op"] != "attn":
        rows = 2 * Hk * sum(_lens(c))
        return {"bytes": rows * (d * {"bf16": 2, "fp16": 2, "fp32": 4}[c["type"]] + d + 1), "flops": 2 * rows * d}
    H, Nq, own_keys = c["H"], c["Nq"], sum(_lens(c))
    row = {"bf16": 2 * d, "cache": d + 1}
    return {"bytes": 4 * B * H * Nq * d + 2 * Hk * (c["Np"] * row[c["prefix"]] + own_keys * row[c["owned"]]),
            "flops": 4 * H * Nq * d * (B * c["Np"] + own_keys)}


def exact(case, seed):
    c = case
    if c["op"] == "attn" and work(c)["flops"] > EXACT_FLOPS:
        return None
    s = prepare(case, seed)
    return {"write": _write_exact, "read": _read_exact, "attn": _attn_exact}[c["op"]](s)


def _value(codes, scales):
    """What codes stand for, from the bits of the format: sign, 4 bits of exponent, 3 of fraction."""
    bits = codes.view(torch.uint8).long()
    e, f = bits >> 3 & 15, (bits & 7).double()
    size = torch.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * torch.exp2((e - 7).double()))
    return torch.where(bits >= 128, -size, size) * torch.exp2(scales.double() - 127)[..., None]


def _tokens(s, b):
    """Pages and rows of request b's tokens, token by token."""
    c = s["case"]
    at = s["start"][b].item() + torch.arange(_lens(c)[b], device=s["pages"].device)
    return s["pages"][b].long()[torch.div(at, c["page"], rounding_mode="floor")], at.remainder(c["page"])


def _write_exact(s):
    """The scaled values before they are rounded to e4m3; the exponents have no such value."""
    c = s["case"]
    out = []
    for i, x in enumerate(_kv(s)):
        y = s["cache"][i].view(torch.uint8).double()    # an empty cache's zeros
        for b in range(c["B"]):
            page, row = _tokens(s, b)
            v = x[b, :, :page.numel()].double()
            e = torch.ceil(torch.log2(v.abs().amax(-1, keepdim=True) / 448) - 1e-9)   # 448 * 2^e itself still fits
            y[page, :, row] = (v / torch.exp2(e)).transpose(0, 1)
        out.append(y)
    return out + [None, None]


def _read_exact(s):
    c = s["case"]
    out = []
    for i in range(2):
        y = torch.zeros((c["B"], c["Hk"], c["N"], c["d"]), device=s["pages"].device, dtype=torch.float32 if c["N"] > 16384 else torch.float64)
        for b in range(c["B"]):
            page, row = _tokens(s, b)
            for h in range(c["Hk"]):
                y[b, h, :page.numel()] = _value(s["cache"][i][:, h].view(torch.uint8)[page, row], s["cache"][2 + i][:, h][page, row])
        out.append(y)
    return tuple(out)


def _attn_exact(s):
    """Request by request and head by head over all keys that it sees, weights from the logarithm of their sum, in 64 bits."""
    c = s["case"]
    B, H, Hk, d, Nq, page = (c[x] for x in ("B", "H", "Hk", "d", "Nq", "page"))
    y = torch.zeros((B, Nq, H, d), device=s["q"].device, dtype=torch.float64)

    def paged(i, pages, h, n):
        pages = pages.long()
        return _value(s["cache"][i][:, h].view(torch.uint8)[pages], s["cache"][2 + i][:, h][pages]).flatten(0, 1)[:n]

    for h in range(Hk):
        prefix = [paged(i, s["prefix_pages"], h, c["Np"]) if c["prefix"] == "cache" else s["prefix"][i][h].double() for i in range(2)]
        for b, n in enumerate(_lens(c)):
            mine = [paged(i, s["pages"][b], h, n) if c["owned"] == "cache" else s["own"][i][b, h, :n].double() for i in range(2)]
            k, v = (torch.cat(x) for x in zip(prefix, mine))
            for j in range(h * H // Hk, (h + 1) * H // Hk):
                for i in range(0, Nq, 4096):
                    t = s["q"][b, j, i:i + 4096].double() @ k.T / math.sqrt(d)
                    t -= torch.logsumexp(t, 1, keepdim=True)
                    y[b, i:i + 4096, j] = t.exp_() @ v
    if c["P"]:
        R = Nq // c["P"]
        return [y[:, p * R:(p + 1) * R].contiguous() for p in range(c["P"])]
    return y.transpose(1, 2).contiguous()
