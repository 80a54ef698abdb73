"""Plain 64-bit forms of the quantised key/value cache and of shared-prefix attention, for the tests."""
import math

import torch

#: What the codes 0..126 of e4m3 stand for (sign 0, 4 bits of exponent, 3 of fraction), in order.
E4M3 = torch.tensor([(c & 7) / 8 * 2.0 ** -6 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7) for c in range(127)],
                    dtype=torch.float64)


def to_codes(x):
    """(codes uint8, scale bytes uint8) of rows x (any type, on the CPU), from the definition."""
    x = x.double()
    big = x.abs().amax(-1)
    bad = ~torch.isfinite(x).all(-1)
    ok = torch.where(bad, torch.zeros_like(big), big)
    e = torch.zeros(big.shape, dtype=torch.int64)
    some = ok > 0
    e[some] = torch.ceil(torch.log2(ok[some] / 448) - 1e-9).long()
    e[some & (ok > 448 * torch.pow(2.0, e.double()))] += 1          # (should log2 have been off)
    e = e.clamp(-120, 119)
    y = x * torch.pow(2.0, -e.double())[..., None]
    size = y.abs().clamp_max(448.0).nan_to_num(0.0)
    hi = torch.searchsorted(E4M3, size).clamp_max(126)                # first code at or above
    lo = (hi - 1).clamp_min(0)
    up, down = E4M3[hi] - size, size - E4M3[lo]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)) | (hi == 0), hi, lo)
    code = code + 128 * torch.signbit(x).long()
    code[bad] = 127
    byte = e + 127
    byte[bad] = 255
    return code.to(torch.uint8), byte.to(torch.uint8)


def values(codes, bytes_):
    """What codes and scale bytes stand for, in 64 bits."""
    c = codes.long()
    table = E4M3.to(c.device)
    size = torch.where((c & 127) == 127, torch.full((), math.nan, dtype=torch.float64, device=c.device), table[(c & 127).clamp_max(126)])
    scale = torch.where(bytes_ == 255, torch.full((), math.nan, dtype=torch.float64, device=c.device),
                        torch.pow(2.0, bytes_.double() - 127))
    return torch.where(c >= 128, -size, size) * scale[..., None]


def prefix_formula(q, prefix, own, lens, scale):
    """q [B, H, Nq, d], prefix (k, v) [Hk, Np, d], own (k, v) [B, Hk, Nk, d], all in 64 bits; lens a list.
    (the result, the same mean of |v|), [B, H, Nq, d] both; rows without keys are zeros."""
    B, H, Nq, d = q.shape
    out, size = torch.zeros_like(q), torch.zeros_like(q)
    Hk = prefix[0].shape[0]
    for b in range(B):
        for h in range(H):
            hk = h * Hk // H
            k = torch.cat([prefix[0][hk], own[0][b, hk, :lens[b]]])
            v = torch.cat([prefix[1][hk], own[1][b, hk, :lens[b]]])
            if k.shape[0] == 0:
                continue
            w = torch.softmax(q[b, h] @ k.T * scale, -1)
            out[b, h], size[b, h] = w @ v, w @ v.abs()
    return out, size
