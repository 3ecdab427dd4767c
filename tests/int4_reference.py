"""Plain implementations of the 4-bit cache and of its attention, on the CPU in
64 bits (the stored bytes: in the fp32 arithmetic that defines them)."""
import math

import torch

B = 16


def quantise(x):
    """Rows [..., d] of 16-bit values -> (codes uint8 [..., d], scales, minima fp16 [..., d / 64])."""
    y = x.float().unflatten(-1, (-1, 64))
    low, high = y.amin(-1), y.amax(-1)
    s, m = ((high - low) / 15.0).half(), low.half()
    bad = ~(torch.isfinite(s) & torch.isfinite(m) & torch.isfinite(y).all(-1))
    s[bad] = float("nan")
    m[bad] = float("nan")
    r = torch.where(s > 0, 1.0 / s.float(), torch.zeros_like(low))
    n = ((y - m.float()[..., None]) * r[..., None]).nan_to_num(0.0).round().clamp(0, 15)
    n[bad] = 0
    return n.flatten(-2).to(torch.uint8), s, m


def pack(n, s, m):
    """Codes [blocks, heads, 16, d] and pairs -> cache bytes [blocks, heads, 9 d]."""
    codes = (n[..., 0::2] | (n[..., 1::2] << 4)).flatten(2)
    # NaN is stored as 0x7fff
    pairs = torch.stack([s, m], -1).contiguous().view(torch.int16)
    pairs = torch.where(torch.isnan(torch.stack([s, m], -1)), torch.full_like(pairs, 0x7FFF), pairs)
    return torch.cat([codes, pairs.contiguous().view(torch.uint8).flatten(2)], -1).contiguous()


def cache_of(x):
    """The cache of rows [blocks, heads, 16, d]."""
    return pack(*quantise(x))


def rows_of(cache, d):
    """Cache bytes [..., 9 d] -> fp64 rows [..., 16, d]."""
    c = cache[..., :8 * d].unflatten(-1, (B, d // 2))
    n = torch.stack([c & 15, c >> 4], -1).flatten(-2).double().unflatten(-1, (-1, 64))
    p = cache[..., 8 * d:].contiguous().view(torch.float16).unflatten(-1, (B, d // 64, 2)).double()
    return (n * p[..., :1] + p[..., 1:]).flatten(-2)


def poison(cache, d, block, row):
    """The pair of a row of a block reads as NaN from now on (every head)."""
    pairs = cache[..., 8 * d:].unflatten(-1, (B, d // 64 * 4))
    pairs[block, :, row, 0::2] = 0xFF
    pairs[block, :, row, 1::2] = 0x7F


def first_key(pos, window, chunk):
    lo = max(0, pos - window + 1) if window else 0
    return max(lo, pos // chunk * chunk) if chunk else lo


def decode(q, kc, vc, tables, lens, scale, window=0, chunk=0):
    """(out, lse) in 64 bits of CPU tensors; q [S, Hq, D]."""
    S, hq, d = q.shape
    hkv = kc.shape[1]
    out = torch.zeros((S, hq, d), dtype=torch.float64)
    lse = torch.full((S, hq), -math.inf, dtype=torch.float64)
    for s in range(S):
        L = int(lens[s])
        if L == 0:
            continue
        lo = first_key(L - 1, window, chunk)
        at = tables[s, lo // B:(L + B - 1) // B].long()
        off = lo // B * B
        k, v = [rows_of(c[at], d).permute(1, 0, 2, 3).reshape(hkv, -1, d)[:, lo - off:L - off] for c in (kc, vc)]
        x = q[s].double().view(hkv, hq // hkv, d) @ k.transpose(1, 2) * scale
        lse[s] = torch.logsumexp(x, -1).reshape(-1)
        out[s] = (torch.softmax(x, -1) @ v).reshape(hq, d)
    return out, lse
