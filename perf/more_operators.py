"""Cases of the 4-bit paged cache and of whole prompts, timed and compared:

* ``pages``   new rows written to 4-bit pages and the pages widened to 16 bits
              (``pa_cache_write`` with a 4-bit cache, ``pa_widen_blocks``)
* ``widen``   the pages of cached prefixes widened to 16 bits, for the chunk
              that follows them (``pa_widen_blocks``)
* ``decode``  decode attention over a 4-bit cache (``pa_decode``)
* ``prompt``  causal attention of packed prompts from their q, k and v rows
              (``pa_prompt_attention``)

A 4-bit row holds, for each group of 64 dims, a scale s and a minimum m in
fp16 and a code n in 0..15 per dim, which stands for s n + m.  A page of one
kv head is its 16 rows' codes (the even dim in the low half of a byte), then
their (s, m) pairs.

``own`` selects what ``run`` computes with: false, elementary torch
operations in 32 bits; true, the library's entry points.
"""
import math
import random

import torch

own = False

DEV = "cuda"
B = 16   # tokens of a cache block
G = 64   # dims that share a scale and a minimum
ACT = {"bf16": torch.bfloat16, "fp16": torch.float16}


# --------------------------------------------------------------------- cases

def listed():
    return [
        # the new tokens of a decode step of 32 sequences, 8 of them padding
        dict(name="pages decode step", op="pages", tokens=32, pad=8, hq=32, hkv=8, d=128, act="bf16"),
        # a long prompt's rows in one go, an odd number of tokens
        dict(name="pages long prompt", op="pages", tokens=16381, pad=0, hq=32, hkv=8, d=128, act="bf16"),
        # a cached prefix of 1024 tokens before a chunk, a small fp16 model
        dict(name="widen short prefix", op="widen", tokens=1024, hq=4, hkv=2, d=64, act="fp16"),
        # four cached documents of 32768 tokens
        dict(name="widen documents", op="widen", tokens=131072, hq=32, hkv=8, d=128, act="bf16"),
        # the smallest batch: an empty sequence and lengths around a block's end
        dict(name="decode tiny", op="decode", lens="0,1,7,16,33", lo=0, hi=0, seqs=5, layout=1, window=0, hq=4, hkv=2,
             d=64, act="bf16"),
        # an ordinary decode batch
        dict(name="decode batch", op="decode", lens="", lo=512, hi=4096, seqs=32, layout=2, window=0, hq=32, hkv=8,
             d=128, act="bf16"),
        # high concurrency, 40 query heads
        dict(name="decode 128 sequences", op="decode", lens="", lo=1024, hi=8192, seqs=128, layout=4, window=0, hq=40,
             hkv=8, d=128, act="bf16"),
        # one long context, an odd length
        dict(name="decode long context", op="decode", lens="131069", lo=0, hi=0, seqs=1, layout=3, window=0, hq=32,
             hkv=8, d=128, act="fp16"),
        # a handful of short questions: a launch's latency
        dict(name="prompt short", op="prompt", lens="1,7,16,33", window=0, hq=4, hkv=2, d=64, act="bf16"),
        # four chunks' worth of prompts arriving together, ragged
        dict(name="prompt batch", op="prompt", lens="512,1531,2048,700,256", window=0, hq=32, hkv=8, d=128, act="bf16"),
        # a local layer of an fp16 model with head_dim 64, a window of 1024
        dict(name="prompt window fp16", op="prompt", lens="4096,3000", window=1024, hq=32, hkv=8, d=64, act="fp16"),
        # one long prompt
        dict(name="prompt long", op="prompt", lens="16384", window=0, hq=32, hkv=8, d=128, act="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = [(32, 8, 128), (40, 8, 128), (16, 1, 128), (8, 8, 128), (4, 2, 64), (32, 8, 64), (6, 2, 128)]


def draw(rng):
    op = rng.choice(["pages", "widen", "decode", "prompt"])
    hq, hkv, d = rng.choice(HEADS)
    case = dict(op=op, hq=hq, hkv=hkv, d=d, act=rng.choice(["bf16", "fp16"]))
    if op == "pages":
        t = _log(rng, 1, 16384)
        case.update(tokens=t, pad=rng.choice([0, 0, min(t - 1, 3)]))
        return case
    if op == "widen":
        case.update(tokens=_log(rng, 1, 131072))
        return case
    case["window"] = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
    if op == "decode":
        while True:
            seqs, hi = _log(rng, 1, 160), _log(rng, 1, 131072)
            if seqs * hi * hkv * d <= 128 * 8192 * 8 * 128 and seqs * hi * hq <= 80_000_000:
                case.update(lens="", lo=rng.choice([0, 1, (hi + 1) // 2, hi]), hi=hi, seqs=seqs,
                            layout=rng.randrange(1 << 20))
                return case
    while True:
        n, top = _log(rng, 1, 40), _log(rng, 1, 16384)
        lens = [rng.choice([top, rng.randint(0, top), _log(rng, 1, top)]) for _ in range(n)]
        if sum(lens) and n * max(lens) ** 2 * hq <= 4_000_000_000:
            case["lens"] = ",".join(map(str, lens))
            return case


def _lens(case):
    if case["lens"]:
        return [int(x) for x in case["lens"].split(",")]
    r = random.Random(case["layout"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]


def _row_bytes(d):
    return d // 2 + d // G * 4


def work(case):
    hq, hkv, d, op = case["hq"], case["hkv"], case["d"], case["op"]
    if op == "pages":
        live = case["tokens"] - case["pad"]
        # rows read, 4-bit rows written, the same rows widened
        return {"bytes": 2 * live * hkv * (2 * d + _row_bytes(d) + 2 * d) + 8 * case["tokens"],
                "flops": 2 * live * hkv * 5 * d}
    if op == "widen":
        t = -(-case["tokens"] // B) * B
        return {"bytes": 2 * t * hkv * (_row_bytes(d) + 2 * d) + 8 * t // B, "flops": 2 * 2 * t * hkv * d}
    lens, w = _lens(case), case["window"]
    if op == "decode":
        seen = [min(x, w) if w else x for x in lens]
        rows = len(lens) * hq
        return {"bytes": 2 * sum(seen) * hkv * _row_bytes(d) + rows * (d * (2 + 4) + 4) + 4 * len(lens)
                + 4 * sum(-(-x // B) for x in seen), "flops": 4 * d * hq * sum(seen)}
    pairs = sum(x * (x + 1) // 2 - (max(0, x - w) * (max(0, x - w) + 1) // 2 if w else 0) for x in lens)
    t = sum(lens)
    return {"bytes": 2 * t * d * (2 * hq + 2 * hkv) + 4 * t * hq + 4 * (len(lens) + 1), "flops": 4 * d * hq * pairs}


# -------------------------------------------------------------------- inputs

def _randn(shape, g, dtype):
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def _quantised(x):
    """(codes, scales, minima) of rows [..., d]: groups of 64 dims."""
    y = x.float().unflatten(-1, (-1, G))
    low, high = y.amin(-1), y.amax(-1)
    s = ((high - low) / torch.full((), 15.0, device=x.device)).half()
    m = low.half()
    r = torch.where(s > 0, torch.reciprocal(s.float()), torch.zeros_like(low))
    n = ((y - m.float()[..., None]) * r[..., None]).round().clamp(0, 15)
    return n.flatten(-2).to(torch.uint8), s, m


def _tiles(n, s, m):
    """Pages [blocks, heads, tile bytes] of codes [blocks, heads, 16, d] and their scales and minima."""
    codes = (n[..., 0::2] | (n[..., 1::2] << 4)).flatten(2)
    pairs = torch.stack([s, m], -1).contiguous().view(torch.uint8).flatten(2)
    return torch.cat([codes, pairs], -1).contiguous()


def _rows_of(tiles, d):
    """fp32 rows [..., 16, d] of pages [..., tile bytes]."""
    cut = B * d // 2
    c = tiles[..., :cut].unflatten(-1, (B, d // 2))
    n = torch.stack([c & 15, c >> 4], -1).flatten(-2).float().unflatten(-1, (-1, G))
    p = tiles[..., cut:].contiguous().view(torch.float16).unflatten(-1, (B, d // G, 2)).float()
    return (n * p[..., :1] + p[..., 1:]).flatten(-2)


def _pool(case, blocks, g):
    """A 4-bit cache full of rows."""
    shape = (blocks, case["hkv"], B, case["d"])
    return _tiles(*_quantised(_randn(shape, g, ACT[case["act"]])))


def _desc(case, blocks, four_bits, window=0):
    from paged_kv_attention_14_gb300 import binding as pa
    kind = {(True, "bf16"): pa.PA_KV_INT4, (True, "fp16"): pa.PA_KV_INT4_F16, (False, "bf16"): pa.PA_KV_BF16,
            (False, "fp16"): pa.PA_KV_F16}[(four_bits, case["act"])]
    return pa.make_desc(blocks, case["hkv"], case["hq"], case["d"], kind, sliding_window=window)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    hq, hkv, d, act, op = case["hq"], case["hkv"], case["d"], ACT[case["act"]], case["op"]
    st = {"case": case}
    if op in ("pages", "widen"):
        pages = -(-case["tokens"] // B)
        blocks = pages + pages // 8 + 2
        ids = 1 + torch.randperm(blocks - 1, generator=g, device=DEV)[:pages]  # block 0 is never written
        st["src"] = ids.to(torch.int32)
        st["dst"] = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        st["kc"], st["vc"] = _pool(case, blocks, g), _pool(case, blocks, g)
        st["k_out"] = torch.zeros((pages, hkv, B, d), dtype=act, device=DEV)
        st["v_out"] = torch.zeros_like(st["k_out"])
    if op == "pages":
        t = case["tokens"]
        # a layer's projection: the keys and values of a token, dense, with the scale and offset of real channels
        centre = torch.randn((2, hkv, d), generator=g, device=DEV)
        st["k"] = (torch.randn((t, hkv, d), generator=g, device=DEV) + 2 * centre[0]).to(act)
        st["v"] = (0.5 * torch.randn((t, hkv, d), generator=g, device=DEV)).to(act)
        i = torch.arange(t, device=DEV)
        slots = ids[i // B] * B + i % B
        if case["pad"]:
            slots[t - case["pad"]:] = -1
        st["slots"] = slots.to(torch.int64).contiguous()
    if op == "decode":
        lens = _lens(case)
        need = [-(-x // B) for x in lens]
        blocks = sum(need) + sum(need) // 8 + 2
        ids = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
        width = max(1, max(need))
        starts = torch.tensor([sum(need[:i]) for i in range(len(need))], device=DEV)
        col = torch.arange(width, device=DEV)
        held = col[None, :] < torch.tensor(need, device=DEV)[:, None]
        at = (starts[:, None] + col).clamp(max=blocks - 1)
        st["tables"] = torch.where(held, ids[at], torch.full_like(ids[at], -1)).contiguous()
        st["lens"], st["max_len"] = torch.tensor(lens, dtype=torch.int32, device=DEV), max(lens)
        st["kc"], st["vc"] = _pool(case, blocks, g), _pool(case, blocks, g)
        st["q"] = _randn((len(lens), hq, d), g, act)
        st["out"] = torch.zeros((len(lens), hq, d), device=DEV)
        st["lse"] = torch.zeros((len(lens), hq), device=DEV)
    if op == "prompt":
        lens = _lens(case)
        t = sum(lens)
        # a projection's output: q, k and v heads of a token side by side
        qkv = _randn((t, (hq + 2 * hkv) * d), g, act)
        st["q"] = qkv[:, :hq * d].view(t, hq, d)
        st["k"] = qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d)
        st["v"] = qkv[:, (hq + hkv) * d:].view(t, hkv, d)
        st["starts"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=DEV)
        st["max_len"], st["seqs"] = max(lens), len(lens)
        st["out"] = torch.zeros((t, hq, d), dtype=act, device=DEV)
        st["lse"] = torch.zeros((t, hq), device=DEV)
    st["softmax_scale"] = 1.0 / math.sqrt(d)
    if own:
        from paged_kv_attention_14_gb300 import binding as pa
        st["desc"] = _desc(case, st["kc"].shape[0] if "kc" in st else 0, op != "prompt", case.get("window", 0))
        if op == "decode":
            st["ws"] = pa.decode_workspace(st["desc"], len(lens), st["max_len"], device=DEV)
    return st


# ----------------------------------------------------------------------- run

def run(st):
    op = st["case"]["op"]
    if own:
        return _run_own(st, op)
    if op == "decode":
        return _plain_decode(st)
    if op == "prompt":
        return _plain_prompt(st)
    d, dst = st["case"]["d"], st["dst"].long()
    for rows, cache in ((st.get("k"), st["kc"]), (st.get("v"), st["vc"])):
        if rows is not None:
            _plain_write(rows, cache, st["slots"], d)
    for cache, out in ((st["kc"], st["k_out"]), (st["vc"], st["v_out"])):
        out[dst] = _rows_of(cache[st["src"].long()], d).to(out.dtype)
    return st["k_out"], st["v_out"]


def _run_own(st, op):
    from paged_kv_attention_14_gb300 import binding as pa
    if op == "decode":
        pa.pa_decode(st["desc"], st["out"], st["q"], st["kc"], st["vc"], st["tables"], st["lens"], st["max_len"],
                     st["softmax_scale"], st["ws"], lse=st["lse"])
        return st["out"], st["lse"]
    if op == "prompt":
        pa.pa_prompt_attention(st["desc"], st["out"], st["q"], st["k"], st["v"], st["starts"], st["max_len"],
                               st["softmax_scale"], lse=st["lse"])
        return st["out"], st["lse"]
    if op == "pages":
        pa.pa_cache_write(st["desc"], st["k"], st["v"], st["kc"], st["vc"], st["slots"])
    pa.pa_widen_blocks(st["desc"], st["kc"], st["vc"], st["src"], st["k_out"], st["v_out"], st["dst"])
    return st["k_out"], st["v_out"]


def _plain_write(rows, cache, slots, d):
    n, s, m = _quantised(rows)
    cut = B * d // 2
    live = (slots >= 0)[:, None, None]
    at = slots.clamp(min=0)
    codes = cache[..., :cut].unflatten(-1, (B, d // 2))
    pairs = cache[..., cut:].unflatten(-1, (B, d // G * 4))
    for part, new in ((codes, n[..., 0::2] | (n[..., 1::2] << 4)),
                      (pairs, torch.stack([s, m], -1).contiguous().view(torch.uint8).flatten(2))):
        # a skipped token puts its place's row back as it was
        part[at // B, :, at % B, :] = torch.where(live, new, part[at // B, :, at % B, :])


def _softmax(x, v, how):
    """(sum of softmax weights times v, log-sum-exp) over x's last axis; masked scores are -inf."""
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    x = x.sub_(top).exp_()
    total = x.sum(-1)
    o = torch.einsum(how, x, v) / total.clamp(min=1e-30)[..., None]
    return o, top[..., 0] + total.log()


def _plain_decode(st):
    case = st["case"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    s, width = st["tables"].shape
    at = st["tables"].clamp(min=0).long()
    lens = st["lens"].long()[:, None]
    t = torch.arange(width * B, device=DEV)[None, :]
    seen = t < lens
    if case["window"]:
        seen &= t >= lens - case["window"]
    k = _rows_of(st["kc"][at], d).transpose(1, 2).reshape(s, hkv, width * B, d)
    q = st["q"].float().view(s, hkv, hq // hkv, d) * st["softmax_scale"]
    x = torch.einsum("shrd,shtd->shrt", q, k).masked_fill_(~seen[:, None, None, :], -math.inf)
    v = _rows_of(st["vc"][at], d).transpose(1, 2).reshape(s, hkv, width * B, d)
    o, lse = _softmax(x, v, "shrt,shtd->shrd")
    return o.reshape(s, hq, d), lse.reshape(s, hq)


def _plain_prompt(st):
    case = st["case"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    starts, n, top = st["starts"].long(), st["seqs"], st["max_len"]
    t = torch.arange(top, device=DEV)
    lens = starts[1:] - starts[:-1]
    rows = (starts[:-1, None] + t).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][rows].float().view(n, top, hkv, hq // hkv, d) * st["softmax_scale"]
    k, v = st["k"][rows].float(), st["v"][rows].float()
    x = torch.einsum("sihrd,sjhd->shrij", q, k)
    seen = t[:, None] >= t[None, :]
    if case["window"]:
        seen &= t[None, :] > t[:, None] - case["window"]
    x.masked_fill_(~seen, -math.inf)
    o, lse = _softmax(x, v, "shrij,sjhd->shrid")
    o, lse = o.permute(0, 3, 1, 2, 4).reshape(n, top, hq, d), lse.permute(0, 3, 1, 2).reshape(n, top, hq)
    held = t[None, :] < lens[:, None]
    return o[held].to(st["q"].dtype), lse[held]


# --------------------------------------------------------------------- exact

def _exact_rows(tiles, d):
    """Rows [heads, tokens, d] in 64 bits of pages [blocks, heads, tile bytes]."""
    f = torch.float64
    at = torch.arange(d, device=DEV)
    codes = tiles[..., :B * d // 2].reshape(*tiles.shape[:2], B, d // 2)[..., at // 2].to(torch.int64)
    codes = (codes >> (4 * (at % 2))) % 16
    pairs = tiles[..., B * d // 2:].contiguous().view(torch.float16).reshape(*tiles.shape[:2], B, d // G, 2).to(f)
    rows = codes.to(f) * pairs[..., at // G, 0] + pairs[..., at // G, 1]
    return rows.permute(1, 0, 2, 3).reshape(tiles.shape[1], -1, d)


def exact(case, seed):
    """The operators' definitions in 64 bits, one sequence, one head or one page range at a time."""
    st = prepare(case, seed)
    f = torch.float64
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    per = hq // hkv
    if case["op"] in ("pages", "widen"):
        outs = []
        for cache, new in ((st["kc"], st.get("k")), (st["vc"], st.get("v"))):
            rows = torch.cat([_exact_rows(cache[lo:lo + 1024], d).reshape(hkv, -1, B, d).transpose(0, 1)
                              for lo in range(0, cache.shape[0], 1024)])
            if new is not None:
                keep = st["slots"] >= 0
                y = new[keep].to(f).reshape(-1, hkv, d // G, G)
                low, high = y.min(-1, keepdim=True).values, y.max(-1, keepdim=True).values
                s, m = ((high - low) / 15).half().to(f), low.half().to(f)
                n = torch.where(s > 0, torch.clamp(torch.round((y - m) / torch.where(s > 0, s, 1.0)), 0, 15), 0.0)
                slot = st["slots"][keep]
                rows[slot // B, :, slot % B] = (n * s + m).reshape(-1, hkv, d)
            out = torch.empty((st["dst"].shape[0], hkv, B, d), dtype=f, device=DEV)
            out[st["dst"].long()] = rows[st["src"].long()]
            outs.append(out)
        return tuple(outs)
    window = case["window"]
    if case["op"] == "decode":
        out = torch.zeros(st["q"].shape, dtype=f, device=DEV)
        lse = torch.full(st["q"].shape[:2], -math.inf, dtype=f, device=DEV)
        for i, length in enumerate(_lens(case)):
            if length == 0:
                continue
            first = max(0, length - window) if window else 0
            at = st["tables"][i, :(length + B - 1) // B].long()
            k, v = [_exact_rows(c[at], d)[:, first:length] for c in (st["kc"], st["vc"])]
            x = st["q"][i].to(f).view(hkv, per, d) @ k.transpose(1, 2) * st["softmax_scale"]
            lse[i] = torch.logsumexp(x, -1).reshape(-1)
            out[i] = (torch.softmax(x, -1) @ v).reshape(hq, d)
        return out, lse
    if 4 * sum(x * x for x in _lens(case)) * hq * d > 8e12:
        return None
    out = torch.zeros(st["q"].shape, dtype=f, device=DEV)
    lse = torch.zeros(st["q"].shape[:2], dtype=f, device=DEV)
    at = 0
    for length in _lens(case):
        # queries in ranges: each sees the keys up to its last one
        for lo in range(0, length, 2048):
            hi = min(length, lo + 2048)
            first = max(0, lo - window + 1) if window else 0
            i, j = torch.arange(lo, hi, device=DEV)[:, None], torch.arange(first, hi, device=DEV)[None, :]
            hidden = (j > i) | (j <= i - window) if window else j > i
            for h in range(hkv):
                q = st["q"][at + lo:at + hi, h * per:(h + 1) * per].to(f).transpose(0, 1)
                k, v = [st[c][at + first:at + hi, h].to(f) for c in ("k", "v")]
                x = (q @ k.T * st["softmax_scale"]).masked_fill_(hidden, -math.inf)
                lse[at + lo:at + hi, h * per:(h + 1) * per] = torch.logsumexp(x, -1).T
                out[at + lo:at + hi, h * per:(h + 1) * per] = (torch.softmax(x, -1) @ v).transpose(0, 1)
        at += length
    return out, lse
