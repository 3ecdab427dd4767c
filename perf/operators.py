"""Cases of the step operators around the paged cache, timed and compared:

* ``norm_rope``   per-head RMS norm of queries and keys and their position
                  rotation in one pass (``pa_qk_norm_rope``)
* ``rope_append`` the same, with the keys and values going to their slots of
                  the paged cache (``pa_rope_cache_write``)
* ``shared``      decode attention of a batch whose sequences share prefixes,
                  each prefix read once for its whole group
                  (``pa_decode_shared``)

``own`` selects what ``run`` computes with: false, elementary torch
operations in 32 bits; true, the library's entry points.
"""
import math
import random

import torch

own = False

DEV = "cuda"
B = 16  # tokens of a cache block
ACT = {"bf16": torch.bfloat16, "fp16": torch.float16}
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}


def _act(case):
    return ACT.get(case["kv"], torch.bfloat16)


# --------------------------------------------------------------------- cases

def listed():
    return [
        # the newest token of one sequence: a launch's latency
        dict(name="norm_rope one token", op="norm_rope", tokens=1, hq=32, hkv=8, d=128, rd=128, inter=False, norm=True,
             kv="bf16", max_pos=40960),
        # a decode batch of 128 sequences, 40 query heads
        dict(name="norm_rope decode batch", op="norm_rope", tokens=128, hq=40, hkv=8, d=128, rd=128, inter=False,
             norm=True, kv="bf16", max_pos=40960),
        # a long prompt's chunk in one go, an odd number of tokens
        dict(name="norm_rope long chunk", op="norm_rope", tokens=16381, hq=32, hkv=8, d=128, rd=128, inter=False,
             norm=True, kv="bf16", max_pos=40960),
        # one decode step of 32 sequences, a quarter of the rows padding (a fixed-size captured step)
        dict(name="rope_append decode step", op="rope_append", tokens=32, hq=32, hkv=8, d=128, rd=128, inter=False,
             norm=True, kv="bf16", max_pos=40960, pad=8),
        # the mixed step's new tokens: 16 decode tokens and 4 chunks of 512
        dict(name="rope_append mixed step", op="rope_append", tokens=2064, hq=32, hkv=8, d=128, rd=128, inter=False,
             norm=True, kv="bf16", max_pos=40960, pad=0),
        # a prompt's chunk into an E4M3 cache, a model without q / k norms
        dict(name="rope_append e4m3 chunk", op="rope_append", tokens=8192, hq=40, hkv=8, d=128, rd=128, inter=False,
             norm=False, kv="e4m3", max_pos=131072, pad=0),
        # an fp16 model with head_dim 64, interleaved rotation of half of each head, an odd batch
        dict(name="rope_append fp16 partial", op="rope_append", tokens=777, hq=4, hkv=2, d=64, rd=32, inter=True,
             norm=False, kv="fp16", max_pos=8192, pad=5),
        # the smallest shared batch: three sequences on a two-block prefix and one alone
        dict(name="shared tiny", op="shared", groups="3,1", prefixes="32,0", suf_lo=1, suf_hi=33, layout=1, hq=4, hkv=2,
             d=64, kv="bf16"),
        # four system prompts of 4096 tokens with 16 conversations each
        dict(name="shared four prompts", op="shared", groups="16,16,16,16", prefixes="4096,4096,4096,4096", suf_lo=16,
             suf_hi=511, layout=2, hq=32, hkv=8, d=128, kv="bf16"),
        # 64 conversations on one 16384-token prompt
        dict(name="shared wide prompt", op="shared", groups="64", prefixes="16384", suf_lo=16, suf_hi=511, layout=3,
             hq=32, hkv=8, d=128, kv="bf16"),
        # an E4M3 cache under 128 sequences, 40 query heads, uneven groups
        dict(name="shared e4m3 batch", op="shared", groups="61,40,20,7", prefixes="8192,2048,1040,16", suf_lo=1,
             suf_hi=1000, layout=4, hq=40, hkv=8, d=128, kv="e4m3"),
        # eight questions on one document of 131072 tokens
        dict(name="shared document", op="shared", groups="8", prefixes="131072", suf_lo=20, suf_hi=300, layout=5, hq=32,
             hkv=8, d=128, kv="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = [(32, 8, 128), (40, 8, 128), (16, 1, 128), (8, 8, 128), (4, 2, 64), (32, 8, 64)]


def draw(rng):
    op = rng.choice(["norm_rope", "rope_append", "shared"])
    hq, hkv, d = rng.choice(HEADS)
    if op != "shared":
        rd = rng.choice([d, d, d // 2, 16])
        case = dict(op=op, tokens=_log(rng, 1, 16384), hq=hq, hkv=hkv, d=d, rd=rd, inter=rng.random() < 0.3,
                    norm=rng.random() < 0.6, kv=rng.choice(["bf16", "bf16", "fp16", "e4m3", "e5m2"]),
                    max_pos=rng.choice([8192, 40960, 131072]))
        if op == "norm_rope":
            case["kv"] = rng.choice(["bf16", "fp16"])
        else:
            case["pad"] = rng.choice([0, 0, min(case["tokens"] - 1, 3)])
        return case
    top = max(work(c)["bytes"] for c in listed())
    while True:
        n_groups = _log(rng, 1, 12)
        groups = [_log(rng, 1, 64) for _ in range(n_groups)]
        prefixes = [rng.choice([0, 1, 1, 1]) * B * _log(rng, 1, 2048) for _ in range(n_groups)]
        hi = _log(rng, 1, 1500)
        case = dict(op="shared", groups=",".join(map(str, groups)), prefixes=",".join(map(str, prefixes)), suf_lo=1,
                    suf_hi=hi, layout=rng.randrange(1 << 20), hq=hq, hkv=hkv, d=d,
                    kv=rng.choice(["bf16", "bf16", "fp16", "e4m3", "e5m2"]))
        w = work(case)
        # no more traffic, and no larger score matrices, than the listed cases have
        if w["bytes"] <= top and sum(groups) <= 160 and sum(groups) * hq * (max(prefixes) + hi) <= 80_000_000:
            return case


def _layout(case):
    """(group sizes, prefix lengths, suffix length of every sequence) of a shared case."""
    sizes = [int(x) for x in case["groups"].split(",")]
    pre = [int(x) for x in case["prefixes"].split(",")]
    r = random.Random(case["layout"])
    return sizes, pre, [r.randint(case["suf_lo"], case["suf_hi"]) for _ in range(sum(sizes))]


def _esz(case):
    return 1 if case["kv"] in FP8 else 2


def work(case):
    if case["op"] == "shared":
        sizes, pre, suf = _layout(case)
        rows = sum(sizes)
        total = sum(n * p for n, p in zip(sizes, pre)) + sum(suf)
        tok = 2 * case["hkv"] * case["d"] * _esz(case)
        blocks = sum(p // B for p in pre) + sum((x + B - 1) // B for x in suf)
        by = (sum(pre) + sum(suf)) * tok + rows * case["hq"] * (case["d"] * (2 + 4) + 4) + 4 * (blocks + rows)
        return {"bytes": by, "flops": 4 * case["d"] * case["hq"] * total}
    t, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
    table = 4 * case["rd"] * min(t, case["max_pos"])
    flops = 3 * t * (hq + hkv) * case["rd"] + (4 * t * (hq + hkv) * d if case["norm"] else 0)
    if case["op"] == "norm_rope":
        return {"bytes": 2 * 2 * t * (hq + hkv) * d + table + 4 * t, "flops": flops}
    live = t - case["pad"]
    kv = 2 * live * hkv * d * (2 + _esz(case))
    return {"bytes": 2 * 2 * t * hq * d + kv + table + 12 * t, "flops": flops}


# -------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(shape, g, dtype):
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def _rope_inputs(case, seed):
    g = _gen(seed)
    t, hq, hkv, d, rd = case["tokens"], case["hq"], case["hkv"], case["d"], case["rd"]
    act = _act(case)
    st = {"case": case}
    # the projection's output: q, k and v heads of a token side by side
    qkv = _randn((t, (hq + 2 * hkv) * d), g, act)
    st["q"] = qkv[:, :hq * d].view(t, hq, d)
    st["k"] = qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d)
    st["v"] = qkv[:, (hq + hkv) * d:].view(t, hkv, d)
    st["q_w"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(act) if case["norm"] else None
    st["k_w"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(act) if case["norm"] else None
    st["eps"] = 1e-6
    # cos | sin of position * base^(-2 i / rd), made in 64 bits
    freq = 1e6 ** (-torch.arange(0, rd, 2, dtype=torch.float64, device=DEV) / rd)
    ang = torch.arange(case["max_pos"], dtype=torch.float64, device=DEV)[:, None] * freq
    st["table"] = torch.cat([ang.cos(), ang.sin()], 1).float()
    if t <= 512:  # a decode batch: every token at a position of its own
        pos = torch.randint(0, case["max_pos"], (t,), generator=g, device=DEV)
    else:  # a chunk: consecutive positions
        first = random.Random(seed).randrange(max(1, case["max_pos"] - t))
        pos = first + torch.arange(t, device=DEV)
        pos = pos % case["max_pos"]
    st["pos"] = pos.to(torch.int32)
    return st, g


def prepare(case, seed):
    if case["op"] == "shared":
        return _prepare_shared(case, seed)
    st, g = _rope_inputs(case, seed)
    t, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
    st["q_out"] = torch.zeros((t, hq, d), dtype=_act(case), device=DEV)
    if case["op"] == "norm_rope":
        st["k_out"] = torch.zeros((t, hkv, d), dtype=_act(case), device=DEV)
        nb = 1
    else:
        nb = (t + B - 1) // B + 3  # block 0 is never written
        shape = (nb, hkv, B, d)
        st["scale"] = (0.01, 0.0125)
        if case["kv"] in FP8:
            st["kc"] = torch.zeros(shape, dtype=torch.uint8, device=DEV)
            st["vc"] = torch.zeros(shape, dtype=torch.uint8, device=DEV)
        else:
            st["kc"], st["vc"] = _randn(shape, g, _act(case)), _randn(shape, g, _act(case))
        perm = B + torch.randperm((nb - 1) * B, generator=g, device=DEV)[:t]
        if case["tokens"] > 512:  # a chunk fills whole pages, in an order of its own
            pages = 1 + torch.randperm(nb - 1, generator=g, device=DEV)
            i = torch.arange(t, device=DEV)
            perm = pages[i // B] * B + i % B
        if case["pad"]:
            perm[t - case["pad"]:] = -1
        st["slots"] = perm.to(torch.int64).contiguous()
    if own:
        from paged_kv_attention_14_gb300 import binding as pa
        st["desc"] = _desc(pa, case, nb, st.get("scale", (0.0, 0.0)))
        st["rope"] = pa.make_rope(st["table"], rotary_dim=case["rd"], interleaved=case["inter"], q_weight=st["q_w"],
                                  k_weight=st["k_w"], eps=st["eps"])
    return st


def _desc(pa, case, num_blocks, scales):
    code = {"bf16": pa.PA_KV_BF16, "fp16": pa.PA_KV_F16, "e4m3": pa.PA_KV_FP8_E4M3, "e5m2": pa.PA_KV_FP8_E5M2}
    ks, vs = scales if case["kv"] in FP8 else (0.0, 0.0)
    return pa.make_desc(num_blocks, case["hkv"], case["hq"], case["d"], code[case["kv"]], k_scale=ks, v_scale=vs)


def _prepare_shared(case, seed):
    g = _gen(seed)
    sizes, pre, suf = _layout(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    n, rows = len(sizes), sum(sizes)
    group_of = [j for j, m in enumerate(sizes) for _ in range(m)]
    lens = [pre[j] + x for j, x in zip(group_of, suf)]
    need = sum(p // B for p in pre) + sum((x + B - 1) // B for x in suf)
    nb = need + need // 8 + 2
    ids = list(range(nb))
    random.Random(seed).shuffle(ids)
    own_pages, at = [], 0
    heads = []
    for p in pre:
        heads.append(ids[at:at + p // B])
        at += p // B
    for x in suf:
        own_pages.append(ids[at:at + (x + B - 1) // B])
        at += (x + B - 1) // B
    width = max((x + B - 1) // B for x in lens)
    table = torch.full((rows, width), -1, dtype=torch.int32)
    for s, j in enumerate(group_of):
        row = heads[j] + own_pages[s]
        table[s, :len(row)] = torch.tensor(row, dtype=torch.int32)
    starts = [sum(sizes[:j]) for j in range(n + 1)]
    st = {"case": case, "tables": table.to(DEV), "lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
          "starts": torch.tensor(starts, dtype=torch.int32, device=DEV),
          "prefixes": torch.tensor(pre, dtype=torch.int32, device=DEV), "max_len": max(lens), "max_pre": max(pre),
          "max_group": max(sizes), "max_suf": max(suf), "softmax_scale": 1.0 / math.sqrt(d)}
    st["group_of"] = torch.tensor(group_of, device=DEV)
    st["q"] = _randn((rows, hq, d), g, _act(case))
    shape = (nb, hkv, B, d)
    if case["kv"] in FP8:
        kind, top = FP8[case["kv"]]
        st["scale"] = (4.5 / top, 5.0 / top)
        st["kc"], st["vc"] = [(torch.randn(shape, generator=g, device=DEV) / s).clamp_(-top, top).to(kind)
                              .view(torch.uint8) for s in st["scale"]]
    else:
        st["scale"] = (1.0, 1.0)
        st["kc"], st["vc"] = _randn(shape, g, _act(case)), _randn(shape, g, _act(case))
    st["out"] = torch.zeros((rows, hq, d), device=DEV)
    st["lse"] = torch.zeros((rows, hq), device=DEV)
    if own:
        from paged_kv_attention_14_gb300 import binding as pa
        st["desc"] = _desc(pa, case, nb, st["scale"])
        st["ws"] = pa.decode_shared_workspace(st["desc"], rows, n, st["max_group"], device=DEV)
    return st


# ----------------------------------------------------------------------- run

def run(st):
    op = st["case"]["op"]
    if own:
        return _run_own(st, op)
    if op == "shared":
        return _plain_shared(st)
    q = _plain_norm_rope(st, st["q"], st["q_w"])
    k = _plain_norm_rope(st, st["k"], st["k_w"])
    if op == "norm_rope":
        return q.to(st["q"].dtype), k.to(st["k"].dtype)
    slots = st["slots"]
    live = (slots >= 0)[:, None, None]
    at = slots.clamp(min=0)
    for_cache = []
    for rows, cache, scale in ((k, st["kc"], st["scale"][0]), (st["v"].float(), st["vc"], st["scale"][1])):
        if st["case"]["kv"] in FP8:
            kind, top = FP8[st["case"]["kv"]]
            new = (rows / scale).clamp(-top, top).to(kind).view(torch.uint8)
        else:
            new = rows.to(cache.dtype)
        # a skipped token puts block 0's first row back as it was
        cache[at // B, :, at % B, :] = torch.where(live, new, cache[0, :, 0, :])
        for_cache.append(cache.view(FP8[st["case"]["kv"]][0]) if st["case"]["kv"] in FP8 else cache)
    return q.to(st["q"].dtype), for_cache[0], for_cache[1]


def _run_own(st, op):
    from paged_kv_attention_14_gb300 import binding as pa
    if op == "norm_rope":
        pa.pa_qk_norm_rope(st["desc"], st["rope"], st["q_out"], st["k_out"], st["q"], st["k"], st["pos"])
        return st["q_out"], st["k_out"]
    if op == "rope_append":
        pa.pa_rope_cache_write(st["desc"], st["rope"], st["q_out"], st["q"], st["k"], st["v"], st["pos"], st["kc"],
                               st["vc"], st["slots"])
        if st["case"]["kv"] in FP8:
            kind = FP8[st["case"]["kv"]][0]
            return st["q_out"], st["kc"].view(kind), st["vc"].view(kind)
        return st["q_out"], st["kc"], st["vc"]
    pa.pa_decode_shared(st["desc"], st["out"], st["q"], st["kc"], st["vc"], st["tables"], st["lens"], st["max_len"],
                        st["starts"], st["prefixes"], st["max_group"], st["max_pre"], st["softmax_scale"], st["ws"],
                        lse=st["lse"])
    return st["out"], st["lse"]


def _plain_norm_rope(st, x, w):
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + st["eps"]) * w.float()
    rd = st["case"]["rd"]
    row = st["table"][st["pos"].long()][:, None, :]
    cos, sin = row[..., :rd // 2], row[..., rd // 2:]
    if st["case"]["inter"]:
        a, b = y[..., 0:rd:2], y[..., 1:rd:2]
        rot = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :rd // 2], y[..., rd // 2:rd]
        rot = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([rot, y[..., rd:]], -1)


def _plain_rows(st, cache, tables, tokens, scale):
    """Rows [table, tokens, heads, d] of a cache in 32 bits: positions `tokens` behind `tables`."""
    at = tables.gather(1, tokens // B).clamp(min=0).long()
    if st["case"]["kv"] in FP8:
        return cache[at, :, tokens % B, :].view(FP8[st["case"]["kv"]][0]).float() * scale
    return cache[at, :, tokens % B, :].float()


def _plain_shared(st):
    case = st["case"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    rows, n = st["lens"].shape[0], st["prefixes"].shape[0]
    per = hq // hkv
    grp, pre = st["group_of"], st["prefixes"].long()
    inner = torch.arange(rows, device=DEV) - st["starts"].long()[grp]
    q = st["q"].float().view(rows, hkv, per, d) * st["softmax_scale"]
    # prefix: the queries of a group side by side
    qg = torch.zeros((n, st["max_group"], hkv, per, d), device=DEV)
    qg[grp, inner] = q
    t = torch.arange(max(st["max_pre"], 1), device=DEV)
    tok = torch.minimum(t[None, :], (pre[:, None] - 1).clamp(min=0))
    first = st["tables"][st["starts"][:-1].long()]
    kp = _plain_rows(st, st["kc"], first, tok, st["scale"][0])
    vp = _plain_rows(st, st["vc"], first, tok, st["scale"][1])
    sp = torch.einsum("gnhrd,gthd->gnhrt", qg, kp)[grp, inner]
    sp = sp.masked_fill((t[None, :] >= pre[grp][:, None])[:, None, None, :], -math.inf)
    # own suffixes
    u = pre[grp][:, None] + torch.arange(st["max_suf"], device=DEV)[None, :]
    lens = st["lens"].long()[:, None]
    tok = torch.minimum(u, lens - 1)
    ks = _plain_rows(st, st["kc"], st["tables"], tok, st["scale"][0])
    vs = _plain_rows(st, st["vc"], st["tables"], tok, st["scale"][1])
    ss = torch.einsum("shrd,sthd->shrt", q, ks).masked_fill((u >= lens)[:, None, None, :], -math.inf)
    top = torch.maximum(sp.amax(-1), ss.amax(-1))
    sp, ss = torch.exp(sp - top[..., None]), torch.exp(ss - top[..., None])
    total = sp.sum(-1) + ss.sum(-1)
    pg = torch.zeros((n, st["max_group"], hkv, per, t.shape[0]), device=DEV)
    pg[grp, inner] = sp
    o = torch.einsum("gnhrt,gthd->gnhrd", pg, vp)[grp, inner] + torch.einsum("shrt,sthd->shrd", ss, vs)
    return (o / total[..., None]).reshape(rows, hq, d), (top + total.log()).reshape(rows, hq)


# --------------------------------------------------------------------- exact

def exact(case, seed):
    """The operators' definitions in 64 bits, one sequence or one token row at a time."""
    st = prepare(case, seed)
    f = torch.float64
    if case["op"] == "shared":
        per = case["hq"] // case["hkv"]
        out = torch.zeros(st["q"].shape, dtype=f, device=DEV)
        lse = torch.zeros(st["q"].shape[:2], dtype=f, device=DEV)
        pools = [c.view(FP8[case["kv"]][0]) if case["kv"] in FP8 else c for c in (st["kc"], st["vc"])]
        for s, length in enumerate(st["lens"].tolist()):
            blocks = st["tables"][s, :(length + B - 1) // B].long()
            k, v = [(p.view(torch.uint8)[blocks].view(p.dtype) if case["kv"] in FP8 else p[blocks]).to(f)
                    .permute(1, 0, 2, 3).reshape(case["hkv"], -1, case["d"])[:, :length] * float(c)
                    for p, c in zip(pools, st["scale"])]
            x = st["q"][s].to(f).view(case["hkv"], per, case["d"]) @ k.transpose(1, 2) * st["softmax_scale"]
            lse[s] = torch.logsumexp(x, -1).reshape(-1)
            out[s] = (torch.softmax(x, -1) @ v).reshape(case["hq"], case["d"])
        return out, lse
    rd = case["rd"]
    i = torch.arange(case["d"], device=DEV)
    # dim -> its partner, its angle and the sign of the partner's share
    if case["inter"]:
        mate, angle, sign = i ^ 1, i // 2, torch.where(i % 2 == 0, -1.0, 1.0).to(f)
    else:
        h = rd // 2
        mate, angle, sign = torch.where(i < h, i + h, i - h), i % h, torch.where(i < h, -1.0, 1.0).to(f)
    mate, angle = torch.where(i < rd, mate, i), torch.where(i < rd, angle, torch.zeros_like(i))
    row = st["table"].to(f)[st["pos"].long()]
    cos = torch.where(i < rd, row[:, angle], torch.ones((), dtype=f, device=DEV))
    sin = torch.where(i < rd, row[:, rd // 2 + angle], torch.zeros((), dtype=f, device=DEV))

    def rotated(x, w):
        y = x.to(f)
        if w is not None:
            y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / case["d"] + st["eps"]) * w.to(f)
        return y * cos[:, None, :] + sign * y[..., mate] * sin[:, None, :]

    q, k = rotated(st["q"], st["q_w"]), rotated(st["k"], st["k_w"])
    if case["op"] == "norm_rope":
        return q, k
    if case["kv"] == "e5m2":  # two bits of mantissa: the rounding to them is most of what 64 bits would show
        return q, None, None
    caches = []
    for new, cache, scale in ((k, st["kc"], st["scale"][0]), (st["v"].to(f), st["vc"], st["scale"][1])):
        if case["kv"] in FP8:
            cache = cache.view(FP8[case["kv"]][0]).to(f)
            new = new / scale
        else:
            cache = cache.to(f)
        for lo in range(0, case["tokens"], 4096):
            s = st["slots"][lo:lo + 4096]
            keep = s >= 0
            cache[s[keep] // B, :, s[keep] % B, :] = new[lo:lo + 4096][keep]
        caches.append(cache)
    return q, caches[0], caches[1]
