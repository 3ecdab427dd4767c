"""How exact pa_decode_shared is, tight enough to see half of a weight go.

The weights P = 2^(score - maximum) enter the products as a pair of 16-bit
values, hi + lo (bf16 with a bf16 cache, else fp16), good to half a step of a
half step: 2^-16 and 2^-22 of P.  hi alone is good to 2^-8 and 2^-11 only."""
import numpy as np
import pytest
import torch

import pa_helpers as H
from paged_kv_attention_14_gb300 import binding as B
from paged_kv_attention_14_gb300 import workloads as W

DEV = "cuda"
KV = [W.KV_BF16, W.KV_F16, W.KV_FP8, W.KV_FP8_E5M2]
PAIR = {W.KV_BF16: 2.0 ** -16}  # else fp16: 2^-22


def _run(b):
    c = b.meta["cascade"]
    gs, pre = c["query_start_loc"], c["prefix_lens"]
    d, t, S = H.desc_of(b), b.block_tables_decode, b.q_decode.shape[0]
    out = torch.full((S, b.num_q_heads, b.head_dim), float("nan"), device=DEV)
    mg = int((gs[1:] - gs[:-1]).max())
    kc, vc = H.gpu_caches(b)
    B.pa_decode_shared(d, out, b.q_decode, kc, vc, t, b.context_lens_decode, t.shape[1] * 16, gs, pre, mg, int(pre.max()),
                       b.scale, B.decode_shared_workspace(d, S, pre.shape[0], mg))
    torch.cuda.synchronize()
    return out


SHORT = [([4], [48]), ([17, 3], [64, 32])]  # narrow items; 68 and 12 rows


def _short(groups, plens, kv, D, device):
    """Queries that pick one column of K each (twice its value: exact scores,
    up to 9.6), positive values: no sum cancels."""
    S = sum(groups)
    b = W.shared_prefix_decode(950 + S + D, groups, plens, [5 * i % 37 + 1 for i in range(S)], 8, 2, D, kv_dtype=kv, scale=1.0,
                               device=device, poison=False)
    b.v_pool = b.v_pool.abs() + 0.25
    b.q_decode.zero_()
    for s in range(S):
        for h in range(8):
            b.q_decode[s, h, (8 * s + 5 * h) % D] = 2
    return b


def _reference(b, halves):
    """The output in 64 bits from the cache's own values; with `halves` False
    each part's weights are rounded to one 16-bit value."""
    code, kc, vc = H.oracle_caches(b)
    kind = {W.KV_FP8: torch.float8_e4m3fn, W.KV_FP8_E5M2: torch.float8_e5m2}.get(b.kv_dtype)

    def values(x, scale):
        if kind is None:
            return x.double()
        return torch.from_numpy(np.ascontiguousarray(x)).view(torch.uint8).view(kind).double() * float(np.float32(scale))

    k, v = values(kc, b.k_scale), values(vc, b.v_scale)
    gs, pre = b.meta["cascade"]["query_start_loc"].tolist(), b.meta["cascade"]["prefix_lens"].tolist()
    S, Hq, D = b.q_decode.shape
    g = Hq // b.num_kv_heads
    out = np.zeros((S, Hq, D))
    for s in range(S):
        n = int(b.context_lens_decode[s])
        P = pre[max(j for j in range(len(pre)) if gs[j] <= s)]
        t = b.block_tables_decode[s, :(n + 15) // 16].long().cpu()
        ks = k[t].permute(1, 0, 2, 3).reshape(b.num_kv_heads, -1, D)[:, :n]
        vs = v[t].permute(1, 0, 2, 3).reshape(b.num_kv_heads, -1, D)[:, :n]
        for h in range(Hq):
            x = ks[h // g] @ b.q_decode[s, h].double().cpu() * b.scale
            w = torch.exp(x - x.max())
            total = w.sum()
            if not halves:
                act = torch.bfloat16 if b.kv_dtype == W.KV_BF16 else torch.float16
                for part in (slice(0, P), slice(P, n)):
                    top = w[part].max()
                    w[part] = (w[part] / top).to(act).double() * top
            out[s, h] = (w[:, None] * vs[h // g]).sum(0) / total
    return out


def _bound(kv):
    """Relative to each (positive) output, worst case:
    the weights: P's pair; the score's distance d from the maximum (log2
    units) through four roundings (three of the scale, one of the difference),
    4 * 2^-24 * d * ln 2, and the mean of d over weights 2^-d of 101 keys, times
    values in a ratio of 20 at most, is at most log2(101 * 20) = 11: 1.9e-6, in
    the numerator and in the sum; the exponential 2^-22 in both;
    the sums: P V of at most 101 keys, 14 products of 16 keys each truncated
    to 2^-23 of the running sum once for their own sum and once when added,
    14 * 2 * 2^-23 = 3.3e-6; l, at most 40 additions of 2^-24, 2.4e-6;
    the join: the parts' log-sum-exps, up to 16 in log2 units, rounded by
    2^-24 of that each, 2 * 16 * 2^-24 * ln 2 = 1.3e-6, two exponentials, two
    products, a division: 2.4e-6."""
    return PAIR.get(kv, 2.0 ** -22) + 2 * 1.9e-6 + 2 * 2.0 ** -22 + 3.3e-6 + 2.4e-6 + 2.4e-6


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("groups,plens", SHORT)
def test_one_16_bit_weight_would_be_seen(groups, plens, D, kv):
    """The inputs below tell a pair from its first half: the oracle with rounded weights is off by four bounds."""
    b = _short(groups, plens, kv, D, "cpu")
    want, single = _reference(b, True), _reference(b, False)
    assert np.abs(single / want - 1).max() > 4 * _bound(kv)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("groups,plens", SHORT)
def test_weights_keep_both_halves(groups, plens, D, kv):
    from paged_kv_attention_14_gb300 import build
    B.load(build.build())
    b = _short(groups, plens, kv, D, DEV)
    want = _reference(b, True)
    err = np.abs(_run(b).double().cpu().numpy() / want - 1).max()
    assert err <= _bound(kv), f"{err:.2e} of {_bound(kv):.2e}"


@pytest.mark.gpu
@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [3, 20])
def test_long_prefixes_in_the_2_norm(n, D, kv):
    """16384 tokens, N(0, 1) rows, narrow items and wide ones.  A chain of 16
    steps loses 256 products' truncation, 256 * 2/3 * 0.72 * 2^-24 = 7.3e-6 of
    its end value (a product loses half of 2^-23 |O| on average, 0.72 of that
    over a binade, and O grows as a random walk); P's pairs add an independent
    2.6e-6 for bf16 (a uniform error within half a step, twice), the scores'
    products 1e-6: 1e-5 covers their sum of squares.  The first half of P alone
    would be off by 2^-11 / sqrt 3 and more, 2e-4."""
    from paged_kv_attention_14_gb300 import build
    B.load(build.build())
    b = W.shared_prefix_decode(970 + n, [n], [16384], [17 * i % 90 + 1 for i in range(n)], 8, 2, D, kv_dtype=kv, device=DEV)
    out = _run(b)
    rows = [0, n - 1]
    o, _ = H.oracle_decode(b, ocaches=H.oracle_caches(b), pairs=[(s, h) for s in rows for h in range(8)])
    e = out[rows].double().cpu().numpy().reshape(-1, D) - o.reshape(-1, D)
    rel = np.linalg.norm(e) / np.linalg.norm(o)
    assert rel <= 1e-5, f"{rel:.2e}"
