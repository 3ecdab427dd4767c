"""pa_decode_shared where sequences end inside their group's prefix."""
import pytest
import torch

import pa_helpers as H
from paged_kv_attention_14_gb300 import binding as B
from paged_kv_attention_14_gb300 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda"
# the error of the scores, the weights and the output of N(0, 1) rows in fp32,
# worst case: 128 products of 2^-24 each on sum |q k| <= 128 * 0.65, times max |v|
TOL, LSE_TOL = 5e-4, 2e-4


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_kv_attention_14_gb300 import build
    B.load(build.build())


def _run(b, caches, lens):
    c = b.meta["cascade"]
    gs, pre = c["query_start_loc"], c["prefix_lens"]
    S, t = lens.shape[0], b.block_tables_decode
    out = torch.full((S, b.num_q_heads, b.head_dim), float("nan"), device=DEV)
    lse = torch.full((S, b.num_q_heads), float("nan"), device=DEV)
    d = H.desc_of(b)
    mg = int((gs[1:] - gs[:-1]).max())
    B.pa_decode_shared(d, out, b.q_decode, caches[0], caches[1], t, lens, t.shape[1] * 16, gs, pre, mg, int(pre.max()),
                       b.scale, B.decode_shared_workspace(d, S, pre.shape[0], mg), lse=lse)
    torch.cuda.synchronize()
    return out, lse


NONFINITE = {  # (NaN, infinity) of each cache type
    W.KV_BF16: (float("nan"), float("inf")), W.KV_F16: (float("nan"), float("-inf")),
    W.KV_FP8: (0x7F, 0xFF),  # (no infinity: NaN of either sign)
    W.KV_FP8_E5M2: (0x7E, 0x7C),
}


@pytest.mark.parametrize("kv", list(NONFINITE))
@pytest.mark.parametrize("groups,plens,Hq,Hkv,D,short", [
    ([7], [96], 8, 2, 128, [0, 1, 37, 48]),        # a narrow item; nothing, one token, inside a block, at a block's end
    ([3, 12], [64, 4096], 32, 8, 128, [33, 2050]),  # 48 rows on a prefix cut between CTAs
    ([40], [1024], 16, 4, 64, [1023, 1009, 16]),    # 160 rows, two tiles, the last key missing
])
def test_tokens_past_a_sequences_end_do_not_reach_it(groups, plens, Hq, Hkv, D, short, kv):
    """Some sequences end inside the prefix that others of their group read on.
    What the cache holds past their ends, NaN and infinity in K or in V, is the
    others' business."""
    S = sum(groups)
    b = W.shared_prefix_decode(900 + S, groups, plens, [3 * i % 41 + 1 for i in range(S)], Hq, Hkv, D, kv_dtype=kv,
                               device=DEV, poison=False)
    caches = H.gpu_caches(b)
    lens = b.context_lens_decode.clone()
    first = S - groups[-1]  # the last group's sequences: every other one is a short one
    ends = {first + 2 * i: n for i, n in enumerate(short)}
    for s, n in ends.items():
        lens[s] = n
    b.context_lens_decode = lens
    good = _run(b, caches, lens)
    live = [s for s in range(S) if int(lens[s]) > 0]
    pairs = [(s, h) for s in live for h in range(Hq)]
    o, x = H.oracle_decode(b, ocaches=H.oracle_caches(b), pairs=pairs)
    H.assert_close(good[0][live].reshape(-1, D), o, TOL, "out")
    H.assert_close(good[1][live].reshape(-1), x, LSE_TOL, "lse")
    for s, n in ends.items():
        if n == 0:
            assert (good[0][s] == 0).all() and (good[1][s] == float("-inf")).all()
    # the tokens from the longest short sequence's end to the prefix's end
    at = torch.arange(max(short), plens[-1], device=DEV)
    blk = b.block_tables_decode[first].long()[at // 16]
    reads = torch.tensor([int(lens[s]) > max(short) and s >= first for s in range(S)], device=DEV)
    for which in (0, 1):
        for value in NONFINITE[kv]:
            c = [t.clone() for t in caches]
            c[which][blk, :, at % 16, D // 2 + 3] = value
            out, lse = _run(b, c, lens)
            assert torch.equal(out[~reads], good[0][~reads]) and torch.equal(lse[~reads], good[1][~reads])
            if which == 1:  # one column of V, for those who read it
                assert not torch.isfinite(out[reads][:, :, D // 2 + 3]).any()
                keep = torch.arange(D, device=DEV) != D // 2 + 3
                assert torch.equal(out[reads][:, :, keep], good[0][reads][:, :, keep])
