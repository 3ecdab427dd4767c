"""pa_decode_shared against the fp64 oracle's plain decode over the whole
tables.  Slots no sequence may read hold NaN.

Tolerance.  A weight's relative error is the P pair's (2^-18 for bf16 hi + lo,
less for fp16), the exponential's (2^-22) and its score's: 128 products
summed in fp32, at worst 128 * 2^-24 * scale * sum |q k| * log2 e, and
sum |q k| <= 128 * 0.65 for N(0, 1) rows, so 9e-5.  The output is off by at
most that times max |v|, about 5: 5e-4.  The log-sum-exp is off by the
scores' error plus the sum's, 2e-4.  An 8-bit cache is widened exactly.
"""
import numpy as np
import pytest
import torch

import oracle
import pa_helpers as H
from paged_kv_attention_14_gb300 import binding as B
from paged_kv_attention_14_gb300 import workloads as W
from paged_kv_attention_14_gb300.step import GraphedStep, MixedStep

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL, LSE_TOL = 5e-4, 2e-4


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_kv_attention_14_gb300 import build
    B.load(build.build())


def _args(b):
    c = b.meta["cascade"]
    gs, pre = c["query_start_loc"], c["prefix_lens"]
    return gs, pre, int((gs[1:] - gs[:-1]).max()), int(pre.max())


def _run(b, caches, gs=None, pre=None, max_group=None, lens=None, tables=None, desc=None, out=None, lse=None, ws=None,
         scale=None, stream=None):
    g0, p0, mg, mp = _args(b)
    gs, pre = g0 if gs is None else gs, p0 if pre is None else pre
    lens = b.context_lens_decode if lens is None else lens
    tables = b.block_tables_decode if tables is None else tables
    S = lens.shape[0]
    d = desc or H.desc_of(b)
    out = torch.full((S, b.num_q_heads, b.head_dim), float("nan"), device=DEV) if out is None else out
    lse = torch.full((S, b.num_q_heads), float("nan"), device=DEV) if lse is None else lse
    ws = B.decode_shared_workspace(d, S, pre.shape[0], mg if max_group is None else max_group) if ws is None else ws
    B.pa_decode_shared(d, out, b.q_decode, caches[0], caches[1], tables, lens, tables.shape[1] * 16, gs, pre,
                       mg if max_group is None else max_group, int(pre.max()) if pre.numel() else 0,
                       b.scale if scale is None else scale, ws, lse=lse, stream=stream)
    torch.cuda.synchronize()
    return out, lse


def _check(b, out, lse, ocaches=None, rows=None, scale_tol=1.0):
    S, Hq, D = b.q_decode.shape
    rows = list(range(S)) if rows is None else rows
    pairs = [(s, h) for s in rows for h in range(Hq)]
    o, x = H.oracle_decode(b, ocaches=ocaches, pairs=pairs)
    H.assert_close(out[rows].reshape(-1, D), o.reshape(-1, D), TOL * scale_tol, "out")
    H.assert_close(lse[rows].reshape(-1), x, LSE_TOL * scale_tol, "lse")


KV = [W.KV_BF16, W.KV_F16, W.KV_FP8, W.KV_FP8_E5M2]
CASES = [
    # (group sizes, prefix lens, own lens, q heads, kv heads, head_dim)
    ([3, 1], [32, 0], [1, 33, 7, 16], 4, 2, 64),
    ([1], [16], [5], 8, 1, 128),
    ([2], [16], [1, 1], 4, 4, 128),
    ([3, 1, 2], [48, 32, 64], [1, 15, 16, 40, 7, 33], 8, 2, 128),       # 12 rows, a single, 8 rows
    ([5, 2], [256, 0], [3, 100, 17, 1, 64, 9, 250], 32, 8, 128),        # 20 rows: two row groups; nothing shared
    ([9, 7], [160, 1040], list(range(1, 17)), 40, 8, 128),              # 45 and 35 rows, g 5
    ([17], [2048], [11 * i + 1 for i in range(17)], 32, 8, 64),         # 68 rows: eight row groups
    ([33, 3], [512, 4096], [37 * i % 300 + 1 for i in range(36)], 16, 4, 128),   # 132 rows: two tiles
    ([9], [400], [i + 1 for i in range(9)], 16, 1, 128),                # g 16: 144 rows of one kv head
    ([40], [96], [3] * 40, 5, 1, 128),                                  # g 5: tiles of 125 rows at most
]


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("groups,plens,slens,Hq,Hkv,D", CASES)
def test_matches_the_oracle(groups, plens, slens, Hq, Hkv, D, kv):
    b = W.shared_prefix_decode(700 + sum(plens) + D, groups, plens, slens, Hq, Hkv, D, kv_dtype=kv, device=DEV)
    _check(b, *_run(b, H.gpu_caches(b)), ocaches=H.oracle_caches(b))


@pytest.mark.parametrize("kv", [W.KV_BF16, W.KV_FP8])
def test_wide_group_on_a_long_prefix(kv):
    """64 sequences on 16384 tokens: 256 rows per kv head, items cut between many CTAs; sampled rows."""
    g = torch.Generator().manual_seed(8)
    slens = torch.randint(1, 300, (64,), generator=g).tolist()
    b = W.shared_prefix_decode(801, [64], [16384], slens, 32, 8, 128, kv_dtype=kv, device=DEV)
    _check(b, *_run(b, H.gpu_caches(b)), ocaches=H.oracle_caches(b), rows=[0, 1, 31, 32, 63])


def test_two_sequences_on_a_very_long_prefix():
    b = W.shared_prefix_decode(802, [2], [65536], [100, 1], 8, 2, 128, device=DEV)
    _check(b, *_run(b, H.gpu_caches(b)))


def test_the_error_does_not_grow_with_the_prefix():
    """131072 tokens, some 108 steps of 128 keys in a piece.  A product adds to
    the output truncated: half of 2^-23 |O| is lost on average, 0.72 of that
    over a binade, towards zero every time.  The output of a chain of 16 steps
    (256 products) grows as a random walk does, so the chain loses
    256 * 2/3 * 0.72 * 2^-24 = 7.3e-6 of its end value; P's pairs add 2^-18
    at most, independent from key to key: 1e-5 in the 2-norm.  (Without chains
    the same sum over 1728 products is 4.9e-5.)"""
    b = W.shared_prefix_decode(827, [8], [131072], [20, 60, 100, 140, 180, 220, 260, 300], 32, 8, 128, device=DEV)
    out, _ = _run(b, H.gpu_caches(b))
    o, _ = H.oracle_decode(b, pairs=[(3, h) for h in range(32)])
    e = out[3].double().cpu().numpy() - o.reshape(32, 128)
    assert np.linalg.norm(e) <= 1e-5 * np.linalg.norm(o)


def test_rising_scores_over_many_chains():
    """Row maxima that rise by more than the raise threshold again and again,
    also between chains, so that the sums are scaled."""
    b = W.shared_prefix_decode(828, [3], [65536], [5, 6, 7], 8, 8, 64, device=DEV, poison=False)
    b.q_decode.zero_()
    b.q_decode[:, :, 0] = 1
    kc = b.k_pool.clone()
    kc[..., 0] = 0
    # the score in log2 units goes up by 12 every 4096 tokens, scattered below by the other columns' zeros
    up = torch.arange(4096, device=DEV) // 256 * (12 * 0.6931471805599453 / b.scale)
    kc[b.block_tables_decode[0, :4096].long(), :, :, 0] = up.to(kc.dtype)[:, None, None]
    b.k_pool = kc
    # scores up to 125 (130 of the derivation's 7.4 units are 18 times as many)
    _check(b, *_run(b, (kc, b.v_pool)), scale_tol=18.0)


def test_no_groups_is_a_plain_decode():
    b = W.shared_prefix_decode(803, [3, 2], [64, 32], [1, 40, 7, 300, 16], 32, 8, 128, device=DEV)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    out, lse = _run(b, H.gpu_caches(b), gs=torch.zeros(1, dtype=torch.int32, device=DEV), pre=none, max_group=0)
    _check(b, out, lse)


def test_groups_that_leave_sequences_out_and_prefixes_that_end_inside_a_block():
    """Group 0 starts at sequence 1, the last sequence belongs to none; a
    prefix of 16 n + 7 tokens is used up to its whole blocks; the largest
    group is twice what max_group_size says."""
    b = W.shared_prefix_decode(804, [6, 5], [96, 208], [9, 50, 1, 16, 33, 17, 8, 2, 300, 31, 90], 32, 8, 128, device=DEV)
    gs = torch.tensor([1, 6, 10], dtype=torch.int32, device=DEV)
    pre = torch.tensor([96 + 7, 208 + 15], dtype=torch.int32, device=DEV)
    _check(b, *_run(b, H.gpu_caches(b), gs=gs, pre=pre, max_group=3))


@pytest.mark.parametrize("kv", [W.KV_BF16, W.KV_FP8])
def test_empty_sequences_and_ones_shorter_than_their_prefix(kv):
    b = W.shared_prefix_decode(805, [6, 3, 4], [96, 32, 64], [9, 50, 1, 16, 33, 17, 5, 6, 7, 1, 2, 3, 4], 32, 8, 128,
                               kv_dtype=kv, device=DEV, poison=False)
    lens = b.context_lens_decode.clone()
    lens[0], lens[2], lens[3] = 0, 96, 37           # empty; exactly the prefix; inside it
    lens[6:9] = torch.tensor([0, 20, 1])            # nobody reaches the prefix's end
    lens[9:13] = 0                                  # a group of padding rows
    b.context_lens_decode = lens
    out, lse = _run(b, H.gpu_caches(b))
    empty = [0, 6, 9, 10, 11, 12]
    assert (out[empty] == 0).all() and (lse[empty] == float("-inf")).all()
    _check(b, out, lse, ocaches=H.oracle_caches(b), rows=[s for s in range(13) if s not in empty])


def test_padding_rows_read_nothing():
    """A group whose unread prefix slots hold NaN: all of its sequences but one are empty or shorter."""
    b = W.shared_prefix_decode(806, [4], [64], [1, 1, 1, 1], 8, 2, 128, device=DEV, poison=False)
    lens = torch.tensor([0, 21, 0, 5], dtype=torch.int32, device=DEV)
    kc, vc = b.k_pool.clone(), b.v_pool.clone()
    blk = int(b.block_tables_decode[1, 1])
    for c in (kc, vc):  # tokens 21 .. 31 of the prefix and its later blocks
        c[blk, :, 5:] = float("nan")
        for j in (2, 3):
            c[int(b.block_tables_decode[1, j])] = float("nan")
    b.context_lens_decode, b.k_pool, b.v_pool = lens, kc, vc
    out, lse = _run(b, (kc, vc))
    _check(b, out, lse, rows=[1, 3])
    assert (out[[0, 2]] == 0).all()


def test_rising_scores():
    """Scores that grow along the keys by far more than the raise threshold, up to hundreds."""
    b = W.shared_prefix_decode(807, [5, 1], [640, 0], [70, 3, 200, 1, 33, 500], 32, 8, 128, device=DEV, poison=False)
    kc = b.k_pool.float()
    for s in range(6):
        n = int(b.context_lens_decode[s])
        for j in range((n + 15) // 16):
            blk = int(b.block_tables_decode[s, j])
            if s in (0, 5) or j >= 40:
                kc[blk] *= 1 + 0.2 * j
    b.k_pool = kc.to(torch.bfloat16)
    # scores (and so their error) are up to 1 + 0.2 * 71 times those of the tolerance's derivation
    _check(b, *_run(b, (b.k_pool, b.v_pool)), scale_tol=16.0)


def test_one_far_larger_score_keeps_the_small_weights():
    """One key 2^18 times as heavy as each other one; the rest together still weigh: fp16 P must not lose them."""
    for kv in (W.KV_F16, W.KV_BF16):
        b = W.shared_prefix_decode(808, [4], [8192], [5, 6, 7, 8], 8, 2, 128, kv_dtype=kv, device=DEV, poison=False)
        b.q_decode.zero_()
        b.q_decode[:, :, 0] = 1
        kc = b.k_pool.clone()
        kc[..., 0] = 0
        kc[int(b.block_tables_decode[0, 3]), :, 4, 0] = 12.48 / b.scale  # e^12.48 = 2^18
        b.k_pool = kc
        _check(b, *_run(b, (kc, b.v_pool)))


def test_nan_and_infinity_stay_in_their_rows():
    b = W.shared_prefix_decode(809, [5], [160], [9, 50, 1, 16, 33], 32, 8, 128, device=DEV)
    good, _ = _run(b, H.gpu_caches(b))
    b.q_decode[2, 5, 3] = float("nan")
    b.q_decode[4, 31, 7] = float("inf")
    out, lse = _run(b, H.gpu_caches(b))
    bad = torch.zeros(5, 32, dtype=torch.bool, device=DEV)
    bad[2, 5] = bad[4, 31] = True
    assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
    assert torch.equal(out[~bad], good[~bad])


def test_same_bits_every_time_and_from_any_workspace():
    b = W.shared_prefix_decode(810, [20, 9], [2048, 304], [37 * i % 200 + 1 for i in range(29)], 32, 8, 128, device=DEV)
    caches = H.gpu_caches(b)
    a = _run(b, caches)
    n = B.pa_decode_shared_workspace_size(H.desc_of(b), 29, 2, 20)
    for fill in (0, 255):
        ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
        for _ in range(2):
            x = _run(b, caches, ws=ws)
            assert torch.equal(x[0], a[0]) and torch.equal(x[1], a[1])


def test_per_head_scales():
    b = W.random_decode(811, [40, 100, 7], 8, 4, 128, kv_dtype=W.KV_FP8, device=DEV, poison=True, per_head_scales=True)
    gs = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    b.meta["cascade"] = dict(query_start_loc=gs, prefix_lens=torch.zeros(1, dtype=torch.int32, device=DEV))
    out, lse = _run(b, H.gpu_caches(b))
    o, x = H.oracle_decode(b)
    # heads of magnitudes up to 2^2: the scores' and the values' errors scale by that
    H.assert_close(out, o, 4 * TOL, "out")
    H.assert_close(lse, x, 4 * LSE_TOL, "lse")
    # a shared block too: the second sequence's first block is the first one's
    t = b.block_tables_decode.clone()
    t[1, 0] = t[0, 0]
    b.block_tables_decode = t
    pre = torch.tensor([16], dtype=torch.int32, device=DEV)
    out, lse = _run(b, H.gpu_caches(b), gs=torch.tensor([0, 2], dtype=torch.int32, device=DEV), pre=pre)
    o, x = H.oracle_decode(b)
    H.assert_close(out, o, 4 * TOL, "out")


def test_checked_indices_are_reported_and_stay_inside():
    ew = torch.zeros(1, dtype=torch.int32, device=DEV)
    b = W.shared_prefix_decode(812, [4, 3], [64, 32], [9, 50, 1, 16, 33, 17, 5], 32, 8, 128, device=DEV, poison=False)
    caches = H.gpu_caches(b)
    d = B.make_desc(b.num_blocks, 8, 32, 128, error_word=ew, check_indices=True)
    out, lse = _run(b, caches, desc=d)
    assert int(ew) == 0
    _check(b, out, lse)
    gs, pre, _, _ = _args(b)
    for what in ("table", "len", "start", "prefix"):
        ew.zero_()
        t, n, g2, p2 = b.block_tables_decode.clone(), b.context_lens_decode.clone(), gs.clone(), pre.clone()
        if what == "table":
            t[0, 1], t[1, 1], t[2, 1], t[3, 1] = [b.num_blocks + 5] * 4
        elif what == "len":
            n[3] = t.shape[1] * 16 + 1
        elif what == "start":
            g2[1] = 70000
        else:
            p2[0] = -16
        B.pa_decode_shared(d, out, b.q_decode, caches[0], caches[1], t, n, t.shape[1] * 16, g2, p2, 4, 64, b.scale,
                           B.decode_shared_workspace(d, 7, 2, 4), lse=lse)
        torch.cuda.synchronize()
        assert int(ew) & B.PA_DEVERR_BAD_INDEX, what


def test_lengths_past_the_table_end_at_it():
    b = W.shared_prefix_decode(826, [3], [64], [48, 48, 33], 8, 2, 128, device=DEV, poison=False)
    b.context_lens_decode = torch.full_like(b.context_lens_decode, b.block_tables_decode.shape[1] * 16)
    want = _run(b, H.gpu_caches(b))
    b.context_lens_decode = b.context_lens_decode + torch.tensor([1, 1000, 2**31 - 1 - 200], dtype=torch.int32, device=DEV)
    out = _run(b, H.gpu_caches(b))
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_a_stalled_pipeline_is_reported_and_the_next_call_is_right():
    ew = torch.zeros(1, dtype=torch.int32, device=DEV)
    b = W.shared_prefix_decode(813, [20, 3], [512, 32], [9] * 23, 32, 8, 128, device=DEV)
    caches = H.gpu_caches(b)
    d = B.make_desc(b.num_blocks, 8, 32, 128, error_word=ew)
    try:
        B.pa_test_stall_pipelines(True)
        _run(b, caches, desc=d)
    finally:
        B._check(B.load().pa_test_stall_pipelines(0, 0))
    assert int(ew) == B.PA_DEVERR_WAIT_TIMEOUT
    ew.zero_()
    _check(b, *_run(b, caches, desc=d))
    assert int(ew) == 0


def test_graph_replay_with_other_lengths_and_two_streams_at_once():
    b = W.shared_prefix_decode(814, [7, 4], [128, 64], [37 * i % 100 + 1 for i in range(11)], 32, 8, 128, device=DEV)
    caches = H.gpu_caches(b)
    d = H.desc_of(b)
    gs, pre, mg, mp = _args(b)
    S = 11
    lens = b.context_lens_decode.clone()
    outs = [torch.zeros(S, 32, 128, device=DEV) for _ in range(3)]
    wss = [B.decode_shared_workspace(d, S, 2, mg) for _ in range(3)]
    maxL = b.block_tables_decode.shape[1] * 16

    def issue(i, n, stream=None):
        B.pa_decode_shared(d, outs[i], b.q_decode, caches[0], caches[1], b.block_tables_decode, n, maxL, gs, pre, mg,
                           mp, b.scale, wss[i], stream=stream)

    step = GraphedStep(lambda: issue(0, lens))
    lens.copy_(torch.clamp(lens - 20, min=1))  # the plan is made anew at every replay
    step()
    full = b.context_lens_decode
    b.context_lens_decode = lens
    o, _ = H.oracle_decode(b)
    H.assert_close(outs[0], o, TOL, "replay")
    b.context_lens_decode = full
    want, _ = _run(b, caches)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, st in enumerate(streams):
            issue(1 + i, full, st)
    torch.cuda.synchronize()
    assert torch.equal(outs[1], want) and torch.equal(outs[2], want)


@pytest.mark.parametrize("kv", [W.KV_BF16, W.KV_F16, W.KV_FP8])
@pytest.mark.parametrize("scale", [-0.08, -1e-3, 0.0, 1e-39])
def test_scales_of_either_sign_and_zero(scale, kv):
    """Wide and narrow items.  A zero scale weighs every key alike."""
    b = W.shared_prefix_decode(819, [24, 2], [528, 64], [37 * i % 90 + 1 for i in range(26)], 32, 8, 128, kv_dtype=kv,
                               device=DEV)
    b.scale = scale
    _check(b, *_run(b, H.gpu_caches(b)), ocaches=H.oracle_caches(b), rows=[0, 5, 23, 24, 25])


@pytest.mark.parametrize("kv", [W.KV_BF16, W.KV_FP8])
@pytest.mark.parametrize("pairs,singles", [(256, 0), (256, 1), (600, 137)])
def test_many_sequences_and_groups(pairs, singles, kv):
    """More sequences, or groups, than one CTA plans from shared memory (512)."""
    S = 2 * pairs + singles
    b = W.shared_prefix_decode(820 + S, [2] * pairs + [1] * singles, [16 * (j % 4) for j in range(pairs)] + [0] * singles,
                               [13 * i % 37 + 1 for i in range(S)], 8, 2, 128, kv_dtype=kv, device=DEV)
    gs, pre, _, _ = _args(b)
    out, lse = _run(b, H.gpu_caches(b))
    _check(b, out, lse, ocaches=H.oracle_caches(b))
    # the singles in no group: the same
    out, lse = _run(b, H.gpu_caches(b), gs=gs[:pairs + 1], pre=pre[:pairs], max_group=2)
    _check(b, out, lse, ocaches=H.oracle_caches(b))


def test_many_empty_groups():
    """700 groups of which only every tenth has sequences."""
    b = W.shared_prefix_decode(821, [3] * 70, [48] * 70, [7 * i % 50 + 1 for i in range(210)], 8, 2, 64, device=DEV)
    gs = torch.tensor([3 * ((i + 9) // 10) for i in range(701)], dtype=torch.int32, device=DEV)
    pre = torch.full((700,), 48, dtype=torch.int32, device=DEV)
    _check(b, *_run(b, H.gpu_caches(b), gs=gs, pre=pre))


@pytest.mark.parametrize("max_group", [0, 1, 8, 1000])
def test_any_largest_group_size(max_group):
    """A bound below the largest group, and far above the batch."""
    b = W.shared_prefix_decode(829, [2, 1], [48, 0], [5, 40, 17], 8, 2, 128, device=DEV)
    _check(b, *_run(b, H.gpu_caches(b), max_group=max_group))


def test_the_largest_batch():
    """65535 sequences in 21845 groups of three; sampled rows, and the same rows as a batch of their own."""
    n = 21845
    b = W.shared_prefix_decode(830, [3] * n, [16 * (j % 3) for j in range(n)], [7 * i % 23 + 1 for i in range(3 * n)], 4, 2,
                               64, device=DEV)
    out, lse = _run(b, H.gpu_caches(b))
    _check(b, out, lse, rows=[0, 1, 2, 3, 511, 512, 513, 32767, 32768, 65531, 65532, 65533, 65534])
    ref = torch.empty_like(out)
    d = H.desc_of(b)
    B.pa_decode(d, ref, b.q_decode, *H.gpu_caches(b), b.block_tables_decode, b.context_lens_decode,
                b.max_context_len_decode(), b.scale, B.decode_workspace(d, 3 * n, b.max_context_len_decode()))
    torch.cuda.synchronize()
    assert float((out - ref).abs().max()) <= 2 * TOL


def test_one_stream_takes_batches_of_different_shapes_through_one_workspace():
    """Calls in a row, each with its own lengths and sizes, not waited for in between."""
    bs = [W.shared_prefix_decode(831 + i, g, p, s, 32, 8, 128, device=DEV) for i, (g, p, s) in enumerate([
        ([9, 7], [160, 1040], list(range(1, 17))), ([1], [0], [700]), ([40], [4096], [3 * i % 70 + 1 for i in range(40)])])]
    ws = B.decode_shared_workspace(H.desc_of(bs[2]), 40, 2, 40)
    outs = []
    for b in bs + bs[::-1]:
        gs, pre, mg, mp = _args(b)
        o = torch.empty_like(b.q_decode, dtype=torch.float32)
        B.pa_decode_shared(H.desc_of(b), o, b.q_decode, b.k_pool, b.v_pool, b.block_tables_decode, b.context_lens_decode,
                           b.block_tables_decode.shape[1] * 16, gs, pre, mg, mp, b.scale, ws)
        outs.append(o)
    torch.cuda.synchronize()
    for i, b in enumerate(bs):
        assert torch.equal(outs[i], outs[5 - i])
        _check(b, outs[i], _run(b, H.gpu_caches(b))[1])


def test_output_in_pinned_host_memory():
    b = W.shared_prefix_decode(815, [4, 1], [64, 0], [9, 50, 1, 16, 33], 32, 8, 128, device=DEV)
    caches = H.gpu_caches(b)
    want = _run(b, caches)
    out, lse = torch.zeros(5, 32, 128).pin_memory(), torch.zeros(5, 32).pin_memory()
    _run(b, caches, out=out, lse=lse)
    assert torch.equal(out, want[0].cpu()) and torch.equal(lse, want[1].cpu())


def test_queries_beyond_fp16_of_an_8bit_cache_are_reported():
    ew = torch.zeros(1, dtype=torch.int32, device=DEV)
    b = W.shared_prefix_decode(816, [3], [32], [5, 6, 7], 8, 2, 128, kv_dtype=W.KV_FP8, device=DEV, poison=False)
    caches = H.gpu_caches(b)
    d = B.make_desc(b.num_blocks, 2, 8, 128, B.PA_KV_FP8_E4M3, b.k_scale, b.v_scale, error_word=ew)
    _run(b, caches, desc=d)
    assert int(ew) == 0
    b.q_decode[1, 2, 3] = 1e5
    _run(b, caches, desc=d)
    assert int(ew) == B.PA_DEVERR_FP16_RANGE


@pytest.mark.parametrize("kv", [W.KV_FP8, W.KV_FP8_E5M2])
def test_every_finite_byte_of_an_8bit_cache(kv):
    """K and V of all the type's finite values, its subnormals among them.
    With the largest one, m, the scale is 1 / (4 m): the bytes' mean magnitude
    is some 0.13 m (E4M3; E5M2: less), so scale * sum |q k| is about 3, less
    than the tolerance's 7.  The output is compared in units of m."""
    b = W.shared_prefix_decode(824, [3, 1], [256, 0], [9, 300, 1, 40], 8, 2, 128, kv_dtype=kv, device=DEV, poison=False)
    t = torch.float8_e4m3fn if kv == W.KV_FP8 else torch.float8_e5m2
    val = torch.arange(256, dtype=torch.uint8).view(t).float()
    finite = torch.isfinite(val)
    top = float(val[finite].max())
    good = torch.arange(256, dtype=torch.uint8)[finite]
    g = torch.Generator().manual_seed(9)
    kc, vc = (good[torch.randint(0, len(good), tuple(b.k_pool.shape), generator=g)] for _ in range(2))
    b.k_scale, b.v_scale, b.scale = 1.0, 1.0, 0.25 / top
    out, lse = _run(b, (kc.to(DEV), vc.to(DEV)))
    code = H.oracle_caches(b)[0]
    o, x = H.oracle_decode(b, ocaches=(code, kc.numpy(), vc.numpy()))
    H.assert_close(out / top, o / top, TOL, "out")
    H.assert_close(lse, x, LSE_TOL, "lse")


@pytest.mark.parametrize("kv", [W.KV_FP8, W.KV_FP8_E5M2])
def test_nan_bytes_of_an_8bit_cache_reach_their_readers_only(kv):
    b = W.shared_prefix_decode(825, [3, 1], [256, 0], [9, 300, 1, 40], 8, 2, 128, kv_dtype=kv, device=DEV, poison=False)
    caches = H.gpu_caches(b)
    good, _ = _run(b, caches)
    blk = int(b.block_tables_decode[1, 17])  # of sequence 1's own part
    for which, byte in ((0, 0x7F), (1, 0xFF)):
        c = [x.clone() for x in caches]
        c[which][blk, 1, 3, 77] = byte
        out, _ = _run(b, c)
        bad = torch.zeros(4, 8, 128, dtype=torch.bool, device=DEV)
        bad[1, 4:, slice(None) if which == 0 else 77] = True
        assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], good[~bad])


def test_misuse_of_the_binding_is_refused():
    b = W.shared_prefix_decode(817, [3], [32], [5, 6, 7], 8, 2, 128, device=DEV)
    caches = H.gpu_caches(b)
    gs, pre, mg, mp = _args(b)
    with pytest.raises(ValueError, match="group_start"):
        _run(b, caches, gs=gs[:-1])
    with pytest.raises(ValueError, match="block_tables"):
        _run(b, caches, tables=b.block_tables_decode[:2])
    with pytest.raises(ValueError, match="num_blocks"):
        _run(b, (caches[0][:-1], caches[1]))
    with pytest.raises(B.PaError) as e:
        _run(b, caches, ws=torch.zeros(1024, dtype=torch.uint8, device=DEV))
    assert e.value.status == B.PA_ERR_WORKSPACE


def test_rotated_append_then_shared_decode():
    """The operators as a step uses them: q, k and v of a projection rotated and
    written into the cache, then attention over the shared prefix, the own
    part and the new token, against the oracle on a cache written by hand."""
    b = W.shared_prefix_decode(818, [6, 2], [160, 48], [9, 50, 1, 16, 33, 17, 5, 100], 32, 8, 128, device=DEV)
    S, Hq, Hkv, D = 8, 32, 8, 128
    g = torch.Generator().manual_seed(4)
    qkv = torch.randn(S, (Hq + 2 * Hkv) * D, generator=g).to(torch.bfloat16).to(DEV)
    q, k, v = (qkv[:, lo * D:hi * D].view(S, hi - lo, D) for lo, hi in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, 48)))
    w = (1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16).to(DEV)
    rope = B.make_rope(B.rope_table(512, D, 1e6, DEV), q_weight=w, k_weight=w)
    pos = (b.context_lens_decode - 1).to(torch.int32)
    at = pos.long()
    slots = b.block_tables_decode.gather(1, (at // 16)[:, None])[:, 0].long() * 16 + at % 16
    d = H.desc_of(b)
    kc, vc = b.k_pool.clone(), b.v_pool.clone()
    q_out = torch.empty(S, Hq, D, dtype=torch.bfloat16, device=DEV)
    B.pa_rope_cache_write(d, rope, q_out, q, k, v, pos, kc, vc, slots)
    b.q_decode = q_out
    out, lse = _run(b, (kc, vc))
    k_rot = torch.empty(S, Hkv, D, dtype=torch.bfloat16, device=DEV)
    B.pa_qk_norm_rope(d, rope, None, k_rot, None, k, pos)
    ok, ov = oracle.cache_write(oracle.KV_BF16, 16, Hkv, D, k_rot.cpu(), v.contiguous().cpu(), slots.cpu(),
                                b.k_pool.cpu(), b.v_pool.cpu())
    assert np.array_equal(kc.view(torch.int16).cpu().numpy().view(np.uint16), ok)
    _check(b, out, lse, ocaches=(oracle.KV_BF16, ok, ov))


@pytest.mark.parametrize("mode", ["fused", "streams", "serial"])
@pytest.mark.parametrize("grouped", [True, False])
def test_a_step_from_projections(mode, grouped):
    """MixedStep.projected: decode sequences and prefill chunks, captured and replayed with other inputs."""
    b = W.shared_prefix_decode(822, [5, 2], [160, 48], [9, 50, 1, 16, 33, 17, 100], 32, 8, 128, device=DEV)
    p = W.random_prefill(823, [70, 1, 40], [70, 33, 100], 32, 8, 128, device=DEV, poison=True)
    S, Tq, Hq, Hkv, D = 7, 111, 32, 8, 128
    # one pool: the chunks' blocks behind the decode sequences'
    kc, vc = (torch.cat([getattr(b, n), getattr(p, n)]) for n in ("k_pool", "v_pool"))
    ptab = torch.where(p.block_tables_prefill >= 0, p.block_tables_prefill + b.num_blocks, p.block_tables_prefill)
    d = B.make_desc(kc.shape[0], Hkv, Hq, D)
    gs, pre, mg, mp = _args(b)
    table = B.rope_table(512, D, 1e6, DEV)
    rope = B.make_rope(table)
    maxL = b.block_tables_decode.shape[1] * 16
    n = b.context_lens_decode - 1
    qsl, plen = p.query_start_loc.cpu(), p.context_lens_prefill.cpu()
    pos = torch.cat([n.cpu()] + [torch.arange(int(plen[i]) - int(qsl[i + 1] - qsl[i]), int(plen[i])) for i in range(3)])
    rows = torch.cat([b.block_tables_decode.cpu().gather(1, (n.cpu().long() // 16)[:, None])[:, 0]] + [
        ptab.cpu()[i, pos[S + int(qsl[i]):S + int(qsl[i + 1])].long() // 16] for i in range(3)])
    pos = pos.to(torch.int32)
    slots = (rows.long() * 16 + pos.long() % 16).to(DEV)
    pos = pos.to(DEV)
    qkv = torch.zeros(S + Tq, (Hq + 2 * Hkv) * D, dtype=torch.bfloat16, device=DEV)
    q, k, v = (qkv[:, lo * D:hi * D].view(-1, hi - lo, D) for lo, hi in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, 48)))
    ws = B.mixed_workspace(d, S, maxL, DEV)
    out, lse = torch.empty(S, Hq, D, device=DEV), torch.empty(S, Hq, device=DEV)
    pout, plse = torch.empty(Tq, Hq, D, device=DEV), torch.empty(Tq, Hq, device=DEV)
    step = MixedStep(d, kc, vc, b.scale, decode_out=out, decode_lse=lse, workspace=ws, max_context_len_decode=maxL,
                     prefill_out=pout, prefill_lse=plse, max_q_len=70, max_context_len_prefill=100, mode=mode,
                     shared_workspace=B.decode_shared_workspace(d, S, 2, mg) if grouped else None)
    q_rot = torch.empty(S + Tq, Hq, D, dtype=torch.bfloat16, device=DEV)
    groups = (gs, pre, mg, mp) if grouped else None

    def issue():
        step.projected(rope, q_rot, q, k, v, pos, slots, (b.block_tables_decode, b.context_lens_decode),
                       (p.query_start_loc, ptab, p.context_lens_prefill), groups)

    graph = GraphedStep(issue)
    before = kc.cpu(), vc.cpu()
    qkv.copy_(torch.randn(qkv.shape, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16))
    graph()
    k_rot = torch.empty(S + Tq, Hkv, D, dtype=torch.bfloat16, device=DEV)
    want_q = torch.empty_like(q_rot)
    B.pa_qk_norm_rope(d, rope, want_q, k_rot, q, k, pos)
    assert torch.equal(want_q, q_rot)
    ok, ov = oracle.cache_write(oracle.KV_BF16, 16, Hkv, D, k_rot.cpu(), v.contiguous().cpu(), slots.cpu(), *before)
    assert np.array_equal(kc.view(torch.int16).cpu().numpy().view(np.uint16), ok)
    b.q_decode = q_rot[:S]
    b.num_blocks = kc.shape[0]
    _check(b, out, lse, ocaches=(oracle.KV_BF16, ok, ov))
    o, x = oracle.prefill(oracle.KV_BF16, 16, Hkv, Hq, D, q_rot[S:].cpu(), qsl, ok, ov, ptab.cpu(), plen, b.scale)
    H.assert_close(pout.reshape(-1, D), o.reshape(-1, D), TOL, "prefill out")
    H.assert_close(plse.reshape(-1), x.reshape(-1), LSE_TOL, "prefill lse")
    if grouped:
        step.shared_workspace = None
        with pytest.raises(ValueError, match="shared_workspace"):
            issue()
