"""Values that are not finite in batches of many prompts: a CTA works through several items one after the other, and a
row of v that is not finite reaches the tokens that see it and no others, whatever the items before and behind it hold.

Which outputs are finite is compared exactly; the finite ones against 64 bits without the bad rows, with the tolerance
of test_gpu_prompt.
"""
import math

import pytest
import torch

from paged_kv_attention_14_gb300 import binding as pa
from test_gpu_prompt import DEV, KIND, U, _first, _rows, _want

pytestmark = pytest.mark.gpu


def _check(lens, hq, hkv, d, bad, act=torch.bfloat16, times=5, seed=0, heads=None, **local):
    """bad: (token, kv head, dim, value) of v.  heads: the query heads looked at (default: all)."""
    q, k, v, starts = _rows(lens, hq, hkv, d, act, seed)
    clean = v.clone()
    for tok, h, x, val in bad:
        v[tok, h, x] = val
    T, g, scale = sum(lens), hq // hkv, 1 / math.sqrt(d)
    out = torch.zeros((T, hq, d), dtype=act, device=DEV)
    desc = pa.make_desc(0, hkv, hq, d, KIND[act], **local)
    first = None
    for _ in range(times):
        out.fill_(7)
        pa.pa_prompt_attention(desc, out, q, k, v, starts, max(lens), scale)
        if first is None:
            first = out.clone()
        assert torch.equal(out.nan_to_num(0.5, 0.25, 0.125), first.nan_to_num(0.5, 0.25, 0.125))
    window, chunk = local.get("sliding_window", 0), local.get("attention_chunk", 0)
    hit = torch.zeros((T, hkv, d), dtype=torch.bool, device=DEV)
    at = 0
    for n in lens:
        for tok, h, x, _ in bad:
            if at <= tok < at + n:
                i = torch.arange(n, device=DEV)
                hit[at:at + n, h, x] |= (i >= tok - at) & (_first(i, window, chunk) <= tok - at)
        at += n
    hit = hit.repeat_interleave(g, 1)
    assert torch.equal(~torch.isfinite(out), hit)
    # a bad row adds to dims in which it is finite what it adds without the bad ones
    heads = list(range(hkv)) if heads is None else heads
    qh = torch.cat([q[:, h * g:(h + 1) * g] for h in heads], 1)
    got = torch.cat([out[:, h * g:(h + 1) * g] for h in heads], 1)
    o, size, _ = _want(qh, k[:, heads], clean[:, heads], lens, scale, window, chunk)
    fine = torch.isfinite(got)
    tol = U[act] * (size + o.abs()) + 2.0 ** -15 * size
    assert ((got.double() - o).abs() <= tol)[fine].all()


def _some(lens, hkv, d, every, seed):
    """A bad value in every `every`-th prompt, at any place of it."""
    g = torch.Generator().manual_seed(seed)
    at, bad = 0, []
    for s, n in enumerate(lens):
        if s % every == 0:
            for _ in range(2):
                r = [int(torch.randint(0, m, (1,), generator=g)) for m in (n, hkv, d, 3)]
                bad.append((at + r[0], r[1], r[2], (float("nan"), float("inf"), -float("inf"))[r[3]]))
        at += n
    return bad


@pytest.mark.parametrize("hq,hkv,d", [(16, 4, 128), (16, 4, 64), (4, 4, 128)])
@pytest.mark.parametrize("rows", [128, 200, 256])  # one tile an item (two CTAs an SM), two tiles, two full ones
@pytest.mark.parametrize("every", [1, 3])
def test_bad_rows_in_some_of_many_items(hq, hkv, d, rows, every):
    n = rows // (hq // hkv)
    lens = [n] * (304 if rows <= 128 else 152)  # four items of each CTA
    _check(lens, hq, hkv, d, _some(lens, hkv, d, every, seed=rows + every))


@pytest.mark.parametrize("hq,hkv,d", [(16, 4, 128), (8, 4, 64)])
def test_bad_rows_in_items_of_one_tile_beside_items_of_two(hq, hkv, d):
    # most items have rows in their first tile only, the second one's warps have
    # nothing to do for several items on end
    g = torch.Generator().manual_seed(d)
    lens = torch.randint(1, 24, (900,), generator=g).tolist()
    for s in range(0, 900, 90):
        lens[s] = 150
    _check(lens, hq, hkv, d, _some(lens, hkv, d, 2, seed=d), seed=1)


def _far(chunk, hkv, d, where):
    """A bad value in each of the tiles `where` (by number) of the first chunk, and one in the second chunk."""
    return [(128 * t + 5 + 3 * i, i % hkv, (7 * i) % d, float("nan")) for i, t in enumerate(where)] + [(chunk + 9, 0, 1, float("inf"))]


@pytest.mark.parametrize("act,hq,hkv,d", [(torch.bfloat16, 8, 2, 128), (torch.float16, 4, 4, 64)])
def test_bad_rows_in_more_partly_seen_tiles_than_have_masks(act, hq, hkv, d):
    # the item over the chunks' boundary sees all 41 tiles of the first chunk in part
    chunk = 40 * 128 + 20
    _check([3 * 128, chunk + 200], hq, hkv, d,
           [(384 + t, *rest) for t, *rest in _far(chunk, hkv, d, (0, 31, 33, 40))], act=act, times=2, seed=2,
           attention_chunk=chunk)


@pytest.mark.parametrize("every", [1, 1000])
def test_a_long_chunk_with_bad_rows_is_within_the_waits_limit(every):
    # 4 heads of 32768 keys behind the masks; every row of v bad, or a few
    hq, hkv, d, chunk = 4, 1, 128, 32768 + 100
    T = chunk + 60
    q, k, v, starts = _rows([T], hq, hkv, d, torch.bfloat16, 3)
    v[::every, :, ::2] = v[chunk, :, ::2] = float("nan")
    out = torch.zeros((T, hq, d), dtype=torch.bfloat16, device=DEV)
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    desc = pa.make_desc(0, hkv, hq, d, attention_chunk=chunk, error_word=word)
    pa.pa_prompt_attention(desc, out, q, k, v, starts, T, 1 / math.sqrt(d))
    assert int(word) == 0
    assert out[:, :, ::2].isnan().all() and torch.isfinite(out[:, :, 1::2]).all()
    rows = torch.tensor([chunk - 70, chunk - 1, chunk, T - 1], device=DEV)
    for h in range(hq):
        x = q[rows, h].double() @ k[:, 0].double().T / math.sqrt(d)
        j = torch.arange(T, device=DEV)
        x = x.masked_fill((j > rows[:, None]) | (j < rows[:, None] // chunk * chunk), -math.inf)
        p, vv = torch.softmax(x, -1), v[:, 0, 1::2].double()
        o, size = p @ vv, p @ vv.abs()
        tol = U[torch.bfloat16] * (size + o.abs()) + 2.0 ** -15 * size
        assert ((out[rows, h, 1::2].double() - o).abs() <= tol).all()
