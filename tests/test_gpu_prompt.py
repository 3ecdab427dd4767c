"""Causal attention of packed prompts from their own rows, against 64 bits.

Tolerance of an output element o = sum_j p_j v_j: the weights are rounded to the
activation type (half a step u of it, 2^-8 for bf16, 2^-11 for fp16, each
relative), the result once more: u (sum_j p_j |v_j| + |o|).  The rest is fp32
(exponents of at most about 64 rounded to 2^-18, an exponential off by 2^-22):
2^-15 sum_j p_j |v_j| on top, and half the smallest step of the type.  lse:
2^-15 of its own exponent range, 5e-5.
"""
import math

import pytest
import torch

from paged_kv_attention_14_gb300 import binding as pa
from paged_kv_attention_14_gb300.step import GraphedStep

pytestmark = pytest.mark.gpu
DEV = "cuda"
KIND = {torch.bfloat16: pa.PA_KV_BF16, torch.float16: pa.PA_KV_F16}
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def _first(pos, window, chunk):
    lo = (pos - window + 1).clamp(min=0) if window else torch.zeros_like(pos)
    return torch.maximum(lo, pos // chunk * chunk) if chunk else lo


def _want(q, k, v, lens, scale, window=0, chunk=0):
    """(out, sum of p |v|, lse) of the prompts' rows in 64 bits."""
    T, hq, d = sum(lens), q.shape[1], q.shape[2]
    g = hq // k.shape[1]
    out = torch.zeros((T, hq, d), dtype=torch.float64, device=q.device)
    size, lse = torch.zeros_like(out), torch.zeros((T, hq), dtype=torch.float64, device=q.device)
    at = 0
    for n in lens:
        i, j = torch.arange(n, device=q.device)[:, None], torch.arange(n, device=q.device)[None, :]
        hidden = (j > i) | (j < _first(i, window, chunk))
        for h in range(hq):
            rows = slice(at, at + n)
            x = (q[rows, h].double() @ k[rows, h // g].double().T * scale).masked_fill(hidden, -math.inf)
            p = torch.softmax(x, -1)
            vv = v[rows, h // g].double()
            out[rows, h], size[rows, h] = p @ vv, p @ vv.abs()
            lse[rows, h] = torch.logsumexp(x, -1)
        at += n
    return out, size, lse


def _rows(lens, hq, hkv, d, act, seed, pad=0, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    T = sum(lens) + pad
    qkv = (torch.randn((T, (hq + 2 * hkv) * d), generator=g, device=DEV) * scale).to(act)
    q, k, v = qkv[:, :hq * d], qkv[:, hq * d:(hq + hkv) * d], qkv[:, (hq + hkv) * d:]
    starts = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=DEV)
    return q.view(T, hq, d), k.view(T, hkv, d), v.view(T, hkv, d), starts


def _check(out, lse, want, act):
    o, size, l64 = want
    n = o.shape[0]
    off = (out[:n].double() - o).abs()
    tol = U[act] * (size + o.abs()) + 2.0 ** -15 * size + torch.finfo(act).smallest_normal
    assert (off <= tol).all(), f"off by {(off / tol).max():.2f} of the bound"
    if lse is not None:
        torch.testing.assert_close(lse[:n].double(), l64, rtol=0, atol=5e-5)


def _run(lens, hq, hkv, d, act, seed=0, pad=0, scale=None, **desc):
    q, k, v, starts = _rows(lens, hq, hkv, d, act, seed, pad)
    T = q.shape[0]
    out = torch.full((T, hq, d), 7.0, dtype=act, device=DEV)
    lse = torch.full((T, hq), 7.0, device=DEV)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    dsc = pa.make_desc(0, hkv, hq, d, KIND[act], error_word=word, **desc)
    pa.pa_prompt_attention(dsc, out, q, k, v, starts, max(lens), scale, lse=lse)
    want = _want(q, k, v, lens, scale, desc.get("sliding_window", 0), desc.get("attention_chunk", 0))
    _check(out, lse, want, act)
    assert int(word) == 0
    n = sum(lens)
    assert (out[n:] == 7).all() and (lse[n:] == 7).all()  # rows behind the last prompt


HEADS = [(4, 2, 64), (32, 8, 128), (5, 1, 128), (16, 1, 64), (3, 3, 128), (12, 2, 64), (7, 1, 64)]


@pytest.mark.parametrize("act", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("lens", [[1], [1, 7, 16, 33], [0, 5, 0, 0, 130, 0], [127, 128, 129], [300]])
def test_prompts(act, hq, hkv, d, lens):
    _run(lens, hq, hkv, d, act, seed=len(lens), pad=3)


@pytest.mark.parametrize("act,hq,hkv,d", [(torch.bfloat16, 8, 2, 128), (torch.float16, 4, 4, 64),
                                          (torch.bfloat16, 6, 1, 128), (torch.bfloat16, 2, 2, 128)])
@pytest.mark.parametrize("lens", [[1111], [2048, 1, 900], [257] * 9])
def test_longer_prompts(act, hq, hkv, d, lens):
    _run(lens, hq, hkv, d, act, seed=3, pad=200)


def test_many_short_prompts_beside_a_long_one():
    # the items are then packed instead of laid out by position
    g = torch.Generator().manual_seed(4)
    lens = torch.randint(0, 40, (300,), generator=g).tolist()
    lens[77], lens[201] = 1500, 700
    _run(lens, 4, 2, 64, torch.bfloat16, seed=4, check_indices=True)


@pytest.mark.parametrize("local", [dict(sliding_window=1), dict(sliding_window=70), dict(sliding_window=200),
                                   dict(attention_chunk=96), dict(attention_chunk=64, sliding_window=40),
                                   dict(attention_chunk=1000)])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (2, 2, 64), (16, 1, 128)])
def test_local_layers(local, hq, hkv, d):
    _run([5, 700, 1301], hq, hkv, d, torch.bfloat16, seed=5, **local)


@pytest.mark.parametrize("scale", [0.0, -0.1, 1.0])
def test_scales(scale):
    _run([200, 90], 4, 2, 64, torch.float16, seed=6, scale=scale)


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (2, 2, 64)])
@pytest.mark.parametrize("local", [dict(), dict(sliding_window=150), dict(attention_chunk=200)])
def test_rows_that_are_not_finite(hq, hkv, d, local):
    """NaN and infinities in k and v reach the tokens that see them and no others."""
    lens = [70, 300, 40]
    act = torch.bfloat16
    q, k, v, starts = _rows(lens, hq, hkv, d, act, 8, pad=130)
    v[370 + 40:] = float("nan")       # rows behind the last prompt
    k[370 + 40:] = float("nan")
    bad = [(70 + 250, 0, float("nan")), (70 + 90, hkv - 1, float("inf")), (30, 0, -float("inf"))]
    for tok, h, x in bad:
        v[tok, h, 3] = x
    k[70 + 280, 0] = float("nan")
    out = torch.zeros((q.shape[0], hq, d), dtype=act, device=DEV)
    lse = torch.zeros((q.shape[0], hq), device=DEV)
    pa.pa_prompt_attention(pa.make_desc(0, hkv, hq, d, pa.PA_KV_BF16, **local), out, q, k, v, starts, 300,
                           1 / math.sqrt(d), lse=lse)
    window, chunk = local.get("sliding_window", 0), local.get("attention_chunk", 0)
    pos = torch.cat([torch.arange(n, device=DEV) for n in lens])
    base = torch.cat([torch.full((n,), sum(lens[:i]), device=DEV) for i, n in enumerate(lens)])
    tok = pos + base
    first = _first(pos, window, chunk) + base
    end = torch.cat([torch.full((n,), sum(lens[:i + 1]), device=DEV) for i, n in enumerate(lens)])
    g = hq // hkv
    for h in range(hq):
        sees = lambda j: (first <= j) & (j <= tok) & (j < end) & (base <= j)  # noqa: E731
        nan_k = sees(350) if h // g == 0 else torch.zeros_like(tok, dtype=torch.bool)
        for d3 in (3, 4):
            x = out[:410, h, d3].float()
            hit = nan_k.clone()
            for j, kvh, _ in bad:
                if d3 == 3 and kvh == h // g:
                    hit |= sees(j)
            assert torch.equal(~torch.isfinite(x), hit)
        assert torch.equal(lse[:410, h].isnan(), nan_k)
    # tokens that see none of it are what they are without it
    v2, k2 = v.nan_to_num(0.0, 0.0, 0.0), k.nan_to_num(0.0)
    want = _want(q[:410], k2[:410], v2[:410], lens, 1 / math.sqrt(d), window, chunk)
    fine = torch.isfinite(out[:410]).all(-1)
    tol = U[act] * (want[1] + want[0].abs()) + 2.0 ** -15 * want[1]
    assert ((out[:410].double() - want[0]).abs() <= tol)[fine].all()


def test_large_values_and_a_rising_maximum():
    lens, hq, hkv, d = [600], 4, 1, 128
    q, k, v, starts = _rows(lens, hq, hkv, d, torch.bfloat16, 9)
    k *= (1 + torch.arange(600, device=DEV) / 60.0)[:, None, None].to(torch.bfloat16)  # scores grow along the keys
    out = torch.zeros((600, hq, d), dtype=torch.bfloat16, device=DEV)
    pa.pa_prompt_attention(pa.make_desc(0, hkv, hq, d), out, q, k, v, starts, 600, 1 / math.sqrt(d))
    _check(out, None, _want(q, k, v, lens, 1 / math.sqrt(d)), torch.bfloat16)


def test_on_another_stream_captured_and_the_same_twice():
    lens, hq, hkv, d = [333, 64, 1000], 8, 2, 128
    q, k, v, starts = _rows(lens, hq, hkv, d, torch.bfloat16, 10)
    out = torch.zeros((q.shape[0], hq, d), dtype=torch.bfloat16, device=DEV)
    lse = torch.zeros((q.shape[0], hq), device=DEV)
    desc = pa.make_desc(0, hkv, hq, d)
    run = lambda: pa.pa_prompt_attention(desc, out, q, k, v, starts, 1000, 1 / math.sqrt(d), lse=lse)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    first = out.clone(), lse.clone()
    graph = GraphedStep(run)
    q.copy_(q.flip(0))
    graph()
    want = _want(q, k, v, lens, 1 / math.sqrt(d))
    _check(out, lse, want, torch.bfloat16)
    q.copy_(q.flip(0))
    graph()
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


def test_two_calls_at_once_and_beside_other_tensor_memory():
    """Prompts on two streams, of the large and the small kind, and a chunked prefill between them."""
    big, small = _rows([900, 300], 8, 2, 128, torch.bfloat16, 13), _rows([30] * 90, 8, 2, 128, torch.bfloat16, 14)
    desc = pa.make_desc(8, 2, 8, 128)
    outs = [torch.zeros(x[0].shape, dtype=torch.bfloat16, device=DEV) for x in (big, small)]
    kc, vc = [torch.randn((8, 2, 16, 128), device=DEV).to(torch.bfloat16) for _ in range(2)]
    pf = torch.zeros((64, 8, 128), device=DEV)
    pq = small[0][:64].contiguous()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    table, lens, loc = torch.arange(8, dtype=torch.int32, device=DEV)[None], i32(128), i32(0, 64)
    torch.cuda.synchronize()
    for _ in range(10):
        for (q, k, v, starts), out, longest, st in zip((big, small), outs, (900, 30), streams):
            pa.pa_prompt_attention(desc, out, q, k, v, starts, longest, 0.1, stream=st)
        pa.pa_prefill_chunk(desc, pf, pq, loc, kc, vc, table, lens, 64, 128, 0.1, stream=streams[0])
    torch.cuda.synchronize()
    for (q, k, v, _), out, lens in zip((big, small), outs, ([900, 300], [30] * 90)):
        _check(out, None, _want(q, k, v, lens, 0.1), torch.bfloat16)


def test_checked_starts():
    q, k, v, _ = _rows([100], 2, 1, 64, torch.bfloat16, 11)
    out = torch.zeros((100, 2, 64), dtype=torch.bfloat16, device=DEV)
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    desc = pa.make_desc(0, 1, 2, 64, error_word=word, check_indices=True)
    for starts, longest, bad in (([0, 40, 100], 60, 0), ([0, 101], 100, 1), ([-1, 100], 100, 1), ([0, 60, 50, 100], 60, 1),
                                 ([0, 100], 99, 1), ([10, 10, 90], 80, 0)):
        word.zero_()
        pa.pa_prompt_attention(desc, out, q, k, v, torch.tensor(starts, dtype=torch.int32, device=DEV), longest, 0.1)
        assert (int(word) == pa.PA_DEVERR_BAD_INDEX) == bool(bad), starts


def test_waits_that_run_out_are_reported():
    q, k, v, starts = _rows([300, 20], 4, 2, 128, torch.bfloat16, 12)
    out = torch.zeros((320, 4, 128), dtype=torch.bfloat16, device=DEV)
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    desc = pa.make_desc(0, 2, 4, 128, error_word=word)
    pa.pa_test_stall_pipelines(True, 2_000_000)
    try:
        pa.pa_prompt_attention(desc, out, q, k, v, starts, 300, 0.1)
        torch.cuda.synchronize()
    finally:
        pa.pa_test_stall_pipelines(False)
    assert int(word) == pa.PA_DEVERR_WAIT_TIMEOUT
    word.zero_()
    pa.pa_prompt_attention(desc, out, q, k, v, starts, 300, 0.1)
    assert int(word) == 0
    _check(out, None, _want(q, k, v, [300, 20], 0.1), torch.bfloat16)
