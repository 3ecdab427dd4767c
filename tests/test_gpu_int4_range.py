"""Decode over 4-bit pages whose scales and minima lie far apart or have any sign, compared in 64 bits with what the
pages read as.

Tolerances: each group of 64 dims of an output against its own values, 5e-5 of the largest (see test_gpu_int4).
"""
import pytest
import torch

import int4_reference as ref
from paged_kv_attention_14_gb300 import binding as pa
from test_gpu_int4 import DEV, TOL, Batch

pytestmark = pytest.mark.gpu


def _pairs(cache, d):
    """The (scale, minimum) pairs of a CPU cache as a writable fp16 view [blocks, heads, 16, d / 64, 2]."""
    return cache[..., 8 * d:].unflatten(-1, (16, -1)).view(torch.float16).unflatten(-1, (-1, 2))


def _run(b):
    for n in ("kc", "vc", "q"):
        b.dev[n] = getattr(b, n).to(DEV)
    b.out.fill_(float("nan"))
    b.run()
    return b.out.cpu().double(), b.lse.cpu().double()


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (16, 2, 64), (16, 1, 128), (5, 1, 64)])
@pytest.mark.parametrize("which", ["all", "every second row"])
def test_scales_of_either_sign(hq, hkv, d, which):
    b = Batch([700, 33, 16, 1], hq, hkv, d, pa.PA_KV_INT4, seed=21)
    for c in (b.kc, b.vc):
        # the same values: codes 15 - n, scale -s, minimum m + 15 s (rounded)
        rows = slice(None, None, 1 if which == "all" else 2)
        p = _pairs(c, d)
        top = (p[..., 1].float() + 15 * p[..., 0].float()).half()
        p[:, :, rows, :, 0] = -p[:, :, rows, :, 0]
        p[:, :, rows, :, 1] = top[:, :, rows]
        codes = c[..., :8 * d].unflatten(-1, (16, -1))
        codes[:, :, rows] = 255 - codes[:, :, rows]
    out, lse = _run(b)
    want, wlse = b.want()
    torch.testing.assert_close(out, want, rtol=0, atol=TOL * b.vmax)
    torch.testing.assert_close(lse, wlse, rtol=0, atol=TOL)


def _size(b):
    """[sequences, heads, groups]: per group of 64 dims, the sum over the tokens of weight x (15 |scale| + |minimum|)."""
    d, hkv = b.d, b.kc.shape[1]
    S, hq, _ = b.q.shape
    size = torch.zeros((S, hq, d // 64), dtype=torch.float64)
    for s in range(S):
        L = int(b.lens[s])
        if L == 0:
            continue
        at = b.tables[s, :(L + 15) // 16].long()
        k = ref.rows_of(b.kc[at], d).permute(1, 0, 2, 3).reshape(hkv, -1, d)[:, :L]
        p = _pairs(b.vc, d)[at].double().permute(1, 0, 2, 3, 4).reshape(hkv, -1, d // 64, 2)[:, :L].abs()
        x = b.q[s].double().view(hkv, hq // hkv, d) @ k.transpose(1, 2) * b.scale
        size[s] = (torch.softmax(x, -1) @ (15 * p[..., 0] + p[..., 1])).reshape(hq, -1)
    return size


def _check(b):
    """Each group of an output within 5e-5 of the sum of its terms' magnitudes: the weights' 2^-15.5 (test_gpu_int4), and
    for products of weight and scale far below the largest seen 2^-29 of that for each of at most 2^13 tokens: 2^-16."""
    out, lse = _run(b)
    want, wlse = b.want()
    off = (out - want).abs().unflatten(-1, (-1, 64)).amax(-1)
    tol = TOL * _size(b)
    assert (off <= tol).all(), f"off by {float((off / tol.clamp(min=1e-300)).max()):.2f} of the bound"
    torch.testing.assert_close(lse, wlse, rtol=0, atol=TOL)
    assert int(b.word) == 0


@pytest.mark.parametrize("hq,hkv", [(8, 2), (16, 2), (16, 1)])
@pytest.mark.parametrize("kind", [pa.PA_KV_INT4, pa.PA_KV_INT4_F16])
@pytest.mark.parametrize("big", [0, 1])
def test_groups_with_scales_far_apart(hq, hkv, kind, big):
    b = Batch([700, 33, 2500, 1], hq, hkv, 128, kind, seed=22)
    p = _pairs(b.vc, 128)
    p[..., big, :] *= 2.0 ** 13
    p[..., 1 - big, :] *= 2.0 ** -10
    _check(b)


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (8, 1, 64), (16, 1, 128)])
@pytest.mark.parametrize("at", [0, 5, 300])
@pytest.mark.parametrize("low", [-20.0, -1.0])
def test_a_token_of_large_values_that_hardly_counts(hq, hkv, d, at, low):
    b = Batch([700, 1100], hq, hkv, d, pa.PA_KV_INT4, seed=23, vscale=1e-3)
    b.q = b.q.abs()
    for s in range(2):
        block, row = int(b.tables[s, at // 16]), at % 16
        _pairs(b.kc, d)[block, :, row] = torch.tensor([0.0, low]).half()
        _pairs(b.vc, d)[block, :, row] *= 2.0 ** 20
    assert torch.isfinite(ref.rows_of(b.vc, d)[b.tables[0, 0]]).all()
    _check(b)


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (8, 1, 64), (16, 1, 128), (4, 4, 64)])
@pytest.mark.parametrize("lens", [[900, 31, 0, 5], [8000]])
def test_scales_of_any_size_in_any_order(hq, hkv, d, lens):
    b = Batch(lens, hq, hkv, d, pa.PA_KV_INT4, seed=24, qscale=4.0)  # (scores of magnitude 20)
    g = torch.Generator().manual_seed(25)
    p = _pairs(b.vc, d)
    p *= torch.exp2(torch.randint(-11, 12, (*p.shape[:-1], 1), generator=g).float()).half()
    _check(b)


@pytest.mark.parametrize("d", [64, 128])
def test_widened_fp16_pages_of_the_largest_values_stay_finite(d):
    # 65504 + 65504 in 15 steps: the scale rounds to 8736, the top reads as 65536
    x = torch.zeros((2, 1, 16, d), dtype=torch.float16)
    x[..., 0::64], x[..., 1::64], x[..., 2::64] = -65504.0, 65504.0, 100.0
    x[1] = -x[1]
    x[1, 0, 3, 5] = float("nan")
    cache = ref.cache_of(x)
    assert ref.rows_of(cache, d).nan_to_num(0.0).max() == 65536.0
    ids = torch.arange(2, dtype=torch.int32, device=DEV)
    ko, vo = [torch.zeros((2, 1, 16, d), dtype=torch.float16, device=DEV) for _ in range(2)]
    pa.pa_widen_blocks(pa.make_desc(2, 1, 1, d, pa.PA_KV_INT4_F16), cache.to(DEV), cache.to(DEV), ids, ko, vo, ids)
    want = ref.rows_of(cache, d).clamp(-65504.0, 65504.0).half()  # (a NaN stays one)
    for got in (ko.cpu(), vo.cpu()):
        assert torch.equal(got.isnan(), want.isnan()) and bool(want.isnan().any())
        assert torch.equal(got.nan_to_num(0.0), want.nan_to_num(0.0))
