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
