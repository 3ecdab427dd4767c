"""Calls of pa_prompt_attention and MixedStep.prompts that the documentation allows."""
import math

import pytest
import torch

from paged_kv_attention_14_gb300 import binding as pa
from paged_kv_attention_14_gb300.step import MixedStep
from test_gpu_prompt import DEV, KIND, U, _check, _rows, _want

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("longest", [101, 8192, 2 ** 31 - 1])
def test_any_bound_of_the_lengths(longest):
    lens, hq, hkv, d = [30, 70], 8, 2, 64
    q, k, v, starts = _rows(lens, hq, hkv, d, torch.bfloat16, 1)
    out = torch.zeros((100, hq, d), dtype=torch.bfloat16, device=DEV)
    lse = torch.zeros((100, hq), device=DEV)
    desc = pa.make_desc(0, hkv, hq, d)
    pa.pa_prompt_attention(desc, out, q, k, v, starts, longest, 1 / math.sqrt(d), lse=lse)
    _check(out, lse, _want(q, k, v, lens, 1 / math.sqrt(d)), torch.bfloat16)
    again = torch.zeros_like(out)
    kc, vc = [torch.zeros((8, hkv, 16, d), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    MixedStep(desc, kc, vc, 1 / math.sqrt(d)).prompts(again, q, k, v, starts, longest)
    assert torch.equal(again, out)


def test_what_a_step_of_prompts_writes_is_dense():
    lens, hq, hkv, d = [20, 12], 4, 2, 64
    q, k, v, starts = _rows(lens, hq, hkv, d, torch.bfloat16, 2)  # slices of a projection
    kc, vc = [torch.zeros((4, hkv, 16, d), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    step = MixedStep(pa.make_desc(4, hkv, hq, d), kc, vc, 0.125)
    slots = torch.arange(32, device=DEV)
    out, want = [torch.zeros((32, hq, d), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    for bad in ((k, v.contiguous()), (k.contiguous(), v)):
        with pytest.raises(ValueError, match="contiguous"):
            step.prompts(out, q, *bad, starts, 20, slots)
    step.prompts(want, q, k, v, starts, 20)
    step.prompts(out, q, k.contiguous(), v.contiguous(), starts, 20, slots)
    assert torch.equal(out, want)
    assert torch.equal(kc.transpose(1, 2).reshape(64, hkv, d)[:32], k)
    # rotated, only v has to be dense
    rot = [torch.empty((32, h, d), dtype=torch.bfloat16, device=DEV) for h in (hq, hkv)]
    pos = torch.arange(32, dtype=torch.int32, device=DEV)
    step.prompts(out, q, k, v.contiguous(), starts, 20, slots, rope=pa.make_rope(pa.rope_table(64, d)), positions=pos,
                 q_rot=rot[0], k_rot=rot[1])
    assert torch.equal(kc.transpose(1, 2).reshape(64, hkv, d)[:32], rot[1])


@pytest.mark.parametrize("act", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (4, 2, 64), (5, 1, 128), (16, 1, 64)])
@pytest.mark.parametrize("lens,local", [([1, 7, 16, 5], {}), ([300, 0, 129], {}), ([257, 256], dict(sliding_window=90)),
                                        ([290], dict(attention_chunk=100))])
@pytest.mark.parametrize("impl", [pa.PA_PREFILL_TCGEN05_PAIR, pa.PA_PREFILL_MMA_SYNC])
def test_weights_as_a_pair(act, hq, hkv, d, lens, local, impl):
    """The weights then carry 16 bits (bf16: half a step of the low half is 2^-17 of them) or 22 (fp16, but for at most
    half its smallest step, 2^-25, a weight, against a sum of weights of at least 1): the output's own rounding, 2^-15 of
    the terms for fp32 as in test_gpu_prompt, and that."""
    q, k, v, starts = _rows(lens, hq, hkv, d, act, 31, pad=5)
    scale = 1 / math.sqrt(d)
    out, single, auto = [torch.full(q.shape, 7.0, dtype=act, device=DEV) for _ in range(3)]
    lse = torch.zeros(q.shape[:2], device=DEV)
    for o, i in ((out, impl), (single, pa.PA_PREFILL_TCGEN05), (auto, pa.PA_PREFILL_AUTO)):
        pa.pa_prompt_attention(pa.make_desc(0, hkv, hq, d, KIND[act], prefill_impl=i, **local), o, q, k, v, starts,
                               max(lens), scale, lse=lse if o is out else None)
    assert torch.equal(single, auto)
    n = sum(lens)
    o64, size, l64 = _want(q, k, v, lens, scale, local.get("sliding_window", 0), local.get("attention_chunk", 0))
    weights = 2.0 ** -17 * size if act == torch.bfloat16 else 2.0 ** -22 * size + max(lens) * 2.0 ** -25 * float(v[:n].abs().max())
    tol = U[act] * o64.abs() + 2.0 ** -15 * size + weights + torch.finfo(act).smallest_normal
    off = (out[:n].double() - o64).abs()
    assert (off <= tol).all(), f"off by {(off / tol).max():.2f} of the bound"
    torch.testing.assert_close(lse[:n].double(), l64, rtol=0, atol=5e-5)
    assert (out[n:] == 7).all()
    if n > 100:  # (a few tokens may round the same way)
        assert (out[:n].double() - o64).norm() < (single[:n].double() - o64).norm()


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (4, 4, 64)])
def test_a_pair_of_weights_and_rows_that_are_not_finite(hq, hkv, d):
    lens = [60, 290]
    q, k, v, starts = _rows(lens, hq, hkv, d, torch.bfloat16, 32)
    v[60 + 200, 0, 5], v[30, hkv - 1, 9] = float("nan"), float("inf")
    outs = [torch.zeros(q.shape, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    for out, impl in zip(outs, (pa.PA_PREFILL_AUTO, pa.PA_PREFILL_TCGEN05_PAIR)):
        pa.pa_prompt_attention(pa.make_desc(0, hkv, hq, d, prefill_impl=impl), out, q, k, v, starts, 290, 0.1)
    assert torch.equal(*(torch.isfinite(x) for x in outs)) and not torch.isfinite(outs[0]).all()
