"""Calls of pa_prompt_attention and MixedStep.prompts that the documentation allows."""
import math

import pytest
import torch

from paged_kv_attention_14_gb300 import binding as pa
from paged_kv_attention_14_gb300.step import MixedStep
from test_gpu_prompt import DEV, _check, _rows, _want

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
