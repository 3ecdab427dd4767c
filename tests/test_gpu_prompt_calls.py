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
