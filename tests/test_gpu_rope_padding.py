"""Padding tokens of pa_rope_cache_write with checked indices, and inputs the
binding must not hand on."""
import pytest
import torch

from paged_kv_attention_14_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
MAXP = 300


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_kv_attention_14_gb300 import build
    B.load(build.build())


@pytest.mark.parametrize("kv", [B.PA_KV_BF16, B.PA_KV_FP8_E4M3])
@pytest.mark.parametrize("tokens", [8, 2500])
def test_positions_of_padding_tokens_are_not_reported(tokens, kv):
    """A negative slot marks a padding token of a fixed-size step, whose
    position may hold anything; both kernels (8 and 2500 tokens)."""
    hq, hkv, d = 32, 8, 128
    g = torch.Generator().manual_seed(tokens)
    ew = torch.zeros(1, dtype=torch.int32, device=DEV)
    nb = tokens // 16 + 2
    desc = B.make_desc(nb, hkv, hq, d, kv, k_scale=0.02, v_scale=0.02, error_word=ew, check_indices=True) \
        if kv == B.PA_KV_FP8_E4M3 else B.make_desc(nb, hkv, hq, d, kv, error_word=ew, check_indices=True)
    rope = B.make_rope(B.rope_table(MAXP, d, device=DEV))
    q, k, v = (torch.randn(tokens, h, d, generator=g).to(torch.bfloat16).to(DEV) for h in (hq, hkv, hkv))
    pos = torch.randint(0, MAXP, (tokens,), generator=g).to(torch.int32).to(DEV)
    slots = torch.randperm(nb * 16, generator=g)[:tokens].to(DEV)
    shape, kind = (nb, hkv, 16, d), torch.uint8 if kv == B.PA_KV_FP8_E4M3 else torch.bfloat16
    kc, vc = torch.zeros(shape, dtype=kind, device=DEV), torch.zeros(shape, dtype=kind, device=DEV)
    q_out = torch.empty_like(q)
    pad = [3, tokens - 1]
    pos[pad] = torch.tensor([-7, MAXP], dtype=torch.int32, device=DEV)
    slots[pad] = torch.tensor([-1, -100], device=DEV)
    B.pa_rope_cache_write(desc, rope, q_out, q, k, v, pos, kc, vc, slots)
    assert int(ew) == 0
    # a token that is written is checked as before
    slots[pad[1]] = nb * 16 - 1
    B.pa_rope_cache_write(desc, rope, q_out, q, k, v, pos, kc, vc, slots)
    assert int(ew) == B.PA_DEVERR_BAD_INDEX
