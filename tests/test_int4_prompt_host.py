"""Refusals of the 4-bit cache's calls and of pa_prompt_attention, before any CUDA
call (no GPU needed)."""
import ctypes

import pytest
import torch

import int4_reference as ref
from paged_kv_attention_14_gb300 import binding as B
from paged_kv_attention_14_gb300 import build as pa_build


@pytest.fixture(scope="module")
def lib():
    return B.load(pa_build.build())


def _desc(**kw):
    d = dict(num_blocks=64, num_kv_heads=2, num_q_heads=4, head_dim=64, kv_dtype=B.PA_KV_INT4)
    d.update(kw)
    return B.make_desc(**d)


def _call(fn, defaults, d, kw):
    a = dict(defaults)
    assert set(kw) <= set(a)
    a.update(kw)
    return fn(ctypes.byref(d) if d else None, *a.values())


def _write(lib, d, **kw):
    return _call(lib.pa_cache_write, dict(k=0x1000, v=0x2000, kc=0x3000, vc=0x4000, slots=0x5000, n=4, stream=None), d, kw)


def _widen(lib, d, **kw):
    return _call(lib.pa_widen_blocks, dict(kc=0x1000, vc=0x2000, src=0x3000, ko=0x4000, vo=0x5000, dst=0x6000, nb=8, n=4,
                                           stream=None), d, kw)


def _prompt(lib, d, **kw):
    return _call(lib.pa_prompt_attention,
                 dict(out=0x1000, lse=0x2000, q=0x3000, qs=0, k=0x4000, ks=0, v=0x5000, vs=0, starts=0x6000, seqs=2,
                      tokens=100, longest=60, scale=0.125, stream=None), d, kw)


def _decode(lib, d, **kw):
    return _call(lib.pa_decode, dict(out=0x1000, lse=None, q=0x2000, kc=0x3000, vc=0x4000, tables=0x5000, width=4,
                                     lens=0x6000, seqs=2, longest=16, scale=0.125, ws=0x7000, wsb=1 << 30, stream=None),
                 d, kw)


@pytest.mark.parametrize("call,empty", [(_write, dict(n=0)), (_widen, dict(n=0)), (_prompt, dict(seqs=0)),
                                        (_prompt, dict(tokens=0, longest=0)), (_prompt, dict(longest=0)),
                                        (_decode, dict(seqs=0))])
def test_an_empty_call_is_accepted_and_a_bad_descriptor_is_not(lib, call, empty):
    for kind in (B.PA_KV_INT4, B.PA_KV_INT4_F16):
        assert call(lib, _desc(kv_dtype=kind), **empty) == B.PA_OK, B.last_error()
    assert call(lib, None, **empty) == B.PA_ERR_INVALID_ARG
    assert call(lib, _desc(head_dim=96), **empty) == B.PA_ERR_UNSUPPORTED
    assert call(lib, _desc(kv_dtype=18), **empty) == B.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("call,bad,word", [
    (_write, dict(n=-1), "num_tokens"), (_write, dict(k=None), "non-NULL"), (_write, dict(vc=0x4008), "aligned"),
    (_write, dict(slots=0x5004), "slot_mapping"),
    (_widen, dict(n=-1), "num_pairs"), (_widen, dict(nb=-1), "num_out_blocks"), (_widen, dict(src=None), "non-NULL"),
    (_widen, dict(ko=0x4008), "aligned"), (_widen, dict(kc=0x1004), "aligned"), (_widen, dict(dst=0x6002), "aligned"),
    (_prompt, dict(seqs=-1), "num_seqs"), (_prompt, dict(tokens=-1), "num_tokens"), (_prompt, dict(longest=-1), "max_q_len"),
    (_prompt, dict(longest=101), "max_q_len"), (_prompt, dict(out=None), "non-NULL"), (_prompt, dict(q=0x3008), "aligned"),
    (_prompt, dict(out=0x1008), "aligned"), (_prompt, dict(starts=0x6001), "aligned"), (_prompt, dict(lse=0x2002), "aligned"),
    (_prompt, dict(qs=255), "strides"), (_prompt, dict(qs=252), "strides"), (_prompt, dict(ks=120), "strides"),
    (_prompt, dict(vs=-8), "strides"), (_prompt, dict(ks=1 << 40), "strides"), (_prompt, dict(scale=float("nan")), "NaN"),
    (_decode, dict(q=None), "non-NULL"), (_decode, dict(kc=0x3008), "aligned"), (_decode, dict(width=0), "max_blocks"),
    (_decode, dict(longest=65), "max_context_len"), (_decode, dict(scale=float("nan")), "NaN"),
])
def test_bad_arguments(lib, call, bad, word):
    assert call(lib, _desc(), **bad) == B.PA_ERR_INVALID_ARG
    assert word in B.last_error()


def test_too_many_rows(lib):
    big = 2 ** 31 - 1
    assert _prompt(lib, _desc(num_kv_heads=64, num_q_heads=1024), tokens=big, longest=big) == B.PA_ERR_UNSUPPORTED


def test_widening_takes_a_4_bit_cache_only(lib):
    assert _widen(lib, _desc(kv_dtype=B.PA_KV_BF16)) == B.PA_ERR_INVALID_ARG


def test_calls_without_a_4_bit_cache(lib):
    d = _desc()
    p = ctypes.byref(d)
    null = None
    assert lib.pa_prefill_chunk(p, 1 << 12, null, 1 << 12, 1 << 12, 1 << 12, 1 << 12, 1 << 12, 4, 1 << 12, 1, 4, 16, 0.1,
                                null) == B.PA_ERR_UNSUPPORTED
    assert "pa_widen_blocks" in B.last_error()
    assert lib.pa_decode_append(p, 1 << 12, null, 1 << 12, 1 << 12, 1 << 12, 1 << 12, 1 << 12, 1 << 12, 4, 1 << 12, 1, 16,
                                0.1, 1 << 12, 1 << 30, null) == B.PA_ERR_UNSUPPORTED
    assert lib.pa_prefix_attention(p, 1 << 12, 1 << 12, 1 << 12, 1 << 12, 1 << 12, 1 << 12, 1 << 12, 4, 1 << 12, 1, 4, 16,
                                   1, 0, 0.1, null) == B.PA_ERR_UNSUPPORTED
    assert lib.pa_decode_shared(p, 1 << 12, null, 1 << 12, 1 << 12, 1 << 12, 1 << 12, 4, 1 << 12, 1, 16, 1 << 12, 1 << 12,
                                1, 1, 16, 0.1, 1 << 12, 1 << 30, null) == B.PA_ERR_UNSUPPORTED
    assert lib.pa_mixed_attention(p, 1 << 12, null, 1 << 12, 1 << 12, 4, 1 << 12, 0, 16, 1 << 12, null, 1 << 12, 1 << 12,
                                  1 << 12, 4, 1 << 12, 0, 4, 16, 1 << 12, 1 << 12, 0.1, 1 << 12, 1 << 30,
                                  null) == B.PA_ERR_UNSUPPORTED
    rope = B.PaRopeDesc(0x1000, 128, 0, 0, 1e-6, None, None)
    assert lib.pa_rope_cache_write(p, ctypes.byref(rope), null, null, 0, 1 << 12, 0, 1 << 12, 0, 1 << 12, 1 << 12, 1 << 12,
                                   1 << 12, 4, null) == B.PA_ERR_UNSUPPORTED
    assert lib.pa_prefill_workspace_size(p, 1, 16) == 0
    assert lib.pa_mixed_workspace_size(p, 1, 16) == 0
    assert lib.pa_decode_shared_workspace_size(p, 1, 1, 1) == 0
    assert lib.pa_prefill_balanced_chosen(p, 1, 16, 16, 4) == -1


def test_scales_belong_to_8_bit_caches(lib):
    d = _desc()
    d.k_scales = 0x1000
    assert _write(lib, d, n=0) == B.PA_ERR_INVALID_ARG


def test_the_binding_refuses_shapes_and_types():
    d = _desc(num_blocks=3)
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    cache = torch.zeros((3, 2, B.int4_tile_bytes(64)), dtype=torch.uint8)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):  # not on a GPU
        B.pa_cache_write(d, x, x, cache, cache, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):  # not a row per slot
        B.pa_cache_write(d, x[:3], x[:3], cache, cache, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        B.pa_widen_blocks(_desc(kv_dtype=B.PA_KV_BF16), cache, cache, torch.zeros(1, dtype=torch.int32), x, x,
                          torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        B.pa_widen_blocks(d, cache, cache, torch.zeros(2, dtype=torch.int32), x, x, torch.zeros(1, dtype=torch.int32))
    with pytest.raises((ValueError, TypeError)):
        B.pa_prompt_attention(d, x, x.float(), x, x, torch.zeros(2, dtype=torch.int32), 4, 0.1)
    with pytest.raises(ValueError):
        B.pa_decode(d, torch.zeros(2, 4, 64), torch.zeros((2, 4, 32), dtype=torch.bfloat16), cache, cache,
                    torch.zeros((2, 1), dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 16, 0.1, cache)


def test_the_reference_reads_what_it_stores():
    g = torch.Generator().manual_seed(0)
    x = torch.randn((2, 3, 16, 128), generator=g).to(torch.bfloat16)
    rows = ref.rows_of(ref.cache_of(x), 128)
    n, s, _ = ref.quantise(x)
    step = s.double().repeat_interleave(64, -1)
    # half a step of the codes, and the rounding of the minimum and of 15 scales to fp16
    assert ((rows - x.double()).abs() <= 0.5 * step + 2.0 ** -11 * 16 * (step + x.double().abs().amax())).all()
    assert int(n.max()) == 15 and int(n.min()) == 0
