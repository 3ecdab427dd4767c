"""Refusals of pa_qk_norm_rope and pa_rope_cache_write, before any CUDA call
(no GPU needed): every argument the header restricts, and the order in which
an empty call is accepted."""
import ctypes

import pytest
import torch

from paged_kv_attention_14_gb300 import binding as B
from paged_kv_attention_14_gb300 import build as pa_build


@pytest.fixture(scope="module")
def lib():
    return B.load(pa_build.build())


def _desc(**kw):
    d = dict(num_blocks=64, num_kv_heads=2, num_q_heads=4, head_dim=64)
    d.update(kw)
    return B.make_desc(**d)


def _rope(**kw):
    f = dict(cos_sin=0x1000, max_position=128, rotary_dim=0, interleaved=0, eps=1e-6, q_weight=None, k_weight=None)
    f.update(kw)
    return B.PaRopeDesc(*f.values())


def _norm(lib, d, r, **kw):
    a = dict(q_out=0x10000, k_out=0x20000, q=0x30000, qs=0, k=0x40000, ks=0, pos=0x50000, n=4)
    a.update(kw)
    return lib.pa_qk_norm_rope(ctypes.byref(d) if d else None, ctypes.byref(r) if r else None, a["q_out"], a["k_out"],
                               a["q"], a["qs"], a["k"], a["ks"], a["pos"], a["n"], None)


def _write(lib, d, r, **kw):
    a = dict(q_out=0x10000, q=0x30000, qs=0, k=0x40000, ks=0, v=0x60000, vs=0, pos=0x50000, kc=0x70000, vc=0x80000,
             slots=0x90000, n=4)
    a.update(kw)
    return lib.pa_rope_cache_write(ctypes.byref(d) if d else None, ctypes.byref(r) if r else None, a["q_out"], a["q"],
                                   a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["pos"], a["kc"], a["vc"], a["slots"],
                                   a["n"], None)


@pytest.mark.parametrize("call", [_norm, _write])
def test_an_empty_call_is_accepted_and_a_bad_descriptor_is_not(lib, call):
    assert call(lib, _desc(), None, n=0) == B.PA_OK and B.last_error() == ""
    assert call(lib, None, _rope()) == B.PA_ERR_INVALID_ARG
    assert call(lib, _desc(head_dim=96), _rope()) == B.PA_ERR_UNSUPPORTED
    assert call(lib, _desc(), _rope(), n=-1) == B.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("call", [_norm, _write])
@pytest.mark.parametrize("bad,word", [
    (dict(cos_sin=None), "cos_sin"), (dict(cos_sin=0x1008), "cos_sin"), (dict(max_position=0), "max_position"),
    (dict(rotary_dim=8), "rotary_dim"), (dict(rotary_dim=80), "rotary_dim"), (dict(rotary_dim=-16), "rotary_dim"),
    (dict(interleaved=2), "interleaved"), (dict(eps=-1e-6), "eps"), (dict(eps=float("nan")), "eps"),
    (dict(eps=float("inf")), "eps"), (dict(q_weight=0x1002), "weight"), (dict(k_weight=0x1008), "weight"),
])
def test_rotation_descriptor(lib, call, bad, word):
    assert call(lib, _desc(), _rope(**bad)) == B.PA_ERR_INVALID_ARG
    assert word in B.last_error()


@pytest.mark.parametrize("call", [_norm, _write])
@pytest.mark.parametrize("bad,word", [
    (dict(pos=None), "positions"), (dict(pos=0x50002), "positions"), (dict(q=0x30008), "aligned"),
    (dict(k=0x40008), "aligned"), (dict(q_out=0x10008), "aligned"), (dict(qs=255), "strides"),
    (dict(qs=248), "strides"), (dict(ks=120), "strides"), (dict(ks=-128), "strides"), (dict(q=None), "q_out"),
    (dict(q_out=None), "q_out"),
])
def test_shared_arguments(lib, call, bad, word):
    assert call(lib, _desc(), _rope(), **bad) == B.PA_ERR_INVALID_ARG
    assert word in B.last_error()


def test_null_rope(lib):
    assert _norm(lib, _desc(), None) == B.PA_ERR_INVALID_ARG and "rope" in B.last_error()
    assert _write(lib, _desc(), None) == B.PA_ERR_INVALID_ARG and "rope" in B.last_error()


def test_norm_rope_sides_come_in_pairs(lib):
    for bad in (dict(k=None), dict(k_out=None), dict(q=None, q_out=None, k=None, k_out=None)):
        assert _norm(lib, _desc(), _rope(), **bad) == B.PA_ERR_INVALID_ARG
        assert "pairs" in B.last_error()


@pytest.mark.parametrize("bad", [dict(k=None), dict(v=None), dict(kc=None), dict(vc=None), dict(slots=None),
                                 dict(slots=0x90004), dict(kc=0x70008), dict(vc=0x80008), dict(v=0x60008),
                                 dict(vs=64), dict(vs=132)])
def test_cache_write_arguments(lib, bad):
    assert _write(lib, _desc(), _rope(), **bad) == B.PA_ERR_INVALID_ARG


def test_binding_refuses_what_it_would_misread():
    """Wrong shapes, strides, types and devices raise before the library is called."""
    cpu = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        B._rows(cpu, torch.bfloat16, 3, 4, 64, "q")
    with pytest.raises(TypeError, match="dtype"):
        B._rows(cpu.half(), torch.bfloat16, 3, 4, 64, "q")
    with pytest.raises(ValueError, match="CUDA"):
        B.make_rope(torch.zeros(8, 64))
    with pytest.raises(ValueError, match="max_position"):
        B.make_rope(torch.zeros(8, 64), rotary_dim=32)


def test_rope_table_angles():
    """Rows are cos | sin of p * base^(-2 i / rd), right to fp32's half step at far positions."""
    t = B.rope_table(100001, 64, base=1e6, device="cpu")
    assert t.shape == (100001, 64) and t.dtype == torch.float32
    p, i = 100000, torch.arange(32, dtype=torch.float64)
    ang = p * 1e6 ** (-2 * i / 64)
    want = torch.cat([ang.cos(), ang.sin()])
    # one rounding of a value of magnitude at most 1, and 64-bit angles off by p * 2^-52
    assert (t[p].double() - want).abs().max() <= 2.0 ** -25 + 1e5 * 2.0 ** -51
    assert torch.equal(t[0], torch.cat([torch.ones(32), torch.zeros(32)]))
