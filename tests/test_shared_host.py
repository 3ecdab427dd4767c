"""Refusals of pa_decode_shared and its workspace size, before any CUDA call (no GPU needed)."""
import ctypes

import pytest

from paged_kv_attention_14_gb300 import binding as B
from paged_kv_attention_14_gb300 import build as pa_build


@pytest.fixture(scope="module")
def lib():
    return B.load(pa_build.build())


def _desc(**kw):
    d = dict(num_blocks=64, num_kv_heads=2, num_q_heads=4, head_dim=64)
    d.update(kw)
    return B.make_desc(**d)


def _call(lib, d, **kw):
    a = dict(out=0x1000, lse=None, q=0x2000, kc=0x3000, vc=0x4000, bt=0x5000, mb=4, cl=0x6000, S=3, maxL=64, gs=0x7000,
             pl=0x8000, G=1, mg=3, mp=32, scale=0.125, ws=0x9000, wsb=1 << 40)
    a.update(kw)
    return lib.pa_decode_shared(ctypes.byref(d) if d else None, a["out"], a["lse"], a["q"], a["kc"], a["vc"], a["bt"],
                                a["mb"], a["cl"], a["S"], a["maxL"], a["gs"], a["pl"], a["G"], a["mg"], a["mp"],
                                a["scale"], a["ws"], a["wsb"], None)


def test_an_empty_batch_is_accepted(lib):
    assert _call(lib, _desc(), S=0, out=None, q=None, kc=None, vc=None, bt=None, cl=None, ws=None) == B.PA_OK
    assert B.last_error() == ""


@pytest.mark.parametrize("bad,status", [
    (dict(S=-1), B.PA_ERR_INVALID_ARG), (dict(G=-1), B.PA_ERR_INVALID_ARG), (dict(mg=-1), B.PA_ERR_INVALID_ARG),
    (dict(S=65536), B.PA_ERR_UNSUPPORTED), (dict(G=65536), B.PA_ERR_UNSUPPORTED),
    (dict(out=None), B.PA_ERR_INVALID_ARG), (dict(q=None), B.PA_ERR_INVALID_ARG),
    (dict(kc=None), B.PA_ERR_INVALID_ARG), (dict(vc=None), B.PA_ERR_INVALID_ARG),
    (dict(bt=None), B.PA_ERR_INVALID_ARG), (dict(cl=None), B.PA_ERR_INVALID_ARG),
    (dict(gs=None), B.PA_ERR_INVALID_ARG), (dict(pl=None), B.PA_ERR_INVALID_ARG),
    (dict(out=0x1008), B.PA_ERR_INVALID_ARG), (dict(q=0x2004), B.PA_ERR_INVALID_ARG),
    (dict(kc=0x3008), B.PA_ERR_INVALID_ARG), (dict(bt=0x5002), B.PA_ERR_INVALID_ARG),
    (dict(gs=0x7002), B.PA_ERR_INVALID_ARG), (dict(pl=0x8001), B.PA_ERR_INVALID_ARG),
    (dict(lse=0xa002), B.PA_ERR_INVALID_ARG), (dict(mb=0), B.PA_ERR_INVALID_ARG),
    (dict(maxL=65), B.PA_ERR_INVALID_ARG), (dict(maxL=-1), B.PA_ERR_INVALID_ARG),
    (dict(mp=65), B.PA_ERR_INVALID_ARG), (dict(mp=-16), B.PA_ERR_INVALID_ARG),
    (dict(scale=float("nan")), B.PA_ERR_INVALID_ARG), (dict(ws=None), B.PA_ERR_WORKSPACE),
    (dict(ws=0x9008), B.PA_ERR_WORKSPACE), (dict(wsb=64), B.PA_ERR_WORKSPACE),
])
def test_arguments(lib, bad, status):
    assert _call(lib, _desc(), **bad) == status
    assert B.last_error() != ""


@pytest.mark.parametrize("field,value,status", [
    ("head_dim", 96, B.PA_ERR_UNSUPPORTED), ("block_size", 32, B.PA_ERR_UNSUPPORTED),
    ("sliding_window", 8, B.PA_ERR_UNSUPPORTED), ("attention_chunk", 64, B.PA_ERR_UNSUPPORTED),
    ("decode_impl", B.PA_DECODE_SIMT, B.PA_ERR_UNSUPPORTED), ("num_blocks", 1 << 30, B.PA_ERR_UNSUPPORTED),
    ("kv_dtype", 9, B.PA_ERR_INVALID_ARG),
])
def test_descriptor(lib, field, value, status):
    d = _desc()
    setattr(d, field, value)
    assert _call(lib, d) == status
    assert lib.pa_decode_shared_workspace_size(ctypes.byref(d), 3, 1, 3) == 0
    assert _call(lib, None) == B.PA_ERR_INVALID_ARG


def test_a_workspace_past_32_bits_of_places_is_refused(lib):
    d = _desc(num_kv_heads=64, num_q_heads=1024, head_dim=128)
    # two parts of 1024 heads x 128 x 4 bytes a sequence
    assert lib.pa_decode_shared_workspace_size(ctypes.byref(d), 32000, 1, 2) > 32000 * (1 << 20)
    assert lib.pa_decode_shared_workspace_size(ctypes.byref(d), 33000, 1, 2) == 0
    assert _call(lib, d, S=33000) == B.PA_ERR_UNSUPPORTED and "32 GB" in B.last_error()


def test_workspace_size(lib):
    d = ctypes.byref(_desc())
    size = lib.pa_decode_shared_workspace_size
    assert size(d, -1, 1, 1) == 0 and size(d, 1, -1, 1) == 0 and size(d, 1, 1, -1) == 0
    a = size(d, 8, 2, 4)
    # two sets of parts per (sequence, head), and more for more of anything
    assert a > 2 * 8 * 4 * 65 * 4
    assert size(d, 9, 2, 4) > a and size(d, 8, 200, 4) > a and size(d, 8, 2, 8) > a
    assert size(d, 8, 2, 64) == size(d, 8, 2, 1 << 30)  # tiles of at most 128 rows
