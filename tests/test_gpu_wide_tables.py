"""Tables of 2^27 blocks a sequence and more, whose tokens a 32-bit length cannot count, with checked indices."""
import math

import pytest
import torch

from paged_kv_attention_14_gb300 import binding as pa

pytestmark = pytest.mark.gpu
DEV = "cuda"
WIDTH = 2 ** 27 + 3


@pytest.fixture(scope="module")
def tables():
    narrow = torch.randperm(20, generator=torch.Generator().manual_seed(1))[None, :9].to(torch.int32).to(DEV)
    wide = torch.full((1, WIDTH), -1, dtype=torch.int32, device=DEV)
    wide[:, :9] = narrow
    return narrow, wide


@pytest.mark.parametrize("kind", [pa.PA_KV_BF16, pa.PA_KV_FP8_E4M3, pa.PA_KV_INT4])
@pytest.mark.parametrize("impl", [pa.PA_DECODE_MMA, pa.PA_DECODE_SIMT])
def test_decode(tables, kind, impl):
    if kind == pa.PA_KV_INT4 and impl == pa.PA_DECODE_SIMT:
        pytest.skip("a 4-bit cache is decoded on the tensor cores")
    hq, hkv, d, L = 4, 2, 128, 140
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    desc = pa.make_desc(20, hkv, hq, d, kind, decode_impl=impl, error_word=word, check_indices=True)
    g = torch.Generator(device=DEV).manual_seed(2)
    rows = [torch.randn((320, hkv, d), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2)]
    shape, dt = {pa.PA_KV_BF16: ((20, hkv, 16, d), torch.bfloat16), pa.PA_KV_FP8_E4M3: ((20, hkv, 16, d), torch.uint8),
                 pa.PA_KV_INT4: ((20, hkv, 9 * d), torch.uint8)}[kind]
    kc, vc = [torch.zeros(shape, dtype=dt, device=DEV) for _ in range(2)]
    pa.pa_cache_write(desc, *rows, kc, vc, torch.arange(320, device=DEV))
    q = torch.randn((1, hq, d), generator=g, device=DEV).to(torch.bfloat16)
    lens = torch.tensor([L], dtype=torch.int32, device=DEV)
    outs = []
    for t in tables:
        out, lse = torch.zeros((1, hq, d), device=DEV), torch.zeros((1, hq), device=DEV)
        pa.pa_decode(desc, out, q, kc, vc, t, lens, L, 1 / math.sqrt(d), pa.decode_workspace(desc, 1, L), lse=lse)
        outs.append((out, lse))
    assert int(word) == 0
    assert torch.isfinite(outs[0][1]).all()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("impl", [pa.PA_PREFILL_MMA_SYNC, pa.PA_PREFILL_TCGEN05])
def test_prefill(tables, impl):
    hq, hkv, d, L, n = 4, 2, 128, 140, 33
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    desc = pa.make_desc(20, hkv, hq, d, prefill_impl=impl, error_word=word, check_indices=True)
    g = torch.Generator(device=DEV).manual_seed(3)
    kc, vc = [torch.randn((20, hkv, 16, d), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2)]
    q = torch.randn((n, hq, d), generator=g, device=DEV).to(torch.bfloat16)
    lens, loc = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([L], [0, n])]
    outs = []
    for t in tables:
        out, lse = torch.zeros((n, hq, d), device=DEV), torch.zeros((n, hq), device=DEV)
        pa.pa_prefill_chunk(desc, out, q, loc, kc, vc, t, lens, n, L, 1 / math.sqrt(d), lse=lse)
        outs.append((out, lse))
    assert int(word) == 0
    assert torch.isfinite(outs[0][1]).all()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
