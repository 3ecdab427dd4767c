"""One decode workspace, zeroed once, through batches of different sizes and layers of different cache types: each call
gives the bits that it gives with a workspace of its own."""
import pytest
import torch

from pa_helpers import desc_of, gpu_caches, gpu_decode, gpu_prefill, prefill_workspace
from paged_kv_attention_14_gb300 import binding as B
from paged_kv_attention_14_gb300 import workloads as W
from test_gpu_int4 import Batch

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Paged:
    """A decode over a 16- or 8-bit cache."""

    def __init__(self, seed, lens, hq, hkv, d, kv, impl=B.PA_DECODE_AUTO):
        self.b, self.impl = W.random_decode(seed, lens, hq, hkv, d, kv_dtype=kv, device=DEV, poison=True), impl
        self.caches = gpu_caches(self.b)
        self.bytes = B.pa_decode_workspace_size(desc_of(self.b, impl), len(lens), max(lens))

    def __call__(self, ws):
        return gpu_decode(self.b, caches=self.caches, decode_impl=self.impl, workspace=ws)


class FourBits:
    def __init__(self, seed, lens, hq, hkv, d, kind=B.PA_KV_INT4):
        self.b = Batch(lens, hq, hkv, d, kind, seed=seed)
        self.bytes = self.b.ws.numel()

    def __call__(self, ws):
        self.b.ws = ws
        self.b.out.fill_(float("nan"))
        self.b.run()
        return self.b.out.clone(), self.b.lse.clone()


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (8, 2, 64), (40, 8, 128), (16, 1, 128), (32, 8, 64)])
def test_one_workspace_for_batches_and_cache_types(hq, hkv, d):
    g = torch.Generator().manual_seed(hq + d)
    many = torch.randint(1, 900, (70,), generator=g).tolist()
    calls = [Paged(1, [3000, 5000], hq, hkv, d, W.KV_BF16), Paged(2, many, hq, hkv, d, W.KV_BF16),
             FourBits(3, [9000, 2500], hq, hkv, d), FourBits(4, many, hq, hkv, d),
             Paged(5, [7000], hq, hkv, d, W.KV_FP8), Paged(6, many, hq, hkv, d, W.KV_FP8),
             Paged(7, many[:9], hq, hkv, d, W.KV_F16), FourBits(8, [4000] * 5, hq, hkv, d, B.PA_KV_INT4_F16)]
    if hq // hkv <= 4:
        calls += [Paged(9, [6000, 10], hq, hkv, d, W.KV_BF16, B.PA_DECODE_SIMT), Paged(10, many, hq, hkv, d, W.KV_BF16, B.PA_DECODE_SIMT)]
    own = [c(torch.zeros(c.bytes, dtype=torch.uint8, device=DEV)) for c in calls]
    ws = torch.zeros(max(c.bytes for c in calls), dtype=torch.uint8, device=DEV)
    order = list(range(len(calls))) + torch.randperm(len(calls), generator=g).tolist() * 2 + list(range(len(calls)))[::-1]
    for i in order:
        out, lse = calls[i](ws)
        assert torch.equal(out, own[i][0]) and torch.equal(lse, own[i][1]), i
        assert int(ws[:4096].sum()) == 0  # the error word and the 4-bit decode's counters


def test_a_mixed_step_and_decodes_share_a_workspace():
    b = W.random_decode(11, [2000, 33, 700], 32, 8, 128, device=DEV, poison=True)
    many = Paged(12, [300] * 64, 32, 8, 128, W.KV_BF16)
    d, maxL = desc_of(b), b.max_context_len_decode()
    n = B.mixed_workspace(d, 3, maxL, DEV).numel()
    ws = torch.zeros(max(n, many.bytes), dtype=torch.uint8, device=DEV)
    want, (want_many, _) = gpu_decode(b)[0], many(torch.zeros_like(ws))
    four = FourBits(13, [5000, 800], 32, 8, 128)
    want4, _ = four(torch.zeros_like(ws))
    for _ in range(3):
        out = torch.full_like(want, float("nan"))
        B.pa_mixed_attention(d, b.k_pool, b.v_pool, b.scale, ws,
                             dec=(out, b.q_decode, b.block_tables_decode, b.context_lens_decode, maxL))
        torch.testing.assert_close(out, want, rtol=0, atol=2e-3)  # cut at other places than pa_decode's: its tolerance
        assert torch.equal(many(ws)[0], want_many)
        assert torch.equal(four(ws)[0], want4)


def test_one_workspace_for_balanced_prefills_of_different_shapes():
    B.pa_test_prefill_schedule(1)
    try:
        bs = [W.random_prefill(20, [64, 200], [3000, 2500], 32, 8, 128, device=DEV, poison=True),
              W.random_prefill(21, [300] * 12, [900] * 12, 32, 8, 128, device=DEV, poison=True),
              W.random_prefill(22, [512], [8000], 32, 8, 128, device=DEV, poison=True),
              W.random_prefill(23, [90] * 40, [400] * 40, 32, 8, 128, kv_dtype=W.KV_FP8, device=DEV, poison=True)]
        caches = [gpu_caches(b) for b in bs]
        sizes = [prefill_workspace(b) for b in bs]
        own = [gpu_prefill(b, caches=c, workspace=w) for b, c, w in zip(bs, caches, sizes)]
        ws = torch.zeros(max(w.numel() for w in sizes), dtype=torch.uint8, device=DEV)
        for i in (0, 1, 2, 3, 1, 0, 3, 2, 1):
            out, lse = gpu_prefill(bs[i], caches=caches[i], workspace=ws)
            assert torch.equal(out, own[i][0]) and torch.equal(lse, own[i][1]), i
    finally:
        B.pa_test_prefill_schedule(0)
