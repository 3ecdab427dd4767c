"""MixedStep.__call__ with groups: the new rows written, the shared decode and
the prefill, in every mode, captured and replayed with other inputs."""
import pytest
import torch

import oracle
import pa_helpers as H
from paged_kv_attention_14_gb300 import binding as B
from paged_kv_attention_14_gb300 import workloads as W
from paged_kv_attention_14_gb300.step import GraphedStep, MixedStep

pytestmark = pytest.mark.gpu
DEV = "cuda"
# worst case of N(0, 1) rows of 128 in fp32, and the prefill's one fp16 P (2^-11, times max |v| of 5)
TOL, PREFILL_TOL = 5e-4, 2.5e-3


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_kv_attention_14_gb300 import build
    B.load(build.build())


@pytest.mark.parametrize("prefill", [True, False])
@pytest.mark.parametrize("mode", MixedStep.MODES)
@pytest.mark.parametrize("append", [False, True])
def test_a_step_with_groups(mode, prefill, append):
    Hq, Hkv, D, S = 32, 8, 128, 7
    b = W.shared_prefix_decode(980, [5, 2], [160, 48], [9, 50, 1, 16, 33, 17, 100], Hq, Hkv, D, device=DEV)
    p = W.random_prefill(981, [70, 1, 40], [70, 33, 100], Hq, Hkv, D, device=DEV, poison=True)
    kc, vc = (torch.cat([getattr(b, n), getattr(p, n)]) for n in ("k_pool", "v_pool"))
    ptab = torch.where(p.block_tables_prefill >= 0, p.block_tables_prefill + b.num_blocks, p.block_tables_prefill)
    d = B.make_desc(kc.shape[0], Hkv, Hq, D)
    c = b.meta["cascade"]
    groups = (c["query_start_loc"], c["prefix_lens"], 5, 160)
    maxL = b.block_tables_decode.shape[1] * 16
    out, lse = torch.zeros(S, Hq, D, device=DEV), torch.zeros(S, Hq, device=DEV)
    pout = torch.zeros(p.q_prefill.shape[0], Hq, D, device=DEV) if prefill else None
    step = MixedStep(d, kc, vc, b.scale, decode_out=out, decode_lse=lse, workspace=B.mixed_workspace(d, S, maxL, DEV),
                     max_context_len_decode=maxL, prefill_out=pout, max_q_len=70, max_context_len_prefill=100, mode=mode,
                     decode_append=append, write_in_step=append, shared_workspace=B.decode_shared_workspace(d, S, 2, 5))
    last = (b.context_lens_decode - 1).long()
    slots = b.block_tables_decode.gather(1, (last // 16)[:, None])[:, 0].long() * 16 + last % 16
    new = torch.zeros(2, S, Hkv, D, dtype=torch.bfloat16, device=DEV)

    def issue():
        step(new[0], new[1], slots, (b.q_decode, b.block_tables_decode, b.context_lens_decode),
             (p.q_prefill, p.query_start_loc, ptab, p.context_lens_prefill) if prefill else None, groups)

    graph = GraphedStep(issue)
    new.copy_(torch.randn(new.shape, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16))
    graph()
    at = slots // 16, slots % 16
    assert torch.equal(kc[at[0], :, at[1]], new[0]) and torch.equal(vc[at[0], :, at[1]], new[1])
    o, x = H.oracle_decode(b, ocaches=(oracle.KV_BF16, kc.cpu(), vc.cpu()))
    H.assert_close(out.reshape(-1, D), o.reshape(-1, D), TOL, "decode out")
    H.assert_close(lse.reshape(-1), x.reshape(-1), TOL, "decode lse")
    if prefill:
        o, _ = oracle.prefill(oracle.KV_BF16, 16, Hkv, Hq, D, p.q_prefill.cpu(), p.query_start_loc.cpu(), kc.cpu(), vc.cpu(),
                              ptab.cpu(), p.context_lens_prefill.cpu(), b.scale)
        H.assert_close(pout.reshape(-1, D), o.reshape(-1, D), PREFILL_TOL, "prefill out")
