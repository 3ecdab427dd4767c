"""What MixedStep hands to the library, with the entry points replaced by a recorder (no GPU needed)."""
import pytest
import torch

from paged_kv_attention_14_gb300 import binding as B
from paged_kv_attention_14_gb300 import build as pa_build
from paged_kv_attention_14_gb300 import step as step_module
from paged_kv_attention_14_gb300.step import MixedStep


@pytest.fixture
def calls(monkeypatch):
    """The names and arguments of the entry points called, in order."""
    B.load(pa_build.build())
    seen = []

    def record(name):
        return lambda *a, **kw: seen.append((name, a, kw))

    for name in ("pa_cache_write", "pa_rope_cache_write", "pa_decode", "pa_decode_append", "pa_decode_shared",
                 "pa_prefill_chunk", "pa_mixed_attention"):
        monkeypatch.setattr(B, name, record(name))
    monkeypatch.setattr(step_module.torch.cuda, "Event", lambda: None)
    return seen


S, HQ, HKV, D = 3, 4, 2, 64


def _step(decode=True, prefill=False, **kw):
    desc = B.make_desc(16, HKV, HQ, D)
    cache = torch.zeros(16, HKV, 16, D, dtype=torch.bfloat16)
    return MixedStep(desc, cache, cache.clone(), 0.125, decode_out=torch.zeros(S, HQ, D) if decode else None,
                     prefill_out=torch.zeros(5, HQ, D) if prefill else None, max_context_len_decode=64, max_q_len=5,
                     max_context_len_prefill=64, mode="serial", shared_workspace=torch.zeros(64, dtype=torch.uint8), **kw)


def _decode_args():
    return (torch.zeros(S, HQ, D, dtype=torch.bfloat16), torch.zeros(S, 4, dtype=torch.int32),
            torch.full((S,), 20, dtype=torch.int32))


GROUPS = (torch.tensor([0, S], dtype=torch.int32), torch.tensor([16], dtype=torch.int32), S, 16)


@pytest.mark.parametrize("append", [False, True])
def test_groups_write_the_new_rows_before_the_shared_decode(calls, append):
    k = torch.zeros(S, HKV, D, dtype=torch.bfloat16)
    slots = torch.arange(S)
    _step(decode_append=append)(k, k, slots, _decode_args(), groups=GROUPS)
    assert [c[0] for c in calls] == ["pa_cache_write", "pa_decode_shared"]
    assert calls[0][1][5] is slots


@pytest.mark.parametrize("append", [False, True])
def test_groups_without_slots_for_the_new_rows_are_refused(calls, append):
    """A step that appends needs no slots, but the shared decode does not append: the new rows would be lost."""
    k = torch.zeros(S, HKV, D, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="slot_mapping"):
        _step(decode_append=append)(k, k, None, _decode_args(), groups=GROUPS)
    assert not calls


def test_groups_without_new_rows_only_attend(calls):
    _step()(None, None, None, _decode_args(), groups=GROUPS)
    assert [c[0] for c in calls] == ["pa_decode_shared"]


@pytest.mark.parametrize("decode", [True, False])
def test_the_chunks_queries_follow_the_decode_sequences(calls, decode):
    """q_rot holds the decode sequences' rows first, also for a step without decode outputs."""
    T = S + 5
    q_rot = torch.arange(T * HQ * D, dtype=torch.float32).to(torch.bfloat16).view(T, HQ, D)
    q = torch.zeros_like(q_rot)
    kv = torch.zeros(T, HKV, D, dtype=torch.bfloat16)
    _, tables, lens = _decode_args()
    pf = (torch.tensor([0, 5], dtype=torch.int32), torch.zeros(1, 4, dtype=torch.int32), torch.tensor([5], dtype=torch.int32))
    _step(decode=decode, prefill=True).projected(None, q_rot, q, kv, kv, torch.zeros(T, dtype=torch.int32),
                                                 torch.arange(T), (tables, lens), pf)
    assert [c[0] for c in calls] == ["pa_rope_cache_write"] + ["pa_decode"] * decode + ["pa_prefill_chunk"]
    rows = calls[-1][1][2]
    assert rows.data_ptr() == q_rot[S:].data_ptr() and rows.shape[0] == 5
