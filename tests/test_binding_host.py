"""What the binding of the norm and rotation refuses before the library sees an address (no GPU needed)."""
import pytest
import torch

from paged_kv_attention_14_gb300 import binding as B


class OnDevice(torch.Tensor):
    """A tensor that says it is on device 0, where its shape and strides are all that is looked at."""

    def get_device(self):
        return 0


def _on_device(t):
    return t.as_subclass(OnDevice)


def _row(h=8, d=128):
    return torch.zeros(1, h, d, dtype=torch.bfloat16)


@pytest.mark.parametrize("tokens,heads", [(2, 8), (5, 8), (5, 1)])
def test_a_token_broadcast_over_the_batch_is_refused(tokens, heads):
    """Its token stride is 0, which the library reads as dense rows: tokens times what the storage holds."""
    x = _on_device(_row(heads).expand(tokens, heads, 128))
    with pytest.raises(ValueError, match="token stride"):
        B._rows(x, torch.bfloat16, tokens, heads, 128, "q")


def test_tokens_that_overlap_are_refused():
    x = torch.zeros(4096, dtype=torch.bfloat16).as_strided((4, 8, 128), (512, 128, 1))
    with pytest.raises(ValueError, match="token stride"):
        B._rows(_on_device(x), torch.bfloat16, 4, 8, 128, "k")


def test_strides_the_library_takes():
    x = torch.zeros(5, 24 * 128, dtype=torch.bfloat16)
    q = _on_device(x[:, 128:9 * 128].view(5, 8, 128))
    assert B._rows(q, torch.bfloat16, 5, 8, 128, "q") == (q.data_ptr(), 24 * 128)
    # of one token, any stride
    one = _on_device(_row().expand(1, 8, 128))
    assert B._rows(one, torch.bfloat16, 1, 8, 128, "q") == (one.data_ptr(), 8 * 128)
    one = _on_device(torch.zeros(8 * 128, dtype=torch.bfloat16).as_strided((1, 8, 128), (0, 128, 1)))
    assert B._rows(one, torch.bfloat16, 1, 8, 128, "q")[1] == 8 * 128
