"""The host side of the bindings (no GPU)."""
import pytest
import torch

from exact_attention_134_b200 import rope


@pytest.mark.parametrize("make", [
    lambda x: torch.cat([torch.zeros(3).bfloat16(), x.flatten()])[3:].view(x.shape),      # contiguous, 6 bytes off
    lambda x: torch.cat([torch.zeros(2, 5, 4).bfloat16(), x], -1)[..., 4:],               # rows of 68
    lambda x: x.transpose(0, 1).contiguous().transpose(0, 1),                             # other order: read as it is
    lambda x: x,
    lambda x: x[:1, :1, :1].expand(x.shape),                                              # a sum's gradient
])
def test_gradients_are_readable(make):
    t = make(torch.randn((2, 5, 64)).bfloat16())
    r = rope._readable(t)
    assert torch.equal(r, t)
    assert r.stride(-1) == 1 and all(s % 8 == 0 for s in r.stride()[:-1]) and r.data_ptr() % 16 == 0


def test_scratch_is_contiguous_and_on_the_device():
    import exact_attention_134_b200 as attn
    t = torch.empty(64, dtype=torch.uint8)
    attn._check_scratch("workspace", None, 0)
    attn._check_scratch("workspace", t, -1)                       # -1: the host, as get_device() has it
    attn._check_scratch("workspace", t.view(torch.float32), -1)
    for bad, index in ((t, 0), (t[::2], -1), (t.view(8, 8).T, -1), (t[:1].expand(64), -1)):
        with pytest.raises(ValueError):
            attn._check_scratch("workspace", bad, index)
