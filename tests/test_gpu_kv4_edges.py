"""Calls of the 4-bit cache and attention over it at the edges of what their
documentation allows."""
import numpy as np
import pytest
import torch

import exact_attention_134_b200 as attn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    attn.lib()


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_tensors_that_calls_write_to_count_as_changed():
    """What autograd goes by when a tensor that it saved was written to."""
    pool = attn.kv4_alloc(4, 2, 64, 16)
    table, lens = _ints([[0], [1]]), _ints([3, 4])
    k = torch.randn((2, 2, 64), device="cuda").bfloat16()
    q = torch.randn((2, 4, 64), device="cuda").bfloat16()
    o, lse, kg, vg = torch.empty_like(q), torch.empty((4, 2), device="cuda"), torch.empty_like(k), torch.empty_like(k)
    for call, written in ((lambda: attn.kv4_append(k, k, pool, table, lens), [pool]),
                          (lambda: attn.kv4_copy_pages(pool, _ints([0]), _ints([2])), [pool]),
                          (lambda: attn.kv4_gather(pool, table, lens, 2, k=kg), [kg]),
                          (lambda: attn.kv4_gather(pool, table, lens, 2, v=vg), [vg]),
                          (lambda: attn.attn_fwd_kv4(q, pool, table, lens, out=o), [o]),
                          (lambda: attn.attn_fwd_kv4(q, pool, table, lens, lse=lse), [lse])):
        everything = [pool, table, lens, k, q, o, lse, kg, vg]
        before = [t._version for t in everything]
        call()
        for t, was in zip(everything, before):
            assert (t._version > was) == any(t is w for w in written)
