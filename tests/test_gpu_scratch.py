"""Workspaces that a caller supplies, at every entry point that takes one."""
import pytest
import torch

import exact_attention_134_b200 as attn
from synthetic import make_qkv

pytestmark = pytest.mark.gpu


def test_strided_workspaces_are_refused():
    """A view of every other element: large enough, but the bytes between are someone else's."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    q, k, v = (t.cuda() for t in make_qkv(1, 2, 2, 256, 256, 64, seed=3))
    o, lse = attn.attn_fwd(q, k, v, causal=True)
    p = [t[0].transpose(0, 1).contiguous() for t in (q, k, v, o)]  # packed: one sequence
    cu = torch.tensor([0, 256], dtype=torch.int32, device="cuda")
    pool = attn.kv4_alloc(40, 2, 64, 16)
    table = torch.arange(40, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([3], dtype=torch.int32, device="cuda")
    attn.kv4_append(p[1][:3], p[2][:3], pool, table, lens)
    w = torch.ones(64, device="cuda")
    calls = [
        lambda ws: attn.qk_norm_rope_bwd(q, k, q, k, q_weight=w, k_weight=w, workspace=ws),
        lambda ws: attn.attn_fwd_kv4(p[0][:1], pool, table, lens, workspace=ws),
        lambda ws: attn.attn_bwd(q, k, v, o, lse, q, causal=True, workspace=ws),
        lambda ws: attn.attn_bwd_varlen(*p, lse[0], p[0], cu, cu, 256, 256, causal=True, workspace=ws),
        lambda ws: attn.attn_fwd_splitkv(q, k, v, num_splits=2, workspace=ws),
        lambda ws: attn.attn_fwd_partial(q, k, v, num_splits=2, workspace=ws),
        lambda ws: attn.attn_fwd_q8(q, k, v, workspace=ws),
        lambda ws: attn.q8_prepass(q, k, v, ws),
        lambda ws: attn.attn_fwd_host(q.cpu(), k.cpu(), v.cpu(), dev_buf=ws),
    ]
    big = torch.empty(1 << 25, dtype=torch.uint8, device="cuda")
    for call in calls:
        call(big)
        for bad in (big[::2], big.cpu()):
            with pytest.raises(ValueError):
                call(bad)
    assert attn.get_status() == (0, 0)
