"""Calls from threads that made no CUDA call before (an autograd engine's
thread whose first node is attention, a server's worker)."""
import threading

import pytest
import torch

import exact_attention_134_b200 as attn
from synthetic import make_qkv

pytestmark = pytest.mark.gpu


def test_first_cuda_call_of_a_thread():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    q, k, v = (t.cuda() for t in make_qkv(1, 2, 2, 200, 200, 64, seed=3))
    want = attn.attn_fwd(q, k, v, causal=True)
    grads = attn.attn_bwd(q, k, v, *want, q, causal=True)
    o, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    dq, dk, dv = (torch.empty_like(t) for t in (q, k, v))
    ws = torch.empty(attn.bwd_workspace_size(1, 2, 2, 200, 200, 64), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    failed = []

    def run(call):
        try:
            call()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    for call in (lambda: attn.attn_fwd(q, k, v, causal=True, out=o, lse=lse),
                 lambda: attn.attn_bwd(q, k, v, *want, q, causal=True, workspace=ws, dq=dq, dk=dk, dv=dv)):
        t = threading.Thread(target=run, args=(call,))
        t.start()
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert torch.equal(dk, grads[1]) and torch.equal(dv, grads[2])
