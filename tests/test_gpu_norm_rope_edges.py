"""Calls of the norm with rotation at the edges of what its documentation allows."""
import pytest
import torch

import exact_attention_134_b200 as attn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    attn.lib()


def _inputs(N, Hq, Hkv, d, seed=0):
    g = torch.Generator().manual_seed(seed)
    q, k = (torch.randn((N, h, d), generator=g).bfloat16().cuda() for h in (Hq, Hkv))
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    inv = (1e4 ** (-torch.arange(d // 2).float() / (d // 2))).cuda()
    wq, wk = ((1 + 0.1 * torch.randn(d, generator=g)).cuda() for _ in range(2))
    return q, k, pos, inv, wq, wk


def test_a_gradient_that_begins_off_a_16_byte_boundary():
    """A result joined behind three other values hands back a contiguous gradient 6 bytes off."""
    q, k, pos, inv, wq, wk = _inputs(9, 4, 2, 64)
    dy = torch.randn((3 + q.numel(),), device="cuda").bfloat16()
    want = attn.qk_norm_rope_bwd(q, k, dy[3:].view(q.shape).clone(), torch.zeros_like(k), pos, inv, wq, wk)
    leaves = [t.detach().requires_grad_() for t in (q, k, wq, wk)]
    yq, _ = attn.norm_rope(leaves[0], leaves[1], pos, inv, *leaves[2:])
    torch.cat([torch.zeros(3, device="cuda").bfloat16(), yq.flatten()]).backward(dy)
    for got, ref in zip(leaves, want):
        assert torch.equal(got.grad, ref)


def test_a_tensor_written_in_place_is_not_used_by_a_backward():
    """norm_rope saves q and k; a call that then writes to one of them makes the backward raise."""
    q, k, pos, inv, wq, wk = _inputs(9, 4, 2, 64)
    for which in (0, 1):
        x = [t.clone().requires_grad_() for t in (q, k)]
        out = attn.norm_rope(*x, pos, inv, wq, wk)
        place = [None, None]
        place[which] = x[which].detach()
        attn.qk_norm_rope(q, k, pos, inv, wq, wk, q_out=place[0], k_out=place[1])
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            (out[0].sum() + out[1].sum()).backward()
    x = [t.clone().requires_grad_() for t in (q, k)]
    out = attn.norm_rope(*x, pos, inv, wq, wk)
    attn.qk_norm_rope_bwd(q, k, q, k, pos, inv, wq, wk, dk=x[1].detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out[0].sum().backward()
    # tensors that the call made itself, or only read, count as they did; inference tensors have no count
    at = [t._version for t in (q, k, pos, inv, wq, wk)]
    y = attn.qk_norm_rope(q, k, pos, inv, wq, wk)
    assert [t._version for t in (q, k, pos, inv, wq, wk)] == at and y[0]._version == 0
    with torch.inference_mode():
        z = torch.empty_like(q)
    attn.qk_norm_rope(q, k, pos, inv, wq, wk, q_out=z)
    assert torch.equal(z, y[0])


@pytest.mark.parametrize("d", [64, 96, 128, 256])
def test_the_largest_rows(d):
    """Rows of values just below 2^59: the sum of their squares is still finite."""
    q, k, pos, inv, wq, wk = _inputs(33, 2, 1, d)
    x = [(torch.sign(t.float()) * 2.0 ** 58 * 1.9921875).bfloat16() for t in (q, k)]
    y = attn.qk_norm_rope(*x, q_weight=wq, k_weight=wk)
    for got, s, w in zip(y, x, (wq, wk)):
        want = torch.sign(s.double()) * w.double()
        assert ((got.double() - want).abs() <= (torch.finfo(torch.bfloat16).eps / 2 + 2.0 ** -18) * want.abs()).all()
    dq, dk, dwq, dwk = attn.qk_norm_rope_bwd(*x, q, k, q_weight=wq, k_weight=wk)
    # dw = sum over rows of dy * sign(x); fp32 sums of fewer than 2^7 terms
    for dw, s, dy in ((dwq, x[0], q), (dwk, x[1], k)):
        terms = dy.double() * torch.sign(s.double())
        assert ((dw.double() - terms.sum((0, 1))).abs() <= 2.0 ** -17 * terms.abs().sum((0, 1))).all()
    assert dq.isfinite().all() and dk.isfinite().all()


def test_a_captured_training_step():
    """Norm and rotation, attention and their backward in one graph, captured as torch asks for it: after
    warm-up on a side stream, with no eager graph of the leaves alive. Replayed with other inputs."""
    N, d = 150, 64
    q0, k0, pos, inv, wq0, wk0 = _inputs(N, 4, 2, d, seed=5)
    q0, k0 = (t.transpose(0, 1)[None].contiguous() for t in (q0, k0))
    v0, dout = torch.randn_like(k0), torch.randn_like(q0)
    leaves = [t.clone().requires_grad_() for t in (q0, k0, v0, wq0, wk0)]

    def step(q, k, v, wq, wk):
        yq, yk = attn.norm_rope(q, k, pos, inv, wq, wk)
        attn.attention(yq, yk, v, causal=True).backward(dout)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            step(*leaves)
            for t in leaves:
                t.grad = None
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*leaves)
    for seed in (6, 7):
        g = torch.Generator(device="cuda").manual_seed(seed)
        with torch.no_grad():
            for t in leaves:
                t.copy_(torch.randn(t.shape, device="cuda", generator=g))
            dout.copy_(torch.randn(dout.shape, device="cuda", generator=g))
        graph.replay()
        torch.cuda.synchronize()
        fresh = [t.detach().clone().requires_grad_() for t in leaves]
        step(*fresh)
        # dQ of attention is summed by atomics, in any order, in fp32: one step of bf16 here and there
        for a, b in zip(leaves, fresh):
            err = (a.grad.double() - b.grad.double()).norm() / b.grad.double().norm()
            assert err <= torch.finfo(torch.bfloat16).eps / 2, err.item()
    assert attn.get_status() == (0, 0)
