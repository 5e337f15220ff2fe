"""The norm of query and key heads with their rotation, and its gradients, on
the GPU against the fp64 oracle.

Tolerances, from the arithmetic: results are rounded once to bf16 (half a step:
2^-8 of the value). Before that, in fp32: the sum of squares (16 values a lane
and up to 4 shuffles: 20 roundings, halved by the root), rsqrt (2 steps), two
products, cos and sin (angle 2^-24 of a turn, function 2 steps) and the rotation
(2 roundings): below 64 * 2^-24 = 2^-18 of |a| + |b|. Gradients take two more sums
of that kind: 2^-16 of the largest of what is summed. Weight gradients: fp32
sums of R rows in slices; a random walk of roundings stays below 2^-22 * (the sum
of |terms|).
"""
import numpy as np
import pytest
import torch

import exact_attention_134_b200 as attn
from oracle import norm_rope

pytestmark = pytest.mark.gpu

HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    attn.lib()


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _case(B, N, Hq, Hkv, d, rot, axes, inter, packed, w, far=100000, seed=0, fused=True):
    g = torch.Generator().manual_seed(seed + 1000 * d + N)
    if fused:  # views of one projection result
        qkv = torch.randn((B, N, Hq + 2 * Hkv, d), generator=g).bfloat16().cuda()
        q, k = qkv[:, :, :Hq].transpose(1, 2), qkv[:, :, Hq:Hq + Hkv].transpose(1, 2)
    else:
        q, k = (torch.randn((B, h, N, d), generator=g).bfloat16().cuda() for h in (Hq, Hkv))
    half = rot // 2
    cuts = [half // axes] * (axes - 1)
    sections = [half - sum(cuts)] + cuts
    pos = torch.randint(-3, far, (axes, B, N), generator=g).int().cuda()
    inv = (10000.0 ** (-torch.arange(half).float() / max(half, 1))).cuda()
    wq = wk = None
    if w is not None:
        wq, wk = ((1 + 0.3 * torch.randn(d, generator=g)).to(w).cuda() for _ in range(2))
    kw = dict(sections=sections, interleaved=inter)
    if packed:
        assert B == 1
        q, k, pos = q[0].transpose(0, 1), k[0].transpose(0, 1), pos[:, 0]
    args = (pos, inv, wq, wk)
    if rot == 0:
        args, kw["sections"] = (None, None, wq, wk), None
    return q, k, args, kw, sections


def _want(x, w, pos, inv, sections, inter, packed, eps=1e-6, dy=None):
    x4 = _np(x)[None].transpose(0, 2, 1, 3) if packed else _np(x)
    ang = None
    if inv is not None:
        p = pos.cpu().numpy()
        ang = norm_rope.rotation_angles(p[:, None] if packed else p, inv.cpu().numpy(), sections)
    w = None if w is None else _np(w)
    if dy is None:
        y, mag = norm_rope.norm_rope_fp64(x4, w, eps, ang, inter)
        return (t[0].transpose(1, 0, 2) if packed else t for t in (y, mag))
    dy4 = _np(dy)[None].transpose(0, 2, 1, 3) if packed else _np(dy)
    dx, dw = norm_rope.norm_rope_bwd_fp64(x4, w, eps, dy4, ang, inter)
    # sizes of what is summed: |g| and |xhat| of a row, rstd
    r = 1.0 / np.sqrt(np.mean(x4 * x4, -1, keepdims=True) + eps)
    big = np.abs(dy4).max(-1, keepdims=True) * 2 * (1.0 if w is None else np.abs(w).max())
    mag = np.broadcast_to((r if w is not None else 1.0) * big * (1 + np.abs(x4 * r).max(-1, keepdims=True) ** 2), x4.shape)
    terms = (np.abs(dy4).max(-1, keepdims=True) * 2 * np.abs(x4 * r)).sum((0, 1, 2))
    if packed:
        dx, mag = dx[0].transpose(1, 0, 2), mag[0].transpose(1, 0, 2)
    return dx, mag, dw, terms


CASES = [
    # B, N, Hq, Hkv, d, rot, axes, interleaved, packed, weights
    (1, 1, 1, 1, 64, 64, 1, False, False, torch.float32),
    (2, 5, 4, 2, 128, 128, 1, False, False, torch.bfloat16),
    (1, 37, 7, 1, 96, 96, 1, True, True, torch.float32),
    (3, 33, 3, 3, 96, 48, 3, False, False, torch.float32),
    (1, 129, 8, 2, 256, 256, 2, False, True, torch.bfloat16),
    (2, 17, 2, 2, 256, 64, 4, True, False, torch.float32),
    (1, 65, 5, 5, 64, 16, 1, False, True, torch.float32),
    (2, 300, 6, 2, 128, 64, 3, True, False, torch.float32),
    (1, 50, 4, 4, 128, 128, 1, False, True, None),
    (2, 9, 4, 1, 64, 0, 1, False, False, torch.float32),
    (2, 3, 40, 8, 128, 32, 1, False, False, torch.float32),
    (1, 2000, 2, 1, 128, 128, 1, True, True, torch.float32),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("fused", [False, True])
def test_forward(case, fused):
    packed = case[8]
    q, k, args, kw, sections = _case(*case, fused=fused)
    yq, yk = attn.qk_norm_rope(q, k, *args, **kw)
    assert attn.get_status()[0] == 0
    assert yq.is_contiguous() and yq.shape == q.shape and yk.shape == k.shape
    for y, x, w in ((yq, q, args[2]), (yk, k, args[3])):
        want, mag = _want(x, w, args[0], args[1], sections, case[7], packed)
        assert (np.abs(_np(y) - want) <= HALF_BF16 * np.abs(want) + 2.0 ** -18 * mag).all()


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("fused", [False, True])
def test_backward(case, fused):
    packed = case[8]
    q, k, args, kw, sections = _case(*case, fused=fused)
    g = torch.Generator().manual_seed(3)
    dyq, dyk = (torch.randn(x.shape, generator=g).bfloat16().cuda() for x in (q, k))
    dq, dk, dwq, dwk = attn.qk_norm_rope_bwd(q, k, dyq, dyk, *args, **kw)
    again = attn.qk_norm_rope_bwd(q, k, dyq, dyk, *args, **kw)
    assert attn.get_status()[0] == 0
    for dx, dw, x, w, dy in ((dq, dwq, q, args[2], dyq), (dk, dwk, k, args[3], dyk)):
        want, mag, want_w, terms = _want(x, w, args[0], args[1], sections, case[7], packed, dy=dy)
        assert (np.abs(_np(dx) - want) <= HALF_BF16 * np.abs(want) + 2.0 ** -16 * mag).all()
        if w is None:
            assert dw is None
        else:
            assert dw.dtype == torch.float32
            assert (np.abs(_np(dw) - want_w) <= 2.0 ** -18 * terms + 2.0 ** -24 * np.abs(want_w)).all()
    for a, b in zip((dq, dk, dwq, dwk), again):  # the same bits every time
        assert (a is None and b is None) or torch.equal(a, b)


def test_without_a_norm_the_gradient_needs_no_input():
    q, k, args, kw, _ = _case(2, 40, 4, 2, 128, 128, 1, False, False, None)
    g = torch.Generator().manual_seed(4)
    dyq, dyk = (torch.randn(x.shape, generator=g).bfloat16().cuda() for x in (q, k))
    a = attn.qk_norm_rope_bwd(None, None, dyq, dyk, *args, **kw)
    b = attn.qk_norm_rope_bwd(q, k, dyq, dyk, *args, **kw)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and a[2] is None and a[3] is None
    # turned back and forth: the rotation of the gradient by -t is the inverse
    yq, _ = attn.qk_norm_rope(dyq, dyk, *args, **kw)
    back = attn.qk_norm_rope_bwd(None, None, yq, dyk, *args, **kw)[0]
    mag = dyq.float().abs().amax(-1, keepdim=True) * 2
    assert ((back.float() - dyq.float()).abs() <= 3 * HALF_BF16 * mag).all()


def test_in_place_in_the_projection():
    g = torch.Generator().manual_seed(8)
    qkv = torch.randn((77, 4 + 2 * 2, 128), generator=g).bfloat16().cuda()
    keep = qkv.clone()
    q, k = qkv[:, :4], qkv[:, 4:6]
    pos = torch.arange(77, dtype=torch.int32, device="cuda")
    inv = (1e4 ** (-torch.arange(64).float() / 64)).cuda()
    w = torch.ones(128, device="cuda")
    yq, yk = attn.qk_norm_rope(keep[:, :4], keep[:, 4:6], pos, inv, w, w)
    out = attn.qk_norm_rope(q, k, pos, inv, w, w, q_out=q, k_out=k)
    assert out[0] is q and out[1] is k
    assert torch.equal(q, yq) and torch.equal(k, yk) and torch.equal(qkv[:, 6:], keep[:, 6:])
    dq, dk, dwq, dwk = attn.qk_norm_rope_bwd(keep[:, :4], keep[:, 4:6], yq, yk, pos, inv, w, w)
    gq, gk = yq.clone(), yk.clone()
    r = attn.qk_norm_rope_bwd(keep[:, :4], keep[:, 4:6], gq, gk, pos, inv, w, w, dq=gq, dk=gk)
    assert torch.equal(gq, dq) and torch.equal(gk, dk) and torch.equal(r[2], dwq) and torch.equal(r[3], dwk)


def test_positions_of_every_shape_and_sign():
    B, N = 3, 21
    q, k, (pos, inv, wq, wk), kw, _ = _case(B, N, 2, 1, 64, 64, 1, False, False, torch.float32)
    kw["sections"] = None
    a = attn.qk_norm_rope(q, k, pos, inv, wq, wk)
    assert torch.equal(attn.qk_norm_rope(q, k, pos[0], inv, wq, wk)[0], a[0])
    shared = pos[:, :1].contiguous()
    b = attn.qk_norm_rope(q, k, shared, inv, wq, wk)
    assert torch.equal(attn.qk_norm_rope(q, k, shared[0, 0], inv, wq, wk)[0], b[0])
    assert torch.equal(attn.qk_norm_rope(q, k, shared.expand(1, B, N), inv, wq, wk)[0], b[0])
    for edge in (0, -1, 2 ** 31 - 1, -2 ** 31):
        p = torch.full((N,), edge, dtype=torch.int32, device="cuda")
        y, _ = attn.qk_norm_rope(q, k, p, inv, wq, wk)
        want, mag = _want(q, wq, p.expand(1, B, N), inv, [32], False, False)
        # an angle of 2^31 radians in 64 bits: 2^-21 of a radian
        assert (np.abs(_np(y) - want) <= HALF_BF16 * np.abs(want) + 2.0 ** -17 * mag).all()


def test_rows_of_zeros_and_of_large_values():
    q, k, (pos, inv, wq, wk), kw, sections = _case(1, 64, 4, 2, 128, 128, 1, False, False, torch.float32)
    q = q.contiguous()
    q[:, 0] = 0
    q[:, 1] *= 2.0 ** 40
    q[:, 2] *= 2.0 ** -30
    y, _ = attn.qk_norm_rope(q, k, pos, inv, wq, wk, eps=1e-5)
    want, mag = _want(q, wq, pos, inv, sections, False, False, eps=1e-5)
    assert (np.abs(_np(y) - want) <= HALF_BF16 * np.abs(want) + 2.0 ** -18 * mag).all()
    assert not y[:, 0].any()
    dy = torch.randn(q.shape, device="cuda").bfloat16()
    dq, _, dwq, _ = attn.qk_norm_rope_bwd(q, k, dy, torch.zeros_like(k), pos, inv, wq, wk, eps=1e-5)
    dx, mag, dw, terms = _want(q, wq, pos, inv, sections, False, False, eps=1e-5, dy=dy)
    assert (np.abs(_np(dq) - dx) <= HALF_BF16 * np.abs(dx) + 2.0 ** -16 * mag).all()
    assert (np.abs(_np(dwq) - dw) <= 2.0 ** -18 * terms + 2.0 ** -24 * np.abs(dw)).all()


def test_autograd_through_attention():
    """A training step: norm and rotation, attention, gradients of everything."""
    g = torch.Generator().manual_seed(21)
    B, N, Hq, Hkv, d = 1, 160, 4, 2, 64
    qkv = (torch.randn((B, N, Hq + 2 * Hkv, d), generator=g)).bfloat16().cuda().requires_grad_()
    wq, wk = ((1 + 0.1 * torch.randn(d, generator=g)).cuda().requires_grad_() for _ in range(2))
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    inv = (1e4 ** (-torch.arange(32).float() / 32)).cuda()
    dout = torch.randn((B, Hq, N, d), generator=g).bfloat16().cuda()
    q, k = qkv[:, :, :Hq].transpose(1, 2), qkv[:, :, Hq:Hq + Hkv].transpose(1, 2)
    v = qkv[:, :, Hq + Hkv:].transpose(1, 2).contiguous()
    yq, yk = attn.norm_rope(q, k, pos, inv, wq, wk)
    attn.attention(yq, yk, v, causal=True).backward(dout)

    ref = qkv.detach().double().requires_grad_()
    rq, rk = (w.detach().double().requires_grad_() for w in (wq, wk))
    ang = pos.double()[:, None] * inv.double()
    c, s = ang.cos(), ang.sin()

    def one(x, w):
        n = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
        a, b = n[..., :32], n[..., 32:]
        return torch.cat([a * c - b * s, a * s + b * c], -1)

    x = ref.transpose(1, 2)
    tq, tk, tv = one(x[:, :Hq], rq), one(x[:, Hq:Hq + Hkv], rk), x[:, Hq + Hkv:]
    rep = Hq // Hkv
    p = (tq @ tk.repeat_interleave(rep, 1).transpose(-1, -2)) / 8.0
    p = p.masked_fill(torch.ones(N, N, device="cuda").triu(1).bool(), -torch.inf).softmax(-1)
    (p @ tv.repeat_interleave(rep, 1)).backward(dout.double())
    # bf16 operands of every product between: a few steps of 2^-8, of the whole tensor's size
    for got, want in ((qkv.grad, ref.grad), (wq.grad, rq.grad), (wk.grad, rk.grad)):
        err = (got.double() - want).norm() / want.norm()
        assert err <= 4 * HALF_BF16, err.item()
    # an expanded gradient, and one output unused
    q2, k2 = (t.detach().requires_grad_() for t in (q, k))
    attn.norm_rope(q2, k2, pos, inv)[0].sum().backward()
    assert q2.grad.shape == q2.shape and not k2.grad.any()


def test_captured_and_replayed_and_on_another_stream():
    q, k, args, kw, _ = _case(2, 70, 4, 2, 128, 128, 3, False, False, torch.float32)
    q, k = q.contiguous(), k.contiguous()
    dy, dyk = torch.randn_like(q), torch.randn_like(k)
    ws = torch.empty(int(attn.lib().attn_qk_norm_rope_bwd_workspace_size(2, 70, 4, 2, 128)), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        first = attn.qk_norm_rope(q, k, *args, **kw) + attn.qk_norm_rope_bwd(q, k, dy, dyk, *args, workspace=ws, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = attn.qk_norm_rope(q, k, *args, **kw) + attn.qk_norm_rope_bwd(q, k, dy, dyk, *args, workspace=ws, **kw)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, out))
    q.copy_(torch.randn_like(q))
    args[0].add_(5)
    want = attn.qk_norm_rope(q, k, *args, **kw) + attn.qk_norm_rope_bwd(q, k, dy, dyk, *args, **kw)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, out))


def test_refusals():
    x = torch.zeros((6, 2, 64), dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(6, dtype=torch.int32, device="cuda")
    inv = torch.ones(32, device="cuda")
    w = torch.ones(64, device="cuda")
    bad = [
        lambda: attn.qk_norm_rope(x.float(), x.float(), pos, inv),
        lambda: attn.qk_norm_rope(x, x[:5], pos, inv), lambda: attn.qk_norm_rope(x, x[None], pos, inv),
        lambda: attn.qk_norm_rope(x.transpose(1, 2), x, pos, inv),
        lambda: attn.qk_norm_rope(x, x, pos.long(), inv), lambda: attn.qk_norm_rope(x, x, pos[:5], inv),
        lambda: attn.qk_norm_rope(x, x, None, inv), lambda: attn.qk_norm_rope(x, x, pos, None),
        lambda: attn.qk_norm_rope(x, x, pos, inv.double()), lambda: attn.qk_norm_rope(x, x, pos.cpu(), inv),
        lambda: attn.qk_norm_rope(x, x, pos, inv, sections=[31]), lambda: attn.qk_norm_rope(x, x, pos, inv, sections=[16, 16]),
        lambda: attn.qk_norm_rope(x, x, pos, inv, w), lambda: attn.qk_norm_rope(x, x, pos, inv, w, w.bfloat16()),
        lambda: attn.qk_norm_rope(x, x, pos, inv, w[:32], w[:32]),
        lambda: attn.qk_norm_rope(x, x, pos, inv, w, w, q_out=x[:, :1].expand(6, 2, 64)),
        lambda: attn.qk_norm_rope(x, x, pos, inv, w, w, q_out=torch.empty_like(x)[:, :1]),
        lambda: attn.qk_norm_rope_bwd(None, None, x, x, pos, inv, w, w),
        lambda: attn.qk_norm_rope_bwd(x, x, x[:5], x, pos, inv, w, w),
        lambda: attn.qk_norm_rope(x, x, torch.zeros((6, 2), dtype=torch.int32, device="cuda")[:, 0], inv),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    y = torch.zeros((6, 2, 72), dtype=torch.bfloat16, device="cuda")
    for call, status in ((lambda: attn.qk_norm_rope(y, y), 2), (lambda: attn.qk_norm_rope(y[..., 4:68], x), 3),
                         (lambda: attn.qk_norm_rope(x, x, pos, inv[:4]), 1),
                         (lambda: attn.qk_norm_rope(x, x, pos, inv, w, w, eps=-1.0), 1),
                         (lambda: attn.qk_norm_rope(x[:0], x[:0], pos[:0], inv), 1),
                         (lambda: attn.qk_norm_rope_bwd(x, x, x, x, pos, inv, w, w,
                                                        workspace=torch.empty(64, dtype=torch.uint8, device="cuda")), 6)):
        with pytest.raises(attn.AttnError) as e:
            call()
        assert e.value.status == status
