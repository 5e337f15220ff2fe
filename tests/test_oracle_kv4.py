"""Pins of the oracles for the norm with rotation and for the 4-bit cache
(CPU only): float64 autograd, complex rotations, finite differences, round
trips, a second reading of a record's layout, plain softmax attention."""
import numpy as np
import pytest
import torch

import oracle
from oracle import kv4, norm_rope
from synthetic import bf16_bits


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot,norm", [(64, True), (32, True), (64, False), (0, True)])
def test_norm_rope_gradients_are_float64_autograd(rot, norm, interleaved):
    g = torch.Generator().manual_seed(5)
    x = torch.randn((2, 3, 5, 64), generator=g, dtype=torch.float64).requires_grad_()
    w = (1 + 0.2 * torch.randn(64, generator=g, dtype=torch.float64)).requires_grad_()
    dy = torch.randn((2, 3, 5, 64), generator=g, dtype=torch.float64)
    ang = torch.randn((2, 5, rot // 2), generator=g, dtype=torch.float64) * 3
    n = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-3) * w if norm else x * 1.0
    if rot:
        pairs = n[..., :rot].unflatten(-1, (rot // 2, 2)) if interleaved else n[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        z = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.ones_like(ang), ang)[:, None]
        z = torch.view_as_real(z)
        z = z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)
        n = torch.cat([z, n[..., rot:]], -1)
    n.backward(dy)
    args = (x.detach().numpy(), w.detach().numpy() if norm else None, 1e-3)
    y, mag = norm_rope.norm_rope_fp64(*args, ang.numpy(), interleaved)
    assert np.allclose(y, n.detach().numpy(), rtol=0, atol=1e-13)
    assert (mag >= np.abs(y) - 1e-13).all()
    dx, dw = norm_rope.norm_rope_bwd_fp64(*args, dy.numpy(), ang.numpy(), interleaved)
    assert np.allclose(dx, x.grad.numpy(), rtol=0, atol=1e-13)
    if norm:
        assert np.allclose(dw, w.grad.numpy(), rtol=0, atol=1e-12)


def test_norm_rope_gradient_is_the_difference_quotient():
    r = np.random.default_rng(1)
    x, w, dy = r.standard_normal((1, 2, 3, 64)), 1 + 0.1 * r.standard_normal(64), r.standard_normal((1, 2, 3, 64))
    ang = r.standard_normal((1, 3, 16))
    dx, dw = norm_rope.norm_rope_bwd_fp64(x, w, 1e-6, dy, ang)
    f = lambda x_, w_: (norm_rope.norm_rope_fp64(x_, w_, 1e-6, ang)[0] * dy).sum()  # noqa: E731
    h = 1e-5
    for at in [(0, 0, 0, 0), (0, 1, 2, 17), (0, 0, 1, 40)]:
        e = np.zeros_like(x)
        e[at] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[at]) < 1e-8
    e = np.zeros_like(w)
    e[9] = h
    assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[9]) < 1e-8


def test_angles_take_their_axis():
    pos = np.array([[[1, 2]], [[10, 20]], [[100, 200]]])
    a = norm_rope.rotation_angles(pos, np.array([1.0, 0.5, 0.25, 0.125]), [2, 0, 2])
    assert np.array_equal(a[0], [[1.0, 0.5, 25.0, 12.5], [2.0, 1.0, 50.0, 25.0]])


def test_quantiser_on_hand():
    def q(x):
        return kv4.quantise(bf16_bits(torch.tensor(x, dtype=torch.float32).bfloat16()))
    codes, s, lo = q([0.0] * 16 + [15.0] * 8 + [3.5, 4.5, 7.0, 14.5] * 2)
    assert oracle.widen_bf16(s)[0] == 1.0 and oracle.widen_bf16(lo)[0] == 0.0
    assert codes.tolist() == [0] * 16 + [15] * 8 + [4, 4, 7, 14] * 2     # ties to even
    codes, s, lo = q([-2.5] * 32)                                        # no spread: the minimum
    assert oracle.widen_bf16(s)[0] == 2.5 * 2.0 ** -13 and oracle.widen_bf16(lo)[0] == -2.5 and not codes.any()
    codes, s, lo = q([0.0] * 32)
    assert s[0] == 0 and lo[0] == 0 and not codes.any()
    for bad in (float("nan"), float("inf"), -float("inf")):
        codes, s, lo = q([1.0] * 31 + [bad])
        assert s[0] == 0x7fc0 and lo[0] == 0 and not codes.any()


@pytest.mark.parametrize("d", [64, 96, 128, 256])
def test_tokens_of_a_record_round_trip_and_share_no_bit(d):
    g = torch.Generator().manual_seed(d)
    x = bf16_bits(torch.randn((2, 16, d), generator=g).bfloat16())
    rec = np.random.default_rng(d).integers(0, 256, 20 * d).astype(np.uint8)
    order = np.random.default_rng(1).permutation(16)
    for r in order:
        kv4.write_token(rec, r, x[0, r], x[1, r])
    for r in range(16):
        k, v, _, _ = kv4.read_token(rec, r)
        for got, bits in ((k, x[0, r]), (v, x[1, r])):
            val = oracle.widen_bf16(bits).reshape(-1, 32)
            codes, s, lo = kv4.quantise(bits)
            assert np.array_equal(got, np.repeat(oracle.widen_bf16(lo), 32) + np.repeat(oracle.widen_bf16(s), 32) * codes)
            s_ = oracle.widen_bf16(s)[:, None]
            assert (np.abs(got.reshape(-1, 32) - val) <= s_ * (0.5 + 15 * 2.0 ** -8)).all()
    # every bit of a record belongs to one token: a second writing changes no other token's
    before = rec.copy()
    kv4.write_token(rec, 5, x[0, 6], x[1, 6])
    for r in range(16):
        if r != 5:
            assert np.array_equal(kv4.read_token(rec, r)[0], kv4.read_token(before, r)[0])
            assert np.array_equal(kv4.read_token(rec, r)[1], kv4.read_token(before, r)[1])


def test_layout_is_that_of_the_measured_plain_form():
    """The records that perf/operators.py packs whole are these, token by token."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "operators.py")
    spec = importlib.util.spec_from_file_location("operators_plain", path)
    plain = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(plain)
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn((3, 2, 32, 96), generator=g).bfloat16() for _ in range(2))
    pool = plain._pack(k.float(), v.float()).numpy()
    kb, vb = bf16_bits(k), bf16_bits(v)
    rec = np.zeros(20 * 96, np.uint8)
    for p, h, t in ((0, 0, 0), (2, 1, 1), (1, 0, 1)):
        for r in range(16):
            kv4.write_token(rec, r, kb[p, h, 16 * t + r], vb[p, h, 16 * t + r])
        assert np.array_equal(rec, pool[p, h, t])


@pytest.mark.parametrize("causal", [False, True])
def test_attention_over_the_cache_is_attention_over_its_values(causal):
    r = np.random.default_rng(3)
    pool = np.zeros((5, 2, 2, 20 * 64), np.uint8)
    table, N = [3, 0, 4], 70
    for j in range(N):
        for h in range(2):
            bits = bf16_bits(torch.tensor(r.standard_normal((2, 64))).bfloat16())
            kv4.write_token(pool[table[j // 32], h, j // 16 % 2], j % 16, bits[0], bits[1])
    caches = [kv4.read_cache(pool, table, N, h) for h in range(2)]
    q = r.standard_normal((4, 4, 64))
    O, L, tO, tL = kv4.attention_kv4_fp64(q, caches, causal, 0.3)
    for h in range(4):
        c = caches[h // 2]
        x = 0.3 * q[:, h] @ c["k"].T
        if causal:
            x = np.where(np.arange(N)[None] <= N - 4 + np.arange(4)[:, None], x, -np.inf)
        p = np.exp(x)
        assert np.allclose(O[:, h], p @ c["v"] / p.sum(1, keepdims=True), atol=1e-12)
        assert np.allclose(L[:, h], np.log(p.sum(1)), atol=1e-12)
    assert (tO > 0).all() and tO.max() < 0.02 and tL.max() < 1e-3
    # rows before the first token see nothing
    few = [kv4.read_cache(pool, table, 2, h) for h in range(2)]
    O, L, _, _ = kv4.attention_kv4_fp64(q, few, True, 0.3)
    assert np.isneginf(L[:2]).all() and not O[:2].any() and np.isfinite(L[2:]).all()
