"""Calls of the 4-bit cache and attention over it at the edges of what their
documentation allows."""
import numpy as np
import pytest
import torch

import exact_attention_134_b200 as attn
from oracle import kv4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    attn.lib()


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _pages_of(n, H, d, page, g):
    """A pool of n full pages, and what each kv head's records of them stand for, page after page."""
    k = torch.randn((n * page, H, d), generator=g) * (1 + 5 * (torch.rand(d, generator=g) < 0.1))
    v = torch.randn((n * page, H, d), generator=g)
    pool = torch.zeros((n, H, page // 16, 20 * d), dtype=torch.uint8, device="cuda")
    attn.kv4_append(k.bfloat16().cuda(), v.bfloat16().cuda(), pool, _ints([list(range(n))]), _ints([n * page]))
    return pool, [kv4.read_cache(pool.cpu().numpy(), list(range(n)), n * page, h) for h in range(H)]


def _repeated_fp64(q, cache, counts, scale, chain):
    """Attention of one row q [d] over the cache's tokens, token j counted counts[j] times:
    (O, LSE, tol_O, tol_LSE). Tolerances as the oracle derives them for a few tokens, with the
    roundings of `chain` additions one behind the other on top: 2^-24 of a sum of weights, 2^-23 of a
    matrix instruction's accumulator, each of the size of all that is summed."""
    x = scale * (cache["k"] @ q)
    there = counts > 0
    m = x[there].max()
    p = counts * np.exp(np.minimum(x - m, 0.0))
    l = p.sum()
    w = p / l
    O, L = w @ cache["v"], m + np.log(l)
    size = scale * ((cache["ks"] * cache["kc"] + np.abs(cache["kl"])) @ np.abs(q))
    ex = 2.0 ** -19 * size[there].max() + 2.0 ** -20
    vs = cache["vs"][there].max()
    ex += 2 * 2.0 ** -24 * np.log(2) * (8 + abs(np.log2(max(vs, 2.0 ** -126))))
    codes, minima = w @ (cache["vs"] * cache["vc"]), w @ np.abs(cache["vl"])
    tO = 2.0 ** -8 * np.abs(O) + (2.0 ** -11 + 2 * ex) * codes + (2.0 ** -15 + 2 * ex) * minima
    tO += 15 * counts.sum() * 2.0 ** -32 * vs / l + chain * (2.0 ** -23 * (codes + minima) + 2.0 ** -24 * np.abs(O))
    return O, L, tO, ex + 2.0 ** -22 * abs(L) + chain * 2.0 ** -24


def _chain(tokens, ctas):
    """Additions behind one another: two for each of a warp's records, then shuffles, warps and parts."""
    return 2 * -(-tokens // (16 * 4 * ctas)) + 700


def test_the_longest_page_tables():
    """2^31 - 65536 tokens in 8 pages that repeat, one row a sequence; lengths beyond that are clamped."""
    d, page, most = 64, 1024, 2 ** 31 - 65536
    g = torch.Generator().manual_seed(21)
    pool, (cache,) = _pages_of(8, 1, d, page, g)
    table = torch.randint(0, 8, (2, most // page), generator=g).int()
    lens = [most, 2 ** 31 - 1]
    q = torch.randn((2, 2, d), generator=g).bfloat16()
    o, lse = attn.attn_fwd_kv4(q.cuda(), pool, table.cuda(), _ints(lens), causal=True)
    assert attn.get_status() == (0, 0)
    for s in range(2):
        counts = np.repeat(np.bincount(table[s].numpy(), minlength=8), page)
        for h in range(2):
            O, L, tO, tL = _repeated_fp64(_np(q[s, h]), cache, counts, 0.125, _chain(2 * most, 296))
            assert abs(float(lse[h, s]) - L) <= tL
            assert (np.abs(_np(o[s, h]) - O) <= tO).all()
    # the last tokens read back, and written
    last = int(table[0, -1])
    k, v = attn.kv4_gather(pool, table.cuda(), _ints(lens), 6)
    whole, _ = attn.kv4_gather(pool, _ints([[last]]), _ints([page]), 3)
    assert torch.equal(k[:3], whole)
    pool2 = pool.clone()
    attn.kv4_append(k[:3] + 1, v[:3], pool, table[:1].cuda(), _ints(lens[:1]))
    attn.kv4_append(k[:3] + 1, v[:3], pool2, _ints([[last]]), _ints([page]))
    assert torch.equal(pool, pool2) and attn.get_status() == (0, 0)


@pytest.mark.parametrize("Hq", [3, 8, 14])
@pytest.mark.parametrize("up", [-120, -112, 0, 90, 102])
def test_queries_of_every_size(Hq, up):
    """Queries and keys of inverse sizes: the same scores; rows whose largest value is 2^106 or more are NaN."""
    g = torch.Generator().manual_seed(22)
    n, d = 70, 128
    k = torch.randn((n, 1, d), generator=g) * 2.0 ** -up
    v = torch.randn((n, 1, d), generator=g)
    q = torch.randn((1, Hq, d), generator=g).clamp(-7, 7) * 2.0 ** up
    pool = torch.zeros((5, 1, 1, 20 * d), dtype=torch.uint8, device="cuda")
    args = pool, _ints([[3, 0, 4, 1, 2]]), _ints([n])
    attn.kv4_append(k.bfloat16().cuda(), v.bfloat16().cuda(), *args)
    cache = kv4.read_cache(pool.cpu().numpy(), [3, 0, 4, 1, 2], n, 0)
    q = q.bfloat16()
    O, L, tO, tL = kv4.attention_kv4_fp64(_np(q), [cache], True, d ** -0.5)
    o, lse = attn.attn_fwd_kv4(q.cuda(), *args, causal=True)
    assert (np.abs(_np(o) - O) <= tO).all() and (np.abs(_np(lse).T - L) <= tL).all()
    for large in (-2.0 ** 106, 2.0 ** 127, float("inf"), float("-inf"), float("nan")):
        bad = q.clone()
        bad[0, 1] = 0
        bad[0, 1, 77] = large
        o2, lse2 = attn.attn_fwd_kv4(bad.cuda(), *args, causal=True)
        assert o2[0, 1].isnan().all() and lse2[1].isnan().all()
        rest = [h for h in range(Hq) if h != 1]
        assert (np.abs(_np(o2) - O) <= tO)[:, rest].all() and (np.abs(_np(lse2).T - L) <= tL)[:, rest].all()
    edge = torch.zeros_like(q)  # the largest allowed: finite
    edge[0, 0, 5] = -255 * 2.0 ** 98
    small = torch.zeros((1, 1, 1, 20 * d), dtype=torch.uint8, device="cuda")
    one = small, _ints([[0]]), _ints([1])
    attn.kv4_append((torch.randn((1, 1, d), generator=g) * 2.0 ** -100).bfloat16().cuda(), v[:1].bfloat16().cuda(), *one)
    o3, lse3 = attn.attn_fwd_kv4(edge.cuda(), *one)
    O, L, tO, tL = kv4.attention_kv4_fp64(_np(edge), [kv4.read_cache(small.cpu().numpy(), [0], 1, 0)], True, d ** -0.5)
    assert (np.abs(_np(o3) - O) <= tO).all() and (np.abs(_np(lse3).T - L) <= tL).all()
    assert attn.get_status() == (0, 0)


@pytest.mark.parametrize("Hq", [4, 8, 13])
@pytest.mark.parametrize("what", ["one large token", "one large group", "large first", "2^-75", "2^-90", "2^-110"])
def test_values_whose_scales_lie_far_apart(Hq, what):
    """What the fp16 range of weights times scales leaves: 2^-32 of the row's largest product, over all
    tokens and groups, where scales below 2^-64 count as 2^-64."""
    g = torch.Generator().manual_seed(23)
    n, d = 150, 128
    k, v = torch.randn((n, 1, d), generator=g), torch.randn((n, 1, d), generator=g)
    if what == "one large token":
        v[77] *= 2.0 ** 24
    elif what == "one large group":
        v[77, :, 32:64] *= 2.0 ** 30
    elif what == "large first":
        v[0] *= 2.0 ** 40
        k[0] = 0
    else:
        v *= 2.0 ** int(what[2:])
    q = torch.randn((1, Hq, d), generator=g).bfloat16()
    pool = torch.zeros((10, 1, 1, 20 * d), dtype=torch.uint8, device="cuda")
    args = pool, _ints([list(range(10))]), _ints([n])
    attn.kv4_append(k.bfloat16().cuda(), v.bfloat16().cuda(), *args)
    o, lse = attn.attn_fwd_kv4(q.cuda(), *args, causal=True)
    assert attn.get_status() == (0, 0)
    cache = kv4.read_cache(pool.cpu().numpy(), list(range(10)), n, 0)
    # the oracle's bound has the largest scale that there is; 2^-64 stands for a smaller one
    O, L, tO, tL = kv4.attention_kv4_fp64(_np(q), [cache], True, d ** -0.5)
    x = d ** -0.5 * (cache["k"] @ _np(q)[0].T)
    low = 15 * n * 2.0 ** -32 * max(0.0, 2.0 ** -64 - cache["vs"].max()) / np.exp(x - x.max(0)).sum(0)
    assert (np.abs(_np(o) - O) <= tO + low[None, :, None]).all()
    assert (np.abs(_np(lse).T - L) <= tL).all()


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
