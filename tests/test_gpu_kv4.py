"""The 4-bit cache on the GPU (append, gather, page copies) and attention over
it, against the integer and fp64 oracle.

What the cache holds is compared bit by bit. Attention's tolerances are derived
where the oracle computes them (oracle/kv4.py: bf16 results, fp16 weights times
scales, 16-bit weights of the minima, fp32 scores).
"""
import numpy as np
import pytest
import torch

import exact_attention_134_b200 as attn
import oracle
from oracle import kv4
from synthetic import bf16_bits

pytestmark = pytest.mark.gpu

HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    attn.lib()


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _table(lens, page, g, spare=3):
    """A page table in random order, entries behind the last page far outside the pool, and the pool's pages."""
    need = [-(-n // page) for n in lens]
    ids = torch.randperm(sum(need) + spare, generator=g).tolist()
    most = max(1, max(need))
    rows = []
    for n in need:
        rows.append([ids.pop() for _ in range(n)] + [10 ** 9] * (most - n))
    return rows, sum(need) + spare


def _keys_values(n, H, d, g):
    k = torch.randn((n, H, d), generator=g) * (1 + 5 * (torch.rand(d, generator=g) < 0.1))
    return k.bfloat16(), torch.randn((n, H, d), generator=g).bfloat16()


def _filled(lens, H, d, page, seed):
    """A pool of random bytes with the records of `lens` tokens written by the oracle's layout (whole, in numpy)."""
    g = torch.Generator().manual_seed(seed)
    rows, pages = _table(lens, page, g)
    pool = torch.randint(0, 256, (pages, H, page // 16, 20 * d), generator=g, dtype=torch.uint8).cuda()
    k, v = _keys_values(max(1, sum(lens)), H, d, g)
    k, v = k[:sum(lens)], v[:sum(lens)]
    if sum(lens):
        attn.kv4_append(k.cuda(), v.cuda(), pool, _ints(rows), _ints(lens), _ints(np.cumsum([0] + lens).tolist()))
    return pool, rows, k, v


# ------------------------------------------------------------ append and gather

@pytest.mark.parametrize("d,page,Hkv", [(64, 16, 1), (96, 32, 3), (128, 64, 2), (256, 1024, 1), (128, 16, 5)])
@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("many", [False, True])
def test_append_writes_the_new_tokens_and_nothing_else(d, page, Hkv, ragged, many):
    g = torch.Generator().manual_seed(d + page)
    lens, new = ([5, 40, 33, 16], [5, 17, 0, 3]) if ragged else ([20, 4, 33], [3, 3, 3])
    if many:  # whole records
        lens, new = ([70, 100, 33, 200, 16], [40, 100, 0, 137, 16]) if ragged else ([64, 50, 91], [48, 48, 48])
    rows, pages = _table(lens, page, g)
    pool = torch.randint(0, 256, (pages, Hkv, page // 16, 20 * d), generator=g, dtype=torch.uint8)
    total = sum(new)
    extra = 2 if ragged else 0        # rows behind the last sequence
    qkv = torch.zeros((total + extra, 2 * Hkv + 1, d))
    qkv[:, 1:1 + Hkv], qkv[:, 1 + Hkv:] = (x.float() for x in _keys_values(total + extra, Hkv, d, g))
    qkv[0, 1, :32] = 2.5                                   # no spread
    qkv[1, 1, 32:64] = torch.linspace(-1e-38, 1e-38, 32)   # spread below what a scale holds
    qkv[2, 2, 5] = float("nan") if Hkv > 1 else 1.0
    qkv[2, 1, 40] = float("inf")
    qkv[2, 1 + Hkv, :32] = torch.tensor([-3.3e38, 3.3e38] * 16)
    qkv = qkv.bfloat16().cuda()
    k, v = qkv[:, 1:1 + Hkv], qkv[:, 1 + Hkv:]
    want = pool.numpy().copy()
    kb, vb = bf16_bits(k.cpu()), bf16_bits(v.cpu())
    t = 0
    for s, (n, m) in enumerate(zip(lens, new)):
        for j in range(n - m, n):
            for h in range(Hkv):
                kv4.write_token(want[rows[s][j // page], h, j // 16 % (page // 16)], j % 16, kb[t, h], vb[t, h])
            t += 1
    pool = pool.cuda()
    cu = _ints(np.cumsum([0] + new).tolist()) if ragged else None
    attn.kv4_append(k, v, pool, _ints(rows), _ints(lens), cu)
    assert attn.get_status()[0] == 0
    assert np.array_equal(pool.cpu().numpy(), want)
    # and back, as the nearest bf16 of what the records stand for
    ko, vo = (torch.full((total + extra, Hkv, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    attn.kv4_gather(pool, _ints(rows), _ints(lens), total + extra, cu, k=ko, v=vo)
    assert attn.get_status()[0] == 0
    t = 0
    for s, (n, m) in enumerate(zip(lens, new)):
        for j in range(n - m, n):
            for h in range(Hkv):
                x, y, _, _ = kv4.read_token(want[rows[s][j // page], h, j // 16 % (page // 16)], j % 16)
                for got, val in ((ko[t, h], x), (vo[t, h], y)):
                    got = got.float().cpu().numpy().astype(np.float64)
                    assert np.array_equal(np.isnan(got), np.isnan(val))
                    ok = ~np.isnan(val)
                    assert (np.abs(got - val)[ok] <= HALF_BF16 * np.abs(val[ok])).all()
            t += 1
    assert (ko[t:] == 7).all() and (vo[t:] == 7).all()     # rows that no sequence owns


@pytest.mark.parametrize("n", [5, 37])
def test_append_of_more_tokens_than_cached_and_gather_before_the_first(n):
    g = torch.Generator().manual_seed(3)
    pool = torch.randint(0, 256, (4, 2, 4, 20 * 64), generator=g, dtype=torch.uint8).cuda()
    k, v = (x.cuda() for x in _keys_values(2 * n, 2, 64, g))
    a, b = pool.clone(), pool.clone()
    attn.kv4_append(k, v, a, _ints([[1], [3]]), _ints([3, n]))             # n rows each: n - 3 are before token 0
    attn.kv4_append(k[n - 3:], v[n - 3:], b, _ints([[1], [3]]), _ints([3, n]), _ints([0, 3, n + 3]))
    assert torch.equal(a, b)
    ko, vo = attn.kv4_gather(a, _ints([[1], [3]]), _ints([3, 0]), 2 * n - 2)
    assert not ko[:n - 4].any() and ko[n - 4:n - 1].any(-1).all() and not ko[n - 1:].any() and not vo[n - 1:].any()
    whole, _ = attn.kv4_gather(a, _ints([[1], [3]]), _ints([3, n]), n + 3, _ints([0, 3, n + 3]))
    assert torch.equal(whole[:3], ko[n - 4:n - 1])
    assert attn.get_status()[0] == 0


def test_ties_of_the_quantiser_go_to_even():
    """Quotients of a half exactly, for every scale of 8 bits: codes k and k + 1 are as near, the even one is held."""
    m = torch.arange(128, 256).float()                                  # scales m * 2^-9
    x = torch.zeros(128, 1, 64)
    x[:, 0, 15] = 15 * m                                                # max, min 0: a span of 15 scales
    x[:, 0, 1:15] = (torch.arange(14) + 0.5) * m[:, None]
    x = x * 2.0 ** -9
    x[:, 0, 32:] = -x[:, 0, :32]
    b = x.bfloat16()
    rows = [[0, 1]]
    want = np.zeros((2, 1, 4, 20 * 64), np.uint8)
    bits = bf16_bits(b)
    for j in range(128):
        kv4.write_token(want[j // 64, 0, j // 16 % 4], j % 16, bits[j, 0], bits[j, 0])
    for new in (128, 1):  # whole records, then single rows
        pool = torch.zeros((2, 1, 4, 20 * 64), dtype=torch.uint8, device="cuda")
        for at in range(0, 128, new):
            attn.kv4_append(b[at:at + new].cuda(), b[at:at + new].cuda(), pool, _ints(rows), _ints([at + new]))
        assert np.array_equal(pool.cpu().numpy(), want)


def test_lengths_are_clamped_to_the_table_and_bad_pages_reported():
    g = torch.Generator().manual_seed(4)
    pool = torch.randint(0, 256, (4, 2, 2, 20 * 64), generator=g, dtype=torch.uint8).cuda()
    k, v = (x.cuda() for x in _keys_values(2, 2, 64, g))
    a, b = pool.clone(), pool.clone()
    attn.kv4_append(k, v, a, _ints([[1], [3]]), _ints([100, 32]))
    attn.kv4_append(k, v, b, _ints([[1], [3]]), _ints([32, 32]))
    assert torch.equal(a, b) and attn.get_status()[0] == 0
    c = pool.clone()
    for bad in (4, -1, 2 ** 31 - 1, -2 ** 31):
        attn.kv4_append(k, v, c, _ints([[bad], [3]]), _ints([7, 32]))
        assert attn.get_status() == (1, 0x510)
        ko, vo = attn.kv4_gather(c, _ints([[bad], [3]]), _ints([7, 32]), 2)
        assert attn.get_status() == (1, 0x520)
        assert not ko[0].any() and not vo[0].any() and ko[1].any()
    ref = pool.clone()
    attn.kv4_append(k[1:], v[1:], ref, _ints([[3]]), _ints([32]))
    assert torch.equal(c, ref) and attn.get_status() == (0, 0)


# ------------------------------------------------------------------ page copies

@pytest.mark.parametrize("layers,pages,H,page,d,n", [(1, 9, 1, 16, 64, 1), (3, 40, 5, 16, 96, 11), (2, 12, 2, 128, 256, 5)])
def test_copy_pages(layers, pages, H, page, d, n):
    g = torch.Generator().manual_seed(n)
    pool = torch.randint(0, 256, (layers, pages, H, page // 16, 20 * d), generator=g, dtype=torch.uint8).cuda()
    ids = torch.randperm(pages, generator=g)
    src, dst = ids[:n].clone(), ids[n:2 * n]
    if n > 2:
        src[1] = src[0]                                    # one page to two places
    want = pool.clone()
    want[:, dst.cuda()] = pool[:, src.cuda()]
    attn.kv4_copy_pages(pool, src.int().cuda(), dst.int().cuda())
    assert torch.equal(pool, want) and attn.get_status()[0] == 0
    one = pool[0].clone()
    attn.kv4_copy_pages(one, src.int().cuda(), src.int().cuda())
    assert torch.equal(one, pool[0])
    attn.kv4_copy_pages(one, _ints([0, pages, -1, 0]), _ints([1, 2, 2, -5]))
    want1 = pool[0].clone()
    want1[1] = want1[0]
    assert torch.equal(one, want1) and attn.get_status() == (1, 0x530)


# -------------------------------------------------------------------- attention

def _check(q, pool, rows, lens, cu, Hkv, page, causal, scale, o, lse):
    pool_np = pool.cpu().numpy()
    o, lse = o.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    for s, n in enumerate(lens):
        a, b = cu[s], cu[s + 1]
        if a == b:
            continue
        caches = [kv4.read_cache(pool_np, rows[s], n, h) for h in range(Hkv)]
        O, L, tO, tL = kv4.attention_kv4_fp64(q[a:b].float().numpy().astype(np.float64), caches, causal, scale)
        empty = np.isneginf(L)
        assert np.array_equal(np.isneginf(lse[:, a:b].T), empty), s
        assert not o[a:b][empty].any()
        err, errl = np.abs(o[a:b] - O), np.abs(np.subtract(lse[:, a:b].T, L, where=~empty, out=np.zeros_like(L)))
        assert (err <= tO).all(), (s, (err / np.maximum(tO, 1e-30)).max())
        assert (errl <= tL).all(), (s, (errl / np.maximum(tL, 1e-30)).max())


LENS = [1, 15, 16, 17, 100, 0, 33]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("nq", [1, 2, 5])
@pytest.mark.parametrize("d,page,Hq,Hkv", [(64, 16, 4, 4), (96, 32, 6, 2), (128, 64, 8, 1), (256, 16, 14, 2), (128, 128, 3, 1)])
def test_attention(d, page, Hq, Hkv, nq, causal):
    pool, rows, _, _ = _filled(LENS, Hkv, d, page, seed=d + nq)
    g = torch.Generator().manual_seed(9)
    q = torch.randn((nq * len(LENS), Hq, d), generator=g).bfloat16()
    o, lse = attn.attn_fwd_kv4(q.cuda(), pool, _ints(rows), _ints(LENS), causal=causal)
    assert attn.get_status() == (0, 0)
    _check(q, pool, rows, LENS, [nq * i for i in range(len(LENS) + 1)], Hkv, page, causal, d ** -0.5, o, lse)


@pytest.mark.parametrize("d,Hq,Hkv,told", [(128, 4, 2, 13), (64, 8, 1, 13), (128, 4, 2, 1), (256, 4, 2, 13), (96, 2, 2, 40)])
def test_ragged_query_rows(d, Hq, Hkv, told):
    """Sequences of other numbers of query rows, none, more than are cached, more than was announced;
    rows that no sequence owns stay as they were."""
    lens, new = [40, 300, 3, 77, 0, 513], [1, 13, 5, 0, 2, 7]
    pool, rows, _, _ = _filled(lens, Hkv, d, 32, seed=d)
    cu = np.cumsum([0] + new).tolist()
    total = cu[-1] + 3
    q = torch.randn((total, Hq, d), generator=torch.Generator().manual_seed(1)).bfloat16()
    out = torch.full((total, Hq, d), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((Hq, total), 3.0, device="cuda")
    attn.attn_fwd_kv4(q.cuda(), pool, _ints(rows), _ints(lens), _ints(cu), told, causal=True, scale=0.2, out=out, lse=lse)
    assert attn.get_status() == (0, 0)
    assert (out[cu[-1]:] == 3).all() and (lse[:, cu[-1]:] == 3).all()
    _check(q, pool, rows, lens, cu, Hkv, 32, True, 0.2, out, lse)


def test_long_and_short_sequences_split_over_the_gpu():
    """Ranges that cut sequences, several sequences in a range, results joined from many."""
    lens = [3000, 1, 700, 16, 2049]
    pool, rows, _, _ = _filled(lens, 2, 64, 64, seed=5)
    q = torch.randn((len(lens), 4, 64), generator=torch.Generator().manual_seed(2)).bfloat16()
    args = (q.cuda(), pool, _ints(rows), _ints(lens))
    o, lse = attn.attn_fwd_kv4(*args, causal=True)
    assert attn.get_status() == (0, 0)
    _check(q, pool, rows, lens, list(range(6)), 2, 64, True, 0.125, o, lse)
    for _ in range(3):  # the same bits every time
        again = attn.attn_fwd_kv4(*args, causal=True)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


def test_many_sequences():
    g = torch.Generator().manual_seed(6)
    lens = torch.randint(0, 60, (301,), generator=g).tolist()
    pool, rows, _, _ = _filled(lens, 1, 64, 16, seed=6)
    q = torch.randn((301, 2, 64), generator=g).bfloat16()
    o, lse = attn.attn_fwd_kv4(q.cuda(), pool, _ints(rows), _ints(lens), causal=True)
    assert attn.get_status() == (0, 0)
    _check(q, pool, rows, lens, list(range(302)), 1, 16, True, 0.125, o, lse)


@pytest.mark.parametrize("what", ["large", "small", "peaked", "spread scales", "rising"])
def test_values_of_unusual_size(what):
    g = torch.Generator().manual_seed(11)
    n, d = 200, 128
    k, v = (x.float() for x in _keys_values(n, 1, d, g))
    q = torch.randn((1, 8, d), generator=g)
    if what == "large":
        v *= 2.0 ** 55
        q *= 2.0 ** 30
        k *= 2.0 ** -30
    elif what == "small":
        v *= 2.0 ** -60
        k *= 2.0 ** -40
    elif what == "peaked":
        q *= 40
    elif what == "spread scales":
        v *= torch.exp2(torch.randint(-6, 7, (n, 1, d // 32), generator=g).float()).repeat_interleave(32, -1)
    else:  # every key's score above the last one's, by a lot
        k = q[:, :1] * torch.linspace(-3, 3, n)[:, None, None] + 0.1 * k
    k, v, q = k.bfloat16(), v.bfloat16(), q.bfloat16()
    rows = [[2, 0, 5, 1]]
    pool = torch.zeros((6, 1, 4, 20 * d), dtype=torch.uint8, device="cuda")
    attn.kv4_append(k.cuda(), v.cuda(), pool, _ints(rows), _ints([n]))
    o, lse = attn.attn_fwd_kv4(q.cuda(), pool, _ints(rows), _ints([n]), causal=True)
    assert attn.get_status() == (0, 0)
    _check(q, pool, rows, [n], [0, 1], 1, 64, True, d ** -0.5, o, lse)


@pytest.mark.parametrize("heads", [1, 2, 6])
def test_a_row_sees_no_nan_behind_its_mask(heads):
    """Keys and values of NaN reach the rows that see them, and no others; what a record
    holds behind the last token (anything at all) reaches none."""
    g = torch.Generator().manual_seed(12)
    n, d = 37, 64
    k, v = _keys_values(n, 1, d, g)
    kn, vn = k.clone(), v.clone()
    kn[36, 0, 3] = float("nan")
    vn[35, 0, 40] = float("inf")
    q = torch.randn((3, heads, d), generator=g).bfloat16()
    pool = torch.full((3, 1, 1, 20 * d), 0xff, dtype=torch.uint8, device="cuda")   # scales and minima of NaN
    clean = torch.zeros_like(pool)
    table, lens = _ints([[0, 1, 2]]), _ints([n])
    attn.kv4_append(kn.cuda(), vn.cuda(), pool, table, lens)
    attn.kv4_append(k.cuda(), v.cuda(), clean, table, lens)
    o, lse = attn.attn_fwd_kv4(q.cuda(), pool, table, lens, causal=True)
    oc, lc = attn.attn_fwd_kv4(q.cuda(), clean, table, lens, causal=True)
    assert torch.equal(o[0], oc[0]) and torch.equal(lse[:, :2], lc[:, :2])
    assert torch.equal(o[1, :, :32], oc[1, :, :32]) and o[1, :, 32:].isnan().all()
    assert o[2].isnan().all() and lse[:, 2].isnan().all()


@pytest.mark.parametrize("Hq,page", [(4, 16), (4, 64), (12, 32), (20, 16)])
def test_bad_pages_are_left_out_and_reported(Hq, page):
    lens = [70, 20]
    pool, rows, _, _ = _filled(lens, 2, 64, page, seed=13)
    q = torch.randn((2, Hq, 64), generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    at = min(2, len(rows[0]) - 1)
    want, wl = attn.attn_fwd_kv4(q[1:], pool, _ints(rows[1:]), _ints(lens[1:]))
    for bad in (pool.shape[0], -1, 2 ** 31 - 1, -2 ** 31):
        broken = [[*rows[0][:at], bad, *rows[0][at + 1:]], rows[1]]
        o, lse = attn.attn_fwd_kv4(q, pool, _ints(broken), _ints(lens))
        assert attn.get_status() == (1, 0x500)
        assert o[0].isfinite().all() and torch.equal(o[1:], want) and torch.equal(lse[:, 1:], wl)
        if at * page + page >= lens[0]:  # the last page: as if the sequence ended before it
            short, sl = attn.attn_fwd_kv4(q[:1], pool, _ints(rows[:1]), _ints([at * page]))
            assert torch.equal(o[:1], short) and torch.equal(lse[:, :1], sl)
    assert attn.get_status() == (0, 0)


def test_offsets_beyond_32_bits():
    """Pages more than 2^32 bytes into the pool."""
    H, page, d = 8, 64, 128
    big = torch.empty(2 ** 32 + 2 ** 28, dtype=torch.uint8, device="cuda")
    pages = big.numel() // attn.kv4_page_bytes(H, d, page)
    pool = big[:pages * attn.kv4_page_bytes(H, d, page)].view(pages, H, page // 16, 20 * d)
    g = torch.Generator().manual_seed(14)
    k, v = (x.cuda() for x in _keys_values(70, H, d, g))
    q = torch.randn((1, 16, d), generator=g).bfloat16().cuda()
    small = torch.zeros((2, H, page // 16, 20 * d), dtype=torch.uint8, device="cuda")
    lens = _ints([70])
    for p, table in ((pool, _ints([[pages - 1, pages - 2]])), (small, _ints([[0, 1]]))):
        attn.kv4_append(k, v, p, table, lens)
    a = attn.attn_fwd_kv4(q, pool, _ints([[pages - 1, pages - 2]]), lens)
    b = attn.attn_fwd_kv4(q, small, _ints([[0, 1]]), lens)
    ka = attn.kv4_gather(pool, _ints([[pages - 1, pages - 2]]), lens, 70)
    kb = attn.kv4_gather(small, _ints([[0, 1]]), lens, 70)
    attn.kv4_copy_pages(pool, _ints([pages - 1]), _ints([0]))
    c = attn.attn_fwd_kv4(q, pool, _ints([[0, pages - 2]]), lens)
    assert attn.get_status() == (0, 0)
    for x in (a, c):
        assert torch.equal(x[0], b[0]) and torch.equal(x[1], b[1])
    assert torch.equal(ka[0], kb[0]) and torch.equal(ka[1], kb[1])


def test_two_streams_with_their_own_workspaces_and_a_replayed_graph():
    lens = [900, 40, 333]
    pool, rows, _, _ = _filled(lens, 2, 128, 16, seed=15)
    g = torch.Generator().manual_seed(4)
    qs = [torch.randn((3, 8, 128), generator=g).bfloat16().cuda() for _ in range(2)]
    table, n = _ints(rows), _ints(lens)
    want = [attn.attn_fwd_kv4(q, pool, table, n, causal=True) for q in qs]
    need = attn.fwd_kv4_workspace_size(8, 2, 1, 128)
    ws = [torch.full((need,), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [(torch.empty_like(w[0]), torch.empty_like(w[1])) for w in want]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for s, q, w, o in zip(streams, qs, ws, outs):
            with torch.cuda.stream(s):
                attn.attn_fwd_kv4(q, pool, table, n, causal=True, workspace=w, out=o[0], lse=o[1])
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert torch.equal(w[0], o[0]) and torch.equal(w[1], o[1])
    # one decode step captured: the lengths grow between the replays
    k, v = (x.cuda() for x in _keys_values(3, 2, 128, g))
    grow = _ints([890, 30, 320])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn.kv4_append(k, v, pool, table, grow)
        o, lse = attn.attn_fwd_kv4(qs[0], pool, table, grow, causal=True, workspace=ws[0])
        grow.add_(1)
    other = pool.clone()
    for step in range(4):
        k.copy_(torch.randn(k.shape, generator=g).bfloat16())
        graph.replay()
        at = _ints([890 + step, 30 + step, 320 + step])
        attn.kv4_append(k, v, other, table, at)
        ref = attn.attn_fwd_kv4(qs[0], other, table, at, causal=True)
        torch.cuda.synchronize()
        assert torch.equal(pool, other) and torch.equal(o, ref[0]) and torch.equal(lse, ref[1])
    assert attn.get_status() == (0, 0)


def test_no_memory_is_allocated_with_everything_supplied():
    lens = [500]
    pool, rows, k, v = _filled(lens, 2, 64, 16, seed=16)
    q = torch.randn((1, 4, 64), device="cuda").bfloat16()
    k, v, table, n = k[:1].cuda(), v[:1].cuda(), _ints(rows), _ints(lens)
    ws = torch.empty(attn.fwd_kv4_workspace_size(4, 2, 1, 64), dtype=torch.uint8, device="cuda")
    o, lse = attn.attn_fwd_kv4(q, pool, table, n, workspace=ws)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated(), torch.cuda.mem_get_info()[0], torch.cuda.memory_stats()["allocation.all.allocated"]
    for _ in range(3):
        attn.kv4_append(k, v, pool, table, n)
        attn.attn_fwd_kv4(q, pool, table, n, workspace=ws, out=o, lse=lse)
        attn.kv4_gather(pool, table, n, 1, k=k, v=v)
    torch.cuda.synchronize()
    assert before == (torch.cuda.memory_allocated(), torch.cuda.mem_get_info()[0],
                      torch.cuda.memory_stats()["allocation.all.allocated"])


# --------------------------------------------------------------- all of it together

def test_serving_two_forks_of_a_prompt():
    """A prompt in two chunks (append, gather, packed attention), forked, then decoded
    token by token with the norm, the rotation and the cache; against attention over what
    the cache holds of every branch's own history."""
    g = torch.Generator().manual_seed(17)
    Hq, Hkv, d, page, chunks, steps = 8, 2, 128, 16, [70, 31], 19
    inv = (1e4 ** (-torch.arange(64).float() / 64)).cuda()
    w = (1 + 0.1 * torch.randn(d, generator=g)).cuda()
    pages = attn.KV4Pages(40, page)
    pool = attn.kv4_alloc(40, Hkv, d, page)
    pool.random_(0, 256)

    def project(n):
        qkv = torch.randn((n, Hq + 2 * Hkv, d), generator=g).bfloat16().cuda()
        return qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]

    a = pages.new()
    history = {a: []}
    at = 0
    for n in chunks:
        q, k, v = project(n)
        pos = torch.arange(at, at + n, dtype=torch.int32, device="cuda")
        at += n
        q, k = attn.qk_norm_rope(q, k, pos, inv, w, w)
        assert pages.extend({a: n}) == []
        table, lens = pages.tables([a])
        attn.kv4_append(k, v, pool, table, lens)
        history[a].append((k, v))
        kc, vc = attn.kv4_gather(pool, table, lens, at)
        o, lse = attn.attn_fwd_varlen(q.contiguous(), kc, vc, _ints([0, n]), _ints([0, at]), n, causal=True)
        o4, lse4 = attn.attn_fwd_kv4(q.contiguous(), pool, table, lens, max_seqlen_q=n, causal=True)
        # one rounds keys, values and weights to bf16, the other does not: one step of 2^-8 each,
        # of scores below 2^4 and values below 2^3
        assert (lse - lse4).abs().max() <= 16 * HALF_BF16 and (o.float() - o4.float()).abs().max() <= 8 * 16 * HALF_BF16
    b = pages.fork(a)
    history[b] = list(history[a])
    for step in range(steps):
        pairs = pages.extend({a: 1, b: 1})
        if pairs:
            attn.kv4_copy_pages(pool, *attn.page_pairs(pairs))
        assert bool(pairs) == (step == 0)
        q, k, v = project(2)
        pos = torch.full((2,), at, dtype=torch.int32, device="cuda")
        at += 1
        q, k = attn.qk_norm_rope(q, k, pos, inv, w, w)
        table, lens = pages.tables([a, b])
        attn.kv4_append(k, v, pool, table, lens)
        history[a].append((k[:1], v[:1]))
        history[b].append((k[1:], v[1:]))
        o, lse = attn.attn_fwd_kv4(q, pool, table, lens, causal=True)
    pairs = pages.compact()
    if pairs:
        attn.kv4_copy_pages(pool, *attn.page_pairs(pairs))
    assert attn.get_status() == (0, 0)
    table, lens = pages.tables([a, b])
    again = attn.attn_fwd_kv4(q, pool, table, lens, causal=True)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)
    # a cache written at once from every branch's history is the same
    fresh = torch.zeros_like(pool)
    rows = [pages.pages(a), [p + 20 for p in range(len(pages.pages(b)))]]
    attn.kv4_append(*(torch.cat([torch.cat([x[i] for x in history[s]]) for s in (a, b)]) for i in (0, 1)), fresh,
                    _ints([list(range(len(rows[0]))), rows[1]]), lens)
    ref = attn.attn_fwd_kv4(q, fresh, _ints([list(range(len(rows[0]))), rows[1]]), lens, causal=True)
    assert torch.equal(ref[0], o) and torch.equal(ref[1], lse)
    _check(q.cpu(), pool, [pages.pages(a), pages.pages(b)], lens.tolist(), [0, 1, 2], Hkv, page, True, d ** -0.5, o, lse)


def test_refusals():
    pool = attn.kv4_alloc(4, 2, 64, 16)
    table, lens = _ints([[0], [1]]), _ints([3, 4])
    k = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    bad = [
        lambda: attn.kv4_append(k.float(), k, pool, table, lens), lambda: attn.kv4_append(k, k[:1], pool, table, lens),
        lambda: attn.kv4_append(k[:, :1], k[:, :1], pool, table, lens), lambda: attn.kv4_append(k, k, pool[:, :, :, :640], table, lens),
        lambda: attn.kv4_append(k, k, pool, table.long(), lens), lambda: attn.kv4_append(k, k, pool, table[0], lens),
        lambda: attn.kv4_append(k, k, pool, table, lens[:1]), lambda: attn.kv4_append(k, k, pool, table, lens, lens),
        lambda: attn.kv4_append(k, k, pool, table.cpu(), lens),
        lambda: attn.kv4_gather(pool, table, lens, 2, k=k.float()), lambda: attn.kv4_gather(pool, table, lens, 4, k=k),
        lambda: attn.attn_fwd_kv4(q.float(), pool, table, lens), lambda: attn.attn_fwd_kv4(q[:, ::2], pool, table, lens),
        lambda: attn.attn_fwd_kv4(q, pool, table, lens, out=torch.empty_like(q)[:1]),
        lambda: attn.attn_fwd_kv4(q, pool, table, lens, lse=torch.empty((2, 4), device="cuda")),
        lambda: attn.attn_fwd_kv4(torch.zeros((2, 4, 128), dtype=torch.bfloat16, device="cuda"), pool, table, lens),
        lambda: attn.kv4_copy_pages(pool, lens, lens[:1]), lambda: attn.kv4_copy_pages(pool, lens.long(), lens.long()),
        lambda: attn.kv4_copy_pages(pool[0], lens, lens),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    small = torch.empty(128, dtype=torch.uint8, device="cuda")
    for call, status in ((lambda: attn.kv4_gather(pool, table, lens, 3), 1), (lambda: attn.kv4_gather(pool, table, lens, 0), 1),
                         (lambda: attn.attn_fwd_kv4(q[:, :3].contiguous(), pool, table, lens), 1),
                         (lambda: attn.attn_fwd_kv4(q, pool, table, lens, scale=0.0), 1),
                         (lambda: attn.attn_fwd_kv4(q, pool, table, lens, workspace=small), 6),
                         (lambda: attn.attn_fwd_kv4(q, pool, _ints([[0] * 33] * 2), lens, workspace=small), 6),
                         (lambda: attn.kv4_copy_pages(pool, lens[:0], lens[:0]), 1)):
        with pytest.raises(attn.AttnError) as e:
            call()
        assert e.value.status == status
