"""Attention over the 4-bit cache where a CTA has much to do: many row blocks of
short caches one after the other, caches of 513 to 1024 tokens that are not
split, ranges of far more units than the ring has stages and one look-up of
pages finds. Sequences share the pages of small pools. Against the fp64 oracle."""
import numpy as np
import pytest
import torch

import exact_attention_134_b200 as attn
from oracle import kv4
from test_gpu_kv4_edges import _chain, _ints, _np, _pages_of, _repeated_fp64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    attn.lib()


@pytest.mark.parametrize("most", [500, 1000])  # tokens of the longest: always whole, whole because they are many
@pytest.mark.parametrize("d,Hq,Hkv,page,seqs,nq,causal", [
    (64, 4, 2, 16, 900, 1, True),       # 4 columns, 1800 row blocks of at most 592 CTAs
    (128, 16, 2, 32, 500, 1, False),    # 8 columns, 1000 of 444
    (128, 12, 1, 64, 700, 1, True),     # 16 columns, 700 of 296
    (256, 6, 2, 16, 330, 1, True),      # 4 columns, 660 of 296
    (96, 4, 2, 32, 300, 3, True),       # 8 columns, 600 of 444
    (64, 10, 1, 16, 320, 5, True),      # 16 columns, four blocks a sequence: 1280 of 444
])
def test_many_row_blocks(d, Hq, Hkv, page, seqs, nq, causal, most):
    g = torch.Generator().manual_seed(d + most)
    pool, caches = _pages_of(64, Hkv, d, page, g)
    table = torch.randint(0, 64, (seqs, -(-most // page)), generator=g)
    lens = torch.randint(0, most + 1, (seqs,), generator=g)
    lens[0], lens[1], lens[-1] = most, 0, most
    q = torch.randn((seqs * nq, Hq, d), generator=g).bfloat16()
    o, lse = attn.attn_fwd_kv4(q.cuda(), pool, table.int().cuda(), lens.int().cuda(), causal=causal)
    assert attn.get_status() == (0, 0)
    o, lse, q64 = _np(o), _np(lse), _np(q)
    for s in range(seqs):
        n, at = int(lens[s]), slice(s * nq, s * nq + nq)
        j = np.arange(n)
        token = table[s].numpy()[j // page] * page + j % page
        O, L, tO, tL = kv4.attention_kv4_fp64(q64[at], [{x: c[x][token] for x in c} for c in caches], causal, d ** -0.5)
        empty = np.isneginf(L)
        assert np.array_equal(np.isneginf(lse[:, at].T), empty), s
        assert (np.abs(o[at] - O) <= tO).all(), s
        assert (np.abs(np.subtract(lse[:, at].T, L, where=~empty, out=np.zeros_like(L))) <= tL).all(), s


@pytest.mark.parametrize("bad", [False, True])
@pytest.mark.parametrize("d,Hq,ctas", [(64, 4, 592), (128, 2, 444), (128, 7, 444), (128, 13, 296), (256, 3, 296), (96, 16, 296)])
def test_ranges_of_many_units(d, Hq, ctas, bad):
    """150 pairs of records a CTA, 37 or 38 a warp: the ring goes round and round, and each warp looks
    pages up twice. With a page that there is not, of the second look-up."""
    page = 128
    g = torch.Generator().manual_seed(d + Hq)
    pool, (cache,) = _pages_of(32, 1, d, page, g)
    lens = [ctas * 140 * 32 + 77, ctas * 10 * 32 - 5]
    table = torch.randint(0, 32, (2, -(-lens[0] // page)), generator=g)
    if bad:  # units 131 and 132 of a range in the middle
        table[0, (140 * (ctas // 2) + 131) * 32 // page] = 32
    q = torch.randn((2, Hq, d), generator=g).bfloat16()
    args = q.cuda(), pool, table.int().cuda(), _ints(lens)
    o, lse = attn.attn_fwd_kv4(*args, causal=True)
    assert attn.get_status() == ((1, 0x500) if bad else (0, 0))
    for s in range(2):
        counts = np.zeros((33, page))
        full, rest = divmod(lens[s], page)
        counts += np.bincount(table[s, :full].numpy(), minlength=33)[:, None]
        counts[int(table[s, full]) if rest else 0, :rest] += 1
        counts = counts[:32].reshape(-1)
        for h in range(Hq):
            O, L, tO, tL = _repeated_fp64(_np(q[s, h]), cache, counts, d ** -0.5, _chain(sum(lens), ctas))
            assert abs(float(lse[h, s]) - L) <= tL, (s, h, float(lse[h, s]), L, tL)
            assert (np.abs(_np(o[s, h]) - O) <= tO).all(), (s, h)
    again = attn.attn_fwd_kv4(*args, causal=True)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    attn.get_status()
