"""The host's bookkeeping of the 4-bit cache's pages (no GPU): random forks,
extensions, truncations and compactions against token lists copied whole."""
import random

import pytest
import torch

from exact_attention_134_b200.kv4_pages import KV4Pages, OutOfPages, page_pairs


class Shadow:
    """The pool as a list of pages of token names, and each sequence's tokens."""

    def __init__(self, pages: KV4Pages):
        self.p = pages
        self.pool = [[None] * pages.page_size for _ in range(pages.num_pages)]
        self.want = {}
        self.count = 0

    def copy(self, pairs, rng):
        src, dst = [a for a, _ in pairs], [b for _, b in pairs]
        assert len(set(dst)) == len(dst) and not set(dst) & set(src)
        pairs = list(pairs)
        rng.shuffle(pairs)  # in any order
        for a, b in pairs:
            self.pool[b] = list(self.pool[a])

    def append(self, tokens):
        ps = self.p.page_size
        for seq, n in tokens.items():
            held = self.p.pages(seq)
            for j in range(self.p.length(seq) - n, self.p.length(seq)):
                self.pool[held[j // ps]][j % ps] = self.count
                self.want[seq].append(self.count)
                self.count += 1

    def check(self):
        ps = self.p.page_size
        seen = set()
        for seq, want in self.want.items():
            held = self.p.pages(seq)
            assert self.p.length(seq) == len(want) and len(held) == -(-len(want) // ps)
            assert [self.pool[held[j // ps]][j % ps] for j in range(len(want))] == want
            seen |= set(held)
        assert self.p.free_pages == self.p.num_pages - len(seen)
        assert len(self.p) == len(self.want)


@pytest.mark.parametrize("seed", range(12))
def test_random_histories(seed):
    rng = random.Random(seed)
    s = Shadow(KV4Pages(rng.choice([7, 24, 60]), 16))
    for _ in range(300):
        seqs = list(s.want)
        what = rng.random()
        if what < 0.12 or not seqs:
            s.want[s.p.new()] = []
        elif what < 0.25:
            a = rng.choice(seqs)
            s.want[s.p.fork(a)] = list(s.want[a])
        elif what < 0.75:
            tokens = {a: rng.choice([0, 1, 1, 5, 16, 33]) for a in rng.sample(seqs, rng.randint(1, min(4, len(seqs))))}
            before = s.p.free_pages
            try:
                pairs = s.p.extend(tokens)
            except OutOfPages:
                assert s.p.free_pages == before
                s.check()
                s.want.pop(a := rng.choice(seqs))
                s.p.free(a)
                continue
            s.copy(pairs, rng)
            s.append(tokens)
        elif what < 0.85:
            a = rng.choice(seqs)
            n = rng.randint(0, len(s.want[a]))
            s.p.truncate(a, n)
            del s.want[a][n:]
        elif what < 0.95:
            a = rng.choice(seqs)
            s.p.free(a)
            del s.want[a]
        else:
            used = s.p.num_pages - s.p.free_pages
            s.copy(s.p.compact(), rng)
            assert all(p < used for a in s.want for p in s.p.pages(a))
        s.check()
    for a in list(s.want):
        s.p.free(a)
    assert s.p.free_pages == s.p.num_pages


def test_last_page_of_many_forks_is_copied_for_all_but_one():
    p = KV4Pages(20, 16)
    a = p.new()
    assert p.extend({a: 20}) == []
    forks = [a] + [p.fork(a) for _ in range(4)]
    last = p.pages(a)[1]
    pairs = p.extend({f: 1 for f in forks})
    assert len(pairs) == 4 and {x for x, _ in pairs} == {last}
    assert len({p.pages(f)[1] for f in forks}) == 5 and len({p.pages(f)[0] for f in forks}) == 1
    b = p.fork(a)
    p.truncate(b, 16)               # a full page is shared without a copy
    assert p.extend({b: 3}) == []


def test_out_of_pages_changes_nothing():
    p = KV4Pages(3, 16)
    a = p.new()
    p.extend({a: 40})
    b = p.fork(a)
    for tokens in ({a: 9}, {b: 1}, {a: 1, b: 1}):
        with pytest.raises(OutOfPages):
            p.extend(tokens)
        assert p.length(a) == 40 and p.pages(a) == p.pages(b) and p.free_pages == 0
    p.free(b)
    assert p.extend({a: 8}) == []
    with pytest.raises(OutOfPages):
        p.extend({a: 1})


def test_refusals():
    for n, size in ((0, 16), (4, 8), (4, 24), (4, 2048)):
        with pytest.raises(ValueError):
            KV4Pages(n, size)
    p = KV4Pages(4, 16)
    a = p.new()
    p.extend({a: 17})
    with pytest.raises(ValueError):
        p.extend({a: -1})
    with pytest.raises(ValueError):
        p.truncate(a, 18)
    with pytest.raises(ValueError):
        p.tables([a], "cpu", max_pages=1)
    p.free(a)
    with pytest.raises(KeyError):
        p.extend({a: 1})


def test_tables_and_pairs():
    p = KV4Pages(9, 16)
    a, b, c = p.new(), p.new(), p.new()
    p.extend({a: 33, b: 5})
    table, lens = p.tables([b, c, a], "cpu")
    assert table.dtype == lens.dtype == torch.int32 and table.tolist() == [[3, 0, 0], [0, 0, 0], [0, 1, 2]]
    assert lens.tolist() == [5, 0, 33]
    assert p.tables([c], "cpu")[0].shape == (1, 1) and p.tables([b], "cpu", max_pages=6)[0].shape == (1, 6)
    src, dst = page_pairs([(1, 2), (5, 6)], "cpu")
    assert src.tolist() == [1, 5] and dst.tolist() == [2, 6] and src.dtype == torch.int32 and src.is_contiguous()
    assert page_pairs([], "cpu")[0].numel() == 0
