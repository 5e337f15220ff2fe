"""The host's bookkeeping of a 4-bit cache's pages: which page holds which
tokens of which sequence, pages shared between forks, and the copies that keep
them apart. Plain Python, no GPU: the calls that move data are kv4_append and
kv4_copy_pages.

    pages = KV4Pages(num_pages, page_size)
    a = pages.new()
    pairs = pages.extend({a: 700})          # 700 tokens to come; copies to make first
    b = pages.fork(a)                       # shares all of a's pages
    pairs = pages.extend({a: 1, b: 1})      # the half full last page is now copied for one of them
    if pairs: kv4_copy_pages(pool, *page_pairs(pairs, pool.device))
    table, lens = pages.tables([a, b], pool.device)
    kv4_append(k, v, pool, table, lens)

All copies of a call may run in any order (no page is written that another pair
reads or writes). Pages that free() or truncate() gives back may be handed out
again at once: the order of the calls on one stream keeps that right.
"""
from __future__ import annotations


class OutOfPages(RuntimeError):
    """The pool has too few free pages for the call, which changed nothing."""


class KV4Pages:
    def __init__(self, num_pages: int, page_size: int):
        if num_pages <= 0 or page_size < 16 or page_size > 1024 or page_size & (page_size - 1):
            raise ValueError("num_pages must be positive and page_size a power of two from 16 to 1024")
        self.num_pages, self.page_size = num_pages, page_size
        self._free = list(range(num_pages - 1, -1, -1))  # taken from the end: low pages first
        self._users = [0] * num_pages                    # sequences that a page belongs to
        self._seqs: dict[int, list[int]] = {}            # pages of each sequence
        self._lens: dict[int, int] = {}
        self._next = 0

    def __len__(self) -> int:
        """Sequences that there are."""
        return len(self._seqs)

    @property
    def free_pages(self) -> int:
        return len(self._free)

    def length(self, seq: int) -> int:
        """Tokens of a sequence."""
        return self._lens[seq]

    def pages(self, seq: int) -> list[int]:
        """Pages of a sequence, in the order of its tokens."""
        return list(self._seqs[seq])

    def _add(self, pages: list[int], tokens: int) -> int:
        seq, self._next = self._next, self._next + 1
        self._seqs[seq], self._lens[seq] = pages, tokens
        return seq

    def new(self) -> int:
        """A sequence without tokens. Returns its id (ids are not used again)."""
        return self._add([], 0)

    def fork(self, seq: int) -> int:
        """A sequence with the same tokens, in the same pages. Returns its id."""
        for page in self._seqs[seq]:
            self._users[page] += 1
        return self._add(list(self._seqs[seq]), self._lens[seq])

    def extend(self, tokens: dict[int, int]) -> list[tuple[int, int]]:
        """Room for tokens[seq] more tokens of every sequence named. Returns the
        page copies (src, dst) to make before they are appended: a last page
        that is not full and that another sequence has too."""
        need, sharers = 0, {}
        for seq, n in tokens.items():
            if n < 0:
                raise ValueError("tokens to add must not be negative")
            held, len_ = self._seqs[seq], self._lens[seq]
            need += -(-(len_ + n) // self.page_size) - len(held)
            if n and len_ % self.page_size:
                last = held[-1]
                left = sharers.get(last, self._users[last])
                need += left > 1
                sharers[last] = left - 1
        if need > len(self._free):
            raise OutOfPages(f"{need} pages are needed and {len(self._free)} are free")
        pairs = []
        for seq, n in tokens.items():
            held = self._seqs[seq]
            if n and self._lens[seq] % self.page_size and self._users[held[-1]] > 1:
                page = self._take()
                pairs.append((held[-1], page))
                self._users[held[-1]] -= 1
                held[-1] = page
            self._lens[seq] += n
            while len(held) * self.page_size < self._lens[seq]:
                held.append(self._take())
        return pairs

    def truncate(self, seq: int, tokens: int) -> None:
        """Keeps the first `tokens` tokens of a sequence (drafted ones turned down, say)."""
        if not 0 <= tokens <= self._lens[seq]:
            raise ValueError(f"sequence {seq} has {self._lens[seq]} tokens")
        held = self._seqs[seq]
        while len(held) > -(-tokens // self.page_size):
            self._give(held.pop())
        self._lens[seq] = tokens

    def free(self, seq: int) -> None:
        """Ends a sequence."""
        self.truncate(seq, 0)
        del self._seqs[seq], self._lens[seq]

    def compact(self) -> list[tuple[int, int]]:
        """Moves the pages in use to the front of the pool (a pool can then be cut
        short or copied out whole). Returns the copies (src, dst) to make."""
        used = self.num_pages - len(self._free)
        src = [p for p in range(used, self.num_pages) if self._users[p]]
        dst = [p for p in range(used) if not self._users[p]]
        to = dict(zip(src, dst))
        for a, b in to.items():
            self._users[b], self._users[a] = self._users[a], 0
        for held in self._seqs.values():
            held[:] = [to.get(p, p) for p in held]
        self._free = list(range(self.num_pages - 1, used - 1, -1))
        return list(to.items())

    def tables(self, seqs: list[int], device="cuda", max_pages: int | None = None):
        """(page_table, seq_lens) of these sequences as the kernels take them:
        int32 [len(seqs), max_pages] (as many as the longest has when not given,
        one at least) and int32 [len(seqs)]. Copied from pinned memory, without
        waiting."""
        import torch
        most = max([1] + [len(self._seqs[s]) for s in seqs])
        if max_pages is None:
            max_pages = most
        elif max_pages < most:
            raise ValueError(f"a sequence has {most} pages, more than max_pages = {max_pages}")
        rows = [self._seqs[s] + [0] * (max_pages - len(self._seqs[s])) for s in seqs]
        table = torch.tensor(rows, dtype=torch.int32).reshape(len(seqs), max_pages)
        lens = torch.tensor([self._lens[s] for s in seqs], dtype=torch.int32)
        return _to_device(table, device), _to_device(lens, device)

    def _take(self) -> int:
        page = self._free.pop()
        self._users[page] = 1
        return page

    def _give(self, page: int) -> None:
        self._users[page] -= 1
        if self._users[page] == 0:
            self._free.append(page)


def _to_device(t, device):
    import torch
    if torch.device(device).type != "cuda":
        return t.to(device)
    return t.pin_memory().to(device, non_blocking=True)


def page_pairs(pairs, device="cuda"):
    """(src, dst) int32 vectors for kv4_copy_pages of the pairs that extend() or compact() returned."""
    import torch
    t = torch.tensor(list(pairs), dtype=torch.int32).reshape(-1, 2).T.contiguous()
    t = _to_device(t, device)
    return t[0], t[1]
