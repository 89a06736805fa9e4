"""A paged key/value cache for answering one token at a time.

:class:`PageTable` is the host side: which pages hold which sequence, what is
free, what is shared.  Sequences are added, extended, forked (the copy shares
its pages; the first write into a shared page gets its own copy of it), freed
and compacted (the pages in use moved to the front of the pool).  It moves no
data itself: what has to be copied comes back as a list of pages.

:class:`PagedCache` joins it with the pages on the device (``nt.KVPages``) and
the library's calls: a step names its sequences and how many tokens each
gains, writes their keys and values (``nt_paged_write``) and attends with one
query token per sequence (``nt_paged_attn``); forks and compaction copy pages
(``nt_paged_copy``).
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Dict, List, Optional, Sequence, Tuple

import torch

from . import nt

Copies = List[Tuple[int, int]]


class OutOfPages(RuntimeError):
    """The pool has not enough free pages; nothing was changed."""


class PageTable:
    """Pages [0, n_pages) of ``page_size`` positions and the sequences in them."""

    def __init__(self, n_pages: int, page_size: int):
        if n_pages < 0 or page_size < 1:
            raise ValueError("n_pages >= 0 and page_size >= 1")
        self.n_pages, self.page_size = n_pages, page_size
        self.refs = [0] * n_pages
        self.free_pages = list(range(n_pages - 1, -1, -1))      # taken from the end: low pages first
        self.pages: Dict[int, List[int]] = {}                   # of each sequence, in order
        self.length: Dict[int, int] = {}
        self._next = 0

    def add(self) -> int:
        """A new, empty sequence's id."""
        seq = self._next
        self._next += 1
        self.pages[seq], self.length[seq] = [], 0
        return seq

    def _known(self, seq: int):
        if seq not in self.pages:
            raise KeyError(f"no sequence {seq}")

    def _drop(self, page: int):
        self.refs[page] -= 1
        if self.refs[page] == 0:
            self.free_pages.append(page)

    def extend(self, seqs: Sequence[int], counts: Sequence[int]) -> Copies:
        """Room for counts[i] more positions in each of ``seqs`` (distinct).
        Returns the (source, destination) pages to copy before they are
        written: the partly filled last pages that other sequences share.
        Raises OutOfPages with nothing changed."""
        if len(seqs) != len(counts) or len(set(seqs)) != len(seqs):
            raise ValueError("one count per sequence, each sequence once")
        # what each needs: new pages, and a page of its own in place of a shared one.  When all sharers of a
        # page extend in one call, the last one left keeps it.
        need, left = 0, {}
        own = []
        for s, n in zip(seqs, counts):
            self._known(s)
            if n < 0:
                raise ValueError("counts must be >= 0")
            have = len(self.pages[s])
            copy = False
            if n > 0 and self.length[s] % self.page_size:
                last = self.pages[s][-1]
                refs = left.setdefault(last, self.refs[last])
                copy = refs > 1
                if copy:
                    left[last] = refs - 1
            own.append(copy)
            need += -(-(self.length[s] + n) // self.page_size) - have + copy
        if need > len(self.free_pages):
            raise OutOfPages(f"{need} pages needed, {len(self.free_pages)} free")
        copies = []
        for s, n, copy in zip(seqs, counts, own):
            pages = self.pages[s]
            if copy:
                dst = self.free_pages.pop()
                copies.append((pages[-1], dst))
                self.refs[dst] = 1
                self.refs[pages[-1]] -= 1                       # stays in use: another sequence holds it
                pages[-1] = dst
            self.length[s] += n
            while len(pages) * self.page_size < self.length[s]:
                page = self.free_pages.pop()
                self.refs[page] = 1
                pages.append(page)
        return copies

    def retract(self, seqs: Sequence[int], counts: Sequence[int], copies: Copies) -> None:
        """Takes back the call of :meth:`extend` before it, which had these
        arguments and returned ``copies``: the table is as it was."""
        copied = {dst: src for src, dst in copies}
        for s, n in zip(reversed(seqs), reversed(counts)):
            pages = self.pages[s]
            self.length[s] -= n
            while len(pages) > -(-self.length[s] // self.page_size):
                self._drop(pages.pop())
            if pages and pages[-1] in copied:
                dst, pages[-1] = pages[-1], copied[pages[-1]]
                self.refs[pages[-1]] += 1
                self._drop(dst)

    def fork(self, seq: int) -> int:
        """A new sequence with the same positions, sharing ``seq``'s pages."""
        self._known(seq)
        new = self.add()
        self.pages[new], self.length[new] = list(self.pages[seq]), self.length[seq]
        for p in self.pages[new]:
            self.refs[p] += 1
        return new

    def free(self, seq: int) -> None:
        """Ends a sequence; pages no other sequence shares become free."""
        self._known(seq)
        for p in self.pages.pop(seq):
            self._drop(p)
        del self.length[seq]

    def compact(self) -> Copies:
        """Moves the pages in use to [0, pages in use): returns the (source,
        destination) pages to copy.  No page is both a source and a
        destination."""
        used = sum(r > 0 for r in self.refs)
        holes = [p for p in range(used) if self.refs[p] == 0]
        moved = [p for p in range(used, self.n_pages) if self.refs[p] > 0]
        to = dict(zip(moved, holes))
        for src, dst in to.items():
            self.refs[dst], self.refs[src] = self.refs[src], 0
        for s, pages in self.pages.items():
            self.pages[s] = [to.get(p, p) for p in pages]
        self.free_pages = list(range(self.n_pages - 1, used - 1, -1))
        return list(to.items())


@dataclass
class Step:
    """One step's sequences as the calls take them: packed offsets of the new
    tokens, the lengths before and after, and the block table."""
    seqs: List[int]
    cu_seqlens: torch.Tensor     # [B + 1] of the new tokens
    pos0: torch.Tensor           # [B] positions before the step
    lengths: torch.Tensor        # [B] positions with the step's
    block_table: torch.Tensor    # [B, max_pages]
    max_new: int                 # longest of the new segments
    tokens: int                  # new tokens of all of them


class PagedCache:
    """Keys and values of many sequences in pages on the device."""

    def __init__(self, n_pages: int, page_size: int, H_kv: int, d: int, dtype: torch.dtype = torch.bfloat16,
                 device="cuda"):
        shape = (n_pages, H_kv, page_size, d)
        self.table = PageTable(n_pages, page_size)
        self.pages = nt.KVPages(torch.empty(shape, dtype=dtype, device=device),
                                torch.empty(shape, dtype=dtype, device=device))

    def add(self) -> int:
        return self.table.add()

    def fork(self, seq: int) -> int:
        return self.table.fork(seq)

    def free(self, seq: int) -> None:
        self.table.free(seq)

    def _copy(self, copies: Copies, stream=None) -> None:
        if copies:
            src, dst = torch.tensor(copies, dtype=torch.int32).T.contiguous()
            nt.nt_paged_copy(self.pages, src, dst, stream=stream)

    def _on(self, stream, what: str):
        """The call's stream, which may not be capturing."""
        on = stream if stream is not None else torch.cuda.current_stream(self.pages.device)
        with torch.cuda.stream(on):
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError(f"{what} on the host: take it outside the capture")
        return on

    def compact(self, stream=None) -> None:
        """The pages in use moved to the front of the pool.  Steps taken
        before hold the old places.  Not while a graph is being captured: the
        table would change now and the pages at a replay."""
        self._on(stream, "compaction moves pages")
        t = self.table
        before = list(t.refs), list(t.free_pages), {s: list(p) for s, p in t.pages.items()}
        try:
            self._copy(t.compact(), stream)
        except BaseException:
            t.refs, t.free_pages, t.pages = before
            raise

    def step(self, seqs: Sequence[int], counts: Sequence[int], stream=None) -> Step:
        """Makes room for counts[i] new tokens of seqs[i] and returns the
        step's device arrays (one copy from pinned memory).  Counts of 1 make
        a decoding step, larger ones a prefill.  Not while a graph is being
        captured: a replay would not make room again."""
        on = self._on(stream, "a step makes room")
        seqs, counts = list(seqs), list(counts)
        copies = self.table.extend(seqs, counts)
        try:
            self._copy(copies, stream)
            return self._arrays(seqs, counts, on)
        except BaseException:
            self.table.retract(seqs, counts, copies)      # no room is made for a step that was not taken
            raise

    def _arrays(self, seqs: List[int], counts: List[int], on) -> Step:
        B = len(seqs)
        lists = [self.table.pages[s] for s in seqs]
        after = [self.table.length[s] for s in seqs]
        width = max([len(p) for p in lists] + [1])
        cu = [0]
        for n in counts:
            cu.append(cu[-1] + n)
        flat = cu + [a - n for a, n in zip(after, counts)] + after
        head = len(flat) + (-len(flat)) % 4
        flat += [0] * (head - len(flat))
        for p in lists:
            flat += p + [-1] * (width - len(p))
        host = torch.tensor(flat, dtype=torch.int32).pin_memory()
        dev = self.pages.device
        with torch.cuda.stream(on):
            arr = host.to(dev, non_blocking=True)
        return Step(seqs, arr[:B + 1], arr[B + 1:2 * B + 1], arr[2 * B + 1:3 * B + 1],
                    arr[head:].view(B, width), max(counts + [0]), cu[-1])

    def write(self, step: Step, k: torch.Tensor, v: torch.Tensor, stream=None) -> None:
        """The step's new keys and values, packed (tokens, H_kv, d): all of
        them, or positions that were never written would be attended to."""
        if k.shape[0] != step.tokens:
            raise ValueError(f"the step has {step.tokens} new tokens, k and v have {k.shape[0]}")
        nt.nt_paged_write(self.pages, k, v, step.cu_seqlens, step.block_table, pos0=step.pos0, stream=stream)

    def attend(self, step: Step, q: torch.Tensor, scale: Optional[float] = None, stream=None) -> torch.Tensor:
        """One query token per sequence, q (B, H, d), over all its positions."""
        return nt.nt_paged_attn(self.pages, q, step.block_table, step.lengths, scale=scale, stream=stream)[0]
