"""The attention half of a decoder served with W4 linears: per block the q, k, v
and o projections (spear_linear_decode / spear_linear_prefill), a paged
key/value cache, and the attention that reads it.

`PagedServer` keeps what a serving process keeps: the blocks' weights, one
cache per block, one page pool for all of them, and workspaces.  A step takes
any mix of sequences and new tokens (one token each: the decode kernels; more:
the prefill kernels), and sequences can be forked, finished and the pool
compacted between steps.  Everything runs in stream order on the GPU; no call
reads an answer back.  A call that the pool would refuse is refused on the host
before anything is launched (PoolFull where pages are short): the server counts
along.  Where the pool's bookkeeping was changed other than by its methods (a
saved state put back, say), recount() has to follow.

Norms, rotary embeddings and the feed-forward half are not part of it: a block
maps its input rows to the o projection's output rows.
"""
from __future__ import annotations

import contextlib
from dataclasses import dataclass
from typing import List, Optional, Sequence

import torch

from . import spear


@dataclass
class AttentionBlock:
    """One block's linears: q [width -> q_heads head_dim], k and v [width -> kv_heads head_dim], o back to width."""
    q: spear.W4Layer
    k: spear.W4Layer
    v: spear.W4Layer
    o: spear.W4Layer
    head_dim: int
    window: int = 0          # keys a token sees, itself among them (0: all)
    sinks: int = 0           # first keys of a sequence that stay visible

    @property
    def q_heads(self) -> int:
        return self.q.N // self.head_dim

    @property
    def kv_heads(self) -> int:
        return self.k.N // self.head_dim


class PoolFull(RuntimeError):
    """A step or fork needs more pages than are free.  Nothing was launched: it can be tried again after finish()."""


class PageCount:
    """The lengths and the number of free pages of a page pool, counted on the host: what spear_kv_reserve,
    spear_kv_fork and spear_kv_free will find on the device, and the calls that they would refuse.

    A row's pages are a list of runs [pages, rows that share them]; a run with more than one row is of whole pages."""

    def __init__(self, num_pages: int, page_size: int, max_seqs: int, max_pages: int):
        self.page_size, self.max_pages, self.num_pages, self.free_pages = page_size, max_pages, num_pages, num_pages
        self.lens = [0] * max_seqs
        self.runs: List[list] = [[] for _ in range(max_seqs)]

    def recount(self, lens: Sequence[int], table: Sequence[Sequence[int]]) -> None:
        """Takes over a pool's lengths and block table."""
        runs = {}                                            # by page: a run of its own
        self.lens, self.runs = list(lens), []
        for n, row in zip(lens, table):
            self.runs.append([runs.setdefault(p, [1, 0]) for p in row[:-(-n // self.page_size)]])
            for run in self.runs[-1]:
                run[1] += 1
        self.free_pages = self.num_pages - len(runs)

    def _check_rows(self, rows: Sequence[int], once: bool) -> None:
        if any(not 0 <= r < len(self.lens) for r in rows):
            raise ValueError(f"rows must be in [0, {len(self.lens)}), got {list(rows)}")
        if once and len(set(rows)) != len(rows):
            raise ValueError(f"a row is listed twice: {list(rows)}")

    def _take(self, pages: int) -> None:
        if pages > self.free_pages:
            raise PoolFull(f"{pages} pages needed, {self.free_pages} free")
        self.free_pages -= pages

    def reserve(self, rows: Sequence[int], counts: Sequence[int]) -> None:
        self._check_rows(rows, True)
        if len(counts) != len(rows) or any(n < 0 for n in counts):
            raise ValueError(f"counts must be one number >= 0 for each of {len(rows)} rows, got {list(counts)}")
        need = []
        for r, n in zip(rows, counts):
            want = self.lens[r] + n
            if want > min(self.max_pages * self.page_size, 0x7fffffff - self.page_size):
                raise ValueError(f"row {r} would hold {want} tokens, a row has {self.max_pages} pages of {self.page_size}")
            need.append(-(-want // self.page_size) - -(-self.lens[r] // self.page_size))
        self._take(sum(need))
        for r, n, pages in zip(rows, counts, need):
            runs = self.runs[r]
            if pages and runs and runs[-1][1] == 1:
                runs[-1][0] += pages
            elif pages:
                runs.append([pages, 1])
            self.lens[r] += n

    def fork(self, parents: Sequence[int], children: Sequence[int]) -> None:
        self._check_rows(children, True)
        self._check_rows(parents, False)
        if len(parents) != len(children):
            raise ValueError(f"{len(parents)} parents, {len(children)} children")
        if any(self.lens[c] for c in children) or set(parents) & set(children):
            raise ValueError(f"children must be empty rows and no parents, got {list(children)}")
        self._take(sum(self.lens[p] % self.page_size > 0 for p in parents))
        for p, c in zip(parents, children):
            part = self.lens[p] % self.page_size > 0         # the last page, which no other row holds
            runs = self.runs[p]
            if part and runs[-1][0] > 1:
                runs[-1][0] -= 1
                runs.append([1, 1])
            shared = runs[:-1] if part else runs
            for run in shared:
                run[1] += 1
            self.runs[c] = list(shared) + ([[1, 1]] if part else [])
            self.lens[c] = self.lens[p]

    def free(self, rows: Sequence[int]) -> None:
        self._check_rows(rows, False)
        for r in rows:
            for run in self.runs[r]:
                run[1] -= 1
                if not run[1]:
                    self.free_pages += run[0]
            self.runs[r], self.lens[r] = [], 0


class PagedServer:
    """Blocks, their caches and the sequences in flight (rows 0 .. max_seqs - 1 of the page pool).

    With a `stream` the server's work runs there and its buffers belong to it.  Each call first waits (on the GPU) for
    the work of the caller's current stream, which in turn waits for the call's before it goes on, so inputs and
    results are used on the caller's stream as with any other call."""

    def __init__(self, blocks: Sequence[AttentionBlock], num_pages: int, page_size: int, max_seqs: int, max_pages: int,
                 device, stream: Optional[torch.cuda.Stream] = None):
        self.blocks: List[AttentionBlock] = list(blocks)
        for i, b in enumerate(self.blocks):
            if b.q.N % b.head_dim or b.k.N % b.head_dim or b.v.N != b.k.N or b.o.K != b.q.N or b.q_heads % b.kv_heads \
                    or not b.q.K == b.k.K == b.v.K == self.blocks[0].q.K:
                sizes = {n: (l.K, l.N) for n, l in (("q", b.q), ("k", b.k), ("v", b.v), ("o", b.o))}
                raise ValueError(f"block {i}: heads of {b.head_dim} do not go with linears of (in, out) {sizes}")
        self.device, self.stream = torch.device(device), stream
        with self._on_stream():
            self.caches = [spear.new_kv_cache(num_pages, page_size, b.kv_heads, b.head_dim, device) for b in self.blocks]
            self.pool = spear.PagePool(num_pages, page_size, max_seqs, max_pages, device)
        self.count = PageCount(num_pages, page_size, max_seqs, max_pages)

    @contextlib.contextmanager
    def _on_stream(self):
        """The server's stream as the current one, after the caller's work so far and before what it does next."""
        if self.stream is None:
            yield
            return
        here = torch.cuda.current_stream(self.device)
        self.stream.wait_stream(here)
        try:
            with torch.cuda.stream(self.stream):
                yield
        finally:
            here.wait_stream(self.stream)

    def _rows(self, *lists: Sequence[int]) -> List[torch.Tensor]:
        """The lists as int32 tensors on the device: one copy from pinned memory, which nothing waits for."""
        flat = torch.tensor([i for x in lists for i in x], dtype=torch.int32).pin_memory()
        return list(flat.to(self.device, non_blocking=True).split([len(x) for x in lists]))

    def _linear(self, layer: spear.W4Layer, x: torch.Tensor) -> torch.Tensor:
        call = spear.spear_linear_decode if x.shape[0] <= 64 else spear.spear_linear_prefill
        return call(layer, x)

    def step(self, x: torch.Tensor, rows: Sequence[int], counts: Sequence[int]) -> List[torch.Tensor]:
        """Runs x (bf16 [sum(counts)][width]: counts[i] new tokens of sequence rows[i], in order) through every block on
        its own input rows, and returns each block's output rows.  (A full decoder would feed each block's output,
        through its norm and feed-forward half, to the next one.)"""
        starts = [0]
        for n in counts:
            starts.append(starts[-1] + n)
        if starts[-1] != x.shape[0]:
            raise ValueError(f"x has {x.shape[0]} rows, counts add up to {starts[-1]}")
        width = self.blocks[0].q.K if self.blocks else None
        if x.dtype != torch.bfloat16 or x.dim() != 2 or width not in (None, x.shape[1]) or not x.is_contiguous() \
                or x.get_device() != self.pool.index:
            raise ValueError(f"x must be a contiguous bfloat16 [tokens][{width}] tensor on {self.pool.device}, "
                             f"got {x.dtype} {tuple(x.shape)} on {x.device}")
        self.count.reserve(rows, counts)                     # (the last check: from here on the tokens count)
        here = torch.cuda.current_stream(self.device)
        with self._on_stream():
            outs = self._step(x, rows, counts, starts)
        if self.stream is not None:                          # used on both streams: not reused before either is done
            x.record_stream(self.stream)
            for y in outs:
                y.record_stream(here)
        return outs

    def _step(self, x: torch.Tensor, rows: Sequence[int], counts: Sequence[int], starts: List[int]) -> List[torch.Tensor]:
        ids, new, dev_starts = self._rows(rows, counts, starts)
        table, lens = self.pool.block_table, self.pool.seq_lens
        one_each = all(n == 1 for n in counts)
        spear.spear_kv_reserve(self.pool, ids, new)
        outs = []
        for b, cache in zip(self.blocks, self.caches):
            T, D = x.shape[0], b.head_dim
            q = self._linear(b.q, x).view(T, b.q_heads, D)
            k = self._linear(b.k, x).view(T, b.kv_heads, D)
            v = self._linear(b.v, x).view(T, b.kv_heads, D)
            spear.spear_kv_append(cache, k, v, table, lens, dev_starts, seq_ids=ids, pool=self.pool)
            kw = dict(seq_ids=ids, window=b.window, sinks=b.sinks)
            if one_each:
                a = spear.spear_attn_decode(q, cache, table, lens, **kw)
            else:
                a = spear.spear_attn_prefill(q, cache, table, lens, dev_starts, **kw)
            outs.append(self._linear(b.o, a.view(T, b.q_heads * D)))
        return outs

    def fork(self, parents: Sequence[int], children: Sequence[int]) -> None:
        """Each empty row children[i] continues from a copy of parents[i]."""
        self.count.fork(parents, children)
        with self._on_stream():
            spear.spear_kv_fork(self.pool, self.caches, *self._rows(parents, children))

    def finish(self, rows: Sequence[int]) -> None:
        """Empties the rows (those that are empty already stay so)."""
        self.count.free(rows)
        with self._on_stream():
            spear.spear_kv_free(self.pool, *self._rows(rows))

    def recount(self) -> None:
        """Counts the pool's pages anew, after a change to it that was not made by these methods.  Waits for the GPU."""
        with self._on_stream():
            self.count.recount(self.pool.seq_lens.tolist(), self.pool.block_table.tolist())

    def compact(self) -> None:
        """Moves the live pages to the front of the pool."""
        with self._on_stream():
            spear.spear_kv_compact(self.pool, self.caches)


__all__ = ["AttentionBlock", "PageCount", "PagedServer", "PoolFull"]
