"""A paged key/value cache with its own page list: serving steps over the paged operators.

Host side only: which pages a sequence holds, how many keys are cached, which
position comes next.  The tensors live on the device and every step of the
computation is one of the library's entry points:

    cache = PagedCache(num_pages=4096, H_kv=8, D=128, freq=mea_rope_frequencies(128))
    a, b = cache.add(), cache.add()
    o, lse = cache.step(q, k, v, [a, b], [512, 1])     # 512 new tokens of a, one of b
    cache.evict([a], n_keep=2048, n_recent=256)        # keep the heaviest and the last
    cache.remove(a)

``step`` rotates q and k, appends k and v, attends, and adds up the attention
that every cached key received; ``evict`` cuts sequences in place by those sums
and returns the pages.  Positions keep counting after an eviction: the rotation
of a kept key stays that of its own position.

The compute steps come from an ``ops`` object so that the page list can be
exercised without a GPU; the default is the CUDA library.
"""

from __future__ import annotations

import math

import torch


class CudaOps:
    """The library's entry points as the compute steps of a cache."""

    def __init__(self):
        import exact_memory_efficient_b200 as m
        self.m = m

    def append(self, q, k, v, cache, cu, kv_len, table, positions):
        return self.m.paged_append(q, k, v, cache.k, cache.v, cache.weights, cu, kv_len, table, positions, cache.freq,
                                   cache.interleaved, cache.mscale)

    def attend(self, q, cache, cu, kv_len, table, max_q, max_kv, scale):
        return self.m.attention_paged(q, cache.k, cache.v, cu, kv_len, table, max_q, max_kv, scale)

    def weigh(self, q, lse, cache, cu, kv_len, table, max_q, max_kv, scale):
        self.m.attention_paged_weights(q, lse, cache.k, cache.weights, cu, kv_len, table, max_q, max_kv, scale)

    def evict(self, cache, table, kv_len, n_keep, n_recent):
        return self.m.paged_evict(cache.k, cache.v, cache.weights, table, kv_len, table, n_keep, n_recent)[0]


class PagedCache:
    """Pages of keys, values and (``bounded``) accumulated weights, shared by any number of sequences."""

    def __init__(self, num_pages: int, H_kv: int, D: int, page_size: int = 64, dtype=torch.bfloat16, device="cuda",
                 freq=None, interleaved: bool = False, mscale: float = 1.0, bounded: bool = True, ops=None):
        self.k = torch.zeros(num_pages, H_kv, page_size, D, dtype=dtype, device=device)
        self.v = torch.zeros_like(self.k)
        self.weights = torch.zeros(num_pages, H_kv, page_size, device=device) if bounded else None
        self.freq = None if freq is None else freq.to(device)
        self.interleaved, self.mscale = interleaved, mscale
        self.page_size = page_size
        self.ops = ops if ops is not None else CudaOps()
        self._free = list(range(num_pages - 1, -1, -1))
        self._pages, self._len, self._pos = {}, {}, {}
        self._next = 0

    # ------------------------------------------------------------- page list

    @property
    def free_pages(self) -> int:
        return len(self._free)

    def length(self, seq: int) -> int:
        """Cached keys of a sequence."""
        return self._len[seq]

    def pages(self, seq: int) -> list:
        return list(self._pages[seq])

    def add(self) -> int:
        """A new, empty sequence."""
        seq, self._next = self._next, self._next + 1
        self._pages[seq], self._len[seq], self._pos[seq] = [], 0, 0
        return seq

    def remove(self, seq: int) -> None:
        """Forget a sequence and return its pages."""
        self._free.extend(reversed(self._pages.pop(seq)))
        del self._len[seq], self._pos[seq]

    def _check(self, seqs) -> list:
        seqs = [int(s) for s in seqs]
        if len(set(seqs)) != len(seqs):
            raise ValueError("a sequence is named twice")
        for s in seqs:
            if s not in self._pages:
                raise KeyError(f"no sequence {s}")
        return seqs

    def _upload(self, *rows):
        """The int32 lists as device tensors, in one copy."""
        flat = torch.tensor([x for r in rows for x in r], dtype=torch.int32)
        if self.k.is_cuda:
            flat = flat.pin_memory().to(self.k.device, non_blocking=True)
        out, at = [], 0
        for r in rows:
            out.append(flat[at:at + len(r)])
            at += len(r)
        return out

    def _table(self, seqs):
        width = max([1] + [len(self._pages[s]) for s in seqs])
        return width, [p for s in seqs for p in self._pages[s] + [-1] * (width - len(self._pages[s]))]

    # ------------------------------------------------------------------ steps

    def step(self, q, k, v, seqs, counts, scale: float | None = None):
        """Append ``counts[i]`` new tokens to sequence ``seqs[i]`` and attend: q [T, H, D], k and v
        [T, H_kv, D] packed in that order (any token stride).  Returns o [T, H, D] and lse [T, H]."""
        seqs, counts = self._check(seqs), [int(c) for c in counts]
        if len(counts) != len(seqs) or any(c < 0 for c in counts):
            raise ValueError("one count of new tokens, not negative, for every sequence")
        if q.shape[0] != sum(counts) or k.shape[0] != sum(counts) or v.shape[0] != sum(counts):
            raise ValueError("q, k and v must hold the new tokens of all sequences")
        need = {s: max(0, -(-(self._len[s] + c) // self.page_size) - len(self._pages[s])) for s, c in zip(seqs, counts)}
        if sum(need.values()) > len(self._free):
            raise MemoryError(f"{sum(need.values())} pages needed, {len(self._free)} free")
        before = [(s, len(self._pages[s]), self._len[s], self._pos[s]) for s in seqs]
        try:
            return self._step(q, k, v, seqs, counts, need, scale)
        except BaseException:   # a refused or interrupted call leaves the page list as it was
            for s, held, length, pos in before:
                self._free.extend(reversed(self._pages[s][held:]))
                del self._pages[s][held:]
                self._len[s], self._pos[s] = length, pos
            raise

    def _step(self, q, k, v, seqs, counts, need, scale):
        cu, positions = [0], []
        for s, c in zip(seqs, counts):
            self._pages[s] += [self._free.pop() for _ in range(need[s])]
            positions += range(self._pos[s], self._pos[s] + c)
            self._len[s] += c
            self._pos[s] += c
            cu.append(cu[-1] + c)
        lens = [self._len[s] for s in seqs]
        width, table = self._table(seqs)
        cu, lens_d, table, positions = self._upload(cu, lens, table, positions)
        table = table.view(len(seqs), width)
        q = self.ops.append(q, k, v, self, cu, lens_d, table, positions)
        max_q, max_kv = max([0] + counts), max([0] + lens)
        if scale is None:
            scale = 1.0 / math.sqrt(q.shape[-1])
        o, lse = self.ops.attend(q, self, cu, lens_d, table, max_q, max_kv, scale)
        if self.weights is not None:
            self.ops.weigh(q, lse, self, cu, lens_d, table, max_q, max_kv, scale)
        return o, lse

    def evict(self, seqs, n_keep: int, n_recent: int):
        """Cut every named sequence to at most ``n_keep`` keys, its last ``n_recent`` among them, and
        return the pages behind.  Returns the kept slots, [len(seqs), H_kv, n_keep], -1 behind them."""
        seqs = self._check(seqs)
        if self.weights is None:
            raise ValueError("the cache keeps no weights")
        if n_keep < 1 or not 0 <= n_recent <= n_keep:
            raise ValueError("0 <= n_recent <= n_keep, 1 <= n_keep")
        width, table = self._table(seqs)
        table, lens = self._upload(table, [self._len[s] for s in seqs])
        kept = self.ops.evict(self, table.view(len(seqs), width), lens, n_keep, n_recent)
        for s in seqs:
            self._len[s] = min(self._len[s], n_keep)
            held = -(-self._len[s] // self.page_size)
            self._free.extend(reversed(self._pages[s][held:]))
            del self._pages[s][held:]
        return kept
