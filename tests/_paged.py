"""Ragged batches over a paged cache for the tests, and the bounds that they enforce.

Bounds, from the arithmetic (u = 2^-24, half a step of fp32; half a step of bf16
is 2^-8 relative with 8 bits of significand: torch.finfo(bf16).eps / 2):
* rope: y = m (a c - b s).  The angle is exact to 2^-50 turns before it is
  rounded to fp32 half turns in [-1, 1]: an error of at most 2^-25 half turns =
  pi u / 2 < 1.6 u radians.  sincospif is off by at most 2 steps = 4 u of a value
  at most 1, the product with m by u, a c and b s by u each, their difference by
  u of the result: at most (1.6 + 4 + 1 + 1 + 1) u < 9 u times m (|a| + |b|);
  then half a step of the result's type.
* attention: the library's stated bounds (tests/_parity.py) and its derived lse
  bound.
* weights: a probability exp(x), x = scale q.k - lse, has the relative error
  exp(dx) - 1, dx = scale gamma_D sum |q k| (fp32 products and sums of D terms)
  + 3 u (|scale q.k| + |lse|) (the two products with log2 e and their
  difference), plus 2^-21 for the approximate exp2; summing n terms adds n u of
  the sum, adding it to the old weight u of the result.
"""

from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24


class Batch:
    """Inputs on the CPU (torch), from a seed: `counts` new tokens and `lens` cached keys per sequence."""

    def __init__(self, counts, lens, H, Hkv, D, page, dtype, seed=0, spare=3, garbage=None, rows=None, front=0,
                 behind=0, max_pages=None, mult=1.0):
        g = torch.Generator().manual_seed(seed)
        self.counts, self.lens, self.H, self.Hkv, self.D, self.page = list(counts), list(lens), H, Hkv, D, page
        self.dtype, B = dtype, len(lens)
        per = [-(-x // page) for x in self.lens]
        self.max_pages = max_pages or max([1] + per)
        self.pages = sum(per) + spare
        order = torch.randperm(self.pages, generator=g).to(torch.int32)
        self.table = torch.full((B, self.max_pages), -1, dtype=torch.int32)
        at = 0
        for b, m in enumerate(per):
            self.table[b, :m] = order[at:at + m]
            at += m
        self.free = order[at:]
        self.cu = torch.tensor([front] + self.counts, dtype=torch.int32).cumsum(0).to(torch.int32)
        self.T = int(self.cu[-1]) + behind
        self.kv_len = torch.tensor(self.lens, dtype=torch.int32)
        rnd = lambda *s: torch.randn(*s, generator=g).to(dtype)  # noqa: E731
        self.k_cache, self.v_cache = rnd(self.pages, Hkv, page, D), rnd(self.pages, Hkv, page, D)
        self.q, self.k, self.v = rnd(self.T, H, D), rnd(self.T, Hkv, D), rnd(self.T, Hkv, D)
        if mult != 1.0:
            self.q, self.k_cache = self.q * mult, self.k_cache * mult
        self.weights = torch.rand(self.pages, Hkv, page, generator=g)
        self.scale = 1.0 / np.sqrt(D)
        self.max_q, self.max_kv = max(self.counts + [0]), max(self.lens + [0])
        if garbage is not None:
            used = torch.zeros(self.pages, page, dtype=torch.bool)
            for b, x in enumerate(self.lens):
                j = torch.arange(x)
                used[self.table[b, j // page].long(), j % page] = True
            for t in (self.k_cache, self.v_cache):
                t.permute(0, 2, 1, 3)[~used] = garbage
        self.used_rows = range(int(self.cu[0]), int(self.cu[-1]))

    def gpu(self, *names):
        return [getattr(self, n).cuda() for n in names]

    def np(self, *names):
        return [f64(getattr(self, n)) for n in names]

    def gathered_k(self, b):
        j = torch.arange(self.lens[b])
        return f64(self.k_cache[self.table[b, j // self.page].long(), :, j % self.page])   # [L, Hkv, D]


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy() if t.is_floating_point() else t.detach().cpu().numpy()


def rope_bound(x, freq, interleaved, mscale, dtype, want):
    """Per-value bound of a rotation of x [..., D] whose exact result is `want`."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    half = len(freq)
    tol = np.zeros_like(x)
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else \
        (slice(0, half), slice(half, 2 * half))
    both = 9 * U * abs(mscale) * (x[..., first] + x[..., second])
    tol[..., first], tol[..., second] = both, both
    step = U if dtype == torch.float32 else torch.finfo(dtype).eps / 2
    return tol * (1 + step) + step * np.abs(want)


def weight_bound(bt, q, lse, want):
    """Per-slot bound of the accumulated weights (module docstring); `want` are the exact ones."""
    tol = U * np.abs(want) + 1e-30
    gamma = bt.D * U / (1 - bt.D * U)
    G = bt.H // bt.Hkv
    for b, L in enumerate(bt.lens):
        n, c = bt.counts[b], int(bt.cu[b])
        if n == 0 or L == 0:
            continue
        k = bt.gathered_k(b)
        j = np.arange(L)
        p, f = bt.table.numpy()[b, j // bt.page], j % bt.page
        seen = np.arange(L)[None, :] < (L - n + np.arange(n) + 1)[:, None]
        for h in range(bt.H):
            qq, kk, ll = q[c:c + n, h], k[:, h // G], lse[c:c + n, h][:, None]
            s = bt.scale * qq @ kk.T
            dx = bt.scale * gamma * np.abs(qq) @ np.abs(kk).T + 3 * U * (np.abs(s) + np.abs(ll))
            with np.errstate(invalid="ignore", over="ignore"):
                e = np.where(seen, np.exp(s - ll) * (np.expm1(dx) + 2.0 ** -21 + n * G * U), 0.0)
            tol[p, h // G, f] += e.sum(0)
    return tol
