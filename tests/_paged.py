"""Plain 64-bit forms of the paged cache's operators, for its tests.

``Model`` holds every sequence as a list of token values and the page map as
Python lists, by the rules of include/fc_paged.h; nothing here is shared with
the library.
"""

from __future__ import annotations

import numpy as np
import torch

EPS = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step


def quantise(x: torch.Tensor):
    """int8 codes and fp32 scales of rows (..., D), decided in 64 bits."""
    x = x.double()
    top = x.abs().amax(-1)
    safe = torch.where(top > 0, top, torch.ones_like(top))
    codes = torch.round(x * 127.0 / safe[..., None]).to(torch.int8)
    return codes, (top / 127.0).float()


def held(x: torch.Tensor, kv: str) -> torch.Tensor:
    """What the cache holds for token rows x, in 64 bits."""
    if kv != "i8":
        return x.double()
    codes, scale = quantise(x)
    return codes.double() * scale.double()[..., None]


def seen(n: int, window: int, sinks: int):
    """Positions a query at the end of n tokens sees."""
    return [t for t in range(n)
            if window == 0 or t >= n - window or t < sinks]


def attend(q, k, v, G, scale, window=0, sinks=0):
    """q (Hq, D), k and v (n, Hk, D), all float64 numpy: (out, lse, bounds):
    ``bounds`` is sum_t p_t |v_t| / l per output and the largest
    sigma sum_d |q_d k_td| and |s_t| per head, for error bounds."""
    Hq, D = q.shape
    keep = seen(k.shape[0], window, sinks)
    out = np.zeros((Hq, D))
    lse = np.full(Hq, -np.inf)
    mag, dots = np.zeros((Hq, D)), np.zeros(Hq)
    if keep:
        for h in range(Hq):
            kk, vv = k[keep, h // G], v[keep, h // G]
            s = scale * (kk @ q[h])
            m = s.max()
            p = np.exp(s - m)
            out[h] = p @ vv / p.sum()
            mag[h] = p @ np.abs(vv) / p.sum()
            lse[h] = m + np.log(p.sum())
            dots[h] = (scale * (np.abs(kk) @ np.abs(q[h]))).max()
    return out, lse, mag, dots


def attend_bound(mag, dots, ref, n, D, out_dtype):
    """How far an output may lie from the exact one.

    Assumed of one tensor-core product: its fp32 sum is off by at most 2^-22 of
    the sum of the magnitudes it adds. Scores: at most 6 products per 16
    channels (three limbs each way), so |ds| <= (6 D/16 + 4) 2^-22 sum |q k|
    sigma, the four for the scalings and roundings of s. The exponential adds
    2^-21 relative and the rounding of its argument, |s| 2^-22 <= dots 2^-22.
    Sums over tokens: at most 6 products per 16 tokens and the joins, each
    2^-22 of sum p |v|. The limbs of p keep 2^-16 (two, bf16 outputs) or
    2^-23 (three). l has the exponentials' error and n 2^-24."""
    ds = (6 * D / 16 + 5) * 2.0 ** -22 * dots[:, None] + 2.0 ** -21
    limbs = 2.0 ** -16 if out_dtype == torch.bfloat16 else 2.0 ** -23
    sums = (6 * n / 16 + 64) * 2.0 ** -22
    rel = 2 * ds + limbs + sums + n * 2.0 ** -24
    return rel * mag + EPS[out_dtype] * np.abs(ref) + 1e-30


class Model:
    """The page map's rules: lowest free page first, reference counts, copy
    before a write to a shared page, compaction into the holes."""

    def __init__(self, n_slots, n_pages, page, max_pages):
        self.page, self.n_pages, self.max_pages = page, n_pages, max_pages
        self.rows = [[] for _ in range(n_slots)]
        self.lens = [0] * n_slots

    def refs(self):
        r = [0] * self.n_pages
        for row in self.rows:
            for p in row:
                r[p] += 1
        return r

    def _take(self):
        r = self.refs()
        return r.index(0) if 0 in r else None

    def begin(self, slots, counts):
        """True and the (old, new) page copies, or False (nothing changed)."""
        rows, lens = [list(r) for r in self.rows], list(self.lens)
        copies = []
        for s, c in zip(slots, counts):
            if c and self.lens[s] % self.page:
                old = self.rows[s][-1]
                if self.refs()[old] > 1:
                    new = self._take()
                    if new is None:
                        self.rows, self.lens = rows, lens
                        return False, []
                    self.rows[s][-1] = new
                    copies.append((old, new))
            self.lens[s] += c
            while len(self.rows[s]) * self.page < self.lens[s]:
                new = self._take()
                if new is None or len(self.rows[s]) == self.max_pages:
                    self.rows, self.lens = rows, lens
                    return False, []
                self.rows[s].append(new)
        return True, copies

    def fork(self, src, dst):
        for a, b in zip(src, dst):
            self.rows[b], self.lens[b] = list(self.rows[a]), self.lens[a]

    def crop(self, slot, keep):
        self.lens[slot] = keep
        del self.rows[slot][-(-keep // self.page):]

    def compact(self):
        r = self.refs()
        live = [p for p in range(self.n_pages) if r[p]]
        holes = [p for p in range(len(live)) if not r[p]]
        to = dict(zip([p for p in live if p >= len(live)], holes))
        self.rows = [[to.get(p, p) for p in row] for row in self.rows]
        return len(live)

    def table(self):
        t = np.full((len(self.rows), self.max_pages), -1, np.int32)
        for i, row in enumerate(self.rows):
            t[i, :len(row)] = row
        return t
