"""Float64 oracle of the serving operators: rotary positions and the paged 8-bit key/value cache.

TEST INFRASTRUCTURE ONLY (see the package docstring): the product path never imports it.  Plain
loops from the definitions; it shares nothing with the CUDA path.

Definitions
  Rotary  pair (x1, x2) -> A (x1 cos a - x2 sin a, x1 sin a + x2 cos a), a = position * theta_i;
          columns behind the rotated ones pass through; the inverse turns by -a.
  e4m3    sign, 4 exponent bits (bias 7), 3 mantissa bits: +-(1 + m / 8) 2^(x - 7), subnormals m 2^-9,
          largest 448, no infinity; rounding to nearest, ties to the even mantissa.
  Scale   of one page and head: 2^e, e the least with amax <= 448 * 2^e over the finite new elements,
          within [-117, 120], and not below the page's exponent if the page holds older tokens.
  Pages   free: no holder.  reserve takes the lowest free ones in batch order; a shared, partly filled
          last page is copied while more than one holder is left.
"""
from __future__ import annotations

import math
from typing import List, Optional

import numpy as np

from .attention import _as64

E_MIN, E_MAX = -117, 120
TOP = 240.0 * 2.0 ** 120


def rope(x, pos, inv_freq, interleaved: bool, amplitude: float = 1.0, inverse: bool = False) -> np.ndarray:
    """x [B, H, S, Dh], pos [B, S], inv_freq [rot / 2]."""
    x = _as64(x).copy()
    a = np.asarray(pos, dtype=np.float64)[:, None, :, None] * np.asarray(inv_freq, dtype=np.float64)
    c, s = amplitude * np.cos(a), amplitude * np.sin(a) * (-1.0 if inverse else 1.0)
    r = 2 * len(inv_freq)
    i1, i2 = (np.arange(0, r, 2), np.arange(1, r, 2)) if interleaved else (np.arange(r // 2), np.arange(r // 2, r))
    x1, x2 = x[..., i1].copy(), x[..., i2].copy()
    x[..., i1], x[..., i2] = x1 * c - x2 * s, x1 * s + x2 * c
    return x


def e4m3(y) -> np.ndarray:
    """Nearest e4m3 value of each y (|y| <= 448 expected), ties to even; NaN stays."""
    y = np.asarray(y, dtype=np.float64)
    _, x = np.frexp(np.abs(np.where(np.isfinite(y), y, 0.0)))
    step = np.ldexp(1.0, np.maximum(x, -5) - 4)     # 3 bits behind the leading one; subnormals 2^-9
    return np.where(np.isnan(y), np.nan, np.round(y / step) * step)


def scale_exponent(amax: float) -> int:
    if amax <= 0.0:
        return E_MIN
    e = math.ceil(math.log2(amax / 448.0)) - 2
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return min(max(e, E_MIN), E_MAX)


class Cache:
    """One layer's values in float64 and the books of the page table."""

    def __init__(self, pages: int, heads: int, page: int, Dh: int, slots: int, max_pages: int):
        self.page, self.heads, self.Dh = page, heads, Dh
        self.codes = {n: np.zeros((pages, heads, page, Dh)) for n in "kv"}     # e4m3 values
        self.exp = {n: np.full((pages, heads), E_MIN) for n in "kv"}
        self.table = np.full((slots, max_pages), -1)
        self.lens = np.zeros(slots, dtype=np.int64)
        self.refs = np.zeros(pages, dtype=np.int64)

    def _count(self, tokens: int) -> int:
        return -(-int(tokens) // self.page)

    def reserve(self, slots: List[int], n_new: List[int]) -> bool:
        """False (nothing changed) when the free pages do not suffice."""
        free = [p for p in range(len(self.refs)) if self.refs[p] == 0]
        plan, refs = [], self.refs.copy()
        for s, n in zip(slots, n_new):
            if s < 0 or n == 0:
                continue
            have, need = self._count(self.lens[s]), self._count(self.lens[s] + n)
            copy_of = None
            if self.lens[s] % self.page:
                last = self.table[s, have - 1]
                if refs[last] > 1:
                    copy_of = last
                    refs[last] -= 1
            plan.append((s, n, have, need, copy_of))
        if sum(need - have + (c is not None) for _, _, have, need, c in plan) > len(free):
            return False
        self.refs = refs
        for s, n, have, need, copy_of in plan:
            if copy_of is not None:
                p = free.pop(0)
                for x in "kv":
                    self.codes[x][p], self.exp[x][p] = self.codes[x][copy_of], self.exp[x][copy_of]
                self.table[s, have - 1] = p
                self.refs[p] = 1
            for j in range(have, need):
                p = free.pop(0)
                self.table[s, j] = p
                self.refs[p] = 1
            self.lens[s] += n
        return True

    def append(self, slots, n_new, k, v) -> None:
        """k, v [B, heads, T, Dh]; the last n_new[b] positions of slots[b] get rows 0 .. n_new[b] - 1."""
        for b, (s, n) in enumerate(zip(slots, n_new)):
            if s < 0:
                continue
            p0, end = self.lens[s] - n, self.lens[s]
            for j in range(p0 // self.page, self._count(end)) if n else []:
                pid = self.table[s, j]
                a, z = max(p0, j * self.page), min(end, (j + 1) * self.page)
                old = a - j * self.page
                for name, x in (("k", k), ("v", v)):
                    for h in range(self.heads):
                        new = _as64(x[b, h, a - p0:z - p0])
                        fin = np.abs(new[np.isfinite(new)])
                        e = scale_exponent(fin.max() if fin.size else 0.0)
                        if old:
                            e0 = self.exp[name][pid, h]
                            e = max(e, e0)
                            c = self.codes[name][pid, h, :old]
                            self.codes[name][pid, h, :old] = e4m3(c * 2.0 ** float(max(e0 - e, -126)))
                        y = np.where(np.isfinite(new), np.clip(np.nan_to_num(new, nan=0.0), -TOP, TOP), np.nan)
                        self.codes[name][pid, h, old:old + z - a] = e4m3(y * 2.0 ** -float(e))
                        self.exp[name][pid, h] = e

    def values(self, name: str, slot: int) -> np.ndarray:
        """[heads, len, Dh] of one sequence."""
        n = int(self.lens[slot])
        pids = self.table[slot, :self._count(n)]
        x = self.codes[name][pids] * np.ldexp(1.0, self.exp[name][pids])[..., None, None]
        return x.transpose(1, 0, 2, 3).reshape(self.heads, -1, self.Dh)[:, :n]

    def attend(self, slot: int, q, n_new: int, scale: Optional[float] = None, causal: bool = True):
        """q [Hq, n_new, Dh] -> (o, lse, and sum_j p_j |v_j| for error bounds)."""
        q = _as64(q)
        k, v = self.values("k", slot), self.values("v", slot)
        Hq, n, g = q.shape[0], k.shape[1], q.shape[0] // self.heads
        scale = scale or self.Dh ** -0.5
        o, size = np.zeros(q.shape), np.zeros(q.shape)
        lse = np.full(q.shape[:2], -np.inf)
        for h in range(Hq):
            for t in range(n_new):
                m = min(n, n - n_new + t + 1) if causal else n
                if m <= 0:
                    continue
                s = k[h // g, :m] @ q[h, t] * scale
                top = s.max()
                p = np.exp(s - top)
                z = p.sum()
                lse[h, t] = top + np.log(z)
                o[h, t] = p @ v[h // g, :m] / z
                size[h, t] = p @ np.abs(v[h // g, :m]) / z
        return o, lse, size

    def fork(self, src, dst) -> None:
        lens = self.lens.copy()
        for s, d in zip(src, dst):
            if s < 0 or self.lens[d]:
                continue
            n = self._count(lens[s])
            self.table[d, :n] = self.table[s, :n]
            self.lens[d] = lens[s]
            for p in self.table[s, :n]:
                self.refs[p] += 1

    def trim(self, slots, keep) -> None:
        for s, n in zip(slots, keep):
            if s < 0 or n >= self.lens[s]:
                continue
            for j in range(self._count(n), self._count(self.lens[s])):
                self.refs[self.table[s, j]] -= 1
                self.table[s, j] = -1
            self.lens[s] = n

    def compact(self) -> None:
        live = [p for p in range(len(self.refs)) if self.refs[p]]
        holes = [p for p in range(len(live)) if not self.refs[p]]
        movers = [p for p in live if p >= len(live)]
        for a, z in zip(movers, holes):
            for x in "kv":
                self.codes[x][z], self.exp[x][z] = self.codes[x][a], self.exp[x][a]
            self.refs[z], self.refs[a] = self.refs[a], 0
            self.table[self.table == a] = z
