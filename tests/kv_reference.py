"""Plain 64-bit forms of the 4-bit mat-vec with group scales and of the paged
key-value cache, written from their definitions (no code of the library's)."""
from __future__ import annotations

import numpy as np


# --- 4-bit weights with group scales ------------------------------------------
def i4_matrix(rng, out, inf, group, zeros=True, scale=0.006):
    """(packed uint8 [out][in/2], scales float16 [out][groups], zeros uint8 [out][groups] or None)."""
    groups = -(-inf // group)
    packed = rng.integers(0, 256, (out, inf // 2), dtype=np.uint8)
    scales = ((rng.random((out, groups)) + 0.5) * scale).astype(np.float16)
    return packed, scales, (rng.integers(0, 16, (out, groups), dtype=np.uint8) if zeros else None)


def i4_weights(packed, scales, zeros, inf, group):
    codes = np.empty((packed.shape[0], inf))
    codes[:, 0::2], codes[:, 1::2] = packed & 15, packed >> 4
    at = np.arange(inf) // group
    zero = 8.0 if zeros is None else zeros.astype(np.float64)[:, at]
    return (codes - zero) * scales.astype(np.float64)[:, at]


def i4_tolerance(w, x):
    """What the products' sums may be off by: x in two binary16 parts is within 2^-22 of itself (and 2^-50 of its column's
    largest value), a float32 chain of additions adds 2^-24 of the sum of magnitudes a step: at most 32 within a matrix
    instruction, one for each 32 weights, 32 for group scales' folding, wavefronts and bias."""
    size = np.abs(x) @ np.abs(w).T
    depth = 64 + w.shape[1] / 32
    return (2.0 ** -22 + depth * 2.0 ** -24) * size + 2.0 ** -50 * np.abs(x).max(initial=0) * np.abs(w).sum(1) + 1e-38


def silu(g):
    return g / (1 + np.exp(-g))


# --- paged cache ----------------------------------------------------------------
class Cache:
    """Host copy of a cache and its sequences.  k, v: float16, or int8 with float32 scales."""

    def __init__(self, rng, fmt, layers, pages, page_size, kv_heads, head_dim, seqs, width, lengths=(), spread=1.0, shuffle=True):
        self.fmt, self.layers, self.pages, self.page_size = fmt, layers, pages, page_size
        self.kv_heads, self.head_dim, self.seqs, self.width = kv_heads, head_dim, seqs, width
        shape = (layers, pages, kv_heads, page_size, head_dim)
        if fmt == "f16":
            self.k, self.v = ((rng.standard_normal(shape) * spread).astype(np.float16) for _ in range(2))
            self.k_scales = self.v_scales = None
        else:
            self.k, self.v = (rng.integers(-127, 128, shape).astype(np.int8) for _ in range(2))
            self.k_scales, self.v_scales = (((rng.random(shape[:-1]) + 0.5) * (spread / 64)).astype(np.float32) for _ in range(2))
        self.table = np.full((seqs, width), -1, np.int32)
        self.lengths = np.zeros(seqs, np.int32)
        self.refs = np.zeros(pages, np.int32)
        order = rng.permutation(pages) if shuffle else np.arange(pages)
        at = 0
        for s, n in enumerate(lengths):
            m = -(-n // page_size)
            self.table[s, :m] = order[at:at + m]
            self.refs[order[at:at + m]] = 1
            self.lengths[s] = n
            at += m

    def rows(self, name, layer, seq, head):
        """[tokens][head_dim] float64 of a sequence, and which tokens have a page."""
        n, p = self.length(seq), self.page_size
        t = np.arange(n)
        page = self.table[seq, t // p]
        there = (page >= 0) & (page < self.pages)
        at = np.where(there, page, 0)
        x = getattr(self, name)[layer, at, head, t % p].astype(np.float64)
        if self.fmt != "f16":
            x = x * getattr(self, name + "_scales")[layer, at, head, t % p].astype(np.float64)[:, None]
        return x, there

    def length(self, seq):
        return int(min(max(int(self.lengths[seq]), 0), self.width * self.page_size))

    def held(self, seq):
        return -(-self.length(seq) // self.page_size)

    def attend(self, layer, q, scale, seq_ids=None):
        """(y, bound) [rows][heads][head_dim]: the exact result, and how far float32 scores, weights and sums of two-part
        operands may be from it (a rounding of the result itself not counted)."""
        rows, heads, d = q.shape
        g = heads // self.kv_heads
        y, bound = np.zeros(q.shape), np.zeros(q.shape)
        for r in range(rows):
            s = r if seq_ids is None else int(seq_ids[r])
            if not 0 <= s < self.seqs:
                continue
            for h in range(heads):
                k, there = self.rows("k", layer, s, h // g)
                v, _ = self.rows("v", layer, s, h // g)
                k, v = k[there], v[there]
                if len(k) == 0:
                    continue
                qh = q[r, h].astype(np.float64)
                score = k @ qh * scale
                p = np.exp(score - score.max())
                total = p.sum()
                y[r, h] = p @ v / total
                # a score: operands within 2^-22 (scale and log2(e) folded into q add two roundings of 2^-24), a chain of
                # at most 32 + d / 32 additions, then its difference from the maximum and the exponential's own error
                size = np.abs(k) @ np.abs(qh) * abs(scale)
                off = (2.0 ** -22 + (36 + d / 32) * 2.0 ** -24) * size + 2.0 ** -22 * (np.abs(score) + np.abs(score.max())) + 2.0 ** -22
                # weights: their scores' errors, two parts; sums: a chain of 64 + tokens / 32 additions, above and below
                each = 2 * off.max() + 2.0 ** -22 + 2 * (96 + len(k) / 32) * 2.0 ** -24
                bound[r, h] = each * (p @ np.abs(v)) / total + 1e-38
        return y, bound

    # page upkeep, one step at a time
    def lowest_free(self):
        return np.flatnonzero(self.refs <= 0)

    def extend(self, seq_ids, counts):
        seen, plan = set(), []
        for s, c in zip(seq_ids, counts):
            if not 0 <= s < self.seqs or s in seen:
                continue
            seen.add(s)
            plan.append((s, self.length(s), self.length(s) + max(int(c), 0)))
        if any(new > self.width * self.page_size for _, _, new in plan):
            return -1
        need = [-(-new // self.page_size) - -(-old // self.page_size) for _, old, new in plan]
        free = self.lowest_free()
        if sum(need) > len(free):
            return sum(need) - len(free)
        at = 0
        for (s, old, new), n in zip(plan, need):
            first = -(-old // self.page_size)
            self.table[s, first:first + n] = free[at:at + n]
            self.refs[free[at:at + n]] = 1
            self.lengths[s] = new
            at += n
        return 0

    def free(self, seq_ids):
        for s in seq_ids:
            if not 0 <= s < self.seqs:
                continue
            for j in range(self.held(s)):
                p = self.table[s, j]
                if 0 <= p < self.pages:
                    self.refs[p] -= 1
                self.table[s, j] = -1
            self.lengths[s] = 0

    def copy_page(self, src, dst):
        for x in (self.k, self.v, self.k_scales, self.v_scales):
            if x is not None:
                x[:, dst] = x[:, src]

    def fork(self, parents, children):
        before, seen, plan = [self.length(s) for s in range(self.seqs)], set(), []
        for p, c in zip(parents, children):
            if not 0 <= c < self.seqs or not 0 <= p < self.seqs or c in seen:
                continue
            seen.add(c)
            if before[c] == 0:
                plan.append((p, c))
        free = self.lowest_free()
        need = sum(before[p] % self.page_size != 0 for p, _ in plan)
        if need > len(free):
            return need - len(free)
        at = 0
        for p, c in plan:
            whole = before[p] // self.page_size
            for j in range(whole):
                page = self.table[p, j]
                self.table[c, j] = page
                if 0 <= page < self.pages:
                    self.refs[page] += 1
            if before[p] % self.page_size:
                old, new = self.table[p, whole], free[at]
                at += 1
                self.table[c, whole] = new
                self.refs[new] = 1
                if 0 <= old < self.pages:
                    self.copy_page(old, new)
            self.lengths[c] = before[p]
        return 0

    def compact(self):
        live = int((self.refs > 0).sum())
        holes = np.flatnonzero(self.refs[:live] <= 0)
        movers = live + np.flatnonzero(self.refs[live:] > 0)
        to = np.arange(self.pages)
        to[movers] = holes
        for a, b in zip(movers, holes):
            self.copy_page(a, b)
        self.refs[holes], self.refs[movers] = self.refs[movers], 0
        for s in range(self.seqs):
            for j in range(self.held(s)):
                p = self.table[s, j]
                if 0 <= p < self.pages:
                    self.table[s, j] = to[p]
        return live

    def append(self, layer, k, v, seq_ids, positions):
        """k, v [rows][kv_heads][head_dim] float32 or float16."""
        for name, x in (("k", k), ("v", v)):
            x = x.astype(np.float64)
            for r in range(len(x)):
                s = int(seq_ids[r])
                if not 0 <= s < self.seqs:
                    continue
                t = int(positions[r])
                if not 0 <= t < self.length(s):
                    continue
                page = self.table[s, t // self.page_size]
                if not 0 <= page < self.pages:
                    continue
                at = (layer, page, slice(None), t % self.page_size)
                if self.fmt == "f16":
                    with np.errstate(over="ignore"):
                        getattr(self, name)[at] = x[r].astype(np.float32).astype(np.float16)
                else:
                    codes, scales = i8_rows(x[r])
                    getattr(self, name)[at] = codes
                    getattr(self, name + "_scales")[at] = scales


def i8_rows(x):
    """Codes and scales of rows: scale = max / 127 (one float32 rounding), the exact quotient rounded half away from zero;
    a row with an infinity or NaN gets scale NaN and codes 0, a row whose scale is 0 codes 0."""
    codes, scales = np.zeros(x.shape, np.int8), np.zeros(x.shape[:-1], np.float32)
    for i in np.ndindex(*x.shape[:-1]):
        row = x[i].astype(np.float64)
        if not np.isfinite(row).all():
            scales[i] = np.nan
            continue
        scale = np.float32(np.float32(np.abs(row).max()) / np.float32(127))
        scales[i] = scale
        if scale > 0:
            # quotient and tie in integers over the scale: 2 |x| against (2 q + 1) scale, both exact in 64 bits
            s, a = np.float64(scale), np.abs(row)
            q = np.floor(a / s)
            q = np.where(a < q * s, q - 1, np.where(a >= (q + 1) * s, q + 1, q))
            q = q + (2 * (a - q * s) >= s)
            codes[i] = (np.sign(row) * np.minimum(q, 127)).astype(np.int8)
    return codes, scales
