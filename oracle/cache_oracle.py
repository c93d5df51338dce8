"""Oracle of the cache's writers, readers and page pool (test infrastructure).

Plain float64 / Python-list statements of what include/mla_paged.h defines; no code is
shared with the CUDA path.  An FP8 token follows the FlashMLA notes, "FP8 KV Cache
Quantization and Dequantization" (512 E4M3 values, four float32 scales, 64 bf16 values);
the float32 scale and the float32 quotient value / scale are part of that format, so they
are computed in float32 here too.
"""

from __future__ import annotations

import numpy as np

BAD_INDEX, NO_PAGES = -6, -11


def rope(x, positions, inv_freq, sections, interleaved):
    """Rotary positions on x [T, H, 64]; positions [axes, T]; float64."""
    x = np.asarray(x, np.float64)
    positions = np.asarray(positions, np.float64)
    out = np.empty_like(x)
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    for i in range(32):
        angle = positions[axis[i]] * np.float64(inv_freq[i])
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + 32)
        a, b = x[..., ia], x[..., ib]
        out[..., ia] = a * c - b * s
        out[..., ib] = a * s + b * c
    return out


def _e4m3_values():
    v = []
    for code in range(127):
        e, m = code >> 3, code & 7
        v.append((m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(v)


def quantise(ckv):
    """Latents [n, 512] -> (codes [n, 512] uint8, scales [n, 4] float32).  The code is the
    nearest E4M3 number to the float32 quotient, ties to the even code; NaN (0x7F) for a
    value that is not finite."""
    tiles = np.asarray(ckv, np.float32).reshape(-1, 4, 128)
    finite = np.isfinite(tiles)
    amax = np.where(finite, np.abs(tiles), 0).max(-1).astype(np.float32)
    scales = np.where(amax > 0, amax / np.float32(448), np.float32(1)).astype(np.float32)
    with np.errstate(invalid="ignore"):
        q = (tiles / scales[..., None]).astype(np.float32)
    table = _e4m3_values()
    mag = np.minimum(np.where(finite, np.abs(q), 0).astype(np.float64), 448.0)
    hi = np.clip(np.searchsorted(table, mag), 0, 126)
    lo = np.maximum(hi - 1, 0)
    below, above = mag - table[lo], table[hi] - mag
    code = np.where(below < above, lo, np.where(above < below, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(finite, code + 128 * np.signbit(q), 0x7F)
    return code.astype(np.uint8).reshape(-1, 512), scales.reshape(-1, 4)


class Pool:
    """The page pool as Python lists, one entry after the other."""

    def __init__(self, table, lens, refs, page_size):
        self.table = [list(map(int, r)) for r in table]
        self.lens = list(map(int, lens))
        self.refs = list(map(int, refs))
        self.ps = page_size

    def blocks(self, n):
        return -(-n // self.ps)

    def row_ok(self, r):
        return 0 <= r < len(self.lens)

    def page_ok(self, p):
        return 0 <= p < len(self.refs)

    def room(self):
        return (len(self.table[0]) if self.table else 0) * self.ps

    def _grant(self, needs):
        """needs: None (invalid) or pages of every entry -> statuses and the pages given."""
        free = [p for p, n in enumerate(self.refs) if n <= 0]
        total, status, pages = 0, [], []
        for need in needs:
            if need is None:
                status.append(BAD_INDEX)
                pages.append([])
                continue
            total += need
            if need and total > len(free):
                status.append(NO_PAGES)
                pages.append([])
            else:
                status.append(0)
                pages.append(free[total - need:total])
        return status, pages

    def extend(self, rows, new, capacity):
        needs, seen = [], set()
        for r, a in zip(rows, new):
            ok = self.row_ok(r) and r not in seen
            if self.row_ok(r):
                seen.add(r)
            if ok:
                n = self.lens[r]
                ok = n >= 0 and a >= 0 and n + a <= self.room()
                if ok and a and n % self.ps:
                    page = self.table[r][n // self.ps]
                    ok = self.page_ok(page) and self.refs[page] == 1
            needs.append(self.blocks(n + a) - self.blocks(n) if ok else None)
        status, pages = self._grant(needs)
        ptr, slots = [0], []
        for r, a, st, pg in zip(rows, new, status, pages):
            if st == 0:
                n = self.lens[r]
                for k, page in enumerate(pg):
                    self.table[r][self.blocks(n) + k] = page
                    self.refs[page] = 1
                slots += [self.table[r][p // self.ps] * self.ps + p % self.ps for p in range(n, n + a)]
                self.lens[r] = n + a
            ptr.append(ptr[-1] + (a if st == 0 else 0))
        return ptr, (slots + [-1] * capacity)[:capacity], status

    def fork(self, parents, children):
        needs, seen, before = [], set(), list(self.lens)
        for p, c in zip(parents, children):
            ok = self.row_ok(c) and c not in seen
            if self.row_ok(c):
                seen.add(c)
            ok = ok and self.row_ok(p) and p != c and before[c] == 0
            if ok:
                n = before[p]
                ok = 0 <= n <= self.room()
                if ok and n % self.ps:
                    ok = self.page_ok(self.table[p][n // self.ps])
            needs.append((1 if n % self.ps else 0) if ok else None)
        status, pages = self._grant(needs)
        src, dst, tokens = [], [], []
        for p, c, st, pg in zip(parents, children, status, pages):
            s, d, t = -1, -1, 0
            if st == 0:
                n = before[p]
                for k in range(n // self.ps):
                    page = self.table[p][k]
                    self.table[c][k] = page
                    if self.page_ok(page):
                        self.refs[page] += 1
                if pg:
                    s, d, t = self.table[p][n // self.ps], pg[0], n % self.ps
                    self.table[c][n // self.ps] = d
                    self.refs[d] = 1
                self.lens[c] = n
            src.append(s)
            dst.append(d)
            tokens.append(t)
        return status, src, dst, tokens

    def free(self, rows):
        for r in rows:
            if not self.row_ok(r):
                continue
            for k in range(min(self.blocks(max(self.lens[r], 0)), len(self.table[r]))):
                page, self.table[r][k] = self.table[r][k], -1
                if self.page_ok(page):
                    self.refs[page] = max(self.refs[page] - 1, 0)
            self.lens[r] = 0

    def compact(self):
        live = sum(1 for n in self.refs if n > 0)
        src = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        dst = [p for p in range(live) if self.refs[p] <= 0]
        new = dict(zip(src, dst))
        for s, d in new.items():
            self.refs[d], self.refs[s] = self.refs[s], 0
        for r, n in enumerate(self.lens):
            for k in range(min(self.blocks(max(n, 0)), len(self.table[r]))):
                self.table[r][k] = new.get(self.table[r][k], self.table[r][k])
        return live, src, dst
