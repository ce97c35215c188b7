"""The attention-side operators as plain numpy: the append operation by operation in fp32, as it is
specified, and attention in 64 bits, with the error that the kernels' number formats allow."""
import numpy as np

LOG2E = 1.4426950408889634


def turn32(x, rope, rot, interleaved):
    """x fp32 [T][heads][D], rope fp32 [T][rot]; every product and sum rounded to fp32."""
    y = x.copy()
    c, s = rope[:, None, : rot // 2], rope[:, None, rot // 2: rot]
    i0 = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    i1 = i0 + (1 if interleaved else rot // 2)
    a, b = x[..., i0], x[..., i1]
    y[..., i0] = (a * c).astype(np.float32) - (b * s).astype(np.float32)
    y[..., i1] = (b * c).astype(np.float32) + (a * s).astype(np.float32)
    return y


def _bf16(x):
    """fp64 -> the values of the nearest bf16 (ties to even), through fp32 with the sticky bit of round to odd."""
    f = x.astype(np.float32)
    u = f.view(np.uint32).astype(np.int64)
    u = np.where(f.astype(np.float64) == x, u, np.where(np.abs(f.astype(np.float64)) > np.abs(x), u - 1, u) | 1)
    u = (u + 0x7FFF + ((u >> 16) & 1)) >> 16 << 16
    return u.astype(np.uint32).view(np.float32).astype(np.float64)


def within(got, want, tol, bf16):
    """(all fine, worst share of the tolerance): |got - want| <= tol, or, for a bf16 result, got between the roundings
    of want - tol and want + tol."""
    err = np.abs(got - want)
    if not bf16:
        return bool(np.all(err <= tol)), float((err / np.maximum(tol, 1e-300)).max(initial=0.0))
    fine = (got >= _bf16(want - tol)) & (got <= _bf16(want + tol))
    return bool(np.all(fine)), float((err / np.maximum(tol + 2.0 ** -8 * np.abs(want), 1e-300)).max(initial=0.0))


class Cache:
    """A paged int8 cache on the host, in the header's layout."""

    def __init__(self, pages, heads, dim, page, rng=None):
        self.pages, self.heads, self.dim, self.page = pages, heads, dim, page
        r = rng or np.random.default_rng(0)
        self.k = r.integers(-127, 128, (pages, heads, page, dim)).astype(np.int8)
        self.v = r.integers(-127, 128, (pages, heads, dim, page)).astype(np.int8)
        self.ks = r.uniform(0.005, 0.05, (pages, heads)).astype(np.float32)
        self.vs = r.uniform(0.005, 0.05, (pages, heads)).astype(np.float32)

    def values(self, table_row, n):
        """k, v fp64 [heads][n][dim] of the first n positions; positions of unnamed pages give NaN."""
        k = np.full((self.heads, n, self.dim), np.nan)
        v = np.full((self.heads, n, self.dim), np.nan)
        for slot in range(-(-n // self.page)):
            pid = int(table_row[slot])
            if not 0 <= pid < self.pages:
                continue
            lo, hi = slot * self.page, min(n, (slot + 1) * self.page)
            k[:, lo:hi] = self.k[pid, :, : hi - lo].astype(np.float64) * self.ks[pid].astype(np.float64)[:, None, None]
            v[:, lo:hi] = (self.v[pid].astype(np.float64) * self.vs[pid].astype(np.float64)[:, None, None]
                           ).transpose(0, 2, 1)[:, : hi - lo]
        return k, v

    def _store(self, codes, scales, pid, r0, x):
        """x fp32 [new][heads][D] into rows r0.. of page pid; codes: a view [heads][page][D] of the page."""
        f = np.float32
        want = np.maximum(np.abs(x).max(axis=(0, 2)), f(1e-5)) / f(127)
        old = scales[pid].copy()
        now = np.maximum(old, want) if r0 else want
        for h in range(self.heads):
            if r0 and now[h] > old[h]:
                codes[h, :r0] = np.rint(codes[h, :r0].astype(f) * (old[h] / now[h])).astype(np.int8)
            q = np.rint(x[:, h] * (f(1) / now[h]))
            codes[h, r0: r0 + len(x)] = np.clip(q, -127, 127).astype(np.int8)
        scales[pid] = now

    def append(self, x, rope, rot, interleaved, table, starts, before, max_new, q_heads):
        """x fp32 [T][q_heads + 2 heads][D].  Returns the turned (q, k) in fp32; rows of no token are NaN."""
        hk = self.heads
        q = np.full((x.shape[0], q_heads, self.dim), np.nan, np.float32)
        k = np.full((x.shape[0], hk, self.dim), np.nan, np.float32)
        for b in range(len(before)):
            n = min(int(starts[b + 1] - starts[b]), max_new)
            for slot in range(before[b] // self.page, -(-(before[b] + n) // self.page) if n > 0 else 0):
                base = slot * self.page
                p0, p1 = max(before[b], base), min(before[b] + n, base + self.page)
                if p0 >= p1:
                    continue
                t = slice(starts[b] + p0 - before[b], starts[b] + p1 - before[b])
                if slot >= table.shape[1]:
                    q[t], k[t] = 0, 0
                    continue
                turned = turn32(x[t, : q_heads + hk], rope[p0:p1], rot, interleaved) if rot else x[t, : q_heads + hk]
                q[t], k[t] = turned[:, :q_heads], turned[:, q_heads:]
                pid = int(table[b, slot])
                if 0 <= pid < self.pages:
                    self._store(self.k[pid], self.ks, pid, p0 - base, turned[:, q_heads:])
                    self._store(self.v[pid].transpose(0, 2, 1), self.vs, pid, p0 - base, x[t, q_heads + hk:])
        return q, k


def softmax_rows(q, k, v, scale, see):
    """q [rows][D], k, v [n][D], see bool [rows][n], fp64.  Returns (out, sum p|v|, largest |score|); rows that see
    nothing give zeros."""
    s = (q @ k.T) * scale
    s = np.where(see, s, -np.inf)
    m = s.max(axis=1, initial=-np.inf, keepdims=True)
    p = np.where(see, np.exp(s - np.where(np.isfinite(m), m, 0.0)), 0.0)
    l = p.sum(axis=1, keepdims=True)
    p = np.divide(p, l, out=np.zeros_like(p), where=l > 0)
    big = np.abs(np.where(see, s, 0.0)).max(axis=1, initial=0.0, keepdims=True)
    return p @ v, p @ np.abs(v), big


def decode(q, cache, table, lengths, scale, fine, q_bits):
    """q fp64 [B][Hq][D].  Returns (out, tolerance).  The tolerance, for a largest |v| of a key head of vmax:
      * weights in digits: each off by at most half a unit, 2^-16 (2^-24 when fine) of the largest weight of
        its 64 tokens, 64 of them: 64 * 2^-16 * vmax in all, as the largest weights of the tiles sum to at most 1;
      * a score off by d changes a weight by d, and the output by at most 2 d vmax: d is half a unit of
        the query's digits, 2^-(q_bits + 1) of its largest value, against sum |k|, plus three fp32 roundings of the score;
      * exp2, the running sums and their joining: 2^-20 vmax (fp32, tens of roundings of 2^-24).
    A bf16 output is the rounding of a value within it (`within`)."""
    B, hq, D = q.shape
    hk = cache.heads
    out, tol = np.zeros_like(q), np.zeros_like(q)
    for b in range(B):
        n = max(0, int(lengths[b]))
        if n == 0:
            continue
        k, v = cache.values(table[b], n)
        there = ~np.isnan(k[0, :, 0])
        k, v = np.nan_to_num(k), np.nan_to_num(v)
        for h in range(hk):
            r = slice(h * (hq // hk), (h + 1) * (hq // hk))
            o, _, big = softmax_rows(q[b, r], k[h], v[h], scale, np.broadcast_to(there, (hq // hk, n)))
            vmax = np.abs(v[h]).max()
            d = 2.0 ** -(q_bits + 1) * 2 * np.abs(q[b, r]).max(1, keepdims=True) * np.abs(k[h]).sum(1).max() * scale
            d = d + 3 * 2.0 ** -24 * big * 2
            out[b, r] = o
            tol[b, r] = (64 * 2.0 ** -(24 if fine else 16) + 2 * d + 2.0 ** -20) * vmax
    return out, tol


def prompt(q, k, v, starts, causal, scale, max_len):
    """fp64 [T][heads][D].  Returns (out, tolerance, rows written).  Tolerance: every weight rounded to bf16 (8 bits: off by
    2^-8 of it at most, against |v|) and fp32 scores, exponents and sums: 2^-15 vmax.  The bf16 output is the rounding
    of a value within it (`within`)."""
    T, hq, D = q.shape
    hk = k.shape[1]
    out, tol, wrote = np.zeros_like(q), np.zeros_like(q), np.zeros(T, bool)
    for lo, hi in zip(starts, starts[1:]):
        n = min(hi - lo, max_len)
        if n <= 0:
            continue
        see = np.tril(np.ones((n, n), bool)) if causal else np.ones((n, n), bool)
        wrote[lo: lo + n] = True
        for h in range(hq):
            kk, vv = k[lo: lo + n, h * hk // hq], v[lo: lo + n, h * hk // hq]
            o, a, _ = softmax_rows(q[lo: lo + n, h], kk, vv, scale, see)
            out[lo: lo + n, h] = o
            tol[lo: lo + n, h] = 2.0 ** -8 * a + 2.0 ** -15 * np.abs(vv).max()
    return out, tol, wrote
