"""Bounds of decode attention's error row by row, from the roundings that the kernel makes, for caches whose scales differ widely:
attn_oracle.decode charges every rounding against the largest value of the whole head, this one against what a row weighs."""
import numpy as np

import attn_oracle as ao

TILE = 64


def decode(q, cache, table, lengths, scale):
    """q fp64 [B][Hq][D], all pages named by `table` present.  Returns (out, tolerance) in fp64:
      * weights: e_j s_j (s_j the scale of j's values) as whole multiples of 1 / (127 * 65536) of the largest of its 64 tokens: off by at most half of
        that, 2^-23.98, against codes of at most 127: 127 * 2^-23.98 * sum over tiles of 64 max_j p_j s_j;
      * a score off by d_j: the output by sum p_j d_j (|v_j| + sum p |v|).  d_j: the query's digits, 2^-31 of a power of two that is at most
        twice its largest value, against sum |k_j|; four digit products, each at most that power of two times sum |k_j|, rounded when they are
        scaled and twice when they are summed; the difference to the tile's and the row's largest score, and the exponent's argument, 4
        roundings of values up to 2 max |s|;
      * what is rounded in the weight and the sums themselves: exponential, scale and unit of a weight, factor of a tile, sums of tiles, waves and
        splits: 2^-20 sum p |v| (tens of roundings of 2^-24).
    A bf16 output is the rounding of a value within it (attn_oracle.within)."""
    B, hq, D = q.shape
    group = hq // cache.heads
    out, tol = np.zeros_like(q), np.zeros_like(q)
    for b in range(B):
        n = max(0, int(lengths[b]))
        if n == 0:
            continue
        k, v = cache.values(table[b], n)
        vs = np.repeat(cache.vs[table[b, : -(-n // cache.page)]].astype(np.float64), cache.page, axis=0)[:n]
        for i in range(hq):
            kk, vv, ss = k[i // group], v[i // group], vs[:, i // group]
            s = (kk @ q[b, i]) * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            a = p @ np.abs(vv)
            reach = 2 * np.abs(q[b, i]).max() * np.abs(kk).sum(1) * scale
            d = reach * 2.0 ** -31 + 3 * reach * 2.0 ** -24 + 4 * 2 * np.abs(s).max() * 2.0 ** -24
            tiles = np.pad(p * ss, (0, -n % TILE)).reshape(-1, TILE).max(1).sum()
            out[b, i] = p @ vv
            tol[b, i] = (127 * 64 * 2.0 ** -23.98 * tiles + (p * d) @ np.abs(vv) + (p @ d) * a + 2.0 ** -20 * a) * 1.001
    return out, tol


def decode_fine(got, q, cache, table, lengths, scale, bf16):
    """(all fine, worst share of the tolerance) of an output against `decode`."""
    want, tol = decode(q, cache, table, lengths, scale)
    return ao.within(got, want, tol, bf16)


def emulate(q, cache, table, lengths, scale, q_bits=30, weight_unit=127 * 65536):
    """Decode attention with the kernel's digits and 64 bits for everything else: queries as whole multiples of 2^-q_bits of the power of two above
    their row's largest, products of weight and value scale as whole multiples of 1 / weight_unit of the largest of their 64."""
    B, hq, D = q.shape
    group = hq // cache.heads
    out = np.zeros_like(q)
    for b in range(B):
        n = max(0, int(lengths[b]))
        k, v = cache.values(table[b], n)
        vs = np.repeat(cache.vs[table[b, : -(-n // cache.page)]].astype(np.float64), cache.page, axis=0)[:n]
        for i in range(hq if n else 0):
            step = 2.0 ** (np.frexp(np.abs(q[b, i]).max())[1] - q_bits)
            s = (k[i // group] @ (np.rint(q[b, i] / step) * step)) * scale
            total, l = np.zeros(D), 0.0
            for t in range(0, n, TILE):
                e, sv = np.exp(s[t: t + TILE] - s[t: t + TILE].max()), vs[t: t + TILE, i // group]
                unit = max((e * sv).max() / weight_unit, 1e-300)
                codes = np.divide(v[i // group, t: t + TILE], sv[:, None], out=np.zeros((len(sv), D)), where=sv[:, None] > 0)
                beta = np.exp(s[t: t + TILE].max() - s.max())
                total += beta * unit * (np.rint(e * sv / unit) @ codes)
                l += beta * e.sum()
            out[b, i] = total / l
    return out
