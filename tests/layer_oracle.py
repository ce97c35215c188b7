"""Plain forms, in 64 bits, of what stands between the products of a decoder layer, and the tolerances that the kernels' own roundings
allow.  The norm's codes are defined in fp32, operation by operation, and are whole numbers to be met exactly."""
import math

import numpy as np
import torch

HALF = 2.0 ** -24  # half a step of fp32, relative
ACTS = ("none", "relu", "relu2", "silu", "gelu")


def rounded(v, dtype):
    """fp32 array rounded to dtype and widened again."""
    return torch.from_numpy(np.ascontiguousarray(v, np.float32)).to(dtype).float().numpy()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------ norm
def add_norm(x, weight, eps, dtype, add=None, slots=None, gates=None):
    """x, add fp32 arrays of values of their types.  Returns (stream, h, codes, s_a), fp32 each operation as the header has them."""
    f = np.float32
    with np.errstate(invalid="ignore", over="ignore"):
        if slots is not None:
            d = np.zeros_like(x)
            for m in range(x.shape[0]):
                for j in range(slots.shape[1]):
                    if 0 <= slots[m, j] < add.shape[0]:
                        d[m] = d[m] + f(gates[m, j]) * add[slots[m, j]]
            x = rounded(x + d, dtype)
        elif add is not None:
            x = rounded(x + add, dtype)
        mean = (x.astype(np.float64) ** 2).sum(-1) / x.shape[1]
        r = (1.0 / np.sqrt(mean + float(f(eps)))).astype(f)
        h = x * r[:, None]
        if weight is not None:
            h = h * weight
        most = np.abs(h).max(-1)
        good = np.isfinite(most)
        top = np.maximum(np.where(good, most, f(1.0)), f(1e-5)).astype(f)
        codes = np.rint(h * (f(127.0) / top)[:, None])
        codes = np.where(good[:, None], codes, 0.0).astype(np.int8)
        return x, h, codes, np.where(good, top / f(127.0), f(np.nan)).astype(f)


# ------------------------------------------------------------------ products
def product(T, S, q, s_a):
    """(z, |terms|) in 64 bits: T [N][K], S [N][K/128], q [M][K], s_a [M]."""
    z = np.zeros((q.shape[0], T.shape[0]))
    mag = np.zeros_like(z)
    for b in range(S.shape[1]):
        a = (q[:, 128 * b: 128 * (b + 1)].astype(np.float64) @ T[:, 128 * b: 128 * (b + 1)].astype(np.float64).T) * S[:, b].astype(np.float64)
        z += a
        mag += np.abs(a)
    s = s_a.astype(np.float64)[:, None]
    return z * s, mag * np.abs(s)


def activation(z, act):
    """(act(z), the largest slope within a hair of z, the rounding of computing it in fp32)."""
    tiny = 2.0 ** -125  # below the smallest normal number: exp overflowed
    if act == "none":
        return z, np.ones_like(z), np.zeros_like(z)
    if act == "relu":
        return np.maximum(z, 0), np.ones_like(z), np.zeros_like(z)
    if act == "relu2":
        a = np.maximum(z, 0) ** 2
        return a, 2 * np.abs(z) * (1 + 1e-4) + 1e-4, HALF * a
    with np.errstate(over="ignore"):
        if act == "silu":
            u, slope = z, 1.1
        else:
            u, slope = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3), 1.13
        a = z / (1 + np.exp(-u))
    # the argument of the exponential, u log2 e: up to 8 roundings; the exponential, the sum and the quotient: 4 more, each a whole step
    part = np.where(u < 40, 1 / (1 + np.exp(np.minimum(u, 700))), 0.0)  # how much of a's relative error the exponential's becomes
    return a, np.full_like(z, slope), np.abs(a) * (8 * 2 * HALF * np.abs(u) * part + 8 * HALF) + tiny


def epilogue(z, mag, blocks, bias, act, gated, residual, dtype):
    """(y, tolerance).  A sum of `blocks` terms, cut over at most 16 waves, scaled once: blocks + 18 roundings of at most the sum of the
    terms' magnitudes; the bias one more of the result; then activation, gate, residual and the output's own rounding."""
    dz = (blocks + 18) * HALF * mag
    if bias is not None:
        z = z + bias
        dz = dz + HALF * (np.abs(z) + dz)
    if gated:
        n = z.shape[1] // 2
        z, up, dz, du = z[:, :n], z[:, n:], dz[:, :n], dz[:, n:]
    a, slope, da = activation(z, act)
    da = da + slope * dz * 1.01 + (dz * dz if act == "relu2" else 0)
    if gated:
        y = a * up
        da = da * (np.abs(up) + du) + np.abs(a) * du
        da = da + HALF * (np.abs(y) + da)
    else:
        y = a
    if residual is not None:
        y = y + residual
        da = da + HALF * (np.abs(y) + da)
    return y, da + (half_step(dtype) if dtype != torch.float32 else 0.0) * (np.abs(y) + da) + 2.0 ** -126


def linear(T, S, q, s_a, bias, act, gated, residual, dtype):
    z, mag = product(T, S, q, s_a)
    return epilogue(z, mag, S.shape[1], bias, act, gated, residual, dtype)


def close(got, want, tol):
    """Whether every value lies within its tolerance; NaN only where NaN is due."""
    got = got.double().cpu().numpy()
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan)
    off = np.abs(got - want)[~nan] - tol[~nan]
    assert off.size == 0 or off.max() <= 0, (off.max(), np.abs(got - want)[~nan].max())
    return True


# ------------------------------------------------------------------ routing
def route(logits, k, over_all):
    """(chosen, gates in 64 bits, starts, rows, slots) of fp32 logits."""
    T, E = logits.shape
    order = np.where(np.isnan(logits), -np.inf, logits).astype(np.float64)
    chosen = np.argsort(-order, axis=1, kind="stable")[:, :k]
    value = np.take_along_axis(order, chosen, 1)
    there = value > -np.inf
    with np.errstate(invalid="ignore"):
        top = np.where(there[:, :1], value[:, :1], 0.0)
        gates = np.where(there, np.exp(value - top), 0.0)
        total = np.exp(order - top).sum(1, keepdims=True) if over_all else gates.sum(1, keepdims=True)
        gates = np.where(there, gates / np.where(there[:, :1], total, 1.0), 0.0)
    chosen = np.where(there, chosen, -1).astype(np.int32)
    starts, rows, slots = [0], np.full(T * k, -1, np.int32), np.full((T, k), -1, np.int32)
    for e in range(E):
        token, place = np.nonzero(chosen == e)
        at = starts[-1] + np.arange(len(token))
        rows[at], slots[token, place] = token, at
        starts.append(starts[-1] + len(token))
    return chosen, gates, np.array(starts, np.int32), rows, slots
