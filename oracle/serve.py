"""Oracle of the serving operators: the product with q4tp weights, the 4-bit
key/value cache and the attention over it, plain numpy in 64 bits.

Inputs are arrays of numbers that the 16-bit type ("bf16" or "f16") holds
exactly.  Only what a definition rounds is rounded: the cache's (s, z) and
codes follow f32 arithmetic with one rounding per operation, its values one
rounding to the type.

Test infrastructure: see the package docstring.
"""
from __future__ import annotations

import math

import numpy as np

F32, F64 = np.float32, np.float64
GROUP, BLOCK = 32, 16
# significand bits, smallest normal exponent, largest number
TYPES = {"bf16": (8, -126, float.fromhex("0x1.fep127")), "f16": (11, -14, 65504.0)}


def round_to(x, dtype):
    """Nearest number of the type, ties to even, from 64 bits (inf past the end)."""
    p, emin, top = TYPES[dtype]
    x = np.asarray(x, dtype=F64)
    with np.errstate(all="ignore"):
        _, e = np.frexp(x)
        ulp = np.ldexp(1.0, np.maximum(e, emin + 1) - p)
        r = np.rint(x / ulp) * ulp
        return np.where(np.isfinite(x), np.where(np.abs(r) > top, np.copysign(np.inf, x), r), x)


def activate(v, act):
    v = np.asarray(v, dtype=F64)
    with np.errstate(all="ignore"):
        if act == "relu":
            return np.where(v < 0, 0.0, v)
        if act == "gelu":
            return 0.5 * v * (1 + np.vectorize(math.erf, otypes=[F64])(v / math.sqrt(2)))
        if act == "gelu_tanh":
            return 0.5 * v * (1 + np.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
        if act == "silu":
            return v / (1 + np.exp(-v))
    return v


def weights(nibbles, rungs, tab):
    """W [rows, n] in 64 bits; a rung above 31 counts as scale 0."""
    tab = np.asarray(tab, dtype=F64)
    rows = tab.shape[0]
    b = np.asarray(nibbles, dtype=np.uint8).reshape(rows, -1)
    n = b.shape[1] * 2
    q = np.empty((rows, n), dtype=F64)
    q[:, 0::2] = (b & 15).astype(F64) - 8
    q[:, 1::2] = (b >> 4).astype(F64) - 8
    r = np.asarray(rungs, dtype=np.int64).reshape(rows, n // GROUP)
    s = np.where(r < 32, np.take_along_axis(tab, np.minimum(r, 31), 1), 0.0)
    return q * np.repeat(s, GROUP, axis=1)


def linear(x, nibbles, rungs, tab, bias=None, act="none", residual=None):
    y = np.asarray(x, dtype=F64) @ weights(nibbles, rungs, tab).T
    if bias is not None:
        y = y + np.asarray(bias, dtype=F64)
    y = activate(y, act)
    return y if residual is None else y + np.asarray(residual, dtype=F64)


def quantise(x, dtype):
    """(codes [..., d] int, s, z [..., d / 32] as numbers of the type); s = z =
    NaN marks a group that cannot be held."""
    x = np.asarray(x, dtype=F32)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    with np.errstate(all="ignore"):
        lo, hi = g.min(-1), g.max(-1)  # numpy's keep a NaN
        s = round_to((hi - lo) * F32(1 / 15), dtype).astype(F32)
        z = round_to(lo - F32(16) * s, dtype).astype(F32)
        bad = ~(np.isfinite(s) & np.isfinite(z))
        s, z = np.where(bad, F32(np.nan), s), np.where(bad, F32(np.nan), z)
        r = np.where(s > 0, F32(1) / np.where(s > 0, s, F32(1)), F32(0)).astype(F32)
        c = np.rint((g - z[..., None]) * r[..., None])
    c = np.clip(np.where(np.isnan(c), 16, c), 16, 31).astype(np.int64) - 16
    return c.reshape(x.shape), s, z


def values(codes, s, z, dtype):
    c = np.asarray(codes, dtype=F64).reshape(*s.shape, GROUP)
    v = z.astype(F64)[..., None] + s.astype(F64)[..., None] * (16 + c)  # exact in 64 bits for any (s, z) near each other
    return round_to(v, dtype).reshape(*s.shape[:-1], -1)


def round_trip(x, dtype):
    """What the cache gives back for x [..., d]."""
    return values(*quantise(x, dtype), dtype)


def pack_block(kc, vc, kp, vp):
    """Bytes of one block of 16 tokens: K codes, K (s, z), V codes, V (s, z).
    kc, vc [16, d] codes; kp, vp [16, d / 32, 2] u16 bit patterns."""
    out = []
    for c, p in ((kc, kp), (vc, vp)):
        c = np.asarray(c, dtype=np.uint8)
        out.append((c[:, 0::2] | (c[:, 1::2] << 4)).reshape(-1))
        out.append(np.ascontiguousarray(p, dtype="<u2").view(np.uint8).reshape(-1))
    return np.concatenate(out)


def attention(q, k, v, lens, group, scale, q_lens=None):
    """q [tokens, heads * group, d]; k, v: one [len, heads, d] array a sequence
    (the cache's values).  Query i of a sequence's nq sees keys 0 .. len - nq + i."""
    q = np.asarray(q, dtype=F64)
    out = np.zeros_like(q)
    at = 0
    for b, ln in enumerate(lens):
        nq = 1 if q_lens is None else q_lens[b]
        for i in range(nq):
            m = ln - nq + i + 1
            if m > 0:
                for h in range(q.shape[1]):
                    kk, vv = k[b][:m, h // group].astype(F64), v[b][:m, h // group].astype(F64)
                    sc = kk @ q[at + i, h] * scale
                    p = np.exp(sc - sc.max())
                    out[at + i, h] = p @ vv / p.sum()
        at += nq
    return out


def gated(x, nibbles, rungs, tab, bias=None, act="silu"):
    """act(x Wg^T + bg) * (x Wu^T + bu): the gate's rows come first."""
    y = linear(x, nibbles, rungs, tab, bias)
    half = y.shape[1] // 2
    with np.errstate(all="ignore"):
        return activate(y[:, :half], act) * y[:, half:]


def angles(positions, turns):
    """Radians [tokens, pairs] of positions times turns (2^64ths of a turn a
    position), modulo one turn: exact in whole numbers but for the last step."""
    return np.array([[2 * math.pi * ((int(p) * int(t)) % 2 ** 64) / 2 ** 64 for t in turns] for p in positions])


def rotary(x, angle, layout="half", gain=1.0):
    """x [tokens, heads, dim] turned by angle [tokens, pairs]."""
    y = np.array(x, dtype=F64)
    n = angle.shape[1]
    i, j = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    a, b = y[..., i].copy(), y[..., j].copy()
    c, s = gain * np.cos(angle)[:, None], gain * np.sin(angle)[:, None]
    with np.errstate(all="ignore"):
        y[..., i], y[..., j] = a * c - b * s, b * c + a * s
    return y


def log_sums(q, k, lens, group, scale, q_lens=None):
    """Logarithm of each row's sum of exp(score), as `attention` sees its keys;
    -inf where a row sees none."""
    q = np.asarray(q, dtype=F64)
    out = np.full(q.shape[:2], -np.inf)
    at = 0
    for b, ln in enumerate(lens):
        nq = 1 if q_lens is None else q_lens[b]
        for i in range(nq):
            m = ln - nq + i + 1
            if m > 0:
                for h in range(q.shape[1]):
                    sc = k[b][:m, h // group].astype(F64) @ q[at + i, h] * scale
                    out[at + i, h] = sc.max() + math.log(np.exp(sc - sc.max()).sum())
        at += nq
    return out


def attention_weights(q, k, lens, group, scale, lse, q_lens=None):
    """One array [heads, len] a sequence: the sum of exp(score - lse) over the
    rows that see a token."""
    q = np.asarray(q, dtype=F64)
    out, at = [], 0
    for b, ln in enumerate(lens):
        nq = 1 if q_lens is None else q_lens[b]
        w = np.zeros((q.shape[1] // group, ln))
        for i in range(nq):
            m = ln - nq + i + 1
            if m > 0:
                for h in range(q.shape[1]):
                    w[h // group, :m] += np.exp(k[b][:m, h // group].astype(F64) @ q[at + i, h] * scale - lse[at + i, h])
        out.append(w)
        at += nq
    return out


def kept(weights, length, keep, recent):
    """Places of one head that stay, in order: the last min(recent, keep) and the
    heaviest of the others, equal ones the earlier first, a NaN the lightest."""
    if length <= keep:
        return list(range(length))
    old = length - min(recent, keep)
    w = np.asarray(weights, dtype=F64)[:old]
    order = sorted(range(old), key=lambda t: (0 if np.isnan(w[t]) else -1, 0.0 if np.isnan(w[t]) else -w[t], t))
    return sorted(order[:keep - (length - old)]) + list(range(old, length))
