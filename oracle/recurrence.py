"""The gated linear recurrence, 8-bit checkpoints and the gated norm's gradients from their
definitions, in 64 bits on the CPU, row by row.  Shares no code with the CUDA library.

The bounds beside the results say how far FP32 arithmetic may be off.  A decay is off by
at most 2 units in the last place (2^-22), and every step of a chain adds a rounding of its product and
one of its sum (2^-24 each): below 2^-21 a step, relative to the chain of absolute values.
With E the recurrence of |x| and N the sum of E along the chain (N_t = a N_{t-1} + E_t), h_t is
therefore within 2^-21 N_t; the gradients likewise.  Below 2^-126 the two units of a decay, or of
1 - a, are 2^-148 whatever its size, and products that fall there are rounded to a multiple of 2^-149:
TINY e stands for that beside the relative part, e being what the decay multiplies.

16-bit arguments of the sigmoid take a faster exponential (coarse, the largest |g|): the product |g| log2(e) is
rounded (|g| 2^-24 of z = exp(-g)), the power of two is within 2^-22, and a = 1 / (1 + z) and z a are
off by no more than z is and 2^-22: |g| 2^-24 + 2^-21 a step in all.  1 - a is then 0 below 2^-126, and a at
least 2^-126."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -21
TINY = 2.0 ** -147 / U


def _scale(coarse):
    """The bounds' factor and the least size of a decay, in units of U, for arguments up to `coarse`."""
    return (1.0, TINY) if not coarse else (1 + coarse * 2.0 ** -24 / U, 2.0 ** -125 / U)


CHUNK, BLOCK = 64, 32


def decays(g, gate):
    """a and 1 - a."""
    if gate == "log":
        return np.exp(g), -np.expm1(g)
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-g)), 1 / (1 + np.exp(g))


def scan(x, g, spans, starts, gate, complement, coarse=0):
    """x, g [rows, D]; spans: (first, end) rows of the sequences; starts [N, D].  Returns (y, final, chunk states, bounds of
    the three); rows of no sequence are NaN, as are the chunk states of such rows."""
    u, tiny = U * _scale(coarse)[0], _scale(coarse)[1]
    a, rest = decays(g, gate)
    b = rest * x if complement else x
    rows, D = x.shape
    y, yb = np.full((rows, D), np.nan), np.full((rows, D), np.nan)
    chunks, cb = np.full((-(-rows // CHUNK), D), np.nan), np.full((-(-rows // CHUNK), D), np.nan)
    final, fb = np.array(starts, np.float64), np.zeros((len(spans), D))
    for n, (first, end) in enumerate(spans):
        h, e, bound = np.array(starts[n], np.float64), np.abs(starts[n]).astype(np.float64), np.zeros(D)
        for t in range(first, end):
            if t % CHUNK == 0:
                chunks[t // CHUNK], cb[t // CHUNK] = h, u * bound
            h = a[t] * h + b[t]
            bound = a[t] * (bound + e) + np.abs(b[t]) + tiny * (e + np.abs(x[t]) + 1)
            e = a[t] * e + np.abs(b[t])
            y[t], yb[t] = h, u * bound
        final[n], fb[n] = h, u * bound
    return y, final, chunks, yb, fb, cb


def scan_backward(dy, x, g, chunks, spans, starts, dfinal, gate, complement, coarse=0):
    """Returns (dx, dg, dstarts) and their bounds; h before a row comes from chunks (every 64 rows) and starts."""
    u, tiny = U * _scale(coarse)[0], _scale(coarse)[1]
    a, rest = decays(g, gate)
    b, c = (rest * x, rest) if complement else (x, np.ones_like(x))
    out = [np.full(dy.shape, np.nan) for _ in range(4)]
    dx, dg, dxb, dgb = out
    ds, dsb = np.array(dfinal, np.float64), np.zeros(dfinal.shape)
    for n, (first, end) in enumerate(spans):
        before, size, off = {}, {}, {}
        for t in range(first, end):
            if t == first or t % CHUNK == 0:
                h = np.array(starts[n] if t == first else chunks[t // CHUNK], np.float64)
                e, bound = np.abs(h), np.zeros_like(h)
            before[t], size[t], off[t] = h, e, bound
            h = a[t] * h + b[t]
            bound = a[t] * (bound + e) + np.abs(b[t]) + tiny * (e + np.abs(x[t]) + 1)
            e = a[t] * e + np.abs(b[t])
        d, e, bound = np.array(dfinal[n], np.float64), np.abs(dfinal[n]).astype(np.float64), np.zeros_like(h if end > first else ds[n])
        for t in range(end - 1, first - 1, -1):
            d, e = dy[t] + d, np.abs(dy[t]) + e
            bound = bound + e
            m, ms, mo = before[t] - x[t] if complement else before[t], size[t] + (np.abs(x[t]) if complement else 0), off[t]
            k = a[t] * rest[t] if gate == "sigmoid" else a[t]
            dx[t], dxb[t] = c[t] * d, u * (c[t] * (bound + 2 * e) + tiny * (e + 1))
            # the product's factors are off by their own bounds, and it rounds five times
            dg[t], dgb[t] = d * m * k, u * (k * (bound * ms + e * mo + 4 * e * ms) + tiny * (e + 1) * (ms + 1))
            d, e, bound = a[t] * d, a[t] * e, a[t] * bound + a[t] * e + tiny * (e + 1)
        ds[n], dsb[n] = d, u * bound
    return dx, dg, ds, dxb, dgb, dsb


def checkpoint(x, largest=float(np.finfo(np.float32).max)):
    """Codes, exponent bytes and values of x [rows, dim] in 64 bits (finite or not); largest: that of x's type."""
    rows, dim = x.shape
    blocks = -(-dim // BLOCK)
    codes, exps, values = np.zeros((rows, dim), np.int8), np.zeros((rows, blocks), np.uint8), np.zeros((rows, dim))
    for r in range(rows):
        for b in range(blocks):
            part = x[r, b * BLOCK:(b + 1) * BLOCK]
            if not np.isfinite(part).all():
                exps[r, b], values[r, b * BLOCK:(b + 1) * BLOCK] = 255, np.nan
                continue
            top, e = np.max(np.abs(part)), -127
            while top > 127 * 2.0 ** e:
                e += 1
            k = np.rint(part / 2.0 ** e)
            k = np.where(np.abs(k) * 2.0 ** e > largest, np.trunc(part / 2.0 ** e), k)
            codes[r, b * BLOCK:(b + 1) * BLOCK], exps[r, b] = k, e + 127
            values[r, b * BLOCK:(b + 1) * BLOCK] = k * 2.0 ** e
    return codes, exps, values


def gated_norm_backward(dy, x, z, w, eps, activation):
    """dx, dz, dw of rows [rows, dim], and sums of absolute values that their errors are relative to."""
    r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    with np.errstate(over="ignore"):
        s, rest = 1 / (1 + np.exp(-z)), 1 / (1 + np.exp(z))
    act, slope = (s, s * rest) if activation == "sigmoid" else (z * s, s * (1 + z * rest))
    steep = s * rest if activation == "sigmoid" else s * (1 + np.abs(z) * rest)
    u, n = dy * w * act, x * r
    dx = r * (u - n * np.mean(u * n, -1, keepdims=True))
    dxs = r * (np.abs(u) + np.abs(n) * np.mean(np.abs(u * n), -1, keepdims=True))
    q = dy * act * n
    return dx, dy * n * w * slope, q.sum(0), dxs, np.abs(dy * n * w) * steep, np.abs(q).sum(0)
