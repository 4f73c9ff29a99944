"""A mixture-of-experts layer from its definition, in 64 bits on the CPU, with
a bound on what fp32 sums and the output's rounding may add."""
import math

import numpy as np

U = 2.0 ** -23     # a whole fp32 step: whatever the matrix core's own rounding is


def choose(logits, k):
    """The k largest logits: NaN before all, ties to the lower index, -inf
    never."""
    def key(e):
        v = logits[e]
        return (0 if math.isnan(v) else 1, 0.0 if math.isnan(v) else -v, e)
    return [e for e in sorted(range(len(logits)), key=key)[:k] if logits[e] != -math.inf]


def layer(x, logits, up, down, k, renormalize, eps, tiny):
    """(y, tolerance), float64 [T, H].  x [T, H], logits [T, E], up [E, 2I, H],
    down [E, H, I], all float64; eps and tiny of the output format."""
    T, H = x.shape
    E, _, I = down.shape
    y, tol = np.zeros((T, H)), np.zeros((T, H))
    absy = np.zeros((T, H))
    for t in range(T):
        chosen = choose(logits[t], k)
        pool = chosen if renormalize else range(E)
        m = max(logits[t][list(pool)], default=0.0)
        total = sum(math.exp(logits[t][j] - m) for j in pool)
        for e in chosen:
            p = math.exp(logits[t][e] - m) / total
            z, absz = up[e] @ x[t], np.abs(up[e]) @ np.abs(x[t])
            dz = (H + 8) * U * absz
            g, u, dg, du = z[:I], z[I:], dz[:I], dz[I:]
            s = g / (1 + np.exp(-g))
            a = s * u
            # silu' stays below 1.1; the value is carried to 2^-16 (two
            # bfloat16 parts: 2^-9 of 2^-9 and some, or two binary16 parts, whose
            # least step is 2^-24)
            da = 1.1 * dg * np.abs(u) + np.abs(s) * du + 1.1 * dg * du + 2.0 ** -16 * np.abs(a) + 2.0 ** -24
            # p: exponentials and a sum of E terms, a few fp32 steps each, and
            # the exponent's own rounding
            dp = p * U * (E + 16 + abs(logits[t][e] - m))
            mag = np.abs(down[e]) @ (np.abs(a) + da)
            y[t] += p * (down[e] @ a)
            absy[t] += p * mag
            tol[t] += p * (np.abs(down[e]) @ da) + dp * mag
    tol += (k * I + k + 16) * U * absy
    return y, tol + (np.abs(y) + tol) * (eps / 2) + tiny / 2
