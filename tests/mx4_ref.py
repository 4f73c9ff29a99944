"""MX FP4 from its definition, in 64 bits on the CPU (numpy): the reference
of the MX4 tests.  Shares nothing with the library."""
import numpy as np

MAG = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
VALUES = np.concatenate([MAG, -MAG])


def blocks(K):
    return -(-K // 32)


def quantize(x):
    """float64 [R, K] -> (data uint8 [R, 16 B], scales uint8 [R, B])."""
    R, K = x.shape
    B = blocks(K)
    p = np.zeros((R, B * 32))
    p[:, :K] = x
    p = p.reshape(R, B, 32)
    bad = ~np.isfinite(p).all(axis=2)
    p = np.where(bad[:, :, None], 0.0, p)
    m = np.abs(p).max(axis=2)
    e = np.full((R, B), -127)
    nz = m > 0
    e[nz] = np.maximum(np.frexp(m[nz])[1] - 1 - 2, -127)
    y = np.abs(p) / np.exp2(e.astype(np.float64))[:, :, None]
    # the nearest magnitude, an exact tie to the even code
    d = np.abs(y[..., None] - MAG)
    best = d.min(axis=-1, keepdims=True)
    tied = d == best
    code = np.argmax(tied, axis=-1)
    second = 7 - np.argmax(tied[..., ::-1], axis=-1)
    code = np.where((second != code) & (code % 2 == 1), second, code)
    code = code + 8 * np.signbit(p)
    code = np.where(bad[:, :, None], 0, code).reshape(R, B * 32).astype(np.uint8)
    scales = np.where(bad, 255, e + 127).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), scales


def values(data, scales, K):
    """float64 [R, K] of an MX4 matrix (NaN in blocks of scale 255)."""
    codes = np.empty((data.shape[0], 2 * data.shape[1]), dtype=np.uint8)
    codes[:, 0::2] = data & 15
    codes[:, 1::2] = data >> 4
    s = np.exp2(scales.astype(np.float64) - 127)
    s[scales == 255] = np.nan
    return (VALUES[codes] * np.repeat(s, 32, axis=1))[:, :K]


def random_codes(rng, R, K, lo=118, hi=132):
    """A random MX4 matrix: codes of every kind, scales lo .. hi, garbage past
    K in the last block."""
    B = blocks(K)
    return (rng.integers(0, 256, (R, 16 * B), dtype=np.uint8),
            rng.integers(lo, hi + 1, (R, B), dtype=np.uint8))


def half_step(dtype_eps, ref, tiny):
    """Half a step of the output format at each reference value: eps/2
    relative, and half the least subnormal."""
    return np.abs(ref) * (dtype_eps / 2) + tiny / 2


def product_tolerance(ref, absum, terms, eps, tiny):
    """|C - ref| of a product summed in fp32 and rounded once.  `terms` fp32
    additions in any order are off by at most terms * 2^-23 times the sum of
    the magnitudes (2^-23: a whole step each, whatever the matrix core's own
    rounding is), and the rounding of the sum by half a step of the output."""
    fp32 = terms * 2.0 ** -23 * absum
    return fp32 + half_step(eps, np.abs(ref) + fp32, tiny)
