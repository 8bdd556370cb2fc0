"""fp64 reference of the AdamW step whose moments are held in 8 bits.

TEST INFRASTRUCTURE ONLY.  Written from the definitions: a moment is a value of a small
floating-point type (e4m3 or e5m2) times a power of two per block of 64 elements; after the step
each value goes to one of its two neighbours in that type, upwards with the probability of its
place between them.  The random bits are Murmur3's finalizer of the element's number and a key.
"""
from __future__ import annotations

import numpy as np

from .adamw import adamw_step

BLOCK = 64
# mantissa bits, lowest normal exponent, exponent of a block's largest value
E4M3, E5M2 = (3, -6, 7), (2, -14, 14)


def _mix(x):
    x = np.asarray(x, dtype=np.uint32)
    x = (x ^ (x >> np.uint32(16))) * np.uint32(0x85EBCA6B)
    x = (x ^ (x >> np.uint32(13))) * np.uint32(0xC2B2AE35)
    return x ^ (x >> np.uint32(16))


def fractions(first, n, seed, step):
    """The two fractions in [0, 1) of elements first .. first + n - 1."""
    with np.errstate(over="ignore"):
        key = _mix(_mix(_mix(seed & 0xFFFFFFFF) ^ np.uint32((seed >> 32) & 0xFFFFFFFF)) ^ np.uint32(step & 0xFFFFFFFF))
        at = np.arange(first, first + n, dtype=np.uint64)
        low, high = (at & np.uint64(0xFFFFFFFF)).astype(np.uint32), (at >> np.uint64(32)).astype(np.uint32)
        bits = _mix((low * np.uint32(0x9E3779B1)) ^ (key + high * np.uint32(0x9E3779B1)))
    return (bits & np.uint32(0xFFFF)) / 65536.0, (bits >> np.uint32(16)) / 65536.0


def blocks(x):
    """x flattened into rows of BLOCK, zeros behind its end."""
    x = np.asarray(x, dtype=np.float64).reshape(-1)
    out = np.zeros((-(-x.size // BLOCK), BLOCK))
    out.reshape(-1)[:x.size] = x
    return out


def widen(values, scale_bytes):
    """What 8-bit values (as floats) and their blocks' scale bytes stand for."""
    values = np.asarray(values, dtype=np.float64)
    scale = np.exp2(np.asarray(scale_bytes, dtype=np.float64) - 127.0)
    return (blocks(values) * scale[:, None]).reshape(-1)[:values.size].reshape(values.shape)


def exponents(x, kind):
    """The scale's exponent of each block of a moment x."""
    big = np.abs(blocks(x))
    big = np.where(np.isfinite(big), big, 0.0).max(1)
    e = np.frexp(big)[1] - 1 - kind[2]
    return np.clip(np.where(big > 0, e, -126), -126, 127)


def places(x, e, kind):
    """(multiples of the grid's distance, that distance) of each element of x in units of its
    block's scale 2^e: a value between the grid's points k and k + 1 has a place in [k, k + 1)."""
    y = blocks(x) * np.exp2(-np.asarray(e, dtype=np.float64))[:, None]
    unit = np.exp2(np.maximum(np.frexp(np.abs(y))[1] - 1, kind[1]) - float(kind[0]))
    size = np.asarray(x).size
    return (y / unit).reshape(-1)[:size], unit.reshape(-1)[:size]


def step(param, grad, exp_avg, exp_avg_sq, **hp):
    """(param, exp_avg, exp_avg_sq) in 64 bits, the moments before they are rounded."""
    r = adamw_step(param, grad, exp_avg, exp_avg_sq, **hp)
    return r.param, r.exp_avg, r.exp_avg_sq
