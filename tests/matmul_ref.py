"""Inputs and float64 references of the NVFP4 matrix products' tests."""
import math

import numpy as np

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6], np.float64)
E2M1 = np.concatenate([E2M1, -E2M1])
_b = np.arange(256)
_e, _m = (_b >> 3) & 15, _b & 7
E4M3 = np.where(_e == 0, _m * 2.0 ** -9, (1 + _m / 8) * 2.0 ** (_e - 7.0))

ACTS = ("none", "gelu", "silu")


def random_matrix(rng, lead, R, C, tiles, spread=3):
    """Random codes (all 16), block scales around 1 (with zeros) and tensor
    scales: dict of codes [lead, R, C/2], scales, s [lead or 1]."""
    srows = R // 16 if tiles else R
    codes = rng.integers(0, 256, lead + (R, C // 2), dtype=np.uint8)
    e = rng.integers(7 - spread, 7 + spread, lead + (srows, C // 16))
    sb = (e * 8 + rng.integers(0, 8, e.shape)).astype(np.uint8)
    sb[rng.random(sb.shape) < 0.05] = 0
    sb[rng.random(sb.shape) < 0.02] = 3                    # subnormal scale
    s = (rng.uniform(0.5, 1.0, lead or (1,)) / (8.0 * math.sqrt(C) ** 0.5)).astype(np.float32)
    return dict(codes=codes, scales=sb, s=s, tiles=tiles)


def decode(m, e=None):
    """float64 values of matrix m (expert e)."""
    codes, sb, s = (m["codes"], m["scales"], m["s"][0]) if e is None else \
        (m["codes"][e], m["scales"][e], m["s"][e])
    v = np.empty((codes.shape[0], 2 * codes.shape[1]))
    v[:, 0::2], v[:, 1::2] = E2M1[codes & 15], E2M1[codes >> 4]
    b = np.repeat(E4M3[sb], 16, axis=1)
    if m["tiles"]:
        b = np.repeat(b, 16, axis=0)
    return v * b * np.float64(s)


def act64(z, act):
    if act == "gelu":
        return 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z / (1 + np.exp(-z))
    return z


def reference(x, w, bias, act, gate, residual):
    """(Y, bound on |Y|'s ingredients) in float64: the second is what the fp32
    steps' errors scale with, sum_k |x w| + |bias| through the gate, plus
    |residual|."""
    z, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    if bias is not None:
        z, mag = z + bias, mag + np.abs(bias)
    y = act64(z, act)
    if gate is not None:
        y, mag = y * gate, mag * np.abs(gate)
    if residual is not None:
        y, mag = y + residual, mag + np.abs(residual)
    return y, mag


def tolerance(y, mag, K, bf16):
    """Allowed |error| for each value.  The tensor core adds the K / 16 block
    products of a sum in fp32 in an order of its own, each addition off by at
    most one fp32 step (2^-23, truncation) of a partial sum that sum |x w|
    bounds; the epilogue has at most 16 more fp32 steps (scale, bias, the
    activation's exponential and quotient at 2 ulp each, whose slopes are below
    1.13, gate, residual) of values mag bounds.  A bf16 result is off by half a
    bf16 step of the value on top."""
    t = mag * (K / 16 + 32) * 2.0 ** -23
    return t + (np.abs(y) + t) * 2.0 ** -8 if bf16 else t
