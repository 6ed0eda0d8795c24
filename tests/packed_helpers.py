"""Plain 64-bit forms of the operators on packed layers, for the tests: numpy, from the definitions."""
from __future__ import annotations

import numpy as np
import torch

from oracle import gptq_oracle as O

ACTS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}
EPS = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}  # half the smallest step


def random_layer(rng, m, n, bits, g, s0=0.02):
    """codes (ints), packed words, scales, zeros of a random packed layer."""
    gw = n if g == -1 else g
    codes = rng.integers(0, 1 << bits, (m, n))
    s = (rng.uniform(0.5, 1.5, (m, n // gw)) * s0 / (1 << bits)).astype(np.float32)
    z = rng.integers(0, 1 << bits, (m, n // gw)).astype(np.float32)
    return codes, O.pack_codes(codes, bits), s, z


def weights64(codes, s, z):
    """(u - z) s in 64 bits, sweep order."""
    g = codes.shape[1] // s.shape[1]
    return (codes - np.repeat(z.astype(np.float64), g, 1)) * np.repeat(s.astype(np.float64), g, 1)


def act64(z, name):
    from math import sqrt

    from scipy.special import erf
    if name == "relu":
        return np.where(z > 0, z, 0.0)
    if name == "gelu":
        return 0.5 * z * (1 + erf(z / sqrt(2)))
    if name == "silu":
        return z / (1 + np.exp(-z))
    return z


def act_grad64(z, name):
    from math import pi, sqrt

    from scipy.special import erf
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "gelu":
        return 0.5 * (1 + erf(z / sqrt(2))) + z * np.exp(-z * z / 2) / sqrt(2 * pi)
    if name == "silu":
        s = 1 / (1 + np.exp(-z))
        return s * (1 + z * (1 - s))
    return np.ones_like(z)


def product_tol(x, w):
    """Bound of a product's error: products of 16-bit values are exact in fp32; at most one rounding
    of 2^-23 of the running sum per 16 terms, the group sums' scaling and addition one each."""
    k = x.shape[1]
    return (k / 16 + 2 * (k / 32) + 8) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T) + 1e-30


def to64(t):
    return t.detach().to(torch.float64).cpu().numpy()
