"""The operators on packed weights over the range of values that their types hold: outliers that an
activation masks, infinities, layers of very small and very large scales."""
import numpy as np
import pytest
import torch

from post_weight_quantization_16_b200 import gptq as G
from tests import packed_helpers as H
from tests.test_gpu_packed_linear import DEV, Case

pytestmark = pytest.mark.gpu
KERNELS = [(20, 256), (300, 9472)]                    # tokens and columns of the single-block and of the pair kernel


def gradient_close(c, got, dY, Z, dtype):
    """dX against the 64-bit formula with the exact weights: every product of dz and a weight is off by at
    most 2^-11 for each of them (2^-10 and the product of the two), a value of dz by 2^-25 of 2^13 times less
    than the token's largest |dz| where it is that small, the sum by its accumulation, dX by its rounding."""
    dz = H.to64(dY) * H.act_grad64(H.to64(Z), c.act)
    W = np.zeros_like(c.W)
    W[:, c.perm_np] = c.W
    want = dz @ W
    tol = (2.0 ** -10 + 2.0 ** -21) * (np.abs(dz) @ np.abs(W)) + H.product_tol(dz, W.T)
    tol += np.abs(dz).max(1, keepdims=True) * 2.0 ** (-13 - 25) * np.abs(W).sum(0)
    # (act' itself is good to 2^-19 of its largest value, 1.13)
    if c.act != "relu":
        tol += 2.0 ** -19 * 1.13 * (np.abs(np.where(np.abs(H.to64(Z)) > 50, 0, H.to64(dY))) @ np.abs(W))
    tol += H.EPS[dtype] * (np.abs(want) + tol) + H.TINY[dtype]
    d = np.abs(H.to64(got) - want)
    assert (d <= tol).all(), float((d / tol).max())
    # the tolerance says something: it is far below the values
    assert np.median(tol / np.abs(want).clip(1e-300)) < 0.1


@pytest.mark.parametrize("T,n", KERNELS)
@pytest.mark.parametrize("act,dtype,outlier", [("relu", "bf16", 2.0 ** 100), ("silu", "bf16", 2.0 ** 60), ("gelu", "bf16", 2.0 ** 60),
                                               ("silu", "fp16", 60000.0)])
def test_an_outlier_that_the_activation_masks(T, n, act, dtype, outlier):
    """A few large dY where act' is zero (or 1e-300): the rest of the token keeps its bits."""
    c = Case(T, 200, n, 4, 128, dtype, act, True)
    dY = torch.from_numpy(c.rng.normal(0, 1e-3, (T, 200))).to(DEV)
    Z = torch.from_numpy(c.rng.normal(0, 1, (T, 200))).to(DEV)
    at = c.rng.integers(0, 200, (T, 3))
    for j in range(3):
        dY[torch.arange(T), at[:, j]] = outlier * (-1.0) ** j
        Z[torch.arange(T), at[:, j]] = -700.0
    dY, Z = dY.to(c.dt), Z.to(c.dt)
    gradient_close(c, G.dequant_linear_backward(dY, *c.layer, act=H.ACTS[act], preact=Z), dY, Z, c.dt)


@pytest.mark.parametrize("T,n", KERNELS)
def test_a_token_with_one_infinity(T, n):
    """Its dX is that infinity times the sign of its row of W: the other values of the token, finite in bf16
    but above fp16's largest, must not become infinite beside it."""
    c = Case(T, 200, n, 4, 128, "bf16", "none", True)
    dY = torch.from_numpy(c.rng.normal(0, 1e7, (T, 200))).to(DEV).to(c.dt)
    r = int(np.argmin((c.W == 0).sum(1)))
    dY[:, r] = float("inf")
    got = H.to64(G.dequant_linear_backward(dY, *c.layer))[:, c.perm_np]
    keep = c.W[r] != 0
    assert keep.mean() > 0.8
    assert np.array_equal(got[:, keep], np.broadcast_to(np.sign(c.W[r][keep]) * np.inf, (T, keep.sum())))
