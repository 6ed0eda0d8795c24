"""Layers with a channel scale (awq_quantize, rtn_quantize given one) in the operators on packed weights: the
codes are those of the scaled weight, so X is divided by the scale before the linear layer and dX after
the gradient.  The scale here is a power of two, so that those divisions are exact."""
import numpy as np
import pytest
import torch

from post_weight_quantization_16_b200 import gptq as G
from tests import packed_helpers as H

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.mark.parametrize("T,dtype", [(3, torch.float16), (40, torch.bfloat16), (300, torch.float16)])
@pytest.mark.parametrize("how", ["awq", "rtn"])
def test_linear_and_gradient_of_a_scaled_layer(T, dtype, how):
    m, n, bits, g = 192, 256, 4, 64
    gen = torch.Generator(device=DEV)
    gen.manual_seed(T)
    cal = torch.randn(512, n, generator=gen, device=DEV)
    cal[:, ::16] *= 10
    W = (torch.randn(m, n, generator=gen, device=DEV) * 0.05).half()
    q = G.awq_quantize(cal.bfloat16(), W, 2.0, bits, g)
    if how == "rtn":
        q = G.rtn_quantize(W, bits, g, sym=False, channel_scale=q["channel_scale"])
    cs = q["channel_scale"]
    assert (cs == 2).any() and (cs == 1).any()
    layer = (q["codes"], q["scales"], q["zeros"], None, bits, g)
    X = torch.randn(T, n, generator=gen, device=DEV).to(dtype)
    w, x = H.to64(q["w_hat"]), H.to64(X)
    y = G.dequant_linear((X / cs.to(dtype)).contiguous(), *layer, out_dtype=torch.float32)
    # w_hat is fp32 (two roundings): 2^-23 of every product beside the product's own bound
    tol = H.product_tol(x, w) + 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)
    want = x @ w.T
    assert (np.abs(H.to64(y) - want) <= tol + 2.0 ** -24 * np.abs(want)).all()
    dY = torch.randn(T, m, generator=gen, device=DEV).to(dtype)
    dX = H.to64(G.dequant_linear_backward(dY, *layer) / cs.to(dtype))
    dy = H.to64(dY)
    dx = dy @ w
    # weights with 11 bits, dX rounded to its type
    tol = (2.0 ** -11 + 2.0 ** -17) * (np.abs(dy) @ np.abs(w)) + H.EPS[dtype] * np.abs(dx) + H.TINY[dtype]
    assert (np.abs(dX - dx) <= tol).all()
    with pytest.raises(ValueError, match="channel_scale"):
        G.stack_experts([q], [q], [q])
