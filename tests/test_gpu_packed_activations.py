"""The activations of the epilogues by themselves, in each of the linear layer's three kernels and in the
gradient's passes, over their whole range.

Each weight row has one weight, 1 times its scale, in the column where X holds the token's value, so that
Z[t][r] = fp32(x[t] * s[r]) to the bit, and Y is fp32.  SiLU: expf within 2 units (2^-22), the sum's
rounding, a division within 2 units, the product's rounding: below 2^-20 of the value.  GELU: the fit
(2^-22.9), its argument and polynomial (2^-21.5), two exponentials (2^-22 each) and products: below 2^-19.
Both: nothing below fp32's normal numbers counts."""
import numpy as np
import pytest
import torch
from scipy.special import expit, log_ndtr, ndtr

from oracle import gptq_oracle as O
from post_weight_quantization_16_b200 import gptq as G

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
KERNELS = [(12, 300), (100, 300), (256, 9473)]


def gelu64(z):
    return z * np.exp(log_ndtr(z))


def silu64(z):
    return z * expit(z)


def layer(m, n, scale):
    """Weight 1 times scale[r] in column 0 of row r; the other columns of X are zero."""
    codes = np.full((m, n), 5)
    codes[:, 0] = 4
    z = torch.full((m, 1), 3.0, device=DEV)
    return torch.from_numpy(O.pack_codes(codes, 4).view(np.int32)).to(DEV), torch.from_numpy(scale).to(DEV).view(m, 1), z


@pytest.mark.parametrize("T,m", KERNELS)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_forward(T, m, dtype, act):
    rng = np.random.default_rng(T)
    n, limit = 128, 80.0 if act == "silu" else 12.5
    x = np.concatenate([np.linspace(-1, 1, T - T // 2), rng.uniform(-1, 1, T // 2) ** 5])
    X = torch.zeros(T, n, dtype=dtype, device=DEV)
    X[:, 0] = torch.from_numpy(x).to(DEV).to(dtype)
    s = (rng.uniform(0.01, 1, m) * limit).astype(np.float32)
    Z = X[:, 0].double().cpu().numpy()[:, None] * s.astype(np.float64)
    Z = Z.astype(np.float32).astype(np.float64)
    got = G.dequant_linear(X, *layer(m, n, s), None, 4, -1, act=G.ACT_SILU if act == "silu" else G.ACT_GELU,
                           out_dtype=torch.float32).double().cpu().numpy()
    want, rel = (silu64(Z), 2.0 ** -20) if act == "silu" else (gelu64(Z), 2.0 ** -19)
    assert np.abs(Z).max() > 0.9 * limit
    d = np.abs(got - want)
    assert (d <= rel * np.abs(want) + 2.0 ** -126).all(), np.log2((d / (np.abs(want) + 1e-37)).max())


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_the_kernels_agree_to_the_bit(act):
    """The same Z in the kernels for few and for many tokens: one form of the activation."""
    n, k = 128, G.ACT_SILU if act == "silu" else G.ACT_GELU
    rng = np.random.default_rng(1)
    s = (rng.uniform(0.01, 1, 9473) * 20).astype(np.float32)
    w = layer(9473, n, s)
    X = torch.zeros(256, n, dtype=torch.float16, device=DEV)
    X[:, 0] = torch.from_numpy(rng.uniform(-1, 1, 256)).to(DEV).half()
    y = G.dequant_linear(X, *w, None, 4, -1, act=k, out_dtype=torch.float32)
    for T in (3, 16, 100):
        assert torch.equal(G.dequant_linear(X[:T], *w, None, 4, -1, act=k, out_dtype=torch.float32), y[:T])


def test_ends_of_the_range():
    """Large and infinite Z: 0 and z, as the formulas' limits but for -infinity, which is a NaN there too."""
    n = 128
    big = torch.tensor([30000.0, -30000.0, 300.0, -300.0, 0.0, -0.0, 25.0, -25.0], device=DEV)
    for T, m in KERNELS:
        X = torch.zeros(T, n, dtype=torch.float16, device=DEV)
        X[:, 0] = big.half().repeat(-(-T // 8))[:T]
        w = layer(m, n, np.ones(m, dtype=np.float32))
        z = X[:, :1].float()
        for k in (G.ACT_SILU, G.ACT_GELU):
            y = G.dequant_linear(X, *w, None, 4, -1, act=k, out_dtype=torch.float32)
            assert ((y - z.clamp(min=0)).abs() <= 25.0 * np.exp(-25.0) * 1.001).all()
            far = z[:, 0].abs() > 100
            assert torch.equal(y[far], z.clamp(min=0).expand(-1, m)[far])


def test_the_largest_values_and_infinity():
    """bf16 holds 3e38: 0 and z again; +infinity stays, -infinity times 0 is a NaN in the formulas too."""
    n = 128
    big = torch.tensor([3e38, -3e38, 1e20, -1e20, 95.0, -95.0, float("inf"), float("-inf")], device=DEV)
    for T, m in KERNELS:
        X = torch.zeros(T, n, dtype=torch.bfloat16, device=DEV)
        X[:, 0] = big.bfloat16().repeat(-(-T // 8))[:T]
        codes, scale, zeros = layer(m, n, np.ones(m, dtype=np.float32))
        codes = torch.full_like(codes, 0x33333333)              # the other weights are 0: 0 times infinity nowhere
        codes[:, 0] += 1
        for k in (G.ACT_SILU, G.ACT_GELU):
            y = G.dequant_linear(X, codes, scale, zeros, None, 4, -1, act=k, out_dtype=torch.float32)
            z = X[:, :1].float().expand(-1, m)
            low = z == float("-inf")
            assert y[low].isnan().all() and torch.equal(y[~low], z[~low].clamp(min=0))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradient_by_the_bias_sum(dtype, act):
    """dbias of one token with dY = 1 is act'(Z) itself, in fp32: off by less than 2^-20 of its largest value,
    1.13, and, where it is a single product far from its zero, by 2^-18 of itself."""
    m, n = 8192, 128
    w = layer(m, n, np.ones(m, dtype=np.float32))
    z = np.concatenate([np.linspace(-60, 60, m // 2), np.linspace(-4, 4, m // 2)])
    Z = torch.from_numpy(z).to(DEV).to(dtype)[None].contiguous()
    one = torch.ones_like(Z)
    k = G.ACT_SILU if act == "silu" else G.ACT_GELU
    got = G.dequant_linear_backward(one, *w, None, 4, -1, act=k, preact=Z, want_dx=False, want_dbias=True)[1]
    got, z = got.double().cpu().numpy(), Z.double().cpu().numpy()[0]
    if act == "silu":
        want = expit(z) * (1 + z * expit(-z))
        far = z < -2
    else:
        want = ndtr(z) + z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
        far = (z < -2) & (z > -12.5)
    d = np.abs(got - want)
    assert (d <= 1.13 * 2.0 ** -20).all(), np.log2(d.max())
    assert (d[far] <= 2.0 ** -18 * np.abs(want[far])).all(), np.log2((d[far] / np.abs(want[far])).max())
