"""The linear layer on packed weights and its gradient (gptq_dequant_linear,
gptq_dequant_linear_backward) against plain 64-bit numpy.

Tolerances, element by element.  Forward: Z is off by at most product_tol (fp32 accumulation of exact
products) plus one fp32 rounding of the bias's addition; an activation's slope is at most 1.13 and its
own evaluation is good to 2^-19 of its value; then an addition of the residual in fp32 and the rounding
of the output (half a step).  Gradient: the operands are W16 = fp16((u - z) s) - the same fp16 values on
both sides - and dz, which is exact for fp16 without an activation, else rounded to fp16 (2^-11; to
2^-22 where it is split in two), below 2^-25 of the token's scale (at most the token's largest |dY| /
2^13); accumulation as above; then the rounding of the output."""
import numpy as np
import pytest
import torch

from oracle import gptq_oracle as O
from post_weight_quantization_16_b200 import gptq as G
from tests import packed_helpers as H

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


class Case:
    def __init__(self, T, m, n, bits, g, dtype, act="none", perm=True, seed=0, outliers=True):
        self.rng = rng = np.random.default_rng(seed * 7919 + T * 31 + m + n + bits)
        self.T, self.m, self.n, self.bits, self.g, self.act, self.dt = T, m, n, bits, g, act, DT[dtype]
        self.codes, packed, s, z = H.random_layer(rng, m, n, bits, g)
        self.perm_np = rng.permutation(n) if perm else np.arange(n)
        self.perm = torch.from_numpy(self.perm_np.astype(np.int32)).to(DEV) if perm else None
        self.layer = [torch.from_numpy(packed.view(np.int32)).to(DEV), torch.from_numpy(s).to(DEV),
                      torch.from_numpy(z).to(DEV), self.perm, bits, g]
        self.packed, self.s, self.z = packed, s, z
        self.W = H.weights64(self.codes, s, z)                      # sweep order
        x = rng.normal(0, 1, (T, n))
        if outliers:
            x[:, rng.choice(n, max(1, n // 100), replace=False)] *= 20
        self.X = self.dev(x)

    def dev(self, a):
        return torch.from_numpy(np.ascontiguousarray(a)).to(DEV).to(self.dt)

    def forward64(self, bias=None, residual=None, X=None):
        """(Y, its tolerance before the output's rounding, Z, its tolerance)"""
        x = H.to64(self.X if X is None else X)[:, self.perm_np]
        z = x @ self.W.T
        tol = H.product_tol(x, self.W)
        if bias is not None:
            z = z + H.to64(bias)
            tol = tol + 2.0 ** -23 * np.abs(z)
        y = H.act64(z, self.act)
        ty = 1.13 * tol + 2.0 ** -19 * np.abs(y)
        if residual is not None:
            y = y + H.to64(residual)
            ty = ty + 2.0 ** -23 * np.abs(y)
        return y, ty, z, tol


def close(got, want, tol, dtype):
    t = tol + H.EPS[dtype] * (np.abs(want) + tol) + H.TINY[dtype]
    d = np.abs(H.to64(got) - want)
    assert np.isfinite(H.to64(got)).all()
    assert (d <= t).all(), float((d / t).max())


FORWARD = [
    # T, m, n, bits, g, dtype, act, perm, bias, residual, fp32 out, preact
    (1, 1, 128, 4, 128, "fp16", "none", False, False, False, False, False),
    (1, 130, 512, 4, 128, "fp16", "none", True, True, True, False, True),
    (1, 300, 4096, 2, 32, "bf16", "silu", True, True, False, False, False),
    (2, 129, 1152, 3, 64, "fp16", "gelu", True, True, False, True, False),
    (3, 256, 768, 8, -1, "bf16", "relu", False, False, True, False, True),
    (5, 77, 640, 8, 32, "fp16", "gelu", False, True, False, True, False),
    (7, 65, 384, 3, 32, "bf16", "none", False, False, False, True, False),
    (8, 200, 2048, 4, 64, "fp16", "silu", False, True, True, False, False),
    (8, 128, 768, 4, 384, "bf16", "none", True, False, False, True, False),
    (9, 131, 1024, 2, 128, "bf16", "relu", True, True, True, False, True),
    (16, 1000, 512, 8, 64, "bf16", "none", True, False, True, False, False),
    (16, 64, 11008, 4, 128, "fp16", "silu", True, False, False, True, False),
    (17, 127, 256, 4, 32, "fp16", "gelu", True, True, True, False, True),
    (32, 129, 384, 3, 128, "bf16", "none", False, False, False, True, False),
    (33, 260, 1280, 8, 128, "fp16", "silu", True, True, False, False, False),
    (64, 255, 512, 2, 64, "bf16", "relu", True, False, True, False, True),
    (65, 384, 1024, 3, 64, "fp16", "none", True, True, False, True, False),
    (128, 100, 2048, 4, -1, "bf16", "gelu", False, True, True, False, False),
    (129, 300, 256, 8, 32, "fp16", "silu", True, True, True, False, True),
    (257, 2500, 384, 4, 128, "bf16", "silu", True, True, True, False, True),     # CTA pairs from here on
    (300, 9473, 256, 3, 32, "fp16", "gelu", False, True, False, True, False),
    (1030, 2570, 512, 2, 64, "bf16", "relu", True, False, True, False, False),
    (2048, 1290, 1152, 8, 128, "fp16", "none", True, True, True, False, True),
    (19, 130, 65536, 4, 128, "bf16", "none", True, False, False, False, False),       # rows too wide for pairs
    (1185, 128, 1024, 4, 64, "fp16", "none", True, False, False, False, False),        # an odd last row of a pair
    (700, 4101, 768, 4, 384, "fp16", "silu", False, True, False, True, False),
]


@pytest.mark.parametrize("T,m,n,bits,g,dtype,act,perm,bias,residual,f32,preact", FORWARD)
def test_linear(T, m, n, bits, g, dtype, act, perm, bias, residual, f32, preact):
    c = Case(T, m, n, bits, g, dtype, act, perm)
    b = c.dev(c.rng.normal(0, 1, m)) if bias else None
    r = c.dev(c.rng.normal(0, 1, (T, m))) if residual else None
    got = G.dequant_linear(c.X, *c.layer, bias=b, act=H.ACTS[act], residual=r,
                           out_dtype=torch.float32 if f32 else None, want_preact=preact)
    y, ty, z, tz = c.forward64(b, r)
    out = got[0] if preact else got
    assert out.dtype == (torch.float32 if f32 else c.dt)
    close(out, y, ty, out.dtype)
    if preact:
        close(got[1], z, tz, c.dt)


BACKWARD = [
    # T, m, n, bits, g, dtype, act, perm, dbias
    (1, 1, 128, 4, 128, "fp16", "none", False, True),
    (3, 130, 256, 2, 32, "bf16", "silu", True, True),
    (16, 7, 384, 3, 64, "fp16", "relu", True, True),
    (17, 200, 512, 8, 128, "bf16", "none", False, False),
    (33, 129, 1152, 4, 384, "fp16", "gelu", True, True),
    (64, 1000, 256, 8, 32, "fp16", "none", True, True),
    (100, 257, 640, 3, -1, "bf16", "gelu", False, True),
    (129, 384, 512, 4, 64, "fp16", "silu", True, False),
    (300, 131, 9472, 4, 128, "bf16", "silu", True, True),      # CTA pairs from here on
    (1100, 300, 2176, 2, 32, "fp16", "gelu", False, True),
    (2050, 100, 1280, 8, 64, "bf16", "none", True, True),
    (515, 264, 3200, 3, 128, "fp16", "none", False, False),
]


def grad64(c, dY, Z):
    dy = H.to64(dY)
    dz = dy * (H.act_grad64(H.to64(Z), c.act) if Z is not None else 1.0)
    W16 = O.dequantize_packed_fp16(c.packed, c.s, c.z, c.perm_np, c.n, c.bits, c.g).astype(np.float64)  # original order
    dx = dz @ W16
    biggest = np.abs(dy).max(1, keepdims=True)
    tol = H.product_tol(dz, W16.T)
    step = 0.0
    if c.dt == torch.bfloat16 or c.act != "none":
        step = 2.0 ** -22 if c.dt == torch.float16 and c.act in ("gelu", "silu") else 2.0 ** -11
        if c.dt == torch.bfloat16 and c.act == "none":
            step = 0.0                                          # bf16 values fit fp16 but for the smallest
    a = np.abs(dz) @ np.abs(W16)
    # (act' itself is good to 2^-19 of its largest value, 1.13)
    tol = tol + step * a + (2.0 ** -19 * 1.13 if c.act in ("gelu", "silu") else 0.0) * (np.abs(dy) @ np.abs(W16))
    tol = tol + biggest * 2.0 ** (-13 - 25) * np.abs(W16).sum(0)
    return dx, tol, dz


@pytest.mark.parametrize("T,m,n,bits,g,dtype,act,perm,dbias", BACKWARD)
def test_gradient(T, m, n, bits, g, dtype, act, perm, dbias):
    c = Case(T, m, n, bits, g, dtype, act, perm)
    dY = c.dev(c.rng.normal(0, 1, (T, m)) * 10.0 ** c.rng.uniform(-3, 1, (T, 1)))   # tokens of very different sizes
    Z = c.dev(c.rng.normal(0, 1.5, (T, m))) if act != "none" else None
    got = G.dequant_linear_backward(dY, *c.layer, act=H.ACTS[act], preact=Z, want_dbias=dbias)
    dx, tol, dz = grad64(c, dY, Z)
    out = got[0] if dbias else got
    assert out.dtype == c.dt
    close(out, dx, tol, c.dt)
    if dbias:
        b = got[1]
        assert b.dtype == torch.float32
        t = (T / 8 + 24) * 2.0 ** -24 * np.abs(dz).sum(0) + 2.0 ** -19 * 1.13 * np.abs(H.to64(dY)).sum(0) * (act != "none")
        assert (np.abs(H.to64(b) - dz.sum(0)) <= t + 1e-30).all()
        only = G.dequant_linear_backward(dY, *c.layer, act=H.ACTS[act], preact=Z, want_dx=False, want_dbias=True)
        assert only[0] is None and torch.equal(only[1], b)


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_gradient_against_differences_of_the_forward(act):
    """<dX, D> against (f(X + hD) - f(X - hD)) / 2h of f(X) = <dY, Y(X)> in 64 bits, for random D.  The
    weights' rounding to fp16 moves dX by at most 2^-11 of sum |dz W|; the difference's own error is
    below h^2 |f'''| / 6 and 2^-52 |f| / h."""
    c = Case(40, 96, 256, 4, 64, "fp16", act, True, outliers=False)
    dY = c.dev(c.rng.normal(0, 1, (40, 96)))
    z = H.to64(c.X)[:, c.perm_np] @ c.W.T
    Z = c.dev(z)
    dX = H.to64(G.dequant_linear_backward(dY, *c.layer, act=H.ACTS[act], preact=Z if act != "none" else None))
    dy, h = H.to64(dY), 1e-4
    f = lambda x: (dy * H.act64(x[:, c.perm_np] @ c.W.T, act)).sum()  # noqa: E731
    x0 = H.to64(c.X)
    W = np.zeros_like(c.W)
    W[:, c.perm_np] = c.W
    for k in range(3):
        D = c.rng.normal(0, 1, x0.shape)
        fd = (f(x0 + h * D) - f(x0 - h * D)) / (2 * h)
        # dX's, W16's, dz's rounding (2^-11 each, as if all fell on one operand: 4), and Z's times the
        # slope's change (|act''| < 1.2).  They are independent with mean near zero, so that their sum over
        # D.size products stays below 6 sqrt(D.size) of the mean one
        scale = np.abs(dy) * (1.13 + (1.2 * np.abs(z) if act != "none" else 0.0))
        tol = 4 * 2.0 ** -11 * (np.abs(D) * (scale @ np.abs(W))).sum() / np.sqrt(D.size) * 6 + 1e-6
        assert abs((dX * D).sum() - fd) <= tol, (k, (dX * D).sum(), fd, tol)


def test_strides_unaligned_outputs_and_residual_in_place():
    for T, m in ((5, 130), (40, 130), (600, 2500)):
        c = Case(T, m, 384, 4, 64, "fp16", "silu", True)
        wide = torch.zeros(T, 384 + 24, dtype=c.dt, device=DEV)
        wide[:, 8:392] = c.X
        x = wide[:, 8:392]
        res = torch.randn(T, m + 3, device=DEV).to(c.dt)[:, 1:m + 1]                 # odd offset and stride
        out = torch.full((T, m + 5), 7.0, dtype=c.dt, device=DEV)
        y = G.dequant_linear(x, *c.layer, act=G.ACT_SILU, residual=res, out=out[:, 3:m + 3])
        want, tol, *_ = c.forward64(None, res)
        close(y, want, tol, c.dt)
        assert (out[:, :3] == 7).all() and (out[:, m + 3:] == 7).all()               # nothing beside the rows
        buf = res.contiguous()
        y2 = G.dequant_linear(x, *c.layer, act=G.ACT_SILU, residual=buf, out=buf)    # in place
        assert y2 is buf and torch.equal(y2, y)
        dY = torch.randn(T, m + 3, device=DEV).to(c.dt)[:, 1:m + 1]
        Z = torch.randn(T, m, device=DEV).to(c.dt)
        dx = torch.full((T, 384 + 9), 7.0, dtype=c.dt, device=DEV)
        g = G.dequant_linear_backward(dY, *c.layer, act=G.ACT_SILU, preact=Z, out=dx[:, 5:389])
        a = G.dequant_linear_backward(dY.contiguous(), *c.layer, act=G.ACT_SILU, preact=Z)
        assert torch.equal(g, a) and (dx[:, :5] == 7).all() and (dx[:, 389:] == 7).all()
        none = Case(T, m, 384, 4, 64, "fp16", "none", False)
        g = G.dequant_linear_backward(dY, *none.layer)                               # copied: TMA cannot read it
        assert torch.equal(g, G.dequant_linear_backward(dY.contiguous(), *none.layer))


@pytest.mark.parametrize("T", [3, 40, 600])
def test_nan_and_infinity_stay_in_their_token(T):
    c = Case(T, 2500, 256, 4, 128, "bf16", "none", True)
    clean = G.dequant_linear(c.X, *c.layer)
    bad = c.X.clone()
    bad[1, 5], bad[2, 7] = float("nan"), float("inf")
    y = G.dequant_linear(bad, *c.layer)
    keep = [t for t in range(T) if t not in (1, 2)]
    assert torch.equal(y[keep], clean[keep]) and y[1].isnan().all() and not y[2].isfinite().any()
    dY = torch.randn(T, 2500, device=DEV).to(c.dt)
    g0 = G.dequant_linear_backward(dY, *c.layer)
    dY2 = dY.clone()
    dY2[1, 3], dY2[2, 9] = float("nan"), float("-inf")
    dY2[0] = 0
    g = G.dequant_linear_backward(dY2, *c.layer)
    keep = [t for t in range(3, T)]
    assert torch.equal(g[keep], g0[keep]) and g[1].isnan().all() and not g[2].isfinite().any() and (g[0] == 0).all()


def test_no_tokens_and_one_row():
    c = Case(4, 33, 256, 4, 64, "fp16", "none", True)
    y = G.dequant_linear(c.X[:0], *c.layer)
    assert y.shape == (0, 33)
    dx, db = G.dequant_linear_backward(y, *c.layer, want_dbias=True)
    assert dx.shape == (0, 256) and (db == 0).all()


@pytest.mark.parametrize("T", [1, 8, 40, 300])
def test_runs_agree_streams_and_graphs(T):
    """The same call again, on another stream, and captured and replayed on changed inputs, with two
    graphs alive, gives the same values."""
    c = Case(T, 2300, 512, 4, 128, "bf16", "silu", True)
    b = torch.randn(2300, device=DEV).to(c.dt)
    ref = G.dequant_linear(c.X, *c.layer, bias=b, act=3)
    for _ in range(5):
        assert torch.equal(G.dequant_linear(c.X, *c.layer, bias=b, act=3), ref)
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream(DEV))
    y = G.dequant_linear(c.X, *c.layer, bias=b, act=3, stream=side)
    side.synchronize()
    assert torch.equal(y, ref)
    x1, x2 = c.X.clone(), torch.zeros_like(c.X)
    graphs = []
    for x in (x1, x2):
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = G.dequant_linear(x, *c.layer, bias=b, act=3)
            dx, db = G.dequant_linear_backward(out, *c.layer, act=3, preact=out, want_dbias=True)
        graphs.append((g, out, dx, db))
    x2.copy_(c.X)
    for g, *_ in graphs:
        g.replay()
    torch.cuda.synchronize()
    eager = G.dequant_linear_backward(ref, *c.layer, act=3, preact=ref, want_dbias=True)
    for g, out, dx, db in graphs:
        assert torch.equal(out, ref) and torch.equal(dx, eager[0]) and torch.equal(db, eager[1])
    x1.mul_(0.5)
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1], G.dequant_linear(x1, *c.layer, bias=b, act=3)) and torch.equal(graphs[1][1], ref)


def test_callers_workspace_and_refusals_on_the_device():
    c = Case(12, 64, 256, 4, 64, "fp16", "none", True)
    need = G.lib().gptq_dequant_linear_workspace_bytes(12, 256, True)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    y = G.dequant_linear(c.X, *c.layer, workspace=ws)
    assert torch.equal(y, G.dequant_linear(c.X, *c.layer))
    assert G.lib().gptq_dequant_matmul_check(ws.data_ptr(), 0, None) == G.OK
    bad = [dict(workspace=ws[:-1]), dict(bias=torch.zeros(63, device=DEV).half()), dict(bias=torch.zeros(64, device=DEV)),
           dict(residual=torch.zeros(12, 64, device=DEV)), dict(out_dtype=torch.bfloat16),
           dict(out=torch.zeros(12, 63, device=DEV).half()), dict(out=torch.zeros(64, 12, device=DEV).half().t())]
    for kw in bad:
        with pytest.raises(ValueError):
            G.dequant_linear(c.X, *c.layer, **kw)
    for x in (c.X.float(), c.X[:, :128], c.X.t().contiguous().t(), c.X.cpu(),
              torch.zeros(12 * 257, device=DEV).half()[1:1 + 12 * 256].view(12, 256)):
        with pytest.raises(ValueError):
            G.dequant_linear(x, *c.layer)
    with pytest.raises(G.GPTQError):
        G.dequant_linear(c.X, *c.layer, act=7)
    with pytest.raises(ValueError):
        G.dequant_linear_backward(torch.zeros(12, 64, device=DEV).half(), *c.layer, act=3)          # no preact
    with pytest.raises(ValueError):
        G.dequant_linear_backward(torch.zeros(12, 64, device=DEV).half(), *c.layer, want_dx=False)


def test_tiny_and_huge_gradients():
    """Tokens of a bf16 dY scaled by powers of two give the same dX, scaled: dz is scaled per token."""
    for T, m in ((20, 200), (300, 200)):
        c = Case(T, m, 9472, 4, 128, "bf16", "none", True)
        dY = torch.randn(T, m, device=DEV).to(c.dt)
        e = torch.from_numpy(c.rng.integers(-110, 118, T)).to(DEV)
        e[0], e[1] = -110, 117
        base = G.dequant_linear_backward(dY, *c.layer).double()
        got = G.dequant_linear_backward(torch.ldexp(dY.double(), e[:, None]).to(c.dt), *c.layer).double()
        want = torch.ldexp(base, e[:, None])
        normal = (want.abs() >= 2.0 ** -120) | (want == 0)      # below, fewer bits are left
        assert torch.equal(got[normal], want[normal]) and normal.float().mean() > 0.9


def test_offsets_past_32_bits():
    """Strides and row counts whose element offsets exceed 2^31: the last rows are checked."""
    big = torch.empty((5 << 30) // 2, dtype=torch.float16, device=DEV)
    for T in (8, 9, 300):
        c = Case(T, 2304, 256, 4, 128, "fp16", "none", True)
        ld = (big.numel() // T - 4096) // 8 * 8
        assert (T - 1) * ld > 1 << 31
        view = lambda at, cols: torch.as_strided(big, (T, cols), (ld, 1), at)  # noqa: E731
        x, res, out, dx = view(0, 256), view(256, 2304), view(256, 2304), view(2816, 256)
        x.copy_(c.X)
        r = torch.randn(T, 2304, device=DEV).half()
        res.copy_(r)
        G.dequant_linear(x, *c.layer, residual=res, out=out)
        assert torch.equal(out, G.dequant_linear(c.X, *c.layer, residual=r))
        G.dequant_linear_backward(out, *c.layer, out=dx)
        assert torch.equal(dx, G.dequant_linear_backward(out.contiguous(), *c.layer))
    del big, x, res, out, dx
    T, m = 33000, 65600
    c = Case(64, m, 128, 4, 128, "fp16", "silu", True, outliers=False)
    X = torch.zeros(T, 128, dtype=c.dt, device=DEV)
    X[-64:] = c.X
    y, z = G.dequant_linear(X, *c.layer, act=G.ACT_SILU, want_preact=True)
    want, tol, wz, tz = c.forward64()
    close(y[-64:], want, tol, c.dt)
    close(z[-64:], wz, tz, c.dt)
    dX = G.dequant_linear_backward(y, *c.layer, act=G.ACT_SILU, preact=z)
    g, tol, _ = grad64(c, y[-64:], z[-64:])
    close(dX[-64:], g, tol, c.dt)
    assert (dX[:-64] == 0).all()


def test_status_words():
    for T in (1, 16, 40, 600):
        c = Case(T, 2304, 256, 4, 128, "bf16", "none", True)
        ws = torch.full((1 << 26,), 255, dtype=torch.uint8, device=DEV)
        check = lambda: G.lib().gptq_dequant_matmul_check(ws.data_ptr(), 0, None)  # noqa: E731
        y = G.dequant_linear(c.X, *c.layer, workspace=ws)
        assert check() == G.OK
        for kw in (dict(want_dbias=True), dict(want_dx=False, want_dbias=True), {}):
            ws.fill_(255)
            G.dequant_linear_backward(y, *c.layer, workspace=ws, **kw)
            assert check() == G.OK


def test_after_quantizing_a_layer():
    """The path's own result in use: quantize a layer with act-order, apply it with bias and SiLU, and
    take the gradient."""
    from post_weight_quantization_16_b200 import synth
    from tests import gpu_helpers as GH
    layer = synth.scaled_layer(synth.WORKLOADS["tiny_256x512"][0], m=192, n=1024, n_tok=2048)
    qs = synth.QuantSetting(4, 128, False, 0.01, True)
    q = GH.run_path(layer, qs)
    dev = [torch.from_numpy(np.ascontiguousarray(a)).to(DEV) for a in (q["packed"].view(np.int32), q["scales"], q["zeros"],
                                                                       q["perm"].astype(np.int32))]
    rng = np.random.default_rng(3)
    X = torch.from_numpy(rng.normal(0, 1, (24, 1024))).to(DEV).half()
    b = torch.from_numpy(rng.normal(0, 1, 192)).to(DEV).half()
    y, z = G.dequant_linear(X, *dev, 4, 128, bias=b, act=G.ACT_SILU, want_preact=True)
    want = H.to64(X) @ q["w_hat"].T + H.to64(b)                   # the path's fp32 dequantized weights
    tol = H.product_tol(H.to64(X), q["w_hat"]) + 2.0 ** -22 * (np.abs(H.to64(X)) @ np.abs(q["w_hat"]).T)
    close(z, want, tol, torch.float16)
    close(y, H.act64(want, "silu"), 1.13 * tol + 2.0 ** -19 * np.abs(want), torch.float16)
    dX, db = G.dequant_linear_backward(y, *dev, 4, 128, act=G.ACT_SILU, preact=z, want_dbias=True)
    dz = H.to64(y) * H.act_grad64(H.to64(z), "silu")
    t = 2.0 ** -10 * (np.abs(dz) @ np.abs(q["w_hat"])) + 2.0 ** -11 * np.abs(dz @ q["w_hat"])
    assert (np.abs(H.to64(dX) - dz @ q["w_hat"]) <= t + 1e-6).all()
    assert np.allclose(H.to64(db), dz.sum(0), rtol=1e-4, atol=1e-4)
