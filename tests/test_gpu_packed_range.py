"""The operators on packed weights over the range of values that their types hold: outliers that an
activation masks, infinities, layers of very small and very large scales."""
import numpy as np
import pytest
import torch

from post_weight_quantization_16_b200 import gptq as G
from tests import packed_helpers as H
from tests.test_gpu_packed_linear import DEV, Case
from tests.test_gpu_packed_moe import Moe

pytestmark = pytest.mark.gpu
KERNELS = [(20, 256), (300, 9472)]                    # tokens and columns of the single-block and of the pair kernel


def gradient_close(c, got, dY, Z, dtype, sharp=True):
    """dX against the 64-bit formula with the exact weights: every product of dz and a weight is off by at
    most 2^-11 for each of them (2^-10 and the product of the two), a value of dz by 2^-25 of 2^13 times less
    than the token's largest |dz| where it is that small, the sum by its accumulation, dX by its rounding."""
    dz = H.to64(dY) * H.act_grad64(H.to64(Z), c.act)
    W = np.zeros_like(c.W)
    W[:, c.perm_np] = c.W
    want = dz @ W
    tol = (2.0 ** -10 + 2.0 ** -21) * (np.abs(dz) @ np.abs(W)) + H.product_tol(dz, W.T) - 1e-30   # (no absolute part: the layers' scales vary)
    tol += np.abs(dz).max(1, keepdims=True) * 2.0 ** (-13 - 25) * np.abs(W).sum(0)
    # a weight is off by 2^-39 of the largest that its 128 columns' scales allow where it is that small
    largest = np.zeros(c.n)
    largest[c.perm_np] = np.repeat(np.repeat(c.s.max(0), c.n // c.s.shape[1]).reshape(-1, 128).max(1), 128) * 2.0 ** c.bits
    tol += 2.0 ** -39 * np.abs(dz).sum(1, keepdims=True) * largest
    # (act' itself is good to 2^-19 of its largest value, 1.13)
    if c.act != "relu":
        tol += 2.0 ** -19 * 1.13 * (np.abs(np.where(np.abs(H.to64(Z)) > 50, 0, H.to64(dY))) @ np.abs(W))
    tol += H.EPS[dtype] * (np.abs(want) + tol) + H.TINY[dtype]
    d = np.abs(H.to64(got) - want)
    assert (d <= tol).all(), float((d / tol).max())
    # the tolerance says something: it is far below the values.  (Not with very many rows: the accumulation's
    # bound grows with their number, 2^-8 of the sum of magnitudes at 270000, and the values with its root.)
    assert not sharp or np.median(tol / np.abs(want).clip(1e-300)) < 0.1


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


def rescaled(c, factor):
    """The case with its scales multiplied (factor: a number or an [m, groups] array)."""
    c.s = (c.s.astype(np.float64) * factor).astype(np.float32)
    c.layer[1] = torch.from_numpy(c.s).to(DEV)
    c.W = H.weights64(c.codes, c.s, c.z)
    return c


@pytest.mark.parametrize("T,n", KERNELS + [(40, 384)])
@pytest.mark.parametrize("bits,g,dtype,act,dy,factor", [
    (8, 128, "bf16", "none", 1.0, 1e-3), (8, 32, "bf16", "silu", 1.0, 1e-6), (4, 64, "fp16", "none", 100.0, 1e-4),
    (4, -1, "bf16", "none", 1.0, 1e7), (2, 32, "fp16", "relu", 1e-3, 1e5), (3, 64, "bf16", "gelu", 1.0, 1e30),
    (4, 128, "bf16", "none", 1.0, 1e-30)])
def test_gradient_of_layers_of_any_scale(T, n, bits, g, dtype, act, dy, factor):
    """The forward pass holds its scales in fp32; the gradient's fp16 weights reach as far."""
    c = rescaled(Case(T, 200, n, bits, g, dtype, act, True), factor)
    dY = c.dev(c.rng.normal(0, dy, (T, 200)))
    Z = c.dev(c.rng.normal(0, 1, (T, 200)))
    gradient_close(c, G.dequant_linear_backward(dY, *c.layer, act=H.ACTS[act], preact=Z), dY, Z, c.dt)


@pytest.mark.parametrize("T,n", KERNELS)
@pytest.mark.parametrize("bits,g", [(4, 128), (8, 64), (3, 32), (2, 256)])
def test_gradient_of_columns_and_rows_of_different_scales(T, n, bits, g):
    """Blocks of 128 columns a factor of up to 2^60 apart do not touch one another's bits; rows inside a
    block may be 2^20 apart, or zero."""
    m = 200
    c = Case(T, m, n, bits, g, "bf16", "none", True)
    per = max(1, g // 128)                                             # blocks of 128 columns that share a group
    blocks = np.repeat(c.rng.integers(-30, 31, -(-n // 128 // per)), per)[: n // 128].astype(float)
    f = 2.0 ** np.repeat(blocks, 128)[:: g] * 2.0 ** c.rng.integers(-20, 1, (m, 1))
    f[:, :: 5] *= (c.rng.random((m, 1)) < 0.9)
    if f.shape[1] >= 8:
        f[:, 0] = 0.0
    rescaled(c, f)
    dY = c.dev(c.rng.normal(0, 1, (T, m)))
    Z = c.dev(np.ones((T, m)))
    gradient_close(c, G.dequant_linear_backward(dY, *c.layer), dY, Z, c.dt)


@pytest.mark.parametrize("T,E,k,h,i,g,dg,dtype,perm", [
    (1, 4, 2, 256, 256, 64, 128, "fp16", True), (6, 8, 3, 384, 128, 32, 32, "fp16", False),
    (12, 2, 1, 256, 640, 128, 128, "fp16", True), (33, 4, 2, 256, 384, 64, 64, "fp16", True),
    (128, 2, 2, 256, 256, 128, 128, "fp16", False), (33, 4, 2, 256, 384, 64, 64, "bf16", True)])
@pytest.mark.parametrize("factor", [2.0 ** 9, 2.0 ** 17])
def test_experts_gated_values_past_fp16(T, E, k, h, i, g, dg, dtype, perm, factor):
    """A twentieth of the gate and up rows with |h| of up to 1e7 or 1e12 in every other expert, and down
    weights there that bring Y back: finite, and as exact as without them."""
    c = Moe(T, E, k, h, i, 4, g, dg, dtype, perm=perm, seed=3)
    for e in range(0, E, 2):
        rows = c.rng.choice(i, i // 20, replace=False)
        for r in (rows, rows + i):
            c.gate_up[1][e, torch.from_numpy(r).to(DEV)] *= factor
            c.Wgu[e][r] *= factor
        c.down[1][e] *= 2.0 ** -2 / factor ** 2
        c.Wd[e] *= 2.0 ** -2 / factor ** 2
    got = c.run()
    assert got[0].isfinite().all()
    c.check(got)
    assert torch.equal(c.run()[0], got[0])


def choices64(x, r, k):
    """The k largest logits of 64 bits, descending, ties to the lower expert; no two of x r^T that the
    choices hang on are closer than 64 bits can tell."""
    logits = x @ r.T
    ids = np.argsort(-logits, axis=1, kind="stable")
    s = np.take_along_axis(logits, ids, 1)
    gap = np.abs(np.diff(s, axis=1))[:, : k]
    noise = 2.0 ** -53 * x.shape[1] ** 0.5 * (np.abs(x) @ np.abs(r).T).max()
    assert (gap > 100 * noise).all()
    return ids[:, :k], logits


@pytest.mark.parametrize("T,E,k,h,dtype", [(1, 64, 8, 2048, "fp16"), (33, 64, 8, 2048, "bf16"), (128, 256, 16, 512, "fp16"),
                                           (17, 34, 5, 4096, "bf16"), (9, 6, 6, 1152, "fp16")])
@pytest.mark.parametrize("outlier", [1.0, 1000.0])
def test_choices_are_those_of_64_bit_logits(T, E, k, h, dtype, outlier):
    """Pairs of experts whose logits agree to far fewer bits than fp32 holds of their sums: half of the
    rows are the others with one entry a step away, and a few channels of X are large."""
    c = Moe(T, E, k, h, 128, 4, 128, 128, dtype, perm=False, seed=5)
    X = c.X.double()
    X[:, torch.from_numpy(c.rng.choice(h, 4, replace=False)).to(DEV)] *= outlier
    X = X.to(c.dt)
    r = c.router.clone()
    for e in range(E // 2):
        r[e + E // 2] = r[e]
        at = int(c.rng.integers(h))
        r[e + E // 2, at] *= 1 + 4 * H.EPS[c.dt]
    x, rr = H.to64(X), H.to64(r)
    near = (rr[: E // 2] != rr[E // 2: 2 * (E // 2)]).sum(1)
    assert (near == 1).all()
    want, logits = choices64(x, rr, k)
    y, ids, w = c.run(X=X, router=r)
    assert np.array_equal(ids.cpu().numpy(), want)
    p = np.exp(logits - logits.max(1, keepdims=True))
    p = np.take_along_axis(p, want, 1)
    p /= p.sum(1, keepdims=True)
    # the chosen weights: fp32 after logits that are off by at most 2^-16 of their products' magnitudes
    b = 2.0 ** -16 * (np.abs(x) @ np.abs(rr).T).max(1, keepdims=True)
    assert (np.abs(H.to64(w) - p) <= p * (4 * np.minimum(b, 1) + 2.0 ** -22) + 1e-30).all()


def test_tokens_of_zeros_and_equal_experts():
    """Padding rows (every logit 0) and routers of equal rows: the lowest experts, in order."""
    c = Moe(20, 40, 4, 256, 128, 4, 64, 64, "bf16")
    X = c.X.clone()
    X[::2] = 0
    y, ids, w = c.run(X=X)
    assert (ids[::2].cpu().numpy() == np.arange(4)).all() and (w[::2] == 0.25).all() and (y[::2] == 0).all()
    r = c.router[:1].expand(40, -1).contiguous()
    y, ids, w = c.run(router=r)
    assert (ids.cpu().numpy() == np.arange(4)).all() and (w == 0.25).all()


@pytest.mark.parametrize("act", ["none", "silu"])
def test_gradient_of_no_tokens(act):
    c = Case(4, 33, 256, 4, 64, "fp16", act, True)
    e = torch.empty(0, 33, dtype=c.dt, device=DEV)
    dx = G.dequant_linear_backward(e, *c.layer, act=H.ACTS[act], preact=e)
    assert dx.shape == (0, 256) and dx.dtype == c.dt


@pytest.mark.parametrize("T,m,n,bits,g", [(5, 40000, 256, 4, 64), (3, 270000, 128, 2, 32), (4, 50, 65536, 4, 32), (3, 30000, 128, 3, -1),
                                          (20, 1100, 65536, 2, 64), (600, 9000, 1152, 4, 384)])
def test_gradient_scales_are_looked_at_in_every_row_and_column(T, m, n, bits, g):
    """One scale of each block of 128 columns, in a row of its own, is 2^14 times the others: fp16 would
    overflow if its slab, or its group among many, were left out."""
    c = Case(T, m, n, bits, g, "bf16", "none", True)
    f = np.ones_like(c.s, dtype=np.float64)
    G_ = f.shape[1]
    per = max(1, 128 * G_ // n)
    for b in range(0, G_, per):
        f[c.rng.integers(m), b + c.rng.integers(per)] = 2.0 ** 14
    f[m - 1, G_ - 1] = f[0, 0] = 2.0 ** 14
    rescaled(c, 16 * f)
    dY = c.dev(c.rng.normal(0, 1, (T, m)))
    Z = c.dev(np.ones((T, m)))
    gradient_close(c, G.dequant_linear_backward(dY, *c.layer), dY, Z, c.dt, sharp=m < 20000)


@pytest.mark.parametrize("T,n", KERNELS)
@pytest.mark.parametrize("act", ["gelu", "silu", "relu"])
def test_gradients_at_the_end_of_bf16(T, n, act):
    """dY up to bf16's largest where the slope is above 1: dz alone is past fp32, dX is not."""
    c = Case(T, 200, n, 4, 128, "bf16", act, True)
    dY = torch.from_numpy(c.rng.choice([-3.3e38, 3.3e38, 1e38, -1e37], (T, 200))).to(DEV).to(c.dt)
    Z = torch.from_numpy(c.rng.uniform(1.2, 2.5, (T, 200))).to(DEV).to(c.dt)
    rescaled(c, 2.0 ** -10)
    gradient_close(c, G.dequant_linear_backward(dY, *c.layer, act=H.ACTS[act], preact=Z), dY, Z, c.dt)


def test_an_expert_whose_router_row_is_infinite_leaves_the_others_order():
    """Its logit is an infinity of either sign: chosen first or last; the others stand as 64-bit logits say."""
    c = Moe(40, 32, 4, 512, 128, 4, 64, 64, "bf16", perm=False, seed=9)
    r = c.router.clone()
    for e in range(16):
        r[e + 16] = r[e]
        r[e + 16, 7 * e] *= 1 + 4 * H.EPS[c.dt]
    r[5] = 0
    r[5, 3] = float("inf")
    x, rr = H.to64(c.X), H.to64(r)
    rr[5] = 0
    logits = x @ rr.T
    logits[:, 5] = np.where(x[:, 3] > 0, np.inf, -np.inf)
    want = np.argsort(-logits, axis=1, kind="stable")[:, :4]
    X = c.X.clone()
    y, ids, w = c.run(X=X, router=r)
    assert (x[:, 3] != 0).all() and np.array_equal(ids.cpu().numpy(), want)


def captured(call):
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    return g, out


@pytest.mark.parametrize("T", [4, 40])
def test_a_graph_s_replays_keep_nothing_of_the_one_before(T):
    """Inputs and weights changed between replays so that what a call finds out about them changes: gated
    values past fp16 and back, choices that stand close and do not, the weights' largest scale."""
    c = Moe(T, 8, 2, 256, 256, 4, 64, 128, "fp16", seed=4)
    c.down[1].mul_(2.0 ** -20)
    X = c.X.clone()
    g, out = captured(lambda: c.run(X=X))
    for factor in (1.0, 200.0, 1.0, 0.0, 200.0, 1.0):
        X.copy_(c.X * factor)
        g.replay()
        torch.cuda.synchronize()
        fresh = c.run(X=X)
        for a, b in zip(out, fresh):
            assert torch.equal(a, b), factor
        assert out[0].isfinite().all()
    for T, n in [(T, 256), (300, 9472)]:
        k = Case(T, 200, n, 4, 128, "bf16", "silu", True)
        dY, Z = k.dev(k.rng.normal(0, 1, (T, 200))), k.dev(k.rng.normal(0, 1, (T, 200)))
        scales, grad = k.layer[1].clone(), dY.clone()
        g, out = captured(lambda: G.dequant_linear_backward(dY, *k.layer, act=G.ACT_SILU, preact=Z, want_dbias=True))
        for ws, gs in ((1.0, 1.0), (2.0 ** 40, 1.0), (2.0 ** -40, 2.0 ** 50), (0.0, 1.0), (1.0, 0.0), (1.0, 1.0)):
            k.layer[1].copy_(scales * ws)
            dY.copy_(grad * gs)
            g.replay()
            torch.cuda.synchronize()
            dx, db = G.dequant_linear_backward(dY, *k.layer, act=G.ACT_SILU, preact=Z, want_dbias=True)
            assert torch.equal(out[0], dx) and torch.equal(out[1], db), (ws, gs)
            if ws and gs:
                k.s = k.layer[1].cpu().numpy()                         # (the tensor stays the graph's)
                k.W = H.weights64(k.codes, k.s, k.z)
                gradient_close(k, dx, dY, Z, k.dt)


def test_two_streams_at_once():
    """Gradients and experts of different inputs on two streams that run together, each as alone."""
    a, b = Case(200, 300, 512, 4, 64, "bf16", "gelu", True, seed=1), Case(200, 300, 512, 4, 64, "fp16", "none", True, seed=2)
    m1, m2 = Moe(20, 8, 2, 256, 256, 4, 64, 64, "fp16", seed=6), Moe(20, 8, 2, 256, 256, 4, 64, 64, "bf16", seed=7)
    Z = a.dev(a.rng.normal(0, 1, (200, 300)))
    d1, d2 = a.dev(a.rng.normal(0, 1, (200, 300))), b.dev(b.rng.normal(0, 1, (200, 300)))
    calls = [(lambda **k: G.dequant_linear_backward(d1, *a.layer, act=G.ACT_GELU, preact=Z, **k), lambda **k: m1.run(**k)[0]),
             (lambda **k: G.dequant_linear_backward(d2, *b.layer, **k), lambda **k: m2.run(**k)[0])]
    want = [[f() for f in fs] for fs in calls]
    streams = [torch.cuda.Stream(DEV) for _ in calls]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(30):
        for k, s in enumerate(streams):
            got[k].append([f(stream=s) for f in calls[k]])
    torch.cuda.synchronize()
    for k in range(2):
        for row in got[k]:
            assert all(torch.equal(x, y) for x, y in zip(row, want[k]))
