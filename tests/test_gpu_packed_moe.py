"""The mixture-of-experts layer on packed experts (gptq_dequant_moe) against plain 64-bit numpy.

Tolerances, element by element.  Logits: the bound of an fp32-accumulated product (product_tol).  A
softmax's p moves by at most 2 p times the largest move of a logit; the weights are fp32, off by another
2^-24 and, when renormalised, by twice that.  The chosen experts are checked by their logits (none left
out is larger by more than twice that bound), and Y is formed with them.  h = act(g) u: the slope of act
is at most 1.13, its evaluation good to 2^-19 of the value, then half a step of dtype.  Y: the error of h
through |Wd|, the second product's own bound, the weights' error, one fp32 rounding per expert and for
the residual, then half a step of dtype."""
import numpy as np
import pytest
import torch

from oracle import gptq_oracle as O
from post_weight_quantization_16_b200 import gptq as G
from tests import packed_helpers as H

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


class Moe:
    def __init__(self, T, E, k, h, i, bits, g, dg, dtype, act="silu", perm=True, renorm=True, seed=0):
        self.rng = rng = np.random.default_rng(seed * 101 + T * 7 + E + h + i)
        self.T, self.E, self.k, self.h, self.i, self.bits, self.g, self.dg = T, E, k, h, i, bits, g, dg
        self.dt, self.act, self.renorm = DT[dtype], act, renorm
        gu = [H.random_layer(rng, 2 * i, h, bits, g, 0.6) for _ in range(E)]
        dn = [H.random_layer(rng, h, i, bits, dg, 0.6) for _ in range(E)]
        st = lambda ls, k: torch.from_numpy(np.stack([x[k].view(np.int32) if k == 1 else x[k] for x in ls])).to(DEV)  # noqa
        self.gate_up, self.down = tuple(st(gu, k) for k in (1, 2, 3)), tuple(st(dn, k) for k in (1, 2, 3))
        self.Wgu = [H.weights64(c, s, z) for c, _, s, z in gu]
        self.Wd = [H.weights64(c, s, z) for c, _, s, z in dn]
        self.perm_np = np.stack([rng.permutation(h) if perm else np.arange(h) for _ in range(E)])
        self.perm = torch.from_numpy(self.perm_np.astype(np.int32)).to(DEV) if perm else None
        self.X = torch.from_numpy(rng.normal(0, 1, (T, h))).to(DEV).to(self.dt)
        self.router = torch.from_numpy(rng.normal(0, 1.5 / np.sqrt(h), (E, h))).to(DEV).to(self.dt)

    def run(self, **kw):
        kw = {"renormalize": self.renorm, "act": H.ACTS[self.act], "down_group_size": self.dg, **kw}
        X, router = kw.pop("X", self.X), kw.pop("router", self.router)
        return G.dequant_moe(X, router, self.gate_up, self.down, self.perm, self.bits, self.g, self.k, **kw)

    def check(self, got, X=None, router=None, residual=None, tokens=None):
        y, ids, w = got
        x = H.to64(self.X if X is None else X)
        r = H.to64(self.router if router is None else router)
        T = x.shape[0]
        assert y.shape == (T, self.h) and ids.shape == w.shape == (T, self.k) and y.dtype == self.dt
        ids, w = ids.cpu().numpy(), w.cpu().numpy().astype(np.float64)
        logits, lt = x @ r.T, H.product_tol(x, r)
        p = np.exp(logits - logits.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        for t in range(T) if tokens is None else tokens:
            e = ids[t]
            assert len(set(e)) == self.k and (0 <= e).all() and (e < self.E).all()
            b = lt[t].max()
            assert (np.diff(logits[t, e]) <= 2 * b).all()
            rest = np.setdiff1d(np.arange(self.E), e)
            assert rest.size == 0 or logits[t, rest].max() <= logits[t, e].min() + 2 * b
            want = p[t, e] / p[t, e].sum() if self.renorm else p[t, e]
            wt = want * (4 * b + 3 * 2.0 ** -24)
            assert (np.abs(w[t] - want) <= wt + 2.0 ** -149).all()
            yy, ty = np.zeros(self.h), np.zeros(self.h)
            for k, ex in enumerate(e):
                xs = x[t:t + 1, self.perm_np[ex]]
                gu = (xs @ self.Wgu[ex].T)[0]
                tg = H.product_tol(xs, self.Wgu[ex])[0]
                gt, up = gu[:self.i], gu[self.i:]
                a = H.act64(gt, self.act)
                ta = 1.13 * tg[:self.i] + 2.0 ** -19 * np.abs(a)
                hh = a * up
                th = ta * np.abs(up) + np.abs(a) * tg[self.i:] + ta * tg[self.i:] + 2.0 ** -23 * np.abs(hh)
                th = th + H.EPS[self.dt] * (np.abs(hh) + th) + H.TINY[self.dt]
                d = self.Wd[ex]
                v = hh @ d.T
                yy += want[k] * v
                ty += want[k] * (th @ np.abs(d).T + H.product_tol((np.abs(hh) + th)[None], d)[0] + 2.0 ** -22 * np.abs(v))
                ty += wt[k] * np.abs(v)
                ty += 2.0 ** -23 * np.abs(yy)
            if residual is not None:
                yy += H.to64(residual)[t]
            tol = ty + 2.0 ** -23 * np.abs(yy) + H.EPS[self.dt] * (np.abs(yy) + ty) + H.TINY[self.dt]
            dd = np.abs(H.to64(y)[t] - yy)
            assert (dd <= tol).all(), (t, float((dd / tol).max()))


CASES = [
    # T, E, k, h, i, bits, g, down g, dtype, act, perm, renormalize
    (1, 8, 2, 256, 128, 4, 128, 128, "fp16", "silu", True, True),
    (1, 1, 1, 128, 128, 2, 32, 64, "bf16", "silu", False, False),
    (2, 5, 5, 384, 256, 3, 64, 128, "fp16", "gelu", True, False),
    (7, 64, 6, 512, 384, 4, 64, 32, "bf16", "silu", True, True),
    (8, 256, 16, 256, 128, 4, 128, 128, "bf16", "silu", False, True),
    (9, 16, 4, 640, 384, 8, 128, 384, "fp16", "relu", True, True),
    (16, 8, 2, 1024, 640, 4, 32, 128, "bf16", "silu", True, True),
    (17, 3, 3, 256, 512, 3, -1, -1, "fp16", "silu", True, True),
    (33, 32, 4, 512, 128, 2, 64, 64, "bf16", "gelu", False, False),
    (64, 8, 2, 256, 256, 8, 32, 128, "bf16", "silu", True, True),
    (100, 7, 1, 384, 128, 4, 128, 128, "fp16", "silu", True, True),
    (128, 64, 8, 256, 128, 3, 128, 32, "fp16", "silu", True, True),
    (128, 1, 1, 256, 384, 4, 128, 128, "bf16", "silu", True, True),
    (128, 2, 2, 256, 256, 3, 32, 128, "fp16", "silu", True, True),
    (127, 3, 1, 384, 512, 8, 64, 64, "bf16", "gelu", False, True),
    (90, 3, 1, 256, 256, 2, -1, 32, "bf16", "silu", True, False),
    (30, 256, 16, 128, 128, 4, 32, 64, "fp16", "silu", True, True),
    (48, 8, 2, 2048, 1408, 4, 128, 128, "bf16", "none", True, True),
]


@pytest.mark.parametrize("T,E,k,h,i,bits,g,dg,dtype,act,perm,renorm", CASES)
def test_moe(T, E, k, h, i, bits, g, dg, dtype, act, perm, renorm):
    c = Moe(T, E, k, h, i, bits, g, dg, dtype, act, perm, renorm)
    r = torch.from_numpy(c.rng.normal(0, 1, (T, h))).to(DEV).to(c.dt) if T % 2 else None
    c.check(c.run(residual=r), residual=r)


def test_ties_go_to_the_lower_expert_and_every_token_to_one():
    c = Moe(40, 12, 3, 256, 128, 4, 64, 64, "fp16")
    router = torch.zeros_like(c.router)                         # every expert equal
    y, ids, w = got = c.run(router=router)
    assert (ids.cpu().numpy() == np.arange(3)).all() and torch.allclose(w, torch.full_like(w, 1 / 3), rtol=1e-6)
    c.check(got, router=router)
    router = c.router.clone()
    router[9] = router[4]                                       # two identical rows, among others
    y, ids, w = got = c.run(router=router)
    c.check(got, router=router)
    for row in ids.cpu().numpy().tolist():
        assert 9 not in row or (4 in row and row.index(4) < row.index(9))
    x = c.X.abs() + 0.5
    router = torch.full_like(c.router, -1.0)
    router[7] = 1.0                                             # logits so far apart that the rest weigh nothing
    y, ids, w = got = c.run(X=x, router=router)
    assert (ids[:, 0] == 7).all() and (ids[:, 1:].cpu().numpy() == [0, 1]).all() and (w[:, 0] == 1).all() and (w[:, 1:] == 0).all()
    c.check(got, X=x, router=router)


@pytest.mark.parametrize("T", [3, 33])
def test_a_token_of_nan_or_infinity_leaves_the_others(T):
    c = Moe(T, 16, 4, 256, 256, 4, 128, 128, "bf16")
    y0, ids0, w0 = c.run()
    x = c.X.clone()
    x[1, 3], x[2, 5] = float("nan"), float("inf")
    y, ids, w = c.run(X=x)
    keep = [t for t in range(T) if t not in (1, 2)]
    assert torch.equal(y[keep], y0[keep]) and torch.equal(ids[keep], ids0[keep]) and torch.equal(w[keep], w0[keep])
    assert not y[1].isfinite().any() and not y[2].isfinite().any()
    assert (ids >= 0).all() and (ids < 16).all()
    for t in (1, 2):
        assert len(set(ids[t].tolist())) == 4


def test_strides_no_tokens_and_residual_in_place():
    c = Moe(19, 8, 2, 384, 256, 4, 128, 128, "fp16")
    wide = torch.zeros(19, 384 + 16, dtype=c.dt, device=DEV)
    wide[:, 8:392] = c.X
    out = torch.full((19, 391), 7.0, dtype=c.dt, device=DEV)
    res = torch.randn(19, 385, device=DEV).to(c.dt)[:, 1:]
    y, ids, w = got = c.run(X=wide[:, 8:392], residual=res, out=out[:, 3:387])
    c.check((y, ids, w), residual=res)
    assert (out[:, :3] == 7).all() and (out[:, 387:] == 7).all()
    buf = res.contiguous()
    y2, *_ = c.run(residual=buf, out=buf)
    assert y2 is buf and torch.equal(y2, y)
    x = c.X.clone()
    y3, *_ = c.run(X=x, residual=x, out=x)                       # a block's input, residual and output in one
    assert y3 is x and torch.equal(x, c.run(residual=c.X)[0])
    x = c.X[:5].clone()                                         # (the kernels that lay out X themselves)
    assert torch.equal(c.run(X=x, residual=x, out=x)[0], c.run(X=c.X[:5], residual=c.X[:5])[0])
    y, ids, w = c.run(X=c.X[:0])
    assert y.shape == (0, 384) and ids.shape == w.shape == (0, 2)


@pytest.mark.parametrize("T", [1, 12, 64])
def test_runs_agree_streams_and_graphs(T):
    c = Moe(T, 24, 4, 512, 384, 4, 128, 128, "bf16")
    ref = c.run()
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(c.run(), ref))
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream(DEV))
    got = c.run(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    x1, x2 = c.X.clone(), torch.zeros_like(c.X)
    graphs = []
    for x in (x1, x2):
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, c.run(X=x)))
    x2.copy_(c.X)
    for g, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    for g, out in graphs:
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
    flipped = c.X.flip(1).contiguous()                          # other experts are chosen in the replay
    x1.copy_(flipped)
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(graphs[0][1], c.run(X=flipped)))
    c.check(graphs[0][1], X=flipped)


def test_two_calls_at_once_on_two_streams():
    c, d = Moe(24, 8, 2, 1024, 512, 4, 128, 128, "bf16"), Moe(24, 8, 2, 1024, 512, 4, 128, 128, "bf16", seed=1)
    want = c.run(), d.run()
    s1, s2 = torch.cuda.Stream(DEV), torch.cuda.Stream(DEV)
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        got.append((c.run(stream=s1), d.run(stream=s2)))
    torch.cuda.synchronize()
    for pair in got:
        for a, b in zip(pair, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_refusals_on_the_device():
    c = Moe(4, 8, 2, 256, 128, 4, 128, 128, "bf16")
    bad = [dict(X=c.X.float()), dict(X=c.X[:, :128]), dict(router=c.router.float()), dict(router=c.router[:0]),
           dict(router=c.router[:4]), dict(router=torch.cat([c.router, c.router])[:, :128]),
           dict(residual=c.X.float()), dict(residual=c.X[:3]), dict(out=torch.zeros(4, 256, device=DEV)),
           dict(workspace=torch.zeros(256, dtype=torch.uint8, device=DEV)), dict(down_group_size=64)]
    for kw in bad:
        with pytest.raises(ValueError):
            c.run(**kw)
    for k in (0, 9, 17):
        with pytest.raises(G.GPTQError):
            G.dequant_moe(c.X, c.router, c.gate_up, c.down, c.perm, 4, 128, k)
    with pytest.raises(G.GPTQError):
        c.run(X=torch.zeros(129, 256, device=DEV, dtype=c.dt))
    with pytest.raises(G.GPTQError):
        c.run(act=9)


def test_a_block_as_it_is_used():
    """Experts quantized by the framework, stacked, and run in a captured step with a projection before
    and its gradient behind: quantize -> stack_experts -> dequant_linear -> dequant_moe ->
    dequant_linear_backward."""
    rng = np.random.default_rng(11)
    E, h, i, T = 4, 256, 384, 9
    w = lambda m, n: torch.from_numpy(rng.normal(0, 1 / np.sqrt(n), (m, n)).astype(np.float16)).to(DEV)  # noqa: E731
    q = lambda W: G.rtn_quantize(W, 4, 64, False)  # noqa: E731
    gates, ups, downs = [[q(w(*s)) for _ in range(E)] for s in ((i, h), (i, h), (h, i))]
    proj = q(w(h, h))
    gate_up, down, perm = G.stack_experts(gates, ups, downs)
    assert perm is None
    router = (w(E, h) * 3).bfloat16()
    X = torch.from_numpy(rng.normal(0, 1, (T, h))).to(DEV).bfloat16()
    layer = [proj["codes"], proj["scales"], proj["zeros"], None, 4, 64]

    def step(x):
        a, z = G.dequant_linear(x, *layer, act=G.ACT_GELU, residual=x, want_preact=True)
        y, ids, wts = G.dequant_moe(a, router, gate_up, down, None, 4, 64, 2, residual=a)
        dx = G.dequant_linear_backward(y, *layer, act=G.ACT_GELU, preact=z)
        return a, z, y, ids, wts, dx

    ref = step(X)
    x2 = torch.zeros_like(X)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(x2)
    x2.copy_(X)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, ref))
    a, z, y, ids, wts, dx = ref

    def dense(d, m, n):
        return H.weights64(O.unpack_codes(d["codes"].cpu().numpy().view(np.uint32), n, 4),
                           d["scales"].cpu().numpy(), d["zeros"].cpu().numpy())

    Wp = dense(proj, h, h)
    zz = H.to64(X) @ Wp.T
    aa = H.act64(zz, "gelu") + H.to64(X)
    tol = 1.13 * H.product_tol(H.to64(X), Wp) + 2.0 ** -19 * np.abs(aa) + 2.0 ** -22 * np.abs(aa)
    assert (np.abs(H.to64(a) - aa) <= tol + 2.0 ** -8 * (np.abs(aa) + tol)).all()
    # the layer on the rounded a (its own input), by its own oracle
    m = Moe.__new__(Moe)
    m.T, m.E, m.k, m.h, m.i, m.bits, m.g, m.dg, m.dt, m.act, m.renorm = T, E, 2, h, i, 4, 64, 64, torch.bfloat16, "silu", True
    m.X, m.router, m.perm_np = a, router, np.tile(np.arange(h), (E, 1))
    m.Wgu = [np.concatenate([dense(gates[e], i, h), dense(ups[e], i, h)]) for e in range(E)]
    m.Wd = [dense(downs[e], h, i) for e in range(E)]
    m.check((y, ids, wts), residual=a)
    dz = H.to64(y) * H.act_grad64(H.to64(z), "gelu")
    t = (2.0 ** -10 + 2.0 ** -14) * (np.abs(dz) @ np.abs(Wp)) + 2.0 ** -8 * np.abs(dz @ Wp)
    assert (np.abs(H.to64(dx) - dz @ Wp) <= t + 2.0 ** -19 * 1.13 * np.abs(H.to64(y)) @ np.abs(Wp)).all()
