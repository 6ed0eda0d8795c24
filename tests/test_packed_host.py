"""Host side of the operators on packed layers (no GPU): argument blocks, sizes, refusals before any
device call, the stacking of experts."""
import ctypes
import re
import struct

import numpy as np
import pytest
import torch

from oracle import gptq_oracle as O
from post_weight_quantization_16_b200 import build as B
from post_weight_quantization_16_b200 import gptq as G

P = 1 << 20  # an aligned address that no check dereferences
Q = 1 << 40  # another, for outputs
NO_DEVICE = -1  # what passes the checks of arguments ends here, with GPTQ_ERR_CUDA


@pytest.fixture(scope="module")
def L():
    B.build()
    return G.lib()


def packed(m=64, n=512, bits=4, g=128, perm=0, codes=P, scales=P, zeros=P):
    return (codes, scales, zeros, perm, m, n, bits, g, 0)


def linear(L, W=None, X=P, T=4, ldx=512, dtype=0, bias=0, res=0, ldr=0, act=0, Y=Q, ldy=64, f32=0, preact=0, ws=P,
           wsb=1 << 20):
    a = G._LINEAR_ARGS.pack(X, T, ldx, dtype, *(W or packed()), bias, res, ldr, act, Y, ldy, f32, preact, ws, wsb)
    return L.gptq_dequant_linear(a, NO_DEVICE, None)


def backward(L, W=None, dY=P, T=4, ld=64, dtype=0, act=0, Z=0, dX=Q, ldx=512, db=0, ws=P, wsb=1 << 20):
    a = G._LINEAR_GRAD_ARGS.pack(dY, T, ld, dtype, *(W or packed()), act, Z, dX, ldx, db, ws, wsb)
    return L.gptq_dequant_linear_backward(a, NO_DEVICE, None)


def moe(L, T=4, E=8, k=2, gu=None, dn=None, X=P, ldx=512, R=P, renorm=1, act=3, dtype=0, res=0, ldr=0, Y=Q, ldy=512, ws=P,
        wsb=1 << 30):
    gu = gu or packed(m=512, n=512)
    dn = dn or packed(m=512, n=256)
    a = G._MOE_ARGS.pack(X, T, ldx, dtype, R, E, k, renorm, act, *gu, *dn, res, ldr, Y, ldy, 0, 0, ws, wsb)
    return L.gptq_dequant_moe(a, NO_DEVICE, None)


def test_argument_blocks_have_the_header_s_layout():
    """Field by field from include/gptq.h: the packed formats place every member where C does."""
    text = open(G.HEADER).read()
    size = {"gptq_qparams": (12, 4), "gptq_packed": (64, 8)}
    for t in ("int64_t", "size_t"):
        size[t] = (8, 8)
    size["int"] = (4, 4)

    def layout(name):
        body = re.search(r"typedef struct \{([^}]*)\} %s;" % name, text).group(1)
        off, total = 0, []
        for decl in re.sub(r"/\*.*?\*/|//[^\n]*", "", body, flags=re.S).split(";"):
            decl = decl.strip()
            if not decl:
                continue
            base = decl.replace("const ", "").split()[0]
            for var in decl.split(",") if "*" not in decl else [decl]:
                s, al = (8, 8) if "*" in decl else size[base]
                off = (off + al - 1) // al * al + s
                total.append(off - s)
        return (off + 7) // 8 * 8, total

    for name, fmt in (("gptq_linear_args", G._LINEAR_ARGS), ("gptq_linear_grad_args", G._LINEAR_GRAD_ARGS),
                      ("gptq_moe_args", G._MOE_ARGS)):
        assert layout(name)[0] == fmt.size, name
    assert layout("gptq_packed")[0] == struct.calcsize("@" + G._PACKED) == 64


def test_workspace_sizes(L):
    f = L.gptq_dequant_linear_workspace_bytes
    assert f(1, 512, 0) >= 256 and f(16, 512, 1) >= 256 + 16 * 512 * 2
    assert f(4096, 512, 0) == 256 and f(4096, 512, 1) >= 256 + 4096 * 512 * 2
    assert f(0, 512, 0) > 0                                                    # no tokens: a no-op call
    for bad in ((-1, 512), ((1 << 22) + 1, 512), (4, 100), (4, 0), (4, 65536 + 128)):
        assert f(*bad, 0) == 0, bad
    b = L.gptq_dequant_linear_backward_workspace_bytes
    assert b(8, 100, 512, 1, 1, 0) >= 8 * 104 * 2 + 8 * 512 * 2
    assert b(8, 100, 512, 0, 0, 3) >= 2 * 8 * 104 * 2                          # fp16, smooth: two parts
    assert b(8, 0, 512, 0, 0, 0) == 0 and b(8, 4, 512, 0, 2, 0) == 0 and b(8, 4, 512, 0, 0, 4) == 0
    m = L.gptq_dequant_moe_workspace_bytes
    assert m(1, 8, 2, 512, 256) > 0 and m(128, 256, 16, 512, 256) > 0
    for bad in ((129, 8, 2, 512, 256), (4, 257, 2, 512, 256), (4, 8, 9, 512, 256), (4, 32, 17, 512, 256), (4, 8, 0, 512, 256),
                (4, 8, 2, 500, 256), (4, 8, 2, 512, 64), (-1, 8, 2, 512, 256)):
        assert m(*bad) == 0, bad


def test_linear_refusals(L):
    E = G.ERR_ARG
    assert L.gptq_dequant_linear(None, 0, None) == E
    for W in (packed(codes=0), packed(scales=0), packed(zeros=0), packed(m=0), packed(n=500), packed(n=0), packed(bits=5),
              packed(g=96), packed(g=16), packed(n=65536 + 128), packed(codes=P + 4), packed(perm=P + 4), packed(scales=P + 2),
              packed(g=384)):
        assert linear(L, W, ldx=max(512, W[5])) == E, W
    for kw in (dict(X=0), dict(X=P + 8), dict(ldx=504), dict(ldx=516), dict(T=-1), dict(T=(1 << 22) + 1), dict(dtype=2),
               dict(act=4), dict(act=-1), dict(Y=0), dict(Y=Q + 1), dict(ldy=63), dict(f32=2), dict(f32=1, Y=Q + 2),
               dict(bias=P + 1), dict(res=P, ldr=63), dict(res=P + 1, ldr=64), dict(preact=P + 1), dict(ws=0), dict(ws=P + 128),
               dict(wsb=255)):
        assert linear(L, **kw) == E, kw
    assert linear(L) == linear(L, act=3, res=P, ldr=64, bias=P) == G.ERR_CUDA   # the defaults are fine
    assert linear(L, T=0, X=0, Y=0, ws=0) == G.OK                              # nothing to do


def test_backward_refusals(L):
    E = G.ERR_ARG
    assert L.gptq_dequant_linear_backward(None, 0, None) == E
    for kw in (dict(W=packed(bits=7)), dict(dY=0), dict(dY=P + 1), dict(ld=63), dict(ldx=511), dict(dX=Q + 1), dict(dtype=3),
               dict(act=9), dict(act=3, Z=0), dict(act=3, Z=P + 1), dict(dX=0), dict(db=P + 2), dict(ws=0), dict(ws=P + 8),
               dict(dtype=1, wsb=256), dict(T=-1)):
        assert backward(L, **kw) == E, kw
    assert backward(L) == backward(L, act=3, Z=P, db=P) == G.ERR_CUDA
    assert backward(L, T=0, dY=0, ws=0) == G.OK


def test_moe_refusals(L):
    E = G.ERR_ARG
    assert L.gptq_dequant_moe(None, 0, None) == E
    for kw in (dict(T=129), dict(T=-1), dict(E=0), dict(E=257), dict(k=0), dict(k=9), dict(X=0), dict(X=P + 2), dict(ldx=520 - 4),
               dict(ldx=256), dict(R=0), dict(R=P + 8), dict(renorm=2), dict(act=4), dict(dtype=2), dict(Y=0), dict(ldy=511),
               dict(res=P, ldr=8), dict(ws=0), dict(ws=P + 64), dict(wsb=1000), dict(gu=packed(m=511, n=512)),
               dict(gu=packed(m=512, n=384)), dict(dn=packed(m=384, n=256)), dict(dn=packed(m=512, n=256, perm=P)),
               dict(dn=packed(m=512, n=256, bits=8)), dict(gu=packed(m=512, n=512, perm=P + 4))):
        assert moe(L, **kw) == E, kw
    assert moe(L) == moe(L, res=P, ldr=512) == G.ERR_CUDA
    assert moe(L, T=0, X=0, Y=0, R=0, ws=0) == G.OK


def test_outputs_that_overlap(L):
    """X [4 x 512], Y and residual [4 x 64], 16-bit: refused where rows share memory, not where column
    slices of one buffer lie side by side."""
    E, ok = G.ERR_ARG, G.ERR_CUDA
    for Y, ldy, want in ((P, 64, E), (P + 3 * 1024 + 1022, 64, E), (P + 4 * 1024, 64, ok), (P - 512, 64, ok), (P - 510, 64, E)):
        assert linear(L, Y=Y, ldy=ldy) == want, (Y - P, ldy)
    for at, want in ((1024, ok), (1022, E), (1152 - 128, ok), (1152 - 126, E), (0, E)):     # rows of 576 values
        assert linear(L, ldx=576, Y=P + at, ldy=576) == want, at
    assert linear(L, ldx=576, Y=P + 1024, ldy=576, f32=1) == E                 # fp32 rows: other strides
    assert linear(L, T=1, ldx=576, Y=P + 1024, ldy=64) == ok
    assert linear(L, res=Q, ldr=64) == ok                                      # in place
    assert linear(L, res=Q, ldr=72) == linear(L, res=Q + 2, ldr=64) == linear(L, res=Q, ldr=64, f32=1) == E
    assert linear(L, T=1, res=Q, ldr=72) == ok
    assert linear(L, preact=Q) == linear(L, preact=P) == linear(L, preact=2 * Q, res=2 * Q, ldr=64) == E
    assert linear(L, preact=2 * Q) == ok
    assert backward(L, dY=Q) == backward(L, dY=Q + 4094) == backward(L, act=3, Z=Q) == E
    assert backward(L, dY=Q + 4096) == backward(L, Z=Q) == ok                  # (Z is not read without an activation)
    assert moe(L, res=Q, ldr=512) == moe(L, Y=P) == ok
    assert moe(L, res=Q + 2, ldr=512) == moe(L, res=Q, ldr=520) == E


def test_a_stream_of_another_device_is_refused():
    class Stream:
        device_index, cuda_stream = 1, 0

    x, c, s = torch.zeros(2, 512, dtype=torch.float16), torch.zeros(4, 64, dtype=torch.int32), torch.zeros(4, 4)
    for call in (lambda: G.dequant_linear(x, c, s, s, None, 4, 128, stream=Stream()),
                 lambda: G.dequant_linear_backward(x, c, s, s, None, 4, 128, stream=Stream()),
                 lambda: G.dequant_moe(x, x, (c, s, s), (c, s, s), None, 4, 128, 1, stream=Stream())):
        with pytest.raises(ValueError, match="stream belongs"):
            call()


def test_binding_refuses_what_is_not_on_a_device():
    x = torch.zeros(2, 512, dtype=torch.float16)
    codes, s = torch.zeros(4, 64, dtype=torch.int32), torch.zeros(4, 4)
    with pytest.raises(ValueError, match="device tensor"):
        G.dequant_linear(x, codes, s, s, None, 4, 128)
    with pytest.raises(ValueError, match="bits"):
        G.dequant_linear(x, codes, s, s, None, 5, 128)
    with pytest.raises(ValueError, match="group_size"):
        G.dequant_linear(x, codes, s, s, None, 4, 100)
    with pytest.raises(ValueError, match="scales"):
        G.dequant_linear(x, codes, s[:, :2], s, None, 4, 128)
    with pytest.raises(ValueError, match="zeros"):
        G.dequant_linear(x, codes, s, s.half(), None, 4, 128)
    with pytest.raises(ValueError, match="perm"):
        G.dequant_linear(x, codes, s, s, torch.zeros(512), 4, 128)
    with pytest.raises(ValueError, match="device tensor"):
        G.dequant_linear_backward(torch.zeros(2, 4), codes, s, s, None, 4, 128)
    with pytest.raises(ValueError, match="router"):
        G.dequant_moe(x, torch.zeros(0, 512), (codes, s, s), (codes, s, s), None, 4, 128, 1)


def test_stack_experts_folds_the_down_order_into_the_rows():
    """h = (x Wg^T) * (x Wu^T), y = h Wd^T from the stacked layout equals it from the separate layers."""
    rng = np.random.default_rng(5)
    H, I, bits, g = 256, 128, 4, 64

    def layer(m, n, perm):
        codes = rng.integers(0, 16, (m, n))
        s, z = rng.uniform(0.01, 0.02, (m, n // g)).astype(np.float32), rng.integers(0, 16, (m, n // g)).astype(np.float32)
        d = {"codes": torch.from_numpy(O.pack_codes(codes, bits).view(np.int32)), "scales": torch.from_numpy(s),
             "zeros": torch.from_numpy(z), "perm": None if perm is None else torch.from_numpy(perm.astype(np.int32))}
        return d, (codes - np.repeat(z, g, 1)) * np.repeat(s, g, 1).astype(np.float64)

    def w64(codes, s, z):
        c = O.unpack_codes(codes.numpy().view(np.uint32), codes.shape[1] * 8, bits)
        return (c - np.repeat(z.numpy(), g, 1)) * np.repeat(s.numpy(), g, 1).astype(np.float64)

    x = rng.normal(0, 1, (3, H))
    gates, ups, downs, want = [], [], [], []
    for _ in range(2):
        pi, pd = rng.permutation(H), rng.permutation(I)
        (gd, wg), (ud, wu), (dd, wd) = layer(I, H, pi), layer(I, H, pi), layer(H, I, pd)
        gates.append(gd), ups.append(ud), downs.append(dd)
        want.append(((x[:, pi] @ wg.T) * (x[:, pi] @ wu.T))[:, pd] @ wd.T)
    gu, dn, perm = G.stack_experts(gates, ups, downs)
    for e in range(2):
        a = x[:, perm[e].numpy()] @ w64(*[t[e] for t in gu]).T
        y = (a[:, :I] * a[:, I:]) @ w64(*[t[e] for t in dn]).T
        assert np.allclose(y, want[e], rtol=1e-12, atol=1e-12)
    ups[1] = dict(ups[1], perm=torch.flip(ups[1]["perm"], [0]))
    with pytest.raises(ValueError, match="different input orders"):
        G.stack_experts(gates, ups, downs)
    with pytest.raises(ValueError, match="one entry per expert"):
        G.stack_experts(gates, ups[:1], downs)
    mixed = [dict(d, perm=None) if e else d for e, d in enumerate(gates)]
    with pytest.raises(ValueError, match="every expert|different"):
        G.stack_experts(mixed, [dict(d, perm=None) if e else gates[0] for e, d in enumerate(gates)], downs)


def test_stack_experts_refuses_layers_with_a_channel_scale():
    """Codes of a channel-scaled weight (AWQ) are not those of the weight: no expert may have them."""
    codes, s = torch.zeros(128, 16, dtype=torch.int32), torch.ones(128, 1)
    plain = {"codes": codes, "scales": s, "zeros": s}
    one = dict(plain, channel_scale=torch.ones(128))
    scaled = dict(plain, channel_scale=torch.cat([torch.ones(127), torch.full((1,), 2.0)]))
    gu, dn, perm = G.stack_experts([plain, one], [plain, one], [one, plain])
    assert gu[0].shape == (2, 256, 16) and dn[0].shape == (2, 128, 16) and perm is None
    for at, name in enumerate(("gate", "up", "down")):
        for e in range(2):
            parts = [[plain, plain] for _ in range(3)]
            parts[at][e] = scaled
            with pytest.raises(ValueError, match=f"expert {e}: {name} has a channel_scale"):
                G.stack_experts(*parts)


def test_gradient_of_no_tokens_without_an_address(L):
    """An empty dX, as an allocator hands it out, has no address: nothing to do, not a missing output."""
    assert backward(L, T=0, dY=0, dX=0, ws=0) == G.OK
    assert backward(L, T=0, dY=0, dX=0, ws=0, act=3, dtype=1) == G.OK
    assert backward(L, T=1, dX=0) == G.ERR_ARG


def test_argument_blocks_hold_every_field_where_c_does():
    """A distinct value for each field of the binding's argument blocks, read back at the offset and with the
    type that the header's declaration gives it."""
    text = re.sub(r"/\*.*?\*/", "", open(G.HEADER).read(), flags=re.S)
    scalars = {"int64_t": "q", "size_t": "Q", "int": "i", "double": "d"}

    def fields(name):
        """[(member, offset, format)] of the flattened structure, its size and its alignment"""
        out, off, most = [], 0, 1
        for decl in re.search(r"typedef struct \{([^}]*)\} %s;" % name, text).group(1).split(";"):
            if not decl.split():
                continue
            base, rest = re.match(r"\s*(?:const\s+)?(\w+)(.*)", decl, re.S).groups()
            for var in rest.split(","):
                if "*" in var or base in scalars:
                    kind = "Q" if "*" in var else scalars[base]
                    sub, size, al = [("", 0, kind)], struct.calcsize(kind), struct.calcsize(kind)
                else:
                    sub, size, al = fields(base)
                off = -(-off // al) * al
                out += [(var.strip(" *\n") + "." + n, off + o, k) for n, o, k in sub]
                off, most = off + size, max(most, al)
        return out, -(-off // most) * most, most

    for name, fmt in (("gptq_linear_args", G._LINEAR_ARGS), ("gptq_linear_grad_args", G._LINEAR_GRAD_ARGS),
                      ("gptq_moe_args", G._MOE_ARGS)):
        want, size, _ = fields(name)
        assert size == fmt.size, name
        block = fmt.pack(*range(101, 101 + len(want)))                        # (as many values as C has members)
        for value, (member, offset, kind) in enumerate(want, 101):
            assert struct.unpack_from("@" + kind, block, offset)[0] == value, (name, member)
