"""Cases that time and check the operators on packed weights: the linear layer with its epilogue
(gptq.dequant_linear), its gradient (gptq.dequant_linear_backward) and the mixture-of-experts layer
for a few tokens (gptq.dequant_moe).

run() computes a case either from elementary torch operations in 32 bits (own = False: the plain
form) or with the library's calls (own = True), on the same inputs; exact() computes it in 64 bits.
All three follow the same definition:

    W[r][k] = (code[r][k] - zero[r][k / g]) * scale[r][k / g]          (sweep order k, code LSB-first)
    linear    Z = X[:, perm] W^T + bias,  Y = act(Z) + residual
    backward  dZ = dY * act'(Z),  dX[:, perm] = dZ W,  dbias = sum over tokens of dZ
    moe       p = softmax(X R^T), the top_k largest per token (ties to the lowest expert), weights p
              (divided by their sum where renormalize), h = silu(x Wg^T) * (x Wu^T) and
              y = sum of weight * h Wd^T over the token's experts, + residual
"""
import torch

own = False

ACT = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}
DTYPE = {"fp16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda"


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------
def _linear(name, T, m, n, bits, group, dtype, act="none", bias=False, residual=False, perm=True, sym=False,
            out_fp32=False, preact=False):
    c = {"op": "linear", "T": T, "m": m, "n": n, "bits": bits, "group": group, "dtype": dtype, "act": act,
         "bias": bias, "residual": residual, "perm": perm, "sym": sym, "out_fp32": out_fp32, "preact": preact}
    return c if name is None else {"name": name, **c}


def _backward(name, T, m, n, bits, group, dtype, act="none", bias=False, perm=True, sym=False):
    c = {"op": "backward", "T": T, "m": m, "n": n, "bits": bits, "group": group, "dtype": dtype, "act": act,
         "bias": bias, "perm": perm, "sym": sym}
    return c if name is None else {"name": name, **c}


def _moe(name, T, E, top_k, H, I, bits, group, dtype, renorm=True, residual=False, perm=True):
    c = {"op": "moe", "T": T, "E": E, "top_k": top_k, "H": H, "I": I, "bits": bits, "group": group,
         "dtype": dtype, "renorm": renorm, "residual": residual, "perm": perm}
    return c if name is None else {"name": name, **c}


def listed():
    return [
        # one user decoding one token: the attention projection of the 4096-wide layer, act-order
        _linear("linear_t1_qproj", 1, 4096, 4096, 4, 128, "fp16"),
        # sixteen users decoding: the MLP's down projection, symmetric codes, added to the residual stream
        _linear("linear_t16_down", 16, 4096, 11008, 4, 128, "bf16", residual=True, sym=True),
        # a short speculative window on an 8-bit per-channel layer (an output head's slice with an odd number
        # of rows, its scores kept in fp32)
        _linear("linear_t5_head_8bit", 5, 1031, 4096, 8, -1, "bf16", act="gelu", bias=True, perm=False,
                out_fp32=True),
        # a ragged prompt chunk through the up projection at 3 bits, groups of 64
        _linear("linear_t77_up_3bit", 77, 11008, 4096, 3, 64, "fp16", act="silu", bias=True),
        # a prompt of 2048 tokens through the same layer, its pre-activation kept for the backward pass
        _linear("linear_t2048_up", 2048, 11008, 4096, 4, 128, "bf16", act="silu", bias=True, preact=True),
        # the largest: a 4096-token prompt through the 70B-shaped down projection
        _linear("linear_t4096_70b", 4096, 8192, 28672, 4, 128, "fp16", residual=True),
        # gradient through the frozen attention projection, a ragged batch of 500 tokens
        _backward("backward_t500_qproj", 500, 4096, 4096, 4, 128, "bf16"),
        # gradient through a small 2-bit layer with odd sizes, narrow groups, ReLU and a trained bias
        _backward("backward_t1023_2bit", 1023, 1000, 2048, 2, 32, "fp16", act="relu", bias=True, perm=False),
        # gradient through the up projection for a 4096-token batch
        _backward("backward_t4096_up", 4096, 11008, 4096, 4, 128, "bf16", act="silu", bias=True),
        # one token through a layer of many small experts, groups of 64
        _moe("moe_t1_e32", 1, 32, 4, 2048, 1024, 4, 64, "bf16", perm=False),
        # a batch of 33 tokens over 64 small experts at 3 bits, act-order
        _moe("moe_t33_e64_3bit", 33, 64, 8, 2048, 768, 3, 64, "fp16", renorm=False),
        # 48 tokens over eight experts of the 7B MLP's size: every expert's weights are read
        _moe("moe_t48_e8_large", 48, 8, 2, 4096, 11008, 4, 128, "bf16", residual=True),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["linear", "linear", "backward", "moe", "moe"])
    bits = rng.choice([2, 3, 4, 4, 4, 8])
    dtype = rng.choice(["fp16", "bf16"])
    flag = lambda: rng.random() < 0.5  # noqa: E731
    if op == "moe":
        E = _log(rng, 4, 64)
        H, I = 128 * _log(rng, 2, 32), 128 * _log(rng, 1, 40)
        E = max(4, min(E, 8 * 4096 * 11008 // (H * I)))
        group = rng.choice([g for g in (32, 64, 128, 256, -1) if g == -1 or (H % g == 0 and I % g == 0)])
        return _moe(None, _log(rng, 1, 64), E, min(E, rng.randint(1, 8)), H, I, bits, group, dtype, flag(), flag(),
                    flag())
    n = 128 * _log(rng, 1, 86)
    group = rng.choice([g for g in (32, 64, 128, 256, -1) if g == -1 or n % g == 0])
    act = rng.choice(list(ACT))
    m = _log(rng, 16, 11008)
    if op == "linear":
        return _linear(None, _log(rng, 1, 4096), m, n, bits, group, dtype, act, flag(), flag(), flag(), flag(),
                       rng.random() < 0.25, rng.random() < 0.25)
    return _backward(None, _log(rng, 16, 4096), m, n, bits, group, dtype, act, flag(), flag(), flag())


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------
def _pack(u, bits):
    """Codes [..., n] (int32) as LSB-first words [..., n * bits / 32]: 32 codes fill `bits` words."""
    *lead, n = u.shape
    if bits != 3:
        per = 32 // bits
        shifts = torch.arange(per, device=u.device, dtype=torch.int32) * bits
        return (u.view(*lead, n // per, per) << shifts).sum(-1, dtype=torch.int32)
    v = u.view(*lead, n // 32, 32).to(torch.int64)
    words = []
    for j in range(3):
        at = [(c, 3 * c - 32 * j) for c in range(32) if 3 * c < 32 * j + 32 and 3 * c + 3 > 32 * j]
        word = sum(((v[..., c] << s) if s >= 0 else (v[..., c] >> -s)) for c, s in at) & 0xFFFFFFFF
        words.append(torch.where(word >= 2 ** 31, word - 2 ** 32, word).to(torch.int32))
    return torch.stack(words, -1).view(*lead, n * 3 // 32)


def _weights(gen, m, n, bits, group, sym):
    """A packed layer as quantization leaves it: bell-shaped codes around each group's zero-point."""
    g = n if group == -1 else group
    levels = 2 ** bits
    u = torch.randn(m, n, generator=gen, device=DEV).mul_(levels / 6).add_((levels - 1) / 2).round_()
    codes = _pack(u.clamp_(0, levels - 1).to(torch.int32), bits)
    del u
    scales = (torch.rand(m, n // g, generator=gen, device=DEV) * 0.6 + 0.7) * (0.12 / levels)
    if sym:
        zeros = torch.full((m, n // g), float(levels // 2), device=DEV)
    else:
        zeros = torch.randn(m, n // g, generator=gen, device=DEV).mul_(0.08 * levels).add_((levels - 1) / 2)
        zeros = zeros.round_().clamp_(0, levels - 1)
    return codes, scales, zeros


def _activations(gen, T, n, dtype, factor):
    """Normal activations with half a percent of outlier channels."""
    x = torch.randn(T, n, generator=gen, device=DEV)
    x[:, torch.randperm(n, generator=gen, device=DEV)[: max(1, n // 200)]] *= factor
    return x.to(dtype)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt = DTYPE[c["dtype"]]
    s = {"case": c}
    perm = lambda n: torch.randperm(n, generator=gen, device=DEV).to(torch.int32)  # noqa: E731
    if c["op"] == "moe":
        T, E, H, I = c["T"], c["E"], c["H"], c["I"]
        s["x"] = _activations(gen, T, H, dt, 5.0)
        s["router"] = (torch.randn(E, H, generator=gen, device=DEV) * (1.5 / H ** 0.5)).to(dt)
        parts = [_weights(gen, 2 * I, H, c["bits"], c["group"], False) for _ in range(E)]
        s["gate_up"] = [torch.stack(p) for p in zip(*parts)]
        parts = [_weights(gen, H, I, c["bits"], c["group"], False) for _ in range(E)]
        s["down"] = [torch.stack(p) for p in zip(*parts)]
        s["perm"] = torch.stack([perm(H) for _ in range(E)]) if c["perm"] else None
        s["residual"] = torch.randn(T, H, generator=gen, device=DEV).to(dt) if c["residual"] else None
        return s
    T, m, n = c["T"], c["m"], c["n"]
    s["w"] = _weights(gen, m, n, c["bits"], c["group"], c["sym"])
    s["perm"] = perm(n) if c["perm"] else None
    if c["op"] == "linear":
        s["x"] = _activations(gen, T, n, dt, 30.0)
        s["bias"] = torch.randn(m, generator=gen, device=DEV).to(dt) if c["bias"] else None
        s["residual"] = torch.randn(T, m, generator=gen, device=DEV).to(dt) if c["residual"] else None
    else:
        s["dy"] = torch.randn(T, m, generator=gen, device=DEV).to(dt)
        s["z"] = (torch.randn(T, m, generator=gen, device=DEV) * 1.5).to(dt) if c["act"] != "none" else None
    return s


# ------------------------------------------------------------------------------------------
# the plain form (own = False) and the library's calls (own = True)
# ------------------------------------------------------------------------------------------
def _dequant(codes, scales, zeros, bits):
    """fp32 [..., n] in sweep order."""
    *lead, words = codes.shape
    n = words * 32 // bits
    if bits != 3:
        shifts = torch.arange(32 // bits, device=codes.device, dtype=torch.int32) * bits
        u = (codes[..., None] >> shifts) & (2 ** bits - 1)
    else:
        w = (codes.to(torch.int64) & 0xFFFFFFFF).view(*lead, n // 32, 3)
        at = torch.arange(32, device=codes.device) * 3
        lo, hi = w[..., at // 32], w[..., torch.clamp(at // 32 + 1, max=2)]
        u = ((lo | (hi << 32)) >> (at % 32)) & 7
    G = scales.shape[-1]
    return ((u.view(*lead, G, n // G).float() - zeros[..., None]) * scales[..., None]).view(*lead, n)


def _act(z, name):
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, name):
    if name == "relu":
        return (z > 0).float()
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (0.5 / torch.pi) ** 0.5
    sig = 1 / (1 + torch.exp(-z))
    return sig * (1 + z * (1 - sig))


def _plain_linear(s, c):
    dt = DTYPE[c["dtype"]]
    x = s["x"].float()
    x = x if s["perm"] is None else x[:, s["perm"]]
    z = x @ _dequant(*s["w"], c["bits"]).t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(z, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    y = y if c["out_fp32"] else y.to(dt)
    return (y, z.to(dt)) if c["preact"] else y


def _plain_backward(s, c):
    dz = s["dy"].float()
    if c["act"] != "none":
        dz = dz * _act_grad(s["z"].float(), c["act"])
    d = dz @ _dequant(*s["w"], c["bits"])
    dx = d
    if s["perm"] is not None:
        dx = torch.empty_like(d)
        dx[:, s["perm"]] = d
    dx = dx.to(DTYPE[c["dtype"]])
    return (dx, dz.sum(0)) if c["bias"] else dx


def _plain_moe(s, c):
    x = s["x"].float()
    T, E, k = c["T"], c["E"], c["top_k"]
    logits = s["x"].double() @ s["router"].double().t()  # 64 bits: a choice stands next to a border
    p = torch.exp(logits - logits.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True)
    top, ids = torch.sort(p, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    w = (top / top.sum(1, keepdim=True) if c["renorm"] else top).float()
    xe = x[None].expand(E, T, c["H"]) if s["perm"] is None else x[:, s["perm"]].transpose(0, 1)
    gu = torch.bmm(xe, _dequant(*s["gate_up"], c["bits"]).transpose(1, 2))
    h = _act(gu[..., : c["I"]], "silu") * gu[..., c["I"]:]
    d = torch.bmm(h, _dequant(*s["down"], c["bits"]).transpose(1, 2))
    share = torch.zeros(T, E, device=x.device).scatter_(1, ids, w)
    y = (share.t()[..., None] * d).sum(0)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(DTYPE[c["dtype"]]), ids.to(torch.int32), w


def _library(s, c):
    from post_weight_quantization_16_b200 import gptq as G

    if c["op"] == "linear":
        return G.dequant_linear(s["x"], *s["w"], s["perm"], c["bits"], c["group"], bias=s["bias"], act=ACT[c["act"]],
                                residual=s["residual"], out_dtype=torch.float32 if c["out_fp32"] else None,
                                want_preact=c["preact"])
    if c["op"] == "backward":
        return G.dequant_linear_backward(s["dy"], *s["w"], s["perm"], c["bits"], c["group"], act=ACT[c["act"]],
                                         preact=s["z"], want_dbias=c["bias"])
    return G.dequant_moe(s["x"], s["router"], s["gate_up"], s["down"], s["perm"], c["bits"], c["group"], c["top_k"],
                         renormalize=c["renorm"], residual=s["residual"])


def run(state):
    c = state["case"]
    if own:
        return _library(state, c)
    return {"linear": _plain_linear, "backward": _plain_backward, "moe": _plain_moe}[c["op"]](state, c)


# ------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------
def _packed_bytes(m, n, bits, group):
    return m * n * bits / 8 + 8 * m * (1 if group == -1 else n // group)


def work(case):
    c = case
    if c["op"] == "moe":
        T, E, H, I = c["T"], c["E"], c["H"], c["I"]
        # experts that get a token: all pairs on different experts at best, every expert when tokens are many
        active = E * (1 - (1 - c["top_k"] / E) ** T)
        expert = _packed_bytes(2 * I, H, c["bits"], c["group"]) + _packed_bytes(H, I, c["bits"], c["group"])
        expert += 4 * H if c["perm"] else 0
        bytes_ = active * expert + 2 * E * H + 2 * T * H * (3 if c["residual"] else 2) + 8 * T * c["top_k"]
        return {"bytes": bytes_, "flops": 2.0 * T * E * H + 6.0 * T * c["top_k"] * H * I}
    T, m, n = c["T"], c["m"], c["n"]
    bytes_ = _packed_bytes(m, n, c["bits"], c["group"]) + (4 * n if c["perm"] else 0)
    if c["op"] == "linear":
        bytes_ += 2 * T * n + (4 if c["out_fp32"] else 2) * T * m + (2 * m if c["bias"] else 0)
        bytes_ += 2 * T * m * (int(c["residual"]) + int(c["preact"]))
    else:
        bytes_ += 2 * T * m * (2 if c["act"] != "none" else 1) + 2 * T * n + (4 * m if c["bias"] else 0)
    return {"bytes": float(bytes_), "flops": 2.0 * T * m * n}


# ------------------------------------------------------------------------------------------
# the definition in 64 bits
# ------------------------------------------------------------------------------------------
def _exact_weights(codes, scales, zeros, bits):
    """fp64 [m, n] by the definition of the bit stream: bit b of code k is bit k * bits + b of the row."""
    m, words = codes.shape
    n = words * 32 // bits
    stream = torch.empty(m, words * 4, dtype=torch.uint8, device=codes.device)
    for byte in range(4):
        stream[:, byte::4] = (codes >> (8 * byte)).bitwise_and_(255).to(torch.uint8)
    one = torch.stack([(stream >> b) & 1 for b in range(8)], -1).view(m, n, bits)
    u = torch.zeros(m, n, dtype=torch.float64, device=codes.device)
    for b in range(bits):
        u += one[..., b].double() * 2.0 ** b
    g = n // scales.shape[1]
    u -= zeros.double().repeat_interleave(g, 1)
    u *= scales.double().repeat_interleave(g, 1)
    return u


def _exact_product(x, w, bits, rows=1024):
    """x W^T, the rows of W dequantized in blocks."""
    codes, scales, zeros = w
    return torch.cat([x @ _exact_weights(codes[i:i + rows], scales[i:i + rows], zeros[i:i + rows], bits).t()
                      for i in range(0, codes.shape[0], rows)], 1)


def _exact_act(z, name):
    import torch.nn.functional as F

    return {"none": lambda v: v, "relu": F.relu, "gelu": F.gelu, "silu": F.silu}[name](z)


def _exact_linear(s, c):
    x = s["x"].double()
    if s["perm"] is not None:
        x = x.index_select(1, s["perm"].long())
    z = _exact_product(x, s["w"], c["bits"])
    if s["bias"] is not None:
        z += s["bias"].double()
    y = _exact_act(z, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].double()
    return (y, z) if c["preact"] else y


def _exact_backward(s, c):
    dz = s["dy"].double()
    if c["act"] != "none":
        z = s["z"].double().requires_grad_(True)
        dz, = torch.autograd.grad(_exact_act(z, c["act"]), z, dz)
    codes, scales, zeros = s["w"]
    dx = torch.zeros(c["T"], c["n"], dtype=torch.float64, device=DEV)
    for i in range(0, c["m"], 1024):
        r = slice(i, i + 1024)
        dx += dz[:, r] @ _exact_weights(codes[r], scales[r], zeros[r], c["bits"])
    if s["perm"] is not None:
        inverse = torch.argsort(s["perm"].long())
        dx = dx.index_select(1, inverse)
    return (dx, dz.sum(0)) if c["bias"] else dx


def _exact_moe(s, c):
    x = s["x"].double()
    p = torch.softmax(x @ s["router"].double().t(), 1)
    y = torch.zeros(c["T"], c["H"], dtype=torch.float64, device=DEV) if s["residual"] is None \
        else s["residual"].double()
    ids = torch.zeros(c["T"], c["top_k"], dtype=torch.int64, device=DEV)
    w = torch.zeros(c["T"], c["top_k"], dtype=torch.float64, device=DEV)
    left = p.clone()
    for j in range(c["top_k"]):  # the first of the largest that are left
        best = left.amax(1, keepdim=True)
        ids[:, j] = (left == best).to(torch.int64).argmax(1)
        w[:, j] = best[:, 0]
        left.scatter_(1, ids[:, j:j + 1], -1.0)
    if c["renorm"]:
        w /= w.sum(1, keepdim=True)
    for e in range(c["E"]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            xe = x[t] if s["perm"] is None else x[t].index_select(1, s["perm"][e].long())
            gu = _exact_product(xe, [v[e] for v in s["gate_up"]], c["bits"])
            h = _exact_act(gu[:, : c["I"]], "silu") * gu[:, c["I"]:]
            y.index_add_(0, t, w[t, j, None] * _exact_product(h, [v[e] for v in s["down"]], c["bits"]))
    return y, ids.to(torch.int32), w


def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _exact_linear, "backward": _exact_backward, "moe": _exact_moe}[case["op"]](s, case)
