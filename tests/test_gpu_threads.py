"""The entry points called from a host thread that has done nothing with CUDA yet: the call itself has to
bind the device's context before its first driver call (the encoding of a tensor map).  The threads make
the C calls alone; tensors, streams and workspaces come from the main thread."""
import threading

import pytest
import torch

from post_weight_quantization_16_b200 import gptq as G

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def in_fresh_thread(call):
    got = []
    t = threading.Thread(target=lambda: got.append(call()))
    t.start()
    t.join()
    torch.cuda.synchronize()
    return got[0]


class Layer:
    def __init__(self, m, n, bits, g, seed, experts=()):
        gen = torch.Generator(device=DEV)
        gen.manual_seed(seed)
        self.m, self.n, self.bits, self.g = m, n, bits, g
        self.codes = torch.randint(-(1 << 31), 1 << 31, (*experts, m, n * bits // 32), generator=gen, device=DEV).to(torch.int32)
        self.scales = torch.rand((*experts, m, n // g), generator=gen, device=DEV) * 0.02
        self.zeros = torch.randint(0, 1 << bits, (*experts, m, n // g), generator=gen, device=DEV).float()
        self.parts = (self.codes, self.scales, self.zeros)
        self.fields = (self.codes.data_ptr(), self.scales.data_ptr(), self.zeros.data_ptr(), 0, m, n, bits, g, 0)


@pytest.mark.parametrize("T,m", [(4, 64), (40, 64), (300, 9473)])
def test_linear_and_gradient(T, m):
    """The three kernels of the linear layer; the gradient without an activation, whose first driver call is
    the tensor map."""
    w = Layer(m, 256, 4, 64, T)
    x = torch.randn(T, 256, device=DEV).half()
    y, dx = torch.empty(T, m, device=DEV).half(), torch.empty(T, 256, device=DEV).half()
    need = G.lib().gptq_dequant_linear_backward_workspace_bytes(T, m, 256, 0, 0, 0)
    ws = torch.empty(max(1 << 20, need), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    a = G._LINEAR_ARGS.pack(x.data_ptr(), T, 256, 0, *w.fields, 0, 0, 0, 0, y.data_ptr(), m, 0, 0, ws.data_ptr(), ws.numel())
    assert in_fresh_thread(lambda: G.lib().gptq_dequant_linear(a, 0, None)) == G.OK
    assert torch.equal(y, G.dequant_linear(x, *w.parts, None, 4, 64))
    b = G._LINEAR_GRAD_ARGS.pack(y.data_ptr(), T, m, 0, *w.fields, 0, 0, dx.data_ptr(), 256, 0, ws.data_ptr(), ws.numel())
    assert in_fresh_thread(lambda: G.lib().gptq_dequant_linear_backward(b, 0, None)) == G.OK
    assert torch.equal(dx, G.dequant_linear_backward(y, *w.parts, None, 4, 64))


def test_experts():
    T, E, H, inner = 5, 4, 256, 128
    gu, dn = Layer(2 * inner, H, 4, 64, 1, (E,)), Layer(H, inner, 4, 64, 2, (E,))
    x, r = torch.randn(T, H, device=DEV).half(), torch.randn(E, H, device=DEV).half()
    y = torch.empty(T, H, device=DEV).half()
    ws = torch.empty(G.lib().gptq_dequant_moe_workspace_bytes(T, E, 2, H, inner), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    a = G._MOE_ARGS.pack(x.data_ptr(), T, H, 0, r.data_ptr(), E, 2, 1, G.ACT_SILU, *gu.fields, *dn.fields, 0, 0,
                         y.data_ptr(), H, 0, 0, ws.data_ptr(), ws.numel())
    assert in_fresh_thread(lambda: G.lib().gptq_dequant_moe(a, 0, None)) == G.OK
    assert torch.equal(y, G.dequant_moe(x, r, gu.parts, dn.parts, None, 4, 64, 2)[0])


def test_hessian():
    x = torch.randn(512, 256, device=DEV).bfloat16()
    with G.GPTQContext(256, 64, 0) as here, G.GPTQContext(256, 64, 0) as there:
        here.accumulate_hessian(x)
        in_fresh_thread(lambda: there.accumulate_hessian(x) or True)
        assert torch.equal(here.get_hessian()[0], there.get_hessian()[0])


def test_dequant_matmul():
    w = Layer(64, 256, 4, 64, 7)
    x = torch.randn(16, 256, device=DEV).half()
    want = G.dequant_matmul(x, *w.parts, None, 4, 64)
    out = torch.empty_like(want)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device=DEV)
    stream = torch.cuda.current_stream(DEV)
    torch.cuda.synchronize()
    in_fresh_thread(lambda: G.dequant_matmul(x, *w.parts, None, 4, 64, out=out, workspace=ws, stream=stream))
    assert torch.equal(out, want)
