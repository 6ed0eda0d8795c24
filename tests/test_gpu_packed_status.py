"""What a caller learns of a bounded wait that ran out in an operator on packed weights.  The wait is not made
to run out: its bit is written into the status word, or the library's check is replaced on the host."""
import pytest
import torch

from post_weight_quantization_16_b200 import gptq as G
from tests.test_gpu_threads import DEV, Layer

pytestmark = pytest.mark.gpu
TIMEOUT_BIT = 2


def calls():
    w, gu, dn = Layer(300, 256, 4, 64, 1), Layer(256, 256, 4, 64, 2, (4,)), Layer(256, 128, 4, 64, 3, (4,))
    x, dy = torch.randn(20, 256, device=DEV).half(), torch.randn(20, 300, device=DEV).half()
    r = torch.randn(4, 256, device=DEV).half()
    return {"linear": lambda n=20, **kw: G.dequant_linear(x[:n], *w.parts, None, 4, 64, **kw),
            "linear_backward": lambda n=20, **kw: G.dequant_linear_backward(dy[:n], *w.parts, None, 4, 64, **kw),
            "moe": lambda n=20, **kw: G.dequant_moe(x[:n], r, gu.parts, dn.parts, None, 4, 64, 2, **kw)}


def test_a_status_word_with_the_timeout_bit_raises_and_the_next_call_clears_it():
    ws = torch.empty(1 << 22, dtype=torch.uint8, device=DEV)
    for name, call in calls().items():
        ws.fill_(255)
        call(workspace=ws)
        G.check_workspace(ws)
        ws[0] = TIMEOUT_BIT
        with pytest.raises(G.GPTQError) as e:
            G.check_workspace(ws)
        assert e.value.status == G.ERR_TIMEOUT, name
        call(workspace=ws, check=True)
        G.check_workspace(ws)
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream(DEV))
    call(workspace=ws, stream=side, check=True)
    G.check_workspace(ws, side)


def test_check_asks_after_every_call_with_tokens(monkeypatch):
    L = G.lib()
    asked = []

    def check(workspace, device, stream):
        asked.append(device)
        return G.ERR_TIMEOUT

    monkeypatch.setattr(L, "gptq_dequant_matmul_check", check)
    for name, call in calls().items():
        call()
        assert not asked
        with pytest.raises(G.GPTQError) as e:
            call(check=True)
        assert e.value.status == G.ERR_TIMEOUT and asked == [0], name
        asked.clear()
        call(0, check=True)
        assert not asked
        side = torch.cuda.Stream(DEV)
        with pytest.raises(G.GPTQError):
            call(check=True, stream=side)
        asked.clear()


def test_what_is_not_a_workspace_is_refused():
    for bad in (torch.zeros(1024, dtype=torch.uint8), torch.zeros(1024, device=DEV), torch.zeros(10, dtype=torch.uint8, device=DEV)):
        with pytest.raises(ValueError, match="workspace"):
            G.check_workspace(bad)
