"""The layers as torch.cuda.make_graphed_callables captures them: forward and backward in
graphs of their own, inside an eager training loop."""
import pytest
import torch

from tests._gpu import needs_gpu, say

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.mark.parametrize("base", ["nf4", "mx4"])
@pytest.mark.parametrize("act8", [False, True])
def test_graphed_layer(base, act8):
    import quantized_fine_tuning_nf4_amd as qn
    say(f"[graphed layer] {base} act8={act8}")
    torch.manual_seed(0)
    W = torch.randn(72, 128, device="cuda") * 0.1
    layers = []
    for _ in range(2):
        torch.manual_seed(1)
        lin = qn.QLoRALinear(W, r=8, alpha=16.0, act8=act8, base=base)
        with torch.no_grad():
            lin.lora_B.normal_(std=0.1)
        layers.append(lin)
    eager, graphed = layers
    sample = torch.randn(40, 128, device="cuda").to(torch.bfloat16).requires_grad_()
    call = torch.cuda.make_graphed_callables(graphed, (sample,))
    for k in range(3):
        g = torch.Generator(device="cuda").manual_seed(20 + k)
        x = torch.randn(40, 128, generator=g, device="cuda").to(torch.bfloat16)
        dy = torch.randn(40, 72, generator=g, device="cuda").to(torch.bfloat16)
        got = []
        for f, lin in ((eager, eager), (call, graphed)):
            v = x.clone().requires_grad_()
            y = f(v)
            y.backward(dy)
            torch.cuda.synchronize()
            got.append([y.detach().clone(), v.grad.clone()] + [p.grad.clone()
                                                              for p in lin.parameters()])
            for p in lin.parameters():
                p.grad = None
        for a, b in zip(*got):
            assert torch.equal(a, b)
