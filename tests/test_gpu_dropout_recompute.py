"""Dropout in layers whose forward is run again for the backward (activation checkpointing):
without a seed the gradients are those of the mask that the loss saw; a seeded layer
raises instead of drawing another."""
import pytest
import torch
from torch.utils.checkpoint import checkpoint

from tests._gpu import needs_gpu, say

pytestmark = [pytest.mark.gpu, needs_gpu]


def _layer(qn, base, act8, **kw):
    torch.manual_seed(0)
    lin = qn.QLoRALinear(torch.randn(72, 128, device="cuda") * 0.1, r=8, alpha=16.0, dropout=0.3,
                         act8=act8, base=base, **kw)
    with torch.no_grad():
        lin.lora_B.normal_(std=0.1)
    return lin


def _grads(lin, x, g, call):
    x = x.clone().requires_grad_()
    y = call(x)
    torch.rand(1), torch.rand(1, device="cuda")  # both generators move on before the backward
    y.backward(g)
    out = [y.detach(), x.grad] + [p.grad for p in lin.parameters()]
    for p in lin.parameters():
        p.grad = None
    return out


@pytest.mark.parametrize("base", ["nf4", "mx4"])
@pytest.mark.parametrize("act8", [False, True])
@pytest.mark.parametrize("reentrant", [False, True])
def test_recomputed_without_a_seed(base, act8, reentrant):
    import quantized_fine_tuning_nf4_amd as qn
    say(f"[recompute] {base} act8={act8} reentrant={reentrant}")
    lin = _layer(qn, base, act8)
    x = torch.randn(40, 128, device="cuda").to(torch.bfloat16)
    g = torch.randn(40, 72, device="cuda").to(torch.bfloat16)
    torch.manual_seed(5)
    want = _grads(lin, x, g, lin)
    torch.manual_seed(5)
    got = _grads(lin, x, g, lambda v: checkpoint(lin, v, use_reentrant=reentrant))
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    again = _grads(lin, x, g, lin)  # the next forward's mask is another
    assert not torch.equal(again[0], want[0]) and not torch.equal(again[2], want[2])
    lin.eval()
    with torch.no_grad():
        assert torch.equal(lin(x), lin(x))


@pytest.mark.parametrize("base", ["nf4", "mx4"])
@pytest.mark.parametrize("reentrant", [False, True])
def test_recomputed_under_a_seed(base, reentrant):
    import quantized_fine_tuning_nf4_amd as qn
    say(f"[recompute seeded] {base} reentrant={reentrant}")
    lin = _layer(qn, base, False, seed=3)
    x = torch.randn(40, 128, device="cuda").to(torch.bfloat16).requires_grad_()
    y = checkpoint(lin, x, use_reentrant=reentrant)
    with pytest.raises(RuntimeError, match="give the layer no seed"):
        y.backward(torch.ones_like(y))
    assert lin.lora_A.grad is None and lin.draws == 1
    lin.eval()  # no mask: nothing to repeat
    y = checkpoint(lin, x, use_reentrant=reentrant)
    y.backward(torch.ones_like(y))
    assert lin.lora_B.grad is not None


def test_seeds_are_checked_where_the_layer_is_made():
    import quantized_fine_tuning_nf4_amd as qn
    say("[recompute seeds]")
    W = torch.randn(8, 64, device="cuda")
    for kw in (dict(seed=-1), dict(seed=1 << 64), dict(seed=1, step=torch.zeros(2, device="cuda")),
               dict(step=torch.zeros(1, dtype=torch.int64, device="cuda"))):
        with pytest.raises(ValueError):
            qn.QLoRALinear(W, r=4, dropout=0.1, **kw)


def test_captured_without_a_seed():
    """A key drawn by the host at the capture would be every replay's."""
    import quantized_fine_tuning_nf4_amd as qn
    say("[recompute capture]")
    lin = _layer(qn, "mx4", False)
    x = torch.randn(40, 128, device="cuda").to(torch.bfloat16)
    with torch.no_grad():
        lin(x)
        torch.cuda.synchronize()
        with pytest.raises(RuntimeError, match="a seed and a step"):
            with torch.cuda.graph(torch.cuda.CUDAGraph()):
                lin(x)
        lin.eval()
        lin(x)
    torch.cuda.synchronize()
