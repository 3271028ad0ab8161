"""A run that goes on from a state dict draws the masks that the run it came from would have
drawn next, alone and inside another module; state dicts without the count load as before."""
import pytest
import torch

from tests._gpu import needs_gpu, say

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.mark.parametrize("base", ["nf4", "mx4"])
def test_resumed(base):
    import quantized_fine_tuning_nf4_amd as qn
    say(f"[drop resume] {base}")
    torch.manual_seed(0)
    W = torch.randn(72, 128, device="cuda") * 0.1
    make = lambda **kw: qn.QLoRALinear(W, r=8, dropout=0.3, base=base, **kw)  # noqa: E731
    x = torch.randn(40, 128, device="cuda").to(torch.bfloat16)
    a = make(seed=5)
    with torch.no_grad():
        a.lora_B.normal_()
        first = [a(x), a(x)]
        state = {k: v.clone() for k, v in a.state_dict().items()}
        assert sorted(state) == ["draws", "lora_A", "lora_B"] and int(state["draws"]) == 2
        nxt = a(x)
        b = make(seed=5)
        assert b.load_state_dict(state) == ([], []) and b.draws == 2 and "draws" in state
        assert torch.equal(b(x), nxt) and not any(torch.equal(nxt, y) for y in first)
        inside = torch.nn.Sequential(make(seed=5))
        inside.load_state_dict(torch.nn.Sequential(a).state_dict())
        assert inside[0].draws == 3 and torch.equal(inside(x), a(x))
        # without the count, and into a layer without a seed
        del state["draws"]
        b.load_state_dict(state)
        assert b.draws == 3
        c = make()
        assert sorted(c.state_dict()) == ["lora_A", "lora_B"]
        c.load_state_dict(a.state_dict())
        assert torch.equal(c.lora_B, a.lora_B) and c.draws == 0
