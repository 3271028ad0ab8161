"""Layers with a seed and a step in captured graphs: no two uses, in one replay or over
several, have the same mask, and each is the mask of the documented key."""
import pytest
import torch

from tests._gpu import needs_gpu, say

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.mark.parametrize("base", ["nf4", "mx4"])
def test_two_uses_a_replay(base):
    import quantized_fine_tuning_nf4_amd as qn
    from quantized_fine_tuning_nf4_amd.mx4 import linear_fwd
    say(f"[drop replays] {base}")
    torch.manual_seed(0)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    lin = qn.QLoRALinear(torch.randn(72, 128, device="cuda") * 0.1, r=8, alpha=16.0, dropout=0.3,
                         base=base, seed=11, step=step)
    x = torch.randn(40, 128, device="cuda").to(torch.bfloat16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.no_grad():
        lin.lora_B.normal_(std=0.1)
        with torch.cuda.stream(s):
            lin(x)  # draw 0, step 0
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                out = [lin(x), lin(x)]  # draws 1 and 2
        torch.cuda.synchronize()
        seen = []
        for k in range(4):
            step.fill_(k)
            graph.replay()
            torch.cuda.synchronize()
            for draw, y in enumerate(out, start=1):
                drop = qn.Dropout(0.3, 11, (draw << 32) + k)
                want, _ = linear_fwd(lin.st, x, lin.lora_A, lin.lora_B, 16.0, drop=drop)
                assert torch.equal(y, want)
                seen.append(y.clone())
    for i in range(len(seen)):
        for j in range(i):
            assert not torch.equal(seen[i], seen[j]), (i, j)
