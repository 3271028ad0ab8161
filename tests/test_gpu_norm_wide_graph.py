"""Block norms past 4096 columns, whose kernels take more LDS than a launch has without
asking, in captured graphs: every replay against the eager result."""
import pytest
import torch

from tests._gpu import needs_gpu, say

pytestmark = [pytest.mark.gpu, needs_gpu]
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def qn():
    import quantized_fine_tuning_nf4_amd as qn
    qn.load_library()
    return qn


@pytest.mark.parametrize("M,D", [(70, 4104), (300, 5120), (37, 8191), (600, 8192), (90, 16384),
                                 (33, 12001)])
@pytest.mark.parametrize("res", [BF, F32])
def test_graph_replays(qn, M, D, res):
    say(f"[norm graph] M={M} D={D} res={res}")
    g = torch.Generator(device="cuda").manual_seed(D)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    h, o, dy, dh = n(M, D).to(res), n(M, D).to(BF), n(M, D).to(BF), n(M, D).to(res)
    w1, w2, gate = n(D), n(D), n(D)

    def step():
        a, y, x8 = qn.block_norm_fwd(h, w2, o=o, w_post=w1, gate=gate, scale=0.5, pack=True)
        return [a, y, x8.codes, x8.exps, *qn.block_norm_bwd(
            dy, a, w2, dh_new=dh, o=o, w_post=w1, gate=gate, scale=0.5)]

    eager = [v.clone() for v in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for k in range(3):
        for v in outs:
            v.zero_()
        step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, eager)), k
