"""More of the MXFP4 linear and of the calls under a Dropout: the product's tiles with the
adapter in LDS past their stages, the scale of rank-stabilized adapters in every
call, and the backward from an 8-bit checkpoint without dropout."""
import pytest
import torch

from tests._gpu import needs_gpu, say
from tests.test_gpu_mx4 import ADAPTED, test_backward as backward, test_forward as forward

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.fixture(scope="module")
def qn():
    import quantized_fine_tuning_nf4_amd as qn
    qn.load_library()
    return qn


def _normal(seed, *shape, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


# on 256 compute units: 256 x 256 tiles, two stages and six steps; 128 x 128 by eight waves,
# four stages, and by four waves, two; 64 x 128; 64 x 64
@pytest.mark.parametrize("M,rows,cols,r", [(2056, 4104, 1344, 16), (2056, 4104, 1088, 3),
                                           (1000, 4096, 1344, 9), (1100, 4104, 1344, 11),
                                           (300, 4096, 1344, 16), (300, 4096, 1600, 7),
                                           (100, 264, 2112, 16)])
@pytest.mark.parametrize("p", [0.0, 0.1])
def test_tiles_past_their_stages(qn, M, rows, cols, r, p):
    forward(qn, M, rows, cols, r, p)


@pytest.mark.parametrize("M,rows,cols,r", ADAPTED)
def test_backward_from_a_checkpoint(qn, M, rows, cols, r):
    backward(qn, M, rows, cols, r, True, 0.0)


# sqrt(r) is a power of two: alpha / sqrt(r) and (alpha sqrt(r)) / r are the same number
@pytest.mark.parametrize("M,rows,cols,r", [(1, 64, 1024, 4), (40, 136, 320, 16), (300, 264, 576, 64)])
@pytest.mark.parametrize("p", [0.0, 0.2])
def test_rank_stabilized(qn, M, rows, cols, r, p):
    say(f"[rslora] M={M} rows={rows} cols={cols} r={r} p={p}")
    W = _normal(1, rows, cols, std=0.1, dtype=torch.float32)
    x, G = _normal(2, M, cols), _normal(3, M, rows)
    A, B = _normal(4, r, cols, std=0.1), _normal(5, rows, r, std=0.1)
    x8, drop = qn.act8_pack(x), qn.Dropout(p, 7, offset=3)
    for w, fwd, bwd, bwd8 in (
            (qn.nf4_quantize_dq(W), qn.qlora_linear_fwd, qn.qlora_linear_bwd,
             qn.qlora_linear_bwd_act8),
            (qn.mx4_quantize(W), qn.mx4_linear_fwd, qn.mx4_linear_bwd, qn.mx4_linear_bwd)):
        def run(alpha, rslora):
            y, u = fwd(w, x, A, B, alpha, drop=drop, rslora=rslora)
            return [y, u, *bwd(w, x, G, A, B, alpha, u, drop=drop, rslora=rslora),
                    *bwd(w, x, G, A, B, alpha, None, drop=drop, rslora=rslora),
                    *bwd8(w, x8, G, A, B, alpha, u, drop=drop, rslora=rslora)]

        plain = run(8.0, False)
        for a, b in zip(run(8.0, True), run(8.0 * r ** 0.5, False)):
            assert torch.equal(a, b)
        assert not torch.equal(run(8.0, True)[4], plain[4])  # dB: the scale is in it


@pytest.mark.parametrize("base", ["nf4", "mx4"])
@pytest.mark.parametrize("act8", [False, True])
def test_rank_stabilized_modules(qn, base, act8):
    say(f"[rslora module] {base} act8={act8}")
    W = _normal(1, 72, 128, std=0.1, dtype=torch.float32)
    x, g = _normal(2, 40, 128), _normal(3, 40, 72)
    got = []
    for kw in (dict(alpha=8.0, rslora=True), dict(alpha=32.0), dict(alpha=8.0)):
        torch.manual_seed(0)
        lin = qn.QLoRALinear(W, r=16, dropout=0.2, act8=act8, base=base, seed=9, **kw)
        with torch.no_grad():
            lin.lora_B.copy_(_normal(6, 72, 16, std=0.1))
        v = x.clone().requires_grad_()
        y = lin(v)
        y.backward(g)
        got.append([y.detach(), v.grad, lin.lora_A.grad, lin.lora_B.grad])
    for a, b, c in zip(*got):
        assert torch.equal(a, b) and not torch.equal(a, c)
