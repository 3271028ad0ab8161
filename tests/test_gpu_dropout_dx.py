"""dX under dropout on the adapter branch's input: the masked share joins the
base product in fp32, so that dX is rounded to bf16 once, as without dropout.

The reference is fp64 with the weight's bf16 values (the products' operand), so
that what is left is the rounding of dX.  Tolerances: an element may be off by
half a bf16 step of its own and by the fp32 sums, at most (rows + 2 r) 2^-24 of
the sum of its terms' magnitudes (and 2^-16 of the adapter's, which enters the
matrix units in two bf16 parts); over all elements the error is that of the
rounding alone up to one part in a hundred (the sums' is a thousandth of it).
A second rounding would make it 1.4 times as large."""
import pytest
import torch

import workloads as wl
from tests._gpu import bf16_dev, f32_dev, needs_gpu, say

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.fixture(scope="module")
def qn():
    import quantized_fine_tuning_nf4_amd as qn
    qn.load_library()
    return qn


def _keep(mask, M, cols):
    bits = torch.arange(8, device="cuda", dtype=torch.uint8)
    return ((mask[:, None] >> bits) & 1).reshape(-1)[:M * cols].view(M, cols).bool()


# M, rows, cols, r, p: 32-row and 128 x 128 tiles of the dequantizing product;
# 128 x 128, 256 x 256 and 256 x 224 tiles of the dense one; rows and columns that
# end inside tiles, ranks of one block of 16 and of several
CASES = [(1, 8, 64, 1, 0.5), (7, 72, 192, 16, 0.1), (32, 256, 320, 20, 0.3),
         (130, 136, 576, 16, 0.05), (300, 64, 1024, 64, 0.2), (257, 200, 4160, 5, 0.1),
         (2050, 72, 2112, 16, 0.05), (2048, 256, 2048, 33, 0.1), (4096, 64, 4096, 16, 0.05),
         (4000, 136, 4160, 48, 0.3), (4096, 72, 4352, 16, 0.05), (4090, 64, 4352, 7, 0.5)]


@pytest.mark.parametrize("M,rows,cols,r,p", CASES)
@pytest.mark.parametrize("act8", [False, True])
def test_one_rounding(qn, M, rows, cols, r, p, act8):
    say(f"[dropout dX] M={M} rows={rows} cols={cols} r={r} p={p} act8={act8}")
    seed = 31 * M + cols + r
    st = qn.nf4_quantize_dq(f32_dev(wl.weight(rows, cols, seed)))
    x = bf16_dev(wl.normal_bf16((M, cols), seed + 1, 1.0))
    # A and B large enough that the share weighs as much as the base product
    A = bf16_dev(wl.normal_bf16((r, cols), seed + 2, 0.1))
    B = bf16_dev(wl.normal_bf16((rows, r), seed + 3, 0.1))
    G = bf16_dev(wl.normal_bf16((M, rows), seed + 4, 1.0))
    alpha = 2.0 * r
    mask = qn.dropout_mask(M, cols, p)
    if act8:
        u = torch.zeros(M, r, device="cuda")
        dX, _, _ = qn.qlora_linear_bwd_act8(st, qn.act8_pack(x), G, A, B, alpha, u,
                                            dropout_mask=mask, dropout_p=p)
    else:
        dX, _, _ = qn.qlora_linear_bwd(st, x, G, A, B, alpha, dropout_mask=mask, dropout_p=p)
    torch.cuda.synchronize()
    keep = _keep(mask, M, cols).double()
    g, W = G.double(), qn.nf4_dequantize(st, torch.bfloat16).double()
    s = alpha / r / (1 - p)
    v = g @ B.double()
    want = g @ W + s * keep * (v @ A.double())
    once = want.to(torch.float32).to(torch.bfloat16).double()
    err, least = (dX.double() - want).norm(), (once - want).norm()
    assert float(err) <= 1.01 * float(least), float(err / least)
    share = s * keep * (v.abs() @ A.double().abs())
    sums = (rows + 2 * r) * 2.0 ** -24 * (g.abs() @ W.abs() + share) + 2.0 ** -16 * share
    step = torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=2.0 ** -126))) - 7)
    # (a value pushed over a power of two by the sums rounds by the step above it)
    edge = torch.exp2(torch.floor(torch.log2((want.abs() + sums).clamp(min=2.0 ** -126))) - 7)
    over = (dX.double() - want).abs() - torch.maximum(step, edge) / 2 - sums
    assert float(over.max()) <= 0.0, float(over.max())


@pytest.mark.parametrize("M,rows,cols,r", [(20, 72, 192, 8), (200, 72, 192, 16),
                                           (4096, 72, 4352, 16), (2050, 72, 2112, 24)])
def test_dropped_elements_take_the_base_product_alone(qn, M, rows, cols, r):
    """Also where the share is NaN."""
    say(f"[dropout dX dropped] M={M} rows={rows} cols={cols} r={r}")
    st = qn.nf4_quantize_dq(f32_dev(wl.weight(rows, cols, 5)))
    x = bf16_dev(wl.normal_bf16((M, cols), 6, 1.0))
    A = bf16_dev(wl.normal_bf16((r, cols), 7, 0.1))
    B = bf16_dev(wl.normal_bf16((rows, r), 8, 0.1))
    G = bf16_dev(wl.normal_bf16((M, rows), 9, 1.0))
    mask = qn.dropout_mask(M, cols, 0.4)
    keep = _keep(mask, M, cols)
    base, _, _ = qn.qlora_linear_bwd(st, x, G, A, torch.zeros_like(B), 2.0 * r)
    A[:, ::3] = float("nan")
    dX, _, _ = qn.qlora_linear_bwd(st, x, G, A, B, 2.0 * r, dropout_mask=mask, dropout_p=0.4)
    torch.cuda.synchronize()
    assert torch.equal(dX[~keep], base[~keep])
    bad = keep.clone()
    bad[:, 1::3] = False
    bad[:, 2::3] = False
    assert torch.equal(torch.isnan(dX), bad)
