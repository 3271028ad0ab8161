"""Infinities in dY of the MXFP4 linear's backward without an adapter: an output is what its
products add up to, an infinity of the sign of weight and gradient, on every route."""
import pytest
import torch

from tests._gpu import needs_gpu, say

pytestmark = [pytest.mark.gpu, needs_gpu]


# The row length of dY is no multiple of the product's step of 64, and the infinities lie in its
# last columns, beside what the step covers past them.  Routes: 16 and 32 rows a
# workgroup, tiles 64 x 64, 64 x 128, 128 x 128 and larger ones.
@pytest.mark.parametrize("M,rows,cols", [(16, 72, 64), (300, 72, 320), (520, 72, 1344),
                                         (520, 8, 1344), (1000, 264, 1152), (1030, 328, 2112),
                                         (4096, 72, 4096)])
def test_infinite_gradients(M, rows, cols):
    import quantized_fine_tuning_nf4_amd as qn
    say(f"[mx4 infinite dY] {M}x{rows}x{cols}")
    g = torch.Generator(device="cuda").manual_seed(M + rows)
    # magnitudes 1 to 6 beside each other: MXFP4's own values, none of them zero
    W = torch.tensor([1.0, 1.5, 2, 3, 4, 6], device="cuda")[
        torch.randint(0, 6, (rows, cols), generator=g, device="cuda")]
    W[:, ::32] = 6.0
    W *= torch.randint(0, 2, (rows, cols), generator=g, device="cuda") * 2 - 1
    dY = torch.randn(M, rows, generator=g, device="cuda").to(torch.bfloat16)
    at = [(0, rows - 1, 1), (M // 2, rows - 8, -1), (M - 1, rows - 3, 1), (M // 3, 0, -1)]
    w = qn.mx4_quantize(W)
    base, _, _ = qn.mx4_linear_bwd(w, None, dY)
    for m, n, sign in at:
        dY[m, n] = sign * float("inf")
    dX, _, _ = qn.mx4_linear_bwd(w, None, dY)
    want = base.clone()
    for m, n, sign in at:
        want[m] = W[n].sign() * (sign * float("inf"))
    assert torch.equal(dX, want)


@pytest.mark.parametrize("M,rows,cols", [(16, 72, 64), (300, 72, 320), (520, 72, 1344),
                                         (520, 8, 1344), (1000, 264, 1152), (1030, 328, 2112),
                                         (4096, 72, 4096), (4096, 8, 4096)])
def test_reads_zero_past_its_rows(M, rows, cols):
    """What lies past the rows of dY counts as zero, whatever the workgroup's memory held before:
    the result is that of the same operands padded with zeros to whole steps, after a product
    that left NaNs there."""
    import quantized_fine_tuning_nf4_amd as qn
    say(f"[mx4 past dY] {M}x{rows}x{cols}")
    g = torch.Generator(device="cuda").manual_seed(M + rows)
    W = torch.randn(rows, cols, generator=g, device="cuda")
    dY = torch.randn(M, rows, generator=g, device="cuda").to(torch.bfloat16)
    more = -rows % 64
    Wp = torch.nn.functional.pad(W, (0, 0, 0, more))
    want, _, _ = qn.mx4_linear_bwd(qn.mx4_quantize(Wp), None,
                                   torch.nn.functional.pad(dY, (0, more)))
    w = qn.mx4_quantize(W)
    wide = qn.mx4_quantize(torch.ones(512, cols, device="cuda"))
    bad = torch.full((M, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    for _ in range(3):
        assert bool(torch.isnan(qn.mx4_linear_bwd(wide, None, bad)[0]).all())
        assert torch.equal(qn.mx4_linear_bwd(w, None, dY)[0], want)
