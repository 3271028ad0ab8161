"""Stored dropout masks that are too short are refused (the kernels read past their end)."""
import pytest
import torch

from tests._gpu import needs_gpu, say

pytestmark = [pytest.mark.gpu, needs_gpu]


def test_short_masks():
    import quantized_fine_tuning_nf4_amd as qn
    say("[mask refusals]")
    torch.manual_seed(0)
    M, rows, cols, r = 40, 72, 128, 8
    normal = lambda *s: torch.randn(*s, device="cuda").to(torch.bfloat16)  # noqa: E731
    st = qn.nf4_quantize_dq(torch.randn(rows, cols, device="cuda"))
    x, G, A, B = normal(M, cols), normal(M, rows), normal(r, cols), normal(rows, r)
    x8, u = qn.act8_pack(x), torch.zeros(M, r, device="cuda")
    calls = [lambda m: qn.qlora_linear_fwd(st, x, A, B, 8.0, dropout_mask=m, dropout_p=0.1),
             lambda m: qn.qlora_linear_bwd(st, x, G, A, B, 8.0, u, dropout_mask=m, dropout_p=0.1),
             lambda m: qn.qlora_linear_bwd_act8(st, x8, G, A, B, 8.0, u, dropout_mask=m,
                                                dropout_p=0.1)]
    mask = qn.dropout_mask(M, cols, 0.1)
    for call in calls:
        call(mask)
        for bad in (mask[:-1], mask[:0], mask.to(torch.int32), mask.cpu()):
            with pytest.raises(ValueError):
                call(bad)
    torch.cuda.synchronize()
