"""Every call that takes a workspace refuses one that is strided or on the host."""
import pytest
import torch

from tests._gpu import needs_gpu, say

pytestmark = [pytest.mark.gpu, needs_gpu]


def _normal(*shape, dtype=torch.bfloat16):
    return torch.randn(*shape, device="cuda").to(dtype)


def test_refused():
    import quantized_fine_tuning_nf4_amd as qn
    say("[workspace refusals]")
    torch.manual_seed(0)
    M, rows, cols, r = 40, 72, 128, 8
    W = _normal(rows, cols, dtype=torch.float32)
    st, w = qn.nf4_quantize_dq(W), qn.mx4_quantize(W)
    x, G, A, B = _normal(M, cols), _normal(M, rows), _normal(r, cols), _normal(rows, r)
    x8, u, drop = qn.act8_pack(x), torch.zeros(M, r, device="cuda"), qn.Dropout(0.1, 1)
    norm = torch.ones(cols, device="cuda")
    calls = [
        lambda ws: qn.nf4_quantize_dq(W, workspace=ws),
        lambda ws: qn.qn_quantize(W, "fp4", workspace=ws),
        lambda ws: qn.qlora_linear_fwd(st, x, A, B, 8.0, workspace=ws),
        lambda ws: qn.qlora_linear_bwd(st, x, G, A, B, 8.0, u, workspace=ws),
        lambda ws: qn.qlora_linear_bwd_act8(st, x8, G, A, B, 8.0, u, workspace=ws),
        lambda ws: qn.qlora_linear_fwd(st, x, A, B, 8.0, workspace=ws, drop=drop),
        lambda ws: qn.qlora_linear_bwd(st, x, G, A, B, 8.0, u, workspace=ws, drop=drop),
        lambda ws: qn.qlora_linear_bwd_act8(st, x8, G, A, B, 8.0, u, workspace=ws, drop=drop),
        lambda ws: qn.mx4_linear_fwd(w, x, A, B, 8.0, workspace=ws, drop=drop),
        lambda ws: qn.mx4_linear_bwd(w, x, G, A, B, 8.0, u, workspace=ws, drop=drop),
        lambda ws: qn.block_norm_bwd(x, x, norm, workspace=ws),
        lambda ws: qn.token_logprobs_fwd(_normal(4, 90000), top_k=3, workspace=ws),
    ]
    n = 1 << 22
    for k, call in enumerate(calls):
        call(torch.zeros(n, dtype=torch.uint8, device="cuda"))
        for bad in (torch.zeros(2 * n, dtype=torch.uint8, device="cuda")[::2],
                    torch.zeros(n, dtype=torch.uint8)):
            with pytest.raises(ValueError):
                call(bad)
                say("taken:", k)
    torch.cuda.synchronize()
