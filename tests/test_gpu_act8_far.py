"""The adapter gradients where their partial sums lie past 2^32 bytes: 17 slices of
2^20 columns at rank 64.  The checkpoint is zero but for a few rows, one in the first
slice and two in the last, so that dA is theirs alone."""
import pytest
import torch

from tests._gpu import needs_gpu, say

pytestmark = [pytest.mark.gpu, needs_gpu]


def test_partial_sums_past_32_bit_offsets():
    import quantized_fine_tuning_nf4_amd as qn
    M, rows, cols, r = 16400, 8, 1 << 20, 64
    say(f"[act8 far] M={M} rows={rows} cols={cols} r={r}")
    g = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    st = qn.nf4_quantize_dq(torch.randn(rows, cols, generator=g, device="cuda"))
    live = torch.tensor([5, 16380, 16399], device="cuda")
    codes = torch.zeros(M, cols, dtype=torch.int8, device="cuda")
    exps = torch.full((M, cols // 64), 127, dtype=torch.uint8, device="cuda")
    codes[live] = torch.randint(-127, 128, (3, cols), generator=g, device="cuda",
                                dtype=torch.int8)
    G, A, B = n(M, rows), n(r, cols), n(rows, r)
    u = torch.randn(M, r, generator=g, device="cuda")
    _, dA, dB = qn.qlora_linear_bwd_act8(st, qn.Act8(codes, exps), G, A, B, float(r), u,
                                         need_dx=False)
    torch.cuda.synchronize()
    v = G.double() @ B.double()
    want = v[live].t() @ codes[live].double()
    # (three products a value, v in fp32 over 8 rows)
    bound = 16 * 2.0 ** -24 * ((G.double().abs() @ B.double().abs())[live].t()
                               @ codes[live].double().abs())
    assert ((dA.double() - want).abs() <= bound).all()
    ref = G.double().t() @ u.double()
    assert float((dB.double() - ref).norm() / ref.norm()) < 1e-6
