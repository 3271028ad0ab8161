"""Linear calls on workspaces that hold NaN everywhere but in the arrival
counters: no value that a call has not written itself may reach a result."""
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


# rows no multiple of 32: the adapter products over dY end inside a 32-wide step
@pytest.mark.parametrize("M,rows,cols,r", [(5, 72, 64, 4), (33, 520, 576, 17), (100, 136, 1024, 32),
                                           (300, 264, 320, 64), (1000, 8, 128, 16)])
def test_results_do_not_depend_on_what_the_workspace_held(qn, M, rows, cols, r):
    say(f"[workspace] M={M} rows={rows} cols={cols} r={r}")
    st = qn.nf4_quantize_dq(f32_dev(wl.weight(rows, cols, 1)))
    x = bf16_dev(wl.normal_bf16((M, cols), 2, 1.0))
    A = bf16_dev(wl.normal_bf16((r, cols), 3, 0.05))
    B = bf16_dev(wl.normal_bf16((rows, r), 4, 0.05))
    G = bf16_dev(wl.normal_bf16((M, rows), 5, 1.0))
    clean = qn.linear_workspace(64 << 20)
    dirty = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    dirty[:4096] = 0
    outs = []
    for ws in (clean, dirty):
        y, u = qn.qlora_linear_fwd(st, x, A, B, 2.0 * r, workspace=ws)
        outs.append([y, u, *qn.qlora_linear_bwd(st, x, G, A, B, 2.0 * r, None, workspace=ws)])
    torch.cuda.synchronize()
    for a, b in zip(*outs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("M,rows,cols,r", [(5, 72, 64, 4), (33, 520, 576, 17), (300, 264, 320, 64),
                                           (2100, 4096, 4096, 8)])
def test_checkpoint_backward_does_not_depend_on_what_the_workspace_held(qn, M, rows, cols, r):
    say(f"[workspace] act8 M={M} rows={rows} cols={cols} r={r}")
    st = qn.nf4_quantize_dq(f32_dev(wl.weight(rows, cols, 1)))
    x8 = qn.act8_pack(bf16_dev(wl.normal_bf16((M, cols), 2, 1.0)))
    A = bf16_dev(wl.normal_bf16((r, cols), 3, 0.05))
    B = bf16_dev(wl.normal_bf16((rows, r), 4, 0.05))
    G = bf16_dev(wl.normal_bf16((M, rows), 5, 1.0))
    u = torch.randn(M, r, device="cuda")
    outs = [qn.qlora_linear_bwd_act8(st, x8, G, A, B, 2.0 * r, u, workspace=torch.full(
        (256 << 20,), fill, dtype=torch.uint8, device="cuda")) for fill in (0, 255)]
    torch.cuda.synchronize()
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_calls_around_the_linear_leave_a_shared_workspace_as_linear_calls_need_it(qn):
    ws = qn.linear_workspace(64 << 20)

    def counters():
        torch.cuda.synchronize()
        return int(ws[:4096].sum())

    h = torch.randn(300, 1000, device="cuda").bfloat16()
    w = torch.ones(1000, device="cuda")
    h_new, y, *_ = qn.block_norm_fwd(h, w, o=h, w_post=w)
    ws[4096:] = 255
    qn.block_norm_bwd(y, h_new, w, o=h, w_post=w, workspace=ws)
    assert counters() == 0
    logits = torch.randn(2, 131072, device="cuda")
    qn.token_logprobs_fwd(logits, torch.zeros(2, dtype=torch.int64, device="cuda"), top_k=5,
                          workspace=ws)
    assert counters() == 0
    st = qn.nf4_quantize_dq(f32_dev(wl.weight(1024, 1024, 1)))
    x = bf16_dev(wl.normal_bf16((4, 1024), 2, 1.0))
    A = bf16_dev(wl.normal_bf16((16, 1024), 3, 0.05))
    B = bf16_dev(wl.normal_bf16((1024, 16), 4, 0.05))
    y, u = qn.qlora_linear_fwd(st, x, A, B, 32.0, workspace=ws)
    for M in (4, 4096):  # slices added by the tiles' last workgroups, and by a launch
        xm, um = x.repeat(M // 4, 1), u.repeat(M // 4, 1)
        qn.qlora_linear_bwd_act8(st, qn.act8_pack(xm), xm, A, B, 32.0, um, workspace=ws)
        assert counters() == 0
    assert torch.equal(y, qn.qlora_linear_fwd(st, x, A, B, 32.0, workspace=ws)[0])
