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
