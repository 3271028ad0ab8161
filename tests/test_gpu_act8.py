"""8-bit activation checkpoints (act8_pack / act8_unpack) and the linear's
backward from them (qlora_linear_bwd_act8) against plain fp64 forms."""
import numpy as np
import pytest
import torch

import workloads as wl
from tests._gpu import REL_TOL, bf16_dev, f32_dev, needs_gpu, say
from tests.test_gpu_block_norm import _codes64

pytestmark = [pytest.mark.gpu, needs_gpu]

# dA and dB: fp32 sums over at most 8192 rows of products whose fp32 factor
# enters the matrix units in bf16 parts of at least 16 bits together
GRAD_TOL = 1e-5


@pytest.fixture(scope="module")
def qn():
    import quantized_fine_tuning_nf4_amd as qn
    qn.load_library()
    return qn


@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (1, 63), (2, 64), (5, 65), (4, 96), (37, 1000),
                                 (130, 1001), (1, 4096), (64, 4104), (257, 4096), (19, 14336),
                                 (3, 14336 + 24)])
def test_pack_and_unpack_exact(qn, M, K):
    say(f"[act8] M={M} K={K}")
    g = torch.Generator().manual_seed(M * 31 + K)
    x = torch.randn(M, K, generator=g) * torch.exp(3 * torch.randn(M, 1, generator=g))
    x[:, ::17] *= 50.0
    x = x.to(torch.bfloat16)
    x8 = qn.act8_pack(x.cuda())
    back = qn.act8_unpack(x8)
    torch.cuda.synchronize()
    codes, exps = _codes64(x)
    assert np.array_equal(x8.exps.cpu().numpy(), exps)
    assert np.array_equal(x8.codes.cpu().numpy(), codes)
    scale = 2.0 ** (np.repeat(exps, 64, axis=1)[:, :K] - 127.0)
    assert np.array_equal(back.cpu().double().numpy(), codes * scale)
    assert x8.nbytes() == M * K + M * ((K + 63) // 64)
    assert np.all(np.abs(codes * scale - x.double().numpy()) <= scale / 2)


def test_pack_every_significand_and_exponent(qn):
    """The block's largest magnitude at every bf16 value: subnormals, ties
    (odd significands lie half way between codes) and the largest finite."""
    bits = np.arange(0x7f80, dtype=np.uint16)
    x = np.zeros((bits.size, 64), np.uint16)
    x[:, 5] = bits
    x[:, 40] = bits // 3  # something smaller beside it
    x[:, 41] = bits | 0x8000
    t = torch.from_numpy(x.view(np.int16)).view(torch.bfloat16)
    x8 = qn.act8_pack(t.cuda())
    codes, exps = _codes64(t)
    assert np.array_equal(x8.exps.cpu().numpy(), exps)
    assert np.array_equal(x8.codes.cpu().numpy(), codes)
    back = qn.act8_unpack(x8).cpu().double().numpy()
    assert np.array_equal(back, codes * 2.0 ** (exps - 127.0))


def test_nonfinite_blocks_read_back_nan(qn):
    x = torch.randn(4, 200, device="cuda").to(torch.bfloat16)
    x[0, 70], x[2, 199], x[3, 0] = float("nan"), float("-inf"), float("inf")
    x8 = qn.act8_pack(x)
    back = qn.act8_unpack(x8)
    bad = torch.zeros(4, 200, dtype=torch.bool, device="cuda")
    bad[0, 64:128] = bad[2, 192:] = bad[3, :64] = True
    assert torch.equal(torch.isnan(back), bad)
    assert (x8.exps == 255).sum() == 3 and not x8.codes[bad].any()


def test_empty_and_out(qn):
    x = torch.randn(6, 128, device="cuda").to(torch.bfloat16)
    assert qn.act8_unpack(qn.act8_pack(x[:0])).shape == (0, 128)
    out = qn.act8_pack(torch.zeros_like(x))
    assert qn.act8_pack(x, out=out) is out
    back = torch.empty_like(x)
    assert qn.act8_unpack(out, out=back) is back
    assert torch.equal(back, qn.act8_unpack(qn.act8_pack(x.view(2, 3, 128))))


def _case(qn, M, rows, cols, r, p, seed, codebook="nf4", dq=True):
    st = qn.qn_quantize(f32_dev(wl.weight(rows, cols, seed)), codebook, dq)
    x = bf16_dev(wl.normal_bf16((M, cols), seed + 1, 1.0))
    A = bf16_dev(wl.normal_bf16((r, cols), seed + 2, 0.05))
    B = bf16_dev(wl.normal_bf16((rows, r), seed + 3, 0.05))
    G = bf16_dev(wl.normal_bf16((M, rows), seed + 4, 1.0))
    mask = qn.dropout_mask(M, cols, p) if p else None
    return st, x, A, B, G, mask


def _ref(qn, st, x8, A, B, G, u, s, mask):
    M, K = x8.codes.shape
    x = qn.act8_unpack(x8).cpu().double()
    keep = None
    if mask is not None:
        bits = np.unpackbits(mask.cpu().numpy(), bitorder="little")[:M * K].reshape(M, K)
        keep = torch.from_numpy(bits.astype(np.float64))
        x = x * keep
    G, A, B = G.cpu().double(), A.cpu().double(), B.cpu().double()
    v = G @ B
    W = qn.nf4_dequantize(st, torch.float32).cpu().double()
    share = s * (v @ A)
    dX = G @ W + (share if keep is None else share * keep)
    return dX, s * (v.t() @ x), s * (G.t() @ u.cpu().double())


def _rel(a, b):
    return float((a.cpu().double() - b).norm() / b.norm().clamp(min=1e-300))


CASES = [  # M, rows, cols, r, dropout p
    (1, 8, 64, 1, 0.0), (5, 64, 64, 3, 0.1), (31, 72, 192, 5, 0.0), (32, 256, 256, 16, 0.05),
    (33, 520, 576, 17, 0.0), (100, 136, 1024, 32, 0.1), (300, 520, 576, 33, 0.0),
    (129, 1024, 640, 48, 0.05), (64, 128, 4160, 64, 0.0), (1000, 264, 320, 64, 0.3),
    (2048, 1024, 1024, 16, 0.0), (4096, 512, 2048, 8, 0.05)]


@pytest.mark.parametrize("M,rows,cols,r,p", CASES)
def test_backward_from_the_checkpoint(qn, M, rows, cols, r, p):
    say(f"[act8 bwd] M={M} rows={rows} cols={cols} r={r} p={p}")
    st, x, A, B, G, mask = _case(qn, M, rows, cols, r, p, seed=M + rows + r)
    x8 = qn.act8_pack(x)
    _, u = qn.qlora_linear_fwd(st, x, A, B, 2.0 * r, dropout_mask=mask, dropout_p=p)
    dX, dA, dB = qn.qlora_linear_bwd_act8(st, x8, G, A, B, 2.0 * r, u, dropout_mask=mask,
                                          dropout_p=p)
    none, dA2, dB2 = qn.qlora_linear_bwd_act8(st, x8, G, A, B, 2.0 * r, u, need_dx=False,
                                              dropout_mask=mask, dropout_p=p)
    torch.cuda.synchronize()
    rX, rA, rB = _ref(qn, st, x8, A, B, G, u, 2.0 / (1 - p), mask)
    assert _rel(dX, rX) <= REL_TOL
    assert _rel(dA, rA) <= GRAD_TOL and _rel(dB, rB) <= GRAD_TOL
    assert none is None and torch.equal(dA, dA2) and torch.equal(dB, dB2)
    # element by element: no column, rank or tail left out
    scale = rA.abs().max(), rB.abs().max()
    assert float((dA.cpu().double() - rA).abs().max()) <= 4 * GRAD_TOL * scale[0]
    assert float((dB.cpu().double() - rB).abs().max()) <= 4 * GRAD_TOL * scale[1]


@pytest.mark.parametrize("codebook,dq", [("nf4", False), ("fp4", True)])
def test_backward_other_formats_and_rslora(qn, codebook, dq):
    st, x, A, B, G, _ = _case(qn, 70, 256, 320, 16, 0.0, 9, codebook, dq)
    x8 = qn.act8_pack(x)
    u = x.float() @ A.float().t()
    dX, dA, dB = qn.qlora_linear_bwd_act8(st, x8, G, A, B, 32.0, u, rslora=True)
    rX, rA, rB = _ref(qn, st, x8, A, B, G, u, 8.0, None)
    assert _rel(dX, rX) <= REL_TOL and _rel(dA, rA) <= GRAD_TOL and _rel(dB, rB) <= GRAD_TOL


def test_backward_agrees_with_the_bf16_path_and_costs_half_a_code(qn):
    """dX and dB do not read x; dA moves by the checkpoint's rounding alone:
    a uniform error of at most 2^(e-1), for a normal x about 0.9% of it."""
    st, x, A, B, G, _ = _case(qn, 2048, 512, 512, 16, 0.0, 3)
    _, u = qn.qlora_linear_fwd(st, x, A, B, 32.0)
    a = qn.qlora_linear_bwd(st, x, G, A, B, 32.0, u)
    b = qn.qlora_linear_bwd_act8(st, qn.act8_pack(x), G, A, B, 32.0, u)
    assert torch.equal(a[0], b[0])
    assert _rel(b[2], a[2].cpu().double()) <= 2 * GRAD_TOL
    assert 1e-4 < _rel(b[1], a[1].cpu().double()) < 1.5e-2


def test_dirty_workspace_reused(qn):
    """One workspace, never cleared, for calls of different shapes."""
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    for M, rows, cols, r, p in [CASES[3], CASES[9], CASES[5], CASES[0], CASES[3]]:
        say(f"[act8 bwd ws] M={M} rows={rows} cols={cols} r={r} p={p}")
        st, x, A, B, G, mask = _case(qn, M, rows, cols, r, p, seed=M)
        u = x.float() @ A.float().t()
        x8 = qn.act8_pack(x)
        args = (st, x8, G, A, B, 2.0 * r, u)
        got = qn.qlora_linear_bwd_act8(*args, workspace=ws, dropout_mask=mask, dropout_p=p)
        ref = qn.qlora_linear_bwd_act8(*args, dropout_mask=mask, dropout_p=p)
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_empty_batch(qn):
    st, x, A, B, G, _ = _case(qn, 4, 64, 128, 8, 0.0, 1)
    x8 = qn.act8_pack(x[:0])
    dX, dA, dB = qn.qlora_linear_bwd_act8(st, x8, G[:0], A, B, 16.0, torch.empty(0, 8, device="cuda"))
    assert dX.shape == (0, 128) and not dA.any() and not dB.any()


def test_nonfinite_activation_reaches_dA(qn):
    st, x, A, B, G, _ = _case(qn, 40, 64, 192, 8, 0.0, 2)
    x[7, 100] = float("inf")
    u = torch.zeros(40, 8, device="cuda")
    _, dA, _ = qn.qlora_linear_bwd_act8(st, qn.act8_pack(x), G, A, B, 16.0, u)
    bad = torch.zeros(8, 192, dtype=torch.bool, device="cuda")
    bad[:, 64:128] = True
    assert torch.equal(torch.isnan(dA), bad)


def test_graph_replays(qn):
    st, x, A, B, G, mask = _case(qn, 256, 520, 576, 16, 0.1, 5)
    u = x.float() @ A.float().t()
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")

    def step():
        x8 = qn.act8_pack(x)
        return [x8.codes, x8.exps, *qn.qlora_linear_bwd_act8(
            st, x8, G, A, B, 32.0, u, workspace=ws, dropout_mask=mask, dropout_p=0.1)]

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


def test_layer_keeps_the_checkpoint(qn):
    torch.manual_seed(0)
    W = torch.randn(256, 192, device="cuda") * 0.02
    ref, lin = qn.QLoRALinear(W, r=8), qn.QLoRALinear(W, r=8, act8=True)
    with torch.no_grad():
        ref.lora_B.normal_(std=0.05)
        for a, b in zip(lin.parameters(), ref.parameters()):
            a.copy_(b)
    x = torch.randn(3, 17, 192, device="cuda").to(torch.bfloat16)
    dy = torch.randn(3, 17, 256, device="cuda").to(torch.bfloat16)
    xs = [x.clone().requires_grad_(True) for _ in range(3)]
    x8 = qn.act8_pack(x)
    ys = [ref(xs[0]), lin(xs[1]), None]
    ga = []
    for k in range(3):
        layer = ref if k == 0 else lin
        layer.zero_grad()
        y = layer(xs[k]) if k < 2 else layer(xs[k], x8=x8)
        y.backward(dy)
        ga.append((y.detach(), xs[k].grad, layer.lora_A.grad.clone(), layer.lora_B.grad.clone()))
    del ys
    assert torch.equal(ga[0][0], ga[1][0]) and torch.equal(ga[0][1], ga[1][1])
    assert all(torch.equal(a, b) for a, b in zip(ga[1], ga[2]))
    assert 0 < _rel(ga[1][2].float(), ga[0][2].cpu().double()) < 2e-2
    with pytest.raises(ValueError):
        ref(x, x8=x8)


# calls long enough that the slices of dA and dB are added by a launch of their
# own at every rank; rows, columns and slices that end inside tiles
LONG = [(4100, 2056, 2112, 16, 0.0), (8195, 1032, 1088, 3, 0.1), (8224, 520, 1664, 11, 0.0),
        (2500, 4104, 2752, 33, 0.05)]


@pytest.mark.parametrize("M,rows,cols,r,p", LONG)
def test_backward_of_long_calls(qn, M, rows, cols, r, p):
    test_backward_from_the_checkpoint(qn, M, rows, cols, r, p)
