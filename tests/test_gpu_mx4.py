"""MXFP4 on the device: storage against the plain form bit for bit, the linear's
product and gradients against 64 bits.

Tolerances.  A bf16 output may be off by half a step of its own (2^-8 of it) and by the
sums: every product of two MXFP4 values is exact, K of them are added in fp32 (at
most K 2^-23 of the sum of their magnitudes, were every addition cut off); the
adapter's share enters in bf16 parts that hold it to 2^-16.  u, dA and dB are fp32 sums
of bf16 products with u and v in parts to 2^-16.
W has bf16 values exactly, so dX is held to the same bound."""
import numpy as np
import pytest
import torch

from tests import _mx4
from tests._gpu import needs_gpu, say

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.fixture(scope="module")
def qn():
    import quantized_fine_tuning_nf4_amd as qn
    qn.load_library()
    return qn


def _normal(seed, *shape, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _np(t):
    return t.detach().double().cpu().numpy()


def _values(w, qn):
    return qn.mx4_dequantize(w, torch.float32).double()


# ------------------------------------------------------------------------ storage
@pytest.mark.parametrize("M,K", [(1, 1), (1, 31), (2, 32), (31, 33), (33, 64), (5, 255), (64, 256),
                                 (3, 257), (40, 1000), (7, 2049)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_store(qn, M, K, dtype):
    say(f"[mx4 store] {M}x{K} {dtype}")
    x = _normal(M + K, M, K, dtype=dtype)
    x *= torch.exp2(torch.randint(-30, 30, (M, 1), device="cuda").float()).to(dtype)
    if K > 3:
        x[0, 3], x[-1, 0] = 0.0, -0.0
    c, E = _mx4.encode(_np(x))
    codes, scales = _mx4.layout(c, E)
    q = qn.mx4_quantize(x)
    assert (q.rows, q.cols) == (M, K)
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    want = torch.from_numpy(_mx4.decode(c, E, K))
    for dt in (torch.float32, torch.bfloat16):
        got = qn.mx4_dequantize(q, dt).double().cpu()
        assert torch.equal(got, want) and torch.equal(torch.signbit(got), torch.signbit(want))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_store_ties_and_range(qn, dtype):
    """Every midpoint at many scales, the largest and the smallest magnitudes, blocks of
    zeros and blocks that are no numbers."""
    say(f"[mx4 ties] {dtype}")
    mid = torch.tensor([4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6.5, 7.5, 7.9375, 0.125, 0.2490234375,
                        0.251953125, 4.96875, 5.03125], dtype=torch.float64)
    row = torch.cat([mid, -mid])
    scales = list(range(-126, 125, 5)) + [-125, -124, 125]
    x = torch.stack([row * 2.0 ** e for e in scales]).to(dtype)
    top = torch.finfo(dtype).max
    tiny = 2.0 ** -126
    extra = torch.zeros(9, 32, dtype=torch.float64)
    extra[1, 4], extra[2, 5], extra[2, 6] = top, -top, 1.0
    extra[3, :8] = torch.tensor([tiny, tiny / 2, -tiny / 4, tiny / 8, tiny * 3, 0, tiny / 64, -tiny])
    extra[4, 0] = tiny / 2
    extra[5, 7], extra[6, 0], extra[7, 31] = float("nan"), float("inf"), -float("inf")
    extra[8] = -0.0
    x = torch.cat([x, extra.to(dtype)]).cuda()
    c, E = _mx4.encode(_np(x))
    q = qn.mx4_quantize(x)
    codes, sc = _mx4.layout(c, E)
    assert np.array_equal(q.scales.cpu().numpy(), sc)
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    want = _mx4.decode(c, E, 32)
    for dt in (torch.float32, torch.bfloat16):
        assert np.array_equal(_np(qn.mx4_dequantize(q, dt)), want, equal_nan=True)


def test_store_takes_rows_that_start_anywhere_and_given_outputs(qn):
    say("[mx4 store views]")
    x = _normal(3, 41, 333)
    for lo in (0, 1, 2, 7):
        part = x[lo:]
        a, b = qn.mx4_quantize(part), qn.mx4_quantize(part.clone())
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    y = _normal(4, 9 * 64 + 1)[1:].view(9, 64)  # on no 16-byte boundary
    out = qn.mx4_quantize(y.clone())
    q = qn.MX4(torch.full_like(out.codes, 255), torch.full_like(out.scales, 255), 9, 64)
    got = qn.mx4_quantize(y, out=q)
    assert got is q and torch.equal(q.codes, out.codes) and torch.equal(q.scales, out.scales)
    buf = torch.full((9 * 64 + 64,), 7.0, device="cuda")
    qn.mx4_dequantize(q, torch.float32, out=buf[:9 * 64].view(9, 64))
    assert torch.equal(buf[9 * 64:], torch.full((64,), 7.0, device="cuda"))
    z = qn.mx4_quantize(torch.zeros(0, 40, device="cuda"))
    assert z.codes.shape == (0, 128) and qn.mx4_dequantize(z).shape == (0, 40)


def test_store_large_offsets(qn):
    """Rows past 2^32 bytes."""
    say("[mx4 far]")
    rows, cols = (1 << 20) + 40, 2304
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-50:] = _normal(5, 50, cols)
    q = qn.mx4_quantize(x)
    near = qn.mx4_quantize(x[rows - 72:].clone())
    assert torch.equal(q.codes[-50:], near.codes[-50:])
    got = qn.mx4_dequantize(q)[-50:]
    assert torch.equal(got, qn.mx4_dequantize(near)[-50:])
    assert int(q.codes[:rows - 50].max()) == 0


# ------------------------------------------------------------------------ forward
def _bound(want, magnitude, K, share=0.0):
    return 2.0 ** -8 * want.abs() + (K + 128) * 2.0 ** -23 * magnitude + 2.0 ** -15 * share


def _check(got, want, tol, name):
    over = ((got.double() - want).abs() - tol).max() if want.numel() else torch.tensor(0.0)
    assert float(over) <= 0.0, (name, float(over))


# M, rows, cols, r: no adapter at odd sizes, then ranks of one block of 16 and several,
# tiles that end inside, one row, few and many
PLAIN = [(1, 1, 1), (1, 5, 32), (8, 300, 1056), (7, 8210, 288), (1, 5, 33), (3, 17, 100), (16, 64, 256), (17, 31, 1000), (33, 257, 511),
         (100, 130, 2048), (128, 128, 64), (129, 129, 300), (300, 1001, 129), (256, 512, 4096),
         (65, 33, 4000), (4001, 4099, 300), (3841, 4096, 1025), (300, 4096, 257), (1000, 4095, 1281),
         (2049, 4097, 130), (130, 520, 2304)]


@pytest.mark.parametrize("M,rows,cols", PLAIN)
def test_product(qn, M, rows, cols):
    say(f"[mx4 product] {M}x{rows}x{cols}")
    x, W = _normal(M + cols, M, cols), _normal(rows, rows, cols, std=0.1)
    w = qn.mx4_quantize(W)
    y = torch.full((M * rows + 32,), 3.0, dtype=torch.bfloat16, device="cuda")
    got, u = qn.mx4_linear_fwd(w, x, y=y[:M * rows].view(M, rows))
    assert u is None and got.data_ptr() == y.data_ptr()
    a, b = torch.from_numpy(_mx4.rounded(_np(x))).cuda(), _values(w, qn)
    _check(got, a @ b.t(), _bound(a @ b.t(), a.abs() @ b.abs().t(), cols), "y")
    assert bool((y[M * rows:] == 3.0).all())  # nothing behind the last row


ADAPTED = [(1, 8, 64, 1), (2, 64, 128, 16), (16, 72, 192, 5), (31, 136, 320, 17), (40, 256, 1024, 64),
           (130, 264, 576, 16), (257, 512, 832, 33), (1, 1024, 4096, 16), (520, 768, 2048, 8),
           (4000, 4104, 320, 16), (3841, 4000, 832, 40), (6150, 72, 128, 20), (6177, 256, 320, 7),
           (50, 72, 640, 64), (33, 64, 2112, 3), (300, 4096, 192, 16), (300, 4096, 1344, 40),
           (1000, 4096, 192, 9), (1000, 4096, 1344, 40), (2056, 4104, 128, 5), (2056, 4104, 128, 40), (60, 72, 8256, 5), (100, 136, 1088, 20),
           (128, 64, 320, 64), (20, 1000, 8192, 33)]


def _linear(qn, M, rows, cols, r, seed=0):
    d = dict(x=_normal(seed + 1, M, cols), A=_normal(seed + 2, r, cols, std=0.1),
             B=_normal(seed + 3, rows, r, std=0.1), dY=_normal(seed + 4, M, rows))
    w = qn.mx4_quantize(_normal(seed + 5, rows, cols, std=0.1, dtype=torch.float32))
    return w, d


def _keep(M, cols, drop):
    k, f = _mx4.keep(M * cols, drop.p, drop.seed, drop.offset + (
        0 if drop.step is None else int(drop.step)))
    return torch.from_numpy(k).view(M, cols).cuda().double(), f


@pytest.mark.parametrize("M,rows,cols,r", ADAPTED)
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_forward(qn, M, rows, cols, r, p):
    say(f"[mx4 fwd] M={M} rows={rows} cols={cols} r={r} p={p}")
    w, d = _linear(qn, M, rows, cols, r, seed=M + rows)
    drop = qn.Dropout(p, 1 << 40, offset=5) if p else None
    keep, f = _keep(M, cols, drop) if p else (torch.ones(M, cols, device="cuda").double(), 1.0)
    for rslora in (False, True):
        y, u = qn.mx4_linear_fwd(w, d["x"], d["A"], d["B"], 2.0 * r, rslora=rslora, drop=drop)
        x, A, B = d["x"].double(), d["A"].double(), d["B"].double()
        s = 2.0 * r / (r ** 0.5 if rslora else r) * f
        want_u = (x * keep) @ A.t()
        _check(u, want_u, (cols * 2.0 ** -23) * ((x * keep).abs() @ A.abs().t()), "u")
        a, b = torch.from_numpy(_mx4.rounded(_np(x))).cuda(), _values(w, qn)
        want = a @ b.t() + s * (want_u @ B.t())
        share = s * ((x * keep).abs() @ A.abs().t() @ B.abs().t())
        _check(y, want, _bound(want, a.abs() @ b.abs().t() + share, cols, share), "y")
        none, no_u = qn.mx4_linear_fwd(w, d["x"], d["A"], d["B"], 2.0 * r, save_u=False,
                                       rslora=rslora, drop=drop)
        assert no_u is None and torch.equal(none, y)


# u in slices ahead of a product by tiles, ragged rows and ranks, two slices to eight
@pytest.mark.parametrize("M,rows,cols,r", [(33, 72, 4160, 5), (40, 264, 8192, 64), (300, 136, 4096, 16),
                                           (530, 72, 2112, 51), (1001, 64, 4096, 23),
                                           (2040, 64, 4352, 1)])
@pytest.mark.parametrize("p", [0.0, 0.1])
def test_forward_in_slices(qn, M, rows, cols, r, p):
    test_forward(qn, M, rows, cols, r, p)


@pytest.mark.parametrize("M", [1, 16, 40, 70, 6145])
@pytest.mark.parametrize("r", [0, 3, 40])
def test_input_is_rounded_as_a_stored_matrix_is(qn, M, r):
    """With W = 2^e I the product is x in MXFP4, times 2^e."""
    say(f"[mx4 input] M={M} r={r}")
    cols = 320
    for e, lo, hi in ((0, -90, 90), (100, -133, -110)):
        x = _normal(M + r, M, cols, dtype=torch.float32)
        x *= torch.exp2(torch.randint(lo, hi, (M, cols // 32), device="cuda").float()
                        ).repeat_interleave(32, dim=1)
        x = x.to(torch.bfloat16)
        x[0, 32:64], x[-1, 5] = 0.0, -0.0
        w = qn.mx4_quantize(torch.eye(cols, device="cuda") * 2.0 ** e)
        A = _normal(1, r, cols) if r else None
        B = torch.zeros(cols, r, dtype=torch.bfloat16, device="cuda") if r else None
        y, _ = qn.mx4_linear_fwd(w, x, A, B, 1.0)
        want = qn.mx4_dequantize(qn.mx4_quantize(x), torch.float32).double() * 2.0 ** e
        assert torch.equal(y.double(), want), (e, float((y.double() - want).abs().max()))


def test_no_numbers_reach_their_rows_alone(qn):
    """A NaN or an infinity in x makes its row NaN, one in W its column."""
    say("[mx4 nan]")
    x, W = _normal(1, 37, 96), _normal(2, 70, 96)
    clean, _ = qn.mx4_linear_fwd(qn.mx4_quantize(W), x)
    x[3, 40], x[36, 0], W[69, 95], W[0, 1] = float("nan"), float("inf"), float("nan"), -float("inf")
    y, _ = qn.mx4_linear_fwd(qn.mx4_quantize(W), x)
    bad = torch.zeros(37, 70, dtype=torch.bool, device="cuda")
    bad[3], bad[36], bad[:, 69], bad[:, 0] = True, True, True, True
    assert torch.equal(torch.isnan(y), bad)
    assert torch.equal(y[~bad], clean[~bad])


def test_forward_reads_nothing_behind_its_inputs(qn):
    """Workspaces and the memory around codes full of NaN patterns change nothing."""
    say("[mx4 dirty]")
    for M, rows, cols, r in [(5, 72, 192, 7), (65, 136, 320, 16)]:
        w, d = _linear(qn, M, rows, cols, r)
        y, u = qn.mx4_linear_fwd(w, d["x"], d["A"], d["B"], 16.0)
        need = qn.load_library().mx4_linear_workspace(M, rows, cols, r, 0, 0, 0)
        ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
        wide = torch.full((M + 2, cols), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[1:-1] = d["x"]
        y2, u2 = qn.mx4_linear_fwd(w, wide[1:-1], d["A"], d["B"], 16.0, workspace=ws)
        assert torch.equal(y, y2) and torch.equal(u, u2)


# ----------------------------------------------------------------------- backward
@pytest.mark.parametrize("M,rows,cols,r", ADAPTED)
@pytest.mark.parametrize("act8,p", [(False, 0.0), (False, 0.2), (True, 0.2)])
def test_backward(qn, M, rows, cols, r, act8, p):
    say(f"[mx4 bwd] M={M} rows={rows} cols={cols} r={r} act8={act8} p={p}")
    w, d = _linear(qn, M, rows, cols, r, seed=M + cols)
    drop = qn.Dropout(p, 99, offset=(1 << 64) - 3) if p else None
    keep, f = _keep(M, cols, drop) if p else (torch.ones(M, cols, device="cuda").double(), 1.0)
    x8 = qn.act8_pack(d["x"])
    x = qn.act8_unpack(x8).double() if act8 else d["x"].double()
    A, B, G, s = d["A"].double(), d["B"].double(), d["dY"].double(), 2.0 * f
    _, u = qn.mx4_linear_fwd(w, d["x"], d["A"], d["B"], 2.0 * r, drop=drop)
    xin = x8 if act8 else d["x"]
    dX, dA, dB = qn.mx4_linear_bwd(w, xin, d["dY"], d["A"], d["B"], 2.0 * r, u, drop=drop)
    v = G @ B
    part = (M + rows) * 2.0 ** -23 + 2.0 ** -15
    _check(dA, s * (v.t() @ (x * keep)),
           part * s * (G.abs() @ B.abs()).t() @ (x * keep).abs(), "dA")
    _check(dB, s * (G.t() @ u.double()), part * s * G.abs().t() @ u.double().abs(), "dB")
    b = _values(w, qn)
    want = G @ b + s * keep * (v @ A)
    share = s * keep * (G.abs() @ B.abs() @ A.abs())
    _check(dX, want, _bound(want, G.abs() @ b.abs() + share, rows + r, share), "dX")
    none, dA2, dB2 = qn.mx4_linear_bwd(w, xin, d["dY"], d["A"], d["B"], 2.0 * r, u, need_dx=False,
                                       drop=drop)
    assert none is None
    _check(dA2, dA.double(), 2 * part * s * (G.abs() @ B.abs()).t() @ (x * keep).abs(), "dA alone")
    _check(dB2, dB.double(), 2 * part * s * G.abs().t() @ u.double().abs(), "dB alone")
    if not act8:  # u formed again
        _, dA3, dB3 = qn.mx4_linear_bwd(w, xin, d["dY"], d["A"], d["B"], 2.0 * r, drop=drop)
        _check(dB3, dB.double(), 2 * part * s * G.abs().t() @ u.double().abs() + 1e-30, "dB, no u")


# a few tiles of each size, the last ones ragged; reductions of one chunk, of one step, of
# one more than the stages
TILES = [(300, 72, 320, 7), (129, 8, 64, 64), (1000, 264, 1152, 16), (1030, 328, 2112, 33),
         (300, 72, 1344, 7), (200, 8, 1024, 64), (2000, 40, 64, 5)]


@pytest.mark.parametrize("M,rows,cols,r", TILES)
@pytest.mark.parametrize("p", [0.0, 0.2])
def test_backward_by_a_few_tiles(qn, M, rows, cols, r, p):
    test_backward(qn, M, rows, cols, r, False, p)


@pytest.mark.parametrize("M,rows,cols,r", TILES)
def test_frozen_backward_by_a_few_tiles(qn, M, rows, cols, r):
    say(f"[mx4 frozen bwd] M={M} rows={rows} cols={cols}")
    w, d = _linear(qn, M, rows, cols, r, seed=M + cols)
    dX, _, _ = qn.mx4_linear_bwd(w, None, d["dY"])
    G, b = d["dY"].double(), _values(w, qn)
    _check(dX, G @ b, _bound(G @ b, G.abs() @ b.abs(), rows, 0), "dX")


def test_no_numbers_in_the_backward(qn):
    """A block of W that is no number makes its columns of dX NaN, a NaN of dY its row."""
    say("[mx4 bwd nan]")
    W = _normal(2, 72, 320)
    clean = qn.mx4_quantize(W)
    W[70, 100], W[3, 0] = float("nan"), float("inf")
    w, G = qn.mx4_quantize(W), _normal(3, 150, 72)
    base, _, _ = qn.mx4_linear_bwd(clean, None, G)
    dX, _, _ = qn.mx4_linear_bwd(w, None, G)
    bad = torch.zeros(150, 320, dtype=torch.bool, device="cuda")
    bad[:, 96:128], bad[:, :32] = True, True
    assert torch.equal(torch.isnan(dX), bad) and torch.equal(dX[~bad], base[~bad])
    G[17, 5] = float("nan")
    dX, _, _ = qn.mx4_linear_bwd(clean, None, G)
    assert bool(torch.isnan(dX[17]).all()) and not bool(torch.isnan(dX[:17]).any())


def test_adapter_gradients_keep_24_bits(qn):
    """u and v enter in three bf16 parts: over all elements dA and dB are within 1e-6 (the
    fp32 sums; two parts leave 2e-6)."""
    say("[mx4 bwd parts]")
    M, rows, cols, r = 1500, 264, 576, 16
    w, d = _linear(qn, M, rows, cols, r, seed=5)
    st = qn.nf4_quantize_dq(_normal(6, rows, cols, dtype=torch.float32))
    drop = qn.Dropout(0.2, 1)
    keep, f = _keep(M, cols, drop)
    G, B, x = d["dY"].double(), d["B"].double(), d["x"].double() * keep
    for fwd, bwd, base in ((qn.mx4_linear_fwd, qn.mx4_linear_bwd, w),
                           (qn.qlora_linear_fwd, qn.qlora_linear_bwd, st)):
        _, u = fwd(base, d["x"], d["A"], d["B"], 32.0, drop=drop)
        _, dA, dB = bwd(base, d["x"], d["dY"], d["A"], d["B"], 32.0, u, drop=drop)
        s = 2.0 * f
        for got, want in ((dA, s * (G @ B).t() @ x), (dB, s * G.t() @ u.double())):
            assert float((got.double() - want).norm() / want.norm()) <= 1e-6


def test_backward_without_adapter(qn):
    say("[mx4 bwd r=0]")
    for M, rows, cols in [(1, 8, 64), (33, 72, 320), (300, 264, 576)]:
        w, d = _linear(qn, M, rows, cols, 1)
        dX, dA, dB = qn.mx4_linear_bwd(w, None, d["dY"])
        assert dA is None and dB is None
        G, b = d["dY"].double(), _values(w, qn)
        _check(dX, G @ b, _bound(G @ b, G.abs() @ b.abs(), rows), "dX")


def test_gradients_against_differences(qn):
    """With W = 0 the linear is u B^T alone, linear in each of x, A and B, so that
    central differences of sum(dY y) with whole steps are its gradients up to the
    rounding of y (2^-8 of each element, both sides): held to that."""
    say("[mx4 differences]")
    M, rows, cols, r = 33, 72, 192, 9
    _, d = _linear(qn, M, rows, cols, r)
    w = qn.mx4_quantize(torch.zeros(rows, cols, device="cuda"))
    drop = qn.Dropout(0.25, 4, offset=1)
    dX, dA, dB = qn.mx4_linear_bwd(w, d["x"], d["dY"], d["A"], d["B"], 18.0, drop=drop)
    G = d["dY"].double()
    for name, grad in (("x", dX), ("A", dA), ("B", dB)):
        step = _normal(77, *d[name].shape, std=float(d[name].double().std()))
        ys = []
        for sign in (1, -1):
            moved = dict(d)
            moved[name] = (d[name] + sign * step).to(torch.bfloat16)
            y, _ = qn.mx4_linear_fwd(w, moved["x"], moved["A"], moved["B"], 18.0, drop=drop)
            ys.append((moved[name].double(), y.double()))
        got = float((grad.double() * (ys[0][0] - ys[1][0])).sum())
        want = float((G * (ys[0][1] - ys[1][1])).sum())
        noise = float((G.abs() * (ys[0][1].abs() + ys[1][1].abs())).sum()) * 2.0 ** -8
        noise += float((grad.double().abs() * (ys[0][0] - ys[1][0]).abs()).sum()) * 2.0 ** -8
        assert abs(got - want) <= noise, (name, got, want, noise)


# ------------------------------------------------------------ how they are called
def test_empty_batches(qn):
    say("[mx4 empty]")
    w, d = _linear(qn, 4, 64, 128, 4)
    x = d["x"][:0]
    y, u = qn.mx4_linear_fwd(w, x, d["A"], d["B"], 8.0)
    assert y.shape == (0, 64) and u.shape == (0, 4)
    dX, dA, dB = qn.mx4_linear_bwd(w, x, d["dY"][:0], d["A"], d["B"], 8.0)
    assert dX.shape == (0, 128) and not dA.any() and not dB.any()


def test_streams_graphs_and_workspaces(qn):
    """Captured and replayed with new inputs and eager calls between, on a stream of
    its own, a workspace shared with the NF4 linear's calls."""
    say("[mx4 graph]")
    M, rows, cols, r = 70, 136, 320, 16
    w, d = _linear(qn, M, rows, cols, r)
    st = qn.nf4_quantize_dq(_normal(8, rows, cols, dtype=torch.float32))
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    drop = qn.Dropout(0.3, 12, offset=2, step=step)
    L = qn.load_library()
    need = max(L.mx4_linear_workspace(M, rows, cols, r, b, 0, 1) for b in (0, 1))
    need = max(need, L.qlora_linear_drop_workspace(M, rows, cols, r, 1, 0))
    ws = qn.linear_workspace(need)

    def both(ws=None):
        y, u = qn.mx4_linear_fwd(w, d["x"], d["A"], d["B"], 32.0, drop=drop, workspace=ws)
        z, v = qn.qlora_linear_fwd(st, d["x"], d["A"], d["B"], 32.0, drop=drop, workspace=ws)
        g = qn.mx4_linear_bwd(w, d["x"], d["dY"], d["A"], d["B"], 32.0, u, drop=drop, workspace=ws)
        h = qn.qlora_linear_bwd(st, d["x"], d["dY"], d["A"], d["B"], 32.0, v, drop=drop, workspace=ws)
        return (y, u, z, v) + g + h

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both(ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = both(ws)
    for k in range(4):
        d["x"].copy_(_normal(100 + k, M, cols))
        step.fill_(k * 3)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = both()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        if k:
            assert not torch.equal(got[1], last)
        last = got[1]


def test_two_calls_at_once(qn):
    say("[mx4 two streams]")
    w, d = _linear(qn, 200, 264, 576, 8)
    want = qn.mx4_linear_fwd(w, d["x"], d["A"], d["B"], 8.0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(qn.mx4_linear_fwd(w, d["x"], d["A"], d["B"], 8.0))
    torch.cuda.synchronize()
    for y, u in got:
        assert torch.equal(y, want[0]) and torch.equal(u, want[1])


def test_refusals_on_the_device(qn):
    say("[mx4 refusals]")
    w, d = _linear(qn, 4, 64, 128, 4)
    x, A, B, G = d["x"], d["A"], d["B"], d["dY"]
    with pytest.raises(ValueError):
        qn.mx4_linear_fwd(w, x.float(), A, B, 8.0)
    with pytest.raises(ValueError):
        qn.mx4_linear_fwd(w, x[:, :64], A, B, 8.0)
    with pytest.raises(ValueError):
        qn.mx4_linear_fwd(w, x, A, None, 8.0)
    with pytest.raises(ValueError):
        qn.mx4_linear_fwd(w, x, A, B[:32], 8.0)
    with pytest.raises(ValueError):
        qn.mx4_linear_fwd(w, x, drop=qn.Dropout(0.1, 1))
    with pytest.raises(ValueError):
        qn.mx4_linear_fwd(qn.MX4(w.codes, w.scales[:1], 64, 128), x, A, B, 8.0)
    with pytest.raises(ValueError):
        qn.mx4_linear_bwd(w, qn.act8_pack(x), G, A, B, 8.0)  # no u
    with pytest.raises(ValueError):
        qn.qlora_linear_fwd(qn.nf4_quantize_dq(_normal(1, 64, 128, dtype=torch.float32)), x, A, B,
                            8.0, drop=qn.Dropout(0.1, 1), dropout_p=0.1)
    odd = qn.mx4_quantize(_normal(1, 63, 128))
    with pytest.raises(qn.QNError):
        qn.mx4_linear_fwd(odd, x, A, B.new_zeros(63, 4), 8.0)


def test_inputs_on_no_boundary(qn):
    say("[mx4 boundaries]")
    w, d = _linear(qn, 6, 64, 128, 4)
    off = lambda t: torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(t.shape)  # noqa: E731
    y, u = qn.mx4_linear_fwd(w, d["x"], d["A"], d["B"], 8.0)
    m = {k: off(v) for k, v in d.items()}
    y2, u2 = qn.mx4_linear_fwd(w, m["x"], m["A"], m["B"], 8.0)
    assert torch.equal(y, y2) and torch.equal(u, u2)
    want = qn.mx4_linear_bwd(w, d["x"], d["dY"], d["A"], d["B"], 8.0, u)
    got = qn.mx4_linear_bwd(w, m["x"], m["dY"], m["A"], m["B"], 8.0, off(u))
    for a, b in zip(got, want):
        assert torch.equal(a, b)
