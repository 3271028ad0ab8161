"""Dropout from a counter: the mask bit for bit, by itself, in the linears on both
base weights, and through the modules."""
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


def _bits(keep):
    """The keep mask as the linear calls take a stored one."""
    return torch.from_numpy(np.packbits(keep, bitorder="little")).cuda()


@pytest.mark.parametrize("n", [1, 7, 8, 9, 4096, 4097, 10007])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("p,seed,offset", [(0.5, 0, 0), (0.1, (1 << 64) - 1, 1 << 33),
                                           (0.999999, 5, 6), (1e-9, 3, 0)])
def test_apply(qn, n, dtype, p, seed, offset):
    say(f"[drop] n={n} {dtype} p={p}")
    x = _normal(n, n, dtype=dtype)
    keep, f = _mx4.keep(n, p, seed, offset)
    scale = torch.tensor(f, dtype=torch.float32)
    want = torch.where(torch.from_numpy(keep), x.float().cpu() * scale, torch.zeros(n)).to(dtype)
    drop = qn.Dropout(p, seed, offset)
    got = qn.dropout_apply(x, drop)
    assert torch.equal(got.cpu(), want)
    buf = torch.cat([x, x.new_full((16,), 9.0)])
    qn.dropout_apply(buf[:n], drop, out=buf[:n])  # in place, nothing behind it
    assert torch.equal(buf[:n].cpu(), want) and bool((buf[n:] == 9.0).all())
    odd = torch.cat([x.new_zeros(1), x])[1:]
    assert torch.equal(qn.dropout_apply(odd, drop).cpu(), want)


def test_apply_drops_what_is_no_number_and_passes_the_rest(qn):
    say("[drop nan]")
    x = torch.full((4096,), float("nan"), device="cuda")
    keep, _ = _mx4.keep(4096, 0.4, 8)
    got = qn.dropout_apply(x, qn.Dropout(0.4, 8)).cpu()
    assert torch.equal(torch.isnan(got), torch.from_numpy(keep))
    assert bool((got[~torch.from_numpy(keep)] == 0).all())
    assert torch.equal(qn.dropout_apply(x[:0], qn.Dropout(0.4, 8)), x[:0])


def test_apply_past_32_bits(qn):
    """Elements and blocks past 2^32."""
    say("[drop far]")
    n = (1 << 32) + 8 * 5 + 3
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    drop = qn.Dropout(0.5, 21)
    qn.dropout_apply(x, drop, out=x)
    first = (1 << 29) - 4
    keep, f = _mx4.keep(n - 8 * first, 0.5, 21, first=first)
    want = torch.from_numpy(np.where(keep, f, 0.0)).to(torch.bfloat16)
    assert torch.equal(x[8 * first:].cpu(), want)


def test_share_and_independence(qn):
    """About p of many elements, in every half word, and no more agreement between
    offsets, seeds or steps than chance: 2^22 draws, six standard deviations."""
    say("[drop share]")
    n, p = 1 << 22, 0.1
    ones = torch.ones(n, device="cuda")
    masks = [qn.dropout_apply(ones, d) == 0 for d in (
        qn.Dropout(p, 1), qn.Dropout(p, 2), qn.Dropout(p, 1, offset=1),
        qn.Dropout(p, 1, step=torch.tensor([2], device="cuda")))]
    t = round(p * 65536) / 65536
    for m in masks:
        for q in range(8):
            share = float(m[q::8].double().mean())
            assert abs(share - t) <= 6 * (t * (1 - t) / (n / 8)) ** 0.5
    for i in range(4):
        for j in range(i):
            both = float((masks[i] & masks[j]).double().mean())
            assert abs(both - t * t) <= 6 * (t * t / n) ** 0.5


def test_gradient_and_step(qn):
    say("[drop grad]")
    x = _normal(1, 33, 77, dtype=torch.float32).requires_grad_()
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    drop = qn.Dropout(0.3, 5, step=step)
    y = qn.dropout(x, drop)
    g = _normal(2, 33, 77, dtype=torch.float32)
    y.backward(g)
    assert torch.equal(x.grad, qn.dropout_apply(g, drop))
    # linear: whole differences are the gradient
    d = _normal(3, 33, 77, dtype=torch.float32)
    diff = qn.dropout_apply(x.detach() + d, drop).double() - qn.dropout_apply(x.detach(), drop)
    lhs, rhs = float((diff * g).sum()), float((x.grad.double() * d).sum())
    mag = float((g.double().abs() * (y.detach().double().abs() + diff.abs())).sum())
    assert abs(lhs - rhs) <= 4 * 2.0 ** -24 * mag
    y = qn.dropout(x, drop)
    step.add_(1)
    with pytest.raises(RuntimeError):  # the mask would be another one
        y.backward(g)
    assert qn.dropout(x, None) is x


# M, rows, cols, r: every route of the NF4 linear: products of 32 rows, of 128 x 128 and
# the dense one, u with ranks up to 16 and past them
LINEAR = [(1, 8, 64, 1), (7, 72, 192, 16), (60, 8208, 320, 5), (100, 136, 1088, 40), (130, 136, 576, 20), (300, 64, 1024, 64),
          (2050, 2112, 72 * 64, 16), (2048, 2048, 256, 33)]


@pytest.mark.parametrize("M,rows,cols,r", LINEAR)
@pytest.mark.parametrize("act8", [False, True])
def test_nf4_linear_takes_the_same_mask(qn, M, rows, cols, r, act8):
    """The results are those of a stored mask of the same bits, up to the order of the
    sums (other routes: fp32 sums of the same bf16 products, then one rounding each: two
    half steps of bf16 apart) and, in dA and dB, to how finely u and v enter."""
    say(f"[drop linear] M={M} rows={rows} cols={cols} r={r} act8={act8}")
    st = qn.nf4_quantize_dq(_normal(1, rows, cols, std=0.02, dtype=torch.float32))
    x, G = _normal(2, M, cols), _normal(3, M, rows)
    A, B = _normal(4, r, cols, std=0.1), _normal(5, rows, r, std=0.1)
    p = 0.125  # exact in both
    drop = qn.Dropout(p, 77, offset=8)
    ones = torch.ones(M * cols, device="cuda")
    keep = (qn.dropout_apply(ones, drop) != 0).cpu().numpy()
    if M * cols < 1 << 16:
        assert np.array_equal(keep, _mx4.keep(M * cols, p, 77, 8)[0])
    mask = dict(dropout_mask=_bits(keep), dropout_p=p)
    y, u = qn.qlora_linear_fwd(st, x, A, B, 16.0, drop=drop)
    y2, u2 = qn.qlora_linear_fwd(st, x, A, B, 16.0, **mask)
    assert torch.equal(u, u2)
    W = qn.nf4_dequantize(st).double().abs()
    k = torch.from_numpy(keep).view(M, cols).cuda()
    s = 16.0 / r / (1 - p)

    def near(a, b, magnitude, terms, name):
        over = (a.double() - b.double()).abs() - 2.0 ** -7 * b.double().abs()
        assert float((over - (terms * 2.0 ** -23 + 2.0 ** -15) * magnitude).max()) <= 0, name

    near(y, y2, x.double().abs() @ W.t() + s * u.double().abs() @ B.double().abs().t(), cols + r, "y")
    if act8:
        x8 = qn.act8_pack(x)
        got = qn.qlora_linear_bwd_act8(st, x8, G, A, B, 16.0, u, drop=drop)
        want = qn.qlora_linear_bwd_act8(st, x8, G, A, B, 16.0, u, **mask)
    else:
        got = qn.qlora_linear_bwd(st, x, G, A, B, 16.0, u, drop=drop)
        want = qn.qlora_linear_bwd(st, x, G, A, B, 16.0, u, **mask)
        again = qn.qlora_linear_bwd(st, x, G, A, B, 16.0, drop=drop)  # u formed again
        assert torch.allclose(again[2], got[2], rtol=0, atol=float(got[2].abs().max()) * 2.0 ** -15)
    xv = (qn.act8_unpack(x8) if act8 else x).double() * k
    v = (G.double().abs() @ B.double().abs())
    tol = ((M + rows) * 2.0 ** -23 + 2.0 ** -15) * s
    near(got[0], want[0], G.double().abs() @ W + s * k * (v @ A.double().abs()), rows + r, "dX")
    assert float(((got[1] - want[1]).double().abs() - tol * v.t() @ xv.abs()).max()) <= 0
    assert float(((got[2] - want[2]).double().abs() - tol * G.double().abs().t() @ u.double().abs()
                  ).max()) <= 0


@pytest.mark.parametrize("M,rows,cols,r", [(300, 136, 320, 7), (1000, 1152, 1088, 16),
                                           (300, 136, 1344, 7), (70, 1344, 8192, 40),
                                           (1030, 2112, 2112, 33)])
def test_nf4_linear_by_a_few_tiles(qn, M, rows, cols, r):
    test_nf4_linear_takes_the_same_mask(qn, M, rows, cols, r, False)


@pytest.mark.parametrize("M,rows,cols,r", [(1, 64, 1024, 8), (3, 4096, 4096, 16), (16, 64, 2048, 40),
                                           (40, 136, 320, 7), (2050, 2112, 4608, 16)])
@pytest.mark.parametrize("p", [0.0, 1e-7])
def test_dropping_nothing_is_the_linear_itself(qn, M, rows, cols, r, p):
    """A threshold of zero: every route of the call without dropout, in workspaces that
    hold anything."""
    say(f"[drop none] M={M} rows={rows} cols={cols} r={r} p={p}")
    st = qn.nf4_quantize_dq(_normal(1, rows, cols, std=0.02, dtype=torch.float32))
    x, G = _normal(2, M, cols), _normal(3, M, rows)
    A, B = _normal(4, r, cols, std=0.1), _normal(5, rows, r, std=0.1)
    drop = qn.Dropout(p, 1)
    L = qn.load_library()
    ws = [torch.full((L.qlora_linear_drop_workspace(M, rows, cols, r, b, 0),), 255,
                     dtype=torch.uint8, device="cuda") for b in (0, 1)]
    want = qn.qlora_linear_fwd(st, x, A, B, 16.0)
    grads = qn.qlora_linear_bwd(st, x, G, A, B, 16.0, want[1])
    for k in range(2):
        got = qn.qlora_linear_fwd(st, x, A, B, 16.0, drop=drop, workspace=ws[0])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        got = qn.qlora_linear_bwd(st, x, G, A, B, 16.0, want[1], drop=drop, workspace=ws[1])
        assert all(torch.equal(a, b) for a, b in zip(got, grads))
    x8 = qn.act8_pack(x)
    want = qn.qlora_linear_bwd_act8(st, x8, G, A, B, 16.0, want[1])
    got = qn.qlora_linear_bwd_act8(st, x8, G, A, B, 16.0, qn.qlora_linear_fwd(st, x, A, B, 16.0)[1],
                                   drop=drop)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("base", ["nf4", "mx4"])
@pytest.mark.parametrize("act8", [False, True])
def test_modules(qn, base, act8):
    """A QLoRALinear under a seed: forward and gradients are the calls', every forward
    draws another mask, evaluation draws none."""
    say(f"[drop module] {base} act8={act8}")
    torch.manual_seed(0)
    lin = qn.QLoRALinear(torch.randn(64, 128, device="cuda") * 0.1, r=8, alpha=16.0, dropout=0.2,
                         act8=act8, base=base, seed=9)
    with torch.no_grad():
        lin.lora_B.copy_(_normal(6, 64, 8, std=0.1))
    x = _normal(7, 2, 17, 128).requires_grad_()
    g = _normal(8, 2, 17, 64)
    y = lin(x)
    y.backward(g)
    x2, g2 = x.detach().view(34, 128), g.view(34, 64)
    drop = qn.Dropout(0.2, 9, offset=0)
    from quantized_fine_tuning_nf4_amd.mx4 import linear_bwd, linear_fwd
    want, u = linear_fwd(lin.st, x2, lin.lora_A, lin.lora_B, 16.0, drop=drop)
    assert torch.equal(y.view(34, 64), want)
    keep = qn.act8_pack(x2) if act8 else x2
    dX, dA, dB = linear_bwd(lin.st, keep, g2, lin.lora_A, lin.lora_B, 16.0, u, drop=drop)
    assert torch.equal(x.grad.view(34, 128), dX)
    assert torch.equal(lin.lora_A.grad, dA.to(torch.bfloat16))
    assert torch.equal(lin.lora_B.grad, dB.to(torch.bfloat16))
    assert not torch.equal(lin(x), y) and lin.draws == 2
    lin.eval()
    with torch.no_grad():
        a, b = lin(x), lin(x)
    assert torch.equal(a, b) and lin.draws == 2


def test_from_fine_tuning_to_serving(qn):
    """A run as it would be used: adapters trained on NF4 weights under a seeded dropout,
    merged, stored in MXFP4, trained on there too, and asked token by token."""
    say("[drop run]")
    torch.manual_seed(1)
    W = torch.randn(512, 256, device="cuda") * 256 ** -0.5
    lin = qn.QLoRALinear(W, r=8, alpha=16.0, dropout=0.1, seed=3)
    opt = [qn.Adam8(p.detach().float().contiguous(), lr=1e-2) for p in lin.parameters()]
    x = _normal(1, 256, 256)
    targets = torch.randint(0, 512, (256,), device="cuda")
    for _ in range(3):
        loss = -qn.token_logprobs(lin(x), targets).logp.mean()
        loss.backward()
        with torch.no_grad():
            for o, p in zip(opt, lin.parameters()):
                o.step(p.grad.float().contiguous(), p.data)
                p.grad = None
    merged = qn.nf4_merge_lora(lin.st, lin.lora_A.detach(), lin.lora_B.detach(), 16.0)
    w = qn.mx4_quantize(merged)
    batch, _ = qn.mx4_linear_fwd(w, x)
    for m in (0, 100, 255):  # one token gives what it gives in the batch, up to the sums' order
        one, _ = qn.mx4_linear_fwd(w, x[m:m + 1])
        tol = 2.0 ** -7 * batch[m].double().abs() + 1e-4
        assert bool(((one[0].double() - batch[m].double()).abs() <= tol).all())
    r = qn.token_logprobs_fwd(batch, targets, top_k=3)
    assert bool(torch.isfinite(r.logp).all()) and int(r.top_ids.min()) >= 0
    served = qn.QLoRALinear(merged, r=8, alpha=16.0, dropout=0.1, base="mx4", seed=4)
    assert torch.equal(served.st.codes, w.codes)
    loss = -qn.token_logprobs(served(x), targets).logp.mean()
    loss.backward()
    assert served.lora_B.grad is not None and bool(torch.isfinite(served.lora_B.grad).all())
