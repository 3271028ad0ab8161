"""Token log probabilities (token_logprobs_fwd / _bwd) against a plain fp64
form on the CPU.

Tolerances.  A logit's t = scale (x - m) is off by 2^-23 |t|, e^t by that and
2^-22 more; the sums S and W run over chains of at most V / 64 terms joined in
trees, all of one sign: at most (V / 64 + 64) 2^-24 relative, and never more
than 2e-5 at the sizes below; ln S is off by that, a log probability by that
plus 2^-22 |t|.  The entropy's two terms cancel at most to their own size.
"""
import math

import numpy as np
import pytest
import torch

from tests._gpu import needs_gpu, say

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.fixture(scope="module")
def qn():
    import quantized_fine_tuning_nf4_amd as qn
    qn.load_library()
    return qn


def _tol(V):
    return (V / 64 + 64) * 2.0 ** -24 + 2.0 ** -20


def _ref(x, targets, scale, k):
    """fp64: logp, entropy, top values and ids (ties to the lower index)."""
    x = x.cpu().double()
    T, V = x.shape
    z = x * scale
    m = z.max(dim=1, keepdim=True).values
    empty = torch.isneginf(m)
    t = z - torch.where(empty, torch.zeros_like(m), m)
    lse = t.exp().sum(1, keepdim=True).log()
    lp = torch.where(torch.isneginf(t), t, t - lse)
    p = lp.exp()
    H = -(p * torch.where(p > 0, lp, torch.zeros_like(lp))).sum(1)
    out = dict(lp=lp, H=H, p=p)
    if targets is not None:
        tg = targets.cpu()
        v = lp.gather(1, tg.clamp(0, V - 1)[:, None])[:, 0]
        v = torch.where(tg < 0, torch.zeros_like(v), v)
        out["logp"] = torch.where(tg >= V, torch.full_like(v, math.nan), v)
    if k:
        ids, vals = np.full((T, k), -1), np.full((T, k), -np.inf)
        xs = x.numpy()
        for r in range(T):
            order = np.lexsort((np.arange(V), -xs[r]))[:k]
            order = order[xs[r][order] > -np.inf]
            ids[r, :len(order)] = order
            vals[r, :len(order)] = lp[r].numpy()[order]
        out["ids"], out["vals"] = ids, vals
    return out


def _same(got, ref, tol, scale=1.0):
    """Equal where the reference is not finite, within tol elsewhere."""
    got, ref = got.detach().cpu().double(), torch.as_tensor(ref).double()
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    assert torch.equal(got[~fin & ~torch.isnan(ref)], ref[~fin & ~torch.isnan(ref)])
    err = (got - ref).abs()[fin]
    lim = (tol * (1.0 + scale * ref.abs()))[fin]
    assert (err <= lim).all(), float((err / lim).max())


def _logits(T, V, f32, seed, std=2.5, pad=0, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, V + pad, generator=g) * std + offset
    x = x.to(torch.float32 if f32 else torch.bfloat16).cuda()
    t = torch.randint(0, V, (T,), generator=g)
    return x[:, :V], t.cuda()


def _check(qn, x, t, scale=1.0, k=0):
    r = qn.token_logprobs_fwd(x, t, scale=scale, top_k=k)
    torch.cuda.synchronize()
    ref = _ref(x, t, scale, k)
    tol = _tol(x.shape[1])
    if t is None:
        assert r.logp is None
    else:
        _same(r.logp, ref["logp"], tol)
    _same(r.entropy, ref["H"], 2 * tol)
    if k:
        assert np.array_equal(r.top_ids.cpu().numpy(), ref["ids"])
        _same(r.top_logp, ref["vals"], tol)
    return r, ref


SIZES = [(1, 1), (3, 2), (2, 7), (5, 63), (4, 64), (7, 65), (1, 511), (6, 513), (3, 1000),
         (2, 2047), (300, 257), (1, 4099), (17, 8192), (2, 32000), (9, 50021), (1, 131072),
         (256, 8192), (100, 30011),
         (5, 131075), (40, 16384), (600, 1024)]


@pytest.mark.parametrize("T,V", SIZES)
@pytest.mark.parametrize("f32", [False, True])
def test_forward(qn, T, V, f32):
    for k in (0, 1, 5, 20, 32):
        if k > V:
            continue
        say(f"[logprobs] T={T} V={V} f32={f32} k={k}")
        x, t = _logits(T, V, f32, seed=T * 3 + V + k, pad=(k * 3) % 7)
        _check(qn, x, t, scale=1.0 if k != 5 else 0.7, k=k)


@pytest.mark.parametrize("f32", [False, True])
def test_ties_go_to_the_lower_index(qn, f32):
    V = 9000
    g = torch.Generator().manual_seed(1)
    for T, few in ((2, 1), (3, 2), (300, 3), (2, 40)):
        x = torch.randint(0, few, (T, V), generator=g).float()
        x = x.to(torch.float32 if f32 else torch.bfloat16).cuda()
        for k in (1, 7, 32):
            say(f"[logprobs ties] T={T} values={few} k={k} f32={f32}")
            _check(qn, x, torch.zeros(T, dtype=torch.int64, device="cuda"), k=k)
    # minus zero equals zero
    x = torch.zeros(1, 300)
    x[0, ::2] = -0.0
    r = qn.token_logprobs_fwd(x.cuda(), top_k=6)
    assert r.top_ids.tolist() == [[0, 1, 2, 3, 4, 5]]


@pytest.mark.parametrize("order", ["up", "down"])
@pytest.mark.parametrize("T", [1, 400])
def test_sorted_rows(qn, T, order):
    """Every logit a new maximum, or none after the first."""
    V = 20000
    x = torch.linspace(-8, 8, V).repeat(T, 1)
    x = (x if order == "up" else x.flip(1)).cuda()
    say(f"[logprobs sorted] T={T} {order}")
    r = qn.token_logprobs_fwd(x, top_k=32)
    want = list(range(V - 1, V - 33, -1)) if order == "up" else list(range(32))
    assert (r.top_ids.cpu() == torch.tensor(want)).all()
    ref = torch.log_softmax(x[0].cpu().double(), 0)
    _same(r.top_logp[0], ref[want], _tol(V))


@pytest.mark.parametrize("f32", [False, True])
def test_masks(qn, f32):
    low = torch.finfo(torch.float32 if f32 else torch.bfloat16).min
    for T in (6, 520):
        say(f"[logprobs masks] T={T} f32={f32}")
        x, t = _logits(T, 5003, f32, seed=5)
        x = x.contiguous()
        x[0] = -math.inf                  # nothing allowed
        x[1] = -math.inf
        x[1, 4321] = 3.0                  # one token allowed
        x[2, ::2] = -math.inf             # a target among the banned ones
        t[2] = 4
        x[3] = low                        # every logit the type's lowest value
        x[4, 1:] = low                    # all but one masked by it
        x[5, :3000] = -math.inf
        t[1], t[0] = 4321, 7
        r, ref = _check(qn, x, t, k=8)
        assert math.isinf(float(r.logp[0])) and float(r.entropy[0]) == 0.0
        assert float(r.entropy[1]) == 0.0 and float(r.logp[1]) == 0.0
        assert abs(float(r.entropy[3]) - math.log(5003)) < 1e-5
        assert torch.isneginf(r.logp[2])
        dx = qn.token_logprobs_bwd(x, t, r.stats, r.entropy, torch.ones(T, device="cuda"),
                                   torch.ones(T, device="cuda"))
        torch.cuda.synchronize()
        assert torch.isfinite(dx).all()
        assert not dx[0].any()
        banned = torch.isneginf(x)
        banned[torch.arange(T), t] = False
        assert not dx[banned].any()


def test_nan_and_inf_rows(qn):
    x, t = _logits(5, 3001, True, seed=6)
    x = x.contiguous()
    x[1, 2000] = math.nan
    x[3, 5] = math.inf
    r = qn.token_logprobs_fwd(x, t, top_k=3)
    for row in range(5):
        bad = row in (1, 3)
        assert bool(torch.isnan(r.logp[row])) == bad
        assert bool(torch.isnan(r.entropy[row])) == bad


@pytest.mark.parametrize("f32", [False, True])
def test_ignored_and_impossible_targets(qn, f32):
    for T in (5, 300):
        x, t = _logits(T, 777, f32, seed=7)
        t[0], t[1], t[2] = -1, -100, 777
        t[3] = 1 << 40
        r, ref = _check(qn, x, t, k=2)
        assert r.logp[0] == 0 and r.logp[1] == 0 and torch.isnan(r.logp[2:4]).all()
        g = torch.ones(T, device="cuda")
        dx = qn.token_logprobs_bwd(x, t, r.stats, r.entropy, g)
        assert not dx[:4].any() and dx[4].any()


def test_large_offsets_keep_their_precision(qn):
    """Logits far from zero: only differences enter."""
    x, t = _logits(4, 4096, True, seed=8)
    y = x + 4096.0
    a = qn.token_logprobs_fwd(y, t)
    ref = _ref(y, t, 1.0, 0)
    _same(a.logp, ref["logp"], _tol(4096))
    dx = qn.token_logprobs_bwd(y, t, a.stats, a.entropy, torch.ones(4, device="cuda"))
    onehot = torch.zeros(4, 4096, dtype=torch.double)
    onehot[torch.arange(4), t.cpu()] = 1
    assert ((dx.cpu().double() - (onehot - ref["p"])).abs() <= 1e-5 * (onehot + ref["p"])).all()


@pytest.mark.parametrize("T,V", [(1, 1), (3, 7), (2, 64), (5, 1001), (300, 333), (4, 32000),
                                 (2, 50021), (1, 131072)])
@pytest.mark.parametrize("f32", [False, True])
def test_backward(qn, T, V, f32):
    for pad, ent, given in ((0, True, True), (3, False, True), (8, True, False)):
        say(f"[logprobs bwd] T={T} V={V} f32={f32} pad={pad} entropy={ent} logp={given}")
        x, t = _logits(T, V, f32, seed=T + V + pad, pad=pad)
        scale = 0.8 if pad == 3 else 1.0
        g = torch.Generator().manual_seed(V)
        dl = torch.randn(T, generator=g).cuda() if given else None
        de = torch.randn(T, generator=g).cuda() if ent else None
        r = qn.token_logprobs_fwd(x, t, scale=scale)
        dx = qn.token_logprobs_bwd(x, t if given else None, r.stats, r.entropy if ent else None,
                                   dl, de, scale=scale)
        torch.cuda.synchronize()
        ref = _ref(x, t, scale, 0)
        p, lp, H = ref["p"], ref["lp"], ref["H"][:, None]
        want, mag = torch.zeros_like(p), torch.zeros_like(p)
        if given:
            hot = torch.zeros_like(p)
            hot[torch.arange(T), t.cpu()] = 1
            d = dl.cpu().double()[:, None]
            want, mag = want + d * (hot - p), mag + d.abs() * (hot + p)
        if ent:
            d = de.cpu().double()[:, None]
            want, mag = want - d * p * (lp + H), mag + d.abs() * p * (lp.abs() + H + 1)
        tol = scale * mag * (_tol(V) * 4 + lp.abs() * 2.0 ** -21) + 1e-37
        got = dx.cpu().double()
        if not f32:
            tol = tol + 2.0 ** -8 * (scale * want).abs()
        assert ((got - scale * want).abs() <= tol).all()


@pytest.mark.parametrize("f32", [False, True])
def test_backward_in_place_and_into_wider_rows(qn, f32):
    for V, pad in ((513, 0), (1024, 8), (1001, 3)):
        x, t = _logits(37, V, f32, seed=V, pad=pad)
        g = torch.randn(37, device="cuda")
        r = qn.token_logprobs_fwd(x, t)
        ref = qn.token_logprobs_bwd(x, t, r.stats, r.entropy, g, g)
        wide = torch.full((37, V + 5), 9.0, dtype=x.dtype, device="cuda")
        qn.token_logprobs_bwd(x, t, r.stats, r.entropy, g, g, out=wide[:, :V])
        assert torch.equal(wide[:, :V], ref) and (wide[:, V:] == 9.0).all()
        got = qn.token_logprobs_bwd(x, t, r.stats, r.entropy, g, g, out=x)
        assert got is x and torch.equal(x, ref)


def test_gradient_against_differences(qn):
    T, V, step = 3, 40, 1e-5
    x, t = _logits(T, V, True, seed=11, std=1.0)
    w = torch.randn(2, T, dtype=torch.double)
    r = qn.token_logprobs_fwd(x, t, scale=1.3)
    dx = qn.token_logprobs_bwd(x, t, r.stats, r.entropy, w[0].float().cuda(),
                               w[1].float().cuda(), scale=1.3).cpu().double()
    base = x.cpu().double()

    def loss(v):
        q = _ref(v, t, 1.3, 0)
        return float((w[0] * q["logp"]).sum() + (w[1] * q["H"]).sum())

    for i in range(T):
        for j in range(0, V, 3):
            a, b = base.clone(), base.clone()
            a[i, j] += step
            b[i, j] -= step
            assert abs((loss(a) - loss(b)) / (2 * step) - float(dx[i, j])) < 2e-6


def test_misaligned_views_and_another_stream(qn):
    """Rows that start on any element, and a caller's own stream."""
    for f32 in (False, True):
        x, t = _logits(9, 3000, f32, seed=12)
        for at in (1, 2, 3, 5, 8):
            v = x[:, at:at + 2001]
            tv = t % 2001
            _check(qn, v, tv, k=4)
        side = torch.cuda.Stream()
        a = qn.token_logprobs_fwd(x, t, top_k=9)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            b = qn.token_logprobs_fwd(x, t, top_k=9)
            db = qn.token_logprobs_bwd(x, t, b.stats, b.entropy, b.logp)
        side.synchronize()
        da = qn.token_logprobs_bwd(x, t, a.stats, a.entropy, a.logp)
        assert all(torch.equal(p, q) for p, q in zip(a, b)) and torch.equal(da, db)


def test_rows_past_32_bit_offsets(qn):
    """A few rows far apart: row starts past 2^32 bytes."""
    V, ld, T = 1000, (1 << 29) + 8, 6
    x = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda").as_strided((T, V), (ld, 1))
    small, t = _logits(T, V, False, seed=13)
    x.copy_(small)
    say(f"[logprobs far rows] T={T} V={V} ld={ld}")
    a = qn.token_logprobs_fwd(x, t, top_k=3)
    b = qn.token_logprobs_fwd(small, t, top_k=3)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    qn.token_logprobs_bwd(x, t, a.stats, a.entropy, a.logp, out=x)
    ref = qn.token_logprobs_bwd(small, t, b.stats, b.entropy, b.logp)
    assert torch.equal(x, ref)


@pytest.mark.parametrize("T", [1, 2, 700])
def test_graph_replays(qn, T):
    x, t = _logits(T, 40000, False, seed=14)
    ones = torch.ones(T, device="cuda")

    def step():
        r = qn.token_logprobs_fwd(x, t, top_k=20)
        return [*r, qn.token_logprobs_bwd(x, t, r.stats, r.entropy, ones, ones)]

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


def test_empty_and_no_targets(qn):
    x, t = _logits(3, 100, False, seed=15)
    r = qn.token_logprobs_fwd(x[:0], t[:0], top_k=2)
    assert r.logp.shape == (0,) and r.top_ids.shape == (0, 2)
    assert qn.token_logprobs_bwd(x[:0], t[:0], r.stats, r.entropy, r.logp).shape == (0, 100)
    _check(qn, x, None, k=4)


def test_autograd(qn):
    x, t = _logits(6, 301, True, seed=16)
    x = x.contiguous().requires_grad_(True)
    t[2] = -1
    r = qn.token_logprobs(x, t, top_k=3)
    loss = -r.logp.sum() / 5 - 0.01 * r.entropy.mean()
    loss.backward()
    y = x.detach().cpu().double().requires_grad_(True)
    lp = torch.log_softmax(y, 1)
    keep = t.cpu() >= 0
    got = lp.gather(1, t.cpu().clamp(min=0)[:, None])[:, 0] * keep
    (-got.sum() / 5 + 0.01 * (lp.exp() * lp).sum(1).mean()).backward()
    assert float((x.grad.cpu().double() - y.grad).norm() / y.grad.norm()) < 1e-5
