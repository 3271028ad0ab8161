"""Block norms (block_norm_fwd / block_norm_bwd) against a plain fp64 form on
the CPU.

Tolerances.  A row's sums are chains of at most 128 terms joined in a tree,
the rest a fixed number of fp32 operations, so a value that is a sum of terms
t_i is off by at most C = 256 * 2^-24 of sum |t_i|; a bf16 output adds half a
unit in its last place (2^-9 relative, one more 2^-24 share where it falls on
the other side of a tie: 2^-8 bounds both).  Sums over M rows take at most
(M + 256) 2^-24 of the sum of magnitudes.
"""
import numpy as np
import pytest
import torch

from tests._gpu import needs_gpu, say

pytestmark = [pytest.mark.gpu, needs_gpu]
C = 256 * 2.0 ** -24


@pytest.fixture(scope="module")
def qn():
    import quantized_fine_tuning_nf4_amd as qn
    qn.load_library()
    return qn


def _inputs(M, D, res32, w32, post, gate, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    wt = torch.float32 if w32 else torch.bfloat16
    rt = torch.float32 if res32 else torch.bfloat16
    t = dict(h=(2 * n(M, D)).to(rt), w_pre=(1 + 0.2 * n(D)).to(wt), o=None, w_post=None, gate=None)
    if post != "none":
        t["o"] = n(M, D).to(torch.bfloat16)
    if post == "norm":
        t["w_post"] = (1 + 0.2 * n(D)).to(wt)
    if gate != "none":
        shape, dt = {"channel": ((D,), wt), "row": ((M, 1), torch.bfloat16),
                     "element": ((M, D), torch.bfloat16)}[gate]
        t["gate"] = (0.7 + 0.3 * n(*shape)).to(dt)
    t["dy"] = n(M, D).to(torch.bfloat16)
    t["dh_new"] = n(M, D).to(rt)
    return t


def _f64(t):
    return {k: None if v is None else v.double() for k, v in t.items()}


def _fwd64(t, scale, eps):
    h, mag = t["h"], t["h"].abs()
    if t["o"] is not None:
        p = t["o"]
        if t["w_post"] is not None:
            p = p / (p.square().mean(1, keepdim=True) + eps).sqrt() * t["w_post"]
        p = scale * p * (1.0 if t["gate"] is None else t["gate"])
        h, mag = h + p, mag + p.abs()
    r = 1 / (h.square().mean(1, keepdim=True) + eps).sqrt()
    return h, mag, h * r * t["w_pre"], mag * r * t["w_pre"].abs()


def _close(name, got, ref, mag, c=C):
    got = got.detach().cpu()
    tol = c * mag
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * ref.abs() + 2.0 ** -133
    else:
        tol = tol + 2.0 ** -23 * ref.abs()
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all(), name
    bad = err > tol
    assert not bad.any(), (name, int(bad.sum()), float((err / (tol + 1e-300)).max()))


def _dev(t):
    return {k: None if v is None else v.cuda() for k, v in t.items()}


def _codes64(y):
    """Codes and exponents of bf16 y by search over the powers of two."""
    v = y.detach().cpu().double().numpy()
    M, D = v.shape
    nb = (D + 63) // 64
    codes, exps = np.zeros((M, D)), np.zeros((M, nb), int)
    for b in range(nb):
        x = v[:, 64 * b:64 * b + 64]
        top = np.abs(x).max(axis=1)
        e = np.full(M, -126)
        for k in range(-126, 121):
            e = np.where(top > 127 * 2.0 ** k, k + 1, e)
        exps[:, b] = e + 127
        c = np.rint(x * 2.0 ** -e[:, None].astype(float))
        codes[:, 64 * b:64 * b + 64] = np.clip(c, -127, 127)
    return codes, exps


SHAPES = [(1, 4096), (3, 1), (2, 7), (5, 8), (4, 63), (7, 64), (3, 65), (300, 128), (33, 520),
          (9, 1000), (17, 1001), (6, 2048), (5, 4096), (4, 4100), (3, 5121), (3, 8192), (2, 8200),
          (2, 16384), (2, 16381), (3, 1024), (5, 1032)]
MODES = [("none", "none"), ("add", "none"), ("add", "row"), ("norm", "none"), ("norm", "channel"),
         ("norm", "row"), ("norm", "element"), ("add", "channel")]


@pytest.mark.parametrize("M,D", SHAPES)
@pytest.mark.parametrize("res32", [False, True])
def test_forward(qn, M, D, res32):
    for k, (post, gate) in enumerate(MODES):
        w32 = bool((k + res32) % 2)
        say(f"[norm fwd] M={M} D={D} res32={res32} w32={w32} post={post} gate={gate}")
        t = _inputs(M, D, res32, w32, post, gate, seed=M * 7 + D + k)
        d = _dev(t)
        hn, y, x8 = qn.block_norm_fwd(d["h"], d["w_pre"], o=d["o"], w_post=d["w_post"],
                                      gate=d["gate"], scale=0.5, eps=1e-6, pack=k % 2 == 0)
        torch.cuda.synchronize()
        rh, mh, ry, my = _fwd64(_f64(t), 0.5, 1e-6)
        if post == "none":
            assert hn is d["h"]
        else:
            _close("h", hn, rh, mh)
        _close("y", y, ry, my)
        if x8 is not None:
            codes, exps = _codes64(y)
            assert np.array_equal(x8.exps.cpu().numpy(), exps)
            assert np.array_equal(x8.codes.cpu().numpy(), codes)


def _bwd64(t, scale, eps):
    """Gradients by the formulas, and the magnitudes their sums run over."""
    h, dy, w = t["h"], t["dy"], t["w_pre"]
    r = 1 / (h.square().mean(1, keepdim=True) + eps).sqrt()
    n, dn = h * r, dy * w
    k, ka = (dn * n).mean(1, keepdim=True), (dn * n).abs().mean(1, keepdim=True)
    dh = t["dh_new"] + r * (dn - n * k)
    mdh = t["dh_new"].abs() + r * (dn.abs() + n.abs() * ka)
    out = dict(dh=(dh, mdh), dw_pre=((dy * n).sum(0), (dy * n).abs().sum(0)))
    if t["o"] is None:
        return out
    o, wp = t["o"], 1.0 if t["w_post"] is None else t["w_post"]
    r1 = 1.0 if t["w_post"] is None else 1 / (o.square().mean(1, keepdim=True) + eps).sqrt()
    q, g = o * r1, 1.0 if t["gate"] is None else t["gate"]
    dg, mdg = scale * q * wp * dh, (scale * q * wp).abs() * mdh
    if t["gate"] is not None:
        if t["gate"].dim() == 1:
            out["dgate"] = dg.sum(0), mdg.sum(0)
        elif t["gate"].shape[1] == 1:
            out["dgate"] = dg.sum(1, keepdim=True), mdg.sum(1, keepdim=True)
        else:
            out["dgate"] = dg, mdg
    a, ma = scale * g * dh, abs(scale) * (g.abs() if t["gate"] is not None else 1.0) * mdh
    if t["w_post"] is None:
        out["do"] = a, ma
        return out
    out["dw_post"] = (a * q).sum(0), (ma * q.abs()).sum(0)
    dq, mdq = a * wp, ma * wp.abs()
    out["do"] = (r1 * (dq - q * (dq * q).mean(1, keepdim=True)),
                 r1 * (mdq + q.abs() * (mdq * q.abs()).mean(1, keepdim=True)))
    return out


@pytest.mark.parametrize("M,D", SHAPES)
@pytest.mark.parametrize("res32", [False, True])
def test_backward(qn, M, D, res32):
    for k, (post, gate) in enumerate(MODES):
        w32, weights = bool((k + res32) % 2), k % 3 != 1
        say(f"[norm bwd] M={M} D={D} res32={res32} w32={w32} post={post} gate={gate} "
            f"weights={weights}")
        t = _inputs(M, D, res32, w32, post, gate, seed=M * 5 + D + k)
        d = _dev(t)
        g = qn.block_norm_bwd(d["dy"], d["h"], d["w_pre"], dh_new=d["dh_new"], o=d["o"],
                              w_post=d["w_post"], gate=d["gate"], scale=0.5, eps=1e-6,
                              need_weights=weights, need_gate=k != 6)
        torch.cuda.synchronize()
        ref = _bwd64(_f64(t), 0.5, 1e-6)
        # each factor of a product of sums brings its share
        _close("dh", g.dh, *ref["dh"], c=4 * C)
        assert (g.do is None) == (post == "none")
        if g.do is not None:
            _close("do", g.do, *ref["do"], c=8 * C)
        assert (g.dgate is None) == (gate == "none" or k == 6)
        if g.dgate is not None:
            _close("dgate", g.dgate, *ref["dgate"], c=8 * C + M * 2.0 ** -24)
        assert (g.dw_pre is None) == (not weights)
        if weights:
            _close("dw_pre", g.dw_pre, *ref["dw_pre"], c=8 * C + M * 2.0 ** -24)
            assert (g.dw_post is None) == (post != "norm")
            if g.dw_post is not None:
                _close("dw_post", g.dw_post, *ref["dw_post"], c=8 * C + M * 2.0 ** -24)


@pytest.mark.parametrize("M,D", [(4096, 256), (2500, 1024), (1100, 4096)])
def test_backward_sums_over_many_rows(qn, M, D):
    say(f"[norm bwd sums] M={M} D={D}")
    t = _inputs(M, D, False, True, "norm", "channel", seed=M + D)
    d = _dev(t)
    outs = []
    for _ in range(2):
        outs.append(qn.block_norm_bwd(d["dy"], d["h"], d["w_pre"], dh_new=None, o=d["o"],
                                      w_post=d["w_post"], gate=d["gate"], scale=0.5))
    torch.cuda.synchronize()
    t["dh_new"] = torch.zeros_like(t["dh_new"])
    ref = _bwd64(_f64(t), 0.5, 1e-6)
    for k in ("dw_pre", "dw_post", "dgate"):
        _close(k, getattr(outs[0], k), *ref[k], c=8 * C + M * 2.0 ** -24)
        assert torch.equal(getattr(outs[0], k), getattr(outs[1], k)), k  # fixed order
    _close("dh", outs[0].dh, *ref["dh"], c=4 * C)
    _close("do", outs[0].do, *ref["do"], c=8 * C)


def test_gradient_against_differences(qn):
    """The backward against central differences of the fp64 forward."""
    M, D, step = 3, 24, 1e-6
    t = _f64(_inputs(M, D, True, True, "norm", "channel", seed=3))
    up_h, up_y = t["dh_new"], t["dy"]
    base = {k: v.clone() for k, v in t.items() if v is not None}

    def loss(v):
        hn, _, y, _ = _fwd64({**t, **v}, 0.5, 1e-3)
        return float((hn * up_h).sum() + (y * up_y).sum())

    hn, _, _, _ = _fwd64(base, 0.5, 1e-3)
    dev = {k: v.to(torch.bfloat16 if k in ("o", "dy") else torch.float32).cuda()
           for k, v in base.items()}
    g = qn.block_norm_bwd(dev["dy"], hn.float().cuda(), dev["w_pre"], dh_new=dev["dh_new"],
                          o=dev["o"], w_post=dev["w_post"], gate=dev["gate"], scale=0.5, eps=1e-3)
    for name, got in (("h", g.dh), ("w_pre", g.dw_pre), ("w_post", g.dw_post), ("gate", g.dgate),
                      ("o", g.do)):
        flat = base[name].reshape(-1)
        num = torch.zeros_like(flat)
        for i in range(0, flat.numel(), 1 if flat.numel() < 30 else 5):
            for sgn in (1, -1):
                v = flat.clone()
                v[i] += sgn * step
                num[i] += sgn * loss({name: v.view(base[name].shape)}) / (2 * step)
        idx = torch.arange(0, flat.numel(), 1 if flat.numel() < 30 else 5)
        a, b = got.cpu().double().reshape(-1)[idx], num[idx]
        # differences: 1e-8 relative to the loss's terms; bf16 do: 2^-9
        assert float((a - b).norm() / b.norm()) < (4e-3 if name == "o" else 1e-5), name


def test_zero_rows_and_rows_of_zeros(qn):
    t = _dev(_inputs(4, 96, False, False, "norm", "channel", seed=1))
    t["o"][1] = 0
    t["h"][2] = 0
    t["o"][2] = 0
    hn, y, x8 = qn.block_norm_fwd(t["h"], t["w_pre"], o=t["o"], w_post=t["w_post"],
                                  gate=t["gate"], pack=True)
    assert torch.equal(hn[1], t["h"][1])
    assert not y[2].any() and not x8.codes[2].any() and (x8.exps[2] == 1).all()
    g = qn.block_norm_bwd(t["dy"], hn, t["w_pre"], o=t["o"], w_post=t["w_post"], gate=t["gate"])
    assert all(torch.isfinite(v).all() for v in g)
    # no rows: empty outputs, zero sums
    e = lambda v: v[:0]  # noqa: E731
    hn, y, x8 = qn.block_norm_fwd(e(t["h"]), t["w_pre"], o=e(t["o"]), w_post=t["w_post"],
                                  gate=t["gate"], pack=True)
    assert y.shape == (0, 96) and x8.codes.shape == (0, 96)
    g = qn.block_norm_bwd(e(t["dy"]), hn, t["w_pre"], o=e(t["o"]), w_post=t["w_post"],
                          gate=t["gate"])
    assert not g.dw_pre.any() and not g.dw_post.any() and not g.dgate.any()


def test_nan_and_inf_stay_in_their_row(qn):
    t = _dev(_inputs(5, 200, False, True, "norm", "channel", seed=2))
    t["o"][1, 3] = float("nan")
    t["h"][3, 7] = float("inf")
    _, y, x8 = qn.block_norm_fwd(t["h"], t["w_pre"], o=t["o"], w_post=t["w_post"],
                                 gate=t["gate"], pack=True)
    back = qn.act8_unpack(x8)
    assert torch.isnan(y[1]).all() and torch.isnan(y[3, 7])
    assert torch.isfinite(y[[0, 2, 4]]).all() and torch.isfinite(back[[0, 2, 4]]).all()
    assert torch.isnan(back[1]).all() and torch.isnan(back[3, :64]).all()


def test_squares_past_fp32(qn):
    """A row whose squares overflow has norm zero in fp32, and harms no other."""
    t = _dev(_inputs(3, 200, True, True, "norm", "channel", seed=9))
    t["o"][1] = 1e30
    t["h"][2] = 1e30
    hn, y, _ = qn.block_norm_fwd(t["h"], t["w_pre"], o=t["o"], w_post=t["w_post"],
                                 gate=t["gate"])
    assert torch.equal(hn[1], t["h"][1]) and not y[2].any()
    assert torch.isfinite(y).all()


def test_leading_dimensions_and_another_stream(qn):
    t = _dev(_inputs(12, 256, False, True, "norm", "row", seed=4))
    v = {k: x.view(3, 4, -1) for k, x in t.items() if x is not None and x.dim() == 2}
    ref = qn.block_norm_fwd(t["h"], t["w_pre"], o=t["o"], w_post=t["w_post"], gate=t["gate"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = qn.block_norm_fwd(v["h"], t["w_pre"], o=v["o"], w_post=t["w_post"], gate=v["gate"])
        g = qn.block_norm_bwd(v["dy"], got[0], t["w_pre"], dh_new=v["dh_new"], o=v["o"],
                              w_post=t["w_post"], gate=v["gate"])
    side.synchronize()
    assert torch.equal(got[0].view(12, 256), ref[0]) and torch.equal(got[1].view(12, 256), ref[1])
    r = qn.block_norm_bwd(t["dy"], ref[0], t["w_pre"], dh_new=t["dh_new"], o=t["o"],
                          w_post=t["w_post"], gate=t["gate"])
    torch.cuda.synchronize()
    assert g.dgate.shape == (3, 4, 1)
    assert torch.equal(g.dgate.view(12, 1), r.dgate) and torch.equal(g.dw_post, r.dw_post)


def test_graph_replays(qn):
    t = _dev(_inputs(64, 1024, False, True, "norm", "channel", seed=6))

    def step():
        hn, y, x8 = qn.block_norm_fwd(t["h"], t["w_pre"], o=t["o"], w_post=t["w_post"],
                                      gate=t["gate"], pack=True)
        g = qn.block_norm_bwd(t["dy"], hn, t["w_pre"], dh_new=t["dh_new"], o=t["o"],
                              w_post=t["w_post"], gate=t["gate"])
        return [hn, y, x8.codes, x8.exps, *g]

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
        for a, b in zip(outs, eager):
            assert torch.equal(a, b), k


def test_autograd(qn):
    norm = qn.BlockNorm(128, post=True, gate=True, scale=0.5)
    t = _inputs(6, 128, True, True, "norm", "channel", seed=8)
    h = t["h"].cuda().requires_grad_(True)
    o = t["o"].cuda().requires_grad_(True)
    hn, y, x8 = norm(h, o, pack=True)
    assert torch.equal(qn.act8_pack(y.detach()).codes, x8.codes)
    torch.autograd.backward([hn, y], [t["dh_new"].cuda(), t["dy"].cuda()])
    g = qn.block_norm_bwd(t["dy"].cuda(), hn.detach(), norm.w_pre.detach(),
                          dh_new=t["dh_new"].cuda(), o=o.detach(), w_post=norm.w_post.detach(),
                          gate=norm.gate.detach(), scale=0.5)
    for a, b in ((h.grad, g.dh), (o.grad, g.do), (norm.w_pre.grad, g.dw_pre),
                 (norm.w_post.grad, g.dw_post), (norm.gate.grad, g.dgate)):
        assert torch.equal(a, b)
    # the first norm of a model, and a gradient through h' alone
    h2 = t["h"].cuda().requires_grad_(True)
    same, y, none = norm(h2)
    assert same is h2 and none is None
    y.sum().backward()
    assert h2.grad is not None and h2.grad.abs().sum() > 0
    h3 = t["h"].cuda().requires_grad_(True)
    norm(h3, o.detach())[0].sum().backward()
    assert torch.allclose(h3.grad, torch.ones_like(h3))


def test_rows_past_32_bit_offsets(qn):
    """More than 2^31 values: the last rows are those of a small call."""
    M, D, k = 1 << 19, 4160, 8
    t = _dev(_inputs(k, D, False, True, "norm", "channel", seed=21))
    say(f"[norm far rows] M={M} D={D}")
    big = {n: torch.zeros(M, D, dtype=torch.bfloat16, device="cuda")
           for n in ("h", "o", "dy", "dh_new")}
    for n, v in big.items():
        v[-k:] = t[n]
    args = dict(w_post=t["w_post"], gate=t["gate"], scale=0.5)
    hn, y, x8 = qn.block_norm_fwd(big["h"], t["w_pre"], o=big["o"], pack=True, **args)
    rh, ry, r8 = qn.block_norm_fwd(t["h"], t["w_pre"], o=t["o"], pack=True, **args)
    assert torch.equal(hn[-k:], rh) and torch.equal(y[-k:], ry)
    assert torch.equal(x8.codes[-k:], r8.codes) and torch.equal(x8.exps[-k:], r8.exps)
    del y
    g = qn.block_norm_bwd(big["dy"], hn, t["w_pre"], dh_new=big["dh_new"], o=big["o"], **args)
    r = qn.block_norm_bwd(t["dy"], rh, t["w_pre"], dh_new=t["dh_new"], o=t["o"], **args)
    assert torch.equal(g.dh[-k:], r.dh) and torch.equal(g.do[-k:], r.do)
    # the zero rows add nothing to the sums, in whatever order
    for a, b in ((g.dw_pre, r.dw_pre), (g.dw_post, r.dw_post), (g.dgate, r.dgate)):
        assert torch.allclose(a, b, rtol=1e-5, atol=1e-5 * float(b.abs().max()))
    # and a checkpoint of as many values, read back
    back = qn.act8_unpack(qn.act8_pack(hn))
    assert torch.equal(back[-k:], qn.act8_unpack(qn.act8_pack(rh)))
