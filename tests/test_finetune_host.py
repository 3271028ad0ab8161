"""Refusals of the calls around the linear: the C ABI's host-side checks (no
GPU: every address is a number that is never dereferenced) and the binding's."""
import ctypes
import math

import pytest
import torch

FAKE = 1 << 20
OFF = FAKE + 4


@pytest.fixture(scope="module")
def qn():
    import quantized_fine_tuning_nf4_amd as qn
    qn.load_library()
    return qn


def test_act8_refusals(qn):
    L = qn.load_library()
    p, u = L.act8_pack, L.act8_unpack
    for M, K in [(-1, 64), (4, 0), (4, (1 << 20) + 1), ((1 << 23) + 1, 64)]:
        assert p(FAKE, M, K, FAKE, FAKE, None) == qn.QN_EINVAL
    assert p(None, 4, 64, FAKE, FAKE, None) == qn.QN_EINVAL
    assert p(FAKE, 4, 64, FAKE, None, None) == qn.QN_EINVAL
    assert p(FAKE, 4, 64, OFF, FAKE, None) == qn.QN_EALIGN
    assert p(None, 0, 64, None, None, None) == qn.QN_OK
    a = qn._Act8(FAKE, FAKE)
    assert u(ctypes.byref(a), 4, 64, None, None) == qn.QN_EINVAL
    assert u(None, 4, 64, FAKE, None) == qn.QN_EINVAL
    assert u(ctypes.byref(qn._Act8(FAKE, None)), 4, 64, FAKE, None) == qn.QN_EINVAL
    assert u(ctypes.byref(qn._Act8(OFF, FAKE)), 4, 64, FAKE, None) == qn.QN_EALIGN
    assert u(ctypes.byref(a), 0, 64, FAKE, None) == qn.QN_OK


def test_linear_bwd_act8_refusals(qn):
    L = qn.load_library()
    st = qn._NF4DQ(FAKE, FAKE, FAKE, FAKE, 8, 64)
    a = qn._Act8(FAKE, FAKE)

    def call(st=st, a=a, dY=FAKE, M=2, A=FAKE, B=FAKE, r=4, opts=None, u=FAKE, dX=FAKE, dA=FAKE,
             dB=FAKE, ws=FAKE, n=1 << 30):
        return L.qlora_linear_bwd_act8(ctypes.byref(st), None if a is None else ctypes.byref(a),
                                       dY, M, A, B, r, 8.0, opts, u, dX, dA, dB, ws, n, None)

    for kw in [dict(a=None), dict(a=qn._Act8(None, FAKE)), dict(a=qn._Act8(FAKE, None)),
               dict(u=None), dict(dY=None), dict(A=None), dict(B=None), dict(dA=None),
               dict(dB=None), dict(ws=None), dict(r=0), dict(r=65), dict(M=-1),
               dict(st=qn._NF4DQ(FAKE, FAKE, FAKE, FAKE, 8, 72)),
               dict(st=qn._NF4DQ(FAKE, FAKE, FAKE, FAKE, 12, 64)),
               dict(opts=ctypes.byref(qn._LoraOpts(0, FAKE, 1.0))),
               dict(opts=ctypes.byref(qn._LoraOpts(2, None, 0.0)))]:
        assert call(**kw) == qn.QN_EINVAL, kw
    for kw in [dict(a=qn._Act8(OFF, FAKE)), dict(a=qn._Act8(FAKE, OFF)), dict(u=OFF),
               dict(dY=OFF), dict(dX=OFF), dict(dA=OFF), dict(ws=FAKE + 16),
               dict(opts=ctypes.byref(qn._LoraOpts(0, FAKE + 8, 0.5)))]:
        assert call(**kw) == qn.QN_EALIGN, kw
    need = L.qlora_linear_bwd_act8_workspace(2, 8, 64, 4, 1)
    assert need > 0 and call(n=need - 1) == qn.QN_EWORKSPACE
    assert L.qlora_linear_bwd_act8_workspace(2, 8, 64, 65, 1) == 0
    assert L.qlora_linear_bwd_act8_workspace(0, 8, 64, 4, 1) >= 0


def _norm(qn, **kw):
    n = qn._BlockNorm(4, 64, FAKE, FAKE, FAKE, qn.QN_BF16, qn.QN_F32, 1, 0.5, 1e-6)
    for k, v in kw.items():
        setattr(n, k, v)
    return ctypes.byref(n)


BAD_NORMS = [dict(M=-1), dict(D=0), dict(D=16385), dict(w_pre=None), dict(res_dtype=2),
             dict(w_dtype=-1), dict(gate_kind=4), dict(gate_kind=0), dict(gate=None),
             dict(eps=0.0), dict(eps=1e-40), dict(eps=-1.0), dict(eps=math.nan), dict(scale=math.inf)]


def test_block_norm_refusals(qn):
    L = qn.load_library()

    def fwd(n, h=FAKE, o=FAKE, hn=FAKE, y=FAKE, codes=FAKE, exps=FAKE):
        return L.block_norm_fwd(n, h, o, hn, y, codes, exps, None)

    def bwd(n, dy=FAKE, dhn=FAKE, hn=FAKE, o=FAKE, dh=FAKE, do=FAKE, dg=FAKE, dw1=FAKE, dw2=FAKE,
            ws=FAKE, size=1 << 30):
        return L.block_norm_bwd(n, dy, dhn, hn, o, dh, do, dg, dw1, dw2, ws, size, None)

    for kw in BAD_NORMS:
        assert fwd(_norm(qn, **kw)) == qn.QN_EINVAL, kw
        assert bwd(_norm(qn, **kw)) == qn.QN_EINVAL, kw
    assert fwd(None) == qn.QN_EINVAL and bwd(None) == qn.QN_EINVAL
    for kw in [dict(h=None), dict(y=None), dict(hn=None), dict(codes=None), dict(exps=None),
               dict(o=None)]:
        assert fwd(_norm(qn), **kw) == qn.QN_EINVAL, kw
    for kw in [dict(h=OFF), dict(o=OFF), dict(hn=OFF), dict(y=OFF), dict(codes=OFF),
               dict(exps=OFF)]:
        assert fwd(_norm(qn), **kw) == qn.QN_EALIGN, kw
    assert fwd(_norm(qn, w_pre=OFF)) == qn.QN_EALIGN
    assert fwd(_norm(qn, gate=OFF)) == qn.QN_EALIGN
    for kw in [dict(dy=None), dict(hn=None), dict(dh=None), dict(do=None), dict(o=None),
               dict(ws=None)]:
        assert bwd(_norm(qn), **kw) == qn.QN_EINVAL, kw
    # gradients of what is not there
    assert bwd(_norm(qn, w_post=None)) == qn.QN_EINVAL
    assert bwd(_norm(qn, gate=None, gate_kind=0)) == qn.QN_EINVAL
    for kw in [dict(dy=OFF), dict(dhn=OFF), dict(hn=OFF), dict(o=OFF), dict(dh=OFF), dict(do=OFF),
               dict(dg=OFF), dict(dw1=OFF), dict(dw2=OFF), dict(ws=FAKE + 16)]:
        assert bwd(_norm(qn), **kw) == qn.QN_EALIGN, kw
    need = L.block_norm_bwd_workspace(_norm(qn), 1, 1)
    assert need > 0 and bwd(_norm(qn), size=need - 1) == qn.QN_EWORKSPACE
    assert L.block_norm_bwd_workspace(_norm(qn, gate_kind=2), 0, 1) == 0
    assert fwd(_norm(qn, M=0), h=None, o=FAKE, hn=None, y=None) == qn.QN_OK


def test_token_logprobs_refusals(qn):
    L = qn.load_library()

    def fwd(x=FAKE, dt=0, T=4, V=100, ld=100, t=FAKE, scale=1.0, k=5, lp=FAKE, ent=FAKE, st=FAKE,
            tl=FAKE, ti=FAKE, ws=FAKE, n=1 << 30):
        return L.token_logprobs_fwd(x, dt, T, V, ld, t, scale, k, lp, ent, st, tl, ti, ws, n, None)

    def bwd(x=FAKE, dt=0, T=4, V=100, ld=100, t=FAKE, scale=1.0, st=FAKE, ent=FAKE, dl=FAKE,
            de=FAKE, dx=FAKE + (1 << 20), ldd=100):
        return L.token_logprobs_bwd(x, dt, T, V, ld, t, scale, st, ent, dl, de, dx, ldd, None)

    for kw in [dict(x=None), dict(dt=2), dict(T=-1), dict(T=(1 << 23) + 1), dict(V=0), dict(ld=99),
               dict(V=(1 << 28) + 1, ld=1 << 29), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=math.nan), dict(scale=math.inf)]:
        assert fwd(**kw) == qn.QN_EINVAL, kw
        assert bwd(**kw) == qn.QN_EINVAL, kw
    for kw in [dict(k=-1), dict(k=33), dict(V=4, ld=4), dict(t=None), dict(lp=None),
               dict(ent=None), dict(st=None), dict(tl=None), dict(ti=None)]:
        assert fwd(**kw) == qn.QN_EINVAL, kw
    for kw in [dict(x=FAKE + 2), dict(t=OFF), dict(lp=OFF), dict(ent=OFF), dict(st=OFF),
               dict(tl=OFF), dict(ti=OFF)]:
        assert fwd(**kw) == qn.QN_EALIGN, kw
    assert fwd(x=FAKE + 1, dt=1) == qn.QN_EALIGN
    for kw in [dict(st=None), dict(dx=None), dict(dl=None, de=None), dict(t=None),
               dict(ent=None), dict(ldd=99), dict(dx=FAKE, ldd=101)]:
        assert bwd(**kw) == qn.QN_EINVAL, kw
    for kw in [dict(x=FAKE + 2), dict(dx=FAKE + 2), dict(st=OFF), dict(dl=OFF)]:
        assert bwd(**kw) == qn.QN_EALIGN, kw
    need = L.token_logprobs_workspace(4, 100000, 0, 5)
    if need:
        assert fwd(V=100000, ld=100000, n=need - 1) == qn.QN_EWORKSPACE
        assert fwd(V=100000, ld=100000, ws=None) == qn.QN_EINVAL
    assert fwd(x=None, T=0) == qn.QN_OK and bwd(x=None, T=0) == qn.QN_OK


def test_binding_refuses_what_the_kernels_do_not_take(qn):
    z = torch.zeros
    with pytest.raises(ValueError):
        qn.act8_pack(z(4, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        qn.act8_unpack(z(4, 64))
    with pytest.raises(ValueError):
        qn.block_norm_fwd(z(4, 64, dtype=torch.float16), z(64))
    with pytest.raises(ValueError):
        qn.block_norm_fwd(z(4, 64), z(64))
    with pytest.raises(ValueError):
        qn.token_logprobs_fwd(z(4, 64))


def test_linear_bwd_act8_workspace_holds_a_weight_copy_for_dx_only(qn):
    L = qn.load_library()
    for M, rows, cols, r in [(1, 8, 64, 1), (300, 1000, 576, 17), (4096, 1024, 4096, 64)]:
        without, with_dx = (L.qlora_linear_bwd_act8_workspace(M, rows, cols, r, d) for d in (0, 1))
        assert with_dx - without >= 2 * rows * cols
        st = qn._NF4DQ(FAKE, FAKE, FAKE, FAKE, rows, cols)
        assert L.qlora_linear_bwd_act8(
            ctypes.byref(st), ctypes.byref(qn._Act8(FAKE, FAKE)), FAKE, M, FAKE, FAKE, r, 8.0, None,
            FAKE, FAKE, FAKE, FAKE, FAKE, without, None) == qn.QN_EWORKSPACE
