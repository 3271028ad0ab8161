"""MXFP4 and counter-based dropout without a GPU: the plain forms the GPU tests
compare with, and what the C calls and the binding refuse."""
import ctypes

import numpy as np
import pytest
import torch

from tests import _mx4

FAKE = 1 << 20  # a non-null, 256-aligned address that is never dereferenced


@pytest.fixture(scope="module")
def qn():
    import quantized_fine_tuning_nf4_amd as qn
    qn.load_library()
    return qn


def test_philox_against_the_published_vectors():
    # the known answers published with the generator
    f, z = 0xffffffff, 0
    for ctr, key, want in [
            ((z, z, z, z), (z, z), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
            ((f, f, f, f), (f, f), (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
            ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
             (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))]:
        assert [int(v) for v in _mx4.philox(ctr, key)] == list(want)


def test_plain_levels():
    x = np.zeros((1, 32))
    x[0, :12] = [4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, 7.9, -0.3, 4.99]
    got = _mx4.rounded(x)[0, :12]
    assert np.array_equal(got, [4, 0, 1, 1, 2, 2, 4, 4, -0.0, 6, -0.5, 4])
    for v in (1.0, 1.999, 2.0 ** -127, 2.0 ** 127, 6.0, 8.0):
        x = np.zeros((1, 32))
        x[0, 3] = v
        assert abs(_mx4.rounded(x)[0, 3] - v) <= 0.25 * v
    x[0, 5] = np.nan
    assert np.isnan(_mx4.rounded(x)).all()


def _mx(rows, cols, codes=FAKE, scales=FAKE):
    from quantized_fine_tuning_nf4_amd import _MX4
    return ctypes.byref(_MX4(codes, scales, rows, cols))


def _do(p=0.1, seed=1, offset=0, step=None):
    from quantized_fine_tuning_nf4_amd import _Dropout
    return ctypes.byref(_Dropout(seed, offset, step, p))


def test_quantize_refusals(qn):
    L = qn.load_library()
    q = lambda x=FAKE, t=0, rows=4, cols=64, c=FAKE, s=FAKE: L.mx4_quantize(  # noqa: E731
        x, t, rows, cols, c, s, None)
    for bad in (dict(t=2), dict(t=-1), dict(rows=-1), dict(cols=0), dict(cols=(1 << 20) + 1),
                dict(rows=(1 << 23) + 1), dict(x=None), dict(c=None), dict(s=None)):
        assert q(**bad) == qn.QN_EINVAL, bad
    for bad in (dict(x=FAKE + 4), dict(x=FAKE + 2, t=1), dict(c=FAKE + 4), dict(s=FAKE + 8),
                dict(x=FAKE + 2, cols=63), dict(x=FAKE + 1, t=1, cols=63)):
        assert q(**bad) == qn.QN_EALIGN, bad
    assert q(x=None, rows=0) == qn.QN_OK
    d = L.mx4_dequantize
    assert d(_mx(4, 64), 2, FAKE, None) == qn.QN_EINVAL
    assert d(None, 0, FAKE, None) == qn.QN_EINVAL
    assert d(_mx(4, 0), 0, FAKE, None) == qn.QN_EINVAL
    assert d(_mx(4, 64), 0, None, None) == qn.QN_EINVAL
    assert d(_mx(4, 64, codes=FAKE + 4), 0, FAKE, None) == qn.QN_EALIGN
    assert d(_mx(4, 64), 0, FAKE + 4, None) == qn.QN_EALIGN
    assert d(_mx(0, 64), 0, None, None) == qn.QN_OK


def test_sizes_past_a_launch(qn):
    """More elements than one launch has threads for are refused, not cut off."""
    L = qn.load_library()
    assert L.dropout_apply(FAKE, 1, (1 << 35) + 1, _do(), FAKE, None) == qn.QN_EINVAL
    assert L.mx4_quantize(FAKE, 1, 1 << 18, 1 << 19, FAKE, FAKE, None) == qn.QN_EINVAL
    assert L.mx4_dequantize(_mx(1 << 18, 1 << 19), 1, FAKE, None) == qn.QN_EINVAL


def test_linear_refusals(qn):
    L = qn.load_library()

    def fwd(rows=64, cols=128, M=4, A=FAKE, B=FAKE, r=4, rslora=0, drop=None, x=FAKE, y=FAKE,
            u=FAKE, ws=FAKE, n=1 << 30, w=None):
        return L.mx4_linear_fwd(w or _mx(rows, cols), x, M, A, B, r, 8.0, rslora, drop, y, u, ws, n,
                                None)

    def bwd(rows=64, cols=128, M=4, x=FAKE, x8=None, dY=FAKE, A=FAKE, B=FAKE, r=4, drop=None,
            u=FAKE, dX=FAKE, dA=FAKE, dB=FAKE, ws=FAKE, n=1 << 30, rslora=0):
        return L.mx4_linear_bwd(_mx(rows, cols), x, x8, dY, M, A, B, r, 8.0, rslora, drop, u, dX, dA,
                                dB, ws, n, None)

    for bad in (dict(rows=63), dict(cols=127), dict(r=65), dict(r=-1), dict(M=-1),
                dict(M=(1 << 23) + 1), dict(rows=(1 << 20) + 8), dict(cols=(1 << 20) + 64),
                dict(A=None), dict(B=None), dict(ws=None), dict(rslora=2), dict(drop=_do(p=1.0)),
                dict(drop=_do(p=-0.1)), dict(drop=_do(p=float("nan")))):
        assert fwd(**bad) == qn.QN_EINVAL, bad
        assert bwd(**bad) == qn.QN_EINVAL, bad
    for bad in (dict(x=FAKE + 2), dict(A=FAKE + 2), dict(B=FAKE + 2), dict(ws=FAKE + 128),
                dict(u=FAKE + 4), dict(drop=_do(step=FAKE + 4))):
        assert fwd(**bad) == qn.QN_EALIGN, bad
        assert bwd(**bad) == qn.QN_EALIGN, bad
    assert fwd(n=100) == qn.QN_EWORKSPACE
    assert bwd(n=100) == qn.QN_EWORKSPACE
    assert fwd(x=None) == fwd(y=None) == qn.QN_EINVAL
    assert fwd(r=0) == qn.QN_EINVAL  # a u without an adapter
    assert fwd(w=_mx(64, 128, scales=None)) == qn.QN_EINVAL
    assert fwd(w=_mx(64, 128, codes=FAKE + 8)) == qn.QN_EALIGN
    assert bwd(x=None) == qn.QN_EINVAL
    assert bwd(x8=ctypes.byref(qn._Act8(FAKE, FAKE))) == qn.QN_EINVAL  # both
    assert bwd(x=None, x8=ctypes.byref(qn._Act8(FAKE, FAKE)), u=None) == qn.QN_EINVAL
    assert bwd(dY=None) == bwd(dA=None) == bwd(dB=None) == qn.QN_EINVAL
    assert bwd(r=0, dX=None) == qn.QN_EINVAL
    assert fwd(M=0, x=None, y=None, ws=None) == qn.QN_OK
    assert L.mx4_linear_workspace(-1, 64, 128, 4, 0, 0, 0) == 0
    assert L.mx4_linear_workspace(4, 64, 128, 65, 0, 0, 0) == 0
    # with a mask's bits beside the rest
    assert (L.mx4_linear_workspace(512, 64, 128, 4, 1, 0, 1)
            >= L.mx4_linear_workspace(512, 64, 128, 4, 1, 0, 0) + 512 * 128 // 8)


def test_dropout_refusals(qn):
    L = qn.load_library()
    f = lambda x=FAKE, t=0, n=8, d=None, out=FAKE: L.dropout_apply(  # noqa: E731
        x, t, n, d or _do(), out, None)
    for bad in (dict(t=2), dict(n=-1), dict(n=(1 << 40) + 1), dict(x=None), dict(out=None),
                dict(d=_do(p=1.0)), dict(d=_do(p=-1.0))):
        assert f(**bad) == qn.QN_EINVAL, bad
    assert L.dropout_apply(FAKE, 0, 8, None, FAKE, None) == qn.QN_EINVAL
    for bad in (dict(x=FAKE + 2), dict(x=FAKE + 1, t=1), dict(out=FAKE + 1, t=1),
                dict(d=_do(step=FAKE + 2))):
        assert f(**bad) == qn.QN_EALIGN, bad
    assert f(n=0, x=None, out=None) == qn.QN_OK
    s = qn._NF4DQ(FAKE, FAKE, FAKE, FAKE, 64, 128)
    args = (ctypes.byref(s), FAKE, 4, FAKE, FAKE, 4, 8.0)
    tail = (FAKE, FAKE, FAKE, 1 << 30, None)
    assert L.qlora_linear_fwd_drop(*args, 2, None, *tail) == qn.QN_EINVAL
    assert L.qlora_linear_fwd_drop(*args, 0, _do(p=1.0), *tail) == qn.QN_EINVAL
    assert L.qlora_linear_fwd_drop(*args, 0, _do(), FAKE, FAKE, FAKE, 100, None) == qn.QN_EWORKSPACE
    b = lambda x, x8, d, n=1 << 30, u=FAKE: L.qlora_linear_bwd_drop(  # noqa: E731
        ctypes.byref(s), x, x8, FAKE, 4, FAKE, FAKE, 4, 8.0, 0, d, u, FAKE, FAKE, FAKE, FAKE, n, None)
    assert b(None, None, _do()) == qn.QN_EINVAL
    assert b(FAKE, ctypes.byref(qn._Act8(FAKE, FAKE)), _do()) == qn.QN_EINVAL
    assert b(FAKE, None, _do(p=2.0)) == qn.QN_EINVAL
    assert b(FAKE, None, _do(), n=100) == qn.QN_EWORKSPACE


def test_binding_refuses(qn):
    for p in (-0.1, 1.0, float("nan")):
        with pytest.raises(ValueError):
            qn.Dropout(p, 1)
    for kw in (dict(seed=-1), dict(seed=1 << 64), dict(seed=1, offset=-1), dict(seed=1.5)):
        with pytest.raises(ValueError):
            qn.Dropout(0.1, **kw)
    with pytest.raises(ValueError):
        qn.Dropout(0.1, 1, step=torch.zeros(1, dtype=torch.int64))  # not on the device
    with pytest.raises(ValueError):
        qn.mx4_quantize(torch.zeros(4, 64))
    with pytest.raises(ValueError):
        qn.dropout_apply(torch.zeros(4), qn.Dropout(0.1, 1))
    with pytest.raises(ValueError):
        qn.QLoRALinear(torch.zeros(8, 64), base="int4")
    with pytest.raises(ValueError):
        qn.QLoRALinear(torch.zeros(8, 64), base="mx4", dropout=0.1)
