"""What the binding of the calls around the linear refuses, on device tensors:
types, shapes, orders and counts that the kernels do not take."""
import pytest
import torch

from tests._gpu import needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def qn():
    import quantized_fine_tuning_nf4_amd as qn
    qn.load_library()
    return qn


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def test_act8(qn):
    ok = qn.act8_pack(z(4, 128))
    for bad in (z(4, 128, dtype=F32), z(128, 4).t(), z(4, 128)[:, ::2], z(4, 0), None):
        with pytest.raises(ValueError):
            qn.act8_pack(bad)
    for out in (qn.Act8(ok.codes[:2], ok.exps), qn.Act8(ok.codes, ok.exps[:, :1]),
                qn.Act8(ok.codes.to(torch.uint8), ok.exps), ok.codes):
        with pytest.raises(ValueError):
            qn.act8_pack(z(4, 128), out=out)
    for x8, out in ((qn.Act8(ok.codes, ok.exps.int()), None), (ok, z(4, 127)),
                    (ok, z(4, 128, dtype=F32)), (qn.Act8(ok.codes.view(-1), ok.exps), None)):
        with pytest.raises(ValueError):
            qn.act8_unpack(x8, out=out)


def test_linear_backward_from_the_checkpoint(qn):
    st = qn.nf4_quantize_dq(torch.randn(64, 128, device="cuda"))
    good = dict(x8=qn.act8_pack(z(4, 128)), dY=z(4, 64), A=z(8, 128), B=z(64, 8), alpha=16.0,
                u=z(4, 8, dtype=F32))
    qn.qlora_linear_bwd_act8(st, **good)
    for kw in (dict(x8=z(4, 128)), dict(x8=qn.act8_pack(z(5, 128))), dict(dY=z(4, 65)),
               dict(dY=z(64, 4).t()), dict(A=z(8, 64)), dict(B=z(64, 9)), dict(u=z(4, 8)),
               dict(u=z(3, 8, dtype=F32)), dict(u=None),
               dict(dropout_mask=torch.zeros(8, dtype=torch.uint8, device="cuda"), dropout_p=0.5)):
        with pytest.raises(ValueError):
            qn.qlora_linear_bwd_act8(st, **{**good, **kw})
    with pytest.raises(qn.QNError):  # rank
        qn.qlora_linear_bwd_act8(st, good["x8"], good["dY"], z(65, 128), z(64, 65), 16.0,
                                 z(4, 65, dtype=F32))
    with pytest.raises(qn.QNError):  # a probability without a mask
        qn.qlora_linear_bwd_act8(st, **good, dropout_p=0.5)


def test_block_norm(qn):
    good = dict(h=z(4, 64), w_pre=z(64), o=z(4, 64), w_post=z(64), gate=z(64))
    qn.block_norm_fwd(**good)
    for kw in (dict(h=z(4, 64, dtype=torch.float16)), dict(h=z(64, 4).t()), dict(h=z(4, 0)),
               dict(w_pre=z(63)), dict(w_pre=z(64, dtype=torch.float16)), dict(o=z(4, 63)),
               dict(o=z(4, 64, dtype=F32)), dict(w_post=z(64, dtype=F32)), dict(w_post=z(4, 64)),
               dict(gate=z(4)), dict(gate=z(4, 1, dtype=F32)), dict(gate=z(64, dtype=F32)),
               dict(gate=1.0), dict(o=None)):
        with pytest.raises(ValueError):
            qn.block_norm_fwd(**{**good, **kw})
    for kw in (dict(eps=0.0), dict(eps=float("nan")), dict(scale=float("inf"))):
        with pytest.raises(qn.QNError):
            qn.block_norm_fwd(**good, **kw)
    with pytest.raises(qn.QNError):
        qn.block_norm_fwd(z(1, 16385), z(16385))
    back = dict(dy=z(4, 64), h_new=z(4, 64), w_pre=z(64), o=z(4, 64), w_post=z(64))
    qn.block_norm_bwd(**back)
    for kw in (dict(dy=z(4, 64, dtype=F32)), dict(dy=z(3, 64)), dict(dh_new=z(4, 64, dtype=F32)),
               dict(dh_new=z(64)), dict(h_new=z(4, 64, dtype=F32), dh_new=z(4, 64))):
        with pytest.raises(ValueError):
            qn.block_norm_bwd(**{**back, **kw})


def test_token_logprobs(qn):
    x, t = z(4, 100), torch.zeros(4, dtype=torch.int64, device="cuda")
    r = qn.token_logprobs_fwd(x, t)
    for a in ((z(4, 100, dtype=torch.float16), t), (z(100, 4).t(), t), (z(4, 200)[:, ::2], t),
              (z(400), t), (z(1, 100).expand(4, 100), t), (x, t.int()), (x, t[:3])):
        with pytest.raises(ValueError):
            qn.token_logprobs_fwd(*a)
    for kw in (dict(top_k=-1), dict(top_k=33)):
        with pytest.raises(ValueError):
            qn.token_logprobs_fwd(x, t, **kw)
    with pytest.raises(ValueError):
        qn.token_logprobs_fwd(z(2, 3), t[:2], top_k=4)
    for scale in (0.0, -1.0, float("nan")):
        with pytest.raises(qn.QNError):
            qn.token_logprobs_fwd(x, t, scale=scale)
    g = z(4, dtype=F32)
    for a in ((None, None), (g[:3], None), (g.double(), None)):
        with pytest.raises(ValueError):
            qn.token_logprobs_bwd(x, t, r.stats, r.entropy, *a)
    with pytest.raises(ValueError):
        qn.token_logprobs_bwd(x, None, r.stats, r.entropy, g)
    with pytest.raises(ValueError):
        qn.token_logprobs_bwd(x, t, r.stats, None, g, g)
    with pytest.raises(ValueError):
        qn.token_logprobs_bwd(x, t, r.stats[:3], r.entropy, g)
    for out in (z(4, 101), z(4, 100, dtype=F32), z(100, 4).t()):
        with pytest.raises(ValueError):
            qn.token_logprobs_bwd(x, t, r.stats, r.entropy, g, out=out)
