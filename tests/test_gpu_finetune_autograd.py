"""What autograd has to know of the calls around the linear: tensors written in place,
checkpoints that do not belong to the input, derivatives that are not there."""
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


def rnd(*shape, dtype=BF):
    return torch.randn(*shape, device="cuda").to(dtype)


def test_a_checkpoint_packed_again_before_the_backward(qn):
    lin = qn.QLoRALinear(rnd(64, 128, dtype=F32), r=4, act8=True)
    x, buf = rnd(5, 128).requires_grad_(True), qn.act8_pack(rnd(5, 128))
    y = lin(x, x8=qn.act8_pack(x.detach(), out=buf))
    qn.act8_pack(rnd(5, 128), out=buf)
    with pytest.raises(RuntimeError, match="inplace"):
        y.sum().backward()


def test_outputs_written_in_place_count_as_modified(qn):
    x8 = qn.act8_pack(rnd(4, 128))
    out = rnd(4, 128)
    before = out._version, x8.codes._version, x8.exps._version
    qn.act8_unpack(x8, out=out)
    qn.act8_pack(out, out=x8)
    assert out._version > before[0]
    assert x8.codes._version > before[1] and x8.exps._version > before[2]
    logits = rnd(3, 50, dtype=F32).requires_grad_(True)
    h = logits * 1.0
    t = torch.zeros(3, dtype=torch.int64, device="cuda")
    r = qn.token_logprobs(h, t)
    qn.token_logprobs_bwd(h.detach(), t, r.stats, r.entropy.detach(),
                          torch.ones(3, device="cuda"), out=h.detach())
    with pytest.raises(RuntimeError, match="inplace"):
        r.logp.sum().backward()
    with torch.inference_mode():  # (such tensors count nothing)
        z = rnd(4, 128)
        qn.act8_unpack(qn.act8_pack(z, out=qn.act8_pack(z)), out=z)


def test_a_checkpoint_of_another_shape_is_refused_in_the_forward(qn):
    lin = qn.QLoRALinear(rnd(64, 128, dtype=F32), r=4, act8=True)
    x = rnd(2, 3, 128)
    good = qn.act8_pack(x)
    assert lin(x, x8=good).shape == (2, 3, 64)
    for bad in (qn.act8_pack(rnd(5, 128)), qn.act8_pack(rnd(6, 64)), qn.act8_pack(rnd(3, 256)),
                qn.Act8(good.codes, good.exps[:, :1].contiguous()),
                qn.Act8(good.codes.float(), good.exps), qn.Act8(good.codes.cpu(), good.exps),
                (good.codes, good.exps)):
        with pytest.raises(ValueError):
            lin(x, x8=bad)


@pytest.mark.parametrize("what", ["linear", "linear_act8", "norm", "norm_alone", "logprobs"])
def test_second_derivatives_are_refused(qn, what):
    """First derivatives under create_graph are right; asking for more of them raises
    (it gave the part that does not go through the call, and no word)."""
    if what.startswith("linear"):
        x = rnd(5, 128).requires_grad_(True)
        lin = qn.QLoRALinear(rnd(64, 128, dtype=F32), r=4, act8=what == "linear_act8")
        f = lambda v: lin(v).float()  # noqa: E731
    elif what.startswith("norm"):
        x, o = rnd(5, 128, dtype=F32).requires_grad_(True), rnd(5, 128)
        norm = qn.BlockNorm(128, post=True, gate=True)
        f = lambda v: norm(v, o if what == "norm" else None)[1].float()  # noqa: E731
    else:
        x = rnd(5, 40, dtype=F32).requires_grad_(True)
        t = torch.arange(5, device="cuda")
        f = lambda v: qn.token_logprobs(v, t).logp  # noqa: E731
    ref, = torch.autograd.grad((f(x) ** 2).sum(), x)
    y = f(x)
    g, = torch.autograd.grad((y ** 2).sum(), x, create_graph=True)
    assert torch.equal(g, ref)
    with pytest.raises(RuntimeError, match="differentiate twice"):
        (g.float().pow(2).sum() + x.float().pow(2).sum()).backward()


@pytest.mark.parametrize("with_o", [False, True])
def test_only_the_residual_stream_has_a_gradient(qn, with_o):
    """y unused and nothing of the block wants a gradient: h's is h''s, also where h'
    is no number (a backward from dy = 0 made those rows NaN)."""
    norm = qn.BlockNorm(96, post=with_o).requires_grad_(False)
    h, o, g = rnd(5, 96, dtype=F32), rnd(5, 96), rnd(5, 96, dtype=F32)
    h[2, 7], h[3, 0] = float("inf"), float("nan")
    h.requires_grad_(True)
    hn, y, _ = norm(h, o if with_o else None)
    hn.backward(g)
    assert torch.equal(h.grad, g)
    h.grad = None
    hn, y, _ = norm(h, o if with_o else None)
    y.float().sum().backward()
    assert torch.isnan(h.grad[2:4]).any(1).all() and torch.isfinite(h.grad[[0, 1, 4]]).all()
