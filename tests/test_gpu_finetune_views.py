"""The calls around the linear on contiguous views that start anywhere in a larger
tensor (slices of rows, of a batch's tokens, of a flat buffer of parameters): the same
results, bit for bit, as on tensors of their own."""
import pytest
import torch

from tests._gpu import needs_gpu, say

pytestmark = [pytest.mark.gpu, needs_gpu]
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def qn():
    import quantized_fine_tuning_nf4_amd as qn
    qn.load_library()
    return qn


def view(t, at=1):
    """t's values in a contiguous view that starts `at` elements into its storage."""
    flat = torch.empty(t.numel() + at, dtype=t.dtype, device=t.device)
    v = flat[at:].view(t.shape)
    v.copy_(t)
    assert v.is_contiguous() and v.data_ptr() % 16 == (at * t.element_size()) % 16
    return v


def rnd(*shape, dtype=BF, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + sum(shape))
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def same(a, b):
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert (x is None) == (y is None)
        if x is not None:
            assert torch.equal(x, y)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,V", [(7, 1001), (3, 40000)])
def test_log_probabilities_of_shifted_tokens(qn, T, V, f32):
    """targets = ids[1:], and every other operand of a row a view as well."""
    say(f"[views logprobs] T={T} V={V} f32={f32}")
    ids = torch.arange(T + 1, device="cuda") * 37 % V
    x, t = rnd(T + 1, V, dtype=F32 if f32 else BF), ids[1:]
    got = qn.token_logprobs_fwd(x[1:], t, top_k=3)
    own = qn.token_logprobs_fwd(x[1:].clone(), t.clone(), top_k=3)
    same(got, own)
    g, h = rnd(T, dtype=F32, seed=1), rnd(T, dtype=F32, seed=2)
    ref = qn.token_logprobs_bwd(x[1:].clone(), t.clone(), own.stats, own.entropy, g, h)
    for at in (1, 2, 3, 5):
        dx = qn.token_logprobs_bwd(x[1:], t, view(own.stats, at), view(own.entropy, at),
                                   view(g, at), view(h, at))
        assert torch.equal(dx, ref)


@pytest.mark.parametrize("Ta", [1, 2, 3, 6])
def test_gradient_of_two_ragged_calls_joined(qn, Ta):
    """torch.cat hands its second operand a gradient that starts Ta floats in."""
    xs = [rnd(Ta, 501, dtype=F32).requires_grad_(True),
          rnd(5, 501, dtype=F32, seed=9).requires_grad_(True)]
    ts = [torch.arange(n, device="cuda") for n in (Ta, 5)]
    w = rnd(Ta + 5, dtype=F32, seed=3)
    r = [qn.token_logprobs(x, t) for x, t in zip(xs, ts)]
    ((torch.cat([r[0].logp, r[1].logp]) + torch.cat([r[0].entropy, r[1].entropy])) * w).sum().backward()
    for x, t, g in zip(xs, ts, (w[:Ta], w[Ta:])):
        s = qn.token_logprobs_fwd(x.detach(), t)
        ref = qn.token_logprobs_bwd(x.detach(), t, s.stats, s.entropy, g.clone(), g.clone())
        assert torch.equal(x.grad, ref)


@pytest.mark.parametrize("D", [5, 64, 1001, 1002, 4096, 4100, 8191, 9000])
@pytest.mark.parametrize("res", [BF, F32])
@pytest.mark.parametrize("gate", ["none", "channel", "row", "element"])
def test_block_norm(qn, D, res, gate):
    say(f"[views norm] D={D} res={res} gate={gate}")
    M = 5
    h, o, dy, dh = rnd(M, D, dtype=res), rnd(M, D, seed=1), rnd(M, D, seed=2), rnd(M, D, dtype=res, seed=3)
    w = [rnd(D, dtype=F32, seed=4), rnd(D, dtype=F32, seed=5)]
    gt = {"none": None, "channel": rnd(D, dtype=F32, seed=6), "row": rnd(M, 1, seed=6),
          "element": rnd(M, D, seed=6)}[gate]

    def run(f):
        v = lambda t: None if t is None else f(t)  # noqa: E731
        a, y, x8 = qn.block_norm_fwd(v(h), v(w[0]), o=v(o), w_post=v(w[1]), gate=v(gt), scale=0.5,
                                     pack=True)
        g = qn.block_norm_bwd(v(dy), v(a), v(w[0]), dh_new=v(dh), o=v(o), w_post=v(w[1]),
                              gate=v(gt), scale=0.5)
        _, y1, _ = qn.block_norm_fwd(v(h), v(w[0]))
        return [a, y, x8.codes, x8.exps, *g, y1]

    own = run(torch.clone)
    for at in (1, 3):
        same(run(lambda t: view(t, at)), own)
    # a slice of rows of an odd width
    same([qn.block_norm_fwd(h[1:], w[0])[1]], [qn.block_norm_fwd(h[1:].clone(), w[0])[1]])


@pytest.mark.parametrize("cols", [1, 63, 64, 320, 1000, 1001])
def test_checkpoints(qn, cols):
    say(f"[views act8] cols={cols}")
    x = rnd(9, cols)
    own = qn.act8_pack(x)
    for at in (1, 2, 5):
        got = qn.act8_pack(view(x, at))
        same([got.codes, got.exps], [own.codes, own.exps])
        part = qn.Act8(view(own.codes, at), view(own.exps, at))
        assert torch.equal(qn.act8_unpack(part), qn.act8_unpack(own))
    part = qn.Act8(own.codes[2:], own.exps[2:])
    assert torch.equal(qn.act8_unpack(part), qn.act8_unpack(own)[2:])


def test_linear_backward_from_a_slice_of_a_checkpoint(qn):
    """One half of a batch: five exponents a row start between 16-byte boundaries."""
    M, rows, cols, r = 42, 72, 320, 5
    st = qn.nf4_quantize_dq(rnd(rows, cols, dtype=F32) * 0.02)
    x8, G = qn.act8_pack(rnd(M, cols)), rnd(M, rows, seed=1)
    A, B, u = rnd(r, cols, seed=2), rnd(rows, r, seed=3), rnd(M, r, dtype=F32, seed=4)
    half = qn.Act8(x8.codes[21:], x8.exps[21:])
    got = qn.qlora_linear_bwd_act8(st, half, G[21:], view(A), view(B, 3), 10.0, u[21:])
    ref = qn.qlora_linear_bwd_act8(st, qn.Act8(half.codes.clone(), half.exps.clone()),
                                   G[21:].clone(), A, B, 10.0, u[21:].clone())
    same(got, ref)


def test_outputs_have_to_start_on_16_bytes(qn):
    """Where the caller names one: it cannot be copied for them."""
    x = rnd(4, 128)
    own = qn.act8_pack(x)
    with pytest.raises(qn.QNError):
        qn.act8_pack(x, out=qn.Act8(view(own.codes), own.exps))
    with pytest.raises(qn.QNError):
        qn.act8_unpack(own, out=view(x))
