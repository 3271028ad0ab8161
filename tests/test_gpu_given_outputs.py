"""Outputs that calls are given: too short, strided, of another type or on the host they are
refused before anything is launched; written, they count as modified."""
import pytest
import torch

from tests._gpu import needs_gpu, say

pytestmark = [pytest.mark.gpu, needs_gpu]
F32, BF16 = torch.float32, torch.bfloat16


def _calls(qn):
    """(name, type of the output, its shape, call with it)"""
    torch.manual_seed(0)
    normal = lambda *s, t=BF16: torch.randn(*s, device="cuda").to(t)  # noqa: E731
    M, rows, cols, r = 40, 72, 128, 8
    W = normal(rows, cols, t=F32)
    st = qn.nf4_quantize_dq(W)
    x, A, B = normal(M, cols), normal(r, cols), normal(rows, r)
    Wb, V = qn.nf4_dequantize(st), normal(M, r, t=F32)
    drop = qn.Dropout(0.1, 1)
    return [
        ("fwd", BF16, (M, rows), lambda y: qn.qlora_linear_fwd(st, x, A, B, 8.0, y=y)[0]),
        ("fwd drop", BF16, (M, rows),
         lambda y: qn.qlora_linear_fwd(st, x, A, B, 8.0, y=y, drop=drop)[0]),
        ("fwd decode", BF16, (1, rows), lambda y: qn.qlora_linear_fwd(st, x[:1], A, B, 8.0, y=y)[0]),
        ("bf16", BF16, (M, rows), lambda y: qn.lora_linear_bf16(x, Wb, V, B, 8.0, y=y)),
        ("dequantize", F32, (rows, cols), lambda y: qn.nf4_dequantize(st, F32, out=y)),
        ("merge", F32, (rows, cols), lambda y: qn.nf4_merge_lora(st, A, B, 8.0, out=y)),
    ]


def test_given_outputs():
    import quantized_fine_tuning_nf4_amd as qn
    for name, t, shape, call in _calls(qn):
        say(f"[given] {name}")
        want = call(None)
        new = lambda *s, dtype=t, device="cuda": torch.zeros(*s, dtype=dtype, device=device)  # noqa: E731
        for bad in (new(shape[0], shape[1] - 1), new(shape[0], 2 * shape[1])[:, ::2],
                    new(*shape, dtype=torch.float16), new(*shape, device="cpu"), new(0)):
            with pytest.raises(ValueError):
                call(bad)
        out = new(*shape)
        p = torch.ones_like(out).requires_grad_()
        z = (p * out).sum()  # keeps out for its backward
        got = call(out)
        assert got.data_ptr() == out.data_ptr() and torch.equal(got, want)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            z.backward()
        with torch.inference_mode():
            assert torch.equal(call(new(*shape)), want)


def test_given_states_and_copies():
    import quantized_fine_tuning_nf4_amd as qn
    say("[given states]")
    W = torch.randn(72, 128, device="cuda")
    want = qn.nf4_quantize_dq(W)
    out = qn.empty_state(72, 128, "cuda")
    assert qn.nf4_quantize_dq(W, out=out) is out and torch.equal(out.packed, want.packed)
    for name in ("packed", "qscale", "scale2", "offset"):
        bad = qn.empty_state(72, 128, "cuda")
        setattr(bad, name, getattr(bad, name)[:-1])
        with pytest.raises(ValueError):
            qn.nf4_quantize_dq(W, out=bad)
    with pytest.raises(ValueError):
        qn.nf4_quantize_dq(W, out=qn.qn_quantize(W, double_quant=False))
    opt = qn.Adam8(torch.zeros(300, device="cuda"))
    with pytest.raises(ValueError):
        opt.step(torch.ones(300, device="cuda"), torch.zeros(299, dtype=BF16, device="cuda"))
    opt.step(torch.ones(300, device="cuda"), torch.zeros(300, dtype=BF16, device="cuda"))
    torch.cuda.synchronize()
