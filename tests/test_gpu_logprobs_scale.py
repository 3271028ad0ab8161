"""Token log probabilities at the ends of their scale (an inverse temperature): any
positive finite fp32 number, on every route of the forward."""
import math

import pytest
import torch

from tests._gpu import needs_gpu, say
from tests.test_gpu_logprobs import _logits, qn  # noqa: F401

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.mark.parametrize("T,V", [(3, 777), (3, 9001), (300, 33000), (3, 70001)])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("scale", [1e30, 2.4e38, 3.4e38])
def test_next_to_no_temperature(qn, T, V, f32, scale):  # noqa: F811
    """All of a row's probability on its largest logits, shared where they are equal."""
    say(f"[logprobs scale] T={T} V={V} f32={f32} scale={scale}")
    x, t = _logits(T, V, f32, seed=V)
    x = x.contiguous()
    x[0, 5], x[1, 7], x[1, V - 1], x[2, V // 2] = 40.0, 40.0, 40.0, 40.0
    t[0], t[1], t[2] = 5, V - 1, 0
    r = qn.token_logprobs_fwd(x, t, scale=scale, top_k=3)
    torch.cuda.synchronize()
    assert float(r.logp[0]) == 0.0 and float(r.entropy[0]) == 0.0
    assert abs(float(r.logp[1]) + math.log(2)) < 1e-6
    assert abs(float(r.entropy[1]) - math.log(2)) < 1e-6
    assert float(r.logp[2]) < -1e30 and float(r.entropy[2]) == 0.0
    assert r.top_ids[0, 0] == 5 and r.top_ids[1, :2].tolist() == [7, V - 1]
    assert float(r.top_logp[0, 0]) == 0.0 and float(r.top_logp[0, 1]) < -1e28
    dx = qn.token_logprobs_bwd(x[:2], t[:2], r.stats[:2].clone(), None, torch.full((2,), 0.5,
                                                                                   device="cuda"),
                               scale=scale)
    want = torch.zeros(2, V)
    want[1, V - 1], want[1, 7] = scale / 4, -scale / 4
    assert torch.allclose(dx.cpu().float(), want, rtol=2.0 ** -8, atol=0.0)


@pytest.mark.parametrize("scale", [1e-45, 1e-38, 1e-20])
def test_no_difference_left(qn, scale):  # noqa: F811
    x, t = _logits(3, 70001, True, seed=2)
    r = qn.token_logprobs_fwd(x, t, scale=scale, top_k=2)
    assert ((r.logp + math.log(70001)).abs() < 1e-5).all()
    assert ((r.entropy - math.log(70001)).abs() < 1e-5).all()
