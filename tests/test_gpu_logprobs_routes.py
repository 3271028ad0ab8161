"""Masks, infinities, NaN and targets out of range on every route of the forward: a
workgroup of four waves a row, one of sixteen, and rows cut in slices that are joined
by four waves and by sixteen.  References and tolerances as in test_gpu_logprobs."""
import math

import pytest
import torch

from tests._gpu import needs_gpu, say
from tests.test_gpu_logprobs import _check, _logits, qn  # noqa: F401

pytestmark = [pytest.mark.gpu, needs_gpu]

ROUTES = [(9, 5003), (9, 9001), (520, 9001), (300, 33000), (9, 70001)]
both = pytest.mark.parametrize("f32", [False, True])
routes = pytest.mark.parametrize("T,V", ROUTES)


@both
@routes
def test_masks(qn, T, V, f32):  # noqa: F811
    say(f"[logprobs routes masks] T={T} V={V} f32={f32}")
    low = torch.finfo(torch.float32 if f32 else torch.bfloat16).min
    x, t = _logits(T, V, f32, seed=V + T)
    x = x.contiguous()
    x[0] = -math.inf                       # nothing allowed: every slice empty
    x[1] = -math.inf
    x[1, V - 3] = 3.0                      # one token, in the last slice
    x[2, ::2] = -math.inf                  # the target banned
    x[3] = low                             # every logit the type's lowest value
    x[4, 1:] = low                         # all but one masked by it
    x[5, : V * 2 // 3] = -math.inf         # the first slices whole
    x[6, V // 3:] = -math.inf              # the last slices whole
    x[7] = -math.inf                       # fewer alternatives than asked for, far apart
    x[7, [5, V // 2, V - 1]] = torch.tensor([1.0, 2.0, 1.0], dtype=x.dtype, device="cuda")
    x[8, 100:] = low                       # the lowest value beside -inf
    x[8, : 50] = -math.inf
    t[0], t[1], t[2], t[7] = 7, V - 3, 4, V - 1
    for k in (0, 8, 32):
        r, ref = _check(qn, x, t, k=k)
        assert torch.isneginf(r.logp[0]) and float(r.entropy[0]) == 0.0
        assert float(r.entropy[1]) == 0.0 and float(r.logp[1]) == 0.0
        assert torch.isneginf(r.logp[2])
    assert r.top_ids[7].tolist() == [V // 2, 5, V - 1] + [-1] * 29
    assert (r.top_ids[0] == -1).all() and torch.isneginf(r.top_logp[0]).all()
    one = torch.ones(T, device="cuda")
    dx = qn.token_logprobs_bwd(x, t, r.stats, r.entropy, one, one)
    torch.cuda.synchronize()
    assert torch.isfinite(dx).all() and not dx[0].any()
    banned = torch.isneginf(x)
    banned[torch.arange(T), t] = False
    assert not dx[banned].any()


@both
@routes
def test_nan_and_inf_in_one_place(qn, T, V, f32):  # noqa: F811
    say(f"[logprobs routes nan] T={T} V={V} f32={f32}")
    x, t = _logits(T, V, f32, seed=V + T + 1)
    x = x.contiguous()
    bad = {0: (0, math.nan), 2: (V - 1, math.nan), 3: (V // 2, math.inf), 5: (V - 1, math.inf),
           6: (V // 3, math.nan), 7: (V // 5, math.inf)}
    for row, (at, v) in bad.items():
        x[row, at] = v
    x[6, : V // 3] = -math.inf             # the NaN the first that is no -inf
    t[7] = -1
    r = qn.token_logprobs_fwd(x, t, top_k=3)
    torch.cuda.synchronize()
    for row in range(9):
        assert bool(torch.isnan(r.entropy[row])) == (row in bad), row
        assert bool(torch.isnan(r.logp[row])) == (row in bad and row != 7), row
    assert r.logp[7] == 0
    good = [i for i in range(T) if i not in bad]
    _check(qn, x[good].contiguous(), t[good].contiguous(), k=3)
    for row in (3, 5, 7):                  # +inf is the best alternative
        assert int(r.top_ids[row, 0]) == bad[row][0]
    assert torch.isnan(r.top_logp[sorted(bad)]).all()


@both
@routes
def test_ignored_and_impossible_targets(qn, T, V, f32):  # noqa: F811
    say(f"[logprobs routes targets] T={T} V={V} f32={f32}")
    x, t = _logits(T, V, f32, seed=V + T + 2)
    t[:6] = torch.tensor([-1, -(1 << 40), V, 1 << 40, 0, V - 1], device="cuda")
    r, _ = _check(qn, x, t, k=2)
    assert (r.logp[:2] == 0).all() and torch.isnan(r.logp[2:4]).all()
    dx = qn.token_logprobs_bwd(x, t, r.stats, r.entropy, torch.ones(T, device="cuda"))
    torch.cuda.synchronize()
    assert not dx[:4].any() and dx[4].any() and dx[5].any()
