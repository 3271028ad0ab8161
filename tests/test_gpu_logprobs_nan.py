"""Alternatives of rows that hold a NaN: a NaN logit is none of them, whichever of the
forward's routes a row takes, and a call repeats itself.  (Their log probabilities
are NaN, as everything that is summed over such a row.)"""
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


# one workgroup of 4 waves a row; of 16; slices joined by 4 waves and by 16
@pytest.mark.parametrize("T,V", [(6, 5003), (300, 777), (6, 9001), (520, 9001), (6, 70001)])
@pytest.mark.parametrize("f32", [False, True])
def test_nan_is_no_alternative(qn, T, V, f32):
    say(f"[logprobs nan] T={T} V={V} f32={f32}")
    g = torch.Generator().manual_seed(V)
    x = torch.randn(T, V, generator=g) * 2.5
    x[0, 3] = math.nan                              # one, early
    x[1, V - 1] = -math.nan                         # one, last
    x[2, torch.rand(V, generator=g) < 0.3] = math.nan
    x[3] = math.nan                                 # nothing else
    x[4] = math.nan
    x[4, V // 2], x[4, V // 3] = 1.0, 2.0           # two alternatives
    x[5, : V // 2] = math.nan
    x[5, V // 2 + 1] = math.inf
    x = x.to(torch.float32 if f32 else torch.bfloat16)
    if f32:  # a signalling NaN
        x.view(torch.int32)[0, 5] = 0x7F800001
    else:
        x.view(torch.int16)[0, 5] = 0x7F81
    vals = x.double().numpy()
    vals = np.where(np.isnan(vals), -np.inf, vals)
    for k in (1, 5, 32):
        want = np.full((T, k), -1)
        for r in range(T):
            order = np.lexsort((np.arange(V), -vals[r]))[:k]
            order = order[vals[r][order] > -np.inf]
            want[r, :len(order)] = order
        first = None
        for _ in range(3):
            r = qn.token_logprobs_fwd(x.cuda(), top_k=k)
            torch.cuda.synchronize()
            assert np.array_equal(r.top_ids.cpu().numpy(), want)
            bad = torch.isnan(x).any(1) | torch.isinf(x).any(1)
            assert torch.equal(torch.isnan(r.entropy.cpu()), bad)
            there = torch.from_numpy(want) >= 0
            assert torch.isnan(r.top_logp.cpu()[bad])[there[bad]].all()
            assert torch.isneginf(r.top_logp.cpu()[~there]).all()
            bits = r.top_logp.view(torch.int32).cpu()
            first = bits if first is None else first
            assert torch.equal(bits, first)
