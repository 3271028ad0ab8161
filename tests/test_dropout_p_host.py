"""Probabilities that 32 bits round to 1 are those of the largest share that can be dropped."""
import ctypes

import pytest


@pytest.mark.parametrize("p", [0.0, 0.3, 1 - 2.0 ** -24, 1 - 2.0 ** -25, 1 - 2.0 ** -30,
                               1 - 2.0 ** -53])
def test_every_probability_below_one_is_taken(p):
    import quantized_fine_tuning_nf4_amd as qn
    c = qn.Dropout(p, 1).c_struct()
    assert c.p < 1.0 and abs(c.p - p) <= 2.0 ** -24
    # (a call without elements looks at its options alone)
    assert qn.load_library().dropout_apply(None, qn.QN_F32, 0, ctypes.byref(c), None,
                                           None) == qn.QN_OK
