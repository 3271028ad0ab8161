"""Tensors of two devices in one call under a Dropout are refused before anything runs."""
from types import SimpleNamespace

import pytest
import torch


def _on(k):
    return SimpleNamespace(device=torch.device("cuda", k))


@pytest.mark.parametrize("other", ["x", "codes", "exps", "A", "B", "u", "packed"])
def test_two_devices(monkeypatch, other):
    from quantized_fine_tuning_nf4_amd import mx4
    monkeypatch.setattr(mx4, "_one_device", lambda: False)
    t = {k: _on(int(k == other)) for k in ("x", "codes", "exps", "A", "B", "u", "packed")}
    act8 = other in ("codes", "exps")
    x8 = SimpleNamespace(codes=t["codes"], exps=t["exps"]) if act8 else None
    with pytest.raises(ValueError, match="one device"):
        mx4._qlora_bwd_drop(SimpleNamespace(packed=t["packed"]), None if act8 else t["x"], x8, _on(0),
                            t["A"], t["B"], 8, 1.0, False, None, t["u"], None, None, None, None)
