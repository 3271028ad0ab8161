"""The workspace that a call is given: used where it is large enough, refused where the bytes
that the call writes in a row may not be there."""
import pytest
import torch


def test_workspaces():
    import quantized_fine_tuning_nf4_amd as qn
    cpu = torch.device("cpu")
    ws = torch.empty(64, dtype=torch.uint8)
    assert qn._room(ws, 64, cpu) is ws and qn._room(ws, 0, cpu) is ws
    for given in (None, ws, ws[::2], ws[:0]):  # too small: a new one
        new = qn._room(given, 65, cpu)
        assert new is not given and new.numel() == 65 and new.dtype == torch.uint8
    assert not qn._room(None, 100, cpu, zeroed=True).any()
    assert qn._room(None, 0, cpu).numel() == 1
    for given in (ws[::2], ws[:1].expand(64), ws.view(8, 8).t()):
        with pytest.raises(ValueError):
            qn._room(given, 16, cpu)
    with pytest.raises(ValueError):
        qn._room(ws, 64, torch.device("meta"))
    wide = torch.empty(16)  # (elements are counted: more bytes than that)
    assert qn._room(wide, 16, cpu) is wide
