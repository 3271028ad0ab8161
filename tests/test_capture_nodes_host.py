"""What the layers' forwards note about their parameters' nodes: whether one belongs to the
default stream while the forward runs on another (a capture's)."""
import pytest
import torch


class Two(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, A, B, other):
        return x + A + B

    @staticmethod
    def backward(ctx, g):
        import quantized_fine_tuning_nf4_amd as qn
        qn._refuse_default_stream(ctx)
        return g, g, g, None


def _call(A, B, stream, x=None):
    import quantized_fine_tuning_nf4_amd as qn
    y = Two.apply(torch.zeros(3) if x is None else x, A, B, "other")
    qn._mark_nodes(y, stream)
    return y


def _meets(y):
    return getattr(y.grad_fn, "meets_default_stream", False)


def test_nodes_and_their_streams():
    A, B = (torch.nn.Parameter(torch.randn(3)) for _ in range(2))
    eager = _call(A, B, 0)
    assert not _meets(eager)  # on the default stream itself
    assert not _meets(_call(A, B, 0))
    assert _meets(_call(A, B, 7)) and _meets(_call(A, B, 9))
    eager.sum().backward()
    assert _meets(_call(A, B, 7))  # a backward that has run leaves the graph with its output
    del eager
    y = _call(A, B, 7)
    assert not _meets(y) and not _meets(_call(A, B, 8))  # of other streams: no fault
    del y
    z = _call(A, B, 0, x=A)  # the same leaf twice
    assert not _meets(z) and _meets(_call(B, A, 7))


def test_graphs_without_parameters():
    A, B = (torch.nn.Parameter(torch.randn(3), requires_grad=False) for _ in range(2))
    assert _call(A, B, 7).grad_fn is None
    x = (torch.zeros(3, requires_grad=True) * 2)
    held = _call(A, B, 0, x=x)
    assert not _meets(held) and not _meets(_call(A, B, 7, x=x))


def test_a_captured_backward_raises(monkeypatch):
    A, B = (torch.nn.Parameter(torch.randn(3)) for _ in range(2))
    eager = _call(A, B, 0)
    y = _call(A, B, 7)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(RuntimeError, match="let go of every eager output"):
        y.sum().backward()
    assert A.grad is None
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    eager.sum().backward()
    assert A.grad is not None
