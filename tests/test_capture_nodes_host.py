"""What a forward under capture finds out about its parameters: whether a graph that is not
the capture's still holds the nodes that add up their gradients."""
import torch


def _nodes(*leaves, stream=7):
    import quantized_fine_tuning_nf4_amd as qn
    return qn._nodes(leaves, stream)


def test_nodes_of_eager_graphs():
    A, B = torch.nn.Parameter(torch.randn(3)), torch.nn.Parameter(torch.randn(3))
    frozen = torch.nn.Parameter(torch.randn(3), requires_grad=False)
    assert _nodes(A, B, None, frozen, torch.nn.Parameter(torch.randn(3)) * 2)[1] is False
    eager = (A * B).sum()
    assert _nodes(A)[1] and _nodes(B, A)[1]
    assert _nodes(A)[1]  # asked again: the same answer
    eager.backward()
    assert _nodes(A)[1]  # a backward that has run leaves the graph with its outputs
    del eager
    assert _nodes(A, B)[1] is False


def test_nodes_of_the_capture():
    A = torch.nn.Parameter(torch.randn(3))
    held, older = _nodes(A)
    y = A.exp()  # the first use takes the node that was looked at
    del held
    assert older is False
    assert _nodes(A)[1] is False  # the second use in the same capture
    assert _nodes(A, stream=8)[1]  # a capture on another stream
    del y
    assert _nodes(A, stream=8)[1] is False
    assert A.grad is None and A.grad_fn is None
