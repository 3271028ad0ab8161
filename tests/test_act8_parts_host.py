"""What the tests of the adapter gradients' three bf16 parts rest on, on the CPU: a
factor of 1 + 2^-9 + 2^-18 a needs all three, and two leave an error past their bound."""
import torch


def _parts(x, n):
    out, rest = [], x.clone()
    for _ in range(n):
        h = rest.to(torch.bfloat16).float()
        out.append(h)
        rest = rest - h
    return out


def test_two_parts_lose_what_the_tests_look_for():
    u = 1.0 + 2.0 ** -9 + torch.arange(3).float() * 2.0 ** -18
    two, three = _parts(u, 2), _parts(u, 3)
    assert torch.equal(sum(three), u) and torch.equal(three[2], torch.arange(3) * 2.0 ** -18)
    assert torch.equal(two[0] + two[1], torch.full((3,), 1.0 + 2.0 ** -9))


def test_two_parts_are_past_the_bound():
    g = torch.Generator().manual_seed(0)
    u = torch.randn(2048, 16, generator=g)
    G = torch.randn(2048, 64, generator=g).to(torch.bfloat16).double()
    want = G.t() @ u.double()

    def off(n):
        got = G.t() @ sum(p.double() for p in _parts(u, n))
        return float((got - want).norm() / want.norm())

    assert off(2) > 1.5e-6 and off(3) < 2e-8
