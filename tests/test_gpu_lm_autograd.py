"""A second derivative through the language-model operators is refused: their backwards have none of their own."""
import pytest
import torch

from linear_recurrence_sequence_amd import autograd
from tests.helpers import say

pytestmark = pytest.mark.gpu


def twice(out, leaf):
    g = torch.autograd.grad(out, leaf, create_graph=True)[0]
    # the leaf's own part keeps the second derivative from failing for want of any graph
    (g.float().pow(2).sum() + leaf.float().pow(2).sum()).backward()


def test_second_derivatives_are_refused():
    say("[lm] second derivatives")
    g = torch.Generator(device="cuda").manual_seed(1)
    h = torch.randn(20, 64, generator=g, device="cuda").bfloat16().requires_grad_()
    w = torch.randn(90, 64, generator=g, device="cuda").bfloat16()
    t = torch.randint(0, 90, (20,), generator=g, device="cuda")
    with pytest.raises(RuntimeError, match="no second derivative"):
        twice(autograd.linear_ce(h, w, t)[0].sum(), h)
    x = torch.randn(20, 64, generator=g, device="cuda").requires_grad_()
    with pytest.raises(RuntimeError, match="no second derivative"):
        twice(autograd.block_norm(x, x.detach(), None, None, None, torch.ones(64, device="cuda"))[1].sum(), x)


def test_create_graph_without_a_second_derivative():
    """The gradients themselves are those of a call without create_graph, and a gradient of something else passes by."""
    say("[lm] create_graph")
    g = torch.Generator(device="cuda").manual_seed(2)
    h = torch.randn(20, 64, generator=g, device="cuda").bfloat16().requires_grad_()
    w = torch.randn(90, 64, generator=g, device="cuda").bfloat16()
    t = torch.randint(0, 90, (20,), generator=g, device="cuda")
    want = torch.autograd.grad(autograd.linear_ce(h, w, t)[0].sum(), h)[0]
    got = torch.autograd.grad(autograd.linear_ce(h, w, t)[0].sum(), h, create_graph=True)[0]
    assert not want.requires_grad and got.requires_grad and torch.equal(got, want)
    (got.detach().float() * h.float()).sum().backward()
    assert torch.equal(h.grad, got.detach())
    with pytest.raises(RuntimeError, match="linear_ce has no second derivative"):
        got.float().sum().backward()
