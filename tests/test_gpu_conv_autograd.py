"""What the differentiable 2-D convolution does with derivatives of its gradients."""
import pytest
import torch

from depthwise_convolution_gb300 import depthwise_conv2d

pytestmark = pytest.mark.gpu


def test_second_derivatives_are_refused():
    g = torch.Generator().manual_seed(1)
    x, w = torch.randn(1, 9, 9, 16, generator=g).cuda(), torch.randn(3, 3, 16, generator=g).cuda()
    leaves = [t.requires_grad_() for t in (x, w, torch.randn(16, generator=g).cuda())]
    out = depthwise_conv2d(*leaves, pad=1)
    up = torch.randn(out.shape, generator=g).cuda().requires_grad_()
    plain = torch.autograd.grad(out, leaves, up.detach(), retain_graph=True)
    first = torch.autograd.grad(out, leaves, up, create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(first, plain))
    reads = [(leaves[1], up), (leaves[0], up), (up,)]  # what dx, dw and db are made of
    for d, made_of in zip(first, reads):
        for t in (*leaves, up):
            total = d.square().sum() + t.square().sum()
            if any(t is r for r in made_of):
                with pytest.raises(NotImplementedError, match="twice"):
                    torch.autograd.grad(total, t, retain_graph=True)
            else:
                assert torch.equal(torch.autograd.grad(total, t, retain_graph=True)[0], 2 * t)
