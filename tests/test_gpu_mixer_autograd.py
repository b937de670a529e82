"""The token mixer's operations as autograd sees them: which gradients arrive, and what is refused rather than lost."""
import pytest
import torch

import depthwise_convolution_gb300 as dw
import mixer_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("with_grad", [True, False])
@pytest.mark.parametrize("with_lengths", [True, False])
@pytest.mark.parametrize("with_bias", [True, False])
def test_the_window_has_its_gradient_with_and_without_a_bias(with_bias, with_lengths, with_grad):
    g = torch.Generator().manual_seed(3)
    x, dy = (torch.randn(3, 40, 24, generator=g).cuda() for _ in range(2))
    w, bias = torch.randn(4, 24, generator=g).cuda(), torch.randn(24, generator=g).cuda() if with_bias else None
    state = torch.randn(3, 3, 24, generator=g).cuda()
    n = torch.tensor([40, 2, 0], dtype=torch.int32).cuda() if with_lengths else None
    want = dw.dwconv_causal_bwd(dy, x, w, bias, state=state, lengths=n, need_db=with_bias, need_dstate=True)
    leaves = [t.clone().requires_grad_() for t in (x, w)] + ([bias.clone().requires_grad_()] if with_bias else [])
    window = state.clone().requires_grad_(with_grad)
    dw.causal_conv(leaves[0], leaves[1], leaves[2] if with_bias else None, state=window, lengths=n).backward(dy)
    for leaf, d in zip(leaves, want):
        assert torch.equal(leaf.grad, d)
    if not with_grad:
        assert window.grad is None
        return
    assert torch.equal(window.grad, want[3])
    ls = ref.leaf(state)
    ry, _ = ref.conv(ref.wide(x), ref.wide(w), ref.wide(bias), "silu", ls, ref.wide(n))
    rs, = torch.autograd.grad(ry, ls, ref.wide(dy))
    # test_gpu_causal_conv.py's bound for gradients, 4e-6 of the summed magnitudes: W taps of at most 1.1 |dy| |w|
    size = 4 * 1.1 * dy.abs().max().item() * w.abs().max().item() * torch.ones_like(rs)
    ref.assert_near(window.grad, rs, "dstate", "fp32", 4e-6, size)
