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


def operations():
    """(name, function of its differentiable inputs, those inputs): each of the three operations."""
    g = torch.Generator().manual_seed(5)
    x, w = torch.randn(2, 30, 16, generator=g).cuda(), torch.randn(4, 16, generator=g).cuda()
    y, one = torch.randn(6, 32, generator=g).cuda(), torch.ones(32).cuda()
    q, k, v = (torch.randn(1, 30, 1, 16, generator=g).cuda() for _ in range(3))
    gate, beta = -torch.rand(1, 30, 1, generator=g).cuda(), torch.rand(1, 30, 1, generator=g).cuda()
    return [("causal_conv", lambda *a: dw.causal_conv(*a), [x, w]),
            ("block_norm", lambda *a: dw.block_norm(a[0], w_post=a[1])[0], [y, one]),
            ("gated_delta_rule", lambda *a: dw.gated_delta_rule(*a, qk_norm=True), [q, k, v, gate, beta])]


@pytest.mark.parametrize("which", range(3))
def test_forward_mode_is_refused(which):
    import torch.autograd.forward_ad as fwd
    name, f, args = operations()[which]
    plain = f(*args)
    for requires in (False, True):
        with fwd.dual_level():
            dual = [fwd.make_dual(a.clone().requires_grad_(requires), torch.ones_like(a)) if i == 0 else a
                    for i, a in enumerate(args)]
            with pytest.raises(RuntimeError, match="forward"):
                f(*dual)
            with torch.no_grad(), pytest.raises(RuntimeError, match="forward"):
                f(*dual)
    assert torch.equal(f(*args), plain)


@pytest.mark.parametrize("which", range(3))
def test_second_derivatives_are_refused(which):
    name, f, args = operations()[which]
    leaves = [a.requires_grad_() for a in args]
    out = f(*leaves)
    for up in (torch.ones_like(out), torch.ones_like(out).requires_grad_()):
        first = torch.autograd.grad(out, leaves, up, create_graph=True)
        plain = torch.autograd.grad(out, leaves, up.detach(), retain_graph=True)
        assert all(torch.equal(a, b) for a, b in zip(first, plain))
        for d in first:  # a penalty on a gradient, beside a term that has a history of its own
            with pytest.raises(RuntimeError, match="twice"):
                torch.autograd.grad(d.square().sum() + leaves[0].square().sum(), leaves, retain_graph=True,
                                    allow_unused=True)
            for leaf in leaves:  # whichever is asked for
                with pytest.raises(RuntimeError, match="twice"):
                    torch.autograd.grad(d.square().sum() + leaf.square().sum(), leaf, retain_graph=True)


def test_states_written_in_place_raise_their_version():
    g = torch.Generator().manual_seed(6)
    scale = torch.randn((), generator=g).cuda().requires_grad_()
    x, w, window = (torch.randn(*s, generator=g).cuda() for s in ((2, 16), (4, 16), (2, 3, 16)))
    q, v, gate = torch.randn(2, 1, 16, generator=g).cuda(), torch.randn(2, 1, 8, generator=g).cuda(), \
        -torch.rand(2, 1, generator=g).cuda()
    state = torch.randn(2, 1, 16, 8, generator=g).cuda()
    out = torch.empty(2, 16, device="cuda")
    seq = [t[:, None] for t in (q, q, v, gate, gate.neg())]
    calls = [(window, lambda: dw.dwconv_causal_step(x, w, window)),
             (window, lambda: dw.dwconv_causal_step(x, w, window, out=out)),
             (out, lambda: dw.dwconv_causal_step(x, w, window, out=out)),
             (state, lambda: dw.dwconv_delta_step(q, q, v, gate, gate.neg(), state)),
             (state, lambda: dw.dwconv_delta_step(q, q, v, gate, gate.neg(), state, stream=torch.cuda.current_stream())),
             (state, lambda: dw.dwconv_delta_fwd(*seq, state=state, state_out=state)),
             (window, lambda: dw.dwconv_causal_fwd(x[:, None], w, state_out=window))]
    for t, call in calls:
        kept = (t * scale).sum()
        before = t._version
        call()
        assert t._version > before
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            kept.backward()
    with torch.inference_mode():  # tensors without a version
        dw.dwconv_causal_step(x, w, torch.zeros(2, 3, 16, device="cuda"))
        dw.dwconv_delta_step(q, q, v, gate, gate.neg(), torch.zeros(2, 1, 16, 8, device="cuda"), out=torch.empty_like(v))


def test_keys_too_wide_for_gradients_are_refused_at_once():
    q, v = torch.randn(1, 20, 1, 200, device="cuda"), torch.randn(1, 20, 1, 16, device="cuda", requires_grad=True)
    gate = torch.zeros(1, 20, 1, device="cuda")
    with pytest.raises(ValueError, match="128"):
        dw.gated_delta_rule(q, q, v, gate, gate)
    with torch.no_grad():
        assert dw.gated_delta_rule(q, q, v, gate, gate).shape == v.shape
    assert dw.gated_delta_rule(q, q, v.detach(), gate, gate).shape == v.shape
