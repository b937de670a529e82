"""What the token mixer's Python functions do with a call that their native forms refuse or that fails.  No GPU."""
import pytest
import torch

import depthwise_convolution_gb300 as dw
from depthwise_convolution_gb300 import mixer_ops

X, W, STATE = torch.zeros(2, 8), torch.zeros(4, 8), torch.zeros(2, 3, 8)
Q, V, G = torch.zeros(2, 1, 8), torch.zeros(2, 1, 4), torch.zeros(2, 1)
POOL = torch.zeros(2, 1, 8, 4)
CALLS = {
    "causal_step": lambda: dw.dwconv_causal_step(X, W, STATE),
    "causal_fwd": lambda: dw.dwconv_causal_fwd(X[None], W),
    "block_norm_fwd": lambda: dw.dwconv_block_norm_fwd(X),
    "delta_step": lambda: dw.dwconv_delta_step(Q, Q, V, G, G, POOL),
    "causal_conv": lambda: dw.causal_conv(X[None], W),
    "block_norm": lambda: dw.block_norm(X),
    "gated_delta_rule": lambda: dw.gated_delta_rule(Q[None], Q[None], V[None], G[None], G[None]),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_call_that_fails_is_not_made_again(name, monkeypatch):
    """A launch that reports a failure may have moved a state: the call ends there."""
    made = []

    def native(*args):
        made.append(args)
        raise RuntimeError("the launch failed")

    monkeypatch.setitem(mixer_ops._NATIVE, name, native)
    monkeypatch.setattr(mixer_ops, "_ll", lambda: pytest.fail("called again"))
    with pytest.raises(RuntimeError, match="the launch failed"):
        CALLS[name]()
    assert len(made) == 1


@pytest.mark.parametrize("name", CALLS)
def test_a_missing_extension_is_said(name, monkeypatch):
    def module():
        raise RuntimeError("g++ failed")

    monkeypatch.setattr(mixer_ops, "_NATIVE", {})
    monkeypatch.setattr(mixer_ops, "_module", module)
    with pytest.raises(RuntimeError, match=r"g\+\+ failed"):
        CALLS[name]()


@pytest.mark.parametrize("name", CALLS)
def test_arguments_that_are_refused_get_words(name):
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        CALLS[name]()
