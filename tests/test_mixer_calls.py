"""What the token mixer's Python functions do with a call that their native forms refuse or that fails.  No GPU."""
import pytest
import torch

import depthwise_convolution_gb300 as dw
from depthwise_convolution_gb300 import _lib, mixer_ops

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


A = 0x7F0000000000  # never dereferenced: validation fails first


@pytest.mark.parametrize("by", [0, 2, -(2 * 3 * 16 - 1) * 2])
def test_a_window_is_not_written_over_the_one_that_is_read(by):
    """B = 2 windows of 3 x 16 bf16: the same buffer, one value on, the last value of one the first of the other."""
    lib = _lib.load()
    assert lib.dwconv_causal_fwd(2, 8, 16, 4, _lib.BF16, A + (1 << 20), 128, 16, A, None, _lib.ACT_SILU, A, None,
                                 A + (1 << 24), A + by, None) == _lib.ERR_INVALID_ARG


@pytest.mark.parametrize("by", [4, -4, (2 * 4 * 8 * 6 - 1) * 4])
def test_a_state_is_written_over_itself_or_apart(by):
    """2 x 4 states of 8 x 6 floats, shifted against each other."""
    lib = _lib.load()
    q = A + (1 << 24)
    assert lib.dwconv_delta_fwd(2, 4, 2, 4, 8, 6, _lib.BF16, _lib.BF16, q, q, q, q, q, None, 0.1, 1, A, None,
                                A + (1 << 28), A + by, None, None, 0, None) == _lib.ERR_INVALID_ARG
