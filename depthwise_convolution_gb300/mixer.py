"""The token mixer as differentiable PyTorch operations.

``causal_conv``, ``gated_delta_rule`` and ``block_norm`` check their arguments and call native autograd nodes (which
only marshal arguments and save inputs, every pass runs in the library's kernels); ``GatedDeltaMixer`` puts them
together as a layer.  They are differentiable once and in reverse: forward mode and the derivative of a gradient raise
NotImplementedError.
"""
from __future__ import annotations

import torch

from . import mixer_ops as ops


def causal_conv(x, w, bias=None, act="silu", state=None, lengths=None):
    """Differentiable short causal depthwise convolution along time: x [B,T,C], w [W,C],
    bias [C] float32, state [B,W-1,C], lengths [B] int32 (see dwconv_causal_fwd)."""
    if isinstance(w, torch.Tensor) and not w.is_contiguous():
        w = w.contiguous()
    out = ops._native("causal_conv")(x, w, bias, state, lengths, ops._act(act))
    if out is NotImplemented:
        ops._causal_sequence(x, w, bias, act, state, lengths)  # says what is wrong with them
        raise ValueError("unsupported arguments")
    return out


def gated_delta_rule(q, k, v, g, beta, scale=None, qk_norm=False, state=None, lengths=None, return_state=False):
    """Differentiable gated delta rule: q, k [B,T,Hk,K], v [B,T,Hv,V], g, beta [B,T,Hv],
    state [B,Hv,K,V] float32 (see dwconv_delta_fwd); K <= 128 for gradients.  Returns o,
    with return_state (o, last state).  Keeps the forward pass's chunk tiles for the
    backward pass where a gradient is wanted."""
    out = ops._native("gated_delta_rule")(q, k, v, g, beta, state, lengths, scale, bool(qk_norm), bool(return_state))
    if out is NotImplemented:
        (_, _), (_, _, K, _), *_ = ops._delta_checks(q, k, v, g, beta, 2, state, (lengths, "lengths"))
        raise ValueError(f"gradients take keys of at most 128 values, got {K}" if K > 128 else "unsupported arguments")
    return out if return_state else out[0]


def block_norm(y, residual=None, gate=None, w_post=None, scale=None, w_pre=None, kind="rms", gate_act="silu",
               eps=1e-6):
    """Differentiable norms around a block: (h, n) with h = residual + scale * post(y) *
    act(gate) and n = pre(h), or n None without w_pre (see dwconv_block_norm_fwd)."""
    codes = ops._choice(ops.NORMS, kind, "norm"), ops._choice(ops.GATES, gate_act, "gate activation")
    out = ops._native("block_norm")(y, residual, gate, w_post, scale, w_pre, *codes, eps)
    if out is NotImplemented:
        ops._norm_checks(((y, "y"), (residual, "residual"), (gate, "gate")),
                         ((w_post, "w_post"), (scale, "scale"), (w_pre, "w_pre")), kind, gate_act)
        raise ValueError("unsupported arguments")
    return (out[0], out[1]) if w_pre is not None else (out[0], None)


class MixerCache:
    """What a mixer keeps of sequences between calls: a slot each with the convolution's
    window [N, W-1, C] and the rule's states [N, Hv, K, V] (float32)."""

    def __init__(self, mixer: "GatedDeltaMixer", slots: int):
        w = mixer.conv_weight
        self.window = torch.zeros(slots, w.shape[0] - 1, w.shape[1], dtype=w.dtype, device=w.device)
        self.state = torch.zeros(slots, mixer.value_heads, mixer.key_width, mixer.value_width, dtype=torch.float32,
                                 device=w.device)


class GatedDeltaMixer(torch.nn.Module):
    """A gated-delta token mixer in a residual stream, the causal convolution in front of
    the gated delta rule and the norms around both.

    Takes the normalised stream n and the stream h [B, T, width] and returns the stream
    with the mixer's contribution and its norm for the next block:
      q, k, v = SiLU(conv(n W)),  o = delta(q, k, v, g, beta),
      h' = h + scale * (norm(o) SiLU(gate)) W_out,  n' = norm(h').
    ``prefill`` and ``step`` do the same against a :class:`MixerCache`.  The projections
    are plain matrix products, decay and write strength plain PyTorch operations on one
    value a head and token; everything else runs in the library's kernels.
    """

    def __init__(self, width, key_heads, value_heads, key_width=128, value_width=128, taps=4, dtype=torch.bfloat16,
                 device="cuda"):
        super().__init__()
        self.key_heads, self.value_heads = key_heads, value_heads
        self.key_width, self.value_width = key_width, value_width
        keys, values = key_heads * key_width, value_heads * value_width
        self.parts = (2 * keys + values, values, value_heads, value_heads)  # to mix, gate, decay, write strength

        def normal(*shape, std, kind=dtype):
            return torch.nn.Parameter((torch.randn(*shape, device=device) * std).to(kind))

        def constant(value, n):
            return torch.nn.Parameter(torch.full((n,), value, device=device))

        self.in_weight = normal(sum(self.parts), width, std=width ** -0.5)
        self.out_weight = normal(width, values, std=values ** -0.5)
        self.conv_weight = normal(taps, self.parts[0], std=taps ** -0.5)
        self.conv_bias = constant(0.0, self.parts[0])
        self.rate = torch.nn.Parameter(torch.linspace(0.5, 8.0, value_heads, device=device).log())
        self.step_bias = constant(-3.0, value_heads)
        self.head_norm = constant(1.0, value_width)
        self.scale = constant(1.0, width)
        self.next_norm = constant(1.0, width)

    def _project(self, n):
        mix, gate, decay, strength = torch.nn.functional.linear(n, self.in_weight).split(self.parts, -1)
        g = -torch.exp(self.rate) * torch.nn.functional.softplus(decay.float() + self.step_bias)
        return mix, gate.unflatten(-1, (self.value_heads, self.value_width)), g, torch.sigmoid(strength.float())

    def _heads(self, mixed):
        keys = self.key_heads * self.key_width
        q, k, v = mixed.split((keys, keys, mixed.shape[-1] - 2 * keys), -1)
        return (q.unflatten(-1, (self.key_heads, self.key_width)), k.unflatten(-1, (self.key_heads, self.key_width)),
                v.unflatten(-1, (self.value_heads, self.value_width)))

    def _finish(self, o, gate, h):
        o, _ = block_norm(o, gate=gate, w_post=self.head_norm)
        y = torch.nn.functional.linear(o.flatten(-2), self.out_weight)
        return block_norm(y, h, scale=self.scale, w_pre=self.next_norm)

    def forward(self, n, h):
        """(h', n') over whole sequences from an empty past; differentiable."""
        mix, gate, g, beta = self._project(n)
        q, k, v = self._heads(causal_conv(mix, self.conv_weight, self.conv_bias))
        return self._finish(gated_delta_rule(q, k, v, g, beta, qk_norm=True), gate, h)

    @torch.no_grad()
    def prefill(self, n, h, cache, lengths=None):
        """(h', n') over sequences that continue the cache's slots 0 .. B-1 (lengths [B] int32: live tokens)."""
        B = n.shape[0]
        mix, gate, g, beta = self._project(n)
        mixed, window = ops.dwconv_causal_fwd(mix, self.conv_weight, self.conv_bias, state=cache.window[:B],
                                              lengths=lengths, return_state=True)
        cache.window[:B] = window
        o = ops.dwconv_delta_fwd(*self._heads(mixed), g, beta, qk_norm=True, state=cache.state[:B], lengths=lengths,
                                 state_out=cache.state[:B])
        return self._finish(o, gate, h)

    @torch.no_grad()
    def step(self, n, h, cache, slots=None):
        """(h', n') for one token per row, n and h [B, width]; slots [B] int32 names each row's slot (idle
        outside [0, N))."""
        mix, gate, g, beta = self._project(n)
        mixed = ops.dwconv_causal_step(mix, self.conv_weight, cache.window, self.conv_bias, slots=slots)
        o = ops.dwconv_delta_step(*self._heads(mixed), g, beta, cache.state, qk_norm=True, slots=slots)
        return self._finish(o, gate, h)
