"""The token mixer at the edges of what it accepts: widths, gates and values where a kernel's form changes or a sum could
leave the finite numbers.  Tolerances are those of the operator's own test file, which derives them."""
import threading

import pytest
import torch

import depthwise_convolution_gb300 as dw
import mixer_reference as ref
import test_gpu_block_norm as norms
import test_gpu_delta as delta
import test_gpu_delta_bwd as delta_bwd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("C", [6672, 6680, 6912, 7040, 7048])
def test_norm_gradients_where_rows_stop_fitting_shared_memory(dtype, C):
    for rows in (3, 400):
        norms.test_gradients(dtype, (rows, C), "rms", "silu", "rgpsn", "both")


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype,shape,parts", [
    ("fp32", (7, 48), "rgpsn"), ("fp32", (5, 5), "rpsn"), ("bf16", (4999, 136), "rgpsn"), ("fp16", (3, 100), "gp"),
    ("fp32", (3001, 96), "gpsn"), ("bf16", (5001, 97), "rpsn"), ("fp16", (2049, 1024), "rpsn"),
])
def test_norm_gradients_without_an_epsilon(dtype, shape, parts, kind):
    """CTAs that hold more rows than there are: what stands in for the missing ones adds nothing to the column sums."""
    args, dh, dn = norms.inputs(dtype, shape, parts, seed=2)
    got = dw.dwconv_block_norm_bwd(dh, dn, *args, kind=kind, gate_act="silu", eps=0.0)
    leaves = [ref.leaf(a) for a in args]
    outs = ref.block_norm(*leaves, kind, "silu", 0.0)
    pairs = [(o, ref.wide(d)) for o, d in zip(outs, (dh, dn)) if o is not None and d is not None]
    want = iter(torch.autograd.grad([o for o, _ in pairs], [x for x in leaves if x is not None], [d for _, d in pairs]))
    want = [None if x is None else next(want) for x in leaves]
    size = sum(d.abs().amax(-1, keepdim=True) for _, d in pairs) * (1 + max(
        a.abs().max().item() for a in args if a is not None))
    for name, a, r in zip(("dy", "dresidual", "dgate"), got[:3], want[:3]):
        if a is not None:
            ref.assert_near(a, r, name, dtype, 2e-5, r.abs().amax(-1, keepdim=True) + 0.1 * size)
    for name, a, r in zip(("dw_post", "dscale", "dw_pre"), got[3:], want[3:]):
        if a is not None:
            ref.assert_near(a, r, name, "fp32", 1e-5, torch.full_like(r, shape[0] ** 0.5 * size.max().item()))


def resets(g, at, value):
    g = g.clone()
    for t in at:
        if t < g.shape[1]:
            g[:, t, ::2] = value
    return g


@pytest.mark.parametrize("value", ["-inf", "lowest"])
@pytest.mark.parametrize("dtype,gates", [("bf16", "bf16"), ("fp16", "fp16"), ("fp16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("T", [8, 150])
def test_gates_that_reset_a_state(T, dtype, gates, value):
    """A log decay of minus infinity, or the lowest value of its type, forgets everything and nothing else: two in a
    row, at both ends of a chunk, within one.  Sequences, their gradients and single tokens."""
    gt = ref.TYPES[gates]
    (q, k, v, g, b), state = delta.inputs(dtype, 2, T, 1, 2, 64, 32, gates=gt, seed=11)
    g = resets(g, (0, 3, 4, 63, 64, 90, 127, 149), float("-inf") if value == "-inf" else torch.finfo(gt).min)
    args = [q, k, v, g, b]
    leaves = [ref.leaf(a) for a in (*args, state)]
    ro, rs = ref.delta(*leaves[:5], None, True, leaves[5], None)
    o, after = dw.dwconv_delta_fwd(*args, qk_norm=True, state=state, return_state=True)
    ref.assert_close_in_norm(o, ro, "o", delta.REL[dtype])
    ref.assert_close_in_norm(after, rs, "state", 2e-5)
    pool = state.clone()
    steps = torch.stack([dw.dwconv_delta_step(*(a[:, t] for a in args), pool, qk_norm=True) for t in range(T)], 1)
    ref.assert_close_in_norm(steps, ro, "single tokens", delta.REL[dtype])
    ref.assert_close_in_norm(pool, rs, "state after single tokens", 2e-5)
    do = torch.randn(v.shape, generator=torch.Generator().manual_seed(12)).to(v.dtype).cuda()
    got = dw.dwconv_delta_bwd(do, *args, qk_norm=True, state=state, need_dstate=True)
    want = torch.autograd.grad((ro * ref.wide(do)).sum(), leaves)
    for name, a, r in zip((*delta_bwd.NAMES, "dstate"), got, want):
        ref.assert_close_in_norm(a, r, name, delta_bwd.REL[dtype])
    assert not got[3][g < -1e4].any()  # nothing depends on how far below


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("what", ["v", "k", "q", "g", "beta"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("t", [0, 5, 17, 63, 64, 100])
def test_values_that_are_no_numbers_leave_earlier_tokens_alone(dtype, what, bad, t):
    """What one token's NaN or infinity does to the outputs is the rule's own: nothing before it, and of v's columns
    only its own; the state and every later output of what it reaches is not finite."""
    args, state = delta.inputs(dtype, 1, 150, 1, 2, 64, 48, seed=13, norm=False)
    names = ("q", "k", "v", "g", "beta")
    want, clean = dw.dwconv_delta_fwd(*args, qk_norm=False, state=state, return_state=True)
    dirty = [a.clone() for a in args]
    hit = dirty[names.index(what)]
    if hit.dim() == 4:
        hit[0, t, 0, 3] = bad
    else:
        hit[0, t, 0] = bad
    o, after = dw.dwconv_delta_fwd(*dirty, qk_norm=False, state=state, return_state=True)
    # A column's power of two is chosen from what a whole chunk adds to it: other splits of the same values.
    ref.assert_close_in_norm(o[:, :t], ref.wide(want[:, :t]), "earlier tokens", delta.REL[dtype])
    reached = torch.zeros_like(want, dtype=torch.bool)
    if what == "v":
        reached[0, t:, 0, 3] = True
    elif what == "q":
        reached[0, t] = True  # both value heads read the query
    elif what == "k":
        reached[0, t:] = True
    else:
        reached[0, t:, 0] = True
    if what in "vq":
        apart = ~reached
        if what == "v":
            apart[0, :, 0, 3] = False
        assert torch.equal(o[apart], want[apart])
    elif what != "k":
        assert torch.equal(o[:, :, 1], want[:, :, 1])
    assert not torch.isfinite(o[reached]).any()
    lost = torch.zeros_like(after, dtype=torch.bool)
    if what == "v":
        lost[0, 0, :, 3] = True
    elif what == "k":
        lost[:] = True
    elif what != "q":
        lost[0, 0] = True
    assert torch.equal(after[~lost], clean[~lost]) and not torch.isfinite(after[lost]).any()


@pytest.mark.parametrize("dtype,shape,kind", [("bf16", (400, 8200), "rms"), ("fp32", (330, 8192), "layer"),
                                              ("bf16", (320, 16384), "rms"), ("fp16", (310, 10001), "layer")])
def test_norm_gradients_of_the_widest_rows_on_many_rows(dtype, shape, kind):
    norms.test_gradients(dtype, shape, kind, "sigmoid", "rgpsn", "both")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_write_strengths_up_to_two(dtype):
    """beta between 0 and 2 turns a key's direction over instead of overwriting it; the rule still does not grow."""
    args, state = delta.inputs(dtype, 2, 200, 1, 2, 64, 48, seed=17)
    args[4] = args[4] * 2
    args[4][:, 70:90] = 2
    do = torch.randn(args[2].shape, generator=torch.Generator().manual_seed(18)).to(args[2].dtype).cuda()
    o, after = dw.dwconv_delta_fwd(*args, qk_norm=True, state=state, return_state=True)
    got = dw.dwconv_delta_bwd(do, *args, qk_norm=True, state=state, need_dstate=True)
    leaves = [ref.leaf(a) for a in (*args, state)]
    ro, rs = ref.delta(*leaves[:5], None, True, leaves[5], None)
    want = torch.autograd.grad((ro * ref.wide(do)).sum(), leaves)
    ref.assert_close_in_norm(o, ro, "o", delta.REL[dtype])
    ref.assert_close_in_norm(after, rs, "state", 2e-5)
    for name, a, r in zip((*delta_bwd.NAMES, "dstate"), got, want):
        ref.assert_close_in_norm(a, r, name, delta_bwd.REL[dtype])


def test_calls_from_two_host_threads():
    """Each thread with a stream and shapes of its own gets what a single one gets."""
    def work(seed, C, T):
        g = torch.Generator().manual_seed(seed)
        x, y = (torch.randn(2, T, C, generator=g).cuda().requires_grad_() for _ in range(2))
        w, one = torch.randn(4, C, generator=g).cuda(), torch.ones(C).cuda()
        gates = -torch.rand(2, T, 1, generator=g).cuda()

        def run():
            heads = dw.causal_conv(x, w).unflatten(-1, (1, C))
            o = dw.gated_delta_rule(heads, heads, heads, gates, gates.neg(), qk_norm=True)
            h, _ = dw.block_norm(o.flatten(-2), y, w_post=one)
            return [h.detach(), *torch.autograd.grad(h.square().sum(), (x, y))]
        return run

    runs = [work(1, 64, 200), work(2, 48, 130)]
    want = [run() for run in runs]
    torch.cuda.synchronize()
    off, failed = [], []

    def thread(run, expected):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(30):
                    got = run()
                    torch.cuda.current_stream().synchronize()
                    off.extend(i for i, (a, b) in enumerate(zip(got, expected)) if not torch.equal(a, b))
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=thread, args=a) for a in zip(runs, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and not off


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T", [1, 2, 70])
def test_an_empty_past_does_not_depend_on_the_first_decay(T, dtype):
    """Without a state the first token's decay acts on zeros: its gradient is zero, whatever follows."""
    args, _ = delta.inputs(dtype, 2, T, 1, 2, 64, 48, seed=19)
    g = torch.Generator().manual_seed(20)
    do, last = torch.randn(args[2].shape, generator=g).to(args[2].dtype).cuda(), torch.randn(2, 2, 64, 48, generator=g).cuda()
    got = dw.dwconv_delta_bwd(do, *args, qk_norm=True, dstate_out=last)
    assert not got[3][:, 0].any() and (T == 1 or got[3][:, 1:].any())
    leaves = [ref.leaf(a) for a in args]
    ro, rs = ref.delta(*leaves, None, True, None, None)
    want = torch.autograd.grad((ro * ref.wide(do)).sum() + (rs * ref.wide(last)).sum(), leaves)
    for name, a, r in zip(delta_bwd.NAMES, got, want):
        ref.assert_close_in_norm(a, r, name, delta_bwd.REL[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("what", ["v", "k", "g", "beta"])
def test_what_is_no_number_behind_strong_decays(dtype, what, bad):
    """The same behind decays that leave nothing, where the inverse of one overflows."""
    args, state = delta.inputs(dtype, 1, 60, 1, 2, 64, 48, seed=23, norm=False)
    args[3][:, 2::7] = -90
    args[3][:, 5::11] = float("-inf")
    want = dw.dwconv_delta_fwd(*args, state=state)
    hit = args[("q", "k", "v", "g", "beta").index(what)]
    for t in (41, 24, 9):
        dirty = hit.clone()
        dirty[(0, t, 0, 3)[:hit.dim()]] = bad
        o, after = dw.dwconv_delta_fwd(*(dirty if a is hit else a for a in args), state=state, return_state=True)
        ref.assert_close_in_norm(o[:, :t], ref.wide(want[:, :t]), "earlier tokens", delta.REL[dtype])
        assert not torch.isfinite(o[0, t:, 0, 3]).any() and not torch.isfinite(after[0, 0, :, 3]).any()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("what", ["v", "k", "q", "g", "beta", "do", "last"])
@pytest.mark.parametrize("t", [0, 5, 63, 100])
def test_gradients_that_are_lost_are_not_made_up(dtype, what, t):
    """Wherever the definition's gradient is no number because an input is none, the kernels' is none."""
    args, state = delta.inputs(dtype, 1, 150, 1, 2, 64, 48, seed=21, norm=False)
    g = torch.Generator().manual_seed(22)
    do, last = torch.randn(args[2].shape, generator=g).to(args[2].dtype).cuda(), torch.randn(1, 2, 64, 48, generator=g).cuda()
    hit = dict(zip(("q", "k", "v", "g", "beta", "do", "last"), (*args, do, last)))[what]
    hit[(0, t, 0, 3)[:hit.dim()] if what != "last" else (0, 0, 7, 3)] = float("nan")
    for past in (state, None):
        leaves = [ref.leaf(a) for a in args] + ([] if past is None else [ref.leaf(past)])
        ro, rs = ref.delta(*leaves[:5], None, False, None if past is None else leaves[5], None)
        want = torch.autograd.grad((ro * ref.wide(do)).sum() + (rs * ref.wide(last)).sum(), leaves)
        saved = torch.empty(dw.dwconv_delta_saved_size(1, 150, 1, 2, 64, 48, args[0].dtype), dtype=torch.uint8, device="cuda")
        dw.dwconv_delta_fwd(*args, state=past, saved=saved)
        for s in (saved, None):
            got = dw.dwconv_delta_bwd(do, *args, state=past, dstate_out=last, need_dstate=past is not None, saved=s)
            for name, a, r in zip((*delta_bwd.NAMES, "dstate"), got, want):
                made_up = torch.isfinite(ref.wide(a)) & ~torch.isfinite(r)
                assert not made_up.any(), f"{name}: {int(made_up.sum())} of {r.numel()}, first {made_up.nonzero()[0].tolist()}"
