"""GPU parity of the attention's backward pass against the float64 oracle.

Every element is held to the bound that the roundings allow (``oracle.backward_bound``), and every
gradient of N(0, 1) inputs to 5e-3 in the 2-norm (independent bf16 roundings of the rotated q and
k, the probabilities, dS and the result: sqrt(5.x) * 1.7e-3 = 4e-3)."""
import numpy as np
import pytest
import torch

import oracle
import pose_retrieved_kv_b200 as P
import synth
from tests._gpu import attention_inputs, f64, need_gpu

pytestmark = pytest.mark.gpu


def case(name="tiny", **kw):
    base = dict(n_heads=2, head_dim=64, grid_h=5, grid_w=7, frames_per_block=3, ref_frames=1,
                ring_slots=3, rope_mode=3, rope_split=(24, 20, 20), rope_base=10000.0,
                block_index=7, valid_mask=0xFF)
    if name == "tiny":
        base = synth.preset("tiny", block_index=7, valid_mask=0xFF)
    base.update(kw)
    if base["head_dim"] == 128 and sum(base["rope_split"]) != 128:
        base["rope_split"] = (44, 42, 42)
    return base


CASES = [
    case(), case(valid_mask=0b001011, block_index=0), case(ring_slots=1),
    case("grid"), case("grid", head_dim=128, n_heads=1),
    case("grid", ref_frames=0, frames_per_block=1, grid_h=1, grid_w=1, ring_slots=2),
    case("grid", grid_h=8, grid_w=16, frames_per_block=1, ring_slots=2),       # whole tiles
    case("grid", grid_h=11, grid_w=12, frames_per_block=1, head_dim=128, ring_slots=2),
    case("grid", valid_mask=0b101010, block_index=8, head_dim=128),
    case("grid", head_dim=128, rope_split=(64, 32, 32)),
    case("grid", head_dim=128, rope_split=(0, 64, 64), n_heads=3, ref_frames=2),
    case("grid", n_heads=24, grid_h=12, grid_w=12),        # several heads per preparing CTA
]


def inputs(cfg, seed, gain=1.0):
    q, k, v = attention_inputs(cfg, seed)
    if gain != 1.0:
        q = (q.float() * gain).bfloat16()
    s = oracle.layout_sizes(cfg)
    do = synth.normal_bf16((s["L_blk"], cfg["n_heads"], cfg["head_dim"]), seed, 3)
    return q, k, v, do


def forward(cfg, q, k, v):
    """The forward's results as the oracle gives them, rounded to what the library stores."""
    out, lse = oracle.attention(cfg, f64(q), f64(k), f64(v))
    return torch.from_numpy(out).bfloat16(), torch.from_numpy(lse).float()


def backward(cfg, q, k, v, do, out, lse, fill=float("nan"), **kw):
    lay = P.make_layout(**cfg)
    scratch = torch.full((P.prsink_attention_backward_scratch_bytes(lay),), 255,
                         dtype=torch.uint8, device="cuda")
    q, k, v, do, out, lse = (x.cuda() for x in (q, k, v, do, out, lse))
    dq = torch.full_like(q, float("nan"))
    dk, dv = torch.full_like(k, fill), torch.full_like(v, fill)
    P.prsink_attention_backward(lay, q, k, v, out, lse, do, dq, dk, dv, scratch, **kw)
    return dq, dk, dv


def check(cfg, got, q, k, v, do, norm=5e-3):
    x = [f64(t) for t in (q, k, v, do)]
    ref, bound = oracle.attention_backward(cfg, *x), oracle.backward_bound(cfg, *x)
    for name, g, r, b in zip(("dq", "dk", "dv"), got, ref, bound):
        g = f64(g)
        assert np.all(np.isfinite(g)), name
        bad = np.abs(g - r) - b
        assert np.all(bad <= 0), f"{name}: excess {bad.max():.3e}"
        if norm and np.linalg.norm(r) > 0:
            assert np.linalg.norm(g - r) <= norm * np.linalg.norm(r), \
                (name, np.linalg.norm(g - r) / np.linalg.norm(r))


@pytest.mark.parametrize("i", range(len(CASES)))
def test_gradient_matches_the_oracle(i):
    need_gpu()
    cfg = CASES[i]
    q, k, v, do = inputs(cfg, 40 + i)
    out, lse = forward(cfg, q, k, v)
    got = backward(cfg, q, k, v, do, out, lse)
    assert P.prsink_sync_status() == P.PRSINK_OK
    single = cfg["grid_h"] * cfg["grid_w"] == 1     # few keys: the mean roundings do not apply
    check(cfg, got, q, k, v, do, norm=None if single else 5e-3)
    again = backward(cfg, q, k, v, do, out, lse)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("gain", [0.0, 4.0])
def test_flat_and_peaked_scores(gain):
    need_gpu()
    cfg = case("grid", head_dim=128)
    q, k, v, do = inputs(cfg, 60, gain)
    got = backward(cfg, q, k, v, do, *forward(cfg, q, k, v))
    check(cfg, got, q, k, v, do, norm=None)


@pytest.mark.parametrize("d", [64, 128])
def test_empty_slots_hold_anything(d):
    """NaN and infinities in the slots without data reach no gradient; their rows get zeros."""
    need_gpu()
    cfg = case("grid", head_dim=d, valid_mask=0b011011, block_index=1)
    q, k, v, do = inputs(cfg, 61)
    out, lse = forward(cfg, q, k, v)
    for s, (a, e) in enumerate(oracle.slot_ranges(cfg)):
        if not (cfg["valid_mask"] >> s) & 1:
            k[:, a:e], v[:, a:e] = float("nan"), float("inf")
    got = backward(cfg, q, k, v, do, out, lse)
    for a, e in [oracle.slot_ranges(cfg)[s] for s in (2, 5)]:
        assert not got[1][:, a:e].any() and not got[2][:, a:e].any()
        k[:, a:e], v[:, a:e] = 0, 0
    check(cfg, got, q, k, v, do)


def test_dynamic_slot_emptied_on_the_device_and_no_keys_at_all():
    need_gpu()
    cfg = case("grid")
    q, k, v, do = inputs(cfg, 62)
    off = dict(cfg, valid_mask=0xFF & ~4)
    out, lse = forward(off, q, k, v)
    dyn = torch.tensor([-1], dtype=torch.int64, device="cuda")
    check(off, backward(cfg, q, k, v, do, out, lse, dyn_src=dyn), q, k, v, do)
    out, lse = forward(cfg, q, k, v)
    dyn.fill_(3)
    check(cfg, backward(cfg, q, k, v, do, out, lse, dyn_src=dyn), q, k, v, do)
    none = dict(cfg, valid_mask=0)
    out, lse = forward(none, q, k, v)
    assert torch.all(lse == -float("inf"))
    assert not any(g.any() for g in backward(none, q, k, v, do, out, lse))


@pytest.mark.parametrize("mask", [0, 1, 1 << 4, 0b101100])
def test_grad_mask_selects_slots_and_leaves_the_rest(mask):
    need_gpu()
    cfg = case("grid", head_dim=128)
    q, k, v, do = inputs(cfg, 63)
    out, lse = forward(cfg, q, k, v)
    full = backward(cfg, q, k, v, do, out, lse)
    part = backward(cfg, q, k, v, do, out, lse, fill=7.0, grad_mask=mask)
    assert torch.equal(full[0], part[0])
    for s, (a, e) in enumerate(oracle.slot_ranges(cfg)):
        for f, g in zip(full[1:], part[1:]):
            if (mask >> s) & 1:
                assert torch.equal(f[:, a:e], g[:, a:e]), s
            else:
                assert torch.all(g[:, a:e] == 7.0), s
    if mask == 0:                                    # the buffers may then be left out
        lay = P.make_layout(**cfg)
        scratch = torch.empty(P.prsink_attention_backward_scratch_bytes(lay), dtype=torch.uint8,
                              device="cuda")
        dq = torch.empty_like(full[0])
        P.prsink_attention_backward(lay, q.cuda(), k.cuda(), v.cuda(), out.cuda(), lse.cuda(),
                                    do.cuda(), dq, None, None, scratch, grad_mask=0)
        assert torch.equal(dq, full[0])


@pytest.mark.parametrize("name,heads", [("tiny", 1), ("480x480", 1), ("384x672_r4", 1)])
def test_after_the_library_s_forward(name, heads):
    """Forward and backward through the library, at the workload's layouts: sampled directional
    derivatives <dq, a> + <dk, b> + <dv, c> against the float64 oracle's gradient."""
    need_gpu()
    cfg = synth.preset(name, block_index=1000, valid_mask=0xFF, n_heads=heads)
    q, k, v, do = inputs(cfg, 64)
    lay = P.make_layout(**cfg)
    s = oracle.layout_sizes(cfg)
    out = torch.empty_like(q, device="cuda")
    lse = torch.empty((heads, s["L_blk"]), device="cuda")
    P.prsink_attention(lay, q.cuda(), k.cuda(), v.cuda(), out, lse)
    got = backward(cfg, q, k, v, do, out.cpu(), lse.cpu())
    assert P.prsink_sync_status() == P.PRSINK_OK
    ref = oracle.attention_backward(cfg, *(f64(t) for t in (q, k, v, do)))
    for g, r in zip(got, ref):
        assert np.linalg.norm(f64(g) - r) <= 5e-3 * np.linalg.norm(r)


def test_gradient_against_differences_of_the_library_s_forward():
    """A step along the gradient changes <d_out, out> by what the gradient says: float64 sums of
    the library's own bf16 outputs at q +- h dq, v +- h dv."""
    need_gpu()
    cfg = case("grid", n_heads=4, head_dim=128)
    lay = P.make_layout(**cfg)
    q, k, v, do = (t.cuda() for t in inputs(cfg, 65))
    s = oracle.layout_sizes(cfg)

    def loss(q, k, v):
        out = torch.empty_like(q)
        lse = torch.empty((4, s["L_blk"]), device="cuda")
        P.prsink_attention(lay, q, k, v, out, lse)
        return (out.double() * do.double()).sum().item(), out, lse
    _, out, lse = loss(q, k, v)
    grads = backward(cfg, q.cpu(), k.cpu(), v.cpu(), do.cpu(), out.cpu(), lse.cpu())
    for which in range(3):
        g = grads[which].float()
        x = [q, k, v]
        h = 0.25 * x[which].float().norm() / g.norm()      # a step of a quarter of the input
        hi, lo = list(x), list(x)
        hi[which] = (x[which].float() + h * g).bfloat16()
        lo[which] = (x[which].float() - h * g).bfloat16()
        step = hi[which].double() - lo[which].double()     # what was really taken
        want = (step * g.double()).sum().item()
        diff = loss(*hi)[0] - loss(*lo)[0]
        # v enters linearly; q and k have a third-order term of the step's size
        assert abs(diff - want) <= (0.02 if which == 2 else 0.25) * abs(want), (which, diff, want)


def test_captured_backward_replays_on_another_stream():
    need_gpu()
    cfg = case("grid", head_dim=128)
    q, k, v, do = inputs(cfg, 66)
    out, lse = forward(cfg, q, k, v)
    want = backward(cfg, q, k, v, do, out, lse)
    lay = P.make_layout(**cfg)
    dev = [x.cuda() for x in (q, k, v, out, lse, do)]
    grads = [torch.empty_like(x) for x in want]
    scratch = torch.empty(P.prsink_attention_backward_scratch_bytes(lay), dtype=torch.uint8,
                          device="cuda")
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        P.prsink_attention_backward(lay, *dev, *grads, scratch)
    for _ in range(2):
        for g in grads:
            g.fill_(float("nan"))
        scratch.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(grads, want))


def test_two_calls_at_once_with_their_own_scratch():
    need_gpu()
    cfgs = [case("grid", head_dim=128), case("grid", n_heads=3)]
    data = [inputs(c, 67 + i) for i, c in enumerate(cfgs)]
    fwd = [forward(c, *x[:3]) for c, x in zip(cfgs, data)]
    want = [backward(c, *x, *f) for c, x, f in zip(cfgs, data, fwd)]
    torch.cuda.synchronize()
    got = []
    for c, x, f in zip(cfgs, data, fwd):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            got.append(backward(c, *x, *f))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_normal():
    need_gpu()
    cfg = case("grid", head_dim=128)
    q, k, v, do = inputs(cfg, 69)
    out, lse = forward(cfg, q, k, v)
    want = backward(cfg, q, k, v, do, out, lse)
    assert P.prsink_sync_status() == P.PRSINK_OK
    P.prsink_debug_attention_stall(200_000)
    got = backward(cfg, q, k, v, do, out, lse)
    assert P.prsink_sync_status() == P.PRSINK_ERR_TIMEOUT
    assert not any(g.any() for g in got)
    again = backward(cfg, q, k, v, do, out, lse)
    assert P.prsink_sync_status() == P.PRSINK_OK
    assert all(torch.equal(a, b) for a, b in zip(want, again))
