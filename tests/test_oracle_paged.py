"""Pins of the oracle's paged cache and of its attention gradient (CPU)."""
import math

import numpy as np
import pytest

import oracle
import synth


def _paged(**kw):
    pg = dict(n_seqs=2, n_heads=4, n_kv_heads=2, head_dim=8, page_size=8, n_pages=9, max_pages=4,
              rope_mode=1, rope_split=(4, 2, 2), rope_base=10000.0, grid_h=2, grid_w=3, n_sink=0,
              window=0)
    return {**pg, **kw}


@pytest.mark.parametrize("mode", [0, 1, 3])
def test_append_places_and_turns_rows(mode):
    """Rows appear at (page, offset) of their token, turned as complex numbers."""
    pg = _paged(rope_mode=mode)
    g = np.random.default_rng(1)
    k, v, q = (g.standard_normal((5, h, 8)) for h in (2, 2, 4))
    kp, vp = g.standard_normal((9, 2, 8, 8)), g.standard_normal((9, 2, 8, 8))
    table, lens, cu = [[3, 1, -1, -1], [0, 8, 4, 2]], [10, 19], [0, 3, 5]
    k2, v2, qr = oracle.paged_append(pg, k, v, kp, vp, table, lens, cu, q, np.zeros_like(q))
    where = [(3, 7, 7), (1, 0, 8), (1, 1, 9), (4, 1, 17), (4, 2, 18)]    # page, row, token
    untouched = np.ones((9, 8), bool)
    for i, (page, row, tok) in enumerate(where):
        untouched[page, row] = False
        split = (8, 0, 0) if mode == 1 else (4, 2, 2)
        pos = (tok, 0, 0) if mode == 1 else (tok // 6, tok % 6 // 3, tok % 3)
        z = np.concatenate([np.exp(1j * pos[a] * 10000.0 ** (-2.0 * np.arange(split[a] // 2)
                                                              / split[a]))
                            for a in range(3) if split[a]])
        if mode == 0:
            z = np.ones(4)
        for got, raw in ((k2[page, :, row], k[i]), (qr[i], q[i])):
            want = (raw[:, 0::2] + 1j * raw[:, 1::2]) * z
            assert np.allclose(got[:, 0::2] + 1j * got[:, 1::2], want, atol=1e-13)
        assert np.array_equal(v2[page, :, row], v[i])
    keep = untouched[:, None, :].repeat(2, 1)
    assert np.array_equal(k2[keep], kp[keep]) and np.array_equal(v2[keep], vp[keep])


def test_paged_attention_is_softmax_over_the_attended_tokens():
    pg = _paged(n_sink=3, window=9)
    g = np.random.default_rng(2)
    q = g.standard_normal((2, 4, 8))
    kp, vp = g.standard_normal((9, 2, 8, 8)), g.standard_normal((9, 2, 8, 8))
    table, lens = [[3, 1, 5, -1], [0, 8, 4, 2]], [20, 0]
    out, lse, avg = oracle.paged_attention(pg, q, kp, vp, table, lens)
    toks = [t for t in range(20) if t < 3 or t >= 11]
    for h in range(4):
        w, num, ab = 0.0, np.zeros(8), np.zeros(8)
        for t in toks:
            page, row = table[0][t // 8], t % 8
            e = math.exp(sum(q[0, h] * kp[page, h // 2, row]) / math.sqrt(8))
            w, num, ab = w + e, num + e * vp[page, h // 2, row], ab + e * abs(vp[page, h // 2, row])
        assert np.allclose(out[0, h], num / w, atol=1e-12) and abs(lse[0, h] - math.log(w)) < 1e-12
        assert np.allclose(avg[0, h], ab / w, atol=1e-12)
    assert not out[1].any() and np.all(lse[1] == -np.inf)


SMALL = dict(n_heads=2, head_dim=8, grid_h=2, grid_w=2, frames_per_block=2, ref_frames=1,
             ring_slots=2, rope_mode=3, rope_split=(4, 2, 2), rope_base=100.0, block_index=3,
             valid_mask=0xFF)


@pytest.mark.parametrize("kw", [{}, dict(rope_mode=1), dict(valid_mask=0b10001),
                                dict(valid_mask=0)])
def test_attention_gradient_matches_differences(kw):
    """Central differences of <d_out, attention(q, k, v)>, element by element."""
    cfg = {**SMALL, **kw}
    s = oracle.layout_sizes(cfg)
    g = np.random.default_rng(3)
    q, do = (g.standard_normal((s["L_blk"], 2, 8)) for _ in range(2))
    k, v = (g.standard_normal((2, s["T"], 8)) for _ in range(2))
    grads = oracle.attention_backward(cfg, q, k, v, do)

    def loss(*x):
        return float((oracle.attention(cfg, *x)[0] * do).sum())
    eps = 1e-5
    for which, grad in enumerate(grads):
        for at in [tuple(g.integers(0, n) for n in grad.shape) for _ in range(25)]:
            hi, lo = ([x.copy() for x in (q, k, v)] for _ in range(2))
            hi[which][at] += eps
            lo[which][at] -= eps
            assert abs((loss(*hi) - loss(*lo)) / (2 * eps) - grad[at]) < 1e-8


def test_gradient_bound_covers_planted_roundings():
    """The bound holds for the gradient computed with every intermediate rounded to bf16, and so
    does the 2-norm bound of the GPU tests: the mean square of a bf16 rounding's relative error is
    (1.7e-3)^2, the score carries two (rms 1 for these inputs), dS, its other factor and the
    result one each, delta one on a smaller term: sqrt(5.x) * 1.7e-3 = 4e-3 < 5e-3.  Leaving delta
    out exceeds it."""
    cfg = synth.preset("tiny", block_index=7, valid_mask=0xFF)
    s = oracle.layout_sizes(cfg)
    import torch
    q, do = (synth.normal_bf16((s["L_blk"], 1, 64), 5, i).double().numpy() for i in (0, 3))
    k, v = (synth.normal_bf16((1, s["T"], 64), 5, i).double().numpy() for i in (1, 2))
    bf = lambda x: torch.from_numpy(np.ascontiguousarray(x)).bfloat16().double().numpy()  # noqa: E731
    exact = oracle.attention_backward(cfg, q, k, v, do)
    bound = oracle.backward_bound(cfg, q, k, v, do)
    kpos, valid = oracle.key_positions(cfg)
    qpos = oracle.query_positions(cfg)
    out, lse = oracle.attention(cfg, q, k, v)
    qr, kr = bf(oracle.rope_rotate(cfg, q[:, 0], qpos)), bf(oracle.rope_rotate(cfg, k[0], kpos))
    p = np.exp(qr @ kr.T / 8 - lse[0][:, None])
    ds = bf(p * (do[:, 0] @ v[0].T - (do[:, 0] * bf(out[:, 0])).sum(1, keepdims=True)) / 8)
    back = lambda x, pos: oracle.rope_rotate(cfg, x, -pos)  # noqa: E731
    no_delta = back(bf(p * (do[:, 0] @ v[0].T) / 8) @ kr, qpos)
    assert np.linalg.norm(no_delta - exact[0][:, 0]) > 5e-3 * np.linalg.norm(exact[0])
    got = (bf(back(ds @ kr, qpos)), bf(back(ds.T @ qr, kpos)), bf(bf(p).T @ do[:, 0]))
    for x, e, b in zip(got, (exact[0][:, 0], exact[1][0], exact[2][0]),
                       (bound[0][:, 0], bound[1][0], bound[2][0])):
        assert np.all(np.abs(x - e) <= b)
        assert np.linalg.norm(x - e) / np.linalg.norm(e) < 5e-3
