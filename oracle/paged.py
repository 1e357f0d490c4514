"""Plain float64 definitions of the paged-cache calls and of the attention's gradient.

TEST INFRASTRUCTURE ONLY, like ``prsink_oracle``; no code is shared with the CUDA library.
A paged cache is a dict of the fields of ``prsink_paged``.
"""
from __future__ import annotations

import math

import numpy as np

from .prsink_oracle import (key_positions, layout_sizes, query_positions, rope_angles,
                            rope_rotate)

__all__ = ["paged_positions", "paged_rotate", "paged_append", "paged_attended",
           "paged_attention", "attention_backward", "backward_bound"]


def paged_positions(pg: dict, index) -> np.ndarray:
    """Position of the tokens with these indices in their sequence: the index (1-D), or the
    (frame, row, column) of a grid_h x grid_w latent frame (3-D)."""
    index = np.asarray(index, dtype=np.int64)
    if pg["rope_mode"] != 3:
        return index
    lf = pg["grid_h"] * pg["grid_w"]
    return np.stack([index // lf, index % lf // pg["grid_w"], index % lf % pg["grid_w"]], -1)


def paged_rotate(pg: dict, x, index) -> np.ndarray:
    """Rows x [n][heads][d] rotated at the positions of the tokens ``index`` [n]."""
    x = np.asarray(x, dtype=np.float64)
    if not pg["rope_mode"]:
        return x.copy()
    return rope_rotate(pg, x, paged_positions(pg, index)[:, None])


def paged_append(pg: dict, k_new, v_new, k_pages, v_pages, table, lens, cu=None, q=None,
                 q_rot=None):
    """New pages (and q_rot): row cu[s] + i becomes token lens[s] - (cu[s+1] - cu[s]) + i of
    sequence s.  Tokens without a page, or outside the table, are left out."""
    k_pages, v_pages = np.array(k_pages, np.float64), np.array(v_pages, np.float64)
    q_rot = None if q is None else np.array(q_rot, np.float64)
    cu = list(range(pg["n_seqs"] + 1)) if cu is None else [int(c) for c in cu]
    for s in range(pg["n_seqs"]):
        for i in range(cu[s], cu[s + 1]):
            t = int(lens[s]) - (cu[s + 1] - i)
            if t < 0 or int(lens[s]) > pg["max_pages"] * pg["page_size"]:
                continue
            if q is not None:
                q_rot[i] = paged_rotate(pg, np.asarray(q)[i:i + 1], [t])[0]
            page = int(table[s][t // pg["page_size"]])
            if not 0 <= page < pg["n_pages"]:
                continue
            k_pages[page, :, t % pg["page_size"]] = paged_rotate(pg, k_new[i:i + 1], [t])[0]
            v_pages[page, :, t % pg["page_size"]] = v_new[i]
    return k_pages, v_pages, q_rot


def paged_attended(pg: dict, table_row, length: int) -> list:
    """(page, row) of every attended token of a sequence."""
    cap = pg["max_pages"] * pg["page_size"]
    length = min(max(int(length), 0), cap)
    out = []
    for t in range(length):
        if pg["window"] and not (t < pg["n_sink"] or t >= length - pg["window"]):
            continue
        page = int(table_row[t // pg["page_size"]])
        if 0 <= page < pg["n_pages"]:
            out.append((page, t % pg["page_size"]))
    return out


def paged_attention(pg: dict, q, k_pages, v_pages, table, lens):
    """(out [n_seqs][H][d], lse [n_seqs][H], absolute [n_seqs][H][d]): the last is the softmax
    average of |v|, the scale that a rounding of the probabilities acts on."""
    q = np.asarray(q, np.float64)
    n, h, d = q.shape
    group = h // pg["n_kv_heads"]
    out, avg = np.zeros_like(q), np.zeros_like(q)
    lse = np.full((n, h), -np.inf)
    for s in range(n):
        at = paged_attended(pg, table[s], lens[s])
        if not at:
            continue
        pages, rows = (np.array(x) for x in zip(*at))
        for j in range(h):
            k = np.asarray(k_pages[pages, j // group, rows], np.float64)
            v = np.asarray(v_pages[pages, j // group, rows], np.float64)
            sc = k @ q[s, j] / math.sqrt(d)
            e = np.exp(sc - sc.max())
            lse[s, j] = sc.max() + math.log(e.sum())
            out[s, j] = e @ v / e.sum()
            avg[s, j] = e @ np.abs(v) / e.sum()
    return out, lse, avg


def _head(cfg, q, k, v, d_out, h, qpos, kpos, valid):
    d = cfg["head_dim"]
    qr = rope_rotate(cfg, np.asarray(q[:, h], np.float64), qpos)
    kr = rope_rotate(cfg, np.asarray(k[h][valid], np.float64), kpos[valid])
    vv, do = np.asarray(v[h][valid], np.float64), np.asarray(d_out[:, h], np.float64)
    sc = qr @ kr.T / math.sqrt(d)
    p = np.exp(sc - sc.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    dp = do @ vv.T
    delta = (p * dp).sum(1, keepdims=True)
    return qr, kr, vv, do, p, dp, delta


def _back(cfg, x, pos):
    """The inverse rotation (by the negative angles)."""
    ang = rope_angles(cfg, pos)
    c, s = np.cos(ang), np.sin(ang)
    out = np.empty_like(x)
    out[..., 0::2] = x[..., 0::2] * c + x[..., 1::2] * s
    out[..., 1::2] = -x[..., 0::2] * s + x[..., 1::2] * c
    return out


def attention_backward(cfg: dict, q, k_cache, v_cache, d_out):
    """Gradient of <d_out, attention(q, k, v)> with respect to raw q, k and v: (dq [L_blk][H][d],
    dk, dv [H][T][d]); rows of empty slots are zero."""
    dq = np.zeros(np.shape(q))
    dk, dv = np.zeros(np.shape(k_cache)), np.zeros(np.shape(v_cache))
    kpos, valid = key_positions(cfg)
    qpos = query_positions(cfg)
    if not valid.any():
        return dq, dk, dv
    for h in range(cfg["n_heads"]):
        qr, kr, vv, do, p, dp, delta = _head(cfg, q, k_cache, v_cache, d_out, h, qpos, kpos, valid)
        ds = p * (dp - delta) / math.sqrt(cfg["head_dim"])
        dq[:, h] = _back(cfg, ds @ kr, qpos)
        dk[h, valid] = _back(cfg, ds.T @ qr, kpos[valid])
        dv[h, valid] = p.T @ do
    return dq, dk, dv


def backward_bound(cfg: dict, q, k_cache, v_cache, d_out, u: float = 2.0 ** -8):
    """Bounds of |computed - exact| for dq, dk, dv when the rotated q and k, the probabilities,
    dS, ``out`` (inside delta) and the results are rounded with relative error u, and everything
    else is exact up to a relative 2^-12 (float32 sums of up to 2^12 terms at 2^-24 each).

    delta s <= (2u + u^2) sum_c |q~_c k~_c| / sqrt(d) =: e;  a probability is off by a factor of at
    most exp(e) (its own lse comes from exact scores), and once more by u;
    delta(delta) <= u sum_c |d_out_c out_c|;  each rounding adds u times the value it acts on."""
    d = cfg["head_dim"]
    f = 2.0 ** -12
    bq = np.zeros(np.shape(q))
    bk, bv = np.zeros(np.shape(k_cache)), np.zeros(np.shape(v_cache))
    kpos, valid = key_positions(cfg)
    qpos = query_positions(cfg)
    if not valid.any():
        return bq, bk, bv
    def spread(x):                       # a rotation mixes the two elements of a pair
        pair = x[..., 0::2] + x[..., 1::2]
        return np.repeat(pair, 2, axis=-1)
    for h in range(cfg["n_heads"]):
        qr, kr, vv, do, p, dp, delta = _head(cfg, q, k_cache, v_cache, d_out, h, qpos, kpos, valid)
        e = (2 * u + u * u) * (np.abs(qr) @ np.abs(kr).T) / math.sqrt(d)
        pe = p * (np.exp(e + f) - 1)                      # error of a probability
        o = p @ vv
        ddelta = u * (np.abs(do) * np.abs(o)).sum(1, keepdims=True)
        absdp = np.abs(do) @ np.abs(vv).T
        ds = p * (dp - delta) / math.sqrt(d)
        dse = (pe * np.abs(dp - delta) + (p + pe) * (ddelta + f * (absdp + np.abs(delta)))) \
            / math.sqrt(d)
        dse = dse + u * (np.abs(ds) + dse)                # rounding of dS
        dq = np.abs(_back(cfg, ds @ kr, qpos))
        dk = np.abs(_back(cfg, ds.T @ qr, kpos[valid]))
        full = np.abs(ds) + dse
        bq[:, h] = spread(dse @ np.abs(kr) + (u + f) * (full @ np.abs(kr)))
        bq[:, h] += u * (dq + bq[:, h])
        x = spread(dse.T @ np.abs(qr) + (u + f) * (full.T @ np.abs(qr)))
        bk[h, valid] = x + u * (dk + x)
        x = (pe + (u + f) * (p + pe)).T @ np.abs(do)
        bv[h, valid] = x + u * (np.abs(p.T @ do) + x)
    return bq, bk, bv
