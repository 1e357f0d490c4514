"""Refusals of the paged-cache calls and of the attention's backward pass on the host: invalid
arguments are rejected before anything is launched (CPU only)."""
import ctypes

import pytest
import torch

import pose_retrieved_kv_b200 as P
import synth

GOOD = dict(n_seqs=2, n_heads=4, n_kv_heads=2, head_dim=64, page_size=16, n_pages=8, max_pages=4)


def _append(pg, **kw):
    a = dict(k=16, v=16, ks=128, vs=128, kp=16, vp=16, table=16, lens=16, n=2, cu=None, q=None,
             qs=0, qr=None)
    a.update(kw)
    return P._lib._lib.prsink_paged_append(
        ctypes.byref(pg) if pg else None, a["k"], a["v"], a["ks"], a["vs"], a["kp"], a["vp"],
        a["table"], a["lens"], a["n"], a["cu"], a["q"], a["qs"], a["qr"], None)


def _attend(pg, **kw):
    a = dict(q=16, kp=16, vp=16, table=16, lens=16, out=16, lse=None, scratch=256, nb=1 << 30)
    a.update(kw)
    return P._lib._lib.prsink_paged_attention(
        ctypes.byref(pg) if pg else None, a["q"], a["kp"], a["vp"], a["table"], a["lens"],
        a["out"], a["lse"], a["scratch"], a["nb"], None)


@pytest.mark.parametrize("bad", [
    dict(n_seqs=-1), dict(n_seqs=65536), dict(n_heads=0), dict(n_kv_heads=0), dict(n_heads=5),
    dict(page_size=0), dict(n_pages=0), dict(max_pages=0), dict(n_sink=-1), dict(window=-1),
    dict(rope_mode=2), dict(rope_base=0.0), dict(rope_base=float("nan")),
    dict(max_pages=1 << 27), dict(n_pages=1 << 30), dict(n_seqs=65535, n_heads=65534),
    dict(rope_mode=3, rope_split=(24, 20, 18), grid_h=4, grid_w=4),
    dict(rope_mode=3, rope_split=(23, 21, 20), grid_h=4, grid_w=4),
    dict(rope_mode=3, rope_split=(24, 20, 20), grid_h=0, grid_w=4)])
def test_invalid_paged_description(bad):
    pg = P.make_paged(**{**GOOD, **bad})
    before = P.prsink_launch_count()
    assert _append(pg) == P.PRSINK_ERR_ARG
    assert _attend(pg) == P.PRSINK_ERR_ARG
    assert P._lib._lib.prsink_paged_attention_scratch_bytes(ctypes.byref(pg)) == -1
    with pytest.raises(P.PRSinkError):
        P.prsink_paged_attention_scratch_bytes(pg)
    assert P.prsink_launch_count() == before


@pytest.mark.parametrize("bad", [dict(head_dim=96), dict(head_dim=256), dict(page_size=12),
                                 dict(page_size=4), dict(page_size=1)])
def test_unsupported_paged_description(bad):
    pg = P.make_paged(**{**GOOD, **bad})
    assert _append(pg, ks=1024, vs=1024) == P.PRSINK_ERR_UNSUPPORTED
    assert _attend(pg) == P.PRSINK_ERR_UNSUPPORTED


def test_paged_pointers_strides_and_counts():
    pg = P.make_paged(**GOOD)
    before = P.prsink_launch_count()
    assert _append(None) == _attend(None) == P.PRSINK_ERR_ARG
    for name in ("k", "v", "kp", "vp", "table", "lens"):
        assert _append(pg, **{name: None}) == P.PRSINK_ERR_ARG
    for name in ("k", "v", "kp", "vp"):
        assert _append(pg, **{name: 8}) == P.PRSINK_ERR_ALIGN
    for name in ("table", "lens", "cu"):
        assert _append(pg, **{name: 18}) == P.PRSINK_ERR_ALIGN
    assert _append(pg, q=16, qs=256) == P.PRSINK_ERR_ARG              # q without q_rot
    assert _append(pg, qr=16) == P.PRSINK_ERR_ARG
    assert _append(pg, q=24, qs=256, qr=32) == P.PRSINK_ERR_ALIGN
    for kw in (dict(ks=127), dict(ks=132), dict(vs=120), dict(ks=-128),
               dict(q=16, qs=255, qr=32), dict(q=16, qs=248, qr=32),
               dict(q=16, qs=264, qr=16)):                            # in place, not contiguous
        assert _append(pg, **kw) == P.PRSINK_ERR_ARG, kw
    assert _append(pg, n=3) == P.PRSINK_ERR_ARG                       # without cu_new: n_seqs
    assert _append(pg, n=-1, cu=16) == P.PRSINK_ERR_ARG
    assert _append(pg, n=0, cu=16) == P.PRSINK_OK                     # nothing to do
    for name in ("q", "kp", "vp", "table", "lens", "out"):
        assert _attend(pg, **{name: None}) == P.PRSINK_ERR_ARG
    for name in ("q", "kp", "vp", "out"):
        assert _attend(pg, **{name: 8}) == P.PRSINK_ERR_ALIGN
    for name in ("table", "lens", "lse"):
        assert _attend(pg, **{name: 18}) == P.PRSINK_ERR_ALIGN
    empty = P.make_paged(**{**GOOD, "n_seqs": 0})
    assert _attend(pg, scratch=None) == _attend(pg, scratch=128) == P.PRSINK_ERR_ARG
    assert _attend(pg, nb=P.prsink_paged_attention_scratch_bytes(pg) - 1) == P.PRSINK_ERR_ARG
    assert _attend(empty) == P.PRSINK_OK and _append(empty, n=0) == P.PRSINK_OK
    assert P.prsink_launch_count() == before


def test_paged_binding_checks_shapes_and_types():
    pg = P.make_paged(**GOOD)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)      # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)        # noqa: E731
    pool = bf(8, 2, 16, 64)
    with pytest.raises(ValueError, match="k_new"):
        P.prsink_paged_append(pg, bf(2, 3, 64), bf(2, 2, 64), pool, pool, i32(2, 4), i32(2))
    with pytest.raises(TypeError, match="k_new"):
        P.prsink_paged_append(pg, bf(2, 2, 64).float(), bf(2, 2, 64), pool, pool, i32(2, 4),
                              i32(2))
    with pytest.raises(ValueError, match="contiguous"):
        P.prsink_paged_append(pg, bf(2, 64, 2).transpose(1, 2), bf(2, 2, 64), pool, pool,
                              i32(2, 4), i32(2))
    with pytest.raises(ValueError, match="CUDA"):
        P.prsink_paged_append(pg, bf(2, 2, 64), bf(2, 2, 64), pool, pool, i32(2, 4), i32(2))
    with pytest.raises(ValueError, match="k_pages"):
        P.prsink_paged_attention(pg, None, bf(7, 2, 16, 64), pool, i32(2, 4), i32(2), None, None)
    with pytest.raises(ValueError, match="q must hold"):
        P.prsink_paged_attention(pg, bf(2, 2, 64), pool, pool, i32(2, 4), i32(2), None, None)


def test_backward_refusals():
    lib = P._lib._lib
    lay = P.make_layout(**synth.preset("tiny"))
    nb = P.prsink_attention_backward_scratch_bytes(lay)
    assert nb >= 256 * 64 * 2 + 48 * 64 * 2
    before = P.prsink_launch_count()

    def call(layout=lay, scratch=256, n=nb, mask=0xFF, dyn=None, **kw):
        names = ("q", "k", "v", "out", "lse", "d_out", "dq", "dk", "dv")
        a = [kw.get(x, 16 * (i + 1)) for i, x in enumerate(names)]
        return lib.prsink_attention_backward(ctypes.byref(layout), *a, mask, dyn, scratch, n, None)
    for name in ("q", "k", "v", "out", "lse", "d_out", "dq", "dk", "dv"):
        assert call(**{name: None}) == P.PRSINK_ERR_ARG, name
    for name in ("q", "k", "v", "out", "d_out", "dq", "dk", "dv"):
        assert call(**{name: 24}) == P.PRSINK_ERR_ALIGN, name
    for name, other in (("dq", 16), ("dk", 32), ("dv", 48), ("dq", 96), ("dk", 112), ("dv", 128)):
        assert call(**{name: other}) == P.PRSINK_ERR_ARG, name        # in another's place
    assert call(lse=18) == P.PRSINK_ERR_ALIGN and call(dyn=12) == P.PRSINK_ERR_ALIGN
    assert call(scratch=None) == P.PRSINK_ERR_ARG and call(scratch=128) == P.PRSINK_ERR_ARG
    assert call(n=nb - 1) == P.PRSINK_ERR_ARG
    for bad in (dict(n_heads=0), dict(ring_slots=9), dict(block_index=-1)):
        lay2 = P.make_layout(**{**synth.preset("tiny"), **bad})
        assert call(layout=lay2) == P.PRSINK_ERR_ARG
        with pytest.raises(P.PRSinkError):
            P.prsink_attention_backward_scratch_bytes(lay2)
    lay96 = P.make_layout(**{**synth.preset("tiny"), "head_dim": 96, "rope_split": (96, 0, 0)})
    assert call(layout=lay96) == P.PRSINK_ERR_UNSUPPORTED
    long = P.make_layout(**{**synth.preset("tiny"), "grid_h": 100, "grid_w": 100})   # 160000 keys
    assert call(layout=long) == P.PRSINK_ERR_UNSUPPORTED
    assert P.prsink_launch_count() == before
