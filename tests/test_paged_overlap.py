"""Buffers that a call writes are its own: overlapping ones are refused on the host (CPU only:
addresses without memory behind them, nothing is launched)."""
import ctypes

import pytest

import pose_retrieved_kv_b200 as P
import synth

GOOD = dict(n_seqs=3, n_heads=4, n_kv_heads=2, head_dim=64, page_size=16, n_pages=8, max_pages=4)
MB = 1 << 20


def _paged():
    return P.make_paged(**GOOD)


def _attend(**kw):
    pg = _paged()
    names = ("q", "kp", "vp", "table", "lens", "out", "lse", "scratch")
    a = {**{x: (i + 1) * MB for i, x in enumerate(names)}, **kw}
    return P._lib._lib.prsink_paged_attention(
        ctypes.byref(pg), *[a[x] for x in names], P.prsink_paged_attention_scratch_bytes(pg), None)


def _append(n=3, ks=128, vs=128, qs=256, **kw):
    pg = _paged()
    names = ("k", "v", "kp", "vp", "table", "lens", "cu", "q", "qr")
    a = {**{x: (i + 1) * MB for i, x in enumerate(names)}, **kw}
    return P._lib._lib.prsink_paged_append(
        ctypes.byref(pg), a["k"], a["v"], ks, vs, a["kp"], a["vp"], a["table"], a["lens"], n,
        a["cu"], a["q"], qs, a["qr"], None)


ROW = 3 * 4 * 64 * 2                                 # bytes of q, out and q_rot
POOL = 8 * 2 * 16 * 64 * 2


@pytest.mark.parametrize("kw", [
    dict(out=1 * MB), dict(out=1 * MB + ROW - 16), dict(out=1 * MB - ROW + 16), dict(out=2 * MB),
    dict(out=3 * MB + POOL - 16), dict(lse=6 * MB + 16), dict(lse=1 * MB), dict(lse=4 * MB),
    dict(lse=5 * MB + 8), dict(scratch=1 * MB), dict(scratch=6 * MB), dict(scratch=2 * MB),
    dict(out=8 * MB + 256)])
def test_attention_writes_over_nothing_it_reads(kw):
    assert _attend(**kw) == P.PRSINK_ERR_ARG
    assert "of their own" in P.prsink_last_error()


@pytest.mark.parametrize("kw", [
    dict(vp=3 * MB), dict(vp=3 * MB + POOL - 16), dict(qr=1 * MB), dict(qr=2 * MB + 256),
    dict(qr=3 * MB), dict(qr=4 * MB + POOL - 16), dict(qr=8 * MB + 16), dict(qr=8 * MB - ROW + 16),
    dict(kp=5 * MB), dict(vp=6 * MB), dict(kp=7 * MB + 16 - POOL), dict(qr=5 * MB),
    dict(ks=4096, qr=1 * MB + 2 * 8192)])
def test_append_writes_over_nothing_it_reads(kw):
    assert _append(**kw) == P.PRSINK_ERR_ARG
    assert "of their own" in P.prsink_last_error()


def test_backward_writes_over_nothing_it_reads():
    lay = P.make_layout(**synth.preset("tiny"))
    nb = P.prsink_attention_backward_scratch_bytes(lay)
    names = ("q", "k", "v", "out", "lse", "d_out", "dq", "dk", "dv")

    def call(mask=0xFF, dyn=None, scratch=30 * MB, **kw):
        a = [kw.get(x, (i + 1) * MB) for i, x in enumerate(names)]
        return P._lib._lib.prsink_attention_backward(ctypes.byref(lay), *a, mask, dyn, scratch, nb,
                                                     None)
    q, k = 48 * 64 * 2, 256 * 64 * 2
    for kw in (dict(dq=1 * MB + q - 16), dict(dq=2 * MB - q + 16), dict(dq=5 * MB),
               dict(dk=2 * MB + k - 16), dict(dv=8 * MB + 16), dict(dk=4 * MB - 16),
               dict(scratch=6 * MB), dict(scratch=7 * MB), dict(scratch=9 * MB),
               dict(dyn=7 * MB + 8)):
        assert call(**kw) == P.PRSINK_ERR_ARG, kw
        assert "of their own" in P.prsink_last_error()


def test_neighbours_are_not_refused():
    """Side by side, in place where that is allowed, and rows between the rows of a wider buffer:
    past the overlap check (the next thing that fails here is the missing device)."""
    if P._lib.torch.cuda.is_available():
        pytest.skip("the addresses have no memory behind them")
    for rc in (_attend(out=1 * MB + ROW), _attend(lse=6 * MB + ROW), _append(qr=8 * MB),
               _append(vp=3 * MB + POOL), _append(k=8 * MB + 512, v=8 * MB + 768, ks=512, vs=512,
                                                  qs=512),
               _append(ks=4096, qr=1 * MB + 256)):
        assert rc == P.PRSINK_ERR_LAUNCH, P.prsink_last_error()
