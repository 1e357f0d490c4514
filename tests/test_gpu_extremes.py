"""GPU tests of the paged calls and the backward pass at the limits that their checks allow: the
most sequences, heads and heads per key head, one page of a prime number of rows.  Tolerances as in
``tests/test_gpu_paged.py`` and ``tests/test_gpu_backward.py``."""
import numpy as np
import pytest
import torch

import oracle
import pose_retrieved_kv_b200 as P
from tests._gpu import f64, need_gpu
from tests.test_gpu_backward import backward, case, check, forward, inputs
from tests.test_gpu_paged import attend, bits, check_attention, make, pools

pytestmark = pytest.mark.gpu
MOST = 65535


def test_most_sequences():
    """65535 sequences of up to 8 tokens, idle ones among them: the newest token of each appended,
    then all attended."""
    need_gpu()
    pg = make(n_seqs=MOST, n_heads=2, n_kv_heads=1, page_size=8, n_pages=MOST, max_pages=1)
    gen = torch.Generator().manual_seed(91)
    lens = torch.randint(0, 9, (MOST,), generator=gen, dtype=torch.int32)
    lens[[0, 1, 255, 256, 257, MOST - 1]] = torch.tensor([0, 8, 0, 0, 1, 3], dtype=torch.int32)
    table = torch.randperm(MOST, generator=gen).int()[:, None]
    k, v = pools(pg, gen)
    q, kn, vn = (torch.randn((MOST, h, 64), generator=gen).bfloat16() for h in (2, 1, 1))
    kd, vd, qr = k.cuda(), v.cuda(), torch.zeros((MOST, 2, 64), dtype=torch.bfloat16, device="cuda")
    P.prsink_paged_append(P.make_paged(**pg), kn.cuda(), vn.cuda(), kd, vd, table.cuda(),
                          lens.cuda(), q=q.cuda(), q_rot=qr)
    assert P.prsink_sync_status() == P.PRSINK_OK
    live = (lens > 0).numpy()
    at = (table[live, 0].long(), 0, (lens[live] - 1).long())
    want = v.clone()
    want[at] = vn[live, 0]
    assert np.array_equal(bits(vd), bits(want))
    turned = oracle.paged_rotate(pg, f64(kn[live]), (lens[live] - 1).numpy())[:, 0]
    assert np.all(np.abs(f64(kd.cpu()[at]) - turned) <= 2.0 ** -8 * np.abs(turned) + 2.0 ** -18)
    out, lse = attend(pg, qr, kd, vd, table.cuda(), lens.cuda())
    assert P.prsink_sync_status() == P.PRSINK_OK
    keys, vals = (x.cpu().double()[table[:, 0].long(), 0] for x in (kd, vd))       # [n][8][64]
    sc = torch.einsum("nhd,ntd->nht", qr.cpu().double(), keys) / 8
    sc = sc.masked_fill(torch.arange(8) >= lens[:, None, None], -float("inf"))
    rl = torch.logsumexp(sc, -1)
    p = torch.exp(sc - rl[..., None]).nan_to_num(0.0)
    ref, avg = p @ vals, p @ vals.abs()
    assert torch.equal(torch.isneginf(lse.cpu()), torch.isneginf(rl))
    assert np.all(np.abs(f64(out) - ref.numpy()) <= (2.0 ** -8 * ref.abs() + (
        2.0 ** -8 + 2.0 ** -12) * avg).numpy())
    err = (lse.cpu().double() - rl)[torch.from_numpy(live)]
    assert err.abs().max() <= 2.0 ** -11


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv", [MOST, 1])
def test_most_heads(kv, d):
    """65535 heads with a key head each, or all of them on one key head."""
    need_gpu()
    pg = make(n_seqs=1, n_heads=MOST, n_kv_heads=kv, head_dim=d, page_size=8, n_pages=3,
              max_pages=2, rope_mode=3)
    gen = torch.Generator().manual_seed(92)
    k, v = pools(pg, gen)
    q, kn, vn = (torch.randn((1, h, d), generator=gen).bfloat16() for h in (MOST, kv, kv))
    table, lens = torch.tensor([[2, 0]], dtype=torch.int32), torch.tensor([13], dtype=torch.int32)
    kd, vd, qr = k.cuda(), v.cuda(), torch.zeros_like(q, device="cuda")
    P.prsink_paged_append(P.make_paged(**pg), kn.cuda(), vn.cuda(), kd, vd, table.cuda(),
                          lens.cuda(), q=q.cuda(), q_rot=qr)
    assert P.prsink_sync_status() == P.PRSINK_OK
    rk, rv, rq = oracle.paged_append(pg, f64(kn), f64(vn), f64(k), f64(v), [[2, 0]], [13], None,
                                     f64(q), np.zeros(q.shape))
    assert np.array_equal(f64(vd), rv)
    for got, want in ((kd, rk), (qr, rq)):
        assert np.all(np.abs(f64(got) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18)
    out, lse = attend(pg, qr, kd, vd, table.cuda(), lens.cuda())
    assert P.prsink_sync_status() == P.PRSINK_OK
    check_attention(pg, out, lse, qr, kd, vd, table, lens)


@pytest.mark.parametrize("d", [64, 128])
def test_one_page_of_a_prime_number_of_rows(d):
    need_gpu()
    rows = 1000003
    pg = make(n_seqs=2, n_heads=3, n_kv_heads=1, head_dim=d, page_size=rows, n_pages=2,
              max_pages=1, n_sink=130, window=rows - 300)
    gen = torch.Generator(device="cuda").manual_seed(93)
    k, v = (torch.randn((2, 1, rows, d), generator=gen, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn((2, 3, d), generator=gen, device="cuda").bfloat16()
    table = torch.tensor([[1], [0]], dtype=torch.int32)
    lens = torch.tensor([rows, 999937], dtype=torch.int32)
    out, lse = attend(pg, q, k, v, table.cuda(), lens.cuda())
    assert P.prsink_sync_status() == P.PRSINK_OK
    check_attention(pg, out, lse, q, k, v, table, lens)


def test_backward_of_most_heads():
    """65535 heads over a layout of one token per frame; some heads against the oracle."""
    need_gpu()
    cfg = case("grid", n_heads=MOST, grid_h=1, grid_w=1)
    some = [0, 1, 275, 276, 40000, MOST - 1]
    q, k, v, do = inputs(cfg, 94)
    few = dict(cfg, n_heads=len(some))
    s = oracle.layout_sizes(cfg)
    out = torch.empty_like(q, device="cuda")
    lse = torch.empty((MOST, s["L_blk"]), device="cuda")
    P.prsink_attention(P.make_layout(**cfg), q.cuda(), k.cuda(), v.cuda(), out, lse)
    assert P.prsink_sync_status() == P.PRSINK_OK
    o1, l1 = forward(few, q[:, some], k[some], v[some])
    out, lse = out.cpu(), lse.cpu()
    out[:, some], lse[some] = o1, l1
    dq, dk, dv = backward(cfg, q, k, v, do, out, lse)
    assert P.prsink_sync_status() == P.PRSINK_OK
    check(few, (dq[:, some], dk[some], dv[some]), q[:, some], k[some], v[some], do[:, some],
          norm=None)
    assert torch.isfinite(dq.float()).all() and torch.isfinite(dk.float()).all()
