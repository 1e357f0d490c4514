"""GPU tests of the paged calls at their edges.

Tolerances: those of ``tests/test_gpu_paged.py`` (derived there)."""
import numpy as np
import pytest
import torch

import oracle
import pose_retrieved_kv_b200 as P
from tests._gpu import f64, need_gpu
from tests.test_gpu_paged import attend, bits, check_attention, make, pools, scattered_table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,length,dead,max_pages", [(3, 480, 300, 30), (8, 8000, 5100, 501)])
def test_scores_of_minus_infinity_weigh_nothing(d, n, length, dead, max_pages):
    """Keys with an element of -inf (a mask folded into the keys) against queries that are positive
    there: whole tiles of such scores at the start of a row, in rows of one CTA (n = 3) and in
    shared ones, beside a key head without any.  One sequence holds nothing else."""
    need_gpu()
    pg = make(n_seqs=n, n_heads=6, n_kv_heads=2, head_dim=d, max_pages=max_pages,
              n_pages=n * max_pages)
    gen = torch.Generator().manual_seed(51)
    lens = torch.tensor([length] * (n - 1) + [dead], dtype=torch.int32)
    table = scattered_table(pg, gen, lens.tolist())
    k, v = pools(pg, gen)
    for s in range(n):
        for t in range(dead):
            k[table[s, t // 16], 0, t % 16, 5] = -float("inf")
    q = torch.randn((n, 6, d), generator=gen).bfloat16()
    q[..., 5] = q[..., 5].abs() + 0.5
    out, lse = attend(pg, q.cuda(), k.cuda(), v.cuda(), table.cuda(), lens.cuda())
    assert P.prsink_sync_status() == P.PRSINK_OK
    assert torch.all(out[-1, :3] == 0) and torch.all(lse[-1, :3] == -float("inf"))
    assert torch.isfinite(lse[-1, 3:]).all()
    check_attention(dict(pg, n_seqs=n - 1), out[:-1], lse[:-1], q[:-1], k, v, table[:-1],
                    lens[:-1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 16, 17, 32, 33, 64, 65, 130])
@pytest.mark.parametrize("page,bound", [(16, (0, 0)), (900, (37, 400))])
def test_every_number_of_heads_on_a_key_head(d, group, page, bound):
    """Both widths with 16, 32 and 64 columns, the last column of each in use and not, and more
    heads than one pass over the keys takes; rows of one tile, several, and shared ones."""
    need_gpu()
    lens = [1700, 0, 129, 1]
    width = -(-2700 // page)
    pg = make(n_seqs=4, n_heads=2 * group, n_kv_heads=2, head_dim=d, page_size=page,
              max_pages=width, n_pages=2 * width, n_sink=bound[0], window=bound[1])
    gen = torch.Generator().manual_seed(52)
    table = scattered_table(pg, gen, lens)
    k, v = pools(pg, gen)
    q = torch.randn((4, 2 * group, d), generator=gen).bfloat16()
    lens = torch.tensor(lens, dtype=torch.int32)
    out, lse = attend(pg, q.cuda(), k.cuda(), v.cuda(), table.cuda(), lens.cuda())
    assert P.prsink_sync_status() == P.PRSINK_OK
    check_attention(pg, out, lse, q, k, v, table, lens)


REFUSED = [dict(table=[[99, -1, 8, 2], [0, 1, 2, 3]]), dict(table=[[4, 5, 6, 7], [1, -(1 << 31), 0, 2]]),
           dict(lens=[65, 20]), dict(lens=[-3, 20]), dict(lens=[2, 20]), dict(lens=[40, 1 << 30])]


@pytest.mark.parametrize("bad", REFUSED)
def test_a_refused_token_leaves_every_other_row_alone(bad):
    """Tables and lengths out of range, against the oracle: V and untouched rows bit for bit, K and
    the rotated queries within a rounding, refused queries as they were."""
    need_gpu()
    pg = make(n_seqs=2)
    a = dict(table=[[4, 5, 6, 7], [0, 1, 2, 3]], lens=[40, 20])
    a.update(bad)
    cu, gen = [0, 4, 6], torch.Generator().manual_seed(53)
    k0, v0 = pools(pg, gen)
    q, k, v = (torch.randn((6, h, 64), generator=gen).bfloat16() for h in (4, 2, 2))
    kd, vd = k0.cuda(), v0.cuda()
    qr = torch.full((6, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()         # noqa: E731
    P.prsink_paged_append(P.make_paged(**pg), k.cuda(), v.cuda(), kd, vd, i32(a["table"]),
                          i32(a["lens"]), cu_new=i32(cu), q=q.cuda(), q_rot=qr)
    assert P.prsink_sync_status() == P.PRSINK_ERR_PAGE
    rk, rv, rq = oracle.paged_append(pg, f64(k), f64(v), f64(k0), f64(v0), a["table"], a["lens"],
                                     cu, f64(q), np.full((6, 4, 64), 7.0))
    same = np.all(rk == f64(k0), axis=-1)
    assert not same.all()                            # (the good sequence's tokens)
    assert np.array_equal(bits(kd)[same], bits(k0)[same]) and np.array_equal(f64(vd), rv)
    assert np.all(np.abs(f64(kd) - rk) <= 2.0 ** -8 * np.abs(rk) + 2.0 ** -18)
    left = np.all(rq == 7.0, axis=(1, 2))
    assert np.array_equal(f64(qr)[left], rq[left])
    assert np.all(np.abs(f64(qr) - rq) <= 2.0 ** -8 * np.abs(rq) + 2.0 ** -18)


@pytest.mark.parametrize("cu", [[0, 9, 6], [0, -5, 6], [3, 4, 6], [0, 4, 2], [7, 8, 9], [-2, -1, 0]])
def test_offsets_out_of_order_write_only_the_last_tokens(cu):
    """Whatever the offsets say, a row is stored where its sequence's newest tokens lie (token
    lens[s] - (cu[s+1] - i) of a sequence s whose range holds i), or not at all."""
    need_gpu()
    pg = make(n_seqs=2)
    table, lens = [[4, 5, 6, 7], [0, 1, 2, 3]], [40, 20]
    gen = torch.Generator().manual_seed(54)
    k0, v0 = pools(pg, gen)
    k, v = (torch.randn((6, 2, 64), generator=gen).bfloat16() for _ in range(2))
    kd, vd = k0.cuda(), v0.cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()         # noqa: E731
    P.prsink_paged_append(P.make_paged(**pg), k.cuda(), v.cuda(), kd, vd, i32(table), i32(lens),
                          cu_new=i32(cu))
    assert P.prsink_sync_status() in (P.PRSINK_OK, P.PRSINK_ERR_PAGE)
    may = {}                                         # (page, row) -> rows of v that may lie there
    for s in range(2):
        for i in range(max(cu[s], 0), min(cu[s + 1], 6)):
            t = lens[s] - (cu[s + 1] - i)
            if 0 <= t < 64:
                may.setdefault((table[s][t // 16], t % 16), []).append(i)
    moved = (bits(vd) != bits(v0)).any(-1).any(1)
    k_moved = (bits(kd) != bits(k0)).any(-1).any(1)
    for page, row in np.argwhere(moved | k_moved):
        rows = may.get((int(page), int(row)), [])
        assert any(torch.equal(vd[page, :, row].cpu(), v[i]) for i in rows), (page, row)


def test_a_timeout_does_not_hide_a_bad_page():
    """Both kinds recorded before the status is read: each is reported once, the timeout first."""
    need_gpu()
    pg = make(n_seqs=1, n_pages=12, max_pages=4)
    gen = torch.Generator().manual_seed(55)
    k, v = (x.cuda() for x in pools(pg, gen))
    q = torch.randn((1, 4, 64), generator=gen).bfloat16().cuda()
    table = torch.tensor([[3, 99, -1, 5]], dtype=torch.int32).cuda()
    attend(pg, q, k, v, table, torch.tensor([64], dtype=torch.int32).cuda())
    P.prsink_debug_wait_timeout(1000)
    assert P.prsink_sync_status() == P.PRSINK_ERR_TIMEOUT
    assert P.prsink_sync_status() == P.PRSINK_ERR_PAGE
    assert P.prsink_sync_status() == P.PRSINK_OK


def test_a_call_may_take_longer_than_a_wait():
    """A call of about 3 s (600 sequences of 2^20 tokens that share one page, 128 heads), longer
    than the limit of a wait: every wait in it is short.  A page repeated r = 2^13 times attends as
    the page itself, its lse log r larger.

    Beside the roundings of a short row: a key's float32 sum takes r additions of 2^-24 each (2^-11),
    an element of the product 8 r of at most 2^-23 (2^-7 of the average of |v|)."""
    need_gpu()
    n, heads, rep = 600, 128, 1 << 13
    pg = make(n_seqs=n, n_heads=heads, n_kv_heads=heads, page_size=128, n_pages=1, max_pages=rep)
    gen = torch.Generator().manual_seed(56)
    k, v = pools(pg, gen)
    q = torch.randn((n, heads, 64), generator=gen).bfloat16()
    table = torch.zeros((n, rep), dtype=torch.int32, device="cuda")
    lens = torch.full((n,), 128 * rep, dtype=torch.int32, device="cuda")
    out, lse = attend(pg, q.cuda(), k.cuda(), v.cuda(), table, lens)
    assert P.prsink_sync_status() == P.PRSINK_OK
    some = [0, 1, 299, 598, 599]
    once = dict(pg, n_seqs=len(some), max_pages=1)
    ref, rl, avg = oracle.paged_attention(once, f64(q[some]), f64(k), f64(v), [[0]] * 5, [128] * 5)
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12 + 2.0 ** -11 + 2.0 ** -7) * avg
    assert np.all(np.abs(f64(out[some]) - ref) <= tol)
    assert np.all(np.abs(f64(lse[some]) - rl - np.log(rep)) <= 2.0 ** -11 + 2.0 ** -11)
