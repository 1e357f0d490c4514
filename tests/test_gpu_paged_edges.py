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
