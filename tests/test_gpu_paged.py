"""GPU parity of the paged-cache append and attention against the float64 oracle.

Tolerances (per element, from the arithmetic; bf16 rounds by at most u = 2^-8 of the value):
  append   V and untouched rows: the same bits.  K and q: one bf16 rounding of a float32 result
           whose two products and cos / sin each carry 2^-24: u |y| + 2^-21 (|x0| + |x1|).
  out      probabilities rounded to bf16 inside the sum (u times the softmax average of |v|),
           the result rounded (u |out|); scores, exponentials and sums in float32: d 2^-24
           sum |q k| / sqrt(d) <= 2^-13 of the average for these inputs.
  lse      2^-12 absolute (the scores' float32 sums) plus 2^-22 relative.
"""
import numpy as np
import pytest
import torch

import oracle
import pose_retrieved_kv_b200 as P
from tests._gpu import f64, need_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


def make(**kw):
    pg = dict(n_seqs=1, n_heads=4, n_kv_heads=2, head_dim=64, page_size=16, n_pages=8,
              max_pages=4, rope_mode=1, rope_split=(0, 0, 0), rope_base=10000.0, grid_h=3,
              grid_w=5, n_sink=0, window=0)
    pg.update(kw)
    if pg["rope_mode"] == 3 and not any(pg["rope_split"]):
        pg["rope_split"] = (44, 42, 42) if pg["head_dim"] == 128 else (24, 20, 20)
    return pg


def bits(t):
    return t.detach().cpu().view(torch.int16).numpy()


def pools(pg, gen, stale=None):
    shape = (pg["n_pages"], pg["n_kv_heads"], pg["page_size"], pg["head_dim"])
    k, v = (torch.randn(shape, generator=gen).bfloat16() for _ in range(2))
    return k, v


def scattered_table(pg, gen, lens):
    """Distinct pages in random order; entries behind the last needed page hold garbage."""
    order = torch.randperm(pg["n_pages"], generator=gen).tolist()
    table = torch.full((pg["n_seqs"], pg["max_pages"]), -7, dtype=torch.int32)
    for s, n in enumerate(lens):
        for i in range(-(-int(n) // pg["page_size"])):
            table[s, i] = order.pop()
    return table


def attend(pg, q, k, v, table, lens, lse=True, stream=None):
    p = P.make_paged(**pg)
    nb = P.prsink_paged_attention_scratch_bytes(p)
    scratch = torch.full((max(nb, 1),), 255, dtype=torch.uint8, device="cuda")  # not zeroed
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    ls = torch.full(q.shape[:2], float("nan"), device="cuda") if lse else None
    P.prsink_paged_attention(p, q, k, v, table, lens, out, scratch, lse=ls, stream=stream)
    return out, ls


def check_attention(pg, out, lse, q, k, v, table, lens):
    ref, rl, avg = oracle.paged_attention(pg, f64(q), f64(k), f64(v), table.tolist(),
                                          lens.tolist())
    got = f64(out)
    assert np.all(np.isfinite(got))
    tol = U * np.abs(ref) + (U + 2.0 ** -12) * avg
    bad = np.abs(got - ref) - tol
    assert np.all(bad <= 0), f"max excess {bad.max():.3e} at {np.unravel_index(bad.argmax(), bad.shape)}"
    gl = f64(lse)
    dead = np.isneginf(rl)
    assert np.array_equal(np.isneginf(gl), dead)
    assert np.all(np.abs(gl[~dead] - rl[~dead]) <= 2.0 ** -12 + 2.0 ** -22 * np.abs(rl[~dead]))


# ------------------------------------------------------------------------------------ append
APPENDS = [
    (dict(n_seqs=3, head_dim=128, n_pages=24, max_pages=8), [5, 1, 9], [5, 40, 128]),
    (dict(n_seqs=3, rope_mode=3, n_pages=40, max_pages=8, page_size=48), [0, 130, 64],
     [300, 131, 64]),
    (dict(n_seqs=2, rope_mode=0, n_heads=6, n_kv_heads=6, n_pages=4, max_pages=2,
          page_size=200), [201, 3], [399, 3]),
    (dict(n_seqs=2, n_heads=5, n_kv_heads=1, head_dim=128, rope_mode=3, n_pages=40, max_pages=40,
          page_size=8), [1, 37], [17, 64]),
    (dict(n_seqs=1, n_heads=40, n_kv_heads=40, head_dim=128, rope_mode=3, n_pages=3, max_pages=2,
          page_size=900, grid_h=30, grid_w=30), [1000], [1001]),
    (dict(n_seqs=1, n_pages=2, max_pages=1 << 21, page_size=512), [2], [3]),
]


@pytest.mark.parametrize("kw,new,lens", APPENDS)
@pytest.mark.parametrize("with_q", [True, False])
def test_append_matches_the_oracle_and_touches_nothing_else(kw, new, lens, with_q):
    need_gpu()
    pg = make(**kw)
    gen = torch.Generator().manual_seed(11)
    H, Hkv, d = pg["n_heads"], pg["n_kv_heads"], pg["head_dim"]
    n, extra = sum(new), 3                       # rows behind the last sequence
    k0, v0 = pools(pg, gen)
    if pg["max_pages"] > 1000:
        table = torch.zeros((1, pg["max_pages"]), dtype=torch.int32)
    else:
        table = scattered_table(pg, gen, lens)
    fused = torch.randn((n + extra, (H + 2 * Hkv) * d + 8), generator=gen).bfloat16()
    fused[n:] = float("nan")
    q, k, v = (x.reshape(n + extra, -1, d) for x in
               (fused[:, :H * d], fused[:, H * d:(H + Hkv) * d],
                fused[:, (H + Hkv) * d:(H + 2 * Hkv) * d]))
    cu = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32)
    dev = fused.cuda()
    cut = lambda a, b: dev[:, a * d:b * d].unflatten(1, (-1, d))      # noqa: E731
    kd, vd = k0.cuda(), v0.cuda()
    qr = torch.full((n + extra, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    P.prsink_paged_append(P.make_paged(**pg), cut(H, H + Hkv), cut(H + Hkv, H + 2 * Hkv), kd, vd,
                          table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                          cu_new=cu.cuda(), q=cut(0, H) if with_q else None,
                          q_rot=qr if with_q else None)
    assert P.prsink_sync_status() == P.PRSINK_OK
    rk, rv, rq = oracle.paged_append(pg, f64(k[:n]), f64(v[:n]), f64(k0), f64(v0), table.tolist(),
                                     lens, cu.tolist(), f64(q[:n]), np.full((n, H, d), 7.0))
    same = np.all(rk == f64(k0), axis=-1)        # rows that were not written
    assert np.array_equal(bits(kd)[same], bits(k0)[same])
    assert np.array_equal(f64(vd), rv)
    pairs = lambda x: np.repeat(np.abs(x[..., 0::2]) + np.abs(x[..., 1::2]), 2, axis=-1)  # noqa: E731
    tol = lambda y: U * np.abs(y) + 2.0 ** -21 * pairs(y) * 1.5      # |x0|+|x1| <= sqrt2 pair sum  # noqa: E731,E501
    assert np.all(np.abs(f64(kd) - rk) <= np.where(same[..., None], 0, tol(rk)))
    if with_q:
        assert np.all(np.abs(f64(qr[:n]) - rq) <= tol(rq)) and torch.all(qr[n:] == 7.0)
    else:
        assert torch.all(qr == 7.0)


def test_append_one_token_each_idle_rows_and_in_place_queries():
    need_gpu()
    pg = make(n_seqs=5, n_pages=30, max_pages=4, head_dim=128)
    gen = torch.Generator().manual_seed(12)
    lens = [1, 0, 33, 64, 16]
    table = scattered_table(pg, gen, lens)
    k0, v0 = pools(pg, gen)
    q, k, v = (torch.randn((5, h, 128), generator=gen).bfloat16() for h in (4, 2, 2))
    kd, vd, qd = k0.cuda(), v0.cuda(), q.cuda()
    P.prsink_paged_append(P.make_paged(**pg), k.cuda(), v.cuda(), kd, vd, table.cuda(),
                          torch.tensor(lens, dtype=torch.int32).cuda(), q=qd, q_rot=qd)
    assert P.prsink_sync_status() == P.PRSINK_OK
    rk, rv, rq = oracle.paged_append(pg, f64(k), f64(v), f64(k0), f64(v0), table.tolist(), lens,
                                     None, f64(q), f64(q))
    assert np.array_equal(f64(vd), rv) and np.array_equal(bits(qd[1]), bits(q[1]))
    assert np.all(np.abs(f64(kd) - rk) <= 2.0 ** -7 * (np.abs(rk) + 1e-3))
    assert np.all(np.abs(f64(qd) - rq) <= 2.0 ** -7 * (np.abs(rq) + 1e-3))


def test_append_far_positions():
    """Angles of far positions: token 2^29 + 12345 (1-D) of a long sequence."""
    need_gpu()
    pg = make(page_size=1024, max_pages=1 << 20, n_pages=2, head_dim=128)
    t = (1 << 29) + 12345
    gen = torch.Generator().manual_seed(13)
    k, v = (torch.randn((1, 2, 128), generator=gen).bfloat16() for _ in range(2))
    kd, vd = (torch.zeros((2, 2, 1024, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.zeros((1, 1 << 20), dtype=torch.int32)
    table[0, t // 1024] = 1
    P.prsink_paged_append(P.make_paged(**pg), k.cuda(), v.cuda(), kd, vd, table.cuda(),
                          torch.tensor([t + 1], dtype=torch.int32).cuda())
    assert P.prsink_sync_status() == P.PRSINK_OK
    want = oracle.paged_rotate(pg, f64(k), [t])[0]
    # the angle itself: 2^30 radians at 2^-52 each
    assert np.all(np.abs(f64(kd[1, :, t % 1024]) - want) <= U * np.abs(want) + 4e-6)
    assert torch.equal(vd[1, :, t % 1024].cpu(), v[0])


BAD = [dict(table=[[99, -1, 8, 2], [0, 1, 2, 3]]),            # pages outside the pool
       dict(lens=[65, 20]), dict(lens=[-3, 20]), dict(lens=[2, 20]),   # too long, negative, short
       dict(cu=[0, 9, 6]), dict(cu=[0, -5, 6]), dict(cu=[3, 4, 6])]


@pytest.mark.parametrize("bad", BAD)
def test_append_refuses_bad_tables_on_the_device(bad):
    """Out-of-range lengths, pages and offsets are recorded and skipped; nothing else moves."""
    need_gpu()
    pg = make(n_seqs=2)
    a = dict(table=[[4, 5, 6, 7], [0, 1, 2, 3]], lens=[40, 20], cu=[0, 4, 6])
    a.update(bad)
    gen = torch.Generator().manual_seed(14)
    k0, v0 = pools(pg, gen)
    k, v = (torch.randn((6, 2, 64), generator=gen).bfloat16() for _ in range(2))
    kd, vd = k0.cuda(), v0.cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()         # noqa: E731
    P.prsink_paged_append(P.make_paged(**pg), k.cuda(), v.cuda(), kd, vd, i32(a["table"]),
                          i32(a["lens"]), cu_new=i32(a["cu"]))
    status = P.prsink_sync_status()
    # offsets out of order may still name a sequence for every row: stored inside the pages then
    assert status == P.PRSINK_ERR_PAGE or bad in (dict(cu=[0, 9, 6]), dict(cu=[0, -5, 6]))
    assert P.prsink_sync_status() == P.PRSINK_OK                      # read and cleared
    moved = (bits(vd) != bits(v0)).any(-1).any(1).sum()               # (page, row) pairs
    assert moved <= 6
    if "lens" in bad:                                                 # the good sequence is stored
        assert torch.equal(vd[1, :, 2:4].cpu().transpose(0, 1), v[4:6])


# --------------------------------------------------------------------------------- attention
ATTENDS = [
    (dict(n_seqs=1, n_heads=1, n_kv_heads=1), [1]),
    (dict(n_seqs=4, n_pages=40, max_pages=10), [0, 160, 17, 1]),
    (dict(n_seqs=3, n_heads=16, n_kv_heads=1, head_dim=128, n_pages=80, max_pages=32), [500, 2, 511]),
    (dict(n_seqs=2, n_heads=40, n_kv_heads=8, head_dim=128, n_pages=60, max_pages=50, page_size=48),
     [2400, 95]),
    (dict(n_seqs=2, n_heads=21, n_kv_heads=1, head_dim=128, n_pages=5, max_pages=3, page_size=900),
     [2699, 901]),
    (dict(n_seqs=1, n_heads=66, n_kv_heads=1, n_pages=5, max_pages=4, page_size=129), [515]),
    (dict(n_seqs=2, n_heads=3, n_kv_heads=3, n_pages=300, max_pages=200, page_size=8), [1599, 63]),
    (dict(n_seqs=1, n_heads=2, n_kv_heads=2, head_dim=128, n_pages=20, max_pages=17,
          page_size=1024), [17000]),
    (dict(n_seqs=70, n_heads=2, n_kv_heads=1, n_pages=600, max_pages=5, page_size=32),
     [(37 * i) % 161 for i in range(70)]),
]
BOUNDS = [(0, 0), (5, 1), (0, 100), (40, 130), (1 << 30, 3), (130, 1 << 30)]


@pytest.mark.parametrize("kw,lens", ATTENDS)
@pytest.mark.parametrize("sink,window", BOUNDS)
def test_attention_matches_the_oracle(kw, lens, sink, window):
    need_gpu()
    pg = make(**kw, n_sink=sink, window=window)
    gen = torch.Generator().manual_seed(21)
    table = scattered_table(pg, gen, lens)
    k, v = pools(pg, gen)
    # rows behind a sequence's end and pages of no sequence hold anything
    used = np.zeros((pg["n_pages"], pg["page_size"]), bool)
    for s, n in enumerate(lens):
        for page, row in oracle.paged_attended(pg, table[s].tolist(), n):
            used[page, row] = True
    dead = torch.from_numpy(~used)[:, None, :, None].expand_as(k)
    k, v = k.masked_fill(dead, float("nan")), v.masked_fill(dead, float("inf"))
    q = torch.randn((pg["n_seqs"], pg["n_heads"], pg["head_dim"]), generator=gen).bfloat16()
    lens = torch.tensor(lens, dtype=torch.int32)
    out, lse = attend(pg, q.cuda(), k.cuda(), v.cuda(), table.cuda(), lens.cuda())
    assert P.prsink_sync_status() == P.PRSINK_OK
    check_attention(pg, out, lse, q, k, v, table, lens)
    again, _ = attend(pg, q.cuda(), k.cuda(), v.cuda(), table.cuda(), lens.cuda(), lse=False)
    assert torch.equal(out, again)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("gain", [0.0, 6.0, 40.0])
def test_attention_peaked_and_flat_scores(gain, d):
    """Flat scores average V; large ones pick single keys, the maximum growing along the cache
    (the running maximum and the rescaled sums)."""
    need_gpu()
    pg = make(n_seqs=2, n_heads=4, n_kv_heads=2, head_dim=d, n_pages=40, max_pages=16,
              page_size=128)
    gen = torch.Generator().manual_seed(22)
    lens = torch.tensor([2000, 700], dtype=torch.int32)
    table = scattered_table(pg, gen, lens.tolist())
    k, v = pools(pg, gen)
    q = torch.randn((2, 4, d), generator=gen)
    for s in range(2):                            # keys of later pages point along the query
        for i in range(-(-int(lens[s]) // 128)):
            for g in range(2):
                k[table[s, i], g] += (q[s, 2 * g] * 0.05 * i).bfloat16()
    q = (q * gain).bfloat16()
    out, lse = attend(pg, q.cuda(), k.cuda(), v.cuda(), table.cuda(), lens.cuda())
    assert P.prsink_sync_status() == P.PRSINK_OK
    ref, rl, avg = oracle.paged_attention(pg, f64(q), f64(k), f64(v), table.tolist(), lens.tolist())
    # float32 scores: d 2^-24 sum |q k| / sqrt(d), here with |q k| summing to at most gain * 4 d
    es = 2.0 ** -24 * d * gain * 4 * d / np.sqrt(d)
    tol = U * np.abs(ref) + (U + np.expm1(2 * es) + 2.0 ** -12) * avg
    assert np.all(np.abs(f64(out) - ref) <= tol)
    assert np.all(np.abs(f64(lse) - rl) <= es + 2.0 ** -12 + 2.0 ** -20 * np.abs(rl))


def test_attention_bad_pages_and_lengths_are_recorded_and_absent():
    need_gpu()
    pg = make(n_seqs=3, n_pages=12, max_pages=4)
    gen = torch.Generator().manual_seed(23)
    k, v = pools(pg, gen)
    table = torch.tensor([[3, 99, -1, 5], [1 << 30, -(1 << 31), 2, 4], [0, 1, 6, 7]],
                         dtype=torch.int32)
    lens = torch.tensor([64, 40, 70], dtype=torch.int32)      # the last one too long
    q = torch.randn((3, 4, 64), generator=gen).bfloat16()
    out, lse = attend(pg, q.cuda(), k.cuda(), v.cuda(), table.cuda(), lens.cuda())
    assert P.prsink_sync_status() == P.PRSINK_ERR_PAGE
    assert P.prsink_sync_status() == P.PRSINK_OK
    check_attention(pg, out, lse, q, k, v, table, lens)
    lens = torch.tensor([0, -5, 16], dtype=torch.int32)
    out, lse = attend(pg, q.cuda(), k.cuda(), v.cuda(), table.cuda(), lens.cuda())
    assert P.prsink_sync_status() == P.PRSINK_ERR_PAGE
    check_attention(pg, out, lse, q, k, v, table, lens)
    table[0, :] = -1                                           # every page missing
    lens = torch.tensor([64, 0, 16], dtype=torch.int32)
    out, lse = attend(pg, q.cuda(), k.cuda(), v.cuda(), table.cuda(), lens.cuda())
    assert P.prsink_sync_status() == P.PRSINK_ERR_PAGE
    check_attention(pg, out, lse, q, k, v, table, lens)


def test_attention_shared_pages():
    """Two sequences that read the same pages (a shared prefix) answer as if they were apart."""
    need_gpu()
    pg = make(n_seqs=2, n_pages=12, max_pages=6)
    gen = torch.Generator().manual_seed(24)
    k, v = pools(pg, gen)
    table = torch.tensor([[3, 1, 5, 7, 8, 2], [3, 1, 5, 7, 9, 0]], dtype=torch.int32)
    lens = torch.tensor([90, 70], dtype=torch.int32)
    q = torch.randn((2, 4, 64), generator=gen).bfloat16()
    out, lse = attend(pg, q.cuda(), k.cuda(), v.cuda(), table.cuda(), lens.cuda())
    check_attention(pg, out, lse, q, k, v, table, lens)


def test_pool_offsets_past_32_bits():
    """A pool of 4.3 GB per tensor (element offsets past 2^31): its last pages are written, read
    and attended."""
    need_gpu()
    pg = make(n_heads=2, n_kv_heads=2, head_dim=128, page_size=1024, n_pages=8300, max_pages=4)
    gen = torch.Generator().manual_seed(25)
    k, v = (torch.zeros((8300, 2, 1024, 128), dtype=torch.bfloat16, device="cuda")
            for _ in range(2))
    table = torch.tensor([[8299, 0, 8298, 8192]], dtype=torch.int32)
    new = 3100
    kn, vn = (torch.randn((new, 2, 128), generator=gen).bfloat16() for _ in range(2))
    lens = torch.tensor([new], dtype=torch.int32)
    P.prsink_paged_append(P.make_paged(**pg), kn.cuda(), vn.cuda(), k, v, table.cuda(),
                          lens.cuda(), cu_new=torch.tensor([0, new], dtype=torch.int32).cuda())
    q = torch.randn((1, 2, 128), generator=gen).bfloat16()
    out, lse = attend(pg, q.cuda(), k, v, table.cuda(), lens.cuda())
    assert P.prsink_sync_status() == P.PRSINK_OK
    pages = [8299, 0, 8298, 8192]
    for i, page in enumerate(pages):
        n = min(1024, new - 1024 * i)
        assert torch.equal(v[page, :, :n].cpu(), vn[1024 * i:1024 * i + n].transpose(0, 1))
    small = dict(pg, n_pages=4)
    check_attention(small, out, lse, q, k[pages].cpu(), v[pages].cpu(),
                    torch.tensor([[0, 1, 2, 3]]), lens)


# ------------------------------------------------------------------------------------ together
def test_prompt_then_single_tokens_in_a_captured_step():
    """Prompts appended, then tokens one by one through one captured step (append with its
    queries, attention) replayed while lengths and inputs change on the device; on a side stream,
    twice into the same scratch."""
    need_gpu()
    pg = make(n_seqs=3, n_heads=10, n_kv_heads=2, head_dim=128, n_pages=30, max_pages=8,
              page_size=32, n_sink=20, window=70)
    p = P.make_paged(**pg)
    gen = torch.Generator().manual_seed(31)
    start, steps = [100, 1, 0], 6
    table = scattered_table(pg, gen, [n + steps for n in start])
    k0, v0 = pools(pg, gen)
    n0 = sum(start)
    kn, vn = (torch.randn((n0 + 3 * steps, 2, 128), generator=gen).bfloat16() for _ in range(2))
    qn = torch.randn((3 * steps, 10, 128), generator=gen).bfloat16()
    kd, vd, td = k0.cuda(), v0.cuda(), table.cuda()
    lens = torch.tensor(start, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 100, 101, 101], dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    k_in, v_in, q_in = kn[:3].cuda(), vn[:3].cuda(), qn[:3].cuda()
    q_rot, out = torch.empty_like(q_in), torch.empty_like(q_in)
    lse = torch.empty((3, 10), device="cuda")
    scratch = torch.empty(max(P.prsink_paged_attention_scratch_bytes(p), 1), dtype=torch.uint8,
                          device="cuda")

    def step():
        P.prsink_paged_append(p, k_in, v_in, kd, vd, td, lens, q=q_in, q_rot=q_rot)
        P.prsink_paged_attention(p, q_rot, kd, vd, td, lens, out, scratch, lse=lse)
    with torch.cuda.stream(stream):
        P.prsink_paged_append(p, kn[:n0].cuda(), vn[:n0].cuda(), kd, vd, td, lens, cu_new=cu)
        graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        step()
    rk, rv, _ = oracle.paged_append(pg, f64(kn[:n0]), f64(vn[:n0]), f64(k0), f64(v0),
                                    table.tolist(), start, cu.tolist())
    for i in range(steps):
        a = n0 + 3 * i
        with torch.cuda.stream(stream):
            lens += 1
            k_in.copy_(kn[a:a + 3])
            v_in.copy_(vn[a:a + 3])
            q_in.copy_(qn[3 * i:3 * i + 3])
            graph.replay()
        assert P.prsink_sync_status(stream) == P.PRSINK_OK
        now = lens.tolist()
        assert now == [n + i + 1 for n in start]
        rk, rv, rq = oracle.paged_append(pg, f64(kn[a:a + 3]), f64(vn[a:a + 3]), rk, rv,
                                         table.tolist(), now, None, f64(qn[3 * i:3 * i + 3]),
                                         np.zeros((3, 10, 128)))
        assert np.array_equal(f64(vd), rv)
        assert np.all(np.abs(f64(kd) - rk) <= 2.0 ** -7 * (np.abs(rk) + 1e-3))
        check_attention(pg, out, lse, q_rot, kd, vd, table, torch.tensor(now))


def test_paged_and_slot_attention_agree():
    """One stream's block attention over the slot-indexed cache (raw keys, rotated inside) and
    the paged attention of the same queries over the same keys, appended with their positions in
    the block's logical order."""
    need_gpu()
    import synth
    cfg = synth.preset("tiny", block_index=5, valid_mask=0xFF, n_heads=2, head_dim=64)
    s = oracle.layout_sizes(cfg)
    lay = P.make_layout(**cfg)
    from tests._gpu import attention_inputs
    q, k, v = attention_inputs(cfg, seed=5)
    out = torch.empty((s["L_blk"], 2, 64), dtype=torch.bfloat16, device="cuda")
    P.prsink_attention(lay, q.cuda(), k.cuda(), v.cuda(), out)
    kpos, _ = oracle.key_positions(cfg)
    order = torch.from_numpy(np.argsort(kpos))               # logical order: positions 0..T-1
    T = s["T"]
    pg = make(n_heads=2, n_kv_heads=2, n_pages=40, max_pages=32, page_size=8)
    p = P.make_paged(**pg)
    table = torch.arange(3, 35, dtype=torch.int32, device="cuda")[None]
    kd, vd = (torch.zeros((40, 2, 8, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    q_rot = torch.zeros((T, 2, 64), dtype=torch.bfloat16, device="cuda")
    q_all = torch.zeros((T, 2, 64), dtype=torch.bfloat16)
    q_all[T - s["L_blk"]:] = q                               # the newest block's positions
    P.prsink_paged_append(p, k[:, order].transpose(0, 1).contiguous().cuda(),
                          v[:, order].transpose(0, 1).contiguous().cuda(), kd, vd, table, lens,
                          cu_new=torch.tensor([0, T], dtype=torch.int32, device="cuda"),
                          q=q_all.cuda(), q_rot=q_rot)
    got = torch.cat([attend(pg, q_rot[i:i + 1].contiguous(), kd, vd, table, lens)[0]
                     for i in range(T - s["L_blk"], T)])
    # both round P, the rotated keys and queries and the result: 2 (u |o| + 3 u avg|v|), |v| < 5
    assert (got.float() - out.float()).abs().max().item() <= 2e-2


@pytest.mark.parametrize("d,group", [(64, 1), (128, 20)])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_normal(d, group):
    need_gpu()
    pg = make(n_seqs=3, n_heads=2 * group, n_kv_heads=2, head_dim=d, n_pages=90, max_pages=40)
    gen = torch.Generator().manual_seed(32)
    lens = torch.tensor([600, 300, 64], dtype=torch.int32)
    table = scattered_table(pg, gen, lens.tolist()).cuda()
    k, v = (x.cuda() for x in pools(pg, gen))
    q = torch.randn((3, 2 * group, d), generator=gen).bfloat16().cuda()
    want = attend(pg, q, k, v, table, lens.cuda())
    assert P.prsink_sync_status() == P.PRSINK_OK
    P.prsink_debug_attention_stall(200_000)
    attend(pg, q, k, v, table, lens.cuda())
    assert P.prsink_sync_status() == P.PRSINK_ERR_TIMEOUT
    again = attend(pg, q, k, v, table, lens.cuda())
    assert P.prsink_sync_status() == P.PRSINK_OK
    assert all(torch.equal(a, b) for a, b in zip(want, again))


def test_not_a_number_in_an_attended_key_reaches_its_heads_only():
    need_gpu()
    pg = make(n_seqs=1, n_heads=4, n_kv_heads=2, n_pages=8, max_pages=6)
    gen = torch.Generator().manual_seed(33)
    k, v = pools(pg, gen)
    k[3, 1, 5, 7] = float("nan")
    v[2, 0, 1, 9] = float("inf")
    table = torch.tensor([[0, 1, 2, 3, 4, 5]], dtype=torch.int32)
    q = torch.randn((1, 4, 64), generator=gen).bfloat16()
    out, lse = attend(pg, q.cuda(), k.cuda(), v.cuda(), table.cuda(),
                      torch.tensor([90], dtype=torch.int32).cuda())
    out, lse = out.cpu()[0], lse.cpu()[0]
    assert torch.isnan(out[2:]).all() and torch.isnan(lse[2:]).all()
    assert torch.isfinite(lse[:2]).all() and torch.isinf(out[:2, 9]).all()
    assert torch.isfinite(out[:2, :9]).all() and torch.isfinite(out[:2, 10:]).all()


def test_append_many_tokens_of_many_sequences():
    """Enough tokens that several share a CTA, and enough sequences that the search for a token's
    sequence takes more than one step; sequences without new tokens among them."""
    need_gpu()
    gen = torch.Generator().manual_seed(41)
    g = np.random.default_rng(41)
    new = g.integers(0, 20, 300)
    new[[0, 7, 8, 299]] = 0
    new[100] = 31
    lens = new + g.integers(0, 40, 300)
    pg = make(n_seqs=300, n_heads=3, n_kv_heads=1, page_size=24, n_pages=1200, max_pages=3)
    assert new.sum() > 16 * 148
    table = scattered_table(pg, gen, lens)
    k0, v0 = pools(pg, gen)
    n = int(new.sum())
    q, k, v = (torch.randn((n, h, 64), generator=gen).bfloat16() for h in (3, 1, 1))
    cu = torch.from_numpy(np.concatenate([[0], np.cumsum(new)])).int()
    kd, vd, qr = k0.cuda(), v0.cuda(), torch.empty_like(q, device="cuda")
    P.prsink_paged_append(P.make_paged(**pg), k.cuda(), v.cuda(), kd, vd, table.cuda(),
                          torch.from_numpy(lens).int().cuda(), cu_new=cu.cuda(), q=q.cuda(),
                          q_rot=qr)
    assert P.prsink_sync_status() == P.PRSINK_OK
    rk, rv, rq = oracle.paged_append(pg, f64(k), f64(v), f64(k0), f64(v0), table.tolist(),
                                     lens.tolist(), cu.tolist(), f64(q), np.zeros((n, 3, 64)))
    assert np.array_equal(f64(vd), rv)
    assert np.all(np.abs(f64(kd) - rk) <= U * np.abs(rk) + 2.0 ** -18)
    assert np.all(np.abs(f64(qr) - rq) <= U * np.abs(rq) + 2.0 ** -18)


@pytest.mark.parametrize("page,d", [(200, 128), (200, 64), (136, 128), (72, 128), (40, 64)])
def test_attention_more_sequences_than_threads_and_odd_pages(page, d):
    """Several sequences per thread of the scan (empty ones among them), rows shared by CTAs,
    pages whose tiles are ragged."""
    need_gpu()
    gen = torch.Generator().manual_seed(42)
    g = np.random.default_rng(page + d)
    lens = torch.from_numpy(g.integers(0, 260, 600)).int()
    lens[[0, 1, 77, 598, 599]] = 0
    lens[[5, 300]] = torch.tensor([900, 1200], dtype=torch.int32)
    width = -(-1200 // page)
    pages = int(sum(-(-int(n) // page) for n in lens)) + 2
    pg = make(n_seqs=600, n_heads=3, n_kv_heads=1, head_dim=d, page_size=page, n_pages=pages,
              max_pages=width)
    table = scattered_table(pg, gen, lens.tolist())
    k, v = pools(pg, gen)
    q = torch.randn((600, 3, d), generator=gen).bfloat16()
    out, lse = attend(pg, q.cuda(), k.cuda(), v.cuda(), table.cuda(), lens.cuda())
    assert P.prsink_sync_status() == P.PRSINK_OK
    check_attention(pg, out, lse, q, k, v, table, lens)


def test_two_captured_calls_that_share_their_scratch():
    """Two graphs with the same scratch, replayed in turn on one stream: neither depends on what
    the other left there."""
    need_gpu()
    gen = torch.Generator().manual_seed(43)
    calls = []
    scratch = None
    for i, lens in enumerate(([2000, 700], [3000])):
        pg = make(n_seqs=len(lens), n_heads=4, n_kv_heads=2, head_dim=128, n_pages=200,
                  max_pages=190)
        p = P.make_paged(**pg)
        if scratch is None:
            scratch = torch.full((P.prsink_paged_attention_scratch_bytes(p),), 255,
                                 dtype=torch.uint8, device="cuda")
        table = scattered_table(pg, gen, lens).cuda()
        k, v = (x.cuda() for x in pools(pg, gen))
        q = torch.randn((len(lens), 4, 128), generator=gen).bfloat16().cuda()
        ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
        want = attend(pg, q, k, v, table, ln)
        out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            P.prsink_paged_attention(p, q, k, v, table, ln, out, scratch, lse=lse)
        calls.append((graph, out, lse, want, (p, q, k, v, table, ln)))
    for _ in range(3):
        for graph, out, lse, want, _ in calls:
            out.fill_(float("nan"))
            lse.fill_(float("nan"))
            graph.replay()
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
