"""Cases of the paged-cache operators and of the attention's backward pass, for timing and for
comparing the library's kernels with plain torch.

Three operators: ``append`` writes new tokens' K/V into a paged cache with the rotary embedding
applied on the way; ``decode`` is the attention of one new token per sequence over that cache;
``backward`` is the gradient of the block attention over the slot-indexed cache.
"""
import math

import torch

own = False                     # True: run() calls the library

BASE = 10000.0
GRID = 30                       # rows and columns of a frame for 3-D positions of paged tokens


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------

def listed():
    return [
        # one token of one short sequence, one head: latency alone (the tiny layout's cache)
        dict(name="decode 1x256 1h d64", op="decode", n_seqs=1, heads=1, kv_heads=1, dim=64,
             page=16, min_len=256, max_len=256, sink=0, window=0),
        # one stream's token over a full 480x480 cache, a page for each latent frame
        dict(name="decode 1x14400 40h", op="decode", n_seqs=1, heads=40, kv_heads=40, dim=128,
             page=900, min_len=14400, max_len=14400, sink=0, window=0),
        # a serving batch of ragged lengths, shared key heads
        dict(name="decode 48x(1..16001) 40h/8", op="decode", n_seqs=48, heads=40, kv_heads=8,
             dim=128, page=16, min_len=1, max_len=16001, sink=0, window=0),
        # long streams bounded to sinks and a rolling window (ref + static, three blocks)
        dict(name="decode 8x(20k..70k) sink+window", op="decode", n_seqs=8, heads=16,
             kv_heads=16, dim=128, page=64, min_len=20011, max_len=70001, sink=3600,
             window=8100),
        # one decoding step's append for a batch of 64
        dict(name="append 64x1 40h/8", op="append", n_seqs=64, new_min=1, new_max=1, heads=40,
             kv_heads=8, dim=128, page=16, past=1000, rope=1),
        # one block of 480x480 tokens, 3-D positions
        dict(name="append 1x2700 40h 3-D", op="append", n_seqs=1, new_min=2700, new_max=2700,
             heads=40, kv_heads=40, dim=128, page=900, past=8100, rope=3),
        # ragged prompts behind existing caches
        dict(name="append 16x(1..2047) 40h/8", op="append", n_seqs=16, new_min=1, new_max=2047,
             heads=40, kv_heads=8, dim=128, page=64, past=77, rope=1),
        # the tiny check's layout: latency
        dict(name="backward tiny 1h d64", op="backward", heads=1, dim=64, gh=4, gw=4, ring=3,
             rope=1, mask=0xFF, block=7),
        # one layer's heads on one of eight GPUs at 384x672, early in a stream (empty slots)
        dict(name="backward 384x672 5h early", op="backward", heads=5, dim=128, gh=24, gw=42,
             ring=3, rope=3, mask=0b011011, block=1),
        # odd grid, 64-wide heads, four ring slots
        dict(name="backward 13x17 12h d64", op="backward", heads=12, dim=64, gh=13, gw=17,
             ring=4, rope=3, mask=0xFF, block=1001),
        # a whole 480x480 layer
        dict(name="backward 480x480 40h", op="backward", heads=40, dim=128, gh=30, gw=30,
             ring=3, rope=3, mask=0xFF, block=1000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "backward"])
    dim = rng.choice([64, 128, 128])
    if op == "backward":
        ring = rng.randint(1, 4)
        gh, gw = _log(rng, 3, 30), _log(rng, 3, 30)
        heads = _log(rng, 1, 40)
        while heads > 1 and heads * (gh * gw) ** 2 * (7 + 3 * ring) > 40 * 900 ** 2 * 16:
            heads -= 1
        rope = 1 if gh * gw + 30 <= 50 else 3
        mask = rng.choice([0xFF, 0xFF, 0b111001, 0b001001, 1 | rng.randint(0, 127)])
        return dict(op=op, heads=heads, dim=dim, gh=gh, gw=gw, ring=ring, rope=rope, mask=mask,
                    block=rng.randint(0, 2000))
    kv = _log(rng, 1, 40)
    group = rng.choice([1, 1, 2, 4, 5, 8, 16])
    while group > 1 and kv * group > 64:
        group = {16: 8, 8: 5, 5: 4, 4: 2, 2: 1}[group]
    page = rng.choice([8, 16, 32, 48, 64, 128, 200, 900])
    if op == "append":
        n_seqs = _log(rng, 1, 64)
        new_max = _log(rng, 1, max(2, 16384 // n_seqs))
        while n_seqs * new_max * (kv * group + 2 * kv) > 2700 * 120:
            new_max = max(1, new_max // 2)
            n_seqs = n_seqs if new_max > 1 else max(1, n_seqs // 2)
        return dict(op=op, n_seqs=n_seqs, new_min=rng.randint(1, new_max), new_max=new_max,
                    heads=kv * group, kv_heads=kv, dim=dim, page=page,
                    past=_log(rng, 1, 4000), rope=rng.choice([1, 1, 3]))
    n_seqs = _log(rng, 1, 96)
    max_len = _log(rng, 1, 70000)
    while n_seqs * max_len * kv > 48 * 16001 * 8:
        max_len = max(1, max_len * 2 // 3)
        n_seqs = max(1, n_seqs - 1)
    bounded = rng.random() < 0.3
    return dict(op=op, n_seqs=n_seqs, heads=kv * group, kv_heads=kv, dim=dim, page=page,
                min_len=rng.randint(min(1, max_len), max_len), max_len=max_len,
                sink=rng.randint(0, max_len) if bounded else 0,
                window=rng.randint(1, max_len) if bounded else 0)


def _spread(lo, hi, n):
    """n numbers from lo to hi, both among them, in a scattered order."""
    if n == 1:
        return [hi]
    step = next(s for s in (7, 11, 13, 17) if n % s)
    return [lo + (hi - lo) * ((i * step) % n) // (n - 1) for i in range(n)]


def _attended(length, sink, window):
    if not window:
        return length
    first = max(0, length - window)
    return min(sink, first) + length - first


def _rope_split(case):
    d = case["dim"]
    if case["rope"] == 1:
        return (d, 0, 0)
    return (44, 42, 42) if d == 128 else (24, 20, 20)


def _append_plan(case):
    """(new tokens, length after the append) of every sequence."""
    new = _spread(case["new_min"], case["new_max"], case["n_seqs"])
    return new, [case["past"] + 3 * i + n for i, n in enumerate(new)]


def _tokens(case):
    lf = case["gh"] * case["gw"]
    return lf, 3 * lf, lf + (2 + case["ring"]) * 3 * lf


def _live_keys(case):
    lf, lblk, _ = _tokens(case)
    return sum((lf if s == 0 else lblk) for s in range(3 + case["ring"])
               if (case["mask"] >> s) & 1)


def work(case):
    d = case["dim"]
    if case["op"] == "append":
        n = sum(_append_plan(case)[0])
        rot = case["heads"] + case["kv_heads"]
        return {"bytes": 4 * n * d * (rot + case["kv_heads"]), "flops": 3 * n * d * rot}
    if case["op"] == "decode":
        keys = sum(_attended(x, case["sink"], case["window"])
                   for x in _spread(case["min_len"], case["max_len"], case["n_seqs"]))
        return {"bytes": 4 * d * (case["kv_heads"] * keys + case["heads"] * case["n_seqs"]),
                "flops": 4 * d * case["heads"] * keys}
    _, lblk, t = _tokens(case)
    h, live = case["heads"], _live_keys(case)
    return {"bytes": 2 * h * d * (4 * lblk + 2 * live + 2 * t) + 4 * h * lblk,
            "flops": 10 * h * lblk * live * d}


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).bfloat16()


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _page_table(gen, lens, page):
    """Pages scattered over the pool: (table [n_seqs][max_pages], pages in the pool)."""
    need = [-(-x // page) for x in lens]
    width = max(max(need), 1)
    pool = sum(need) + 3
    order = torch.randperm(pool, generator=gen, device="cuda").int()
    table = torch.zeros((len(lens), width), dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table, pool


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    d, h = case["dim"], case["heads"]
    if case["op"] == "backward":
        lf, lblk, t = _tokens(case)
        st = dict(case=case, q=_normal(gen, lblk, h, d), k=_normal(gen, h, t, d),
                  v=_normal(gen, h, t, d), d_out=_normal(gen, lblk, h, d))
        kpos, qpos, valid = _positions(case)
        st.update(kpos=kpos, qpos=qpos, valid=valid)
        p, lse, _, _ = _probs(st)
        st["out"] = torch.einsum("hqk,hkd->qhd", p, st["v"].float()).bfloat16()
        st["lse"] = lse
        st["dq"], st["dk"] = torch.empty_like(st["q"]), torch.empty_like(st["k"])
        st["dv"] = torch.empty_like(st["v"])
        return st
    kv, page = case["kv_heads"], case["page"]
    if case["op"] == "append":
        new, lens = _append_plan(case)
        n = sum(new)
        table, pool = _page_table(gen, lens, page)
        first = [sum(new[:i]) for i in range(len(new) + 1)]
        return dict(case=case, q=_normal(gen, n, h, d), k=_normal(gen, n, kv, d),
                    v=_normal(gen, n, kv, d), k_pages=_normal(gen, pool, kv, page, d),
                    v_pages=_normal(gen, pool, kv, page, d), table=table, lens=_i32(lens),
                    first=_i32(first), q_rot=torch.empty((n, h, d), dtype=torch.bfloat16,
                                                         device="cuda"))
    lens = _spread(case["min_len"], case["max_len"], case["n_seqs"])
    table, pool = _page_table(gen, lens, page)
    n = len(lens)
    return dict(case=case, q=_normal(gen, n, h, d), k_pages=_normal(gen, pool, kv, page, d),
                v_pages=_normal(gen, pool, kv, page, d), table=table, lens=_i32(lens),
                out=torch.empty((n, h, d), dtype=torch.bfloat16, device="cuda"),
                lse=torch.empty((n, h), dtype=torch.float32, device="cuda"))


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------

def run(state):
    if own:
        return _own(state)
    return {"append": _append, "decode": _decode, "backward": _backward}[
        state["case"]["op"]](state)


def _own(state):
    import pose_retrieved_kv_b200 as P
    case = state["case"]
    if case["op"] == "backward":
        if "scratch" not in state:
            state["layout"] = P.make_layout(
                n_heads=case["heads"], head_dim=case["dim"], grid_h=case["gh"],
                grid_w=case["gw"], ring_slots=case["ring"], rope_mode=case["rope"],
                rope_split=_rope_split(case), rope_base=BASE, block_index=case["block"],
                valid_mask=case["mask"])
            state["scratch"] = torch.empty(
                P.prsink_attention_backward_scratch_bytes(state["layout"]), dtype=torch.uint8,
                device="cuda")
            state["out"] = state["out"].contiguous()
        P.prsink_attention_backward(state["layout"], state["q"], state["k"], state["v"],
                                    state["out"], state["lse"], state["d_out"], state["dq"],
                                    state["dk"], state["dv"], state["scratch"])
        return dict(dq=state["dq"], dk=state["dk"], dv=state["dv"])
    if "paged" not in state:
        rope = case.get("rope", 0)
        state["paged"] = P.make_paged(
            n_seqs=case["n_seqs"], n_heads=case["heads"], n_kv_heads=case["kv_heads"],
            head_dim=case["dim"], page_size=case["page"], n_pages=state["k_pages"].shape[0],
            max_pages=state["table"].shape[1], rope_mode=rope,
            rope_split=_rope_split(case) if rope else (0, 0, 0), rope_base=BASE, grid_h=GRID,
            grid_w=GRID, n_sink=case.get("sink", 0), window=case.get("window", 0))
        if case["op"] == "decode":
            state["scratch"] = torch.empty(
                P.prsink_paged_attention_scratch_bytes(state["paged"]), dtype=torch.uint8,
                device="cuda")
    if case["op"] == "append":
        P.prsink_paged_append(state["paged"], state["k"], state["v"], state["k_pages"],
                              state["v_pages"], state["table"], state["lens"],
                              cu_new=state["first"], q=state["q"], q_rot=state["q_rot"])
        return dict(k_pages=state["k_pages"], v_pages=state["v_pages"], q_rot=state["q_rot"])
    P.prsink_paged_attention(state["paged"], state["q"], state["k_pages"], state["v_pages"],
                             state["table"], state["lens"], state["out"], state["scratch"],
                             lse=state["lse"])
    return dict(out=state["out"], lse=state["lse"])


def _angles(case, pos):
    """Angles [..., d/2] of positions [..., 3] (1-D: [..., 1]), in 64 bits."""
    parts = []
    for axis, da in enumerate(_rope_split(case)):
        if da:
            theta = BASE ** (-torch.arange(0, da, 2, device="cuda", dtype=torch.float64) / da)
            parts.append(pos[..., axis, None].double() * theta)
    return torch.cat(parts, -1)


def _turn(x, angle):
    """Rotate the interleaved pairs of x [..., d] by angles [..., d/2]."""
    c, s = torch.cos(angle).float(), torch.sin(angle).float()
    x0, x1 = x[..., 0::2].float(), x[..., 1::2].float()
    return torch.stack([x0 * c - x1 * s, x0 * s + x1 * c], -1).flatten(-2)


def _append(state):
    case = state["case"]
    first, lens, page = state["first"].long(), state["lens"].long(), case["page"]
    tok = torch.arange(state["k"].shape[0], device="cuda")
    seq = torch.searchsorted(first, tok, right=True) - 1
    pos = lens[seq] - first[seq + 1] + tok
    if case["rope"] == 1:
        grid = pos[:, None]
    else:
        grid = torch.stack([pos // GRID ** 2, pos // GRID % GRID, pos % GRID], -1)
    angle = _angles(case, grid)[:, None, :]
    at = state["table"][seq, pos // page].long()
    state["k_pages"][at, :, pos % page] = _turn(state["k"], angle).bfloat16()
    state["v_pages"][at, :, pos % page] = state["v"]
    state["q_rot"].copy_(_turn(state["q"], angle))
    return dict(k_pages=state["k_pages"], v_pages=state["v_pages"], q_rot=state["q_rot"])


def _decode(state):
    case = state["case"]
    n, h, kv, d = case["n_seqs"], case["heads"], case["kv_heads"], case["dim"]
    at = state["table"].long()
    k = state["k_pages"][at].float().transpose(2, 3).reshape(n, -1, kv, d)
    v = state["v_pages"][at].float().transpose(2, 3).reshape(n, -1, kv, d)
    q = state["q"].float().reshape(n, kv, h // kv, d)
    s = torch.einsum("ngjd,ntgd->ngjt", q, k) / math.sqrt(d)
    i, size = torch.arange(k.shape[1], device="cuda"), state["lens"][:, None]
    keep = i < size
    if case["window"]:
        keep &= (i < case["sink"]) | (i >= size - case["window"])
    s = torch.where(keep[:, None, None, :], s, -math.inf)
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - m)
    total = e.sum(-1, keepdim=True)
    o = torch.einsum("ngjt,ntgd->ngjd", e / total, v)
    return dict(out=o.reshape(n, h, d).bfloat16(),
                lse=(m + torch.log(total)).reshape(n, h))


def _positions(case):
    """Positions of the cache's keys and of the block's queries [., 3] (1-D: [., 1]), and which
    keys are valid; logical order ref, static, dynamic, ring oldest..newest."""
    lf, lblk, t = _tokens(case)
    ring, b = case["ring"], case["block"]
    row = torch.arange(t, device="cuda")
    slot = torch.where(row < lf, 0, 1 + (row - lf) // lblk)
    rank = torch.where(slot < 3, slot, 3 + (slot - 3 - (b - ring + 1)) % ring)
    inside = torch.where(row < lf, row, (row - lf) % lblk)
    kf = torch.where(slot == 0, 0, 1 + 3 * (rank - 1)) * lf + inside
    qf = (1 + 3 * (1 + ring)) * lf + torch.arange(lblk, device="cuda")
    valid = ((case["mask"] >> slot) & 1).bool()
    if case["rope"] == 1:
        return kf[:, None], qf[:, None], valid
    gw = case["gw"]
    kp, qp = (torch.stack([p // lf, p % lf // gw, p % gw], -1) for p in (kf, qf))
    return kp, qp, valid


def _probs(st):
    """P [H][Lq][T], lse [H][Lq] and the rotated q, k (head-major), in 32 bits."""
    case = st["case"]
    q = _turn(st["q"], _angles(case, st["qpos"])[:, None, :]).transpose(0, 1)
    k = _turn(st["k"], _angles(case, st["kpos"]))
    s = torch.matmul(q, k.transpose(1, 2)) / math.sqrt(case["dim"])
    s = s.masked_fill_(~st["valid"], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    s = s.sub_(m).exp_()
    total = s.sum(-1, keepdim=True)
    p = s.div_(torch.where(total > 0, total, 1.0))
    return p, (m + torch.log(total)).squeeze(-1), q, k


def _backward(st):
    case = st["case"]
    p, _, q, k = _probs(st)
    do = st["d_out"].float().transpose(0, 1)
    dv = torch.matmul(p.transpose(1, 2), do)
    ds = torch.matmul(do, st["v"].float().transpose(1, 2))
    delta = (p * ds).sum(-1, keepdim=True)
    ds = ds.sub_(delta).mul_(p).mul_(1 / math.sqrt(case["dim"]))
    dq = _turn(torch.matmul(ds, k).transpose(0, 1), -_angles(case, st["qpos"])[:, None, :])
    dk = _turn(torch.matmul(ds.transpose(1, 2), q), -_angles(case, st["kpos"]))
    return dict(dq=dq.bfloat16(), dk=dk.bfloat16(), dv=dv.bfloat16())


# ------------------------------------------------------------------------------------------
# in 64 bits, from the definitions
# ------------------------------------------------------------------------------------------

def _rotation(case, pos):
    """Complex unit numbers e^(i angle) [n, d/2] of positions given as rows of axis values."""
    columns = []
    for axis, da in enumerate(_rope_split(case)):
        for j in range(da // 2):
            columns.append(pos[:, axis].double() / BASE ** (2.0 * j / da))
    a = torch.stack(columns, 1)
    return torch.polar(torch.ones_like(a), a)


def _complex(x):
    return torch.view_as_complex(x.double().reshape(*x.shape[:-1], -1, 2).contiguous())


def _real(z):
    return torch.view_as_real(z).flatten(-2)


def exact(case, seed):
    st = prepare(case, seed)
    d, page = case["dim"], case.get("page")
    if case["op"] == "append":
        k_pages, v_pages = st["k_pages"].double(), st["v_pages"].double()
        q_rot = torch.empty_like(st["q_rot"], dtype=torch.float64)
        new, lens = _append_plan(case)
        at = 0
        for s, (n, length) in enumerate(zip(new, lens)):
            pos = torch.arange(length - n, length, device="cuda")
            if case["rope"] == 1:
                grid = pos[:, None]
            else:
                f, r = pos // (GRID * GRID), pos % (GRID * GRID)
                grid = torch.stack([f, r // GRID, r % GRID], 1)
            turn = _rotation(case, grid)[:, None, :]
            pages, rows = st["table"][s].long()[pos // page], pos % page
            k_pages[pages, :, rows] = _real(_complex(st["k"][at:at + n]) * turn)
            v_pages[pages, :, rows] = st["v"][at:at + n].double()
            q_rot[at:at + n] = _real(_complex(st["q"][at:at + n]) * turn)
            at += n
        return dict(k_pages=k_pages, v_pages=v_pages, q_rot=q_rot)
    if case["op"] == "decode":
        lens = _spread(case["min_len"], case["max_len"], case["n_seqs"])
        group = case["heads"] // case["kv_heads"]
        out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(st["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
        for s, length in enumerate(lens):
            tok = torch.arange(length, device="cuda")
            if case["window"]:
                tok = tok[(tok < case["sink"]) | (tok >= length - case["window"])]
            pages, rows = st["table"][s].long()[tok // page], tok % page
            k = st["k_pages"][pages, :, rows].double()
            v = st["v_pages"][pages, :, rows].double()
            for g in range(case["kv_heads"]):
                heads = slice(g * group, (g + 1) * group)
                score = st["q"][s, heads].double() @ k[:, g].T / math.sqrt(d)
                lse[s, heads] = torch.logsumexp(score, -1)
                out[s, heads] = torch.softmax(score, -1) @ v[:, g]
        return dict(out=out, lse=lse)
    qt, kt = _rotation(case, st["qpos"]), _rotation(case, st["kpos"][st["valid"]])
    dq = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    dk = torch.zeros(st["k"].shape, dtype=torch.float64, device="cuda")
    dv = torch.zeros(st["v"].shape, dtype=torch.float64, device="cuda")
    if not bool(st["valid"].any()):
        return dict(dq=dq, dk=dk, dv=dv)
    for head in range(case["heads"]):
        q = _real(_complex(st["q"][:, head]) * qt)
        k = _real(_complex(st["k"][head][st["valid"]]) * kt)
        v, do = st["v"][head][st["valid"]].double(), st["d_out"][:, head].double()
        p = torch.softmax(q @ k.T / math.sqrt(d), -1)
        dp = do @ v.T
        ds = p * (dp - (dp * p).sum(-1, keepdim=True)) / math.sqrt(d)
        dv[head, st["valid"]] = p.T @ do
        dq[:, head] = _real(_complex(ds @ k) * qt.conj())
        dk[head, st["valid"]] = _real(_complex(ds.T @ q) * kt.conj())
    return dict(dq=dq, dk=dk, dv=dv)
