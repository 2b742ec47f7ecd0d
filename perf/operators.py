"""Workloads of the paged serving step: page tables and slot maps, the append of new
tokens to paged compressed caches, and attention of drafted token trees over them.

A case names an operator (`op`) and its sizes.  `run` computes it in elementary torch
operations, or with the library's calls where `own` is true; `exact` restates the
definition in 64 bits, one sequence at a time.

  tables   pages of every sequence taken from / given back to the free list as its
           length goes from t_old to t_new, then the cache slot of every new token
  append   the new tokens of every sequence: raw-state ring, rotated window rows and the
           compressed entries that leave the window, in the cache's format
  tree     attention of the drafted nodes of every sequence over its compressed entries
           (all of them, or each node's selected ones), window rows and drafted ancestors
"""
import math
import random

import torch

own = False

W, D, ROPE, BASE = 128, 512, 64, 10000.0
BF16, FP8, FP4, FP8R = 0, 1, 2, 3
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step of a serving batch: a few accepted tokens per sequence, a page now and then
        dict(name="tables_step", op="tables", batch=32, stride=4, page=256, t=131072, new=4, kind="step"),
        # prompts admitted and finished requests released in one step, ragged up to 65536 tokens
        dict(name="tables_prompts", op="tables", batch=48, stride=4, page=64, t=65536, new=65536, kind="prompts"),
        # accepted tokens of a verification step, c4a layer
        dict(name="append_step_c4a", op="append", batch=32, stride=4, fmt=BF16, page=256, t=131072, new=8, kind="step"),
        # the same for a c128a layer with an fp8 cache and an odd batch
        dict(name="append_step_c128a_fp8", op="append", batch=61, stride=128, fmt=FP8, page=128, t=262144, new=5, kind="step"),
        # whole prompts, ragged
        dict(name="append_prompts_c4a", op="append", batch=6, stride=4, fmt=BF16, page=64, t=16384, new=16384, kind="prompts"),
        dict(name="append_prompts_c128a_fp8", op="append", batch=4, stride=128, fmt=FP8, page=64, t=40000, new=40000,
             kind="prompts"),
        # one short conversation with a handful of drafted tokens: latency
        dict(name="tree_one_short", op="tree", batch=1, heads=64, nodes=5, t=4099, stride=128, fmt=BF16, page=64, k=0),
        # a serving batch of the dense (c128a) layer
        dict(name="tree_b8", op="tree", batch=8, heads=64, nodes=16, t=131072, stride=128, fmt=BF16, page=128, k=0),
        # a quarter of the heads (tensor-parallel shard), fp8 cache, odd batch
        dict(name="tree_b13_h16_fp8", op="tree", batch=13, heads=16, nodes=31, t=262144, stride=128, fmt=FP8, page=256, k=0),
        # the longest contexts with wide trees
        dict(name="tree_long", op="tree", batch=4, heads=64, nodes=64, t=1 << 20, stride=128, fmt=BF16, page=256, k=0),
        # the sparse (c4a) layer: every node has its own selected entries
        dict(name="tree_sparse", op="tree", batch=8, heads=64, nodes=12, t=131072, stride=4, fmt=BF16, page=256, k=512),
        dict(name="tree_sparse_fp8", op="tree", batch=16, heads=64, nodes=7, t=40000, stride=4, fmt=FP8, page=64, k=512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "tree", "tree"])
    page = rng.choice([64, 128, 256])
    stride = rng.choice([4, 128])
    if op == "tables":
        kind = rng.choice(["step", "prompts"])
        batch = _log(rng, 1, 256)
        t = _log(rng, 200, (1 << 21) // batch)
        return dict(op=op, batch=batch, stride=stride, page=page, t=t, new=t if kind == "prompts" else rng.randint(1, 16), kind=kind)
    if op == "append":
        kind = rng.choice(["step", "prompts", "chunk"])
        fmt = rng.choice([BF16, FP8, FP8R])
        if kind == "step":
            return dict(op=op, batch=_log(rng, 1, 128), stride=stride, fmt=fmt, page=page, t=_log(rng, 200, 262144),
                        new=rng.randint(1, 16), kind=kind)
        batch = _log(rng, 1, 8)
        t = _log(rng, 300, 98304 // batch)
        return dict(op=op, batch=batch, stride=stride, fmt=fmt, page=page, t=t,
                    new=t if kind == "prompts" else rng.randint(18, 200), kind=kind)
    heads, nodes = rng.choice([8, 16, 20, 32, 64]), _log(rng, 1, 64)
    if rng.random() < 0.4:
        stride, k = 4, rng.choice([64, 200, 512])
        batch = _log(rng, 1, max(1, 160 // nodes))
        return dict(op=op, batch=batch, heads=heads, nodes=nodes, t=_log(rng, 40, 131072), stride=4, fmt=rng.choice([BF16, FP8, FP4, FP8R]),
                    page=page, k=k)
    t = _log(rng, 40, 1 << 20)
    most = 4 * 64 * 64 * (8192 + 200) // (heads * nodes * (t // 128 + 200))
    return dict(op=op, batch=_log(rng, 1, max(1, min(most, 24))), heads=heads, nodes=nodes, t=t, stride=128,
                fmt=rng.choice([BF16, FP8, FP4, FP8R]), page=page, k=0)


LOOKAHEAD = 16  # most drafted tokens an appended state prepares entries for (tables and append)


# ------------------------------------------------------------------ inputs
def _sizes(case):
    """Lengths go by the case alone (every seed's outputs have the same shapes); pages and values by the seed."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _lengths(case, rng):
    """(t_old, t_new) per sequence."""
    b, t, new, kind = case["batch"], case["t"], case["new"], case["kind"]
    if kind == "step":
        old = [max(0, t - rng.randint(0, t // 2)) for _ in range(b)]
        return old, [o + rng.randint(1, new) for o in old]
    if kind == "chunk":
        old = [rng.randint(0, t) for _ in range(b)]
        return old, [o + rng.randint(max(1, new // 2), new) for o in old]
    old = [0] * b
    new_ = [rng.randint((t + 1) // 2, t) for _ in range(b)]
    if case["op"] == "tables":  # every fourth request ends instead of starting
        for i in range(3, b, 4):
            old[i], new_[i] = new_[i], 0
    return old, new_


def _rows(t, stride, look=0):
    """Cache rows of a sequence of t tokens (stride 0: the window cache)."""
    return min(t, W) if stride == 0 else max(0, (t + look - W) // stride)


def _pages(counts, page, rng, spare=0, width=None):
    """A shuffled page assignment: (table, free pages behind it, pages in the pool)."""
    need = [-(-c // page) for c in counts]
    total = sum(need) + spare
    perm = list(range(total))
    rng.shuffle(perm)
    width = max(1, width or 0, *need)
    table, o = [], 0
    for m in need:
        table.append(perm[o:o + m] + [-1] * (width - m))
        o += m
    return table, perm[o:], total


def _dev(x, dtype):
    return torch.tensor(x, dtype=dtype, device="cuda")


def _fp8_rows(rows, dim, g):
    x = torch.randn(rows, dim, generator=g, device="cuda")
    s = x.abs().amax(1) / 448
    return (x / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8), s


def _cache_rows(rows, fmt, g):
    """Random cache rows of a format: (codes, scales)."""
    rows = max(rows, 1)
    if fmt == BF16:
        return torch.randn(rows, D, generator=g, device="cuda", dtype=torch.bfloat16), None
    if fmt == FP8:
        return _fp8_rows(rows, D, g)
    if fmt == FP8R:
        body, s = _fp8_rows(rows, D - ROPE, g)
        rot = torch.randn(rows, ROPE, generator=g, device="cuda", dtype=torch.bfloat16)
        return torch.cat([body, rot.view(torch.uint8)], 1), s
    codes = torch.randint(0, 256, (rows, D // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.rand(rows, D // 16, generator=g, device="cuda") * 0.3 + 0.2).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, s


def _empty_rows(rows, fmt):
    rows = max(rows, 1)
    if fmt == BF16:
        return torch.zeros(rows, D, device="cuda", dtype=torch.bfloat16), None
    width = {FP8: D, FP4: D // 2, FP8R: D + ROPE}[fmt]
    codes = torch.zeros(rows, width, device="cuda", dtype=torch.uint8)
    if fmt == FP4:
        return codes, torch.zeros(rows, D // 16, device="cuda", dtype=torch.uint8)
    return codes, torch.ones(rows, device="cuda")


def prepare(case, seed):
    g, rng = _gen(seed), random.Random(seed)
    s = dict(case=case)
    if case["op"] == "tree":
        _prepare_tree(case, s, g, rng)
    else:
        old, new = _lengths(case, _sizes(case))
        b, stride, page = case["batch"], case["stride"], case["page"]
        # a few tokens of head room: a captured step takes up to `new` tokens per sequence
        total = sum(max(0, y - x) for x, y in zip(old, new))
        cap = total if case["op"] == "append" else total + 5
        s.update(t_old=_dev(old, torch.int64), t_new=_dev(new, torch.int64), t_max=max(old + new), cap=cap)
        held = [_rows(t, stride, LOOKAHEAD) for t in (old if case["op"] == "tables" else new)]
        most = max(_rows(max(o, n), stride, LOOKAHEAD) for o, n in zip(old, new))
        grow = sum(max(0, -(-_rows(n, stride, LOOKAHEAD) // page) - -(-_rows(o, stride, LOOKAHEAD) // page))
                   for o, n in zip(old, new)) if case["op"] == "tables" else 0
        table, free, pool = _pages(held, page, rng, grow + 7, -(-most // page) + 1)
        wt, _, wpool = _pages([W] * b, page, rng)
        s.update(table=_dev(table, torch.int32), pool=pool, win_table=_dev(wt, torch.int32), win_pool=wpool)
        s["free"] = _dev(free + [0] * (pool - len(free)), torch.int32)
        s["count"] = _dev([len(free)], torch.int64)
        if case["op"] == "append":
            fmt, taps = case["fmt"], 8 if stride == 4 else 128
            s["max_new"] = max(y - x for x, y in zip(old, new))
            s["w"] = torch.softmax(torch.randn(taps, D, generator=g, device="cuda"), 0)
            s["states"] = torch.randn(cap, D, generator=g, device="cuda", dtype=torch.bfloat16)
            s["ring0"] = torch.randn(b, W + taps, D, generator=g, device="cuda", dtype=torch.bfloat16)
            s["ring"] = s["ring0"].clone()
            s["comp"] = _empty_rows(pool * page, fmt)
            s["win"] = _empty_rows(wpool * page, fmt)
            plan = _slots_plain(s, case)  # the step's slot map, as the caller's plan gave it
            s.update(zip(("cu", "seq", "pos", "win_slot", "comp_slot"), plan))
    if own:
        _prepare_own(s, case)
    return s


def _prepare_tree(case, s, g, rng):
    b, m, t, stride, fmt, page = (case[x] for x in ("batch", "nodes", "t", "stride", "fmt", "page"))
    size = _sizes(case)
    ts = [max(0, t - size.randint(0, t // 4)) for _ in range(b)]
    ms = [size.randint((m + 1) // 2, m) for _ in range(b)]
    ts[0], ms[0] = t, m
    parents = []
    for mb in ms:  # drafted trees: mostly chains that branch now and then
        parents += [-1 if j == 0 else max(-1, j - 1 - min(rng.randint(0, 6), rng.randint(0, 6))) for j in range(mb)]
    total = sum(ms)
    held = [_rows(x, stride, mb) for x, mb in zip(ts, ms)]
    table, _, pool = _pages(held, page, rng)
    wt, _, wpool = _pages([W] * b, page, rng)
    cu = [0]
    for mb in ms:
        cu.append(cu[-1] + mb)
    s.update(t_seq=_dev(ts, torch.int64), t_max=t, cu=_dev(cu, torch.int32), parent=_dev(parents, torch.int32),
             table=_dev(table, torch.int32), win_table=_dev(wt, torch.int32), pool=pool, win_pool=wpool, total=total)
    s["q"] = torch.randn(total, case["heads"], D, generator=g, device="cuda", dtype=torch.bfloat16)
    s["comp"] = _cache_rows(pool * page, fmt, g)
    s["win"] = _cache_rows(wpool * page, fmt, g)
    s["draft"] = _cache_rows(total, fmt, g)
    s["n_max"], s["idx"] = max(held), None
    if case["k"]:  # ascending entries below every node's own count, -1 behind them
        n = _dev([_rows(x, stride) for x, mb in zip(ts, ms) for _ in range(mb)], torch.int64)
        pick = (torch.rand(total, case["k"], generator=g, device="cuda", dtype=torch.float64) * n[:, None]).long()
        pick = pick.sort(1).values
        again = torch.zeros_like(pick, dtype=torch.bool)
        again[:, 1:] = pick[:, 1:] == pick[:, :-1]
        pick = torch.where(again | (n[:, None] == 0), n.max() + 1, pick).sort(1).values
        s["idx"] = torch.where(pick > n.max(), -1, pick).to(torch.int32)


def _prepare_own(s, case):
    """What a serving program keeps from step to step: descriptors, output buffers and workspaces."""
    import compressed_sparse_kv_b200 as K
    fmt = case.get("fmt", BF16)
    comp, win = s.get("comp", (s["table"], None)), s.get("win", (s["win_table"], None))
    if case["op"] == "tables":
        comp = win = (torch.empty(1, device="cuda"), None)
    s["comp_c"] = K.PagedCache(fmt, comp[0], s["table"], case["page"], comp[1])
    s["win_c"] = K.PagedCache(fmt, win[0], s["win_table"], case["page"], win[1])
    if case["op"] == "tree":
        s["draft_c"] = K.Cache(fmt, s["draft"][0][None], None if s["draft"][1] is None else s["draft"][1][None])
        s["out"] = torch.empty(s["q"].shape, dtype=torch.bfloat16, device="cuda")
        s["ws"] = K.new_workspace(K.tree_decode_paged_workspace_bytes(
            case["batch"], case["heads"], case["nodes"], s["total"], s["t_max"], W, case["stride"], case["k"] if s["idx"] is not None else None))
        return
    s["ws"] = K.new_workspace(K.paged_step_workspace_bytes(case["batch"]))
    if case["op"] == "tables":
        s["comp_c"] = K.PageTable(s["table"], case["page"], s["pool"])
        s["win_c"] = K.PageTable(s["win_table"], case["page"], s["win_pool"])
        s["count_out"] = torch.empty(1, dtype=torch.int64, device="cuda")
        s["slots"] = K.new_slot_map(case["batch"], s["cap"])
    else:
        s["slots"] = K.SlotMap(*(s[x] for x in ("cu", "seq", "pos", "win_slot", "comp_slot")))


# ------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    if case["op"] == "tables":
        return _tables_own(s, case) if own else _tables_plain(s, case)
    if case["op"] == "append":
        if case["kind"] == "chunk":  # the ring is overwritten by the chunk: every pass starts from the same one
            s["ring"].copy_(s["ring0"])
        if own:
            _append_own(s, case)
        else:
            _append_plain(s, case)
        return _append_out(s, case)
    return _tree_own(s, case) if own else _tree_plain(s, case)


def _tables_own(s, case):
    import compressed_sparse_kv_b200 as K
    K.block_table_update(s["t_old"], s["t_new"], s["comp_c"], s["free"], s["count"], s["t_max"], window=W,
                         stride=case["stride"], lookahead=LOOKAHEAD, free_count_out=s["count_out"], ws=s["ws"])
    m = K.slot_map(s["t_old"], s["t_new"], s["comp_c"], s["win_c"], s["cap"], s["t_max"], window=W,
                   stride=case["stride"], lookahead=LOOKAHEAD, out=s["slots"], ws=s["ws"])
    return dict(table=s["table"], free=s["free"], count=s["count_out"], cu=m.cu, seq=m.seq, pos=m.pos,
                win_slot=m.win_slot, comp_slot=m.comp_slot)


def _append_own(s, case):
    import compressed_sparse_kv_b200 as K
    K.append_paged(s["states"], s["w"], s["slots"], s["ring"], s["win_c"], s["comp_c"], stride=case["stride"],
                   window=W, lookahead=LOOKAHEAD, max_new=s["max_new"], ws=s["ws"])


def _tree_own(s, case):
    import compressed_sparse_kv_b200 as K
    return K.tree_decode_paged(s["q"], s["comp_c"], s["win_c"], s["draft_c"], s["cu"], s["parent"], s["t_seq"],
                               s["t_max"], case["nodes"], window=W, stride=case["stride"], idx=s["idx"],
                               out=s["out"], ws=s["ws"])


def _append_out(s, case):
    """The updated state; 8-bit codes as the values they stand for beside their scales."""
    out = dict(ring=s["ring"])
    for name in ("comp", "win"):
        codes, scales = s[name]
        if case["fmt"] == BF16:
            out[name] = codes
            continue
        body = codes if case["fmt"] == FP8 else codes[:, :D - ROPE]
        out[name] = body.view(torch.float8_e4m3fn)
        out[name + "_scale"] = scales
        if case["fmt"] == FP8R:
            out[name + "_rope"] = codes.view(torch.bfloat16)[:, (D - ROPE) // 2:]
    return out


# ------------------------------------------------------------------ plain forms
def _rows_t(t, stride):
    """_rows of a tensor of lengths."""
    return (t - W).clamp(min=0) // stride


def _tables_plain(s, case):
    t_old, t_new, table, free, count = (s[x] for x in ("t_old", "t_new", "table", "free", "count"))
    page, cap = case["page"], free.shape[0]
    old = (_rows_t(t_old + LOOKAHEAD, case["stride"]) + page - 1) // page
    new = (_rows_t(t_new + LOOKAHEAD, case["stride"]) + page - 1) // page
    rel, add = (old - new).clamp(min=0), (new - old).clamp(min=0)
    j = torch.arange(table.shape[1], device=table.device)[None]
    # pages given back go behind the free ones, in order of sequence and row
    rank = count + (rel.cumsum(0) - rel)[:, None] + j - new[:, None]
    back = (j >= new[:, None]) & (j < old[:, None])
    grown = torch.cat([free, free.new_zeros(1)])
    grown.scatter_(0, torch.where(back, rank, cap).reshape(-1), table.reshape(-1))
    # new pages come from the end of the free ones
    take = count + rel.sum() - 1 - ((add.cumsum(0) - add)[:, None] + j - old[:, None])
    want = (j >= old[:, None]) & (j < new[:, None])
    page_of = torch.where(take >= 0, grown[take.clamp(0, cap - 1)], -1)
    table = torch.where(want, page_of, table)
    count_out = (count + rel.sum() - add.sum()).clamp(min=0)
    cu, seq, pos, win_slot, comp_slot = _slots_plain(dict(s, table=table), case)
    return dict(table=table, free=grown[:cap], count=count_out, cu=cu, seq=seq, pos=pos, win_slot=win_slot, comp_slot=comp_slot)


def _slots_plain(s, case):
    """Sequence, position and the window and compressed slots of every new token."""
    t_old, t_new, stride, page = s["t_old"], s["t_new"], case["stride"], case["page"]
    n = (t_new - t_old).clamp(min=0)
    cu = torch.cat([n.new_zeros(1), n.cumsum(0)])
    i = torch.arange(s["cap"], device=n.device)
    seq = torch.searchsorted(cu[1:], i, right=True)
    real = seq < n.shape[0]
    b = seq.clamp(max=n.shape[0] - 1)
    pos = t_old[b] + i - cu[b]

    def slot(table, row):
        pg = table[b, (row // page).clamp(0, table.shape[1] - 1)].long()
        return torch.where(pg >= 0, pg * page + row % page, -1)

    w = torch.where(pos >= t_new[b] - W, slot(s["win_table"], pos % W), -1)
    e1, e0 = _rows_t(pos + 1 + LOOKAHEAD, stride), _rows_t(pos + LOOKAHEAD, stride)
    c = torch.where(e1 > e0, slot(s["table"], e0), -1)
    none = torch.full_like(pos, -1)
    ints = [torch.where(real, x, none).to(torch.int32) for x in (seq, w, c)]
    return cu.to(torch.int32), ints[0], torch.where(real, pos, none), ints[1], ints[2]


def _rotate(x, pos):
    """Rotary pairs of the last ROPE channels of x [..., D] (fp32) by pos * theta_m."""
    m = torch.arange(ROPE // 2, device=x.device, dtype=torch.float64)
    a = pos.double()[..., None] * BASE ** (-2 * m / ROPE)
    c, sn = a.cos().to(x.dtype), a.sin().to(x.dtype)
    p, q = x[..., D - ROPE::2], x[..., D - ROPE + 1::2]
    return torch.cat([x[..., :D - ROPE], torch.stack([p * c - q * sn, p * sn + q * c], -1).flatten(-2)], -1)


def _store(cache, slot, x, fmt):
    """Rows x (fp32) into the cache rows `slot` (negative: dropped)."""
    keep = slot >= 0
    x, slot = x[keep], slot[keep].long()
    codes, scales = cache
    if fmt == BF16:
        codes[slot] = x.to(torch.bfloat16)
        return
    body = x if fmt == FP8 else x[:, :D - ROPE]
    top = body.abs().amax(1)
    sc = torch.where(top > 0, top / 448, torch.ones_like(top))
    q = (body / sc[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    if fmt == FP8R:
        q = torch.cat([q, x[:, D - ROPE:].to(torch.bfloat16).view(torch.uint8)], 1)
    codes[slot] = q
    scales[slot] = sc.to(scales.dtype)


def _append_plain(s, case):
    stride, ring, x, w, fmt = case["stride"], s["ring"], s["states"], s["w"], case["fmt"]
    seq, pos, cu = s["seq"].long(), s["pos"], s["cu"].long()
    taps, r = w.shape[0], ring.shape[1]
    t_old = pos[cu[:-1].clamp(max=pos.shape[0] - 1)]
    t_new = t_old + cu[1:] - cu[:-1]
    emit = (s["comp_slot"] >= 0).nonzero()[:, 0]
    b, first = seq[emit], pos[emit] + 1 + LOOKAHEAD - W - taps
    p = first[:, None] + torch.arange(taps, device=x.device)[None]  # positions of the taps
    fresh = (p >= t_old[b][:, None]) & (p >= 0)
    rows = torch.where(fresh[..., None], x[(cu[b][:, None] + p - t_old[b][:, None]).clamp(0, x.shape[0] - 1)],
                       ring[b[:, None], p.clamp(min=0) % r])
    rows = torch.where((p >= 0)[..., None], rows, 0)
    entry = (rows.float() * w[None]).sum(1)
    at = first + taps - stride  # position of the entry's block
    _store(s["comp"], s["comp_slot"][emit], _rotate(entry, at), fmt)
    _store(s["win"], s["win_slot"], _rotate(x.float(), pos), fmt)
    keep = (pos >= t_new[seq] - r).nonzero()[:, 0]
    ring[seq[keep], pos[keep] % r] = x[keep]


def _values(cache, at, fmt):
    """fp32 values of the cache rows `at`."""
    codes, scales = cache
    c = codes[at]
    if fmt == BF16:
        return c.float()
    if fmt == FP4:
        lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=c.device)
        v = torch.stack([lut[(c & 15).long()], lut[(c >> 4).long()]], -1).flatten(-2)
        return v * scales[at].view(torch.float8_e4m3fn).float().repeat_interleave(16, -1)
    body = (c if fmt == FP8 else c[..., :D - ROPE].contiguous()).view(torch.float8_e4m3fn).float() * scales[at][..., None]
    if fmt == FP8:
        return body
    return torch.cat([body, c[..., D - ROPE:].contiguous().view(torch.bfloat16).float()], -1)


def _attend(q, rows, seen):
    """softmax(q . rows / sqrt(D)) over the rows that are seen, times the rows; zero where none is."""
    x = (q @ rows.transpose(-1, -2)) * D ** -0.5
    x = torch.where(seen, x, -torch.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top > -torch.inf, top, 0))
    return (p @ rows) / p.sum(-1, keepdim=True).clamp(min=1e-30)


def _tree_plain(s, case):
    h, m, stride, fmt, page = (case[x] for x in ("heads", "nodes", "stride", "fmt", "page"))
    cu, t, dev, total = s["cu"].long(), s["t_seq"], s["q"].device, s["total"]
    b = cu.shape[0] - 1
    i = torch.arange(total, device=dev)
    seq = torch.searchsorted(cu[1:], i, right=True)
    node = i - cu[seq]
    # ancestors: paths of the parent matrix, (I - A)^-1 - I
    up = torch.zeros(b, m, m + 1, device=dev)
    up[seq, node, s["parent"].long() % (m + 1)] = 1
    eye = torch.eye(m, device=dev)
    anc = torch.linalg.solve_triangular(eye - up[..., :m], eye.expand(b, m, m).contiguous(), upper=False, unitriangular=True) - eye
    anc = anc > 0.5
    pos = t[:, None] + anc.sum(-1)  # [b, m] position of every node
    n = _rows_t(pos, stride)
    # window rows lie at position % W; a node sees those less than W behind it
    r = torch.arange(W, device=dev)[None]
    at = t[:, None] - 1 - (t[:, None] - 1 - r) % W
    there = r < t[:, None].clamp(max=W)
    wrow = s["win_table"].long().gather(1, (r // page).expand(b, W)) * page + r % page
    tail = torch.cat([torch.where(there[..., None], _values(s["win"], wrow.clamp(min=0), fmt), 0),
                      _values(s["draft"], (cu[:-1, None] + torch.arange(m, device=dev)).clamp(max=total - 1), fmt)], 1)
    near = torch.cat([there[:, None] & (at[:, None] >= pos[..., None] - W), anc], -1)
    if s["idx"] is None:
        e = torch.arange(max(s["n_max"], 1), device=dev)[None]
        pg = s["table"].long().gather(1, (e // page).expand(b, -1))
        have = e < n.amax(1, keepdim=True)
        comp = torch.where(have[..., None], _values(s["comp"], (pg * page + e % page).clamp(min=0), fmt), 0)
        q = torch.zeros(b, m, h, D, device=dev)
        q[seq, node] = s["q"].float()
        seen = torch.cat([e[:, None] < n[..., None], near], -1)
        seen = seen[:, :, None].expand(-1, -1, h, -1).reshape(b, m * h, -1)
        o = _attend(q.view(b, m * h, D), torch.cat([comp, tail], 1), seen).view(b, m, h, D)[seq, node]
    else:
        e = s["idx"].long()
        have = (e >= 0) & (e < n[seq, node][:, None])
        pg = s["table"].long()[seq[:, None], (e.clamp(min=0) // page).clamp(max=s["table"].shape[1] - 1)]
        comp = torch.where(have[..., None], _values(s["comp"], (pg * page + e % page).clamp(min=0), fmt), 0)
        o = _attend(s["q"].float(), torch.cat([comp, tail[seq]], 1), torch.cat([have, near[seq, node]], -1)[:, None])
    return _rotate(o, -pos[seq, node][:, None]).to(torch.bfloat16)


# ------------------------------------------------------------------ the definitions in 64 bits
def _turn(x, pos):
    """x [n, D] rotated at pos [n], as complex numbers."""
    theta = torch.pow(torch.tensor(BASE, dtype=torch.float64, device=x.device),
                      -torch.arange(0, ROPE, 2, dtype=torch.float64, device=x.device) / ROPE)
    z = torch.view_as_complex(x[:, D - ROPE:].reshape(x.shape[0], ROPE // 2, 2).contiguous())
    a = pos.double()[:, None] * theta[None]
    z = z * torch.polar(torch.ones_like(a), a)
    return torch.cat([x[:, :D - ROPE], torch.view_as_real(z).reshape(x.shape[0], ROPE)], 1)


def _decode64(cache, at, fmt):
    codes, scales = cache
    c = codes.index_select(0, at)
    if fmt == BF16:
        return c.double()
    sc = scales.index_select(0, at)
    if fmt == FP4:
        out = torch.empty(c.shape[0], D, dtype=torch.float64, device=c.device)
        for half, nib in ((0, c & 15), (1, c >> 4)):
            mag, exp = (nib & 1).double(), ((nib >> 1) & 3).double()
            v = torch.where(exp == 0, mag / 2, (1 + mag / 2) * 2 ** (exp - 1))
            out[:, half::2] = torch.where((nib & 8) > 0, -v, v)
        return (out.view(-1, D // 16, 16) * sc.view(torch.float8_e4m3fn).double()[..., None]).reshape(-1, D)
    k = D if fmt == FP8 else D - ROPE
    v = c[:, :k].contiguous().view(torch.float8_e4m3fn).double() * sc.double()[:, None]
    return v if fmt == FP8 else torch.cat([v, c[:, k:].contiguous().view(torch.bfloat16).double()], 1)


def _exact_tree(case, s):
    h, stride, fmt, page = case["heads"], case["stride"], case["fmt"], case["page"]
    cu, parent, ts = s["cu"].tolist(), s["parent"].tolist(), s["t_seq"].tolist()
    out = torch.empty(s["total"], h, D, dtype=torch.float64, device="cuda")

    def paged(cache, table, rows):
        return _decode64(cache, table.long()[rows // page] * page + rows % page, fmt)

    for b, t in enumerate(ts):
        lo, hi = cu[b], cu[b + 1]
        paths = []
        for j in range(hi - lo):
            up = parent[lo + j]
            paths.append([] if up < 0 else paths[up] + [up])
        draft = _decode64(s["draft"], torch.arange(lo, hi, device="cuda"), fmt)
        w = torch.arange(min(t, W), device="cuda")
        held = torch.tensor([max(p for p in range(max(0, t - W), t) if p % W == r) for r in range(min(t, W))], device="cuda")
        win = paged(s["win"], s["win_table"][b], w)
        n_all = _rows(t + max(len(p) for p in paths), stride)
        comp = paged(s["comp"], s["table"][b], torch.arange(n_all, device="cuda")) if s["idx"] is None else None
        for j, path in enumerate(paths):
            p = t + len(path)
            n = _rows(p, stride)
            if comp is None:
                e = s["idx"][lo + j].long()
                rows = paged(s["comp"], s["table"][b], e[(e >= 0) & (e < n)])
            else:
                rows = comp[:n]
            rows = torch.cat([rows, win[held >= p - W], draft[path]])
            if rows.shape[0] == 0:
                out[lo + j] = 0
                continue
            a = torch.softmax(s["q"][lo + j].double() @ rows.T / math.sqrt(D), 1) @ rows
            out[lo + j] = _turn(a, torch.full((h,), -p, device="cuda"))
    return out


def _exact_append(case, s):
    stride, fmt, page = case["stride"], case["fmt"], case["page"]
    old, new = s["t_old"].tolist(), s["t_new"].tolist()
    ring, w = s["ring0"].double(), s["w"].double()
    taps, r = w.shape[0], ring.shape[1]
    state = {}
    for name in ("comp", "win"):
        codes, scales = s[name]
        state[name] = [torch.zeros(codes.shape[0], D, dtype=torch.float64, device="cuda"),
                       None if scales is None else scales.double()]
    out_ring = ring.clone()
    lo = 0
    for b, (a, z) in enumerate(zip(old, new)):
        x = s["states"][lo:lo + z - a].double()
        lo += z - a
        past = [p for p in range(max(0, a - r), a)]
        hist = torch.zeros(taps + r + z - a, D, dtype=torch.float64, device="cuda")  # position p at index p - a + r + taps
        if past:
            hist[[p - a + r + taps for p in past]] = ring[b, [p % r for p in past]]
        hist[r + taps:] = x
        first, last = _rows(a, stride, LOOKAHEAD), _rows(z, stride, LOOKAHEAD)
        ent = torch.arange(first, last, device="cuda")
        acc = torch.zeros(last - first, D, dtype=torch.float64, device="cuda")
        for j in range(taps):
            p = ent * stride + stride - taps + j
            acc += torch.where((p >= 0)[:, None], hist[(p - a + r + taps).clamp(min=0)], 0) * w[j]
        near = torch.arange(max(a, z - W), z, device="cuda")
        for name, table, rows, vals, at in (("comp", s["table"], ent, acc, ent * stride),
                                            ("win", s["win_table"], near % W, x[near - a], near)):
            if rows.numel():
                slot = table[b].long()[rows // page] * page + rows % page
                vals, sc = _code64(_turn(vals, at), fmt)
                state[name][0][slot] = vals
                if sc is not None:
                    state[name][1][slot] = sc
        keep = torch.arange(max(a, z - r), z, device="cuda")
        out_ring[b, keep % r] = x[keep - a]
    out = dict(ring=out_ring)
    for name in ("comp", "win"):
        vals, scales = state[name]
        out[name] = vals if fmt != FP8R else vals[:, :D - ROPE]
        if fmt != BF16:
            out[name + "_scale"] = scales
        if fmt == FP8R:
            out[name + "_rope"] = vals[:, D - ROPE:]
    return out


def _code64(x, fmt):
    """The 8-bit values and scales that rows x round to."""
    if fmt == BF16:
        return x, None
    body = x if fmt == FP8 else x[:, :D - ROPE]
    sc = body.abs().amax(1) / 448
    sc = torch.where(sc > 0, sc, 1.0)
    q = (body / sc[:, None]).to(torch.float8_e4m3fn).double()
    return (q if fmt == FP8 else torch.cat([q, x[:, D - ROPE:]], 1)), sc


def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers
    s = prepare(case, seed)
    return _exact_tree(case, s) if case["op"] == "tree" else _exact_append(case, s)


# ------------------------------------------------------------------ what a pass cannot do without
def _row_bytes(fmt):
    return {BF16: 2 * D, FP8: D + 4, FP4: D // 2 + D // 16, FP8R: D + ROPE + 4}[fmt]


def work(case):
    b, stride = case["batch"], case["stride"]
    if case["op"] == "tree":
        h, m, t, k = case["heads"], case["nodes"], case["t"], case["k"]
        nodes = max(1.0, 0.75 * m * b)  # a sequence has between half and all of `nodes`, and t is ragged
        n = 0.875 * max(0, t - W) / stride
        near = min(t, W) + 0.5 * m
        if k:
            n = min(k, n)
            rows, pairs = nodes * n + b * near, nodes * (n + near)
        else:
            rows, pairs = b * (n + near), nodes * (n + near)
        return dict(bytes=rows * _row_bytes(case["fmt"]) + nodes * h * D * 4, flops=4 * D * h * pairs)
    if case["kind"] == "prompts":
        tokens = 0.75 * b * case["t"] * (0.75 if case["op"] == "tables" else 1)
    else:
        tokens = 0.75 * b * case["new"]
    entries = tokens / stride
    if case["op"] == "tables":
        # token: sequence, position and two slots written; a page read and written per page_rows entries
        return dict(bytes=tokens * 20 + entries / case["page"] * 8 + 24 * b, flops=10 * tokens)
    taps = 8 if stride == 4 else 128
    kept = min(tokens, W * b) if case["kind"] == "prompts" else tokens
    return dict(bytes=tokens * 2 * D + entries * _row_bytes(case["fmt"]) + kept * (_row_bytes(case["fmt"]) + 2 * D)
                + taps * D * 4 + (min(entries, b * 4.0) * taps * 2 * D if case["kind"] != "prompts" else 0),
                flops=2 * D * taps * entries + 6 * D * (entries + kept))
