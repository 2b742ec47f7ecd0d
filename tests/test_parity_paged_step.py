"""Block tables, slot maps and the paged append against the oracle."""
import numpy as np
import pytest
import torch

import compressed_sparse_kv_b200 as K
from oracle import formats as OF
from oracle import serving as S
from tests._serving import DEQUANT, FORMATS, ROW_BYTES

pytestmark = pytest.mark.gpu


def dev(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def step_case(seed, t_old, t_new, page, window, stride, lookahead, spare=0):
    """Tables that hold t_old, and a free list of what else t_new needs plus `spare` (may be negative)."""
    rng = np.random.default_rng(seed)
    rows = lambda ts: [S.cache_rows(t, window, stride, lookahead) for t in ts]  # noqa: E731
    o, n = ([-(-r // page) for r in rows(ts)] for ts in (t_old, t_new))
    width = max(1, *o, *n)
    more = max(0, sum(max(0, b - a) for a, b in zip(o, n)) + spare)
    perm = rng.permutation(sum(o) + more)
    table, at = [], 0
    for m in o:
        table.append([int(x) for x in perm[at:at + m]] + [-1] * (width - m))
        at += m
    return table, [int(x) for x in perm[at:]], len(perm)


CASES = [
    ([0], [1]), ([5], [5]), ([1000, 0, 700], [1001, 900, 0]), ([300] * 40, list(range(280, 320))),
    ([0] * 600, [200 + 7 * i % 900 for i in range(600)]), ([64 * i for i in range(513)], [64 * (512 - i) for i in range(513)]),
]


@pytest.mark.parametrize("page,window,stride,lookahead", [(64, 128, 4, 0), (64, 128, 4, 16), (64, 0, 1, 0),
                                                          (128, 128, 128, 5), (64, 200, 0, 0)])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_block_tables_equal_the_sequential_stack(case, page, window, stride, lookahead):
    t_old, t_new = CASES[case]
    table, free, pool = step_case(case, t_old, t_new, page, window, stride, lookahead, spare=3)
    want_t, want_f = S.block_table_update(t_old, t_new, table, free, page, window, stride, lookahead)
    pages = K.PageTable(dev(table), page, max(pool, 1))
    fl = dev(free + [-7] * (pool + 5 - len(free)))
    count, ws = dev([len(free)], torch.int64), K.new_workspace(K.paged_step_workspace_bytes(len(t_old)))
    kw = dict(t_max=max(t_old + t_new), window=window, stride=stride, lookahead=lookahead, ws=ws)
    old, new = dev(t_old, torch.int64), dev(t_new, torch.int64)
    for _ in range(2):      # with another word for the count the call can be repeated
        out = K.block_table_update(old, new, pages, fl, count, **kw)
        assert out.item() == len(want_f) and count.item() == len(free)
        assert fl[:len(want_f)].tolist() == want_f
        assert pages.table.tolist() == want_t
    K.block_table_update(old, new, pages, fl, count, free_count_out=count, **kw)
    assert count.item() == len(want_f) and pages.table.tolist() == want_t
    assert K.workspace_status(ws) == 0 and not ws.any()


def test_block_tables_flags():
    t_old, t_new = [0, 300, 0], [300, 0, 400]
    table, free, pool = step_case(1, t_old, t_new, 64, 0, 1, 0, spare=-6)
    want_t, want_f = S.block_table_update(t_old, t_new, table, free, 64, 0, 1)
    pages, ws = K.PageTable(dev(table), 64, pool), K.new_workspace(16)
    fl = dev(free + [0] * pool)
    call = lambda p, f, c, o=t_old, n=t_new: K.block_table_update(  # noqa: E731
        dev(o, torch.int64), dev(n, torch.int64), p, f, c, 400, window=0, stride=1, ws=ws)
    out = call(pages, fl, dev([len(free)], torch.int64))
    assert K.workspace_status(ws) == K.DEV_NO_PAGES and out.item() == 0 and pages.table.tolist() == want_t
    ws.zero_()      # a full free list: what does not fit is dropped
    assert call(K.PageTable(dev([[0] * 7, [1, 2, 3, 4, 5, 0, 0], [0] * 7]), 64, 9), dev([8, 7]), dev([2], torch.int64),
                n=[0, 0, 0]).item() == 2
    assert K.workspace_status(ws) == K.DEV_NO_PAGES
    ws.zero_()      # a page number outside the pool is not handed out
    p = K.PageTable(dev([[-1] * 7] * 3), 64, 9)
    call(p, dev([3, 99, 4]), dev([3], torch.int64), o=[0, 0, 0], n=[192, 0, 0])
    assert K.workspace_status(ws) == K.DEV_BAD_PAGE and p.table[0].tolist() == [4, -1, 3, -1, -1, -1, -1]
    ws.zero_()      # lengths and counts outside their range are clamped
    p = K.PageTable(dev([[-1] * 7] * 3), 64, 9)
    assert call(p, dev([3, 5, 4]), dev([77], torch.int64), o=[-5, 0, 0], n=[64, 0, 0]).item() == 2
    assert K.workspace_status(ws) == K.DEV_BAD_LENGTH and p.table[0, 0].item() == 4


@pytest.mark.parametrize("page,window,stride,lookahead", [(64, 128, 4, 0), (64, 128, 4, 16), (64, 0, 1, 0),
                                                          (128, 128, 128, 5), (64, 200, 3, 200)])
@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("room", [0, 7])
def test_slot_maps(case, page, window, stride, lookahead, room):
    t_old, t_new = CASES[case]
    table, _, pool = step_case(case, t_new, t_new, page, window, stride, lookahead)
    width = max(len(r) for r in table)
    most = max(1, -(-max(S.cache_rows(t, window, stride, lookahead) for t in t_old + t_new) // page))
    table = [r + [-1] * (max(width, most) - len(r)) for r in table]
    wt, _, wpool = step_case(case + 50, [window] * len(t_old), [window] * len(t_old), 64, window, 0, 0)
    want = S.slot_map(t_old, t_new, table, wt, page, 64, window, stride, lookahead)
    cap = want[0][-1] + room
    ws = K.new_workspace(16)
    m = K.slot_map(dev(t_old, torch.int64), dev(t_new, torch.int64), K.PageTable(dev(table), page, max(pool, 1)),
                   K.PageTable(dev(wt), 64, max(wpool, 1)) if window else None, cap, max(t_old + t_new), window=window,
                   stride=stride, lookahead=lookahead, ws=ws)
    assert K.workspace_status(ws) == 0
    assert m.cu.tolist() == want[0]
    for got, ref in zip((m.seq, m.pos, m.win_slot, m.comp_slot), want[1:]):
        assert got.tolist() == ref + [-1] * room


def test_slot_map_flags():
    ws = K.new_workspace(16)
    pt, wt = K.PageTable(dev([[0], [-1]]), 64, 1), K.PageTable(dev([[0, 5], [0, 1]]), 64, 2)
    m = K.slot_map(dev([100, 3], torch.int64), dev([140, 9], torch.int64), pt, wt, 20, 140, ws=ws)
    assert K.workspace_status(ws) == K.DEV_BAD_LENGTH | K.DEV_BAD_PAGE      # over the capacity; page 5 of 2
    assert m.cu.tolist() == [0, 20, 20] and m.win_slot[:20].tolist() == [-1] * 20 and m.seq.tolist() == [0] * 20
    ws.zero_()
    m = K.slot_map(dev([-3, 3], torch.int64), dev([2, 500], torch.int64), pt, wt, 160, 140, ws=ws)
    assert K.workspace_status(ws) & K.DEV_BAD_LENGTH and m.cu.tolist() == [0, 2, 139]


# ------------------------------------------------------------------ append
class Appender:
    """Paged caches of a few growing sequences and the oracle's copies of what they hold."""

    def __init__(self, seed, batch, fmt, stride, taps, window, lookahead, longest, page=64):
        self.rng = np.random.default_rng(seed)
        self.fmt, self.stride, self.window, self.lookahead, self.page = fmt, stride, window, lookahead, page
        w = self.rng.random((taps, 512)).astype(np.float32)
        self.w = w / w.sum(0)
        self.w_d = torch.from_numpy(self.w).cuda()
        self.hist = [np.zeros((0, 512)) for _ in range(batch)]
        rows = S.cache_rows(longest, window, stride, lookahead)
        per, wper = max(1, -(-rows // page)), max(1, -(-window // page))
        perm, wperm = self.rng.permutation(batch * per + 1), self.rng.permutation(batch * wper + 1)
        self.table = perm[:batch * per].reshape(batch, per).astype(np.int32)
        self.wtable = wperm[:batch * wper].reshape(batch, wper).astype(np.int32)

        def cache(table, pages):
            dt = torch.bfloat16 if fmt == K.BF16 else torch.uint8
            codes = torch.zeros(pages * page, ROW_BYTES[fmt] // dt.itemsize, dtype=dt, device="cuda")
            sc = None
            if fmt == K.FP4_E2M1_G16:
                sc = torch.zeros(pages * page, 32, dtype=torch.uint8, device="cuda")
            elif fmt != K.BF16:
                sc = torch.zeros(pages * page, device="cuda")
            return K.PagedCache(fmt, codes, torch.from_numpy(table).cuda(), page, sc)

        self.comp, self.win = cache(self.table, len(perm)), cache(self.wtable, len(wperm))
        self.ring = torch.zeros(batch, window + taps, 512, dtype=torch.bfloat16, device="cuda")
        self.want_c, self.want_w, self.want_r = {}, {}, {}
        self.ws = K.new_workspace(16)

    def step(self, counts, pad=0, max_new=None):
        old = [len(h) for h in self.hist]
        new = [o + c for o, c in zip(old, counts)]
        total = sum(counts)
        x = torch.from_numpy(self.rng.normal(size=(total + pad, 512)).astype(np.float32)).to(torch.bfloat16).cuda()
        xv, at = x.double().cpu().numpy(), 0
        for b, c in enumerate(counts):
            self.hist[b] = np.concatenate([self.hist[b], xv[at:at + c]])
            at += c
            win, ents, raw = S.append_rows(self.hist[b], old[b], new[b], self.w, self.window, self.stride, self.lookahead)
            slot = lambda t, r: int(t[b][r // self.page]) * self.page + r % self.page  # noqa: E731,B023
            self.want_w.update({slot(self.wtable, r): v for r, v in win.items()})
            self.want_c.update({slot(self.table, r): v for r, v in ents.items()})
            self.want_r.update({(b, r): v for r, v in raw.items()})
        kw = dict(window=self.window, stride=self.stride, lookahead=self.lookahead, ws=self.ws)
        m = K.slot_map(dev(old, torch.int64), dev(new, torch.int64), self.comp, self.win if self.window else None,
                       total + pad, max(new), **kw)
        K.append_paged(x, self.w_d, m, self.ring, self.win if self.window else None, self.comp, max_new=max_new, **kw)
        assert K.workspace_status(self.ws) == 0

    def check(self):
        ring = self.ring.double().cpu().numpy()
        for b in range(ring.shape[0]):
            for r in range(ring.shape[1]):
                assert np.array_equal(ring[b, r], self.want_r.get((b, r), np.zeros(512))), (b, r)
        taps = self.w.shape[0]
        for cache, want, terms in ((self.comp, self.want_c, taps), (self.win, self.want_w, 0)):
            codes = cache.codes.cpu()
            if self.fmt == K.BF16:
                got = codes.double().numpy()
            else:
                got = DEQUANT[self.fmt](codes.numpy(), cache.scales.cpu().numpy())
            for r in range(len(got)):
                if r not in want:
                    assert not np.any(got[r]), r                       # rows nothing was due for are left
                    continue
                ref = want[r]
                # fp32 sums of `terms` products of weights that add up to one, then the rotation's few roundings
                # and its angle to 2^-23 of a turn
                acc = (terms + 16) * 2.0 ** -24 * max(1.0, np.abs(np.stack(self.hist[0])).max())
                lim = np.full(512, acc)
                a = np.abs(ref)
                if self.fmt == K.BF16:
                    lim += a * 2.0 ** -8
                elif self.fmt == K.FP4_E2M1_G16:
                    g = a.reshape(32, 16).max(1)
                    s = np.repeat(np.maximum(g / 6, 2.0 ** -9), 16)     # E4M3 scale, half a step of 2^-4 (or 2^-10) off
                    y = a / s
                    lim += s * (1 + 2.0 ** -4) * np.where(y > 3.7, 1.0, np.where(y > 1.8, 0.5, 0.25)) + s * 2.0 ** -4
                else:
                    n = 512 if self.fmt == K.FP8_E4M3_ROW else 448
                    s = a[:n].max() / 448
                    lim[:n] += np.maximum(a[:n] * 2.0 ** -4, s * 2.0 ** -10) * (1 + 2.0 ** -10)
                    lim[n:] += a[n:] * 2.0 ** -8
                off = np.abs(got[r] - ref) - lim
                assert off.max() <= 0, (r, int(off.argmax()), got[r][off.argmax()], ref[off.argmax()], lim[off.argmax()])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("stride,taps", [(4, 8), (128, 128)])
@pytest.mark.parametrize("lookahead", [0, 16])
def test_append_prompts_then_steps(fmt, stride, taps, lookahead):
    a = Appender(7 + fmt + stride, 4, fmt, stride, taps, 128, lookahead, 1500)
    a.step([700, 129, 1, 300])
    a.step([1, 2, 17, 0], pad=5, max_new=17)        # a verification step: some tokens each
    for _ in range(6):
        a.step([1, 1, 1, 1], max_new=1)
    a.step([200, 0, 400, 3])                        # a chunk longer than the lookahead: two launches
    a.check()


@pytest.mark.parametrize("stride,taps,window,lookahead", [(1, 1, 0, 0), (3, 5, 7, 7), (5, 40, 33, 2), (2, 33, 64, 64)])
def test_append_other_shapes(stride, taps, window, lookahead):
    a = Appender(90 + taps, 3, K.BF16, stride, taps, window, lookahead, 900)
    for counts in ([90, 1, 40], [1, 0, 3], [2, 2, 1], [300, 5, 80], [1, 1, 1]):
        a.step(counts)
    a.check()


def test_append_equals_the_uniform_append():
    """One sequence, one token at a time, bf16: the rings and rows of dsv4kv_append (whose rotation is in fp64: one
    bf16 step apart at most)."""
    a = Appender(5, 1, K.BF16, 4, 8, 128, 0, 300, page=64)
    raw = torch.zeros(1, 136, 512, dtype=torch.bfloat16, device="cuda")
    win = torch.zeros(1, 128, 512, dtype=torch.bfloat16, device="cuda")
    comp = torch.zeros(1, 64, 512, dtype=torch.bfloat16, device="cuda")
    for t in range(300):
        a.step([1])
        K.append(torch.from_numpy(a.hist[0][-1:]).to(torch.bfloat16).cuda(), a.w_d, t, 4, 128, raw, win, comp)
    assert torch.equal(a.ring, raw)
    for cache, ref in ((a.comp, comp), (a.win, win)):
        i = torch.arange(43 if cache is a.comp else 128, device="cuda")
        rows = cache.codes[cache.table[0].long()[i // 64] * 64 + i % 64].double()
        ref = ref[0, :len(i)].double()
        assert torch.all((rows - ref).abs() <= 2.0 ** -7 * ref.abs() + 2.0 ** -30)


def test_append_flags_and_skips_bad_slots():
    a = Appender(6, 2, K.BF16, 4, 8, 128, 0, 300)
    a.step([200, 180])
    before = [x.clone() for x in (a.comp.codes, a.win.codes, a.ring)]
    x = torch.ones(4, 512, dtype=torch.bfloat16, device="cuda")

    def call(seq, pos, ws_, cs, cu=(0, 4, 4), max_new=4):
        a.ws.zero_()
        K.append_paged(x, a.w_d, K.SlotMap(dev(cu), dev(seq), dev(pos, torch.int64), dev(ws_), dev(cs)), a.ring, a.win,
                       a.comp, stride=4, ws=a.ws, max_new=max_new)
        return K.workspace_status(a.ws)

    none = [-1] * 4
    assert call([5, -2, 2, 9], [200, 201, 202, 203], none, none) == K.DEV_BAD_LENGTH
    assert call([0, 0, 0, 0], [-9, -8, -7, -6], none, none) == K.DEV_BAD_LENGTH
    assert call([0, 0, 0, 0], [200, 201, 202, 203], none, none, cu=(0, 9, 9)) == K.DEV_BAD_LENGTH
    assert call([0, 0, 0, 0], [200, 201, 202, 203], none, none, max_new=2) == K.DEV_BAD_LENGTH
    assert call([-1] * 4, [-1] * 4, none, none) == 0
    assert all(torch.equal(x, y) for x, y in zip(before, (a.comp.codes, a.win.codes, a.ring)))
    rows = a.comp.codes.shape[0]
    assert call([0, 0, 0, 0], [200, 201, 202, 203], [1 << 30, -5, -1, -1], [-1, rows, -1, -7]) == K.DEV_BAD_PAGE
    assert torch.equal(before[0], a.comp.codes) and torch.equal(before[1], a.win.codes)


def test_a_serving_loop_in_one_graph():
    """Tables, slots, append and tree attention as one captured step; every replay is checked against a decode of each
    node with its path appended (the oracle on the rows the caches hold)."""
    W, s, L, page, H, B, M = 128, 4, 16, 64, 16, 2, 4
    rng = np.random.default_rng(12)
    w = rng.random((8, 512)).astype(np.float32)
    w_d = torch.from_numpy(w / w.sum(0)).cuda()
    pool, wpool, cap = 16, 4, 2 * 200
    comp = K.PagedCache(0, torch.zeros(pool * page, 512, dtype=torch.bfloat16, device="cuda"),
                        torch.full((B, 6), -1, dtype=torch.int32, device="cuda"), page)
    win = K.PagedCache(0, torch.zeros(wpool * page, 512, dtype=torch.bfloat16, device="cuda"), dev([[2, 0], [1, 3]]), page)
    free, count = dev(list(range(pool))), dev([pool], torch.int64)
    t_old, t_new, t_max = dev([0, 0], torch.int64), dev([0, 0], torch.int64), 1200
    ring = torch.zeros(B, W + 8, 512, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros(cap, 512, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(B * M, H, 512, dtype=torch.bfloat16, device="cuda")
    draft = K.Cache(0, torch.zeros(1, B * M, 512, dtype=torch.bfloat16, device="cuda"))
    cu, parent = dev([0, M, 2 * M]), dev([-1, 0, 0, 2, -1, 0, 1, 2])
    out = torch.zeros(B * M, H, 512, device="cuda")
    slots = K.new_slot_map(B, cap)
    ws, ws_t = K.new_workspace(16), K.new_workspace(K.tree_decode_paged_workspace_bytes(B, H, M, B * M, t_max, W, s))

    def step():
        kw = dict(window=W, stride=s, lookahead=L, ws=ws)
        K.block_table_update(t_old, t_new, comp, free, count, t_max, free_count_out=count, **kw)
        K.slot_map(t_old, t_new, comp, win, cap, t_max, out=slots, **kw)
        K.append_paged(x, w_d, slots, ring, win, comp, **kw)
        K.tree_decode_paged(q, comp, win, draft, cu, parent, t_new, t_max, M, window=W, stride=s, out_fp32=True, out=out,
                            ws=ws_t)

    step()                                       # (nothing is appended yet: every length is zero)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    hist, t = [np.zeros((0, 512))] * B, [0, 0]
    for counts in ([190, 131], [3, 1], [1, 4], [2, 2], [0, 5]):
        t_old.copy_(dev(t, torch.int64))
        t = [a + c for a, c in zip(t, counts)]
        t_new.copy_(dev(t, torch.int64))
        n = sum(counts)
        x[:n] = torch.from_numpy(rng.normal(size=(n, 512)).astype(np.float32)).to(torch.bfloat16).cuda()
        xv = x[:n].double().cpu().numpy()
        hist = [np.concatenate([hist[0], xv[:counts[0]]]), np.concatenate([hist[1], xv[counts[0]:]])]
        q.copy_(torch.from_numpy(rng.normal(size=(B * M, H, 512)).astype(np.float32)))
        draft.codes.copy_(torch.from_numpy(rng.normal(size=(1, B * M, 512)).astype(np.float32)))
        g.replay()
        torch.cuda.synchronize()
        assert K.workspace_status(ws) == 0 and K.workspace_status(ws_t) == 0
        got = out.double().cpu().numpy()
        for b in range(B):
            wr, ents, _ = S.append_rows(hist[b], 0, t[b], w_d.double().cpu().numpy(), W, s, L)
            ents = OF.round_bf16(np.stack([ents[i] for i in range(len(ents))])) if ents else np.zeros((0, 512))
            wrows = OF.round_bf16(np.stack([wr[r] for r in range(min(t[b], W))]))
            lo = b * M
            ref = S.tree_decode(q[lo:lo + M].double().cpu().numpy(), ents, wrows,
                                draft.codes[0, lo:lo + M].double().cpu().numpy(), parent[lo:lo + M].tolist(), t[b], W, s)
            # bf16 weights and cache rows one bf16 step apart: 2^-8 of the rows' mean magnitude for either
            assert np.abs(got[lo:lo + M] - ref).max() <= 3 * 2.0 ** -8 * 2, (t, b)
            assert np.linalg.norm(got[lo:lo + M] - ref) <= 5e-3 * np.linalg.norm(ref)
    used = sum(-(-S.cache_rows(x, W, s, L) // page) for x in t)
    assert count.item() == pool - used


def test_a_pool_without_a_page():
    """No sequence is long enough for a compressed entry, nor has a page for one."""
    old, new = dev([0, 50], torch.int64), dev([9, 100], torch.int64)
    ws = K.new_workspace(K.paged_step_workspace_bytes(2))
    pages, wpages = K.PageTable(dev([[-1], [-1]]), 64, 0), K.PageTable(dev([[2, 0], [1, 3]]), 64, 4)
    count = dev([0], torch.int64)
    K.block_table_update(old, new, pages, dev([]), count, t_max=100, window=128, stride=4, lookahead=16,
                         free_count_out=count, ws=ws)
    m = K.slot_map(old, new, pages, wpages, 64, 100, window=128, stride=4, lookahead=16, ws=ws)
    assert K.workspace_status(ws) == 0 and count.item() == 0 and pages.table.tolist() == [[-1], [-1]]
    assert m.cu.tolist() == [0, 9, 59]
    want = [128 + i for i in range(9)] + [64 + p if p < 64 else 192 + p - 64 for p in range(50, 100)]
    assert m.win_slot[:59].tolist() == want and torch.all(m.comp_slot[:59] < 0)


def test_the_largest_batch():
    """4096 sequences, most of them idle, from tables to cache rows."""
    B, W, page = 4096, 128, 64
    rng = np.random.default_rng(8)
    t_old = rng.integers(0, 600, B)
    t_new = t_old + np.where(rng.random(B) < 0.1, rng.integers(1, 40, B), 0)
    table, free, pool = step_case(8, t_old.tolist(), t_new.tolist(), page, W, 4, 0)
    want_t, want_f = S.block_table_update(t_old.tolist(), t_new.tolist(), table, free, page, W, 4, 0)
    wt = rng.permutation(2 * B).reshape(B, 2)
    comp = K.PagedCache(0, torch.zeros(pool * page, 512, dtype=torch.bfloat16, device="cuda"), dev(table), page)
    win = K.PagedCache(0, torch.zeros(2 * B * page, 512, dtype=torch.bfloat16, device="cuda"), dev(wt.tolist()), page)
    ws, count = K.new_workspace(K.paged_step_workspace_bytes(B)), dev([len(free)], torch.int64)
    old, new, fl = dev(t_old.tolist(), torch.int64), dev(t_new.tolist(), torch.int64), dev(free)
    cap, t_max = int((t_new - t_old).sum()), int(t_new.max())
    K.block_table_update(old, new, K.PageTable(comp.table, page, pool), fl, count, t_max=t_max, window=W, stride=4,
                         lookahead=0, free_count_out=count, ws=ws)
    assert comp.table.tolist() == want_t and count.item() == len(want_f)
    m = K.slot_map(old, new, K.PageTable(comp.table, page, pool), K.PageTable(win.table, page, 2 * B), cap, t_max,
                   window=W, stride=4, lookahead=0, ws=ws)
    want_seq = np.repeat(np.arange(B), t_new - t_old)
    want_pos = np.concatenate([np.arange(a, b) for a, b in zip(t_old, t_new)])
    assert np.array_equal(m.seq.cpu().numpy(), want_seq) and np.array_equal(m.pos.cpu().numpy(), want_pos)
    w = torch.zeros(8, 512, device="cuda")
    w[7] = 1.0                                   # an entry is its last tap's state
    ring = torch.zeros(B, W + 8, 512, dtype=torch.bfloat16, device="cuda")
    x = dev(rng.integers(1, 200, cap).tolist(), torch.bfloat16)[:, None].expand(cap, 512).contiguous()
    K.append_paged(x, w, m, ring, win, comp, stride=4, window=W, lookahead=0, max_new=40, rope_dim=0, ws=ws)
    assert K.workspace_status(ws) == 0
    seq, pos = torch.from_numpy(want_seq).cuda(), torch.from_numpy(want_pos).cuda()
    assert torch.equal(ring[seq, pos % (W + 8)], x)
    at = win.table[seq, (pos % W) // page].long() * page + pos % W % page
    assert torch.equal(win.codes[at], x)


@pytest.mark.parametrize("fmt", [K.BF16, K.FP8_E4M3_ROW])
@pytest.mark.parametrize("stride,taps,window,lookahead", [(100, 300, 128, 16), (7, 129, 20, 20), (16, 97, 0, 0)])
def test_append_of_more_taps_than_are_summed_at_a_time(fmt, stride, taps, window, lookahead):
    a = Appender(190 + taps, 3, fmt, stride, taps, window, lookahead, 1500)
    for counts in ([700, 1, 40], [1, 0, 3], [2, 2, 1], [300, 500, 80], [1, 1, 1], [0, 90, 333]):
        a.step(counts)
    a.check()


def test_append_of_many_long_entries():
    """Every token emits an entry of 40 taps, which all weigh nothing but the 14th."""
    n, taps = 9000, 40
    rng = np.random.default_rng(3)
    table = torch.from_numpy(rng.permutation(2 * 141).reshape(2, 141).astype(np.int32)).cuda()
    comp = K.PagedCache(0, torch.zeros(2 * 141 * 64, 512, dtype=torch.bfloat16, device="cuda"), table, 64)
    w = torch.zeros(taps, 512, device="cuda")
    w[13] = 1.0
    ring = torch.zeros(2, taps, 512, dtype=torch.bfloat16, device="cuda")
    ws = K.new_workspace(K.paged_step_workspace_bytes(2))
    x = torch.from_numpy(rng.normal(size=(2, n, 512)).astype(np.float32)).to(torch.bfloat16).cuda()
    old = 0
    for new in (n - 1000, n):           # (the second call reads the first one's ring)
        m = K.slot_map(dev([old] * 2, torch.int64), dev([new] * 2, torch.int64), comp, None, 2 * (new - old), n, window=0,
                       stride=1, lookahead=0, ws=ws)
        K.append_paged(x[:, old:new].reshape(-1, 512).contiguous(), w, m, ring, None, comp, stride=1, window=0,
                       lookahead=0, rope_dim=0, ws=ws)
        old = new
    assert K.workspace_status(ws) == 0
    e = torch.arange(n, device="cuda")
    for b in range(2):
        got = comp.codes[table[b][e // 64].long() * 64 + e % 64]
        assert not got[:26].any() and torch.equal(got[26:], x[b, :n - 26])


@pytest.mark.parametrize("stride,taps", [(4, 8), (128, 128)])
def test_append_replayed_and_on_two_streams(stride, taps):
    """A captured append replayed on new states, and two appends at once on streams and workspaces of their own."""
    W, t, page = 128, [900, 31, 400], 64
    rng = np.random.default_rng(12)
    rows = [S.cache_rows(x, W, stride, 0) for x in t]
    width = max(1, *(-(-r // page) for r in rows))
    table = dev(rng.permutation(3 * width).reshape(3, width).tolist())
    wtable = dev(rng.permutation(6).reshape(3, 2).tolist())
    w = torch.softmax(torch.from_numpy(rng.normal(size=(taps, 512)).astype(np.float32)).cuda(), 0)
    new = lambda: (K.PagedCache(0, torch.zeros(3 * width * page, 512, dtype=torch.bfloat16, device="cuda"), table, page),  # noqa: E731
                   K.PagedCache(0, torch.zeros(6 * page, 512, dtype=torch.bfloat16, device="cuda"), wtable, page),
                   torch.zeros(3, W + taps, 512, dtype=torch.bfloat16, device="cuda"), K.new_workspace(16))
    first, _, _, ws0 = new()
    m = K.slot_map(dev([0, 0, 0], torch.int64), dev(t, torch.int64), first, new()[1], sum(t), max(t), window=W,
                   stride=stride, lookahead=0, ws=ws0)
    x = [torch.from_numpy(rng.normal(size=(sum(t), 512)).astype(np.float32)).to(torch.bfloat16).cuda() for _ in range(2)]

    def run(states, c, stream=None):
        K.append_paged(states, w, m, c[2], c[1], c[0], stride=stride, window=W, lookahead=0, ws=c[3], stream=stream)

    want = [new() for _ in x]
    for s, c in zip(x, want):
        run(s, c)
    torch.cuda.synchronize()

    def same(c, d):
        return all(torch.equal(a, b) for a, b in ((c[0].codes, d[0].codes), (c[1].codes, d[1].codes), (c[2], d[2])))
    static, c = x[0].clone(), new()
    run(static, c)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(static, c)
    for s, d in zip(x[::-1] + x, want[::-1] + want):
        static.copy_(s)
        g.replay()
        assert same(c, d)
    streams, got = [torch.cuda.Stream() for _ in x], [new() for _ in x]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, c, st in zip(x, got, streams):
            run(s, c, stream=st)
    torch.cuda.synchronize()
    assert all(same(c, d) and K.workspace_status(c[3]) == 0 for c, d in zip(got, want))


@pytest.mark.parametrize("batch,pool", [(3, 10), (40, 700), (4096, 5000)])
def test_a_stack_that_ran_out_is_whole_again(batch, pool):
    """More pages are asked for than there are, over several steps, some are given back in between (runs with and without
    pages in any mixture), in the end all: the stack then holds the pool's pages, and admits again."""
    rng = np.random.default_rng(batch)
    page, width = 64, 24
    table, free = [[-1] * width for _ in range(batch)], [int(x) for x in rng.permutation(pool)]
    pages, fl = K.PageTable(dev(table), page, pool), dev(free)
    count, ws, t = dev([pool], torch.int64), K.new_workspace(K.paged_step_workspace_bytes(batch)), [0] * batch

    def step(new, flags):
        nonlocal table, free, t
        table, free = S.block_table_update(t, new, table, free, page, 0, 1)
        K.block_table_update(dev(t, torch.int64), dev(new, torch.int64), pages, fl, count, page * width, window=0, stride=1,
                             free_count_out=count, ws=ws)
        assert count.item() == len(free) and fl[:len(free)].tolist() == free and pages.table.tolist() == table
        assert K.workspace_status(ws) == flags
        ws.zero_()
        t = new

    most = pool * page * 13 // (10 * batch)
    step([min(page * width, int(x)) for x in rng.integers(most, 2 * most, batch)], K.DEV_NO_PAGES)
    for _ in range(4):
        ran_out = len(free)
        new = [int(x) for x in np.where(rng.random(batch) < 0.5, rng.integers(0, page * width + 1, batch), t)]
        asked = sum(max(0, -(-b // page) - -(-a // page)) for a, b in zip(t, new))
        back = sum(sum(x >= 0 for x in table[i][-(-b // page):-(-a // page)]) for i, (a, b) in enumerate(zip(t, new)))
        step(new, K.DEV_NO_PAGES if asked > ran_out + back else 0)
    step([0] * batch, 0)
    assert sorted(free) == list(range(pool))
    some = [page * (pool // batch)] * batch if pool // batch <= width else [page * width] * batch
    step(some, 0)
    assert min(min(r[:some[0] // page]) for r in table) >= 0


def test_entries_outside_the_pool_are_not_given_back():
    ws, fl, count = K.new_workspace(16), dev([3, 0, 0, 0, 0, 0, 0, 0]), dev([1], torch.int64)
    p = K.PageTable(dev([[4, 99, 6, -5, 1], [-1, 2, -1, -1, -1]]), 64, 8)
    out = K.block_table_update(dev([320, 128], torch.int64), dev([0, 0], torch.int64), p, fl, count, 320, window=0, stride=1,
                               ws=ws)
    assert K.workspace_status(ws) == K.DEV_BAD_PAGE and out.item() == 5 and fl[:5].tolist() == [3, 4, 6, 1, 2]


@pytest.mark.parametrize("fmt", [f for f in FORMATS if f != K.BF16])
@pytest.mark.parametrize("stride,taps", [(4, 8), (128, 128)])
def test_appended_codes_are_the_nearest_ones(fmt, stride, taps):
    """Scales are what the rows' largest magnitudes round to and codes the nearest to value / scale: no code further off
    than the nearest, but for the error of the fp32 sums, rotation and quotient."""
    a = Appender(300 + fmt + taps, 3, fmt, stride, taps, 128, 16, 1500)
    for counts in ([900, 260, 300], [1, 2, 17], [0, 300, 5]):
        a.step(counts)
    e4m3 = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    e4m3 = np.unique(e4m3[np.isfinite(e4m3)])
    e2m1 = np.array([-6, -4, -3, -2, -1.5, -1, -0.5, 0, 0.5, 1, 1.5, 2, 3, 4, 6])

    def nearest(grid, x):
        i = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
        return np.minimum(np.abs(grid[i - 1] - x), np.abs(grid[i] - x))

    acc = (taps + 16) * 2.0 ** -24 * max(1.0, max(np.abs(h).max() for h in a.hist))
    rows = 0
    for cache, want in ((a.comp, a.want_c), (a.win, a.want_w)):
        codes = cache.codes.cpu().numpy()
        got = DEQUANT[fmt](codes, cache.scales.cpu().numpy())
        for r, ref in want.items():
            rows += 1
            if fmt == K.FP4_E2M1_G16:
                top = np.abs(ref).reshape(32, 16).max(1) / 6
                s = cache.scales[r].cpu().view(torch.float8_e4m3fn).double().numpy()
                assert np.all(np.abs(s - top) <= nearest(e4m3, top) + acc / 3 + 2.0 ** -23 * top)
                s, grid, n = np.repeat(s, 16), e2m1, 512
            else:
                n, grid = 512 if fmt == K.FP8_E4M3_ROW else 448, e4m3
                top, s = np.abs(ref[:n]).max() / 448, float(cache.scales[r])
                assert abs(s - top) <= acc / 448 + 2.0 ** -23 * top
            x = ref[:n] / np.where(s > 0, s, 1.0)
            lim = s * nearest(grid, x) + 2 * acc + 2.0 ** -23 * np.abs(ref[:n])
            off = np.abs(got[r, :n] - ref[:n])
            assert np.all(off <= np.where(s > 0, lim, np.abs(ref[:n]))), (r, int(np.argmax(off - lim)))
            assert np.all(np.abs(got[r, n:] - ref[n:]) <= acc + 2.0 ** -8 * np.abs(ref[n:]))
    assert rows > 3 * 128
