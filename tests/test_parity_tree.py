"""dsv4kv_tree_decode_paged against the float64 oracle: every format, head
counts that do and do not divide a group of 64 query rows, lengths from none to
long, trees of one node to many, cut and whole groups, selected entries."""
import numpy as np
import pytest
import torch

import compressed_sparse_kv_b200 as K
from tests._serving import FORMATS, TreeCase

pytestmark = pytest.mark.gpu

RAGGED_T = [300, 0, 1, 5, 127, 128, 129, 9000]
RAGGED_M = [4, 1, 3, 0, 6, 2, 9, 5]


def both(case):
    ws = case.workspace()
    got = case.run(ws=ws)
    case.check(got)
    case.check(case.run(ws=ws, out_fp32=False), bf16=True)
    assert K.workspace_status(ws) == 0
    return got


def test_one_node_one_short_sequence():
    both(TreeCase(1, [130], [1], 64, K.BF16))


def test_full_tiles_by_tma():
    both(TreeCase(2, [128 * 400], [2], 64, K.BF16))        # 399 entries: three whole tiles and a tail


@pytest.mark.parametrize("fmt", FORMATS)
def test_ragged_batch(fmt):
    both(TreeCase(10 + fmt, RAGGED_T, RAGGED_M, 64, fmt, page=64, pad=3))


@pytest.mark.parametrize("heads", [1, 5, 16, 20, 32, 65, 128])
def test_head_counts(heads):
    both(TreeCase(20 + heads, [700, 140, 33], [7, 3, 5], heads, K.BF16, page=128, stride=4))


@pytest.mark.parametrize("fmt,heads", [(K.FP8_E4M3_ROW, 16), (K.FP4_E2M1_G16, 8), (K.FP8_E4M3_ROW_ROPE_BF16, 24)])
def test_quantised_shared_groups(fmt, heads):
    both(TreeCase(30 + fmt, [2000, 260], [9, 11], heads, fmt, page=256, stride=4))


def test_a_long_chain_deeper_than_the_window():
    chain = [list(range(-1, 39))]
    both(TreeCase(41, [70], [40], 32, K.BF16, window=16, stride=4, parents=chain))


def test_wide_tree_of_256_nodes():
    both(TreeCase(42, [257, 90], [256, 17], 4, K.BF16, page=64, stride=128))


@pytest.mark.parametrize("stride,window", [(1, 0), (3, 7), (128, 200)])
def test_other_windows_and_strides(stride, window):
    both(TreeCase(43 + stride, [411, 64, 3], [5, 4, 2], 24, K.BF16, window=window, stride=stride))


def test_groups_cut_between_ctas():
    """Few long groups: their tiles are spread over the SMs and merged."""
    both(TreeCase(50, [40000, 9000, 200], [2, 1, 2], 64, K.BF16, stride=4, page=256))
    both(TreeCase(51, [30000], [3], 48, K.FP8_E4M3_ROW, stride=4, page=128))


def test_more_groups_than_sms():
    both(TreeCase(52, [300, 513, 140], [90, 80, 70], 64, K.BF16, page=64))


@pytest.mark.parametrize("fmt,heads,k", [(K.BF16, 64, 512), (K.FP8_E4M3_ROW, 16, 100), (K.FP4_E2M1_G16, 64, 64),
                                         (K.FP8_E4M3_ROW_ROPE_BF16, 80, 130), (K.BF16, 3, 1)])
def test_selected_entries(fmt, heads, k):
    both(TreeCase(60 + fmt + k, [5000, 90, 640, 132], [4, 2, 6, 3], heads, fmt, stride=4, k=k))


@pytest.mark.parametrize("fmt", [K.BF16, K.FP8_E4M3_ROW])
def test_growing_scores_raise_the_maximum(fmt):
    """Scores that grow along the rows pass the running maximum tile after tile."""
    def grow(comp, win, draft):
        for c in comp:
            c *= np.linspace(0.1, 6, len(c))[:, None] if len(c) else 1.0
    both(TreeCase(70 + fmt, [6000, 900], [3, 5], 32, fmt, stride=4, q_scale=3.0, edit=grow))


def test_repeated_calls_and_workspace_reuse_are_bitwise_equal():
    a, b = TreeCase(80, [20000], [2], 64, K.BF16, stride=4), TreeCase(81, [300, 70], [3, 4], 16, K.BF16)
    ws = K.new_workspace(max(a.workspace().numel(), b.workspace().numel()))
    first = a.run(ws=ws).clone()
    other = b.run(ws=ws).clone()
    assert torch.equal(a.run(ws=ws), first) and torch.equal(b.run(ws=ws), other)


def test_rows_behind_the_last_sequence_are_left():
    c = TreeCase(82, [200, 50], [3, 2], 16, K.BF16, pad=6)
    out = torch.full((c.rows, 16, 512), 7.0, device="cuda")
    c.run(out=out)
    c.check(out)
    assert torch.all(out[c.total:] == 7.0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("heads", [64, 8])
def test_bad_rows_stay_with_the_nodes_that_see_them(heads, bad):
    """A sibling's drafted row, a window row that deeper nodes have left behind and an entry that shallow ones do not
    see yet hold an infinity or NaN: only the nodes that attend to them are affected."""
    parents = [[-1, 0, 0, 2, 3]]                            # node 1 is nobody's ancestor; 4 sees 0, 2, 3
    clean = TreeCase(90, [256 + 126], [5], heads, K.BF16, parents=parents)

    def spoil(comp, win, draft):
        assert len(comp[0]) == 2                            # entry 1 is seen from depth 2 on
        comp[0][1, 5] = bad
        draft[0][1, 7] = bad
        win[0][(382 - 128) % 128, 9] = bad                  # position 254: seen by depth 0 only
    c = TreeCase(90, [256 + 126], [5], heads, K.BF16, parents=parents, edit=spoil)
    got, want = c.run(), clean.run()
    for j, clear in enumerate([False, True, True, False, False]):   # depths 0, 1, 1, 2, 3
        if clear:
            assert torch.equal(got[j], want[j])
        else:
            assert not torch.isfinite(got[j]).all()


def test_a_bad_query_stays_in_its_row():
    c = TreeCase(91, [300], [4], 16, K.BF16)
    want = c.run().clone()
    c.q[1, 3, 11] = float("nan")
    got = c.run()
    assert torch.isnan(got[1, 3]).all()
    got[1, 3] = want[1, 3]
    assert torch.equal(got, want)


def test_bad_inputs_are_flagged_not_faulted():
    c = TreeCase(92, [2000, 600], [4, 3], 16, K.BF16, stride=4)

    def flags(**kw):
        d = TreeCase.__new__(TreeCase)
        d.__dict__.update(c.__dict__, **kw)
        ws = d.workspace()
        out = d.run(ws=ws)
        assert torch.isfinite(out[:c.total]).all() or "cu_d" in kw
        return K.workspace_status(ws)

    assert flags(parent=torch.tensor([0, 0, 9, -3, 2, 0, 1], dtype=torch.int32, device="cuda")) == K.DEV_BAD_TREE
    assert flags(t_seq=torch.tensor([2000, -4], device="cuda")) == K.DEV_BAD_LENGTH
    assert flags(cu_d=torch.tensor([0, 5, 3], dtype=torch.int32, device="cuda")) & K.DEV_BAD_LENGTH
    assert flags(cu_d=torch.tensor([-2, 4, 90], dtype=torch.int32, device="cuda")) & K.DEV_BAD_LENGTH
    tab = c.comp.table.clone()
    tab[0, 1], tab[0, 2] = -1, c.comp.pool_pages
    assert flags(comp=K.PagedCache(c.fmt, c.comp.codes, tab, c.comp.page_rows)) == K.DEV_BAD_PAGE
    wtab = c.win.table.clone()
    wtab[1, 0] = 1 << 30
    assert flags(win=K.PagedCache(c.fmt, c.win.codes, wtab, c.win.page_rows)) == K.DEV_BAD_PAGE
    s = TreeCase(93, [2000], [2], 16, K.BF16, stride=4, k=8)
    s.idx[0, 3] = 100000
    ws = s.workspace()
    assert torch.isfinite(s.run(ws=ws)).all() and K.workspace_status(ws) == K.DEV_BAD_INDEX


def test_captured_and_replayed_with_new_lengths():
    """One graph for a serving loop: lengths, trees and queries change between replays."""
    a = TreeCase(100, [900, 300], [5, 4], 16, K.BF16, stride=4)
    b = TreeCase(101, [850, 120], [4, 5], 16, K.BF16, stride=4)
    ws, out = a.workspace(), torch.empty(9, 16, 512, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a.run(ws=ws, out=out)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run(ws=ws, out=out)
    g.replay()
    a.check(out)
    # b's inputs moved into a's buffers
    rows = b.comp.codes.shape[0], b.win.codes.shape[0]
    assert rows[0] <= a.comp.codes.shape[0] and rows[1] <= a.win.codes.shape[0]
    a.comp.codes[:rows[0]], a.win.codes[:rows[1]] = b.comp.codes, b.win.codes
    a.comp.table.fill_(-1)
    a.comp.table[:, :b.comp.table.shape[1]] = b.comp.table
    a.win.table.copy_(b.win.table)
    a.draft.codes.copy_(b.draft.codes)
    for x, y in ((a.q, b.q), (a.cu_d, b.cu_d), (a.parent, b.parent), (a.t_seq, b.t_seq)):
        x.copy_(y)
    g.replay()
    b.check(out)


def test_two_streams_at_once():
    a, b = TreeCase(110, [20000], [3], 64, K.BF16, stride=4), TreeCase(111, [16000], [2], 64, K.FP8_E4M3_ROW, stride=4)
    want = a.run().clone(), b.run().clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        got = a.run(stream=s[0]), b.run(stream=s[1])
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_tiny_and_zero_row_scales():
    """Rows whose fp8 scale is 0 (a row of zeros), below the smallest normal number or many powers of two below the
    others' keep their place in the softmax."""
    c = TreeCase(120, [900, 300], [4, 3], 16, K.FP8_E4M3_ROW, stride=4)
    for b, (t, vals) in enumerate(zip(c.ts, c.comp_v)):
        for r, scale in ((3, 0.0), (5, 2.0 ** -140), (9, 2.0 ** -60), (20, 2.0 ** -90)):
            at = int(c.comp.table[b, r // 64]) * 64 + r % 64
            vals[r] *= scale / float(c.comp.scales[at])
            c.comp.scales[at] = scale
    c.check(c.run())


def test_rows_past_four_gib_of_the_pool():
    """Pages at the end of a pool of more than 2^32 bytes."""
    c = TreeCase(121, [9000, 200], [3, 2], 64, K.BF16, stride=4, page=64)
    rows, far = c.comp.codes.shape[0], (5 << 30) // 1024 // 64 * 64
    pool = torch.empty(far + rows, 512, dtype=torch.bfloat16, device="cuda")
    pool[far:] = c.comp.codes
    table = torch.where(c.comp.table >= 0, c.comp.table + far // 64, -1).to(torch.int32)
    c.comp = K.PagedCache(K.BF16, pool, table, 64)
    c.check(c.run())
    s = TreeCase(122, [9000], [3], 16, K.BF16, stride=4, page=64, k=40)
    pool = torch.empty(far + s.comp.codes.shape[0], 512, dtype=torch.bfloat16, device="cuda")
    pool[far:] = s.comp.codes
    s.comp = K.PagedCache(K.BF16, pool, torch.where(s.comp.table >= 0, s.comp.table + far // 64, -1).to(torch.int32), 64)
    s.check(s.run())


def test_a_selected_entry_named_twice_counts_twice():
    c = TreeCase(123, [900], [2], 16, K.BF16, stride=4, k=6)
    c.idx[0] = torch.tensor([7, 7, 7, 3, 190, -1], dtype=torch.int32)
    c.idx_v[0][0] = [7, 7, 7, 3, 190]
    c.check(c.run())


def test_no_drafted_nodes_at_all():
    c = TreeCase(124, [900, 10], [2, 3], 16, K.BF16, stride=4)
    out = torch.full((c.rows, 16, 512), 3.0, device="cuda")
    ws = c.workspace()
    c.cu_d.zero_()
    c.run(ws=ws, out=out)
    assert torch.all(out == 3.0) and K.workspace_status(ws) == 0


def test_a_large_batch():
    rng = np.random.default_rng(5)
    b = 1024
    c = TreeCase(125, [int(t) for t in rng.integers(0, 400, b)], [int(m) for m in rng.integers(0, 3, b)], 4, K.BF16, stride=4)
    both(c)


def test_two_graphs_share_a_workspace():
    a, b = TreeCase(126, [20000], [2], 64, K.BF16, stride=4), TreeCase(127, [16000, 300], [1, 3], 64, K.BF16, stride=4)
    ws = K.new_workspace(max(a.workspace().numel(), b.workspace().numel()))
    outs, graphs = [], []
    for c in (a, b):
        out = torch.empty(c.rows, 64, 512, device="cuda")
        c.run(ws=ws, out=out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(ws=ws, out=out)
        outs.append(out)
        graphs.append(g)
    for k in (0, 1, 0, 0, 1):
        outs[k].zero_()
        graphs[k].replay()
        (a, b)[k].check(outs[k])
    assert K.workspace_status(ws) == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("k", [0, 8])
def test_pools_without_a_page(fmt, k):
    """Contexts too short for a compressed entry need no pool, empty ones no window pool either."""
    c = TreeCase(128, [100, 12], [3, 5], 16, fmt, stride=128)
    empty = lambda x: K.PagedCache(fmt, x.codes[:0], x.table, x.page_rows, None if x.scales is None else x.scales[:0])  # noqa: E731
    c.comp = empty(c.comp)
    if k:
        c.k, c.idx, c.idx_v = k, torch.full((c.rows, k), -1, dtype=torch.int32, device="cuda"), [[[]] * m for m in c.ms]
        c.idx[1, 0] = 0                     # (not an entry of that node)
    c.check(c.run())
    c = TreeCase(129, [0, 0], [3, 5], 16, fmt, stride=128)
    c.comp, c.win = empty(c.comp), empty(c.win)
    c.check(c.run())


def test_scores_near_the_lowest_number():
    """One row, whose score is far below -1e30 for half of the heads, has all the weight."""
    def large(comp, win, draft):
        win[0][:] = 1e17
    c = TreeCase(130, [1], [1], 16, K.BF16, q_scale=1e17, edit=large)
    assert ((c.q_v @ c.win_v[0].T).min()) < -1e35
    both(c)


def test_zero_rows_beside_large_scales():
    """A row of zeros counts in the denominator however large the other rows' scales are."""
    def large(comp, win, draft):
        comp[0] *= 2.0 ** 12
    c = TreeCase(131, [900], [2], 16, K.FP8_E4M3_ROW, stride=4, q_scale=2.0 ** -12, edit=large)
    for r in range(0, len(c.comp_v[0]), 2):
        at = int(c.comp.table[0, r // 64]) * 64 + r % 64
        c.comp_v[0][r] = 0.0
        c.comp.scales[at] = 0.0
    both(c)


def test_a_part_of_half_a_million_tiles():
    """A pair whose first part takes seconds goes on to its next one: the one-second limits are for single steps.  Every
    entry lies in one page; with queries of zeros and rows of unit vectors all sums are whole numbers below 2^24."""
    pairs, t, heads = torch.cuda.get_device_properties(0).multi_processor_count // 2, 1 << 26, 128
    nodes = pairs + 1                                   # one group each: a long one a pair, and a short one behind them
    codes = torch.zeros(64, 512, dtype=torch.uint8, device="cuda")
    codes[torch.arange(512, device="cuda") % 64, torch.arange(512, device="cuda")] = 0x38       # 1.0
    ones = lambda n: torch.ones(n, device="cuda")       # noqa: E731
    comp = K.PagedCache(K.FP8_E4M3_ROW, codes, torch.zeros(2, t // 64, dtype=torch.int32, device="cuda"), 64, ones(64))
    win = K.PagedCache(K.FP8_E4M3_ROW, codes[:0], torch.zeros(2, 1, dtype=torch.int32, device="cuda"), 64, ones(0))
    draft = K.Cache(K.FP8_E4M3_ROW, torch.zeros(1, nodes, 512, dtype=torch.uint8, device="cuda"), ones(nodes)[None])
    dev = lambda x, dt: torch.tensor(x, dtype=dt, device="cuda")    # noqa: E731
    ws = K.new_workspace(K.tree_decode_paged_workspace_bytes(2, heads, pairs, nodes, t, 0, 1))
    out = K.tree_decode_paged(torch.zeros(nodes, heads, 512, dtype=torch.bfloat16, device="cuda"), comp, win, draft,
                              dev([0, pairs, nodes], torch.int32), dev([-1] * nodes, torch.int32),
                              dev([t, 128], torch.int64), t, pairs, window=0, stride=1, rope_dim=0, out_fp32=True, ws=ws)
    assert K.workspace_status(ws) == 0
    assert torch.all(out == 1 / 64)


@pytest.mark.parametrize("k", [0, 60])
def test_zero_scales_beside_rotary_channels(k):
    """A scale of 0 makes the fp8 channels zeros whatever their codes; the bf16 rotary channels have no scale."""
    c = TreeCase(132, [900, 300], [4, 3], 16, K.FP8_E4M3_ROW_ROPE_BF16, stride=4, k=k)

    def zero(cache, row, vals):
        cache.scales.view(-1)[row] = 0.0
        vals[:448] = 0.0
    for b in range(2):
        for r in range(0, len(c.comp_v[b]), 3):
            zero(c.comp, int(c.comp.table[b, r // 64]) * 64 + r % 64, c.comp_v[b][r])
        for r in (0, 7, 100):
            zero(c.win, int(c.win.table[b, r // 64]) * 64 + r % 64, c.win_v[b][r])
    zero(c.draft, 1, c.draft_v[0][1])
    both(c)


BAD_ROWS = [(K.FP8_E4M3_ROW, "code", 0x7F), (K.FP8_E4M3_ROW, "scale", float("nan")), (K.FP8_E4M3_ROW, "scale", float("inf")),
            (K.FP4_E2M1_G16, "scale", 0x7F), (K.FP8_E4M3_ROW_ROPE_BF16, "code", 0xFF),
            (K.FP8_E4M3_ROW_ROPE_BF16, "scale", float("nan")),
            (K.FP8_E4M3_ROW_ROPE_BF16, "scale", float("inf")), (K.FP8_E4M3_ROW_ROPE_BF16, "rotary", float("inf")),
            (K.FP8_E4M3_ROW_ROPE_BF16, "rotary", float("-inf")), (K.FP8_E4M3_ROW_ROPE_BF16, "rotary", float("nan"))]


@pytest.mark.parametrize("k", [0, 2])
@pytest.mark.parametrize("heads", [64, 8])
@pytest.mark.parametrize("fmt,where,bad", BAD_ROWS)
def test_bad_quantised_rows_stay_with_the_nodes_that_see_them(fmt, where, bad, heads, k):
    """As for bf16: a drafted row, a window row and an entry that only some nodes see, made non-finite one at a time."""
    parents = [[-1, 0, 0, 2, 3]]                            # depths 0, 1, 1, 2, 3; node 1 is nobody's ancestor

    case = lambda: TreeCase(140, [256 + 126], [5], heads, fmt, parents=parents, k=k)    # noqa: E731
    want = case().run()
    assert torch.isfinite(want).all()
    # (window row 126 holds position 254, which depth 0 alone still sees; entry 1 is seen from depth 2 on)
    for name, row, sees in (("draft", 2, [3, 4]), ("draft", 1, []), ("win", 126, [0]), ("comp", 1, [3, 4])):
        c = case()
        cache = getattr(c, name)
        if name != "draft":
            row = int(cache.table[0, row // 64]) * 64 + row % 64
        codes = cache.codes.view(-1, cache.codes.shape[-1])
        if where == "code":
            codes[row, 300] = bad
        elif where == "rotary":
            codes.view(torch.bfloat16)[row, (448 + 2 * 11) // 2] = bad
        else:
            cache.scales.view(len(codes), -1)[row, -1] = bad
        got = c.run()
        for j in range(5):
            if j in sees:
                assert torch.isnan(got[j]).any(dim=-1).all(), (name, row, j)
            else:
                assert torch.equal(got[j], want[j]), (name, row, j)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("k", [0, 40])
def test_a_query_that_is_not_finite(fmt, bad, k):
    """Its own row is NaN, the others' are untouched."""
    c = TreeCase(141, [300], [4], 16, fmt, stride=4, k=k)
    want = c.run().clone()
    c.q[1, 3, 11] = bad
    got = c.run()
    assert torch.isnan(got[1, 3]).all()
    got[1, 3] = want[1, 3]
    assert torch.equal(got, want)


def test_one_workspace_for_the_decodes_and_the_serving_step():
    """Every call but the index ones takes a workspace as another has left it; an index call takes it zero-filled."""
    c = TreeCase(142, [20000], [2], 64, K.BF16, stride=4)
    size = max(c.workspace().numel(), K.lib().dsv4kv_dense_decode_paged_workspace_bytes(1, 64, 512, c.t_max, 128, 4),
               K.index_topk_workspace_bytes(3, 900, 64), K.paged_step_workspace_bytes(1))
    ws, q = K.new_workspace(size), c.q[:1]
    pages, one = K.PageTable(torch.full((1, 2), -1, dtype=torch.int32, device="cuda"), 64, 4), torch.tensor([0], device="cuda")
    free, count = torch.arange(4, dtype=torch.int32, device="cuda"), torch.tensor([4], device="cuda")
    qi = torch.randint(-8, 9, (3, 128), device="cuda").to(torch.bfloat16)
    keys = K.Cache(0, torch.randint(-8, 9, (3, 900, 128), device="cuda").to(torch.bfloat16), None, 128)

    def decode(w):
        return K.dense_decode_paged(q, c.comp, c.win, c.t_seq, c.t_max, stride=4, ws=w)

    def update(w):
        K.block_table_update(one, one + 100, pages, free, count, 100, window=0, stride=1, ws=w)
        return pages.table.clone()

    calls = [c.run, decode, update]
    want = [c.run(ws=c.workspace()).clone(), decode(K.new_workspace(size)), update(K.new_workspace(16))]
    for i in (0, 1, 2, 0, 2, 1, 0):
        assert torch.equal(calls[i](ws) if i else c.run(ws=ws), want[i]), i
    assert K.workspace_status(ws) == 0 and ws[16:].any()
    ws.zero_()
    for a, b in zip(K.index_topk(qi, keys, 900, 64, ws=ws), K.index_topk(qi, keys, 900, 64)):
        assert torch.equal(a, b)
    assert torch.equal(c.run(ws=ws), want[0])
