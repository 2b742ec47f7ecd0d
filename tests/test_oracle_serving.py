"""Pins of oracle/serving.py: closed forms, the uniform oracle functions and brute force."""
import numpy as np

from oracle import attention as OA
from oracle import compress as OC
from oracle import rope as OR
from oracle import serving as S


def test_pages_are_given_back_before_they_are_taken():
    # 4 rows a page, one row per token behind a window of 0
    table = [[7, 3, -1], [5, 1, 2], [-1, -1, -1]]
    t, f = S.block_table_update([8, 12, 0], [8, 2, 9], table, [9, 8], 4, 0, 1)
    assert t == [[7, 3, -1], [5, 1, 2], [2, 1, 8]] and f == [9]       # 1, 2 pushed; popped 2, 1, 8
    t, f = S.block_table_update([0], [9], [[-1] * 3], [4], 4, 0, 1)
    assert t == [[4, -1, -1]] and f == []                             # the stack runs out


def test_window_cache_keeps_its_pages():
    assert [S.cache_rows(t, 128, 0) for t in (0, 5, 128, 1000)] == [0, 5, 128, 128]
    assert [S.cache_rows(t, 128, 4, 16) for t in (0, 112, 116, 1000)] == [0, 0, 1, 222]


def test_slots_of_a_ragged_step():
    cu, seq, pos, win, comp = S.slot_map([130, 0], [133, 2], [[2, 0], [1, 3]], [[0, 5], [4, 6]], 64, 64, 128, 4)
    assert cu == [0, 3, 5] and seq == [0, 0, 0, 1, 1] and pos == [130, 131, 132, 0, 1]
    assert win == [2, 3, 4, 256, 257]                                 # rows p % 128 of pages 0 and 4
    assert comp == [-1, 128, -1, -1, -1]                              # entry 0 leaves the window at t + 1 = 132
    far = S.slot_map([0], [300], [[0, 1]], [[0, 1]], 64, 64, 128, 4)[3]
    assert far[:172] == [-1] * 172 and min(far[172:]) >= 0 and len(set(far[172:])) == 128


def test_append_in_steps_is_the_whole_history():
    rng = np.random.default_rng(3)
    hist, w = rng.normal(size=(500, 96)), rng.random((8, 96))
    ents, rows, t = {}, {}, 0
    for step in (1, 3, 140, 2, 354):
        win, e, raw = S.append_rows(hist[:t + step], t, t + step, w, 128, 4, 0)
        ents.update(e)
        rows.update(win)
        t += step
    want = OC.compress(hist, w, 4, 128)
    assert sorted(ents) == list(range(len(want)))
    assert np.allclose(np.stack([ents[i] for i in range(len(want))]), want, atol=1e-12)
    assert all(np.allclose(rows[p % 128], OR.rope(hist[p], p)) for p in range(372, 500))
    early = S.append_rows(hist, 0, 500, w, 128, 4, 16)[1]             # a lookahead only writes more of the same entries
    assert len(early) == len(want) + 4 and all(np.allclose(early[i], want[i]) for i in range(len(want)))


def test_window_positions_by_brute_force():
    for t in (0, 1, 5, 127, 128, 129, 1000):
        for r, p in enumerate(S.window_positions(t, 128)):
            assert p == max(x for x in range(max(0, t - 128), t) if x % 128 == r)


def test_a_path_of_the_tree_is_a_sequence_of_decode_steps():
    """Every node gives what the uniform decode gives once its path has been appended to the caches."""
    rng = np.random.default_rng(5)
    t, window, stride, m, d = 150, 16, 4, 7, 128
    parent = [-1, 0, 1, 1, 3, -1, 5]
    hist, w = rng.normal(size=(t, d)), rng.random((8, d))
    draft, q = rng.normal(size=(m, d)), rng.normal(size=(m, 3, d))
    ent = OC.compress(np.concatenate([hist, np.zeros((window, d))]), w, stride, window)   # entries of positions ahead
    held = S.window_positions(t, window)
    rows = np.stack([OR.rope(hist[p], p) for p in held])
    drot = np.stack([OR.rope(draft[j], t + len(a)) for j, a in enumerate(S.ancestors(parent))])
    got = S.tree_decode(q, ent, rows, drot, parent, t, window, stride, scale=d ** -0.5)
    for j, path in enumerate(S.ancestors(parent)):
        full = np.concatenate([hist, draft[path]])
        pos, win, e = OC.append_state(full, w, stride, window)
        ref = OA.dense_decode(q[j][None], e[None], win[None], len(full), d ** -0.5)[0]
        assert np.allclose(got[j], ref, atol=1e-10), j


def test_a_node_without_rows_gives_zeros():
    q = np.ones((2, 1, 128))
    out = S.tree_decode(q, np.zeros((0, 128)), np.zeros((0, 128)), np.ones((2, 128)), [-1, 0], 0, 8, 4)
    assert np.all(out[0] == 0) and np.any(out[1] != 0)


def test_entries_without_a_page_give_none_back():
    t, f = S.block_table_update([0, 0], [12, 20], [[-1] * 5, [-1] * 5], [4, 9, 1, 7], 4, 0, 1)
    assert t == [[7, 1, 9, -1, -1], [4, -1, -1, -1, -1]] and f == []
    t, f = S.block_table_update([12, 20], [4, 0], t, f, 4, 0, 1)
    assert f == [1, 9, 4]                                             # and 7 is still the first sequence's
