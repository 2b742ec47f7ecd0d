"""Set-up of paged caches, drafted trees and error bounds for the serving-step tests."""
import numpy as np
import torch

import compressed_sparse_kv_b200 as K
from oracle import formats as OF
from oracle import serving as S
from oracle.compress import n_entries
from oracle.rope import rope

DEQUANT = {K.BF16: None, K.FP8_E4M3_ROW: OF.dequant_fp8_rows, K.FP4_E2M1_G16: OF.dequant_fp4_rows,
           K.FP8_E4M3_ROW_ROPE_BF16: OF.dequant_fp8_rope_rows}
FORMATS = [K.BF16, K.FP8_E4M3_ROW, K.FP4_E2M1_G16, K.FP8_E4M3_ROW_ROPE_BF16]
ROW_BYTES = {K.BF16: 1024, K.FP8_E4M3_ROW: 512, K.FP4_E2M1_G16: 256, K.FP8_E4M3_ROW_ROPE_BF16: 576}


def store(x, fmt):
    """Rows x [n][512] (fp32 numpy) as (codes, scales) on the GPU and their float64 values."""
    x = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda()
    if fmt == K.BF16:
        c = x.to(torch.bfloat16)
        return c, None, c.double().cpu().numpy()
    if not len(x):
        codes = torch.empty(0, ROW_BYTES[fmt], dtype=torch.uint8, device="cuda")
        sc = torch.empty((0, 32) if fmt == K.FP4_E2M1_G16 else 0,
                         dtype=torch.uint8 if fmt == K.FP4_E2M1_G16 else torch.float32, device="cuda")
        return codes, sc, np.zeros((0, 512))
    c, s = K.quantize(x, fmt)
    return c, s, DEQUANT[fmt](c.cpu().numpy(), s.cpu().numpy())


def nan_pool(rows, fmt):
    """A pool in which every row is NaN: what a call must not read shows."""
    if fmt == K.BF16:
        return torch.full((rows, 512), float("nan"), dtype=torch.bfloat16, device="cuda"), None
    codes = torch.full((rows, ROW_BYTES[fmt]), 0x7F, dtype=torch.uint8, device="cuda")
    if fmt == K.FP4_E2M1_G16:
        return codes, torch.full((rows, 32), 0x7F, dtype=torch.uint8, device="cuda")
    return codes, torch.full((rows,), float("nan"), device="cuda")


def tables(rng, counts, page, spare=2, width=None):
    """Shuffled pages for `counts` rows per sequence: (table int32 numpy, -1 where unused; pool pages)."""
    need = [-(-c // page) for c in counts]
    perm = rng.permutation(sum(need) + spare).astype(np.int32)
    table = np.full((len(counts), max(1, width or 0, *need)), -1, dtype=np.int32)
    o = 0
    for b, m in enumerate(need):
        table[b, :m] = perm[o:o + m]
        o += m
    return table, len(perm)


def paged(rng, rows_of, page, fmt, width=None):
    """A paged cache of per-sequence rows (list of [n][512]); (PagedCache, list of float64 values)."""
    table, pages = tables(rng, [len(r) for r in rows_of], page, width=width)
    codes, scales = nan_pool(pages * page, fmt)
    vals = []
    for b, r in enumerate(rows_of):
        c, s, v = store(r, fmt)
        vals.append(v)
        i = np.arange(len(r))
        at = torch.from_numpy(table[b][i // page].astype(np.int64) * page + i % page).cuda()
        codes[at] = c
        if scales is not None:
            scales[at] = s
    return K.PagedCache(fmt, codes, torch.from_numpy(table).cuda(), page, scales), vals


def random_tree(rng, m):
    return [-1 if j == 0 else int(rng.integers(max(-1, j - 5), j)) for j in range(m)]


class TreeCase:
    """A batch of drafted trees over paged caches: GPU inputs and the oracle's."""

    def __init__(self, seed, ts, ms, heads, fmt, page=64, window=128, stride=128, k=0, q_scale=1.0, parents=None,
                 pad=0, edit=None):
        rng = np.random.default_rng(seed)
        self.ts, self.ms, self.heads, self.fmt, self.window, self.stride, self.k = ts, ms, heads, fmt, window, stride, k
        self.parents = parents or [random_tree(rng, m) for m in ms]
        deep = [max([0] + [len(a) for a in S.ancestors(p)]) for p in self.parents]
        comp = [rng.normal(size=(n_entries(t + d, window, stride), 512)) for t, d in zip(ts, deep)]
        win = [rng.normal(size=(min(t, window), 512)) for t in ts]
        draft = [rng.normal(size=(m, 512)) for m in ms]
        if edit:
            edit(comp, win, draft)
        self.total, self.rows = sum(ms), sum(ms) + pad
        self.comp, self.comp_v = paged(rng, comp, page, fmt)
        self.win, self.win_v = paged(rng, win, page, fmt)
        codes, scales = nan_pool(self.rows, fmt)
        c, s, v = store(np.concatenate(draft) if draft else np.zeros((0, 512)), fmt)
        codes[:self.total] = c
        if scales is not None:
            scales[:self.total] = s
        self.draft = K.Cache(fmt, codes[None], None if scales is None else scales[None])
        self.cu = np.concatenate([[0], np.cumsum(ms)]).astype(np.int32)
        self.draft_v = [v[a:b] for a, b in zip(self.cu[:-1], self.cu[1:])]
        q = torch.from_numpy((rng.normal(size=(self.rows, heads, 512)) * q_scale).astype(np.float32))
        self.q = q.to(torch.bfloat16).cuda()
        self.q_v = self.q.double().cpu().numpy()
        self.idx = self.idx_v = None
        if k:
            idx = np.full((self.rows, k), -1, dtype=np.int32)
            self.idx_v = []
            for b, (t, par) in enumerate(zip(ts, self.parents)):
                own = []
                for j, path in enumerate(S.ancestors(par)):
                    n = n_entries(t + len(path), window, stride)
                    e = np.sort(rng.permutation(n)[:k]).astype(np.int32)
                    idx[self.cu[b] + j, :len(e)] = e
                    own.append(list(e))
                self.idx_v.append(own)
            self.idx = torch.from_numpy(idx).cuda()
        par = np.full(self.rows, -1, dtype=np.int32)
        par[:self.total] = np.concatenate([np.asarray(p, dtype=np.int32) for p in self.parents if p] or [np.zeros(0, np.int32)])
        dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        self.parent, self.cu_d, self.t_seq = dev(par), dev(self.cu), dev(np.asarray(ts, dtype=np.int64))
        self.t_max, self.max_nodes = max(ts), max(1, *ms)

    def workspace(self):
        return K.new_workspace(K.tree_decode_paged_workspace_bytes(
            len(self.ts), self.heads, self.max_nodes, self.rows, self.t_max, self.window, self.stride, self.k or None))

    def run(self, ws=None, **kw):
        kw.setdefault("out_fp32", True)
        return K.tree_decode_paged(self.q, self.comp, self.win, self.draft, self.cu_d, self.parent, self.t_seq, self.t_max,
                                   self.max_nodes, window=self.window, stride=self.stride, idx=self.idx, ws=ws, **kw)

    def reference(self):
        """(out [total][H][512], bound of its error) in float64.

        With weights p_r (1 + e_r), |e_r| <= E, and their own sum as denominator the output is off by at most
        E sum p_r |v_r - o|; where the denominator sums the unrounded weights (row-scale formats) by E sum p_r |v_r|.
        E is half a step of the weights' type plus twice the scores' error: fp32 sums of 512 products (512 x 2^-24 of
        their absolute sum), f16 queries below 2^-14 (2^-25 each) and, with bf16 rotary channels, those rounded to f16
        (2^-11 of them).  f16 weights below 2^-14 add 2^-25 each; the sums over the rows their count x 2^-24."""
        f16 = self.fmt != K.BF16
        scaled = self.fmt in (K.FP8_E4M3_ROW, K.FP8_E4M3_ROW_ROPE_BF16)
        out, tol = [], []
        for b, (t, par) in enumerate(zip(self.ts, self.parents)):
            held = S.window_positions(t, self.window)
            for j, path in enumerate(S.ancestors(par)):
                p = t + len(path)
                n = n_entries(p, self.window, self.stride)
                c = self.comp_v[b][:n] if self.idx is None else self.comp_v[b][self.idx_v[b][j]]
                rows = np.concatenate([c, self.win_v[b][held >= p - self.window], self.draft_v[b][path]])
                q = self.q_v[self.cu[b] + j]
                if not len(rows):
                    out.append(np.zeros(q.shape))
                    tol.append(np.zeros(q.shape))
                    continue
                sc = 512 ** -0.5
                x = (q @ rows.T) * sc
                a = np.abs(q) @ np.abs(rows).T * sc
                d = 512 * 2.0 ** -24 * a.max()
                if f16:
                    d += 2.0 ** -25 * sc * np.abs(rows).sum(1).max()
                if self.fmt == K.FP8_E4M3_ROW_ROPE_BF16:
                    d += 2.0 ** -11 * sc * (np.abs(q[:, 448:]) @ np.abs(rows[:, 448:]).T).max()
                w = np.exp(x - x.max(1, keepdims=True))
                w /= w.sum(1, keepdims=True)
                o = w @ rows
                half = 2.0 ** -11 if f16 else 2.0 ** -8
                e = half + 2 * d + 2.0 ** -20
                spread = w @ np.abs(rows) if scaled else np.stack(
                    [wh @ np.abs(rows - oh) for wh, oh in zip(w, o)])
                if scaled:
                    spread = spread * half + 2 * d * np.stack([wh @ np.abs(rows - oh) for wh, oh in zip(w, o)])
                else:
                    spread = spread * e
                big = np.abs(rows).max(0)
                lim = spread + (len(rows) * 2.0 ** -24 + 2.0 ** -20) * (w @ np.abs(rows))
                if f16:
                    lim = lim + 2.0 ** -25 * len(rows) * big
                if self.fmt == K.FP8_E4M3_ROW_ROPE_BF16:
                    lim[:, 448:] += 2.0 ** -11 * (w @ np.abs(rows[:, 448:]))
                both = lim[:, 448::2] + lim[:, 449::2] + 2.0 ** -20 * (np.abs(o[:, 448::2]) + np.abs(o[:, 449::2]))
                lim[:, 448::2] = lim[:, 449::2] = both
                out.append(rope(o, -p))
                tol.append(lim)
        return np.stack(out), np.stack(tol)

    def check(self, got, bf16=False):
        ref, tol = self.reference()
        got = got[:self.total].double().cpu().numpy()
        if bf16:
            tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
        assert np.all(np.isfinite(got))
        off = np.abs(got - ref) - tol
        worst = np.unravel_index(np.argmax(off), off.shape)
        assert off.max() <= 0, (f"node {worst[0]} head {worst[1]} channel {worst[2]}: got {got[worst]:.6g}, "
                                f"reference {ref[worst]:.6g}, bound {tol[worst]:.3g}; {int((off > 0).sum())} outputs off")
