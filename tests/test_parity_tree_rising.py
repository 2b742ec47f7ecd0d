"""dsv4kv_tree_decode_paged where the running maxima rise tile after tile: the accumulator is rescaled between products
many times a run, for the queries of one CTA of a pair, of the other, or of both."""
import numpy as np
import pytest
import torch

import compressed_sparse_kv_b200 as K
from oracle import serving as S
from oracle.compress import n_entries
from oracle.rope import rope
from tests._serving import FORMATS, TreeCase

pytestmark = pytest.mark.gpu

TILE, LEVELS, STEP = 128, 20, 6.0     # rows of a tile; levels of a sawtooth; a level in units of the scores (8 / log2(e) = 5.5 raise)


class Rising(TreeCase):
    """Row i of the listed rows is c(i // 128) u plus noise, u a vector of +-1: every query along u sees its scores rise
    by STEP from tile to tile; the other queries are orthogonal to u."""

    def __init__(self, seed, fmt, nodes, heads, entries, k, along):
        rng = np.random.default_rng(seed)
        u = np.where(rng.random(512) < 0.5, -1.0, 1.0)

        def edit(comp, win, draft):
            level = (np.arange(len(comp[0])) // TILE) % LEVELS * STEP * 512 ** -0.5
            comp[0][:] = level[:, None] * u + 0.3 * comp[0]

        t = 128 + 4 * entries
        super().__init__(seed, [t], [nodes], heads, fmt, page=256, stride=4, parents=[[-1] * nodes], edit=edit)
        q = rng.normal(size=(nodes, heads, 512))
        q -= (q @ u)[..., None] / 512 * u
        rows = np.arange(nodes * heads).reshape(nodes, heads)
        second = np.arange(heads) >= (heads + 1) // 2 if k else rows % 128 >= 64     # the query's CTA of the pair
        pick = np.broadcast_to({"first": ~second, "second": second, "both": second | ~second}[along], rows.shape)
        q[pick] = u + 0.1 * q[pick]
        self.q = torch.from_numpy(q.astype(np.float32)).to(torch.bfloat16).cuda()
        self.q_v = self.q.double().cpu().numpy()
        if k:
            self.k = k
            self.idx = torch.arange(k, dtype=torch.int32, device="cuda").repeat(nodes, 1).contiguous()

    def reference(self):
        """As TreeCase's, with |v| + |o| for |v - o|, in torch's float64 (roots only: every node at position t)."""
        t, fmt = self.ts[0], self.fmt
        n = n_entries(t, self.window, self.stride)
        held = S.window_positions(t, self.window)
        rows = np.concatenate([self.comp_v[0][:min(n, self.k) if self.k else n], self.win_v[0][held >= t - self.window]])
        r = torch.from_numpy(rows).cuda()
        q, sc, f16 = self.q.double().view(-1, 512), 512 ** -0.5, fmt != K.BF16
        w = torch.softmax(q @ r.T * sc, 1)
        o, mag = w @ r, w @ r.abs()
        a = q.abs() @ r.abs().T * sc
        d = 512 * 2.0 ** -24 * a.amax(1, keepdim=True)
        if f16:
            d = d + 2.0 ** -25 * sc * r.abs().sum(1).max()
        if fmt == K.FP8_E4M3_ROW_ROPE_BF16:
            d = d + 2.0 ** -11 * sc * (q[:, 448:].abs() @ r[:, 448:].abs().T).amax(1, keepdim=True)
        lim = ((2.0 ** -11 if f16 else 2.0 ** -8) + 2 * d + 2.0 ** -20) * (mag + o.abs())
        # a weight passes a rescale for every raise before the product that it is in: one rounding of 2^-24 and an
        # exponential's 2^-22 each
        lim = lim + (len(rows) * 2.0 ** -24 + 2.0 ** -20 + 2 * LEVELS * 2.0 ** -22) * mag
        if f16:
            lim = lim + 2.0 ** -25 * len(rows) * r.abs().amax(0)
        if fmt == K.FP8_E4M3_ROW_ROPE_BF16:
            lim[:, 448:] += 2.0 ** -11 * mag[:, 448:]
        both = lim[:, 448::2] + lim[:, 449::2] + 2.0 ** -20 * (o[:, 448::2].abs() + o[:, 449::2].abs())
        lim[:, 448::2] = lim[:, 449::2] = both
        shape = (self.total, self.heads, 512)
        return rope(o.cpu().numpy(), -t).reshape(shape), lim.cpu().numpy().reshape(shape)


@pytest.mark.parametrize("along", ["first", "second", "both"])
@pytest.mark.parametrize("k", [0, 2048])
@pytest.mark.parametrize("fmt", FORMATS)
def test_rescales_between_products(fmt, k, along):
    c = Rising(200 + fmt, fmt, 150 if k else 16, 64, 2048 if k else TILE * 160, k, along)
    ws = c.workspace()
    first = c.run(ws=ws).clone()
    c.check(first)
    for _ in range(20):
        assert torch.equal(c.run(ws=ws), first)
    assert K.workspace_status(ws) == 0
