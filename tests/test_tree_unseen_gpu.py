"""Drafted tokens that no row of their sequence sees (the padding of a tree, masks without a token's own bit, tokens past the masks'
words): whatever their K, V and fields hold, the other rows' results stay within the bounds of attention without them."""
import numpy as np
import pytest
import torch

from paged_kv_gqa_block_gb300 import workloads as wl
from tests import plain_tokens as pt
from tests.tree_cases import TreeCase

pytestmark = pytest.mark.gpu

BF16, FP8, TQ4 = wl.KV_BF16, wl.KV_FP8_E4M3, wl.KV_TQ4
KVS = [BF16, FP8, TQ4]


@pytest.fixture(scope="module")
def pda():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_gqa_block_gb300 as pda
    return pda


class Unseen(TreeCase):
    """NaN, or the largest finite values, in K, V and fields of what no row sees of the drafted tokens."""

    def __init__(self, *args, hold="nan", padding=None, **kw):
        self.hold, self.padding = hold, padding
        super().__init__(*args, **kw)

    def poison(self):
        if self.padding is not None:      # the last `padding` tokens of each sequence: rows that see nothing, seen by none
            for b, n in enumerate(self.counts):
                real = max(0, n - self.padding)
                self.masks[b] = [[j for j in row if j < real] if i < real else [] for i, row in enumerate(self.masks[b])]
            self.see = [pt.tree_sight(n, m, self.masks[b], self.window, self.first)
                        for b, (n, m) in enumerate(zip(self.lens, self.counts))]
        super().poison()
        c = self.c
        data, meta = wl.cache_views(c.w, c.cache)
        self.unseen = 0
        for b, see in enumerate(self.see):
            for j in range(self.counts[b]):
                t = self.lens[b] + j
                if see[:, t].any():
                    continue
                self.unseen += 1
                at = c.table[b, t // c.BS], t % c.BS
                if self.hold == "nan":
                    data[at] = 0xFFFF if c.kv == BF16 else 0xFF
                    if meta is not None:
                        meta[at[0], :, :, at[1]] = np.nan if c.kv == FP8 else 0xFFFF
                else:
                    data[at] = 0x7F7F if c.kv == BF16 else 0x7E if c.kv == FP8 else 0xF0
                    if meta is not None:
                        meta[at[0], :, :, at[1]] = 3e38 if c.kv == FP8 else 0x7BFF


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("hold", ["nan", "largest"])
@pytest.mark.parametrize("window,first", [(0, 0), (60, 4)])
def test_padded_trees(pda, kv, hold, window, first):
    """Row tiles held twice (up to 64 rows), of one tile, of two, and of more than one row tile."""
    for counts in ([6, 3, 8, 1], [16, 9, 12, 10], [30, 17, 25, 32], [70, 40, 33, 64], [5, 140, 20, 33]):
        t = Unseen(kv, 2, 8, 16, [100, 0, 250, 123], counts, "tree", window, first, seed=sum(counts), hold=hold, padding=2)
        assert t.unseen >= 7
        t.check(pda)


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("hold", ["nan", "largest"])
@pytest.mark.parametrize("BS,QG", [(16, 6), (32, 16)])
def test_masks_that_are_no_trees(pda, kv, hold, BS, QG):
    rng = np.random.default_rng(BS)
    lens, counts = [int(x) for x in rng.integers(0, 400, 40)], [int(x) for x in rng.choice([1, 2, 3, 5, 9, 17, 33, 40, 65], 40)]
    t = Unseen(kv, 2, QG, BS, lens, counts, "anything", seed=5, hold=hold)
    assert t.unseen >= 10
    t.check(pda)


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("hold", ["nan", "largest"])
def test_tokens_past_the_masks_words(pda, kv, hold):
    """Of 200 drafted tokens the masks name 64 at most: steps wholly of tokens that no row sees."""
    t = Unseen(kv, 1, 8, 16, [70, 5], [200, 100], "tree", seed=3, words=1, hold=hold)
    assert t.unseen == 136 + 36
    t.check(pda)


@pytest.mark.parametrize("kv", KVS)
def test_nothing_is_seen(pda, kv):
    """No cached token, and no bit in any mask: zeros."""
    t = Unseen(kv, 2, 8, 16, [0, 0], [7, 40], "tree", seed=3, padding=40)
    assert t.unseen == 47
    assert bool((t.check(pda) == 0).all())


@pytest.mark.parametrize("kv", KVS)
def test_large_trees(pda, kv):
    """Many words of many rows, and row tiles that follow one another in a CTA."""
    t = Unseen(kv, 1, 6, 16, [40, 3], [1100, 130], "tree", seed=6, padding=70)
    assert t.unseen == 140
    t.check(pda)
