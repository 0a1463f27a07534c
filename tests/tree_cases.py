"""Cases of drafted tokens over a cache, and their results in 64 bits.  Test-side only."""
from __future__ import annotations

import numpy as np
import torch

from paged_kv_gqa_block_gb300 import workloads as wl
from tests import plain_tokens as pt

BF16, FP8 = wl.KV_BF16, wl.KV_FP8_E4M3


def tree(rng, n):
    """Every token below one of those before it, or a root of its own."""
    seen = []
    for j in range(n):
        up = int(rng.integers(-1, j)) if j else -1
        seen.append((seen[up] if up >= 0 else []) + [j])
    return seen


def anything(rng, n):
    """Masks that are no tree's: any tokens, none, all."""
    out = [sorted(rng.choice(n, size=int(rng.integers(0, n + 1)), replace=False).tolist()) for _ in range(n)]
    out[0] = []
    if n > 2:
        out[-1] = list(range(n))
        out[1] = [n - 1]
    return out


class TreeCase:
    def __init__(self, kv, Hk, QG, BS, lens, counts, kind="tree", window=0, first=0, seed=0, before=0, after=0, words=None,
                 q_scale=1.0, MB=None, v_spread=0.5):
        c = self.c = pt.Pool(kv, Hk, QG, BS, [n + m for n, m in zip(lens, counts)], seed=seed, MB=MB, v_spread=v_spread)
        rng = c.rng
        self.kv, self.Hk, self.QG, self.BS, self.B = kv, Hk, QG, BS, c.B
        self.lens, self.counts, self.window, self.first = list(lens), list(counts), window, first
        self.starts = before + np.concatenate([[0], np.cumsum(counts)]).astype(int)
        self.N = int(self.starts[-1]) + after
        self.q = wl.round_bf16((rng.standard_normal((self.N, Hk * QG, 128)) * q_scale).astype(np.float32))
        self.masks = None
        if kind != "chain":
            self.masks = [(tree if kind == "tree" else anything)(rng, n) if n else [] for n in counts]
        self.words = words or (max(1, -(-max(counts) // 64)) if self.masks is not None else 0)
        if self.masks is not None:      # tokens past the words' bits are seen by none
            self.masks = [[[j for j in row if j < 64 * self.words] for row in m] for m in self.masks]
        self.see = [pt.tree_sight(n, m, None if self.masks is None else self.masks[b], window, first)
                    for b, (n, m) in enumerate(zip(lens, counts))]
        self.poison()

    def poison(self):
        """What no row of a sequence sees of its cached tokens before the window: NaN, and no block's table entries."""
        c = self.c
        data, meta = wl.cache_views(c.w, c.cache)
        for b, see in enumerate(self.see):
            if not self.window or not len(see):
                continue
            start = max(0, self.lens[b] + 1 - self.window)
            if start <= self.first:
                continue
            t = np.arange(self.first, start)
            assert not see[:, t].any()
            data[c.table[b, t // c.BS], t % c.BS] = 0xFFFF if c.kv == BF16 else 0xFF
            if meta is not None:
                meta[c.table[b, t // c.BS], :, :, t % c.BS] = np.nan if c.kv == FP8 else 0xFFFF
            for j in range(-(-self.first // c.BS), start // c.BS):
                c.table[b, j] = -1 if j % 2 else c.NB + j

    def mask_words(self):
        m = np.zeros((self.N, self.words), np.uint64)
        m[:] = 0xA5A5A5A5A5A5A5A5      # rows of nobody, and bits past a sequence's tokens
        for b, rows in enumerate(self.masks):
            for i, row in enumerate(rows):
                x = sum(1 << j for j in row)
                x |= (0x5A5A << 64 * self.words - 16) >> self.counts[b] << self.counts[b]
                m[self.starts[b] + i] = [(x >> 64 * w) & (1 << 64) - 1 for w in range(self.words)]
        return m

    def device(self, index=0):
        dev = f"cuda:{index}"
        i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(dev)
        c = self.c
        return dict(query=torch.from_numpy(self.q.view(np.int16)).to(dev).view(torch.bfloat16),
                    kv_cache=torch.from_numpy(c.cache).to(dev), num_cache_blocks=c.NB, block_table=i32(c.table),
                    context_lens=i32(self.lens), token_starts=i32(self.starts),
                    tree_masks=None if self.masks is None else torch.from_numpy(self.mask_words().view(np.int64)).to(dev),
                    window=self.window, num_first=self.first,
                    centroids=None if c.book is None else torch.from_numpy(c.book).to(dev))

    def plan(self, pda, **kw):
        return pda.plan(self.B, self.Hk, self.QG, self.BS, self.c.MB, kv_dtype=self.kv, **kw)

    def reference(self, fill=0.0):
        c, QG = self.c, self.QG
        out, bound = np.full((self.N, self.Hk * QG, 128), fill), np.zeros((self.N, self.Hk * QG, 128))
        q = wl.bf16_bits_to_f32(self.q).astype(np.float64)
        for b, n in enumerate(self.counts):
            if n == 0:
                continue
            rows = slice(self.starts[b], self.starts[b] + n)
            used = self.see[b].any(0)
            t = np.flatnonzero(used)         # what nobody sees is left out: its values are NaN
            for h in range(self.Hk):
                k, v, vs, vz = pt.token_values(c.w, c.cache, c.table[b, t // c.BS], t % c.BS, h, c.book)
                r = slice(h * QG, (h + 1) * QG)
                see = np.repeat(self.see[b][:, t], QG, 0)
                o, e = pt.attend(q[rows, r].reshape(n * QG, 128), k, v, see, self.kv, tree=True, vscale=vs, vzero=vz, step=t // 128)
                out[rows, r], bound[rows, r] = o.reshape(n, QG, 128), e.reshape(n, QG, 128)
        return out, bound

    def run(self, pda, d=None, dtype=torch.float32, fill=7.0, p=None, **kw):
        d = d or self.device()
        out = torch.full((self.N, self.Hk * self.QG, 128), fill, dtype=dtype, device=d["kv_cache"].device)
        err = torch.zeros(1, dtype=torch.int32, device=d["kv_cache"].device)
        pda.decode_tree(p or self.plan(pda), **d, out=out, err_word=err, **kw)
        torch.cuda.synchronize()
        return out, int(err.item())

    def check(self, pda, **kw):
        out, err = self.run(pda, **kw)
        assert err == 0
        want, bound = self.reference(fill=7.0)
        off = np.abs(out.cpu().double().numpy() - want)
        worst = float((off / np.maximum(bound, 1e-30)).max())
        assert np.isfinite(off).all() and (off <= bound).all(), (worst, float(off.max()))
        out16, err = self.run(pda, dtype=torch.bfloat16, **kw)
        assert err == 0 and torch.equal(out16, out.to(torch.bfloat16))
        return out
