"""How far a decode step over shared prefixes may be from its result in 64 bits, term by term.  Test-side only.

With p_t the weight of token t (their sum is 1) and V_t its value, the result is sum p_t V_t.  What the step may do to it:
  logits   128 products of q and k are summed in fp32, each addition off by at most a step 2^-23 of |q| |k| (the tensor cores
           may truncate), two more for the scale: 130 of them, ds, move a weight by ds, and the weights' sum by as much
  P        bf16: 2^-8 of the weight.  f16: 2^-11 of it, or 2^-32 of the row's largest where that is more, but no more than itself:
           the reference is 7 below the maximum, and half a step of f16's smallest is 2^-25
  V (fp8)  its scale to f16 and the scaled value to f16, 2^-11 each, in units F <= f / 2, f the largest scale of the token's aligned
           128 tokens: half a step of f16's smallest is 2^-25 F <= 2^-26 f, for a scale below 2^-15 f (times the code) and for
           a value below 2^-15 f
  sums     over T tokens in fp32, in any order, each addition off by at most a step 2^-23 of sum p |V|; 64 more for ex2, the
           factors, the rescales and the join of the pieces
The own tokens' part is the library's partition pass: fewer roundings than the prefix's, but its f16 weights times V's scale (fp8) are
off by half a step of f16's smallest, 2^-25 of its largest value, where they are small.
"""
from __future__ import annotations

import numpy as np

from paged_kv_gqa_block_gb300 import workloads as wl
from tests import plain_pages as pp

BF16 = wl.KV_BF16


def tokens(c, b, drop=None):
    """K ids of sequence b: (block ids, slots, is a prefix token, the token's aligned 128 tokens) of every token, prefix first.
    drop = (first, last): these prefix tokens are left out."""
    ids, slots, prefix, span = [], [], [], []
    for g in range(len(c.plens)):
        if c.starts[g] <= b < c.starts[g + 1]:
            t = np.arange(c.plens[g])
            if drop:
                t = t[(t < drop[0]) | (t >= drop[1])]
            ids.append(c.ptable[g, t // c.BS])
            slots.append(t % c.BS)
            prefix.append(np.ones(len(t), bool))
            span.append(t // 128 + 1000000 * g)
    t = np.arange(c.lens[b])
    ids.append(c.table[b, t // c.BS])
    slots.append(t % c.BS)
    prefix.append(np.zeros(len(t), bool))
    span.append(np.full(len(t), -1))
    return [np.concatenate(x) for x in (ids, slots, prefix, span)]


def result(c, scale=128 ** -0.5, drop=None, rows=None):
    """(out, bound) in 64 bits, of the sequences `rows` (all)."""
    K, V = pp.block_values(c.w, c.cache)
    _, meta = wl.cache_views(c.w, c.cache)
    q = wl.bf16_bits_to_f32(c.q).astype(np.float64)
    shape = (c.B, c.Hk * c.QG, 128)
    out, bound = np.zeros(shape), np.zeros(shape)
    for b in range(c.B) if rows is None else rows:
        ids, slots, prefix, span = tokens(c, b, drop)
        T = len(ids)
        if T == 0:
            continue
        for h in range(c.Hk):
            k, v = K[ids, slots, h], V[ids, slots, h]
            r = slice(h * c.QG, (h + 1) * c.QG)
            s = scale * q[b, r] @ k.T
            p = np.exp(s - s.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            out[b, r] = p @ v
            top = p.max(-1, keepdims=True)
            ds = scale * (np.abs(q[b, r]) @ np.abs(k).T).max(-1, keepdims=True) * 130 * 2.0 ** -23
            a = np.abs(v)
            e = (2 * ds + (T + 64) * 2.0 ** -23) * (p @ a)
            if c.kv == BF16:
                e += 2.0 ** -8 * (p @ a)
            else:
                eps = 2.0 ** -11
                w = np.maximum(eps * p, np.minimum(p, 2.0 ** -32 * top * (1 + ds)))          # the weights' rounding
                f16 = 2 * eps * a                                                            # V's two
                sv = np.abs(np.asarray(meta, np.float64)[ids, h, 1, slots])
                f = np.zeros(T)
                for g in np.unique(span):
                    f[span == g] = sv[span == g].max()
                code = a / np.where(sv == 0, 1, sv)[:, None]
                f16 += np.where((sv < 2.0 ** -15 * f)[:, None], 2.0 ** -26 * f[:, None] * code, 0)
                f16 += np.where(a < 2.0 ** -15 * f[:, None], 2.0 ** -26 * f[:, None], 0)
                e += (1 + 2.0 ** -9) * (w @ a + p @ f16)                                     # second orders
                if (~prefix).any():
                    e += (~prefix).sum() * 2.0 ** -25 * top * a[~prefix].max()
            bound[b, r] = e
    return out, bound
