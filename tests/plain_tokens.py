"""Definitions of the token operators in 64 bits, and how far attention over them may be, term by term.  Test-side only.

With p_t the weight of token t (their sum is 1) and V_t its value, a row's result is sum p_t V_t over the tokens that it sees.  What
the kernels may do to it:
  logits   128 products of q and k are summed in fp32, each addition off by at most a step 2^-23 of |q| |k| (the tensor cores may
           truncate), two more for the scale: 130 of them.  TQ4: centroids are rounded to f16, 2^-11 of every product.  Drafted
           trees, fp8: q, times the power of two that brings its row's largest into [2^7, 2^8), is the sum of two e4m3 parts: the
           high one is off by at most half a step, 2^(e-4) for |q| in [2^e, 2^(e+1)), and that rest is a multiple of q's own
           last bit 2^(e-7), so 4 bits, exact where 2^(e-7) is no less than e4m3's smallest step 2^-9; below, it is off by at
           most 2^-10, 2^-17 of the row's largest; and 256 fp32 additions in place of 128.  A logit off by d moves a weight by
           a factor e^d, and the weights' sum by as much
  P        drafted trees: bf16 KV 2^-8 of the weight; else f16, 2^-11 of it, or 2^-32 of the row's largest where that is more, but
           no more than itself (the reference is 7 below the maximum, half a step of f16's smallest is 2^-25)
           windows (the partition pass): bf16 KV 2^-16 (two bf16 terms); else its product with V's scale to f16, 2^-11, or
           2^-25 of the step's largest scale
  V        drafted trees, fp8: its scale and the scaled value to f16, 2^-11 each, in units F <= f / 2, f the largest scale of the
           step's 128 tokens: half a step of f16's smallest is 2^-25 F <= 2^-26 f.  TQ4: the value to f16 once, 2^-11, in units
           F <= f / 256, f the largest 15 |v_scale| + |v_zero|: 2^-33 f; the fp32 sum before it 2^-21 of 32 |v_scale| + |v_zero|
  sums     over T tokens in fp32, in any order, each addition off by at most a step 2^-23 of sum p |V|; 64 more for ex2, the
           factors, the rescales and the joins
"""
from __future__ import annotations

import numpy as np

from paged_kv_gqa_block_gb300 import workloads as wl
from tests import plain_pages as pp

BF16, FP8, TQ4 = wl.KV_BF16, wl.KV_FP8_E4M3, wl.KV_TQ4
SCALE = 128 ** -0.5


def attend(q, k, v, see, kv, *, tree, vscale=None, vzero=None, step=None, used=None, scale=SCALE):
    """(out, bound) [rows][128] of rows q over tokens k, v that they see (see [rows][T]).  tree: the tensor-core pass; else the
    partition pass.  vscale, vzero [T]: V's fields; step [T]: the step a token belongs to; used [T]: some row sees it."""
    rows, T = see.shape
    out, bound = np.zeros((rows, 128)), np.zeros((rows, 128))
    live = see.any(-1)
    if not live.any():
        return out, bound
    used = see.any(0) if used is None else used
    k, v = np.where(used[:, None], k, 0.0), np.where(used[:, None], v, 0.0)      # what nobody sees may hold anything
    s = np.where(see, scale * q @ k.T, -np.inf)
    top = np.where(live, s.max(-1), 0.0)[:, None]
    p = np.exp(s - top)
    p /= np.where(live, p.sum(-1), 1.0)[:, None]
    out = p @ v
    a = np.abs(v)
    reach = np.where(see, scale * np.abs(q) @ np.abs(k).T, 0.0).max(-1, keepdims=True)
    ds = reach * (130 * 2.0 ** -23 + (2.0 ** -11 * 1.001 if kv == TQ4 else 0.0))
    if kv == FP8 and tree:
        size = np.where(see, np.abs(k).sum(-1), 0.0).max(-1, keepdims=True)
        ds = ds + reach * 1.1 * 128 * 2.0 ** -23 + 2.0 ** -17 * scale * np.abs(q).max(-1, keepdims=True) * size
    e = (np.expm1(2 * ds) + (T + 64) * 2.0 ** -23) * (p @ a)
    big = p.max(-1, keepdims=True)
    eps = 2.0 ** -11
    if kv == BF16:
        e += (2.0 ** -8 if tree else 2.0 ** -16) * (p @ a)
    elif tree:
        w = np.maximum(eps * p, np.minimum(p, 2.0 ** -32 * big * (1 + ds)))
        f = np.zeros(T)
        size = np.abs(vscale) if kv == FP8 else 15 * np.abs(vscale) + np.abs(vzero)
        size = np.where(used, size, 0.0)
        for g in np.unique(step):
            f[step == g] = size[step == g].max()
        if kv == FP8:
            code = a / np.where(size == 0, 1, size)[:, None]
            f16 = 2 * eps * a + np.where((size < 2.0 ** -15 * f)[:, None], 2.0 ** -26 * f[:, None] * code, 0)
            f16 = f16 + np.where(a < 2.0 ** -15 * f[:, None], 2.0 ** -26 * f[:, None], 0)
        else:
            f16 = eps * a + 2.0 ** -33 * f[:, None] + 2.0 ** -21 * np.where(used, 32 * np.abs(vscale) + np.abs(vzero), 0.0)[:, None]
        e += (1 + 2.0 ** -9) * (1 + np.expm1(2 * ds)) * (w @ a + p @ f16)
    else:
        size = np.where(used, np.abs(vscale), 0.0)
        # codes times (weight times scale): the product with the scale is what is rounded
        code = a if kv == FP8 else np.abs(v - np.where(used, vzero, 0.0)[:, None])
        per = code / np.where(size == 0, 1, size)[:, None]
        e += (1 + 2.0 ** -9) * (eps * (p @ code) + 2.0 ** -25 * 64 * size.max() * (big * (p > 0)) @ per)
        if kv == TQ4:   # code * v_scale and v_zero are summed apart
            e += (T + 64) * 2.0 ** -23 * (p @ (code + np.abs(np.where(used, vzero, 0.0))[:, None]))
    return out, e * live[:, None]


class Pool:
    """Sequences of total[b] tokens in one pool whose unused slots hold NaN; K, V ~ N(0, 1) with a few large."""

    def __init__(self, kv, Hk, QG, BS, total, seed=0, MB=None, v_spread=0.0, spare=3):
        rng = self.rng = np.random.default_rng(seed)
        self.kv, self.Hk, self.QG, self.BS, self.B = kv, Hk, QG, BS, len(total)
        self.total = [int(n) for n in total]
        need = [-(-n // BS) for n in self.total]
        self.MB = MB or max(1, max(need, default=1))
        self.NB = sum(need) + spare
        self.w = wl.Workload("tokens", self.B, Hk, QG, BS, self.MB, self.NB, ("list", tuple(self.total)), seed=0, kv_dtype=kv)
        self.cache = wl.empty_cache(self.w)
        self.book = wl.tq4_codebook() if kv == TQ4 else None
        ids, at = rng.permutation(self.NB).astype(np.int32), 0
        self.table = np.full((self.B, self.MB), -1, np.int32)
        for b, n in enumerate(self.total):
            row = ids[at:at + need[b]]
            at += need[b]
            self.table[b, :need[b]] = row
            k = rng.standard_normal((n, Hk, 128)).astype(np.float32)
            v = (rng.standard_normal((n, Hk, 128)) * np.exp(v_spread * rng.standard_normal((n, Hk, 1)))).astype(np.float32)
            if n and kv == BF16:
                k, v = (wl.bf16_bits_to_f32(wl.round_bf16(x)) for x in (k, v))
            wl.write_tokens(self.w, self.cache, row, k, v, self.book)

    def values(self, b, h, n=None):
        """K, V [n][128] of the first n tokens of a sequence and head, and V's fields (None without), in 64 bits."""
        n = self.total[b] if n is None else n
        t = np.arange(n)
        return token_values(self.w, self.cache, self.table[b, t // self.BS], t % self.BS, h, self.book)


def token_values(w, cache, ids, slots, h, book=None):
    data, meta = wl.cache_views(w, cache)
    x = data[ids, slots, h]
    if w.kv_dtype == BF16:
        f = wl.bf16_bits_to_f32(x).astype(np.float64)
        return f[:, 0], f[:, 1], None, None
    if w.kv_dtype == FP8:
        m = meta[ids, h, :, slots].astype(np.float64)
        import torch
        f = torch.from_numpy(np.ascontiguousarray(x)).view(torch.float8_e4m3fn).double().numpy()
        return f[:, 0] * m[:, :1], f[:, 1] * m[:, 1:], m[:, 1], np.zeros(len(m))
    m = meta[ids, h, :, slots].view(np.float16).astype(np.float64)
    code = np.stack([x & 15, x >> 4], -1).reshape(len(x), 2, 128)
    return (np.asarray(book, np.float64)[code[:, 0]] * m[:, :1], code[:, 1] * m[:, 1:2] + m[:, 2:], m[:, 1], m[:, 2])


def tq4_keys(K, book):
    """wl.quantize_tq4_k with the norm rounded to f16 once (the generator goes by way of fp32, which can round twice: 10.5429684
    lies below 10.54296875, the middle of two f16 values, and its fp32 value on it)."""
    norm = np.sqrt((K.astype(np.float64) ** 2).sum(-1)).astype(np.float16)
    unit = K / np.where(norm > 0, norm, np.float16(1)).astype(np.float32)[..., None]
    return np.searchsorted((book[1:] + book[:-1]) / 2, unit, side="left").astype(np.uint8), norm.view(np.uint16)


def quantised(kv, K, V, book):
    """The cache's bytes and fields of token rows K, V [n][Hk][128] (fp32 of bf16 values): data [n][Hk][2][bytes] uint8 and
    fields [n][Hk][F], by the generator's quantisers but for tq4_keys."""
    if kv == BF16:
        return np.stack([wl.round_bf16(K), wl.round_bf16(V)], 2).view(np.uint8), None
    if kv == FP8:
        (kc, ks), (vc, vs) = wl.quantize_e4m3_rows(K), wl.quantize_e4m3_rows(V)
        return np.stack([kc, vc], 2), np.stack([ks, vs], -1)
    kc, kn = tq4_keys(K, book)
    vc, vs, vz = wl.quantize_tq4_v(V)
    return np.stack([wl.pack_nibbles(kc), wl.pack_nibbles(vc)], 2), np.stack([kn, vs, vz], -1)


def store(w, cache, ids, slots, data, fields):
    d, m = wl.cache_views(w, cache)
    d[ids, slots] = data.view(np.uint16) if w.kv_dtype == BF16 else data
    if m is not None:
        m[ids, :, :, slots] = fields


def tree_sight(ctx, n, masks, window, first):
    """[n][ctx + n]: what drafted token i of a sequence sees.  masks: n lists of indices, or None for a chain."""
    see = np.zeros((n, ctx + n), bool)
    t = np.arange(ctx)
    for i in range(n):
        row = [j for j in (masks[i] if masks is not None else range(i + 1)) if j < n]
        pos = ctx + len([j for j in row if j != i])
        see[i, :ctx] = True if not window else (pos - t < window) | (t < first)
        for j in row:
            if masks is not None or not window or ctx + i - (ctx + j) < window or ctx + j < first:
                see[i, ctx + j] = True
    return see
