"""The page operations and the block-sparse operators by definition: sequential numpy on the host,
64 bits for everything that is computed.  Test-side only."""
from __future__ import annotations

import numpy as np

from paged_kv_gqa_block_gb300 import workloads as wl

BAD_LEN, BAD_ID, BAD_POS, BAD_SEQ, NO_BLOCKS = 1, 2, 8, 16, 32


def copy(src, dst, pairs, block_bytes, same):
    """dst after the pairs (src and dst flat uint8); `same`: dst is src's pool."""
    a, out, err = src.reshape(-1, block_bytes), dst.copy().reshape(-1, block_bytes), 0
    for s, d in pairs:
        if s < 0 or d < 0:
            continue
        if s >= len(a) or d >= len(out):
            err |= BAD_ID
            continue
        out[d] = a[s]
    return out.reshape(-1), err


def fork(cache, block_bytes, BS, table, lens, refs, parents, grow):
    """(cache, out_table, out_lens, out_refs, error word) of pda_fork_sequences."""
    B, MB = table.shape
    NB, err = len(refs), 0
    blocks = cache.copy().reshape(NB, block_bytes)
    out_refs = refs.copy()
    lens = [int(x) for x in lens]
    for b in range(B):
        if lens[b] < 0 or lens[b] > MB * BS:
            lens[b], err = 0, err | BAD_LEN
        for j in range(-(-lens[b] // BS)):
            i = int(table[b, j])
            if 0 <= i < NB:
                out_refs[i] -= 1
            else:
                err |= BAD_ID
    free = [i for i in range(NB) if refs[i] == 0]
    out_table = np.full((len(parents), MB), -1, np.int32)
    out_lens = np.zeros(len(parents), np.int32)
    at, seen = 0, set()
    for r, p in enumerate(parents):
        p = int(p)
        if p < 0:
            continue
        if p >= B:
            err |= BAD_SEQ
            continue
        L, g = lens[p], 0 if grow is None else int(grow[r])
        if g < 0 or L + g > MB * BS:
            err |= BAD_POS
            continue
        first = p not in seen
        seen.add(p)
        full, h0, h1 = L // BS, -(-L // BS), -(-(L + g) // BS)
        ids = [int(x) for x in table[p, :h0]]
        copied = h0 > full and 0 <= ids[full] < NB and not (first and refs[ids[full]] == 1)
        need = int(copied) + h1 - h0
        if at + need > len(free) and need > 0:
            err |= NO_BLOCKS
            at += need
            continue
        fresh = free[at:at + need]
        at += need
        if copied:
            blocks[fresh[0]] = blocks[ids[full]]
            ids[full] = fresh.pop(0)
        ids += fresh
        out_table[r, :h1] = ids
        out_lens[r] = L + g
        for i in ids:
            if 0 <= i < NB:
                out_refs[i] += 1
    return blocks.reshape(-1), out_table, out_lens, out_refs, err


def compact(cache, block_bytes, BS, table, lens, refs):
    """(cache, out_table, out_refs, remap, U, error word) of pda_compact_blocks."""
    NB, MB, err = len(refs), table.shape[1], 0
    blocks = cache.copy().reshape(NB, block_bytes)
    U = int((refs > 0).sum())
    remap = np.where(refs > 0, np.arange(NB), -1).astype(np.int32)
    movers = [i for i in range(U, NB) if refs[i] > 0]
    holes = [i for i in range(U) if refs[i] <= 0]
    out_refs = np.where((np.arange(NB) < U) & (refs > 0), refs, 0).astype(np.int32)
    for a, b in zip(movers, holes):
        blocks[b] = blocks[a]
        remap[a], out_refs[b] = b, refs[a]
    out_table = np.full(table.shape, -1, np.int32)
    for b in range(len(lens)):
        L = int(lens[b])
        if L < 0 or L > MB * BS:
            err |= BAD_LEN
            continue
        for j in range(-(-L // BS)):
            i = int(table[b, j])
            if 0 <= i < NB and remap[i] >= 0:
                out_table[b, j] = remap[i]
            else:
                err |= BAD_ID
    return blocks.reshape(-1), out_table, out_refs, remap, U, err


# ------------------------------------------------------------------------------------------------
def block_values(w: wl.Workload, cache, centroids=None):
    """float64 K and V of every block: [NB][BS][Hk][D] each, from the stored bits alone."""
    data, meta = wl.cache_views(w, cache)
    with np.errstate(invalid="ignore"):
        if w.kv_dtype == wl.KV_BF16:
            x = wl.bf16_bits_to_f32(data).astype(np.float64)
            return x[..., 0, :], x[..., 1, :]
        if w.kv_dtype == wl.KV_FP8_E4M3:
            import torch
            x = torch.from_numpy(np.ascontiguousarray(data)).view(torch.float8_e4m3fn).to(torch.float64).numpy()
            sc = np.asarray(meta, dtype=np.float64).transpose(0, 3, 1, 2)[..., None]      # [NB][BS][Hk][2][1]
            x = x * sc
            return x[..., 0, :], x[..., 1, :]
        packed = np.asarray(data)
        codes = np.stack([packed & 15, packed >> 4], axis=-1).reshape(*packed.shape[:-1], 128)
        f = np.ascontiguousarray(meta).view(np.float16).astype(np.float64).transpose(0, 3, 1, 2)[..., None]  # [NB][BS][Hk][3][1]
        k = np.asarray(centroids, np.float32).astype(np.float64)[codes[..., 0, :]] * f[..., 0, :]
        return k, codes[..., 1, :] * f[..., 1, :] + f[..., 2, :]


def attention(q, k, v, scale):
    """softmax(scale q k^T) v in float64; a query without keys gives zeros."""
    if len(k) == 0:
        return np.zeros_like(q)
    s = scale * q @ k.T
    p = np.exp(s - s.max(-1, keepdims=True))
    return p @ v / p.sum(-1, keepdims=True)


def select(scores, lens, BS, K, first, last):
    """Logical indices of the selected blocks, ascending: a list per (sequence, KV head)."""
    out = []
    for b in range(scores.shape[0]):
        nb = -(-int(lens[b]) // BS)
        for h in range(scores.shape[1]):
            s = scores[b, h, :nb]
            if nb <= K:
                out.append(list(range(nb)))
                continue
            forced = set(range(min(first, nb))) | set(range(max(0, nb - last), nb))
            rest = sorted((j for j in range(nb) if j not in forced),
                          key=lambda j: (np.isnan(s[j]), -s[j] if not np.isnan(s[j]) else 0.0, j))
            out.append(sorted(forced | set(rest[:K - len(forced)])))
    return out
