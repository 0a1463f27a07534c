"""Inputs of the shared-prefix tests that hold the tight bound.  Test-side only."""
from __future__ import annotations

import numpy as np

from paged_kv_gqa_block_gb300 import workloads as wl
from tests.test_shared_gpu import Case

FORMATS = [wl.KV_BF16, wl.KV_FP8_E4M3]

# Hk, QG, BS, prefix lengths, group sizes, own lengths; "lost": whether any lost step shows (not where its weights are near zero, nor
# beside the fp32 sums of 20000 tokens)
CASES = {
    "one piece": dict(a=(1, 8, 16, [300], [3], [5, 1, 40])),
    "ragged": dict(a=(2, 6, 32, [1000], [7], [0, 1, 32, 33, 70, 5, 260])),
    "pieces of two groups": dict(a=(2, 8, 32, [5000, 777], [40, 2], [3] * 42)),
    "one piece each": dict(a=(2, 8, 32, [5000, 777], [40, 2], [3] * 42), plans=dict(prefix_tile_groups=1000)),
    "two row tiles": dict(a=(1, 16, 16, [2049], [33], [17] * 33)),
    "long": dict(a=(1, 8, 32, [20000], [5], [0, 0, 100, 3, 1]), lost=False),
    "spread values": dict(a=(1, 8, 16, [1500], [20], [30] * 20), kw=dict(v_spread=3.0), lost=False),
    "large logits": dict(a=(1, 8, 16, [1500], [20], [30] * 20), kw=dict(q_scale=8.0, v_spread=1.0), lost=False),
    "offset keys": dict(a=(2, 6, 16, [900], [50], [9] * 50), kw=dict(q_scale=1e-3, k_bias=3.0)),
    "sink": dict(a=(1, 8, 32, [32768], [4], [0, 3, 1, 0]), sink=17.5, lost=False),
    "sink in one piece": dict(a=(1, 8, 32, [32768], [4], [0, 3, 1, 0]), sink=17.5, plans=dict(prefix_tile_groups=1000), lost=False),
    "far sink": dict(a=(1, 8, 32, [20000], [4], [0, 0, 0, 0]), sink=21.0, lost=False),
    "sink in the middle": dict(a=(1, 8, 32, [16384], [2], [0, 5]), sink=16.0, at=9000, lost=False),
}


def make(name, kv):
    x = CASES[name]
    Hk, QG, BS, plens, sizes, lens = x["a"]
    c = Case(kv, Hk, QG, BS, plens, sizes, lens, seed=sum(map(ord, name)), **x.get("kw", {}))
    c.plan_kw = x.get("plans", {})
    if "sink" in x:
        # One key far along every query's first dimension, whose value is zero, and a long remainder of nearly equal logits `sink`
        # below it (natural units), whose values add up.
        rng = np.random.default_rng(1)
        n = plens[0]
        q = (0.1 * rng.standard_normal((c.B, Hk * QG, 128))).astype(np.float32)
        q[..., 0] = 64.0
        c.q = wl.round_bf16(q)
        k = rng.standard_normal((n, Hk, 128)).astype(np.float32)
        k[..., 0] = 0.0
        v = (1.0 + 0.5 * rng.standard_normal((n, Hk, 128))).astype(np.float32)
        at = x.get("at", 0)
        k[at], v[at] = 0.0, 0.0
        k[at, :, 0] = x["sink"] * 128 ** 0.5 / 64.0
        wl.write_tokens(c.w, c.cache, c.ptable[0], k, v)
    return c
