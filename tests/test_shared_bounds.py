"""The bound that the GPU tests of shared prefixes use tells a step of lost tokens from rounding (no GPU needed)."""
import numpy as np
import pytest

from paged_kv_gqa_block_gb300 import workloads as wl
from tests import plain_pages as pp
from tests import shared_bounds as sb
from tests.shared_cases import CASES, FORMATS, make


@pytest.mark.parametrize("kv", FORMATS)
@pytest.mark.parametrize("name", [n for n in CASES if CASES[n].get("lost", True)])
def test_a_lost_step_is_further_off_than_the_bound(kv, name):
    c = make(name, kv)
    row = c.starts[int(np.argmax(c.plens))]                  # a sequence of the longest prefix's group
    T = max(c.plens)
    out, bound = sb.result(c, rows=[row])
    steps = list(range(0, T, 128))
    for s in steps[::max(1, len(steps) // 6)] + steps[-1:]:
        n = min(T, s + 128) - s
        less, _ = sb.result(c, drop=(s, s + n), rows=[row])
        over = (np.abs(less - out) / bound.clip(1e-300))[row].max()
        assert over > (1.3 if n > 8 else 0.6), (s, n, over)


def test_rounding_weights_to_f16_at_the_maximum_is_outside_the_bound():
    """The loss that a sink key shows: weights below 2^-25 of the largest become zero where the reference is the maximum, and keep
    eleven bits where it is 7 below."""
    c = make("sink", FORMATS[1])
    out, bound = sb.result(c, rows=[0])
    K, V = pp.block_values(c.w, c.cache)
    ids, slots, _, _ = sb.tokens(c, 0)
    q = wl.bf16_bits_to_f32(c.q).astype(np.float64)
    s = 128 ** -0.5 * q[0, :c.QG] @ K[ids, slots, 0].T / np.log(2)
    for below, inside in ((0, False), (7, True)):
        P = 2.0 ** (s - s.max(-1, keepdims=True) + below)
        got = P.astype(np.float16).astype(np.float64) @ V[ids, slots, 0] / P.sum(-1, keepdims=True)
        assert (np.abs(got - out[0, :c.QG]) <= bound[0, :c.QG]).all() == inside
