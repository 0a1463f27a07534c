"""Writes and reads of many tokens, which take up to four heads of a token at a time and several tokens per CTA: byte for byte
against the generator's quantisers, and against the same tokens in small calls."""
import numpy as np
import pytest
import torch

from paged_kv_gqa_block_gb300 import workloads as wl
from tests import plain_tokens as pt
from tests.test_tokens_gpu import bf16, expected_write, i32, places, setup, write

pytestmark = pytest.mark.gpu

BF16, FP8, TQ4 = wl.KV_BF16, wl.KV_FP8_E4M3, wl.KV_TQ4
KVS = [BF16, FP8, TQ4]
FEW = 4 * 152 * 8      # rows (tokens times heads) of a call that takes one at a time


@pytest.fixture(scope="module")
def pda():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_gqa_block_gb300 as pda
    return pda


def case(pda, kv, Hk, BS, tokens):
    """About so many tokens: sequences of very unlike length, some without a place, rows of nobody around them."""
    counts = [tokens // 2, 0, 1, tokens // 4 + 3, 37, tokens // 4, 5]
    positions = [3, 9, 0, 1000, -1, BS - 1, -4]
    return setup(pda, kv, Hk, BS, positions, counts, seed=Hk + BS, before=5, after=11)


def read_back(pda, c, cache, dtype, starts=None):
    out = [torch.full((c.N, c.Hk, 128), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pda.read_kv(c.p, cache, c.NB, i32(c.table), i32(c.starts if starts is None else starts), i32(c.positions), *out, centroids=c.cent,
                err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return out


def expected_read(c, dtype):
    want = np.full((2, c.N, c.Hk, 128), 7.0)
    for b in range(c.B):
        if c.positions[b] >= 0 and c.starts[b + 1] > c.starts[b]:
            for h in range(c.Hk):
                k, v, _, _ = pt.token_values(c.w, c.cache, *places(c, b), h, c.book)
                want[0, c.starts[b]:c.starts[b + 1], h], want[1, c.starts[b]:c.starts[b + 1], h] = k, v
    return torch.from_numpy(want).float().to(dtype)


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("Hk,BS", [(1, 16), (2, 32), (3, 16), (4, 32), (5, 16), (6, 32), (7, 16), (8, 16), (13, 32)])
def test_bytes_and_values(pda, kv, Hk, BS):
    """Heads in fours with a rest of one, two, three or none; a CTA's tokens in whole rounds of its warps."""
    c = case(pda, kv, Hk, BS, FEW // Hk + 700)
    assert c.N * Hk > FEW
    cache = torch.from_numpy(c.cache).cuda()
    assert write(pda, c, cache) == 0
    c.cache = expected_write(c)
    assert np.array_equal(cache.cpu().numpy(), c.cache)
    for dtype in (torch.float32, torch.bfloat16):
        for got, want in zip(read_back(pda, c, cache, dtype), expected_read(c, dtype)):
            assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("Hk", [3, 8])
def test_large_calls_are_many_small_ones(pda, kv, Hk):
    """More tokens than one wave of CTAs takes (32 each, 16 in reads), and the same rows in calls of one row at a time per warp."""
    c = case(pda, kv, Hk, 16, 24000)
    assert c.N > 32 * 4 * 152
    one, many = (torch.from_numpy(c.cache).cuda() for _ in range(2))
    assert write(pda, c, many) == 0
    whole = read_back(pda, c, many, torch.float32)
    k, v = bf16(c.bits[0]), bf16(c.bits[1])
    step = FEW // Hk
    for first in range(0, c.N, step):
        n = min(step, c.N - first)
        # this part of every sequence: it begins inside those that an earlier part has begun
        starts = np.clip(c.starts - first, 0, n)
        skipped = np.clip(first - c.starts[:-1], 0, np.diff(c.starts))
        positions = np.where(np.array(c.positions) < 0, -1, np.array(c.positions) + skipped)
        pda.write_kv(c.p, k[first:first + n], v[first:first + n], one, c.NB, i32(c.table), i32(starts), i32(positions), centroids=c.cent)
        part = [torch.full((n, Hk, 128), 7.0, device="cuda") for _ in range(2)]
        pda.read_kv(c.p, many, c.NB, i32(c.table), i32(starts), i32(positions), *part, centroids=c.cent)
        for a, b in zip(part, whole):
            assert torch.equal(a, b[first:first + n])
    assert torch.equal(one, many)
