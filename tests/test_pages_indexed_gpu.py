"""Page operators with what else block ids index: other pools under the same tables, and block summaries."""
import numpy as np
import pytest
import torch

from paged_kv_gqa_block_gb300 import workloads as wl
from tests import plain_pages as pp
from tests.test_pages_gpu import batch, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pda():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_gqa_block_gb300 as pda
    return pda


def model(pda, layers, lens, NB, MB, seed=0):
    """Pools of several layers under one set of tables."""
    rng = np.random.default_rng(seed)
    BS, Hk = 16, 2
    table, refs = batch(rng, lens, BS, MB, NB)
    w = wl.Workload("layers", len(lens), Hk, 8, BS, MB, NB, ("list", tuple(int(x) for x in lens)), seed=0)
    caches = []
    for _ in range(layers):
        c = wl.empty_cache(w)
        wl.write_tokens(w, c, np.arange(NB, dtype=np.int32), *(rng.standard_normal((NB * BS, Hk, 128)).astype(np.float32) for _ in range(2)))
        caches.append(c)
    return w, table, refs, caches


def test_other_layers_follow_a_fork_and_a_compaction(pda):
    lens = np.array([33, 16, 5, 47, 0], np.int32)
    w, table, refs, caches = model(pda, 2, lens, 60, 6)
    NB, BS, MB, B, R = 60, 16, 6, 5, 7
    p, pR = pda.plan(B, 2, 8, BS, MB), pda.plan(R, 2, 8, BS, MB)
    parents, grow = np.array([0, 0, 3, 3, 1, 2, -1], np.int32), np.array([1, 1, 0, 20, 1, 0, 0], np.int32)
    want = [pp.fork(c, p.cache_block_bytes, BS, table, lens, refs, parents, grow) for c in caches]
    d = [dev(c) for c in caches]
    t, l, r = dev(table), dev(lens), dev(refs)
    nt, nl, nr = torch.empty((R, MB), dtype=torch.int32, device="cuda"), torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty_like(r)
    par = dev(parents)
    pda.fork_sequences(p, d[0], NB, t, l, r, par, nt, nl, nr, pda.page_workspace(p, R, NB, "cuda"), new_tokens=dev(grow))
    # the copies of the other layers, as the documentation states them
    alive = par.clamp(min=0).long()
    old = l[alive]
    j = (old // BS).long().clamp(max=MB - 1)
    src, dst = t[alive, j], nt.gather(1, j[:, None])[:, 0]
    copied = (par >= 0) & (old % BS != 0) & (src != dst) & (nl > 0)
    pairs = torch.where(copied[:, None], torch.stack([src, dst], 1), -1).int().contiguous()
    pda.copy_blocks(p, d[1], NB, d[1], NB, pairs)
    for x, y in zip(d, want):
        assert np.array_equal(x.cpu().numpy(), y[0])
    refs2, table2, lens2 = nr.cpu().numpy(), nt.cpu().numpy(), nl.cpu().numpy()
    before = [x.cpu().numpy() for x in d]
    ct, cr, remap, used = torch.empty_like(nt), torch.empty_like(nr), torch.empty_like(nr), torch.empty(1, dtype=torch.int32, device="cuda")
    pda.compact_blocks(pR, d[0], NB, nt, nl, nr, ct, cr, remap, used, pda.page_workspace(pR, 0, NB, "cuda"))
    pda.copy_blocks(pR, d[1], NB, d[1], NB, torch.stack([torch.arange(NB, dtype=torch.int32, device="cuda"), remap], 1).contiguous())
    for x, y in zip(d, before):
        assert np.array_equal(x.cpu().numpy(), pp.compact(y, p.cache_block_bytes, BS, table2, lens2, refs2)[0])


def test_summaries_after_pages_move(pda):
    """Scores and selections are the same before a compaction and after it, once the summaries' rows moved with their blocks, or were
    renewed; a forked batch selects as its parents did, once the copied blocks' rows are renewed."""
    lens = np.array([300, 700, 37, 512], np.int32)
    B, BS, MB, NB, K = 4, 16, 50, 300, 6
    w, table, refs, (cache,) = model(pda, 1, lens, NB, MB, seed=2)
    p = pda.plan(B, 2, 8, BS, MB)
    t, l, r, c = dev(table), dev(lens), dev(refs), dev(cache)
    q = torch.randn((B, 16, 128), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()

    def chosen(p, q, summ, t, l):
        n = len(l)
        scores = torch.full((n, 2, MB), -7.0, device="cuda")
        sel = torch.empty((n, 2, K), dtype=torch.int32, device="cuda")
        blocks, tokens = torch.empty_like(sel), torch.empty((n, 2), dtype=torch.int32, device="cuda")
        pda.score_blocks(p, q, summ, NB, t, l, scores)
        pda.select_blocks(p, scores, t, l, K, 1, 1, sel, tokens, sel_blocks=blocks)
        return scores, blocks, tokens

    summ = pda.block_summaries(p, NB, "cuda").fill_(9.0)     # what earlier use of an id left behind scores highest
    pda.summarize_blocks(p, c, NB, t, l, summ)
    want = chosen(p, q, summ, t, l)
    ct, cr, remap, used = torch.empty_like(t), torch.empty_like(r), torch.empty_like(r), torch.empty(1, dtype=torch.int32, device="cuda")
    pda.compact_blocks(p, c, NB, t, l, r, ct, cr, remap, used, pda.page_workspace(p, 0, NB, "cuda"))
    assert not torch.equal(chosen(p, q, summ, ct, l)[1], want[1])          # the rows are still the old ids'
    moved, held = summ.clone(), remap >= 0
    moved[remap[held].long()] = summ[held]
    renewed = torch.full_like(summ, 9.0)
    pda.summarize_blocks(p, c, NB, ct, l, renewed)
    for x in (moved, renewed):
        for a, b in zip(chosen(p, q, x, ct, l), want):
            assert torch.equal(a, b)
    # fork: two children each, the second with a copy of the last block
    par = torch.tensor([0, 0, 1, 1, 2, 2, 3, 3], dtype=torch.int32, device="cuda")
    p8 = pda.plan(8, 2, 8, BS, MB)
    ft, fl, fr = torch.empty((8, MB), dtype=torch.int32, device="cuda"), torch.empty(8, dtype=torch.int32, device="cuda"), torch.empty_like(cr)
    pda.fork_sequences(p, c, NB, ct, l, cr, par, ft, fl, fr, pda.page_workspace(p, 8, NB, "cuda"))
    pda.summarize_blocks(p8, c, NB, ft, fl, moved, since=fl - 1)
    for a, b in zip(chosen(p8, q[par.long()].contiguous(), moved, ft, fl), want):
        assert torch.equal(a, b[par.long()])
