"""A shared step whose every input is written by kernels directly in front of it on the stream, many steps without a pause: each
gives what it gives alone.  Of a step's two passes the second starts while the first still runs, so it must not see what the step
before it read.  Both orders of the passes: short prefixes first, own tokens first."""
import numpy as np
import pytest
import torch

from paged_kv_gqa_block_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

# sequences, KV heads, groups, prefix tokens, whether the prefix pass is the first (the host's rule on sizes)
SIZES = {"prefix first": (32, 8, 2, 1500), "own first": (40, 8, 3, 5000), "small": (3, 1, 1, 250)}
N = 12                                                       # variants of the inputs


@pytest.fixture(scope="module")
def pda():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_gqa_block_gb300 as pda
    return pda


class Stage:
    """A pool full of finite tokens, N variants of every input, and the live inputs that kernels write before each step."""

    def __init__(self, pda, kv, sizes):
        self.pda, self.kv = pda, kv
        B, Hk, NG, prefix = sizes
        BS, MB, MP = 16, 6, -(-prefix // 16)
        self.B, self.Hk, self.NG, self.MB, self.BS = B, Hk, NG, MB, BS
        rng = np.random.default_rng(B)
        NB = self.NB = NG * MP + 2 * B * MB + 7
        w = wl.Workload("order", B, Hk, 8, BS, MB, NB, ("list", (1,) * B), seed=0, kv_dtype=kv)
        cache = wl.empty_cache(w)
        kvs = [rng.standard_normal((NB * BS, Hk, 128)).astype(np.float32) for _ in range(2)]
        wl.write_tokens(w, cache, np.arange(NB, dtype=np.int32), *kvs)
        dev = lambda x, t=np.int32: torch.from_numpy(np.ascontiguousarray(x, t)).cuda()
        self.cache0 = dev(cache, np.uint8)
        self.cache = self.cache0.clone()
        ids = rng.permutation(NB).astype(np.int32)
        own = ids[NG * MP:NG * MP + B * MB].reshape(B, MB)
        v = dict(starts=[], ptable=[], plens=[], table=[], lens=[], q=[], k=[], v=[])
        for _ in range(N):
            cut = np.sort(rng.integers(0, B + 1, NG + 1)) if NG > 1 else np.array([0, B])
            v["starts"].append(cut)
            v["ptable"].append(rng.permutation(ids[:NG * MP]).reshape(NG, MP))
            v["plens"].append(rng.integers(0, prefix + 1, NG))
            v["table"].append(own[rng.permutation(B)])
            v["lens"].append(rng.integers(1, MB * BS, B))
            v["q"].append(rng.standard_normal((B, Hk * 8, 128)))
            v["k"].append(rng.standard_normal((B, Hk, 128)))
            v["v"].append(rng.standard_normal((B, Hk, 128)))
        bf = ("q", "k", "v")
        self.variants = {n: dev(np.stack(x), np.float32).bfloat16() if n in bf else dev(np.stack(x)) for n, x in v.items()}
        self.live = {n: x[0].clone() for n, x in self.variants.items()}
        self.positions = self.live["lens"].clone()
        self.pp, self.p = pda.shared_plans(B, NG, Hk, 8, BS, MP, MB, kv_dtype=kv)
        self.ws = pda.shared_workspace(self.pp, self.p, "cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def write(self, i):
        """The live inputs of variant i (a one-element index on the device), and its new tokens into the cache."""
        for n, x in self.variants.items():
            if n in ("q", "k", "v"):
                torch.index_select(x.view(torch.int16).view(N, -1), 0, i, out=self.live[n].view(torch.int16).view(1, -1))
            else:
                torch.index_select(x.view(N, -1), 0, i, out=self.live[n].view(1, -1))
        torch.sub(self.live["lens"], 1, out=self.positions)
        self.pda.append_kv(self.p, self.live["k"], self.live["v"], self.cache, self.NB, self.live["table"], self.positions,
                           err_word=self.err)

    def step(self, out, table=None, lens=None):
        x = self.live
        self.pda.decode_shared(self.pp, self.p, x["q"], self.cache, self.NB, x["starts"], x["ptable"], x["plens"],
                               x["table"] if table is None else table, x["lens"] if lens is None else lens, ws=self.ws, out=out,
                               err_word=self.err)


def bits(x):
    return x.view(torch.int32)


@pytest.mark.parametrize("kv", [wl.KV_BF16, wl.KV_FP8_E4M3])
@pytest.mark.parametrize("name", list(SIZES))
def test_inputs_written_right_before_the_step(pda, kv, name):
    s = Stage(pda, kv, SIZES[name])
    rounds = 8
    index = [torch.tensor([i], device="cuda") for i in range(N)]
    outs = torch.empty((2, rounds * N, s.B, s.Hk * 8, 128), device="cuda")
    for once, pause in ((0, True), (1, False)):
        s.cache.copy_(s.cache0)
        torch.cuda.synchronize()
        for r in range(rounds * N):
            i = (5 * r + r // N) % N
            s.write(index[i])
            if pause:
                torch.cuda.synchronize()
            s.step(outs[once, r])
            if pause:
                torch.cuda.synchronize()
    torch.cuda.synchronize()
    assert int(s.err.item()) == 0 and torch.isfinite(outs).all()
    assert torch.equal(bits(outs[0]), bits(outs[1]))
    assert not torch.equal(bits(outs[0, 0]), bits(outs[0, 1]))


@pytest.mark.parametrize("kv", [wl.KV_BF16, wl.KV_FP8_E4M3])
@pytest.mark.parametrize("name", list(SIZES))
def test_inputs_written_right_before_a_captured_step(pda, kv, name):
    """The writers and the step in one graph, replayed without a pause; a counter on the device picks the variant."""
    s = Stage(pda, kv, SIZES[name])
    total = 5 * N
    order = torch.tensor([(7 * r + r // N) % N for r in range(total)], device="cuda")
    at, out = torch.zeros(1, dtype=torch.long, device="cuda"), torch.empty((s.B, s.Hk * 8, 128), device="cuda")
    outs = torch.empty((2, total, *out.shape), device="cuda")
    keep = torch.empty_like(outs[0])

    def step():
        s.write(torch.index_select(order, 0, at))
        s.step(out)
        keep.index_copy_(0, at, out[None])
        at.add_(1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step()
    for once, pause in ((0, True), (1, False)):
        s.cache.copy_(s.cache0)
        at.zero_()
        keep.fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(total):
            g.replay()
            if pause:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        outs[once].copy_(keep)
    assert int(s.err.item()) == 0 and torch.isfinite(outs).all()
    assert torch.equal(bits(outs[0]), bits(outs[1]))


@pytest.mark.parametrize("kv", [wl.KV_BF16, wl.KV_FP8_E4M3])
@pytest.mark.parametrize("name", list(SIZES))
def test_a_fork_right_before_the_step(pda, kv, name):
    """The step's own tables and lengths come from fork_sequences, whose second launch ends right before the step."""
    s = Stage(pda, kv, SIZES[name])
    B, NB = s.B, s.NB
    rng = np.random.default_rng(7)
    table, lens = s.live["table"].clone(), s.live["lens"].clone().clamp_(max=s.MB * s.BS - 20)
    refs = torch.zeros(NB, dtype=torch.int32, device="cuda")
    refs[s.live["ptable"].flatten().long()] = 1
    for b in range(B):
        refs[table[b, :-(-int(lens[b]) // s.BS)].long()] += 1
    parents = torch.from_numpy(rng.integers(0, B, (N, B)).astype(np.int32)).cuda()
    grow = torch.from_numpy(rng.integers(0, 18, (N, B)).astype(np.int32)).cuda()
    new_table, new_lens, new_refs = torch.empty_like(table), torch.empty_like(lens), torch.empty_like(refs)
    pws = pda.page_workspace(s.p, B, NB, "cuda")
    rounds = 6
    outs = torch.empty((2, rounds * N, B, s.Hk * 8, 128), device="cuda")
    for once, pause in ((0, True), (1, False)):
        s.cache.copy_(s.cache0)
        torch.cuda.synchronize()
        for r in range(rounds * N):
            i = (5 * r + r // N) % N
            pda.fork_sequences(s.p, s.cache, NB, table, lens, refs, parents[i], new_table, new_lens, new_refs, pws,
                               new_tokens=grow[i], err_word=s.err)
            if pause:
                torch.cuda.synchronize()
            s.step(outs[once, r], new_table, new_lens)
            if pause:
                torch.cuda.synchronize()
    torch.cuda.synchronize()
    assert int(s.err.item()) & ~pda.ERRW_OUT_OF_BLOCKS == 0 and torch.isfinite(outs).all()
    assert torch.equal(bits(outs[0]), bits(outs[1]))
