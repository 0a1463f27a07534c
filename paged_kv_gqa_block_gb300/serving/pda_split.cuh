// pda_split.cuh -- which rows and which tokens a CTA of pda_decode_shared's prefix pass takes.  Only integers and warp-wide
// exchanges, so that the same code also compiles for the host, where its pieces are checked.
#pragma once

#include <cstdint>

#include "pda.h"

namespace pda {

constexpr uint32_t kLanes = 0xFFFFFFFFu;
constexpr int kStep = 128;                 // tokens per step
constexpr int kUnitRows = 256;             // query rows of a row tile
constexpr int kSwitch = 3;                 // what a change of row tiles costs a CTA, in steps

struct SharedArgs {
    const uint16_t* query;       // bf16 [B][Hk*QG][D]
    const int* group_starts;     // [NG + 1]
    const int* prefix_table;     // [NG][MP]
    const int* prefix_lens;      // [NG]
    float* part_o;               // [B][Hk][slots][QG][D]
    float* part_l;               // [B][Hk][slots][QG]
    float* part_m;
    int* pieces;                 // [B][Hk][QG]: partials of a row
    int* err_word;
    long long num_cache_blocks;
    int B, NG, Hk, QG, MP, BS, P, slots;
    int first;                   // this pass comes before the own tokens' one
    float qk_scale_log2;
    unsigned long long timeout_ns;
};

struct Unit {
    int g, h, rt;          // group, KV head, row tile
    int seq0, rows;        // first sequence and query rows of the group
    int len;               // prefix length
    int step0, steps;      // this piece
    int rot;               // the piece's steps are taken from step0 + rot on, then from step0
    int slot, pieces;      // its number, and how many the row tile has
};

struct Group {
    int seq0, rows, len;   // first sequence, query rows, prefix length
    int tiles, steps;      // row tiles and steps of each; a group's steps: tiles * Hk * steps
};
// An out-of-range length or range counts as empty.
__device__ __forceinline__ Group group_shape(const SharedArgs& a, int g, int& bad) {
    Group x = {};
    if (g >= a.NG) return x;
    const int s0 = __ldcg(a.group_starts + g), s1 = __ldcg(a.group_starts + g + 1);
    x.len = __ldcg(a.prefix_lens + g);
    if (x.len < 0 || x.len > a.MP * a.BS) {
        bad |= PDA_ERRW_BAD_CONTEXT_LEN;
        x.len = 0;
    }
    x.seq0 = s0;
    if (s0 < 0 || s1 < s0 || s1 > a.B)
        bad |= PDA_ERRW_BAD_GROUP;
    else
        x.rows = (s1 - s0) * a.QG;
    x.tiles = (x.rows + kUnitRows - 1) / kUnitRows;
    x.steps = (x.len + kStep - 1) / kStep;
    return x;
}
// Of numbers that are not negative.  A CTA waits for this code's first fetch longer than for its execution, so
// quotients that are wanted together are computed by lanes of one warp.
__device__ __forceinline__ int quotient(int x, int d) { return (int)((unsigned)x / (unsigned)d); }

// How one warp sees the split: lane i holds group i (and re-reads the others where there are more
// than 32).  The host has made sure that the places of all steps of ascending groups fit an int.
struct Split {
    Group mine;
    int before, total;     // places of the groups before lane i's (of the first 32), and of all
    int per;               // places of a CTA's run
    int whole;             // if not 0: places of every row tile
    // Places of a row tile: its steps, and unused ones after them.  A CTA whose run goes on into another row tile
    // pays for it (store the rows, load others, refill the pipeline: kSwitch steps); either that is counted
    // as places between two tiles, or every tile has whole runs of its own.
    __device__ __forceinline__ int span(int steps) const { return steps == 0 ? 0 : whole ? whole : steps + kSwitch; }
};

// `per`: an even share of all places, or, where that is no longer, the longest tile's share of the runs that every
// tile can have; and at least 1/P of the longest prefix, so that a row tile is cut into at most P + 1 pieces
// (the workspace's slots).
__device__ __forceinline__ Split make_split(const SharedArgs& a, int ctas, bool report) {
    const int lane = threadIdx.x & 31;
    Split s;
    int bad = 0;
    s.mine = group_shape(a, lane, bad);
    int tiles = s.mine.steps > 0 ? s.mine.tiles * a.Hk : 0, steps = tiles * s.mine.steps;
    int longest = tiles > 0 ? s.mine.steps : 0;
#pragma unroll 1
    for (int g = lane + 32; g < a.NG; g += 32) {
        const Group x = group_shape(a, g, bad);
        const int n = x.steps > 0 ? x.tiles * a.Hk : 0;
        tiles += n;
        steps += n * x.steps;
        if (n > 0) longest = max(longest, x.steps);
    }
    tiles = __reduce_add_sync(kLanes, tiles);
    steps = __reduce_add_sync(kLanes, steps);
    longest = __reduce_max_sync(kLanes, longest);
    const int q = quotient(lane == 0 ? longest + a.P - 1 : lane == 1 ? steps + kSwitch * tiles + ctas - 1 : ctas,
                           lane == 0 ? a.P : lane == 1 ? ctas : max(tiles, 1));
    const int least = max(__shfl_sync(kLanes, q, 0), 1), even = max(__shfl_sync(kLanes, q, 1), least);
    const int runs = __shfl_sync(kLanes, q, 2);
    const int own = runs > 0 ? max(quotient(longest + runs - 1, runs), least) : even + 1;
    s.per = min(own, even);
    s.whole = own <= even ? quotient(longest + own - 1, own) * own : 0;   // the first CTAs work: they start first
    const int mine = s.mine.tiles * a.Hk * s.span(s.mine.steps);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(kLanes, incl, o);
        if (lane >= o) incl += x;
    }
    s.before = incl - mine;
    s.total = __shfl_sync(kLanes, incl, 31);
    if (a.NG > 32) {
        int more = 0;
#pragma unroll 1
        for (int g = lane + 32; g < a.NG; g += 32) {
            const Group x = group_shape(a, g, bad);
            more += x.tiles * a.Hk * s.span(x.steps);
        }
        s.total += __reduce_add_sync(kLanes, more);
    }
    // groups that are not ascending may overlap, and name more rows than there are: no prefix then
    if (__any_sync(kLanes, bad & PDA_ERRW_BAD_GROUP)) s.total = 0;
    if (report && bad && a.err_word) atomicOr(a.err_word, bad);
    return s;
}

// One warp: the piece that starts at place `at` of the run of all places, or after the unused ones there, and ends
// with its row tile or at `end`; `at` moves past it.  Without steps: there is none.
__device__ __forceinline__ Unit find_unit(const SharedArgs& a, const Split& s, int& at, int end) {
    const int lane = threadIdx.x & 31;
    Unit u = {};
#pragma unroll 1
    while (at < end) {
        Group x = s.mine;
        int lo = s.before, g0 = 0;
        unsigned hit;
#pragma unroll 1
        for (;;) {
            const int n = x.tiles * a.Hk * s.span(x.steps);
            hit = __ballot_sync(kLanes, lo <= at && at < lo + n);
            if (hit || (g0 += 32) >= a.NG) break;
            const int next = __shfl_sync(kLanes, lo + n, 31);   // the next 32 groups
            int bad = 0;
            x = group_shape(a, g0 + lane, bad);
            const int m = x.tiles * a.Hk * s.span(x.steps);
            int incl = m;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(kLanes, incl, o);
                if (lane >= o) incl += y;
            }
            lo = next + incl - m;
        }
        if (!hit) break;
        const int src = __ffs(hit) - 1;
        const int nt = __shfl_sync(kLanes, x.tiles, src), ns = __shfl_sync(kLanes, x.steps, src);
        const int base = __shfl_sync(kLanes, lo, src), span = s.span(ns);
        const int tile = quotient(at - base, span), first = base + tile * span;   // the row tile's own first place
        u.step0 = at - first;
        if (u.step0 >= ns) {
            at = first + span;
            continue;
        }
        u.g = g0 + src;
        u.seq0 = __shfl_sync(kLanes, x.seq0, src);
        u.rows = __shfl_sync(kLanes, x.rows, src);
        u.len = __shfl_sync(kLanes, x.len, src);
        u.steps = min(ns - u.step0, end - at);
        const int q = quotient(lane == 0 ? tile : lane == 1 ? first : lane == 2 ? at : lane == 3 ? first + ns - 1 : u.step0 + s.per - 1,
                               lane == 0 ? nt : s.per);
        u.h = __shfl_sync(kLanes, q, 0);
        u.rt = tile - u.h * nt;
        const int c0 = __shfl_sync(kLanes, q, 1);
        u.slot = __shfl_sync(kLanes, q, 2) - c0;
        u.pieces = __shfl_sync(kLanes, q, 3) - c0 + 1;
        // The row tiles of one (group, KV head) read the same tokens, but are cut at different places.
        // Taking the steps of a piece from the first multiple of `per` on makes every CTA read, at
        // time t, tokens of step t mod per of its tile: the copies of other row tiles then hit L2.
        const int s0 = __shfl_sync(kLanes, q, 4) * s.per;
        u.rot = s0 < u.step0 + u.steps ? s0 - u.step0 : 0;
        at += u.steps;
        break;
    }
    return u;
}

}  // namespace pda
