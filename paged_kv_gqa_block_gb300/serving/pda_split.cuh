// pda_split.cuh -- which rows and which tokens a CTA of the prefix pass (pda_prefix.cuh) takes: of pda_decode_shared's prefixes,
// or of pda_decode_tree's sequences.  Only integers and warp-wide exchanges, so that the same code also compiles for the host,
// where its pieces are checked.
#pragma once

#include <cstdint>

#include "pda.h"

namespace pda {

constexpr uint32_t kLanes = 0xFFFFFFFFu;
constexpr int kStep = 128;                 // tokens per step
constexpr int kUnitRows = 256;             // query rows of a row tile
constexpr int kSwitch = 3;                 // what a change of row tiles costs a CTA, in steps: of prefixes

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
    static constexpr int kBadStarts = PDA_ERRW_BAD_GROUP;
    static constexpr int kSwitchSteps = kSwitch, kUncut = 0;
};

// pda_decode_tree: a group is a sequence, its rows are those of its drafted tokens, and its tokens are the cached ones and,
// behind them, the drafted.  group_starts: token_starts, over B = num_tokens tokens; prefix_table, prefix_lens: block_table,
// context_lens.
struct TreeArgs : SharedArgs {
    const uint32_t* masks;       // [B][words], or null: token i sees the drafted tokens 0 .. i
    const float* centroids;      // TQ4: [16]
    int* refused;                // set to 1 by a call whose token_starts do not ascend, else to 0
    uint8_t* seen;               // [B]: some row sees the drafted token; of sequences of which one does not see itself
    int words;                   // 32-bit words of a mask
    int window, num_first;       // window 0: none
    const uint8_t* cache;        // the pool, for what is not copied by tensor map
    long long block_bytes, meta_bytes;   // of a block; where its metadata start
    void* out;                   // [B][Hk*QG][D]
    int out_f32;
    static constexpr int kBadStarts = PDA_ERRW_BAD_TOKENS;
    // 64 sequences of up to 6 tokens in a window of 4096 fp8 tokens 101 -> 97 us with 4 in place of 3 for a change of row tiles, of 4
    // over 1000 79 -> 76 (5: 75, but 16 over 4096 48 -> 53); 16 of 32 tokens over 4096 bf16 tokens 82 -> 64 us with runs of their own
    // where those end up to 3 steps later, and fp8 96 -> 86 (6: the same).
    static constexpr int kSwitchSteps = 4, kUncut = 3;
};

// What a sequence's drafted tokens see of it: every one of them misses tokens hole0 .. hole1-1, and the steps at, ..,
// at + skip - 1 lie wholly within those.
struct Sight {
    int ctx, drafted;
    int hole0, hole1;
    int at, skip;
};
__device__ __forceinline__ Sight sight_of(const TreeArgs& a, int len, int drafted) {
    Sight x = {};
    x.ctx = len - drafted;
    x.drafted = drafted;
    // the first of them stands at position ctx at the earliest
    const int start = a.window > 0 && a.window <= x.ctx ? x.ctx - a.window + 1 : 0;
    if (start > a.num_first) {
        x.hole0 = a.num_first;
        x.hole1 = start;
        x.at = (int)(((long long)a.num_first + kStep - 1) / kStep);
        x.skip = start / kStep > x.at ? start / kStep - x.at : 0;
    }
    return x;
}

struct Unit {
    int g, h, rt;          // group, KV head, row tile
    int seq0, rows;        // first sequence and query rows of the group
    int len;               // prefix length
    int step0, steps;      // this piece
    int rot;               // the piece's steps are taken from step0 + rot on, then from step0
    int slot, pieces;      // its number, and how many the row tile has
    int hidden;            // drafted tokens: one of them does not see itself (set by the kernel)
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
__device__ __forceinline__ Group group_shape(const TreeArgs& a, int g, int& bad) {
    Group x = {};
    if (g >= a.NG) return x;
    const int s0 = __ldcg(a.group_starts + g), s1 = __ldcg(a.group_starts + g + 1), ctx = __ldcg(a.prefix_lens + g);
    x.seq0 = s0;
    if (s0 < 0 || s1 < s0 || s1 > a.B) {
        bad |= PDA_ERRW_BAD_TOKENS;
        return x;
    }
    const int drafted = s1 - s0;
    if (ctx < 0 || ctx > a.MP * a.BS) {
        bad |= PDA_ERRW_BAD_CONTEXT_LEN;
    } else if (drafted > a.MP * a.BS - ctx) {
        bad |= PDA_ERRW_BAD_POSITION;
    } else if (drafted > 0) {
        x.len = ctx + drafted;
        x.rows = drafted * a.QG;
        x.tiles = (x.rows + kUnitRows - 1) / kUnitRows;
        x.steps = (x.len + kStep - 1) / kStep - sight_of(a, x.len, drafted).skip;
    }
    return x;
}
// Of numbers that are not negative.  A CTA waits for this code's first fetch longer than for its execution, so
// quotients that are wanted together are computed by lanes of one warp.
__device__ __forceinline__ int quotient(int x, int d) { return (int)((unsigned)x / (unsigned)d); }

// How one warp sees the split: lane i holds group i (and re-reads the others where there are more
// than 32).  The host has made sure that the places of all steps of ascending groups fit an int.
template <int SWITCH>
struct SplitBy {
    Group mine;
    int before, total;     // places of the groups before lane i's (of the first 32), and of all
    int per;               // places of a CTA's run
    int whole;             // if not 0: places of every row tile
    bool refused;          // starts that do not ascend: there are no steps
    // Places of a row tile: its steps, and unused ones after them.  A CTA whose run goes on into another row tile
    // pays for it (store the rows, load others, refill the pipeline: SWITCH steps); either that is counted
    // as places between two tiles, or every tile has whole runs of its own.
    __device__ __forceinline__ int span(int steps) const { return steps == 0 ? 0 : whole ? whole : steps + SWITCH; }
};
using Split = SplitBy<kSwitch>;

// `per`: an even share of all places, or, where that is no longer, the longest tile's share of the runs that every
// tile can have; and at least 1/P of the longest prefix, so that a row tile is cut into at most P + 1 pieces
// (the workspace's slots).
template <class Args>
__device__ __forceinline__ SplitBy<Args::kSwitchSteps> make_split(const Args& a, int ctas, bool report) {
    const int lane = threadIdx.x & 31;
    SplitBy<Args::kSwitchSteps> s;
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
    const int q = quotient(lane == 0 ? longest + a.P - 1 : lane == 1 ? steps + Args::kSwitchSteps * tiles + ctas - 1 : ctas,
                           lane == 0 ? a.P : lane == 1 ? ctas : max(tiles, 1));
    const int least = max(__shfl_sync(kLanes, q, 0), 1), even = max(__shfl_sync(kLanes, q, 1), least);
    const int runs = __shfl_sync(kLanes, q, 2);
    const int own = runs > 0 ? max(quotient(longest + runs - 1, runs), least) : even + 1;
    // Runs of their own also where they end up to Args::kUncut steps later: what is not cut needs no partials and no join.
    const bool whole = own <= even || (runs > 0 && own <= even + Args::kUncut);
    s.per = whole ? own : even;
    s.whole = whole ? quotient(longest + own - 1, own) * own : 0;   // the first CTAs work: they start first
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
    s.refused = __any_sync(kLanes, bad & Args::kBadStarts);
    if (s.refused) s.total = 0;
    if (report && bad && a.err_word) atomicOr(a.err_word, bad);
    return s;
}

// One warp: the piece that starts at place `at` of the run of all places, or after the unused ones there, and ends
// with its row tile or at `end`; `at` moves past it.  Without steps: there is none.
template <class Args>
__device__ __forceinline__ Unit find_unit(const Args& a, const SplitBy<Args::kSwitchSteps>& s, int& at, int end) {
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
