// pda_prefix.cuh -- attention of many query rows over the tokens of one (sequence or group, KV head), on the tensor cores: the
// prefix pass of pda_decode_shared, and the only pass of pda_decode_tree.
//
// pda_decode_shared: for query row r of sequence b in group g,
//   out = softmax(scale [q.K_g ; q.K_b]) [V_g ; V_b],
// with K_g, V_g the group's prefix and K_b, V_b the sequence's own tokens.  The two parts are
// computed apart as (m, l, o), a reference near the maximum, the sum of exponentials from it and the normalised
// output, and joined: w = l e^(m - M), out = sum w o / sum w, M the largest m.  The own part is the cluster kernel of
// pda_selected.cuh.  The prefix part is one matrix product per group and KV head for the
// query rows of all its sequences, n_g * QG of them, and this file's kernel.
//
// pda_decode_tree: a group is one sequence, its rows are those of its drafted tokens, its tokens the cached ones and the
// drafted behind them.  A row does not see every token: see Visible.
//
// The prefix pass.  A CTA holds 256 query rows of one (group, KV head) in two tiles of 128 and walks
// the prefix in steps of 128 tokens: S = Q K^T and O += P V by tcgen05.mma (M = N = 128), S, P and
// O in tensor memory (two tiles x (128 + 128) columns = all 512; P, 16-bit, lies over the S it was
// made of).  Warps take one role each:
//   0-3, 4-7  softmax of tile 0, tile 1: one query row per thread, so a row's maximum and sum need
//             no shuffles; S is read from TMEM, P written back
//   8         copies: K and V blocks by TMA into a ring of shared-memory slots (32 KB each); drafted tokens: K's (TQ4: both)
//   9         the matrix products (one thread issues)
//   10        fp8 and TQ4: the scales of a step; drafted tokens, bf16 and fp8: the copies of V, with the scales
//   11        the split: which rows and which tokens this CTA takes
//   12-15     fp8 and TQ4: codes to f16 between the copy and the product
// The softmax warps hold a whole row of S (128 registers); the other warps give registers up for them.
// The products are issued in the order PV(0, j), QK(0, j+1), PV(1, j), QK(1, j+1): while one tile's
// softmax runs the tensor cores work for the other.  A tile's reference point m moves only when a
// row's maximum passes it by 2^8 (log2 units 8), so the rescale of O, the one read-modify-write of
// TMEM, is rare; a reference below the true maximum leaves the quotient as it is.
// P is announced in halves, so that PV starts while the second half is computed.
// Drafted tokens have few rows as a rule, and many short units: see products_tree and halves.
// P is rounded to bf16 (bf16 KV: by at most 2^-8 of each weight) or f16 (fp8 KV: 2^-11; V carries two more such
// roundings, see the conversion); m, l, S and O are fp32.  f16 has few exponents: below 2^-14 a value loses bits, and
// below 2^-25 it is zero, while l counts it; a long even prefix behind one large weight would lose a share of the
// output.  So with f16 the reference is 7 below the maximum: with the 8 of its lazy move P still ends at 2^15, weights
// keep their 11 bits down to 2^-21 of the largest, and smaller ones are off by at most 2^-32 of it.
//
// Work is split over the CTAs (one per SM) by steps, not by units: the steps of all (group, KV head,
// row tile) are laid end to end and every CTA takes an equal run; a row tile that is cut leaves one
// partial per piece.  A change of row tiles is counted as steps too, or every tile gets runs of its own, whichever
// ends sooner (64 sequences of 64 heads in 3 groups 37.2 -> 33.0 us, 100 of 32 heads in 7 groups 49.3 -> 34.5).
// Nothing depends on how lengths and groups fall.  Bound by the tensor cores
// where a group has many rows (4 * 256 * D flops per token and pair of tiles), by HBM where it has few.
//
// Measured, whole calls from a graph: 128 sequences of 64 query heads over 32768 bf16 tokens 99.4 us (1.39 PFLOP/s; this
// pass 82 us, 141 MB read of a prefix of 134 MB), 64 over 77824 bf16 tokens 109 us, fp8 149 us.  A further step of 256
// rows costs a CTA 1.4 us (bf16), of which its products' 2048 cycles are 1.3 at the clock of this load; fp8 1.95 us:
// 350 KB of shared-memory traffic (operands 192, conversion 96, copies 32, scales 32) at 128 bytes per cycle, which
// account for 1.4 to 1.5 of it.  Few rows: 4 sequences with up to 20 tokens of their own over 38912 tokens 40 us (bf16,
// 4.0 TB/s with the launches) and 46 us (fp8, which converts every token whatever the rows: 1.55 us per step).  The
// launches, first copies, last stores and the join around the steps take 10 to 20 us, more with more rows: a call of two
// steps per CTA is 13.4 us with 4 sequences, 17.0 us with 32.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>
#include <type_traits>

#include "pda.h"
#include "pda_internal.h"
#include "pda_ptx.cuh"
#include "pda_split.cuh"
#include "pda_tc.cuh"

namespace pda {

constexpr int kConvertWarps = 4;
constexpr int kTileRows = 128;
constexpr int kSlotBytes = 32768;          // 128 tokens x 128 dimensions, 16 bits
constexpr int kRawBytes = 16384;           // the same in 8 bits
constexpr float kLog2eS = 1.4426950408889634f, kLn2S = 0.6931471805599453f;
constexpr float kLazy = 8.f;               // log2 units that a row's maximum may rise before its reference follows
constexpr float kBelow = 7.f;              // f16 P: the reference below the maximum

constexpr int kBarBytes = 784;             // barriers and scalars

// What a KV format and a kind of call take of shared memory, barriers and threads.  Q8 (drafted tokens over fp8 KV): the score
// product takes K's codes as they are, so that only V is converted, in halves of 64 tokens.
template <int KV, class Args>
struct SharedCfg {
    static constexpr bool kF16 = KV != PDA_KV_BF16;              // f16 products, converter warps
    static constexpr bool kTq = KV == PDA_KV_TQ4, kTree = std::is_same<Args, TreeArgs>::value, kQ8 = kTree && KV == PDA_KV_FP8_E4M3;
    static constexpr int kScaleBytes = kTq ? 1536 : 1024;        // 128 tokens x {K scale, V scale (, V zero)}
    static constexpr int kTiles = kTq ? 1 : 2;                   // copies of a step: a TQ4 row holds K and V
    static constexpr int kSlots = kF16 ? 3 : 5;
    static constexpr int kRaw = 3, kScales = kQ8 ? 4 : 3;                  // fp8, TQ4: raw slots, scale stages
    static constexpr int kThreads = kF16 ? 512 : 384;
    static constexpr int kOffQ = 0;                               // 2 tiles x 32 KB
    static constexpr int kKeys = 3, kHalves = 3;                  // Q8: slots of K's codes, and of converted halves of V; bf16 trees:
    static constexpr int kValues = kSlots - kKeys;                // the first three slots are K's, the others V's
    static constexpr int kOffKeys = 2 * kSlotBytes;
    static constexpr int kOffSlots = kOffKeys + (kQ8 ? kKeys * kRawBytes : 0);
    static constexpr int kOffRaw = kOffSlots + (kQ8 ? kHalves * kRawBytes : kSlots * kSlotBytes);
    static constexpr int kOffScales = kOffRaw + (kF16 ? kRaw * kRawBytes : 0);
    static constexpr int kOffBars = kOffScales + (kF16 ? kScales * kScaleBytes : 0);
    static constexpr int kOffTable = kOffBars + kBarBytes;        // TQ4: the centroids of a byte's two codes, f16
    static constexpr int kOffPair = kOffBars + kBarBytes + (kTq ? 1024 : 0);   // drafted tokens: (m, l) of rows' halves
    static constexpr int kSmem = kTree ? kOffPair + 2048 : kTq ? kOffTable + 1024 : kOffBars + 448;
    static_assert(kSmem <= 232448, "shared memory of a CTA");
    static constexpr int kReaders = kF16 ? 15 : kTree ? 11 : 10;  // warps that take units
};
// barriers and scalars after kOffBars
enum {
    kBarFull = 0,        // [5] a slot holds its tile
    kBarEmpty = 40,      // [5] the products that read a slot are done
    kBarQ = 80,          // [2] a tile's query rows are in shared memory
    kBarS = 96,          // [2] S is in TMEM
    kBarP = 112,         // [2] the first half of P (64 tokens) is in TMEM
    kBarO = 128,         // [2] the unit's last product of a tile is done
    kBarRawFull = 144,   // [3]
    kBarRawEmpty = 168,  // [3]
    kBarScFull = 192,    // [3] scales are laid out
    kBarScEmpty = 216,   // [3]
    kBarDrain = 240,
    kTmemAt = 248,       // TMEM address
    kAbortAt = 252,      // a wait gave up
    kFAt = 256,          // [3] (Q8: 4) what a step's V scales are divided by
    kBarP2 = 272,        // [2] the second half of P is in TMEM
    kBarScRaw = 288,     // [3] scales as copied
    kBarUnitFull = 312,  // [2] the next unit is in shared memory
    kBarUnitEmpty = 328, // [2]
    kUnitAt = 352,       // [2] units, 48 bytes each
    kPowerAt = 448,      // TQ4: 1 over the power of two that the table's centroids carry
    kBarHalf = 504,      // [2] drafted tokens: the product of the first half of P is done
    kBarScFull8 = 520,   // [4] Q8: the scales' barriers and F, of four stages
    kBarScEmpty8 = 552,
    kBarScRaw8 = 584,
    kBarWhole = 616,     // [2] that of the second half too
    kBarPairFull = 648,  // [8] drafted tokens: a softmax warp has handed a part of its rows over
    kBarPairEmpty = 712, // [8] it has taken what it was handed
    kBarS2 = 632,        // [2] drafted tokens: a tile's S is in the second place (kBarS: in the first)
    kBarVFull = 456,     // [3] Q8: a half of V is converted
    kBarVEmpty = 480     // [3] the products that read it are done
};

// ------------------------------------------------------------------------- the prefix pass
__device__ __forceinline__ uint64_t l2_policy_evict_normal() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// 16 bytes global -> shared, of which `bytes` (16 or 0) are read and the rest are zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// One arrival on `bar` when this thread's asynchronous copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ uint32_t lds32v(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void sts32v(uint32_t addr, uint32_t v) {
    asm volatile("st.volatile.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
// Two fp32 operations per instruction.
__device__ __forceinline__ void mul2(uint32_t& x, uint32_t& y, uint32_t a, uint32_t b) {
    asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\t"
        "mul.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "+r"(x), "+r"(y)
        : "r"(a), "r"(b));
}
__device__ __forceinline__ void fma2(uint32_t& x, uint32_t& y, float c, float d) {   // x c + d
    asm("{\n\t.reg .b64 p, q, r;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %2};\n\tmov.b64 r, {%3, %3};\n\t"
        "fma.rn.f32x2 p, p, q, r;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "+r"(x), "+r"(y)
        : "f"(c), "f"(d));
}
__device__ __forceinline__ void add2(float2& x, const float2& y) {
    asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\t"
        "add.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "+f"(x.x), "+f"(x.y)
        : "f"(y.x), "f"(y.y));
}

template <int KV, class Args>
struct Prefix {
    using Cfg = SharedCfg<KV, Args>;
    using Split = SplitBy<Args::kSwitchSteps>;
    static constexpr bool F16 = Cfg::kF16, TQ = Cfg::kTq, TREE = Cfg::kTree, Q8 = Cfg::kQ8;
    static constexpr uint32_t kScFull = Q8 ? kBarScFull8 : kBarScFull, kScEmpty = Q8 ? kBarScEmpty8 : kBarScEmpty,
                              kScRaw = Q8 ? kBarScRaw8 : kBarScRaw;
    static constexpr uint32_t kIdescQ8 = umma_idesc_e4m3(128, 128);
    static constexpr uint32_t kIdescQK = umma_idesc(!F16, false, 128, 128), kIdescPV = umma_idesc(!F16, true, 128, 128);

    const Args& a;
    const uint32_t sm;         // shared memory base
    const uint32_t bars;
    unsigned units = 0;        // units taken (or given) by this warp
    unsigned busy = 0;         // their steps
    const bool poll;           // TREE: a short limit; and the limit in 1024 ns, half an hour at most
    const uint32_t patience;

    __device__ __forceinline__ Prefix(const Args& args, uint32_t base)
        : a(args), sm(base), bars(base + Cfg::kOffBars), poll(args.timeout_ns < 1000000ull),
          patience((uint32_t)min(args.timeout_ns >> 10, 0x7FFFFFFFull)) {}

    // A whole warp waits (bounded).  False once any wait of the CTA has given up.
    // TREE: in less code, since there is a wait in every other line (fp8 steps 2 to 4 % shorter): the first test does not sleep, and
    // time is counted in 1024 ns and 32 bits.
    __device__ __forceinline__ bool wait_short(uint32_t bar, uint32_t parity, uint32_t limit) const {
        if (__all_sync(kLanes, mbar_test_wait(bar, parity))) return true;
        const uint32_t t0 = (uint32_t)(global_timer_ns() >> 10);
        for (;;) {
            const bool ok = poll ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity);
            if (__all_sync(kLanes, ok)) return true;
            const bool late = (uint32_t)(global_timer_ns() >> 10) - t0 > limit;
            if (__any_sync(kLanes, late || lds32v(bars + kAbortAt) != 0u)) {
                sts32v(bars + kAbortAt, 1u);
                return false;
            }
        }
    }
    __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) const {
        if constexpr (TREE) return wait_short(bar, parity, patience);
        const bool poll = a.timeout_ns < 1000000ull;   // try_wait may sleep past a short limit
        bool ok = poll ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity);
        if (__all_sync(kLanes, ok)) return true;
        return wait_on(bar, parity, poll, a.timeout_ns);
    }
    __device__ __forceinline__ bool wait_on(uint32_t bar, uint32_t parity, bool poll, uint64_t limit) const {
        const uint64_t t0 = global_timer_ns();
        for (;;) {
            const bool ok = poll ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity);
            if (__all_sync(kLanes, ok)) return true;
            const bool late = global_timer_ns() - t0 > limit;
            if (__any_sync(kLanes, late || lds32v(bars + kAbortAt) != 0u)) {
                sts32v(bars + kAbortAt, 1u);
                return false;
            }
        }
    }

    // One warp looks the CTA's units up, ahead of the others, which read them from shared memory; a unit without
    // steps is the end.  (Looked up by every warp for itself, the split took registers from the softmax.)
    // A unit, or its place, may come only when warps that are behind have finished one that was taken before: the
    // limit is that of their waits, a few per step (long limits, from 0.27 s on, do for any unit).
    __device__ __forceinline__ bool wait_unit(uint32_t bar, uint32_t parity) const {
        if constexpr (TREE)
            return wait_short(bar, parity, patience >> 18 ? patience : (uint32_t)min((patience + 1) * (64 + 8ull * busy), 0x7FFFFFFFull));
        const uint64_t limit = a.timeout_ns >> 28 ? a.timeout_ns : a.timeout_ns * (64 + 8ull * busy);
        const bool poll = a.timeout_ns < 1000000ull;
        if (__all_sync(kLanes, poll ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity))) return true;
        return wait_on(bar, parity, poll, limit);
    }
    __device__ __forceinline__ void put(const Unit& u) const {
        const uint32_t at = bars + kUnitAt + (units & 1) * 48;
        if ((threadIdx.x & 31) == 0) {
            sts128(at, u.g, u.h, u.rt, u.seq0);
            sts128(at + 16, u.rows, u.len, u.step0, u.steps);
            sts128(at + 32, u.rot, u.slot, u.pieces, TREE ? u.hidden : 0);
        }
    }
    __device__ void give(const Split& split, Unit u, int at, int end) {   // the first one is there already
        for (;;) {
            __syncwarp();
            if ((threadIdx.x & 31) == 0) mbar_arrive(bars + kBarUnitFull + 8 * (units & 1));
            ++units;
            if (u.steps == 0) return;
            busy += u.steps;
            u = find_unit(a, split, at, end);
            if (units > 1 && !wait_unit(bars + kBarUnitEmpty + 8 * (units & 1), (units >> 1) - 1 & 1)) return;
            put(u);
        }
    }
    // TREE: the same, with the first one looked up here too.
    __device__ void give_all(const Split& split, int at, int end) {
        int noted = -1, hidden = 0;   // of the last sequence looked at
        for (;;) {
            Unit u = find_unit(a, split, at, end);
            if (a.masks && u.steps > 0) {
                if (u.g != noted) hidden = note_hidden(u);
                noted = u.g;
                u.hidden = hidden;
            }
            if (units > 1 && !wait_unit(bars + kBarUnitEmpty + 8 * (units & 1), (units >> 1) - 1 & 1)) return;
            put(u);
            __syncwarp();
            if ((threadIdx.x & 31) == 0) mbar_arrive(bars + kBarUnitFull + 8 * (units & 1));
            ++units;
            if (u.steps == 0) return;
            busy += u.steps;
        }
    }
    __device__ __forceinline__ bool next(Unit& u) {
        const uint32_t slot = units & 1, at = bars + kUnitAt + slot * 48;
        if (!wait_unit(bars + kBarUnitFull + 8 * slot, units >> 1 & 1)) return false;
        uint32_t x[12];
#pragma unroll
        for (int i = 0; i < 12; i += 4) lds128(at + 4 * i, x[i], x[i + 1], x[i + 2], x[i + 3]);
        u.g = x[0], u.h = x[1], u.rt = x[2], u.seq0 = x[3], u.rows = x[4], u.len = x[5], u.step0 = x[6], u.steps = x[7];
        u.rot = x[8], u.slot = x[9], u.pieces = x[10];
        u.hidden = TREE ? x[11] : 0;
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(bars + kBarUnitEmpty + 8 * slot);
        ++units;
        busy += u.steps;
        return u.steps > 0;
    }
    // What the unit's rows see (TREE); constant, and gone, without.
    __device__ __forceinline__ Sight sight(const Unit& u) const {
        if constexpr (TREE)
            return sight_of(a, u.len, u.rows / a.QG);
        else
            return Sight{};
    }
    // Step number of the piece's j-th step, and its tokens.
    __device__ __forceinline__ static int step_of(const Unit& u, const Sight& x, int j) {
        const int i = j + u.rot, n = u.step0 + (i < u.steps ? i : i - u.steps);
        return TREE && n >= x.at ? n + x.skip : n;
    }
    __device__ __forceinline__ static int tokens_of(const Unit& u, const Sight& x, int j) {
        return min(kStep, u.len - step_of(u, x, j) * kStep);
    }
    // Whether token t of the sequence, below its length, is one that all rows miss.
    __device__ __forceinline__ static bool missed(const Sight& x, int t) { return TREE && t >= x.hole0 && t < x.hole1; }
    // Row of the group that a tile starts with.  TREE: a row tile of at most 128 rows is either tile's.
    __device__ __forceinline__ static int first_row(const Unit& u, int tile) {
        return u.rt * kUnitRows + (!TREE || active(u, 1) ? tile * kTileRows : 0);
    }
    // TREE: of at most 64 rows every one is there twice, 64 rows apart: the first half of each step's tokens is one's, the second the
    // other's, so that a step's softmax takes a warp half as long (fp8, steps of 36 rows: 1.7 -> 1.3 us with everything); the two
    // are joined at the end.
    __device__ __forceinline__ static bool halves(const Unit& u) { return TREE && u.rows - u.rt * kUnitRows <= 64; }
    __device__ __forceinline__ static bool active(const Unit& u, int tile) {
        return u.rt * kUnitRows + tile * kTileRows < u.rows;
    }
    // Drafted tokens that no row sees may hold anything, and a weight of zero silences neither a NaN nor a scale that the others
    // vanish beside, so their values and fields count as zeros.  In a chain every token is seen, and in a tree by itself as a rule.
    // Where one is not, the warp that looks the units up notes for each whether some row sees it, and says so with the unit.
    __device__ __forceinline__ bool note_hidden(const Unit& u) const {
        const int lane = threadIdx.x & 31, drafted = u.rows / a.QG;
        const uint32_t* m = a.masks + (long long)u.seq0 * a.words;
        bool own = true;
#pragma unroll 1
        for (int j = lane; j < drafted; j += 32) own = own && j >> 5 < a.words && (__ldcg(m + (long long)j * a.words + (j >> 5)) >> lane & 1);
        if (__all_sync(kLanes, own)) return false;
#pragma unroll 1
        for (int j = 0; j < drafted; j += 32, ++m) {   // a word of every row
            uint32_t any = 0;
            if (j >> 5 < a.words) {
#pragma unroll 1
                for (int i = lane; i < drafted; i += 32) any |= __ldcg(m + (long long)i * a.words);
            }
            any = __reduce_or_sync(kLanes, any);
            if (j + lane < drafted) a.seen[u.seq0 + j + lane] = any >> lane & 1;
        }
        return true;
    }
    // Whether token t of the sequence, below its length, is such a one.
    __device__ __forceinline__ bool hidden(const Unit& u, const Sight& x, int t) const {
        if constexpr (TREE)
            return u.hidden && t >= x.ctx && !a.seen[u.seq0 + (t - x.ctx)];
        else
            return false;
    }

    // ---------------------------------------------------------------- copies
    // Slot order K(0), V(0), K(1), V(1), ...  Each lane copies one (block, 64-dimension half): box
    // {128 bytes, BS tokens}; the halves are 16 KB apart, so that a slot is the products' operand as
    // it lands ([half][token][128 bytes], swizzled).  fp8 rows are one 128-byte piece, copied to the
    // raw slots with the step's scales.
    __device__ void copies(const CUtensorMap* kv_map, const CUtensorMap* sc_map) {
        const int lane = threadIdx.x & 31;
        constexpr int kHalves = F16 ? 1 : 2, kNS = F16 ? Cfg::kRaw : Cfg::kSlots;
        constexpr uint32_t kFull0 = F16 ? kBarRawFull : kBarFull, kEmpty0 = F16 ? kBarRawEmpty : kBarEmpty;
        constexpr int kBytes = F16 ? kRawBytes : kSlotBytes;
        const uint32_t base = sm + (F16 ? Cfg::kOffRaw : Cfg::kOffSlots);
        const int nblk = kStep / a.BS;
        const int blk = lane / kHalves, half = lane % kHalves;
        const uint64_t once = l2_policy_evict_first(), again = l2_policy_evict_normal();
        unsigned seq = 0, step = 0;
        bool ok = true;
        Unit u;
        while (ok && next(u)) {
            const Sight x = sight(u);
            const uint64_t policy = u.rows > kUnitRows ? again : once;   // other row tiles read it too
            const int* table = a.prefix_table + (long long)u.g * a.MP;
            const int last = (u.len + a.BS - 1) / a.BS;   // blocks of the prefix
            int id = 0;
            int b0 = step_of(u, x, 0) * nblk;
            if (blk < nblk && b0 + blk < last) id = __ldcg(table + b0 + blk);
            for (int j = 0; ok && j < u.steps; ++j, ++step) {
                const int n = min(nblk, last - b0);
                const bool mine = blk < n;
                int nid = 0, b1 = 0;
                if (j + 1 < u.steps) {
                    b1 = step_of(u, x, j + 1) * nblk;
                    if (blk < nblk && b1 + blk < last) nid = __ldcg(table + b1 + blk);
                }
                if (mine && half == 0 && (id < 0 || id >= a.num_cache_blocks) && a.err_word)
                    atomicOr(a.err_word, PDA_ERRW_BAD_BLOCK_ID);
                const unsigned st = step % Cfg::kScales;
                if (F16 && step >= Cfg::kScales && !wait(bars + kScEmpty + 8 * st, (step / Cfg::kScales - 1) & 1)) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int v = 0; v < 2; ++v, ++seq) {   // K, then V
                    const int s = seq % kNS;
                    if (seq >= kNS && !wait(bars + kEmpty0 + 8 * s, (seq / kNS - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = bars + kFull0 + 8 * s;
                    const uint32_t row_bytes = (uint32_t)n * a.BS * 128u * kHalves;
                    const bool scales = F16 && v == 0;
                    if (lane == 0) {
                        if (scales) mbar_arrive_expect_tx(bars + kScRaw + 8 * st, (uint32_t)n * a.BS * 8u);
                        mbar_arrive_expect_tx(bar, row_bytes);
                    }
                    __syncwarp();
                    if (mine) {
                        tma_load_5d(base + s * kBytes + half * 16384 + blk * a.BS * 128, kv_map, bar, 0, 0,
                                    v * kHalves + half, u.h, id, policy);
                        if (scales)
                            tma_load_4d(sm + Cfg::kOffScales + st * Cfg::kScaleBytes + blk * a.BS * 8, sc_map,
                                        bars + kScRaw + 8 * st, 0, 0, u.h, id, policy);
                    }
                    __syncwarp();
                }
                id = nid;
                b0 = b1;
            }
        }
        // no copy may land in this CTA's memory after it leaves, whichever role gave up
        for (int s = 0; s < kNS; ++s)
            if (seq > (unsigned)s) {
                const unsigned q = (seq - 1 - s) / kNS;   // the slot's last use
                (void)mbar_wait(bars + kFull0 + 8 * s, q & 1, kDefaultTimeoutNs);
            }
        if (F16) {
            const unsigned issued = (seq + 1) / 2;   // steps whose scales were asked for
            for (int s = 0; s < Cfg::kScales; ++s)
                if (issued > (unsigned)s)
                    (void)mbar_wait(bars + kScRaw + 8 * s, (issued - 1 - s) / Cfg::kScales & 1, kDefaultTimeoutNs);
        }
    }

    // The same for drafted tokens, one warp for K (TQ4: for all) and one for V (Q8: with the scales, which are plain asynchronous
    // copies of 16 bytes): a tensor copy takes its warp 26 ns (50
    // cycles), and 32 of them, of 16 tokens and 64 dimensions each, more than the products of a step of few rows.
    __device__ __forceinline__ void copies_tree(const CUtensorMap* kv_map, const CUtensorMap* sc_map, int v) {
        const int lane = threadIdx.x & 31;
        constexpr int kHalves = F16 ? 1 : 2;
        constexpr uint32_t kBytes = F16 ? kRawBytes : kSlotBytes, kField = TQ ? 6u : 8u;   // of a token's scales
        // a ring for each; TQ4: one for both
        const bool keys = Q8 && v == 0;
        const uint32_t ring = !F16 ? (v ? Cfg::kValues : Cfg::kKeys) : keys ? Cfg::kKeys : Cfg::kRaw, at = !F16 && v ? Cfg::kKeys : 0;
        const uint32_t full = bars + (F16 && !keys ? kBarRawFull : kBarFull) + 8 * at;
        const uint32_t empty = bars + (F16 && !keys ? kBarRawEmpty : kBarEmpty) + 8 * at;
        const uint32_t base = sm + (keys ? Cfg::kOffKeys : F16 ? Cfg::kOffRaw : Cfg::kOffSlots) + at * kBytes;
        const int nblk = kStep / a.BS, blk = lane / kHalves, half = lane % kHalves;
        const uint64_t once = l2_policy_evict_first(), again = l2_policy_evict_normal();
        unsigned filled = 0, step = 0;   // copies of this warp, in slots; steps whose scales were asked for
        uint32_t s = 0, ph = 1, st = 0, st_ph = 1;
        bool ok = true;
        Unit u;
        while (ok && next(u)) {
            const Sight x = sight(u);
            const uint64_t policy = u.rows > kUnitRows ? again : once;   // other row tiles read it too
            const int* table = a.prefix_table + (long long)u.g * a.MP;
            const int last = (u.len + a.BS - 1) / a.BS;   // blocks of the sequence
            int id = 0, b0 = step_of(u, x, 0) * nblk;
            if (blk < nblk && b0 + blk < last) id = __ldcg(table + b0 + blk);
            for (int j = 0; j < u.steps; ++j) {
                // a block that all rows miss may be another's by now, or none: it is not looked at
                const bool mine = blk < min(nblk, last - b0) && !((b0 + blk) * a.BS >= x.hole0 && (b0 + blk + 1) * a.BS <= x.hole1);
                const int n = __popc(__ballot_sync(kLanes, mine && half == 0));
                int nid = 0, b1 = 0;
                if (j + 1 < u.steps) {
                    b1 = step_of(u, x, j + 1) * nblk;
                    if (blk < nblk && b1 + blk < last) nid = __ldcg(table + b1 + blk);
                }
                const bool scales = Q8 ? v == 1 : F16;
                if (mine && half == 0 && v == 0 && (id < 0 || id >= a.num_cache_blocks) && a.err_word)
                    atomicOr(a.err_word, PDA_ERRW_BAD_BLOCK_ID);
                ok = (!scales || wait(bars + kScEmpty + 8 * st, st_ph)) && wait(empty + 8 * s, ph);   // both start free
                if (!ok) break;
                if (lane == 0) {
                    if (!Q8 && scales) mbar_arrive_expect_tx(bars + kScRaw + 8 * st, (uint32_t)n * a.BS * kField);
                    mbar_arrive_expect_tx(full + 8 * s, (uint32_t)n * a.BS * 128u * kHalves);
                }
                __syncwarp();
                if (mine) {
                    tma_load_5d(base + s * kBytes + half * 16384 + blk * a.BS * 128, kv_map, full + 8 * s, 0, 0, v * kHalves + half, u.h, id,
                                policy);
                    if (!Q8 && scales)
                        tma_load_4d(sm + Cfg::kOffScales + st * Cfg::kScaleBytes + blk * a.BS * 8, sc_map, bars + kScRaw + 8 * st, 0, 0, u.h,
                                    id, policy);
                }
                __syncwarp();
                if constexpr (Q8) if (scales) {
                    const int mask = (int)__ballot_sync(kLanes, mine && id >= 0 && id < a.num_cache_blocks);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {   // 16 bytes c of the step's 1024; a block's are BS * 8
                        const int c = lane + 32 * i, b = a.BS == 32 ? c >> 4 : c >> 3;
                        const long long from = __shfl_sync(kLanes, id, b) * a.block_bytes + a.meta_bytes +
                                               (long long)u.h * a.BS * 8 + (c * 16 & (a.BS * 8 - 1));
                        const bool there = mask >> b & 1;
                        cp_async16(sm + Cfg::kOffScales + st * Cfg::kScaleBytes + 16 * c, there ? a.cache + from : a.cache, there ? 16u : 0u);
                    }
                    cp_async_arrive(bars + kScRaw + 8 * st);
                }
                ++filled;
                if (++s == ring) {
                    s = 0;
                    ph ^= 1;
                }
                if (scales) {
                    ++step;
                    if (++st == Cfg::kScales) {
                        st = 0;
                        st_ph ^= 1;
                    }
                }
                id = nid;
                b0 = b1;
            }
        }
        // no copy may land in this CTA's memory after it leaves, whichever role gave up: the last use of every slot
        for (uint32_t i = 0; i < ring && i < filled; ++i) {
            s = s > 0 ? s - 1 : ring - 1;
            if (s + 1 == ring) ph ^= 1;
            (void)mbar_wait(full + 8 * s, ph ^ 1, kDefaultTimeoutNs);
        }
        if constexpr (Q8) cp_async_wait_all();
        for (uint32_t i = 0; !Q8 && i < Cfg::kScales && i < step; ++i) {
            st = st > 0 ? st - 1 : Cfg::kScales - 1;
            if (st + 1 == Cfg::kScales) st_ph ^= 1;
            (void)mbar_wait(bars + kScRaw + 8 * st, st_ph ^ 1, kDefaultTimeoutNs);
        }
    }

    // ---------------------------------------------------------------- conversion (fp8)
    // One warp lays a step's scales out as [128 K scales][128 V scales / F]: the K scales for the softmax, the
    // others for the conversion.  F keeps V in f16's range (the accumulator counts in units of F): 16 F is the
    // step's largest V scale f, and F stays as it is while f lies in [2F, 128F].  So the largest products stay
    // below 448 * 128 = 57344, and a scale keeps its 11 bits down to 2^-15 f (2 F * 2^-15 = 2^-14 F).
    // TQ4: a token's values lie within 15 |v_scale| + |v_zero|; f is the largest such bound, 2048 F = f, and F stays while f lies
    // in [256 F, 32768 F].  The values are computed in 32 bits and rounded to f16 once.
    __device__ void scales() {
        const int lane = threadIdx.x & 31;
        unsigned st = 0, ph = 0;
        float F = 1.f;
        Unit u;
        while (next(u)) {
            const Sight x = sight(u);
            for (int j = 0; j < u.steps; ++j) {
                const int valid = tokens_of(u, x, j), t0 = step_of(u, x, j) * kStep;
                uint32_t gone = 0;
                if (u.hidden && t0 + kStep > x.ctx)
#pragma unroll 1
                    for (int i = 0; i < 4; ++i) gone |= (uint32_t)(lane + 32 * i < valid && hidden(u, x, t0 + lane + 32 * i)) << i;
                if (!wait(bars + kScRaw + 8 * st, ph)) return;
                const uint32_t sc = sm + Cfg::kOffScales + st * Cfg::kScaleBytes;
                float ks[4], vs[4], vz[4], f = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int tok = lane + 32 * i;
                    const bool there = tok < valid && !missed(x, t0 + tok) && !(gone >> i & 1);
                    if constexpr (TQ) {
                        ks[i] = there ? field_at(sc, tok, 0) : 0.f;
                        vs[i] = there ? field_at(sc, tok, 1) : 0.f;
                        vz[i] = there ? field_at(sc, tok, 2) : 0.f;
                        f = fmaxf(f, fmaf(15.f, fabsf(vs[i]), fabsf(vz[i])));
                    } else {
                        ks[i] = there ? __uint_as_float(lds32v(scale_at(sc, tok, 0))) : 0.f;
                        vs[i] = there ? __uint_as_float(lds32v(scale_at(sc, tok, 1))) : 0.f;
                        vz[i] = 0.f;
                        f = fmaxf(f, fabsf(vs[i]));
                    }
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) f = fmaxf(f, __shfl_xor_sync(kLanes, f, o));
                if (!(f > 0.f)) f = 1.f;
                constexpr float kHigh = TQ ? 32768.f : 128.f, kLow = TQ ? 256.f : 2.f, kMid = TQ ? 1.f / 2048.f : 0.0625f;
                if (j == 0 || f > F * kHigh || f < F * kLow) F = fmaxf(f * kMid, 1e-37f);   // 1 / F is finite
                const float rF = 1.f / F;
#pragma unroll
                for (int i = 0; i < 4; ++i) {   // the shuffles above come after every lane's reads
                    sts32v(sc + (lane + 32 * i) * 4, __float_as_uint(ks[i]));
                    sts32v(sc + 512 + (lane + 32 * i) * 4, __float_as_uint(vs[i] * rF));
                    if constexpr (TQ) sts32v(sc + 1024 + (lane + 32 * i) * 4, __float_as_uint(vz[i] * rF));
                }
                if (lane == 0) sts32v(bars + kFAt + 4 * st, __float_as_uint(F));
                fence_proxy_async_shared();   // the next copy into this stage comes after these stores
                __syncwarp();
                if (lane == 0) mbar_arrive(bars + kScFull + 8 * st);
                if (++st == Cfg::kScales) {
                    st = 0;
                    ph ^= 1;
                }
            }
        }
    }
    // Thread t of the converting warps turns token t's 128 codes into f16: K as it is (exact: every e4m3 value is
    // an f16 value; the factor is 1), V times its token's scale over F (two roundings to f16, 2^-11 each, beside
    // P's one; it spares the softmax a product per weight).  Rows past the prefix become zeros, since a
    // weight of zero does not silence a NaN.  This chain (raw codes landed, read, convert, store, announce) paces the fp8
    // pass, so nothing else stands in it: no scales, no branches, and the reads are requested before the slot is free.
    __device__ void convert() {
        if constexpr (TQ)
            convert_tq4();
        else if constexpr (Q8)
            convert_values();
        else
            convert_fp8();
    }
    // Q8: V alone, in halves of 64 tokens, two warps each.  Thread t takes token t's 128 codes times the token's scale over F, as
    // in convert_fp8.  One warp has its processor's quarter to itself for most of a step, so its time is its longest chain: one
    // wait of each kind, all reads at once, no division but where F moves.
    __device__ __forceinline__ void convert_values() {
        const int t = threadIdx.x - 384, lane = t & 31, sw = t & 7, second = t >> 6;
        const uint32_t raw0 = sm + Cfg::kOffRaw + t * 128, slot0 = sm + Cfg::kOffSlots + (t & 63) * 128;
        const uint32_t mine = scale_at(sm + Cfg::kOffScales, t, 1), four = scale_at(sm + Cfg::kOffScales, 4 * lane, 1);
        unsigned s = 0, ph = 0, h = second, h_ph = 1;   // the slots start free
        uint32_t st = 0, st_ph = 0;
        float F = 1.f, rF = 1.f;
        Unit u;
        while (next(u)) {
            const Sight x = sight(u);
            for (int j = 0; j < u.steps; ++j) {
                const int valid = tokens_of(u, x, j), t0 = step_of(u, x, j) * kStep;
                const uint32_t sc = st * Cfg::kScaleBytes;
                // F as in `scales`, by each of the warps for itself; the first tells the softmax
                if (!wait(bars + kScRaw + 8 * st, st_ph)) return;
                uint32_t v[4];
                lds128(four + sc, v[0], v[1], v[2], v[3]);
                float vs = __uint_as_float(lds32v(mine + sc));
                bool zero = false;
                if (valid < kStep || (t0 < x.hole1 && t0 + kStep > x.hole0)) {   // a token that is not there may have any scale and codes
                    zero = t >= valid || missed(x, t0 + t);
                    if (zero) vs = 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (4 * lane + i >= valid || missed(x, t0 + 4 * lane + i)) v[i] = 0u;
                }
                if (u.hidden && t0 + kStep > x.ctx) {
                    zero = zero || hidden(u, x, t0 + t);   // not past the sequence's end
                    if (zero) vs = 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (4 * lane + i < valid && hidden(u, x, t0 + 4 * lane + i)) v[i] = 0u;
                }
                // magnitudes are ordered like their bits; a NaN counts for nothing
                uint32_t y = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i] &= 0x7FFFFFFFu;
                    y = max(y, v[i] > 0x7F800000u ? 0u : v[i]);
                }
                y = __reduce_max_sync(kLanes, y);
                const float top = y ? __uint_as_float(y) : 1.f;
                if (j == 0 || top > F * 128.f || top < F * 2.f) {
                    F = fmaxf(top * 0.0625f, 1e-37f);   // 1 / F is finite
                    rF = 1.f / F;
                }
                if (t == 0) {
                    sts32v(bars + kFAt + 4 * st, __float_as_uint(F));
                    mbar_arrive(bars + kScFull + 8 * st);
                }
                __syncwarp();
                vs *= rF;
                const uint32_t vs2 = pack_f16(vs, vs);
                if (!wait(bars + kBarRawFull + 8 * s, ph)) return;
                const uint32_t src = raw0 + s * kRawBytes, dst = slot0 + h * kRawBytes;
                if (!wait(bars + kBarVEmpty + 8 * h, h_ph)) return;
#pragma unroll 2
                for (int c = 0; c < 8; ++c) {
                    uint32_t w[4], o[8];
                    lds128(src + ((c ^ sw) << 4), w[0], w[1], w[2], w[3]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) e4m3x4_to_f16x2x2(zero ? 0u : w[i], o[2 * i], o[2 * i + 1]);
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = mul_f16x2(o[i], vs2);
                    const uint32_t d = dst + (c >> 2) * 8192;
                    const int k = 2 * (c & 3);
                    sts128(d + ((k ^ sw) << 4), o[0], o[1], o[2], o[3]);
                    sts128(d + (((k + 1) ^ sw) << 4), o[4], o[5], o[6], o[7]);
                }
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bars + kBarVFull + 8 * h);
                    mbar_arrive(bars + kBarRawEmpty + 8 * s);
                    mbar_arrive(bars + kScEmpty + 8 * st);
                }
                h += 2;
                if (h >= Cfg::kHalves) {
                    h -= Cfg::kHalves;
                    h_ph ^= 1;
                }
                if (++s == Cfg::kRaw) {
                    s = 0;
                    ph ^= 1;
                }
                if (++st == Cfg::kScales) {
                    st = 0;
                    st_ph ^= 1;
                }
            }
        }
    }
    __device__ __forceinline__ void convert_fp8() {
        const int t = threadIdx.x - 384, lane = t & 31, sw = t & 7;
        const uint32_t raw0 = sm + Cfg::kOffRaw + t * 128, slot0 = sm + Cfg::kOffSlots + t * 128;
        const uint32_t scale0 = sm + Cfg::kOffScales + 512 + t * 4;
        static_assert(!F16 || Cfg::kRaw == Cfg::kSlots, "a raw slot and its slot are counted together");
        unsigned s = 0, ph = 0, st = 0, st_ph = 0;
        Unit u;
        while (next(u)) {
            const Sight x = sight(u);
            for (int j = 0; j < u.steps; ++j) {
                const bool zero = t >= tokens_of(u, x, j) || missed(x, step_of(u, x, j) * kStep + t);
#pragma unroll 1
                for (int v = 0; v < 2; ++v) {
                    if (!wait(bars + kBarRawFull + 8 * s, ph)) return;
                    const uint32_t src = raw0 + s * kRawBytes, dst = slot0 + s * kSlotBytes;
                    uint32_t w[8][4];
#pragma unroll
                    for (int c = 0; c < 8; ++c) lds128(src + ((c ^ sw) << 4), w[c][0], w[c][1], w[c][2], w[c][3]);
                    float vs = 1.f;
                    if (v) {
                        if (!wait(bars + kScFull + 8 * st, st_ph)) return;
                        vs = __uint_as_float(lds32v(scale0 + st * Cfg::kScaleBytes));
                        if (++st == Cfg::kScales) {
                            st = 0;
                            st_ph ^= 1;
                        }
                    }
                    const uint32_t vs2 = pack_f16(vs, vs);
                    if (!wait(bars + kBarEmpty + 8 * s, ph ^ 1)) return;   // the slots start free
                    if (zero) {
#pragma unroll
                        for (int c = 0; c < 8; ++c) w[c][0] = w[c][1] = w[c][2] = w[c][3] = 0u;
                    }
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        uint32_t o[8];
#pragma unroll
                        for (int i = 0; i < 4; ++i) e4m3x4_to_f16x2x2(w[c][i], o[2 * i], o[2 * i + 1]);
#pragma unroll
                        for (int i = 0; i < 8; ++i) o[i] = mul_f16x2(o[i], vs2);
                        const uint32_t d = dst + (c >> 2) * 16384;
                        const int k = 2 * (c & 3);
                        sts128(d + ((k ^ sw) << 4), o[0], o[1], o[2], o[3]);
                        sts128(d + (((k + 1) ^ sw) << 4), o[4], o[5], o[6], o[7]);
                    }
                    fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(bars + kBarFull + 8 * s);
                        mbar_arrive(bars + kBarRawEmpty + 8 * s);
                    }
                    if (++s == Cfg::kSlots) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
        }
    }
    // TQ4.  Thread t turns token t's 64 + 64 bytes of codes into f16: K's through the table of byte pairs (centroids times a
    // power of two; k_norm is the step's K scale), V as code * v_scale + v_zero over F in 32 bits, rounded once.  Step by step
    // K, then V, out of one raw slot.
    __device__ __forceinline__ void convert_tq4() {
        const int t = threadIdx.x - 384, lane = t & 31, sw = t & 7;
        const uint32_t raw0 = sm + Cfg::kOffRaw + t * 128, slot0 = sm + Cfg::kOffSlots + t * 128;
        const uint32_t scale0 = sm + Cfg::kOffScales + 512 + t * 4, table = sm + Cfg::kOffTable;
        unsigned s = 0, ph = 0, rs = 0, rph = 0, st = 0, st_ph = 0;
        Unit u;
        while (next(u)) {
            const Sight x = sight(u);
            for (int j = 0; j < u.steps; ++j) {
                const bool zero = t >= tokens_of(u, x, j) || missed(x, step_of(u, x, j) * kStep + t);
                if (!wait(bars + kBarRawFull + 8 * rs, rph)) return;
                const uint32_t src = raw0 + rs * kRawBytes;
                if (!wait(bars + kBarEmpty + 8 * s, ph ^ 1)) return;   // the slots start free
                uint32_t dst = slot0 + s * kSlotBytes;
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {   // 32 dimensions, in 16 bytes of codes
                    uint32_t w[4];
                    lds128(src + ((q ^ sw) << 4), w[0], w[1], w[2], w[3]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {   // 16 bytes of f16 from 4 of codes
                        const uint32_t code = zero ? 0u : w[c];
                        uint32_t o[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[i] = lds32v(table + ((code >> (8 * i)) & 0xFFu) * 4);
                        sts128(dst + (q >> 1) * 16384 + (((4 * (q & 1) + c) ^ sw) << 4), o[0], o[1], o[2], o[3]);
                    }
                }
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(bars + kBarFull + 8 * s);
                if (++s == Cfg::kSlots) {
                    s = 0;
                    ph ^= 1;
                }
                if (!wait(bars + kScFull + 8 * st, st_ph)) return;
                // 1 + code / 16 costs one instruction: V = (1 + code / 16) 16 v_scale + (v_zero - 16 v_scale).  A token that is
                // not there has both 0.  Off, in units of 2^-24, by 2 v_scale code + 2 v_zero for 1 / F and the products with it, by
                // 16 v_scale + v_zero for the difference and by the value for the sum: below 2^-18 |v_scale| + 2^-21 |v_zero|.
                const float vs = 16.f * __uint_as_float(lds32v(scale0 + st * Cfg::kScaleBytes));
                const float vz = __uint_as_float(lds32v(scale0 + st * Cfg::kScaleBytes + 512)) - vs;
                if (++st == Cfg::kScales) {
                    st = 0;
                    st_ph ^= 1;
                }
                if (!wait(bars + kBarEmpty + 8 * s, ph ^ 1)) return;
                dst = slot0 + s * kSlotBytes;
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    uint32_t w[4];
                    lds128(src + (((4 + q) ^ sw) << 4), w[0], w[1], w[2], w[3]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t code = zero ? 0u : w[c];
                        uint32_t o[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float lo = __uint_as_float(((code >> (8 * i)) & 0xFu) << 19 | 0x3F800000u);
                            const float hi = __uint_as_float(((code >> (8 * i + 4)) & 0xFu) << 19 | 0x3F800000u);
                            o[i] = pack_f16(fmaf(lo, vs, vz), fmaf(hi, vs, vz));
                        }
                        sts128(dst + (q >> 1) * 16384 + (((4 * (q & 1) + c) ^ sw) << 4), o[0], o[1], o[2], o[3]);
                    }
                }
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bars + kBarFull + 8 * s);
                    mbar_arrive(bars + kBarRawEmpty + 8 * rs);
                }
                if (++s == Cfg::kSlots) {
                    s = 0;
                    ph ^= 1;
                }
                if (++rs == Cfg::kRaw) {
                    rs = 0;
                    rph ^= 1;
                }
            }
        }
    }
    // One warp lays out the table of the centroids, times a power of two that brings the largest into [2^14, 2^15), in f16.
    __device__ __forceinline__ void make_table() const {
        const int lane = threadIdx.x & 31;
        const float c = __ldcg(a.centroids + (lane & 15));
        float top = fabsf(c);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kLanes, top, o));
        int e = top > 0.f ? 14 - ((int)(__float_as_uint(top) >> 23 & 0xFF) - 127) : 0;
        e = max(-100, min(100, e));
        if (lane == 0) sts32v(bars + kPowerAt, (uint32_t)(127 - e) << 23);
        const uint32_t h = __half_as_ushort(__float2half_rn(c * __uint_as_float((uint32_t)(e + 127) << 23)));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int x = 8 * lane + i;
            const uint32_t lo = __shfl_sync(kLanes, h, x & 15), hi = __shfl_sync(kLanes, h, x >> 4);
            sts32v(sm + Cfg::kOffTable + 4 * x, lo | hi << 16);
        }
    }
    // A TQ4 field of token tok as copied: [block][field][BS], f16.
    __device__ __forceinline__ float field_at(uint32_t sc, int tok, int field) const {
        const int b = a.BS == 32 ? tok >> 5 : tok >> 4;
        const uint32_t at = sc + b * a.BS * 8 + (field * a.BS + (tok - b * a.BS)) * 2;   // a copy starts at 128 bytes
        const uint32_t w = lds32v(at & ~3u);
        return __half2float(__ushort_as_half((uint16_t)(at & 2u ? w >> 16 : w & 0xFFFFu)));
    }
    // Address of token tok's K (field 0) or V (field 1) scale as copied: [block][field][BS].
    __device__ __forceinline__ uint32_t scale_at(uint32_t sc, int tok, int field) const {
        const int b = a.BS == 32 ? tok >> 5 : tok >> 4;
        return sc + (b * a.BS * 2 + field * a.BS + (tok - b * a.BS)) * 4;
    }

    // ---------------------------------------------------------------- products
    static constexpr uint32_t kSlot16 = kSlotBytes >> 4;   // descriptors count 16 bytes
    static __device__ __forceinline__ void qk(uint32_t leader, uint32_t d, uint64_t q, uint64_t k) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t o = ((i >> 2) * 16384 + (i & 3) * 32) >> 4;
            umma_ss(leader, d, q + o, k + o, kIdescQK, i > 0);
        }
    }
    template <int HALF>
    static __device__ __forceinline__ void pv(uint32_t leader, uint32_t d, uint32_t p, uint64_t v, bool accumulate) {
#pragma unroll
        for (int i = 4 * HALF; i < 4 * HALF + 4; ++i)
            umma_ts(leader, d, p + i * 8, v + ((i * 2048) >> 4), kIdescPV, accumulate || i > 0);
    }
    __device__ void products(uint32_t tmem_base) {
        if constexpr (TREE)
            products_tree(tmem_base);
        else
            products_f16(tmem_base);
    }
    // Products in flight read shared memory and TMEM: let them end, whichever role gave up.
    __device__ __forceinline__ void drain(uint32_t leader, uint32_t bar) const {
        umma_commit(leader, bar + kBarDrain);
        __syncwarp();
        (void)mbar_wait(bars + kBarDrain, 0, kDefaultTimeoutNs);
    }
    // Drafted tokens.  The units of two tiles as in the prefix pass.  Those of one, at most 128 rows, go to the tiles by turns, so that
    // one tile's first rows are fetched and its last ones stored beside the other's steps, and their steps use the two places for
    // S by turns: S of step g + 2 is computed where S and P of step g were as soon as the product of that P is issued, so that the
    // softmax of a step finds its S there already.
    // Q8: S = Qhi K^T + Qlo K^T, e4m3 each, and V comes in halves.
    // Measured, sequences with 4 drafted tokens of 8 heads and 8 query rows each: 64 of 4096 bf16 tokens 194 -> 176 us (6.1 TB/s), of
    // 1000 66 -> 59; 64 of 4096 fp8 tokens 217 -> 202, and with the halves (see there) 166.
    __device__ __forceinline__ void products_tree(uint32_t tmem_base) {
        const int lane = threadIdx.x & 31;
        const uint32_t leader = elect_one(), tmem = uniform(tmem_base), smu = uniform(sm), bar = uniform(bars);
        constexpr uint32_t kRaw16 = kRawBytes >> 4, kKey16 = Q8 ? kRaw16 : kSlot16;
        // TQ4: K and V in turn in one ring
        constexpr uint32_t kVAt = TQ || Q8 ? 0 : Cfg::kKeys, kStride = TQ ? 2 : 1, kKRing = TQ ? Cfg::kSlots : Cfg::kKeys;
        constexpr uint32_t kVFull = Q8 ? kBarVFull : kBarFull + 8 * kVAt, kVEmpty = Q8 ? kBarVEmpty : kBarEmpty + 8 * kVAt;
        constexpr uint32_t kVRing = Q8 ? Cfg::kHalves : TQ ? Cfg::kSlots : Cfg::kValues;
        const uint64_t q0 = umma_desc(smu + Cfg::kOffQ, 16, 1024), k0 = umma_desc(smu + (Q8 ? Cfg::kOffKeys : Cfg::kOffSlots), 16, 1024);
        const uint64_t v0 = umma_desc(smu + Cfg::kOffSlots + kVAt * kSlotBytes, Q8 ? 8192 : 16384, 1024);
        uint32_t ks = 0, kph = 0, vs = TQ ? 1 : 0, vph = 0;   // the next slot of K, and of V
        uint32_t q_ph = 0, p_ph = 0;                          // a bit per tile, and per place
        uint32_t place = 0;                                   // of the next step of a unit of one tile
        auto move = [](uint32_t& slot, uint32_t& ph, uint32_t stride, uint32_t ring) {
            slot += stride;
            if (slot >= ring) {
                slot -= ring;
                ph ^= 1;
            }
        };
        auto scores = [&](uint32_t tile, uint32_t to) {
            const uint64_t q = q0 + tile * kSlot16, k = k0 + ks * kKey16;
            if constexpr (Q8) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {   // 32 dimensions at a time, first of the high parts, then of the low ones
                    const uint32_t o = (i & 3) * 32 >> 4;
                    umma_ss_f8(leader, tmem + to * 128, q + (i >> 2) * kRaw16 + o, k + o, kIdescQ8, i > 0);
                }
            } else {
                qk(leader, tmem + to * 128, q, k);
            }
            umma_commit(leader, bar + (to ? kBarS2 : kBarS) + 8 * tile);
        };
        auto release_keys = [&] {
            umma_commit(leader, bar + kBarEmpty + 8 * ks);
            move(ks, kph, kStride, kKRing);
        };
        // bf16 rows that nobody sees may hold anything: a weight of zero does not silence a NaN
        auto clear = [&](int valid, int h0, int h1, uint32_t unseen) -> bool {   // unseen: see unseen_of
            if (!wait(bar + kVFull + 8 * vs, vph)) return false;
            const uint32_t s = sm + Cfg::kOffSlots + (kVAt + vs) * kSlotBytes;
            for (int i = lane; i < kStep * 8; i += 32)
                if (const int r = i >> 3; r >= valid || (r >= h0 && r < h1)) {
                    sts128(s + i * 16, 0u, 0u, 0u, 0u);
                    sts128(s + 16384 + i * 16, 0u, 0u, 0u, 0u);
                }
            if (__any_sync(kLanes, unseen))   // rare, and apart: in the loop above its test cost every last step 0.3 us
#pragma unroll 1
                for (int i = lane; i < kStep * 8; i += 32)
                    if (__shfl_sync(kLanes, unseen, i >> 5) >> (i >> 3 & 3) & 1) {
                        sts128(s + i * 16, 0u, 0u, 0u, 0u);
                        sts128(s + 16384 + i * 16, 0u, 0u, 0u, 0u);
                    }
            fence_proxy_async_shared();
            __syncwarp();
            return true;
        };
        // O += P V of a step for one tile, in halves; opens, closes: the step's first and last tile.
        auto values = [&](uint32_t tile, uint32_t from, bool accumulate, bool opens, bool closes) -> bool {
            uint32_t v1 = vs, v1ph = vph;   // of the second half
            if constexpr (Q8) move(v1, v1ph, 1, kVRing);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint32_t slot = half ? v1 : vs;
                if (opens && (Q8 || half == 0) && !wait(bar + kVFull + 8 * slot, half ? v1ph : vph)) return false;
                if (!wait(bar + (half ? kBarP2 : kBarP) + 8 * from, p_ph >> from & 1)) return false;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    umma_ts(leader, tmem + 256 + tile * 128, tmem + from * 128 + (4 * half + k) * 8,
                            v0 + slot * kKey16 + (((Q8 ? k : 4 * half + k) * 2048) >> 4), kIdescPV, accumulate || half > 0 || k > 0);
                umma_commit(leader, bar + (half ? kBarWhole : kBarHalf) + 8 * tile);
                if (closes && (Q8 || half == 1)) umma_commit(leader, bar + kVEmpty + 8 * slot);
            }
            p_ph ^= 1u << from;
            return true;
        };
        auto next_values = [&] {
            move(vs, vph, kStride, kVRing);
            if constexpr (Q8) move(vs, vph, 1, kVRing);
        };
        // Hidden tokens of a step, a bit each: of tokens 4 i .. 4 i + 3 in lane i.
        auto unseen_of = [&](const Unit& u, const Sight& x, int t0) -> uint32_t {
            uint32_t unseen = 0;
            if (u.hidden && t0 + kStep > x.ctx)
#pragma unroll 1
                for (int t = t0 + 4 * lane + 3, i = 0; i < 4; --t, ++i) unseen = 2 * unseen + (t < u.len && hidden(u, x, t));
            return unseen;
        };
        auto two_tiles = [&](const Unit& u, const Sight& x) -> bool {
            const int steps = uniform(u.steps);
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                if (!wait(bar + kBarQ + 8 * w, q_ph >> w & 1)) return false;
                if (w == 0 && !wait(bar + kBarFull + 8 * ks, kph)) return false;
                tc_fence_after();
                scores(w, w);
            }
            q_ph ^= 3;
            release_keys();
            for (int j = 0; j < steps; ++j) {
                const bool more = j + 1 < steps;
                if constexpr (!F16) {
                    const int t0 = uniform(step_of(u, x, j) * kStep), valid = min(kStep, u.len - t0);
                    const int h0 = min(max(x.hole0 - t0, 0), kStep), h1 = min(max(x.hole1 - t0, 0), kStep);
                    const uint32_t unseen = unseen_of(u, x, t0);
                    if ((valid < kStep || h0 < h1 || (u.hidden && t0 + kStep > x.ctx)) && !clear(valid, h0, h1, unseen)) return false;
                }
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    if (!values(w, w, j > 0, w == 0, w == 1)) return false;
                    if (more) {
                        if (w == 0 && !wait(bar + kBarFull + 8 * ks, kph)) return false;
                        scores(w, w);
                    } else {
                        umma_commit(leader, bar + kBarO + 8 * w);
                    }
                }
                if (more) release_keys();
                next_values();
            }
            return true;
        };
        // A step of a unit of one tile: its tile and place, and whether it is the unit's first or last.
        enum : uint32_t { kPlace = 2, kFirst = 4, kLast = 8, kClear = 16 };
        Unit u;
        Sight x = {};
        int j = 0, out = 0;
        u.steps = 0;
        bool more = true;
        uint32_t first = 0, second = 0;   // steps whose product with V is to come
        uint32_t first_unseen = 0, second_unseen = 0;
        auto all = [&] {
            for (;;) {
                if (more && j == u.steps) {
                    more = uniform((int)next(u));
                    x = sight(u);
                    j = 0;
                }
                if (uniform((int)(more && out < 2))) {
                    if (uniform((int)active(u, 1))) {
                        if (out == 0) {
                            if (!two_tiles(u, x)) return;
                            j = u.steps;
                            place = 0;
                            continue;
                        }
                    } else {
                        // The first S of a unit waits for the tile's rows; not while a product is to come: they may come only after it.
                        const uint32_t tile = uniform(units & 1);
                        bool ok = true;
                        if (j == 0) {
                            if (out) {
                                ok = __all_sync(kLanes, mbar_test_wait(bar + kBarQ + 8 * tile, q_ph >> tile & 1));
                            } else if (!wait(bar + kBarQ + 8 * tile, q_ph >> tile & 1)) {
                                return;
                            }
                        }
                        if (uniform((int)ok)) {
                            if (j == 0) q_ph ^= 1u << tile;
                            if (!wait(bar + kBarFull + 8 * ks, kph)) return;
                            tc_fence_after();
                            scores(tile, place);
                            release_keys();
                            uint32_t turn = tile | place << 1 | (j == 0 ? kFirst : 0);
                            if (++j == u.steps) turn |= kLast;
                            if constexpr (!F16) {
                                const int t0 = uniform(step_of(u, x, j - 1) * kStep), valid = min(kStep, u.len - t0);
                                const int h0 = min(max(x.hole0 - t0, 0), kStep), h1 = min(max(x.hole1 - t0, 0), kStep);
                                if (valid < kStep || h0 < h1 || (u.hidden && t0 + kStep > x.ctx)) turn |= kClear | valid << 8 | h0 << 16 | h1 << 24;
                                (out == 0 ? first_unseen : second_unseen) = unseen_of(u, x, t0);
                            }
                            if (out == 0)
                                first = turn;
                            else
                                second = turn;
                            place ^= 1;
                            ++out;
                            continue;
                        }
                    }
                }
                if (out == 0) return;
                const uint32_t turn = uniform(first), tile = turn & 1;
                if (!F16 && (turn & kClear) && !clear(turn >> 8 & 255, turn >> 16 & 255, turn >> 24, first_unseen)) return;
                if (!values(tile, turn >> 1 & 1, !(turn & kFirst), true, true)) return;
                next_values();
                if (turn & kLast) umma_commit(leader, bar + kBarO + 8 * tile);
                first = second;
                first_unseen = second_unseen;
                --out;
            }
        };
        all();
        drain(leader, bar);
    }
    __device__ __forceinline__ void products_f16(uint32_t tmem_base) {
        const int lane = threadIdx.x & 31;
        const uint32_t leader = elect_one(), tmem = uniform(tmem_base), smu = uniform(sm);
        const uint64_t q0 = umma_desc(smu + Cfg::kOffQ, 16, 1024);
        const uint64_t k0 = umma_desc(smu + Cfg::kOffSlots, 16, 1024), v0 = umma_desc(smu + Cfg::kOffSlots, 16384, 1024);
        const uint32_t bar = uniform(bars);
        constexpr uint32_t NS = Cfg::kSlots;
        // Position in the ring: slot and parity of its full barrier.
        struct Pos {
            uint32_t slot, ph;
            __device__ __forceinline__ Pos next() const {
                return slot + 1 == NS ? Pos{0, ph ^ 1} : Pos{slot + 1, ph};
            }
        };
        Pos pos = {0, 0};        // the next tile
        uint32_t unit0 = 0, unit1 = 0, p0 = 0, p1 = 0;
        bool ok = true;
        Unit u;
        auto full = [&](const Pos& x) { return wait(bar + kBarFull + 8 * x.slot, x.ph); };
        while (ok && uniform((int)next(u))) {
            const int tiles = uniform(active(u, 1) ? 2 : 1), steps = uniform(u.steps);
            const Sight x = sight(u);
            // the step that holds the prefix's last, partly filled tile (-1: none)
            int ragged = -1;
            if (!F16 && u.len % kStep) {
                const int i = u.len / kStep - u.step0 - u.rot;
                if (u.len / kStep < u.step0 + u.steps) ragged = i < 0 ? i + u.steps : i;
            }
            ragged = uniform(ragged);
            if (!(ok = full(pos))) break;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                if (w >= tiles) break;
                uint32_t& n = w ? unit1 : unit0;
                if (!(ok = wait(bar + kBarQ + 8 * w, n))) break;
                n ^= 1;
                tc_fence_after();
                qk(leader, tmem + w * 128, q0 + w * kSlot16, k0 + pos.slot * kSlot16);
                umma_commit(leader, bar + kBarS + 8 * w);
            }
            if (!ok) break;
            umma_commit(leader, bar + kBarEmpty + 8 * pos.slot);
            if (!(ok = full(pos.next()))) break;
            // Between one step's last product and the next step's first only the wait for P stands: K(j + 1) is
            // waited for while PV(0, j) runs, V(j + 1) while QK(0, j + 1) does.
            for (int j = 0; j < steps; ++j) {
                const bool more = j + 1 < steps;
                const Pos v = pos.next(), k = v.next();   // V(j), K(j + 1)
                if (j == ragged) {
                    // bf16 rows past the prefix may hold anything: a weight of zero does not silence a NaN
                    const int valid = u.len % kStep;
                    const uint32_t s = sm + Cfg::kOffSlots + v.slot * kSlotBytes;
                    for (int i = valid * 8 + lane; i < kStep * 8; i += 32) {
                        sts128(s + i * 16, 0u, 0u, 0u, 0u);
                        sts128(s + 16384 + i * 16, 0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_shared();
                    __syncwarp();
                }
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    if (w >= tiles) break;
                    uint32_t& n = w ? p1 : p0;
                    if (!(ok = wait(bar + kBarP + 8 * w, n))) break;
                    tc_fence_after();
                    pv<0>(leader, tmem + 256 + w * 128, tmem + w * 128, v0 + v.slot * kSlot16, j > 0);
                    if (!(ok = wait(bar + kBarP2 + 8 * w, n))) break;
                    n ^= 1;
                    tc_fence_after();
                    pv<1>(leader, tmem + 256 + w * 128, tmem + w * 128, v0 + v.slot * kSlot16, true);
                    if (w == 0 && more && !(ok = full(k))) break;
                    if (more) qk(leader, tmem + w * 128, q0 + w * kSlot16, k0 + k.slot * kSlot16);
                    umma_commit(leader, bar + (more ? kBarS : kBarO) + 8 * w);
                    if (w == 0 && more && !(ok = full(k.next()))) break;
                }
                if (!ok) break;
                umma_commit(leader, bar + kBarEmpty + 8 * v.slot);
                if (more) umma_commit(leader, bar + kBarEmpty + 8 * k.slot);
                pos = k;   // after the last step: the next unit's K(0)
            }
        }
        drain(leader, bar);
    }

    // ---------------------------------------------------------------- softmax
    // Four values as the sum of e4m3 pairs (packed, the first in the low byte).
    static __device__ __forceinline__ void split_e4m3(float x0, float x1, float x2, float x3, uint32_t& hi, uint32_t& lo) {
        const uint32_t h0 = f32x2_to_e4m3x2(x0, x1), h1 = f32x2_to_e4m3x2(x2, x3);
        hi = h0 | h1 << 16;
        uint32_t f0, f1;
        e4m3x4_to_f16x2x2(hi, f0, f1);
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&f0)), b = __half22float2(*reinterpret_cast<const __half2*>(&f1));
        lo = f32x2_to_e4m3x2(x0 - a.x, x1 - a.y) | f32x2_to_e4m3x2(x2 - b.x, x3 - b.y) << 16;
    }
    // The warp's 32 query rows into its tile's operand, two rows (16 lanes each) per asynchronous copy; returns
    // the factor from S to log2 units of this lane's own row, 32 * (warp % 4) + lane.  The loops stay
    // rolled: a short prefix waits for this code's first fetch longer than for its execution.
    __device__ __forceinline__ float load_q(const Unit& u, int tile) const {
        const int lane = threadIdx.x & 31, r0 = threadIdx.x & 96, half = lane >> 4, w = lane & 15;
        const uint32_t base = sm + Cfg::kOffQ + tile * kSlotBytes;
        {
            // 16 bytes w of a row; Q8: neighbours 16 KB apart, where the parts of their 16 dimensions will lie
            const uint32_t dst = base + (Q8 ? w & 1 : w >> 3) * 16384;
            const int place = Q8 ? w >> 1 : w & 7;
            const int row0 = first_row(u, tile) + (halves(u) ? r0 & 63 : r0) + half;
            int seq = row0 / a.QG, q = row0 - seq * a.QG;
            const uint16_t* src = a.query + ((long long)(u.seq0 + seq) * a.Hk + u.h) * a.QG * kHeadDim + 8 * w;
            const long long skip = (long long)a.Hk * a.QG * kHeadDim;
#pragma unroll 2
            for (int i = 0; i < 16; ++i) {
                const int r = r0 + 2 * i + half;
                const bool live = row0 + 2 * i < u.rows;   // else: zeros, and no read
                cp_async16(dst + r * 128 + ((place ^ (r & 7)) << 4), live ? src + q * kHeadDim : a.query, live ? 16u : 0u);
                q += 2;
                if (q >= a.QG) {   // the group size is above 2
                    q -= a.QG;
                    src += skip;
                }
            }
            cp_async_wait_all();
            __syncwarp();
        }
        float c = a.qk_scale_log2;
        if constexpr (TQ) c *= __uint_as_float(lds32v(bars + kPowerAt));
        if constexpr (Q8) {
            // This lane's row times a power of two that brings its largest |q| into [2^7, 2^8), as the sum of two e4m3 parts: the
            // high one has 4 of bf16's 8 bits, and what is left fits 4 more down to 2^-2.  A smaller |q| is off by at most half a
            // step of e4m3's smallest, 2^-10: 2^-17 of the row's largest.
            const uint32_t row = base + (r0 + lane) * 128;
            const int x = lane & 7;
            uint32_t mx = 0;
#pragma unroll 4
            for (int i = 0; i < 16; ++i) {
                uint32_t v[4];
                lds128(row + (i >> 3) * 16384 + (((i & 7) ^ x) << 4), v[0], v[1], v[2], v[3]);   // in any order
                mx = __vmaxs2(mx, __vmaxs2(__vmaxs2(v[0] & 0x7FFF7FFFu, v[1] & 0x7FFF7FFFu),
                                           __vmaxs2(v[2] & 0x7FFF7FFFu, v[3] & 0x7FFF7FFFu)));
            }
            const int top = max(mx & 0xFFFFu, mx >> 16);   // bf16 bits
            int e = top ? 7 - ((top >> 7) - 127) : 0;
            e = max(-100, min(100, e));
            const float pw = __uint_as_float((uint32_t)(e + 127) << 23);
            c *= __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {   // 16 dimensions
                const uint32_t at = row + ((i ^ x) << 4);
                uint32_t v[2][4], hi[4], lo[4];
                lds128(at, v[0][0], v[0][1], v[0][2], v[0][3]);
                lds128(at + 16384, v[1][0], v[1][1], v[1][2], v[1][3]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t a0 = v[k >> 1][2 * (k & 1)], a1 = v[k >> 1][2 * (k & 1) + 1];
                    split_e4m3(bf16_lo(a0) * pw, bf16_hi(a0) * pw, bf16_lo(a1) * pw, bf16_hi(a1) * pw, hi[k], lo[k]);
                }
                sts128(at, hi[0], hi[1], hi[2], hi[3]);
                sts128(at + 16384, lo[0], lo[1], lo[2], lo[3]);
            }
        } else if constexpr (F16) {
            // This lane's row times a power of two that brings its largest |q| into [2^14, 2^15): f16 then
            // keeps every bf16 bit.  The magnitudes of bf16 values order like their bits.
            const uint32_t row = base + (r0 + lane) * 128;
            const int x = lane & 7;
            uint32_t mx = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                uint32_t v[4];
                lds128(row + (i >> 3) * 16384 + (((i & 7) ^ x) << 4), v[0], v[1], v[2], v[3]);
                mx = __vmaxs2(mx, __vmaxs2(__vmaxs2(v[0] & 0x7FFF7FFFu, v[1] & 0x7FFF7FFFu),
                                           __vmaxs2(v[2] & 0x7FFF7FFFu, v[3] & 0x7FFF7FFFu)));
            }
            const int top = max(mx & 0xFFFFu, mx >> 16);   // bf16 bits
            int e = top ? 14 - ((top >> 7) - 127) : 0;
            e = max(-100, min(100, e));
            const float pw = __uint_as_float((uint32_t)(e + 127) << 23);
            c *= __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll 8
            for (int i = 0; i < 16; ++i) {
                const uint32_t at = row + (i >> 3) * 16384 + (((i & 7) ^ x) << 4);
                uint32_t v[4];
                lds128(at, v[0], v[1], v[2], v[3]);
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = pack_f16(bf16_lo(v[k]) * pw, bf16_hi(v[k]) * pw);
                sts128(at, v[0], v[1], v[2], v[3]);
            }
        }
        fence_proxy_async_shared();
        return c;
    }

    // Query rows of one unit for this thread's tile.
    struct Rows {
        bool on, live;       // the tile has rows; this thread has one
        long long head;      // (sequence, KV head)
        int q;
        float c;             // from S to log2 units
        int i, lo;           // TREE: drafted token; the first token of its window
        uint32_t m0, m1;     // the first words of its mask
    };
    __device__ __forceinline__ Rows start_unit(const Unit& u, int tile, int r) const {
        Rows w;
        w.on = TREE || active(u, tile);
        const int row = first_row(u, tile) + (halves(u) ? r & 63 : r);
        w.live = row < u.rows;
        w.head = (long long)(u.seq0 + row / a.QG) * a.Hk + u.h;
        w.q = row % a.QG;
        w.c = 0.f;
        w.i = w.lo = 0;
        w.m0 = w.m1 = 0;
        if constexpr (TREE) {
            w.i = row / a.QG;
            if (a.masks && w.live) {   // asked for now, needed at the unit's last step
                const uint32_t* m = a.masks + (long long)(u.seq0 + w.i) * a.words;
                w.m0 = __ldcg(m);
                w.m1 = __ldcg(m + 1);
            }
            if (a.window > 0 && w.live) {
                // its position: behind the cached tokens and the drafted ones that it sees
                int before = w.i;
                if (a.masks) {
                    const int drafted = u.rows / a.QG;
                    const uint32_t* m = a.masks + (long long)(u.seq0 + w.i) * a.words;
                    before = 0;
                    for (int k = 0; k < a.words && 32 * k < drafted; ++k) {
                        uint32_t bits = __ldcg(m + k) & below(drafted - 32 * k);
                        if (w.i >> 5 == k) bits &= ~(1u << (w.i & 31));
                        before += __popc(bits);
                    }
                }
                w.lo = max(0, u.len - u.rows / a.QG + before + 1 - min(a.window, 1 << 30));
            }
        }
        if (w.on) {   // every product with the last unit's rows has ended: their S was read
            // TREE: a warp whose rows are nobody's leaves what is there
            if (!TREE || first_row(u, tile) + (r & (halves(u) ? 32 : 96)) < u.rows) w.c = load_q(u, tile);
            __syncwarp();
            if ((threadIdx.x & 31) == 0) mbar_arrive(bars + kBarQ + 8 * tile);
        }
        return w;
    }

    static __device__ __forceinline__ uint32_t below(int n) {   // bits 0 .. n-1
        return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u;
    }
    // The tokens t0 .. t0+31 of the sequence that this row sees, a bit each.  Cached token t: inside the row's window, or one of
    // the first.  Drafted token j: its bit of the row's mask; without masks j <= i, and the window as for cached tokens.
    __device__ __forceinline__ uint32_t visible(const Unit& u, const Rows& w, const Sight& x, int t0) const {
        uint32_t in = 0xFFFFFFFFu;
        if (a.window > 0) in = below(a.num_first - t0) | ~below(w.lo - t0);
        const uint32_t old = below(x.ctx - t0);
        const int j0 = t0 - x.ctx;                  // drafted token of bit 0
        const uint32_t fresh = below(x.drafted - j0) & ~old;
        if (!a.masks) return in & (old | (fresh & below(w.i + 1 - j0)));
        uint32_t bits = 0;
        if (fresh && w.live) {
            const uint32_t* m = a.masks + (long long)(u.seq0 + w.i) * a.words;
            auto word = [&](int k) { return k == 0 ? w.m0 : k == 1 ? w.m1 : k >= 0 && k < a.words ? __ldcg(m + k) : 0u; };
            const int k = j0 >> 5, sh = j0 & 31;    // floor and remainder, also below zero
            bits = __funnelshift_r(word(k), sh ? word(k + 1) : 0u, sh);
        }
        return (in & old) | (fresh & bits);
    }

    __device__ void softmax(uint32_t tmem_base, int tile) {
        const int r = threadIdx.x & 127, lane = threadIdx.x & 31;
        const uint32_t lanes = (uint32_t)(r & ~31) << 16;
        const uint32_t tS = tmem_base + tile * 128 + lanes, tO = tmem_base + 256 + tile * 128 + lanes;
        unsigned ns = 0, no = 0, step = 0;
        Unit u;
        while (next(u)) {
            const Rows w = start_unit(u, tile, r);
            const Sight x = sight(u);
            constexpr float below = F16 ? kBelow : 0.f;
            float m = 0.f, l = 0.f, F = 1.f;   // m: the reference, which l and O count from
            for (int j = 0; j < u.steps; ++j, ++step) {
                const int valid = tokens_of(u, x, j);
                const unsigned st = step % Cfg::kScales;
                if (F16 && !wait(bars + kScFull + 8 * st, step / Cfg::kScales & 1)) return;
                if (w.on) {
                    if (!wait(bars + kBarS + 8 * tile, ns++ & 1)) return;
                    tc_fence_after();
                    uint32_t s[4][32];
#pragma unroll
                    for (int k = 0; k < 4; ++k) tmem_ld32(s[k], tS + 32 * k);
                    tmem_wait_ld();
                    if constexpr (F16) {   // the K scales
                        const uint32_t sc = sm + Cfg::kOffScales + st * Cfg::kScaleBytes;
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            uint32_t f[16];
#pragma unroll
                            for (int i = 0; i < 16; i += 4) lds128(sc + (16 * k + i) * 4, f[i], f[i + 1], f[i + 2], f[i + 3]);
#pragma unroll
                            for (int i = 0; i < 16; i += 2) {
                                const int c = (k & 1) * 16 + i;
                                mul2(s[k >> 1][c], s[k >> 1][c + 1], f[i], f[i + 1]);
                            }
                        }
                    }
                    if (valid < kStep) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (32 * k + i >= valid) s[k][i] = 0xFF800000u;   // -inf
                    }
                    float t0 = -INFINITY, t1 = -INFINITY, t2 = -INFINITY, t3 = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        t0 = fmaxf(t0, fmaxf(__uint_as_float(s[0][i]), __uint_as_float(s[0][i + 1])));
                        t1 = fmaxf(t1, fmaxf(__uint_as_float(s[1][i]), __uint_as_float(s[1][i + 1])));
                        t2 = fmaxf(t2, fmaxf(__uint_as_float(s[2][i]), __uint_as_float(s[2][i + 1])));
                        t3 = fmaxf(t3, fmaxf(__uint_as_float(s[3][i]), __uint_as_float(s[3][i + 1])));
                    }
                    const float top = fmaxf(fmaxf(fmaxf(t0, t1), fmaxf(t2, t3)) * w.c, -1e30f);
                    float nF = 1.f;
                    if constexpr (F16) nF = __uint_as_float(lds32v(bars + kFAt + 4 * st));
                    if (j == 0) {
                        m = top - below;
                    } else {
                        const bool up = top > m + (kLazy + below);
                        if (__any_sync(kLanes, up || nF != F)) {
                            float f = F / nF;
                            if (nF == F) f = 1.f;
                            if (up) {
                                const float e = ex2(m - (top - below));
                                m = top - below;
                                l *= e;
                                f *= e;
                            }
                            rescale(tO, f);
                        }
                    }
                    F = nF;
                    float2 la = make_float2(0.f, 0.f), lb = make_float2(0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t p[16];
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            fma2(s[k][i], s[k][i + 1], w.c, -m);
                            fma2(s[k][i + 2], s[k][i + 3], w.c, -m);
                            float2 x, y;
                            x.x = ex2(__uint_as_float(s[k][i]));
                            x.y = ex2(__uint_as_float(s[k][i + 1]));
                            y.x = ex2(__uint_as_float(s[k][i + 2]));
                            y.y = ex2(__uint_as_float(s[k][i + 3]));
                            add2(la, x);
                            add2(lb, y);
                            p[i / 2] = F16 ? pack_f16(x.x, x.y) : pack_bf16(x.x, x.y);
                            p[i / 2 + 1] = F16 ? pack_f16(y.x, y.y) : pack_bf16(y.x, y.y);
                        }
                        tmem_st16(tS + 16 * k, p);   // over S, which is in registers
                        if (k & 1) {   // the product of the first half runs while the second is computed
                            tmem_wait_st();
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(bars + (k == 1 ? kBarP : kBarP2) + 8 * tile);
                        }
                    }
                    l += (la.x + la.y) + (lb.x + lb.y);
                }
                if (F16) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bars + kScEmpty + 8 * st);
                }
            }
            if (!w.on) continue;
            if (!wait(bars + kBarO + 8 * tile, no++ & 1)) return;
            tc_fence_after();
            store_rows(u, tile, tO, w, m, l, l > 0.f ? F / l : 0.f);
            tc_fence_before();   // the next unit's products overwrite O once this warp's next P is announced
        }
    }

    // The same for drafted tokens, whose rows do not see every token.  In few instructions: 64 tokens at a time in a rolled loop,
    // in place of a whole row in registers and straight code.  The reference may move before the second half too, whose weights
    // then wait for the first half's product, since O counts from it.  The code of all roles of an SM has to fit its instruction
    // cache: with the straight code 21 % of the fp8 kernel's requests missed it, and a step of few rows took 2.0 us, half of it
    // without an instruction.
    __device__ __forceinline__ void softmax_tree(uint32_t tmem_base, int tile) {
        const int r = threadIdx.x & 127, lane = threadIdx.x & 31;
        const uint32_t lanes = (uint32_t)(r & ~31) << 16;
        const uint32_t tO = tmem_base + 256 + tile * 128 + lanes;
        constexpr float below = F16 ? kBelow : 0.f;
        unsigned own = 0, no = 0, np = 0;   // this tile's steps and units, and those of them with rows held twice
        unsigned step = 0, turn = 0;        // steps and turns of both tiles
        uint32_t s_ph = 0;                              // a bit per place
        Unit u;
        while (next(u)) {
            const bool both = active(u, 1);
            if (!both && (units & 1) != tile) {   // the other tile's
                step += u.steps;
                turn += u.steps;
                continue;
            }
            const Rows w = start_unit(u, tile, r);
            const int releases = both ? 1 : 2;
            const bool part = halves(u), idle = first_row(u, tile) + (r & (part ? 32 : 96)) >= u.rows;   // no row of the warp's
            const int k0 = part ? r >> 6 : 0, k1 = part ? k0 + 1 : 2;
            const Sight x = sight(u);
            float m = 0.f, l = 0.f, F = 1.f;   // m: the reference, which l and O count from
            if (both) turn = tile;
            for (int j = 0; j < u.steps; ++j, ++own) {
                const unsigned st = step % Cfg::kScales, place = turn & 1;
                const uint32_t sc = sm + Cfg::kOffScales + st * Cfg::kScaleBytes, tS = tmem_base + place * 128 + lanes;
                const int t0 = step_of(u, x, j) * kStep;
                // a unit's first comes when all before it are through
                const uint32_t bar = bars + (place ? kBarS2 : kBarS) + 8 * tile, ph = s_ph >> place & 1;
                if (!(j == 0 ? wait_unit(bar, ph) : wait(bar, ph))) return;
                s_ph ^= 1u << place;
                // only now: the other tile may have had the steps between, and S says that they are through
                if (F16 && !wait(bars + kScFull + 8 * st, step / Cfg::kScales & 1)) return;
                ++step;
                turn += both ? 2 : 1;
                tc_fence_after();
                if (!idle) {
                    // only the steps with drafted tokens and those where some row's window starts are looked at bit by bit
                    const bool hidden = t0 + kStep > x.ctx || (a.window > 0 && t0 < u.len - a.window && t0 + kStep > a.num_first);
                    if (hidden) hide(u, w, x, t0, tS, sc, 4 * k0, 4 * k1);
                    float nF = 1.f;
                    if constexpr (F16) nF = __uint_as_float(lds32v(bars + kFAt + 4 * st));
                    float f = nF == F ? 1.f : F / nF;   // what O is to be multiplied by
                    F = nF;
#pragma unroll 1
                    for (int k = k0; k < k1; ++k) {   // 64 tokens
                        uint32_t s[2][32];
                        read_scores(s, tS, 64 * k, sc, hidden);
                        float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                t[c] = fmaxf(t[c], fmaxf(__uint_as_float(s[c][i]), __uint_as_float(s[c][i + 1])));
                                t[c + 2] = fmaxf(t[c + 2], fmaxf(__uint_as_float(s[c][i + 2]), __uint_as_float(s[c][i + 3])));
                            }
                        const float top = fmaxf(fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * w.c, -1e30f);
                        if (j == 0 && k == k0) {
                            m = top - below;
                            f = 1.f;
                        }
                        const bool up = top > m + (kLazy + below);
                        if (__any_sync(kLanes, up || f != 1.f)) {
                            if (up) {
                                const float e = ex2(m - (top - below));
                                m = top - below;
                                l *= e;
                                f *= e;
                            }
                            if (j > 0 || k > k0) {   // the last step's product may be under way, and that of this one's first half
                                if (j > 0 && !wait(bars + kBarWhole + 8 * tile, own - 1 & 1)) return;
                                if (k > k0 && !wait(bars + kBarHalf + 8 * tile, own & 1)) return;
                                tc_fence_after();
                                rescale(tO, f);
                            }
                            f = 1.f;
                        }
                        float2 la = make_float2(0.f, 0.f), lb = make_float2(0.f, 0.f);
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            uint32_t p[16];
#pragma unroll
                            for (int i = 0; i < 32; i += 4) {
                                fma2(s[c][i], s[c][i + 1], w.c, -m);
                                fma2(s[c][i + 2], s[c][i + 3], w.c, -m);
                                float2 y, z;
                                y.x = ex2(__uint_as_float(s[c][i]));
                                y.y = ex2(__uint_as_float(s[c][i + 1]));
                                z.x = ex2(__uint_as_float(s[c][i + 2]));
                                z.y = ex2(__uint_as_float(s[c][i + 3]));
                                add2(la, y);
                                add2(lb, z);
                                p[i / 2] = F16 ? pack_f16(y.x, y.y) : pack_bf16(y.x, y.y);
                                p[i / 2 + 1] = F16 ? pack_f16(z.x, z.y) : pack_bf16(z.x, z.y);
                            }
                            tmem_st16(tS + 32 * k + 16 * c, p);   // over S of the first 64 tokens, which has been read
                        }
                        if (part) {   // no weights for the other half
                            uint32_t p[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) p[i] = 0u;
                            tmem_st16(tS + 32 * (1 - k), p);
                            tmem_st16(tS + 32 * (1 - k) + 16, p);
                        }
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            if (part || k == 0) mbar_arrive(bars + kBarP + 8 * place);
                            if (part || k == 1) mbar_arrive(bars + kBarP2 + 8 * place);
                        }
                        l += (la.x + la.y) + (lb.x + lb.y);
                    }
                } else if (lane == 0) {   // its rows of P are whatever S was, and make rows of O that are nobody's
                    mbar_arrive(bars + kBarP + 8 * place);
                    mbar_arrive(bars + kBarP2 + 8 * place);
                }
                if (F16) {
                    __syncwarp();
                    if (lane == 0)
                        for (int k = 0; k < releases; ++k) mbar_arrive(bars + kScEmpty + 8 * st);
                }
            }
            if (both) turn = 0;
            if (!wait(bars + kBarO + 8 * tile, no++ & 1)) return;
            tc_fence_after();
            if (!idle) {
                const uint32_t mine = 8 * (4 * tile + (r >> 5)), other = mine ^ 16;
                if (part) {
                    hand_over(tile, k0, tO, m, l, F);
                    if (lane == 0) mbar_arrive(bars + kBarPairFull + mine);
                    if (!wait(bars + kBarPairFull + other, np & 1)) return;
                }
                store_tree(u, tile, part, k0, tO, w, m, l, F);
                if (part) {   // the other's next rows come to where this warp's were handed over
                    if (lane == 0) mbar_arrive(bars + kBarPairEmpty + mine);
                    if (!wait(bars + kBarPairEmpty + other, np++ & 1)) return;
                }
            }
            tc_fence_before();   // the next unit's products overwrite O once this warp's next P is announced
        }
    }
    // Rows that are there twice: each of the two warps stores one half of the columns.  A warp gives the other's half of its rows of
    // O, counted from its reference and in units of its F, and (m, l), through its own rows' places in the query operand (no product
    // reads them any more).
    __device__ __forceinline__ uint32_t place(int tile, int r, int c) const {   // 16 bytes c of the 256 of row r
        return sm + Cfg::kOffQ + tile * kSlotBytes + (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
    }
    __device__ __forceinline__ void hand_over(int tile, int k0, uint32_t tO, float m, float l, float F) const {
        const int r = threadIdx.x & 127;
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
            uint32_t o[32];
            tmem_ld32(o, tO + 64 * (1 - k0) + 32 * k);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float f = l > 0.f ? F : 0.f;
                const uint32_t* x = o + 4 * i;
                sts128(place(tile, r, 8 * k + i), __float_as_uint(__uint_as_float(x[0]) * f), __float_as_uint(__uint_as_float(x[1]) * f),
                       __float_as_uint(__uint_as_float(x[2]) * f), __float_as_uint(__uint_as_float(x[3]) * f));
            }
        }
        const uint32_t at = sm + Cfg::kOffPair + (tile * 128 + r) * 8;
        sts32v(at, __float_as_uint(m));
        sts32v(at + 4, __float_as_uint(l));
        __syncwarp();
    }
    // The K scales of 16 tokens from `first` on (a multiple of 16): Q8: where the copies put them.
    __device__ __forceinline__ uint32_t key_scales(uint32_t sc, int first) const { return Q8 ? scale_at(sc, first, 0) : sc + first * 4; }
    // 64 columns of S, times their K scales unless they carry them already.
    __device__ __forceinline__ void read_scores(uint32_t (&s)[2][32], uint32_t tS, int first, uint32_t sc, bool scaled) const {
        tmem_ld32(s[0], tS + first);
        tmem_ld32(s[1], tS + first + 32);
        tmem_wait_ld();
        if (F16 && !scaled) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t f[16];
#pragma unroll
                for (int i = 0; i < 16; i += 4) lds128(key_scales(sc, first + 16 * k) + 4 * i, f[i], f[i + 1], f[i + 2], f[i + 3]);
#pragma unroll
                for (int i = 0; i < 16; i += 2) mul2(s[k >> 1][(k & 1) * 16 + i], s[k >> 1][(k & 1) * 16 + i + 1], f[i], f[i + 1]);
            }
        }
    }
    // A step's S times its K scales, and -inf where the row does not see the token (whatever stands there: the choice comes last).
    __device__ __forceinline__ void hide(const Unit& u, const Rows& w, const Sight& x, int t0, uint32_t tS, uint32_t sc, int k0, int k1) const {
#pragma unroll 1
        for (int k = k0; k < k1; ++k) {   // 16 tokens
            const uint32_t see = visible(u, w, x, t0 + 16 * k);
            uint32_t s[16];
            tmem_ld16(s, tS + 16 * k);
            tmem_wait_ld();
            if constexpr (F16) {
                uint32_t f[16];
#pragma unroll
                for (int i = 0; i < 16; i += 4) lds128(key_scales(sc, 16 * k) + 4 * i, f[i], f[i + 1], f[i + 2], f[i + 3]);
#pragma unroll
                for (int i = 0; i < 16; i += 2) mul2(s[i], s[i + 1], f[i], f[i + 1]);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (!(see >> i & 1u)) s[i] = 0xFF800000u;
            tmem_st16(tS + 16 * k, s);
        }
        tmem_wait_st();
    }
    // The rows that no unit holds: of a sequence in error zeros, of nobody what is there.  The join leaves rows of one piece alone.
    __device__ void settle() const {
        const int lane = threadIdx.x & 31, row = a.Hk * a.QG;
        const int first = __ldcg(a.group_starts), last = __ldcg(a.group_starts + a.NG);
        for (long long i = (long long)blockIdx.x * 32 + lane; i < (long long)(first + a.B - last) * row; i += gridDim.x * 32)
            a.pieces[i < (long long)first * row ? i : i + (long long)(last - first) * row] = 1;
        for (int g = blockIdx.x; g < a.NG; g += gridDim.x) {
            const int s0 = __ldcg(a.group_starts + g), s1 = __ldcg(a.group_starts + g + 1), ctx = __ldcg(a.prefix_lens + g);
            if (ctx >= 0 && ctx <= a.MP * a.BS && s1 - s0 <= a.MP * a.BS - ctx) continue;
            const long long r0 = (long long)s0 * row, n = (long long)(s1 - s0) * row;
            for (long long i = lane; i < n; i += 32) a.pieces[r0 + i] = 1;
            uint4* out = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + r0 * kHeadDim * (a.out_f32 ? 4 : 2));
            for (long long i = lane; i < n * (a.out_f32 ? 32 : 16); i += 32) out[i] = make_uint4(0, 0, 0, 0);
        }
    }

    // The warp's 32 rows of O, times inv, to the partials.  A thread holds a row, and storing rows from
    // there would touch 32 lines per instruction; each half (64 columns) goes through the warp's own rows of
    // its tile's query operand, which no product reads any more, and out two rows per instruction.
    __device__ __forceinline__ void store_rows(const Unit& u, int tile, uint32_t tO, const Rows& w, float m, float l,
                                               float inv) const {
        const int lane = threadIdx.x & 31, r0 = threadIdx.x & 96;
        const uint32_t stage = sm + Cfg::kOffQ + tile * kSlotBytes + r0 * 128;
        auto at = [&](int r, int c) {   // 16 bytes c of the half row r
            return stage + (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
        };
        const int row0 = u.rt * kUnitRows + tile * kTileRows + r0;
        const int rows = min(32, u.rows - row0);   // may be negative
        const long long mine = (w.head * a.slots + u.slot) * a.QG + w.q;
        if (w.live) {
            a.part_l[mine] = l;
            a.part_m[mine] = m * kLn2S;
            if (u.slot == 0) a.pieces[w.head * a.QG + w.q] = u.pieces;
        }
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
            uint32_t s[2][32];
            tmem_ld32(s[0], tO + 64 * half);
            tmem_ld32(s[1], tO + 64 * half + 32);
            tmem_wait_ld();
            __syncwarp();
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                const uint32_t* x = &s[c >> 3][(c & 7) * 4];
                sts128(at(lane, c), __float_as_uint(__uint_as_float(x[0]) * inv),
                       __float_as_uint(__uint_as_float(x[1]) * inv), __float_as_uint(__uint_as_float(x[2]) * inv),
                       __float_as_uint(__uint_as_float(x[3]) * inv));
            }
            __syncwarp();
            const int c = lane & 15;
#pragma unroll 4
            for (int i = 0; i < 16; ++i) {
                const int r = 2 * i + (lane >> 4);
                const long long dst = __shfl_sync(kLanes, mine, r);
                uint32_t v0, v1, v2, v3;
                lds128(at(r, c), v0, v1, v2, v3);
                if (r < rows)
                    *reinterpret_cast<uint4*>(a.part_o + dst * kHeadDim + 64 * half + 4 * c) = make_uint4(v0, v1, v2, v3);
            }
        }
        __syncwarp();   // the next unit's query rows are written by other lanes
    }
    // TREE: the same, over l, to the partials or to a result of one piece; of rows that are there twice one half of the columns,
    // with what the other warp has handed over.
    __device__ __forceinline__ void store_tree(const Unit& u, int tile, bool part, int k0, uint32_t tO, const Rows& w, float m, float l,
                                               float F) const {
        const int lane = threadIdx.x & 31, r0 = part ? threadIdx.x & 32 : threadIdx.x & 96;
        const int from = (threadIdx.x & 96) ^ (part ? 64 : 0);   // rows whose places are used
        const int rows = min(32, u.rows - (first_row(u, tile) + r0));
        const bool whole = u.pieces == 1, bf16 = whole && !a.out_f32;
        const long long row = w.head * a.QG + w.q, mine = whole ? row : (w.head * a.slots + u.slot) * a.QG + w.q;
        float* const to = whole ? static_cast<float*>(a.out) : a.part_o;
        float f0 = l > 0.f ? F : 0.f, f1 = 0.f;
        if (part) {
            const uint32_t at = sm + Cfg::kOffPair + (tile * 128 + from + lane) * 8;
            const float m1 = __uint_as_float(lds32v(at)), l1 = __uint_as_float(lds32v(at + 4));
            const float M = l > 0.f && !(l1 > 0.f && m1 > m) ? m : m1;   // the larger of those that count
            const float e = l > 0.f ? ex2(m - M) : 0.f;
            f1 = l1 > 0.f ? ex2(m1 - M) : 0.f;
            f0 *= e;
            l = k0 ? l1 * f1 + l * e : l * e + l1 * f1;
            m = M;
        }
        const float inv = l > 0.f ? 1.f / l : 0.f;   // a row that sees nothing gives zeros
        f0 *= inv;
        f1 *= inv;
        if (w.live && !k0) {
            if (u.slot == 0) a.pieces[row] = u.pieces;
            if (!whole) {
                a.part_l[mine] = l;
                a.part_m[mine] = m * kLn2S;
            }
        }
#pragma unroll 1
        for (int half = part ? k0 : 0; half < (part ? k0 + 1 : 2); ++half) {
#pragma unroll 1
            for (int q = 0; q < 2; ++q) {   // 32 columns
                uint32_t s[32];
                tmem_ld32(s, tO + 64 * half + 32 * q);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) s[i] = __float_as_uint(__uint_as_float(s[i]) * f0);
                if (part) {
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        uint32_t v[4];
                        lds128(place(tile, from + lane, 8 * q + c), v[0], v[1], v[2], v[3]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) s[4 * c + i] = __float_as_uint(fmaf(__uint_as_float(v[i]), f1, __uint_as_float(s[4 * c + i])));
                    }
                }
#pragma unroll
                for (int c = 0; c < 8; ++c) sts128(place(tile, from + lane, 8 * q + c), s[4 * c], s[4 * c + 1], s[4 * c + 2], s[4 * c + 3]);
            }
            __syncwarp();
            if (bf16) {
                const int c = lane & 7;   // four rows, 16 bytes per lane
#pragma unroll 2
                for (int i = 0; i < 8; ++i) {
                    const int r = 4 * i + (lane >> 3);
                    const long long dst = __shfl_sync(kLanes, mine, r);
                    uint32_t v[8];
                    lds128(place(tile, from + r, 2 * c), v[0], v[1], v[2], v[3]);
                    lds128(place(tile, from + r, 2 * c + 1), v[4], v[5], v[6], v[7]);
                    if (r >= rows) continue;
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] = pack_bf16(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1]));
                    uint16_t* const p = static_cast<uint16_t*>(a.out) + dst * kHeadDim + 64 * half + 8 * c;
                    *reinterpret_cast<uint4*>(p) = make_uint4(v[0], v[1], v[2], v[3]);
                }
            } else {
                const int c = lane & 15;
#pragma unroll 4
                for (int i = 0; i < 16; ++i) {
                    const int r = 2 * i + (lane >> 4);
                    const long long dst = __shfl_sync(kLanes, mine, r);
                    uint32_t v[4];
                    lds128(place(tile, from + r, c), v[0], v[1], v[2], v[3]);
                    if (r < rows) *reinterpret_cast<uint4*>(to + dst * kHeadDim + 64 * half + 4 * c) = make_uint4(v[0], v[1], v[2], v[3]);
                }
            }
        }
        __syncwarp();   // the next unit's query rows are written by other lanes
    }
    // O *= f, one row per thread (rare; few registers, since S is held meanwhile).
    static __device__ __forceinline__ void rescale(uint32_t tO, float f) {
#pragma unroll 1
        for (int k = 0; k < 8; ++k) {
            uint32_t o[16];
            tmem_ld16(o, tO + 16 * k);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st16(tO + 16 * k, o);
        }
        tmem_wait_st();
    }
};

template <int KV, class Args>
__global__ void __launch_bounds__(SharedCfg<KV, Args>::kThreads, 1)
    pda_prefix_kernel(const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ CUtensorMap sc_map,
                      const Args a) {
    using Cfg = SharedCfg<KV, Args>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sm = smem_addr(smem);
    const uint32_t bars = sm + Cfg::kOffBars;
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < Cfg::kSlots; ++i) {
            mbar_init(bars + kBarFull + 8 * i, Cfg::kF16 && !Cfg::kQ8 ? kConvertWarps : 1);
            mbar_init(bars + kBarEmpty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bars + kBarQ + 8 * i, 4);
            mbar_init(bars + kBarS + 8 * i, 1);
            mbar_init(bars + kBarP + 8 * i, 4);
            mbar_init(bars + kBarP2 + 8 * i, 4);
            mbar_init(bars + kBarO + 8 * i, 1);
            if (Cfg::kTree) {
                mbar_init(bars + kBarHalf + 8 * i, 1);
                mbar_init(bars + kBarWhole + 8 * i, 1);
                mbar_init(bars + kBarS2 + 8 * i, 1);
                for (int k = 0; k < 4; ++k) {
                    mbar_init(bars + kBarPairFull + 32 * i + 8 * k, 1);
                    mbar_init(bars + kBarPairEmpty + 32 * i + 8 * k, 1);
                }
            }
        }
        for (int i = 0; i < 3; ++i) {
            mbar_init(bars + kBarRawFull + 8 * i, 1);
            mbar_init(bars + kBarRawEmpty + 8 * i, kConvertWarps);
            mbar_init(bars + kBarScRaw + 8 * i, 1);
            mbar_init(bars + kBarScFull + 8 * i, 1);
            mbar_init(bars + kBarScEmpty + 8 * i, 8);
            if (Cfg::kQ8) {
                mbar_init(bars + kBarVFull + 8 * i, kConvertWarps / 2);   // of 64 tokens
                mbar_init(bars + kBarVEmpty + 8 * i, 1);
            }
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bars + kBarUnitFull + 8 * i, 1);
            mbar_init(bars + kBarUnitEmpty + 8 * i, Cfg::kReaders);
        }
        if (Cfg::kQ8)
            for (int i = 0; i < 4; ++i) {
                mbar_init(bars + kBarScRaw8 + 8 * i, 32);
                mbar_init(bars + kBarScFull8 + 8 * i, 1);
                mbar_init(bars + kBarScEmpty8 + 8 * i, 8 + kConvertWarps);
            }
        mbar_init(bars + kBarDrain, 1);
        sts32v(bars + kAbortAt, (sm & 1023u) ? 1u : 0u);   // the operands' swizzle needs the alignment
        fence_mbar_init();
        prefetch_tensormap(&kv_map);
        if (Cfg::kF16) prefetch_tensormap(&sc_map);
    }
    // Behind the pass over the sequences' own tokens there is no wait for it here: every CTA of that pass has waited for
    // everything before the step before it lets this grid start, and nothing of its own is read.  What was written
    // before the step lies in L2 then, and every read of it in this grid goes there (ld.cg, cp.async.cg, TMA): a line
    // that an earlier grid left in this SM's L1 is not looked at.
    if (a.first) grid_dependency_wait();
    Prefix<KV, Args> p(a, sm);
    SplitBy<Args::kSwitchSteps> split;
    Unit first;
    int at, end;
    if (warp == 11) {
        split = make_split(a, gridDim.x, blockIdx.x == 0);
        if constexpr (std::is_same<Args, TreeArgs>::value)
            if (blockIdx.x == 0 && (threadIdx.x & 31) == 0) *a.refused = split.refused;
        at = (int)min((long long)blockIdx.x * split.per, (long long)split.total);
        end = at + min(split.per, split.total - at);
        if constexpr (!Cfg::kTree) {
            first = find_unit(a, split, at, end);
            p.put(first);
        }
    }
    if constexpr (Cfg::kTq) {
        if (warp == 12) p.make_table();
    }
    if (warp == 9) tmem_alloc(bars + kTmemAt, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = lds32v(bars + kTmemAt);
    allow_dependent_launch();
    // registers at launch: 384 x 168 = 64512 = 256 x 200 + 128 x 104; 512 x 128 = 65536 = 256 x 192 + 256 x 64, of drafted tokens
    // 256 x 160 + 256 x 96
    const bool fine = lds32v(bars + kAbortAt) == 0u;
    if (warp < 8) {
        if constexpr (Cfg::kTree && Cfg::kF16)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
        else if constexpr (Cfg::kF16)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        else
            asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        if (fine) {
            if constexpr (Cfg::kTree)
                p.softmax_tree(tmem, warp >> 2);
            else
                p.softmax(tmem, warp >> 2);
        }
    } else {
        if constexpr (Cfg::kTree && Cfg::kF16)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
        else if constexpr (Cfg::kF16)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        else
            asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        if (fine) {
            // The conversion first: where its code lies decides over a tenth of an fp8 step (64 sequences of 4 drafted tokens over 4096
            // tokens 156 us, in the warps' order 174; TQ4 258 and 273), since the code is larger than the instruction cache.
            if (Cfg::kF16 && warp >= 12)
                p.convert();
            else if (warp == 8 || (Cfg::kTree && !Cfg::kTq && warp == 10)) {
                if constexpr (Cfg::kTree)
                    p.copies_tree(&kv_map, &sc_map, warp == 10);
                else
                    p.copies(&kv_map, &sc_map);
            }
            else if (warp == 9)
                p.products(tmem);
            else if (warp == 11) {
                if constexpr (Cfg::kTree)
                    p.give_all(split, at, end);
                else
                    p.give(split, first, at, end);
                if constexpr (Cfg::kTree)
                    if (!split.refused) p.settle();
            }
            else if (Cfg::kF16 && !Cfg::kQ8 && warp == 10)
                p.scales();
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x == 0 && lds32v(bars + kAbortAt) && a.err_word) atomicOr(a.err_word, PDA_ERRW_PIPELINE_TIMEOUT);
    if (warp == 9) tmem_free(tmem, 512);
    grid_dependency_wait();   // behind the own pass this grid ends after it: the join waits for one grid alone
}

template <int KV, class Args>
static int launch_prefix(const Args& a, const CUtensorMap& kv_map, const CUtensorMap& sc_map, int ctas,
                         cudaStream_t stream) {
    using Cfg = SharedCfg<KV, Args>;
    static bool attr_set[64] = {false};
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PDA_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!attr_set[dev]) {
            if (cudaFuncSetAttribute(pda_prefix_kernel<KV, Args>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem) !=
                cudaSuccess)
                return PDA_ERR_LAUNCH;
            attr_set[dev] = true;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(Cfg::kThreads);
    cfg.dynamicSmemBytes = Cfg::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, pda_prefix_kernel<KV, Args>, kv_map, sc_map, a) == cudaSuccess ? PDA_OK : PDA_ERR_LAUNCH;
}

}  // namespace pda
