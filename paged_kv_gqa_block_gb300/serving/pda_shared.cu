// pda_shared.cu -- pda_decode_shared: a decode step for sequences that share prefixes in groups.
//
// For query row r of sequence b in group g,
//   out = softmax(scale [q.K_g ; q.K_b]) [V_g ; V_b],
// with K_g, V_g the group's prefix and K_b, V_b the sequence's own tokens.  The two parts are
// computed apart as (m, l, o), a reference near the maximum, the sum of exponentials from it and the normalised
// output, and joined: w = l e^(m - M), out = sum w o / sum w, M the largest m.  The own part is the cluster kernel of
// pda_selected.cuh.  The prefix part is one matrix product per group and KV head for the
// query rows of all its sequences, n_g * QG of them, and this file's first kernel.
//
// The prefix pass.  A CTA holds 256 query rows of one (group, KV head) in two tiles of 128 and walks
// the prefix in steps of 128 tokens: S = Q K^T and O += P V by tcgen05.mma (M = N = 128), S, P and
// O in tensor memory (two tiles x (128 + 128) columns = all 512; P, 16-bit, lies over the S it was
// made of).  Warps take one role each:
//   0-3, 4-7  softmax of tile 0, tile 1: one query row per thread, so a row's maximum and sum need
//             no shuffles; S is read from TMEM, P written back
//   8         copies: K and V blocks by TMA into a ring of shared-memory slots (32 KB each)
//   9         the matrix products (one thread issues)
//   10        fp8 only: the scales of a step
//   11        the split: which rows and which tokens this CTA takes
//   12-15     fp8 only: e4m3 codes to f16 between the copy and the product
// The softmax warps hold a whole row of S (128 registers); the other warps give registers up for them.
// The products are issued in the order PV(0, j), QK(0, j+1), PV(1, j), QK(1, j+1): while one tile's
// softmax runs the tensor cores work for the other.  A tile's reference point m moves only when a
// row's maximum passes it by 2^8 (log2 units 8), so the rescale of O, the one read-modify-write of
// TMEM, is rare; a reference below the true maximum leaves the quotient as it is.
// P is announced in halves, so that PV starts while the second half is computed.
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
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

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
constexpr int kScaleBytes = 1024;          // 128 tokens x {K scale, V scale}
constexpr float kLog2eS = 1.4426950408889634f, kLn2S = 0.6931471805599453f;
constexpr float kLazy = 8.f;               // log2 units that a row's maximum may rise before its reference follows
constexpr float kBelow = 7.f;              // f16 P: the reference below the maximum

template <int KV>
struct SharedCfg {
    static constexpr bool kF16 = KV != PDA_KV_BF16;              // f16 products, converter warps
    static constexpr int kSlots = kF16 ? 3 : 5;
    static constexpr int kRaw = 3, kScales = 3;                  // fp8: raw slots, scale stages
    static constexpr int kThreads = kF16 ? 512 : 384;
    static constexpr int kOffQ = 0;                               // 2 tiles x 32 KB
    static constexpr int kOffSlots = 2 * kSlotBytes;
    static constexpr int kOffRaw = kOffSlots + kSlots * kSlotBytes;
    static constexpr int kOffScales = kOffRaw + (kF16 ? kRaw * kRawBytes : 0);
    static constexpr int kOffBars = kOffScales + (kF16 ? kScales * kScaleBytes : 0);
    static constexpr int kSmem = kOffBars + 448;
    static constexpr int kReaders = kF16 ? 15 : 10;               // warps that take units
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
    kFAt = 256,          // [3] what a step's V scales are divided by
    kBarP2 = 272,        // [2] the second half of P is in TMEM
    kBarScRaw = 288,     // [3] scales as copied
    kBarUnitFull = 312,  // [2] the next unit is in shared memory
    kBarUnitEmpty = 328, // [2]
    kUnitAt = 352        // [2] units, 48 bytes each
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

template <int KV>
struct Prefix {
    using Cfg = SharedCfg<KV>;
    static constexpr bool F16 = Cfg::kF16;
    static constexpr uint32_t kIdescQK = umma_idesc(!F16, false, 128, 128), kIdescPV = umma_idesc(!F16, true, 128, 128);

    const SharedArgs& a;
    const uint32_t sm;         // shared memory base
    const uint32_t bars;
    unsigned units = 0;        // units taken (or given) by this warp
    unsigned busy = 0;         // their steps

    __device__ __forceinline__ Prefix(const SharedArgs& args, uint32_t base)
        : a(args), sm(base), bars(base + Cfg::kOffBars) {}

    // A whole warp waits (bounded).  False once any wait of the CTA has given up.
    __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) const {
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
            sts128(at + 32, u.rot, u.slot, u.pieces, 0);
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
    __device__ __forceinline__ bool next(Unit& u) {
        const uint32_t slot = units & 1, at = bars + kUnitAt + slot * 48;
        if (!wait_unit(bars + kBarUnitFull + 8 * slot, units >> 1 & 1)) return false;
        uint32_t x[12];
#pragma unroll
        for (int i = 0; i < 12; i += 4) lds128(at + 4 * i, x[i], x[i + 1], x[i + 2], x[i + 3]);
        u.g = x[0], u.h = x[1], u.rt = x[2], u.seq0 = x[3], u.rows = x[4], u.len = x[5], u.step0 = x[6], u.steps = x[7];
        u.rot = x[8], u.slot = x[9], u.pieces = x[10];
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(bars + kBarUnitEmpty + 8 * slot);
        ++units;
        busy += u.steps;
        return u.steps > 0;
    }
    // Step number of the piece's j-th step, and its tokens.
    __device__ __forceinline__ static int step_of(const Unit& u, int j) {
        const int i = j + u.rot;
        return u.step0 + (i < u.steps ? i : i - u.steps);
    }
    __device__ __forceinline__ static int tokens_of(const Unit& u, int j) {
        return min(kStep, u.len - step_of(u, j) * kStep);
    }
    __device__ __forceinline__ static bool active(const Unit& u, int tile) {
        return u.rt * kUnitRows + tile * kTileRows < u.rows;
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
            const uint64_t policy = u.rows > kUnitRows ? again : once;   // other row tiles read it too
            const int* table = a.prefix_table + (long long)u.g * a.MP;
            const int last = (u.len + a.BS - 1) / a.BS;   // blocks of the prefix
            int id = 0;
            int b0 = step_of(u, 0) * nblk;
            if (blk < nblk && b0 + blk < last) id = __ldcg(table + b0 + blk);
            for (int j = 0; ok && j < u.steps; ++j, ++step) {
                const int n = min(nblk, last - b0);
                const bool mine = blk < n;
                int nid = 0, b1 = 0;
                if (j + 1 < u.steps) {
                    b1 = step_of(u, j + 1) * nblk;
                    if (blk < nblk && b1 + blk < last) nid = __ldcg(table + b1 + blk);
                }
                if (mine && half == 0 && (id < 0 || id >= a.num_cache_blocks) && a.err_word)
                    atomicOr(a.err_word, PDA_ERRW_BAD_BLOCK_ID);
                const unsigned st = step % Cfg::kScales;
                if (F16 && step >= Cfg::kScales && !wait(bars + kBarScEmpty + 8 * st, (step / Cfg::kScales - 1) & 1)) {
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
                        if (scales) mbar_arrive_expect_tx(bars + kBarScRaw + 8 * st, (uint32_t)n * a.BS * 8u);
                        mbar_arrive_expect_tx(bar, row_bytes);
                    }
                    __syncwarp();
                    if (mine) {
                        tma_load_5d(base + s * kBytes + half * 16384 + blk * a.BS * 128, kv_map, bar, 0, 0,
                                    v * kHalves + half, u.h, id, policy);
                        if (scales)
                            tma_load_4d(sm + Cfg::kOffScales + st * kScaleBytes + blk * a.BS * 8, sc_map,
                                        bars + kBarScRaw + 8 * st, 0, 0, u.h, id, policy);
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
                    (void)mbar_wait(bars + kBarScRaw + 8 * s, (issued - 1 - s) / Cfg::kScales & 1, kDefaultTimeoutNs);
        }
    }

    // ---------------------------------------------------------------- conversion (fp8)
    // One warp lays a step's scales out as [128 K scales][128 V scales / F]: the K scales for the softmax, the
    // others for the conversion.  F keeps V in f16's range (the accumulator counts in units of F): 16 F is the
    // step's largest V scale f, and F stays as it is while f lies in [2F, 128F].  So the largest products stay
    // below 448 * 128 = 57344, and a scale keeps its 11 bits down to 2^-15 f (2 F * 2^-15 = 2^-14 F).
    __device__ void scales() {
        const int lane = threadIdx.x & 31;
        unsigned st = 0, ph = 0;
        float F = 1.f;
        Unit u;
        while (next(u)) {
            for (int j = 0; j < u.steps; ++j) {
                const int valid = tokens_of(u, j);
                if (!wait(bars + kBarScRaw + 8 * st, ph)) return;
                const uint32_t sc = sm + Cfg::kOffScales + st * kScaleBytes;
                float ks[4], vs[4], f = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int tok = lane + 32 * i;
                    ks[i] = tok < valid ? __uint_as_float(lds32v(scale_at(sc, tok, 0))) : 0.f;
                    vs[i] = tok < valid ? __uint_as_float(lds32v(scale_at(sc, tok, 1))) : 0.f;
                    f = fmaxf(f, fabsf(vs[i]));
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) f = fmaxf(f, __shfl_xor_sync(kLanes, f, o));
                if (!(f > 0.f)) f = 1.f;
                if (j == 0 || f > F * 128.f || f < F * 2.f) F = fmaxf(f * 0.0625f, 1e-37f);   // 1 / F is finite
                const float rF = 1.f / F;
#pragma unroll
                for (int i = 0; i < 4; ++i) {   // the shuffles above come after every lane's reads
                    sts32v(sc + (lane + 32 * i) * 4, __float_as_uint(ks[i]));
                    sts32v(sc + 512 + (lane + 32 * i) * 4, __float_as_uint(vs[i] * rF));
                }
                if (lane == 0) sts32v(bars + kFAt + 4 * st, __float_as_uint(F));
                fence_proxy_async_shared();   // the next copy into this stage comes after these stores
                __syncwarp();
                if (lane == 0) mbar_arrive(bars + kBarScFull + 8 * st);
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
        const int t = threadIdx.x - 384, lane = t & 31, x = t & 7;
        const uint32_t raw0 = sm + Cfg::kOffRaw + t * 128, slot0 = sm + Cfg::kOffSlots + t * 128;
        const uint32_t scale0 = sm + Cfg::kOffScales + 512 + t * 4;
        static_assert(!F16 || Cfg::kRaw == Cfg::kSlots, "a raw slot and its slot are counted together");
        unsigned s = 0, ph = 0, st = 0, st_ph = 0;
        Unit u;
        while (next(u)) {
            for (int j = 0; j < u.steps; ++j) {
                const bool zero = t >= tokens_of(u, j);
#pragma unroll 1
                for (int v = 0; v < 2; ++v) {
                    if (!wait(bars + kBarRawFull + 8 * s, ph)) return;
                    const uint32_t src = raw0 + s * kRawBytes, dst = slot0 + s * kSlotBytes;
                    uint32_t w[8][4];
#pragma unroll
                    for (int c = 0; c < 8; ++c) lds128(src + ((c ^ x) << 4), w[c][0], w[c][1], w[c][2], w[c][3]);
                    float vs = 1.f;
                    if (v) {
                        if (!wait(bars + kBarScFull + 8 * st, st_ph)) return;
                        vs = __uint_as_float(lds32v(scale0 + st * kScaleBytes));
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
                        sts128(d + ((k ^ x) << 4), o[0], o[1], o[2], o[3]);
                        sts128(d + (((k + 1) ^ x) << 4), o[4], o[5], o[6], o[7]);
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
        // products in flight read shared memory and TMEM: let them end, whichever role gave up
        umma_commit(leader, bar + kBarDrain);
        __syncwarp();
        (void)mbar_wait(bars + kBarDrain, 0, kDefaultTimeoutNs);
    }

    // ---------------------------------------------------------------- softmax
    // The warp's 32 query rows into its tile's operand, two rows (16 lanes each) per asynchronous copy; returns
    // the factor from S to log2 units of this lane's own row, 32 * (warp % 4) + lane.  The loops stay
    // rolled: a short prefix waits for this code's first fetch longer than for its execution.
    __device__ __forceinline__ float load_q(const Unit& u, int tile) const {
        const int lane = threadIdx.x & 31, r0 = threadIdx.x & 96, half = lane >> 4, w = lane & 15;
        const uint32_t base = sm + Cfg::kOffQ + tile * kSlotBytes;
        {
            const uint32_t dst = base + (w >> 3) * 16384;
            const int row0 = u.rt * kUnitRows + tile * kTileRows + r0 + half;
            int seq = row0 / a.QG, q = row0 - seq * a.QG;
            const uint16_t* src = a.query + ((long long)(u.seq0 + seq) * a.Hk + u.h) * a.QG * kHeadDim + 8 * w;
            const long long skip = (long long)a.Hk * a.QG * kHeadDim;
#pragma unroll 2
            for (int i = 0; i < 16; ++i) {
                const int r = r0 + 2 * i + half;
                const bool live = row0 + 2 * i < u.rows;   // else: zeros, and no read
                cp_async16(dst + r * 128 + (((w & 7) ^ (r & 7)) << 4), live ? src + q * kHeadDim : a.query, live ? 16u : 0u);
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
        if constexpr (F16) {
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
    };
    __device__ __forceinline__ Rows start_unit(const Unit& u, int tile, int r) const {
        Rows w;
        w.on = active(u, tile);
        const int row = u.rt * kUnitRows + tile * kTileRows + r;
        w.live = row < u.rows;
        w.head = (long long)(u.seq0 + row / a.QG) * a.Hk + u.h;
        w.q = row % a.QG;
        w.c = 0.f;
        if (w.on) {   // every product with the last unit's rows has ended: their S was read
            w.c = load_q(u, tile);
            __syncwarp();
            if ((threadIdx.x & 31) == 0) mbar_arrive(bars + kBarQ + 8 * tile);
        }
        return w;
    }

    __device__ void softmax(uint32_t tmem_base, int tile) {
        const int r = threadIdx.x & 127, lane = threadIdx.x & 31;
        const uint32_t lanes = (uint32_t)(r & ~31) << 16;
        const uint32_t tS = tmem_base + tile * 128 + lanes, tO = tmem_base + 256 + tile * 128 + lanes;
        unsigned ns = 0, no = 0, step = 0;
        Unit u;
        while (next(u)) {
            const Rows w = start_unit(u, tile, r);
            constexpr float below = F16 ? kBelow : 0.f;
            float m = 0.f, l = 0.f, F = 1.f;   // m: the reference, which l and O count from
            for (int j = 0; j < u.steps; ++j, ++step) {
                const int valid = tokens_of(u, j);
                const unsigned st = step % Cfg::kScales;
                if (F16 && !wait(bars + kBarScFull + 8 * st, step / Cfg::kScales & 1)) return;
                if (w.on) {
                    if (!wait(bars + kBarS + 8 * tile, ns++ & 1)) return;
                    tc_fence_after();
                    uint32_t s[4][32];
#pragma unroll
                    for (int k = 0; k < 4; ++k) tmem_ld32(s[k], tS + 32 * k);
                    tmem_wait_ld();
                    if constexpr (F16) {   // the K scales
                        const uint32_t sc = sm + Cfg::kOffScales + st * kScaleBytes;
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
                    if (lane == 0) mbar_arrive(bars + kBarScEmpty + 8 * st);
                }
            }
            if (!w.on) continue;
            if (!wait(bars + kBarO + 8 * tile, no++ & 1)) return;
            tc_fence_after();
            store_partial(u, tile, tO, w, m, l, l > 0.f ? F / l : 0.f);
            tc_fence_before();   // the next unit's products overwrite O once this warp's next P is announced
        }
    }

    // The warp's 32 rows of O, times inv, to the partials.  A thread holds a row, and storing rows from
    // there would touch 32 lines per instruction; each half (64 columns) goes through the warp's own rows of
    // its tile's query operand, which no product reads any more, and out two rows per instruction.
    __device__ __forceinline__ void store_partial(const Unit& u, int tile, uint32_t tO, const Rows& w, float m, float l,
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

template <int KV>
__global__ void __launch_bounds__(SharedCfg<KV>::kThreads, 1)
    pda_prefix_kernel(const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ CUtensorMap sc_map,
                      const SharedArgs a) {
    using Cfg = SharedCfg<KV>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sm = smem_addr(smem);
    const uint32_t bars = sm + Cfg::kOffBars;
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < Cfg::kSlots; ++i) {
            mbar_init(bars + kBarFull + 8 * i, Cfg::kF16 ? kConvertWarps : 1);
            mbar_init(bars + kBarEmpty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bars + kBarQ + 8 * i, 4);
            mbar_init(bars + kBarS + 8 * i, 1);
            mbar_init(bars + kBarP + 8 * i, 4);
            mbar_init(bars + kBarP2 + 8 * i, 4);
            mbar_init(bars + kBarO + 8 * i, 1);
        }
        for (int i = 0; i < 3; ++i) {
            mbar_init(bars + kBarRawFull + 8 * i, 1);
            mbar_init(bars + kBarRawEmpty + 8 * i, kConvertWarps);
            mbar_init(bars + kBarScRaw + 8 * i, 1);
            mbar_init(bars + kBarScFull + 8 * i, 1);
            mbar_init(bars + kBarScEmpty + 8 * i, 8);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bars + kBarUnitFull + 8 * i, 1);
            mbar_init(bars + kBarUnitEmpty + 8 * i, Cfg::kReaders);
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
    Prefix<KV> p(a, sm);
    Split split;
    Unit first;
    int at, end;
    if (warp == 11) {
        split = make_split(a, gridDim.x, blockIdx.x == 0);
        at = (int)min((long long)blockIdx.x * split.per, (long long)split.total);
        end = at + min(split.per, split.total - at);
        first = find_unit(a, split, at, end);
        p.put(first);
    }
    if (warp == 9) tmem_alloc(bars + kTmemAt, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = lds32v(bars + kTmemAt);
    allow_dependent_launch();
    // registers at launch: 384 x 168 = 64512 = 256 x 200 + 128 x 104; 512 x 128 = 65536 = 256 x 192 + 256 x 64
    const bool fine = lds32v(bars + kAbortAt) == 0u;
    if (warp < 8) {
        if constexpr (Cfg::kF16)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        else
            asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        if (fine) p.softmax(tmem, warp >> 2);
    } else {
        if constexpr (Cfg::kF16)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        else
            asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        if (fine) {
            if (warp == 8)
                p.copies(&kv_map, &sc_map);
            else if (warp == 9)
                p.products(tmem);
            else if (warp == 11)
                p.give(split, first, at, end);
            else if (Cfg::kF16 && warp == 10)
                p.scales();
            else if (Cfg::kF16 && warp >= 12)
                p.convert();
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

// ------------------------------------------------------------------------- the join
struct JoinArgs {
    const int* group_starts;
    const int* prefix_lens;
    const int* context_lens;
    const float* part_o[2];   // prefix pieces [B][Hk][slots][QG][D]; own tokens [B][Hk][QG][D]
    const float* part_l[2];
    const float* part_m[2];
    const int* pieces;
    void* out;
    int B, NG, Hk, QG, MP, MB, BS, slots, out_f32;
};

// One CTA per (sequence, KV head), one warp per query row: lane i holds (m, l) of partials i, i + 32,
// ... of both parts, prefix pieces first; each lane then sums four dimensions over the partials in
// that order, eight loads in flight.  Bound by latency (a row's partials are a few KB, in L2): a call of 32
// sequences of 64 heads without prefixes or tokens, its three launches, takes 5.5 us.
__global__ void __launch_bounds__(512) pda_shared_join_kernel(const JoinArgs a) {
    grid_dependency_wait();
    const int b = blockIdx.x / a.Hk, lane = threadIdx.x & 31, q = threadIdx.x >> 5;
    const long long unit = blockIdx.x;
    // asked for at once, whether or not the sequence has a prefix (the row's entry is then not used)
    const int pieces = __ldg(a.pieces + unit * a.QG + q);
    int ctx = __ldg(a.context_lens + b);
    bool in = false, bad = false;   // as the prefix pass: one group that is not ascending, and there is no prefix
    for (int g = lane; g < a.NG; g += 32) {
        const int s0 = __ldg(a.group_starts + g), s1 = __ldg(a.group_starts + g + 1);
        const int len = __ldg(a.prefix_lens + g);
        bad |= s0 < 0 || s1 < s0 || s1 > a.B;
        in |= s0 <= b && b < s1 && len > 0 && len <= a.MP * a.BS;
    }
    const bool prefix = __any_sync(kLanes, in) && !__any_sync(kLanes, bad);
    const int np = prefix ? max(0, min(a.slots, pieces)) : 0;
    if (ctx < 0 || ctx > a.MB * a.BS) ctx = 0;   // reported by the own pass
    const int total = np + (ctx > 0 ? 1 : 0);
    const long long row0 = unit * a.slots * a.QG + q, row1 = unit * a.QG + q;
    auto at = [&](int i, int& part) {   // index of partial i's row in its part
        part = i >= np;
        return part ? row1 : row0 + (long long)i * a.QG;
    };
    auto stats = [&](int i, float& m, float& l) {
        m = -INFINITY;
        l = 0.f;
        if (i < total) {
            int part;
            const long long k = at(i, part);
            m = __ldcg((part ? a.part_m[1] : a.part_m[0]) + k);
            l = __ldcg((part ? a.part_l[1] : a.part_l[0]) + k);
        }
    };
    float m0, l0;   // of the first 32 partials
    stats(lane, m0, l0);
    float M = m0;
    for (int i = lane + 32; i < total; i += 32) {
        float m, l;
        stats(i, m, l);
        M = fmaxf(M, m);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kLanes, M, o));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    for (int i0 = 0; i0 < total; i0 += 32) {
        if (i0 > 0) stats(i0 + lane, m0, l0);
        const float w = i0 + lane < total ? partition_weight(l0, m0, M) : 0.f;
        sum += w;
        const int n = min(32, total - i0);
        for (int j0 = 0; j0 < n; j0 += 8) {
            float4 o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                int part;
                const long long k = at(i0 + min(j0 + j, n - 1), part);
                o[j] = __ldcg(reinterpret_cast<const float4*>((part ? a.part_o[1] : a.part_o[0]) + k * kHeadDim) + lane);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float f = __shfl_sync(kLanes, w, (j0 + j) & 31);
                if (j0 + j < n) {
                    acc.x = fmaf(f, o[j].x, acc.x);
                    acc.y = fmaf(f, o[j].y, acc.y);
                    acc.z = fmaf(f, o[j].z, acc.z);
                    acc.w = fmaf(f, o[j].w, acc.w);
                }
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kLanes, sum, o);
    const float inv = total > 0 ? 1.f / sum : 0.f;
    const long long orow = unit * a.QG + q;
    if (a.out_f32) {
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + orow * kHeadDim + 4 * lane) =
            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    } else {
        uint2 v;
        v.x = pack_bf16(acc.x * inv, acc.y * inv);
        v.y = pack_bf16(acc.z * inv, acc.w * inv);
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + orow * kHeadDim + 4 * lane) = v;
    }
}

// ------------------------------------------------------------------------- host side
static long long up256(long long x) { return (x + 255) & ~255ll; }

struct SharedLayout {
    long long o0, l0, m0, pieces, o1, l1, m1, bytes;   // the prefix pieces', and the own part's one partial per row
};
static SharedLayout shared_layout(const pda_plan_t* pp, const pda_plan_t* p) {
    const long long heads = (long long)p->num_seqs * p->num_kv_heads * p->query_group_size;
    SharedLayout s;
    const long long r0 = heads * (pp->num_partitions + 1), r1 = heads;
    s.o0 = 0;
    s.l0 = s.o0 + up256(r0 * kHeadDim * 4);
    s.m0 = s.l0 + up256(r0 * 4);
    s.pieces = s.m0 + up256(r0 * 4);
    s.o1 = s.pieces + up256(heads * 4);
    s.l1 = s.o1 + up256(r1 * kHeadDim * 4);
    s.m1 = s.l1 + up256(r1 * 4);
    s.bytes = s.m1 + up256(r1 * 4);
    return s;
}
static bool plans_agree(const pda_plan_t* pp, const pda_plan_t* p) {
    return pp && p && pda_workspace_size(pp) >= 0 && pda_workspace_size(p) >= 0 && pp->num_kv_heads == p->num_kv_heads &&
           pp->query_group_size == p->query_group_size && pp->kv_block_size == p->kv_block_size &&
           pp->kv_dtype == p->kv_dtype && pp->resolved_softmax_scale == p->resolved_softmax_scale;
}
// The most steps that the groups can have.
static long long most_steps(const pda_plan_t* pp, const pda_plan_t* p) {
    const long long tiles = ((long long)p->num_seqs * p->query_group_size + kUnitRows - 1) / kUnitRows + pp->num_seqs;
    return tiles * p->num_kv_heads * (((long long)pp->max_blocks_per_seq * pp->kv_block_size + kStep - 1) / kStep);
}
// The row tiles that the groups can have.
static long long most_tiles(const pda_plan_t* p, int groups) {
    return (((long long)p->num_seqs * p->query_group_size + kUnitRows - 1) / kUnitRows + groups - 1) * p->num_kv_heads;
}
// A prefix CTA takes a whole SM.  Where the prefixes can keep half of the SMs busy at most, their pass comes first and
// the own tokens run beside it (32 sequences of 32 heads over 6000 bf16 tokens 23.7 -> 18.8 us), unless they are few and
// there is room for both anyway: the join then waits for one launch less (2 sequences of 8 heads over 250 tokens 12.4
// -> 11.4 us; but with 63 pieces, 4 sequences over 16000 tokens, 17.8 us against 17.0).
// Else the own tokens come first, and the prefix pass, which wants every SM, starts on each as its short work ends.
static bool prefix_first(const pda_plan_t* pp, const pda_plan_t* p, int sms) {
    const long long steps = ((long long)pp->max_blocks_per_seq * pp->kv_block_size + kStep - 1) / kStep;
    const long long pieces = pp->num_partitions < steps ? pp->num_partitions : steps;
    const long long work = most_tiles(p, pp->num_seqs) * pieces;
    return 2 * work <= sms && (work > 16 || work + own_clusters_ctas(p, sms) > sms);
}
static bool odd(const void* p, unsigned a) { return ((uintptr_t)p & (a - 1)) != 0; }

template <int KV>
static int launch_prefix(const SharedArgs& a, const CUtensorMap& kv_map, const CUtensorMap& sc_map, int ctas,
                         cudaStream_t stream) {
    using Cfg = SharedCfg<KV>;
    static bool attr_set[64] = {false};
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PDA_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!attr_set[dev]) {
            if (cudaFuncSetAttribute(pda_prefix_kernel<KV>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem) !=
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
    return cudaLaunchKernelEx(&cfg, pda_prefix_kernel<KV>, kv_map, sc_map, a) == cudaSuccess ? PDA_OK : PDA_ERR_LAUNCH;
}

}  // namespace pda

using namespace pda;

extern "C" {

int pda_shared_tile_groups(const pda_plan_t* plan, int num_groups, int prefix_blocks) {
    if (!plan || pda_workspace_size(plan) < 0 || num_groups < 1 || prefix_blocks < 1) return PDA_ERR_INVALID_ARG;
    int sms = device_sm_count();
    if (sms <= 0) sms = 152;   // planned without a GPU
    // row tiles that work at the same time; with several groups the longest prefix may be twice the
    // average, and is then cut into twice as many pieces
    const long long rows = ((long long)plan->num_seqs * plan->query_group_size + kUnitRows - 1) / kUnitRows;
    const long long tiles = (rows > num_groups ? rows : num_groups) * plan->num_kv_heads;
    const long long pieces = (sms + tiles - 1) / tiles * (num_groups > 1 ? 2 : 1);
    const long long tokens = (long long)prefix_blocks * plan->kv_block_size;
    // pieces of 256 or 512 tokens where half of the SMs hold them all, and the own tokens run beside them (32 sequences
    // of 64 heads over 1500 bf16 tokens 15.7 us in pieces of 256, 18.1 of 512, 21.2 of 1024); more and shorter
    // pieces cost the join more than they save (8 sequences of 64 heads over 4000: 20.4 us in 128 pieces, 15.6 in 64)
    for (int G = 1; G <= 2; ++G)
        if (2 * most_tiles(plan, num_groups) * ((tokens + G * kTokensPerTileGroup - 1) / (G * kTokensPerTileGroup)) <= sms)
            return G;
    const long long G = (tokens + pieces * kTokensPerTileGroup - 1) / (pieces * kTokensPerTileGroup);
    return (int)(G < 2 ? 2 : G > (1 << 22) ? (1 << 22) : G);
}

long long pda_shared_workspace_size(const pda_plan_t* prefix_plan, const pda_plan_t* plan) {
    if (!plans_agree(prefix_plan, plan)) return -1;
    return shared_layout(prefix_plan, plan).bytes;
}

int pda_decode_shared(const pda_plan_t* prefix_plan, const pda_plan_t* plan, const void* query, const void* kv_cache,
                      long long num_cache_blocks, const int* group_starts, const int* prefix_table,
                      const int* prefix_lens, const int* block_table, const int* context_lens, void* workspace,
                      long long workspace_bytes, void* out, int out_dtype, int* err_word, void* stream) {
    if (!plans_agree(prefix_plan, plan) || (out_dtype != PDA_OUT_BF16 && out_dtype != PDA_OUT_F32))
        return PDA_ERR_INVALID_ARG;
    if (plan->kv_dtype == PDA_KV_TQ4) return PDA_ERR_UNSUPPORTED;
    if (plan->num_seqs == 0) return PDA_OK;
    if (prefix_plan->num_seqs == 0) return PDA_ERR_INVALID_ARG;   // no groups: that is pda_decode
    if (!query || !kv_cache || !group_starts || !prefix_table || !prefix_lens || !block_table || !context_lens ||
        !workspace || !out)
        return PDA_ERR_INVALID_ARG;
    if (num_cache_blocks < 1 || num_cache_blocks > (1ll << 31) - 1) return PDA_ERR_INVALID_ARG;
    if (odd(query, 16) || odd(kv_cache, 16) || odd(workspace, 32) || odd(group_starts, 4) || odd(prefix_table, 4) ||
        odd(prefix_lens, 4) || odd(block_table, 4) || odd(context_lens, 4) || odd(err_word, 4) ||
        odd(out, out_dtype == PDA_OUT_F32 ? 16 : 8))
        return PDA_ERR_INVALID_ARG;
    const SharedLayout w = shared_layout(prefix_plan, plan);
    if (workspace_bytes < w.bytes) return PDA_ERR_WORKSPACE_TOO_SMALL;
    if (most_steps(prefix_plan, plan) > 2000000000ll / (1 + kSwitch)) return PDA_ERR_INVALID_ARG;   // places are ints
    const int sms = device_sm_count();
    if (sms <= 0) return PDA_ERR_CUDA;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    auto f32 = [&](long long at) { return reinterpret_cast<float*>(ws + at); };
    SharedArgs a = {};
    a.query = static_cast<const uint16_t*>(query);
    a.group_starts = group_starts;
    a.prefix_table = prefix_table;
    a.prefix_lens = prefix_lens;
    a.part_o = f32(w.o0);
    a.part_l = f32(w.l0);
    a.part_m = f32(w.m0);
    a.pieces = reinterpret_cast<int*>(ws + w.pieces);
    a.err_word = err_word;
    a.num_cache_blocks = num_cache_blocks;
    a.B = plan->num_seqs;
    a.NG = prefix_plan->num_seqs;
    a.Hk = plan->num_kv_heads;
    a.QG = plan->query_group_size;
    a.MP = prefix_plan->max_blocks_per_seq;
    a.BS = plan->kv_block_size;
    a.P = prefix_plan->num_partitions;
    a.slots = a.P + 1;
    a.qk_scale_log2 = plan->resolved_softmax_scale * kLog2eS;
    a.timeout_ns = prefix_plan->wait_timeout_ns > 0 ? (unsigned long long)prefix_plan->wait_timeout_ns : kDefaultTimeoutNs;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CUtensorMap kv_map, sc_map;
    if (!encode_block_map(&kv_map, kv_cache, plan, num_cache_blocks)) return PDA_ERR_LAUNCH;
    a.first = prefix_first(prefix_plan, plan, sms);
    auto own = [&] {
        return decode_own(plan, a.first, query, kv_cache, num_cache_blocks, block_table, context_lens, f32(w.o1), f32(w.l1),
                          f32(w.m1), err_word, s);
    };
    int rc = a.first ? PDA_OK : own();
    if (rc != PDA_OK) return rc;
    const long long most = most_steps(prefix_plan, plan);   // no more CTAs than there can be steps
    const int ctas = (int)(most < sms ? most : sms);
    if (plan->kv_dtype == PDA_KV_BF16) {
        rc = launch_prefix<PDA_KV_BF16>(a, kv_map, kv_map, ctas, s);
    } else {
        if (!encode_block_scale_map(&sc_map, kv_cache, plan, num_cache_blocks)) return PDA_ERR_LAUNCH;
        rc = launch_prefix<PDA_KV_FP8_E4M3>(a, kv_map, sc_map, ctas, s);
    }
    if (rc == PDA_OK && a.first) rc = own();
    if (rc != PDA_OK) return rc;
    JoinArgs j = {};
    j.group_starts = group_starts;
    j.prefix_lens = prefix_lens;
    j.context_lens = context_lens;
    j.part_o[0] = f32(w.o0);
    j.part_l[0] = f32(w.l0);
    j.part_m[0] = f32(w.m0);
    j.part_o[1] = f32(w.o1);
    j.part_l[1] = f32(w.l1);
    j.part_m[1] = f32(w.m1);
    j.pieces = a.pieces;
    j.out = out;
    j.B = a.B;
    j.NG = a.NG;
    j.Hk = a.Hk;
    j.QG = a.QG;
    j.MP = a.MP;
    j.MB = plan->max_blocks_per_seq;
    j.BS = a.BS;
    j.slots = a.slots;
    j.out_f32 = out_dtype == PDA_OUT_F32;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)a.B * a.Hk));
    cfg.blockDim = dim3(a.QG * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, pda_shared_join_kernel, j) == cudaSuccess ? PDA_OK : PDA_ERR_LAUNCH;
}

}  // extern "C"
