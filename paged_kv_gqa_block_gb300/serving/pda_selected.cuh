// pda_selected.cuh -- attention over short lists in one launch: the tiles of a (sequence, KV head) are split
// over the warps of a thread-block cluster, whose results are joined in shared memory.  Three lists: the selected
// blocks of each (sequence, KV head) (pda_decode_selected) and the first and last tokens of a sequence
// (WINDOW, pda_decode_window), whose result is the output, and a sequence's own tokens beside a shared prefix
// (OWN, pda_decode_shared), whose result is a partial for the join there.
//
// Such lists are a few thousand tokens and of like length, so a unit needs neither partials in
// global memory nor a second launch: C CTAs of nw warps take an equal run of its 16-token tiles each,
// with the arithmetic and the private copy rings of the head-warp kernel (pda_decode.cuh); each warp
// leaves (m, l, o), the maximum, the sum of exponentials and the normalised output of its run, in its
// ring; the CTA joins its warps, w = l 2^(m - M), and the cluster its CTAs through distributed shared
// memory, each CTA a share of the rows.  Bound by HBM for large batches (lists of
// blocks of their own: 800 units of 4096 bf16 tokens 245 us, 6.9 TB/s; 512 of 2048 fp8 tokens 47.8 us, 5.8 TB/s, of
// which the last, uneven round of units is a part) and by the chain of one warp (lengths, table, copies, 0.6 us per two
// tiles) for small ones (32 units of 2048 bf16 tokens 11.5 us, 2.9 TB/s; 8 units 7.7 us).
#pragma once

#include <cooperative_groups.h>

#include "pda_decode.cuh"
#include "pda_window.cuh"

namespace pda {

namespace cg = cooperative_groups;

constexpr int kSelRows = 16;   // query rows of a unit, at most
enum { kListSelected = 0, kListOwn = 1, kListWindow = 2 };

template <int KV, int S>
struct SelectedCfg {
    static constexpr int kRing = S * DecodeCfg<KV, S>::kTileBytes;     // a multiple of 1024
    static constexpr int kScales = S * DecodeCfg<KV, S>::kScaleBytes;
    // per warp: ring, scales, the rows' m and l, barriers; per CTA: the joined rows' m and l (the rows themselves
    // take the place of the first warp's: with 8 KB of their own, one CTA fewer fitted an SM)
    static constexpr int bytes(int nw) {
        return nw * (kRing + kScales + S * 8 + 2 * kSelRows * 4) + 2 * kSelRows * 4 + 1024;
    }
};

__device__ __forceinline__ void store_row4(void* out, int f32, long long row, int c, float4 v) {
    if (f32) {
        *reinterpret_cast<float4*>(static_cast<float*>(out) + row * kHeadDim + 4 * c) = v;
    } else {
        uint2 u;
        u.x = pack_bf16(v.x, v.y);
        u.y = pack_bf16(v.z, v.w);
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + row * kHeadDim + 4 * c) = u;
    }
}

// A row's joined result: o = sum w_i o_i (to be divided by L), M and L as above (log2 units).
template <bool OWN>
__device__ __forceinline__ void store_joined(const DecodeArgs& a, long long row, int c, float4 o, float M, float L) {
    const float r = L == 0.f ? 0.f : 1.f / L;
    const float4 v = make_float4(o.x * r, o.y * r, o.z * r, o.w * r);
    if constexpr (OWN) {
        store_row4(a.partial_out, 1, row, c, v);
        if (c == 0) {
            a.exp_sums[row] = L;
            a.max_logits[row] = M * kLn2;
        }
    } else {
        store_row4(a.out, a.out_f32, row, c, v);
    }
}

// The sequence that stands at place `pos` when those of many tiles come first: by eighths of the most tiles that a window has,
// and by index in some order that is every CTA's.  Called by all threads of a CTA; `counts` [warps][8].
__device__ __forceinline__ int longest_first(const int* lens, int B, int max_ctx, int window, int num_first, int most, int pos,
                                             int (*counts)[8]) {
    const int nw = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float eighth = 7.999f / (float)most;
    auto kind = [&](int b) {   // 0: the most tiles; 8: none there
        if (b >= B) return 8;
        return 7 - min(7, (int)((float)WindowTiles(sanitize_ctx(__ldg(lens + b), max_ctx), window, num_first).tiles * eighth));
    };
    int mine = 0;   // of kind `lane`
    for (int b = 32 * warp; b < B; b += 32 * nw) {
        const int k = kind(b + lane);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int n = __popc(__ballot_sync(kFull, k == i));
            if (lane == i) mine += n;
        }
    }
    if (lane < 8) counts[warp][lane] = mine;
    __syncthreads();
    int of_kind = 0;
    if (lane < 8)
        for (int w = 0; w < nw; ++w) of_kind += counts[w][lane];
    int before = of_kind;   // of kinds 0 .. lane, then of those before
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        const int x = __shfl_up_sync(kFull, before, o);
        if (lane >= o) before += x;
    }
    before -= of_kind;
    const int k = 31 - __clz((int)__ballot_sync(kFull, lane < 8 && before <= pos));   // the last kind that starts no later
    int r = pos - __shfl_sync(kFull, before, k), w = 0;
    while (w + 1 < nw && r >= counts[w][k]) r -= counts[w++][k];
    for (int b = 32 * w; b < B; b += 32 * nw) {
        const unsigned all = __ballot_sync(kFull, kind(b + lane) == k);
        const int n = __popc(all);
        if (r < n) return b + (int)__fns(all, 0, r + 1);
        r -= n;
    }
    return 0;   // not reached
}

template <int KV, int NT, int S, int NWMAX, int MINB, int LIST>
__global__ void __launch_bounds__(32 * NWMAX, MINB)
    pda_selected_kernel(const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ CUtensorMap sc_map,
                        const DecodeArgs a, const int C, const int behind, const int window, const int num_first, const int most) {
    constexpr bool OWN = LIST == kListOwn, WINDOW = LIST == kListWindow;
    using D = Decode<KV, NT, S, false>;
    using Cfg = DecodeCfg<KV, S>;
    using Sel = SelectedCfg<KV, S>;
    constexpr bool FP8 = D::FP8, TQ = D::TQ, F16 = D::F16;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t tq_lut[TQ ? 256 : 1];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int nw = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
    static_assert(Sel::kRing >= kSelRows * kHeadDim * 4, "a ring holds its warp's rows");
    uint8_t* ring = smem + warp * Sel::kRing;
    uint8_t* scales = smem + nw * Sel::kRing + warp * Sel::kScales;
    float* stats = reinterpret_cast<float*>(smem + nw * (Sel::kRing + Sel::kScales));   // [nw][2: m, l][16]
    float* jm = stats + nw * 2 * kSelRows;                                               // joined: m [16], l [16]
    float* jl = jm + kSelRows;
    const uint32_t bar0 = smem_addr(jl + kSelRows) + warp * S * 8;
    const uint32_t sring = smem_addr(ring), sscale = smem_addr(scales);
    if (lane == 0) {
        for (int s = 0; s < S; ++s) mbar_init(bar0 + 8 * s, 1);
        fence_mbar_init();
        prefetch_tensormap(&kv_map);
        if (F16) prefetch_tensormap(&sc_map);
    }
    __syncwarp();
    // Own tokens and the prefix pass read nothing of one another's.  The first of the two waits for everything
    // before them and then lets the other start; the second waits for the first before it ends (one CTA of it: the
    // others make room), so that the join waits for both.  The second has not waited when it reads the step's inputs:
    // they lie in L2 by then, and it reads them there (ld.cg, TMA), past any line that an earlier grid left in L1.
    if constexpr (!OWN) allow_dependent_launch();
    if (!OWN || !behind) grid_dependency_wait();
    if constexpr (OWN) allow_dependent_launch();
    auto leave = [&] {
        if (OWN && behind && blockIdx.x == gridDim.x - 1) grid_dependency_wait();
    };

    const int unit = blockIdx.x / C, rank = blockIdx.x - unit * C;
    const int head = unit % a.sel_heads;
    int list = OWN || WINDOW ? unit / a.sel_heads : unit;   // the table row and length
    const int max_ctx = a.MB * a.BS;
    if constexpr (WINDOW) {
        // more clusters than fit at once: the long ones start first, and the short ones fill the end
        __shared__ int counts[NWMAX][8];
        if (most > 0) list = longest_first(a.context_lens, a.B / a.sel_heads, max_ctx, window, num_first, most, list, counts);
    }
    const int rows_of = WINDOW ? list * a.sel_heads + head : unit;   // the query rows and the result's
    // What a warp needs first is asked for at once: the length, its part of the table as if the list were full (a
    // selected list mostly is, and the first warp's part does not depend on it), and the query rows.
    const int ts = a.bs_shift - 4, n = C * nw, wi = rank * nw + warp;
    const int* table = a.block_table + (long long)list * a.MB;
    auto run_of = [&](int tiles, int& t0, int& t1) {   // runs of whole pairs: a step takes two tiles
        const long long pairs = (tiles + 1) >> 1;
        t0 = 2 * (int)(wi * pairs / n);
        t1 = min(tiles, 2 * (int)((wi + 1) * pairs / n));
    };
    int t0, t1;
    run_of(max_ctx >> 4, t0, t1);
    int e0 = t0 >> ts;
    int ent = !WINDOW && e0 + lane < a.MB ? load_input<OWN>(table + e0 + lane) : 0;
    const int raw = load_input<OWN>(a.context_lens + list);
    uint32_t qn[NT][16];
    {
        UnitIt u = {rows_of, 0, 0, 0, 0, 0};
        D::template load_q<OWN>(a, u, qn, lane);
    }
    if ((raw < 0 || raw > max_ctx) && rank == 0 && threadIdx.x == 0 && (!(OWN || WINDOW) || head == 0) && a.err_word)
        atomicOr(a.err_word, PDA_ERRW_BAD_CONTEXT_LEN);
    const int ctx = sanitize_ctx(raw, max_ctx);
    if (OWN && ctx == 0) return leave();   // every CTA of the cluster
    const WindowTiles win(WINDOW ? ctx : 0, window, num_first);
    run_of(WINDOW ? win.tiles : (ctx + 15) >> 4, t0, t1);
    bool ok = true;

    if (t0 < t1) {
        float cent = 0.f;
        if constexpr (TQ) cent = __ldg(a.centroids + (lane & 15));
        const int entries = WINDOW ? (ctx + a.BS - 1) >> a.bs_shift : ((t1 - 1) >> ts) + 1;
        if constexpr (WINDOW) {
            e0 = win.token(t0) >> a.bs_shift;
            ent = e0 + lane < entries ? __ldg(table + e0 + lane) : 0;
        } else if (e0 != t0 >> ts) {
            e0 = t0 >> ts;
            ent = e0 + lane < entries ? load_input<OWN>(table + e0 + lane) : 0;
        }
        const uint64_t policy = l2_policy_evict_first();
        int issued = 0;
        auto issue = [&](int t, int stage) {   // tiles in order
            const int e = WINDOW ? win.token(t) >> a.bs_shift : t >> ts;
            if (e - e0 >= 32) {
                e0 = WINDOW ? e : e0 + 32;
                ent = e0 + lane < entries ? load_input<OWN>(table + e0 + lane) : 0;
            }
            const int phys = __shfl_sync(kFull, ent, e - e0);
            if (lane == 0) {
                const int slot0 = WINDOW ? win.token(t) & (a.BS - 1) : (t & ((1 << ts) - 1)) * kTileTokens;
                const uint32_t bar = bar0 + 8 * stage;
                mbar_arrive_expect_tx(bar, Cfg::kTileBytes + Cfg::kScaleTx);
                tma_load_5d(sring + stage * Cfg::kTileBytes, &kv_map, bar, 0, slot0, 0, head, phys, policy);
                if constexpr (F16)   // whole tiles of scales: a copy's innermost coordinate keeps its 16 bytes' alignment
                    tma_load_4d(sscale + stage * Cfg::kScaleBytes, &sc_map, bar, WINDOW ? slot0 & ~15 : slot0, 0, head, phys, policy);
                if ((phys < 0 || (long long)phys >= a.num_cache_blocks) && a.err_word)
                    atomicOr(a.err_word, PDA_ERRW_BAD_BLOCK_ID);
            }
            ++issued;
        };
        int next = t0;
        for (int s = 0; s < S && next < t1; ++s) issue(next++, s);

        // the TQ4 centroid table: every warp writes the same values and reads its own
        float cscale = 1.f;
        if constexpr (TQ) {
            float amax = fabsf(cent);
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
            int e = 0;
            if (amax > 0.f) e = 14 - ((int)((__float_as_uint(amax) >> 23) & 0xFF) - 127);
            e = max(-100, min(100, e));
            cscale = __uint_as_float((uint32_t)(127 - e) << 23);
            const uint32_t h16 = (uint32_t)__half_as_ushort(__float2half_rn(cent * __uint_as_float((uint32_t)(e + 127) << 23)));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int x = 8 * lane + i;
                const uint32_t lo = __shfl_sync(kFull, h16, x & 15), hi16 = __shfl_sync(kFull, h16, x >> 4);
                tq_lut[x] = lo | (hi16 << 16);
            }
            __syncwarp();
        }
        uint32_t qf[NT][8][2];
        float cq = a.qk_scale_log2;
        if constexpr (!F16) {
#pragma unroll
            for (int m = 0; m < NT; ++m)
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    qf[m][kk][0] = qn[m][2 * kk];
                    qf[m][kk][1] = qn[m][2 * kk + 1];
                }
        } else {   // Q times a power of two that brings it into f16's range, as in the head-warp kernel
            float amax = 0.f;
#pragma unroll
            for (int m = 0; m < NT; ++m)
#pragma unroll
                for (int c = 0; c < 16; ++c) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(qn[m][c])), fabsf(bf16_hi(qn[m][c]))));
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
            int e = 0;
            if (amax > 0.f) e = 14 - ((int)((__float_as_uint(amax) >> 23) & 0xFF) - 127);
            e = max(-100, min(100, e));
            const float pw = __uint_as_float((uint32_t)(e + 127) << 23);
            cq = a.qk_scale_log2 * __uint_as_float((uint32_t)(127 - e) << 23) * cscale;
#pragma unroll
            for (int m = 0; m < NT; ++m)
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    const uint32_t x = qn[m][2 * kk], y = qn[m][2 * kk + 1];
                    qf[m][kk][0] = pack_f16(bf16_lo(x) * pw, bf16_hi(x) * pw);
                    qf[m][kk][1] = pack_f16(bf16_lo(y) * pw, bf16_hi(y) * pw);
                }
        }

        float acc[NT][8][4];
        float m2[NT][2], mt[NT][2], ls[NT][2], zs[NT][2];
        float F = 1.f, rF = 1.f;
#pragma unroll
        for (int m = 0; m < NT; ++m) {
#pragma unroll
            for (int c = 0; c < 8; ++c) acc[m][c][0] = acc[m][c][1] = acc[m][c][2] = acc[m][c][3] = 0.f;
            m2[m][0] = m2[m][1] = mt[m][0] = mt[m][1] = -INFINITY;
            ls[m][0] = ls[m][1] = zs[m][0] = zs[m][1] = 0.f;
        }
        int cs = 0;
        uint32_t cph = 0;
        for (int t = t0; t < t1;) {
            // only a step's last tile may be partly seen
            const bool two = t + 1 < t1 && (!WINDOW || win.count(t) == kTileTokens);
            const int s0 = cs, s1 = s0 + 1 == S ? 0 : s0 + 1;
            const uint32_t ph0 = cph, ph1 = s0 + 1 == S ? cph ^ 1u : cph;
            if (!mbar_wait_warp(bar0 + 8 * s0, ph0, a.timeout_ns) || (two && !mbar_wait_warp(bar0 + 8 * s1, ph1, a.timeout_ns))) {
                ok = false;
                break;
            }
            const int v0 = WINDOW ? win.count(t) : ctx - t * kTileTokens, v1 = WINDOW ? (two ? win.count(t + 1) : 0) : v0 - kTileTokens;
            const uint32_t a0 = sring + s0 * Cfg::kTileBytes, a1 = sring + s1 * Cfg::kTileBytes;
            const uint8_t* c0 = scales + s0 * Cfg::kScaleBytes;
            const uint8_t* c1 = scales + s1 * Cfg::kScaleBytes;
            if constexpr (WINDOW && F16) {   // the tile in which the window begins: its tokens' scales start as far into their tile
                constexpr int field = FP8 ? 4 : 2;
                c0 += (win.token(t) & 15) * field;
                if (two) c1 += (win.token(t + 1) & 15) * field;
            }
            if (two) {
                const uint32_t st[2] = {a0, a1};
                const int vv[2] = {v0, v1};
                if constexpr (TQ) {
                    const __half* const sc[2] = {reinterpret_cast<const __half*>(c0), reinterpret_cast<const __half*>(c1)};
                    D::template step_tq<2>(st, sc, vv, cq, tq_lut, qf, acc, m2, mt, ls, zs, F, rF, lane);
                } else if constexpr (FP8) {
                    const float* const sc[2] = {reinterpret_cast<const float*>(c0), reinterpret_cast<const float*>(c1)};
                    D::template step_fp8<2>(st, sc, vv, cq, qf, acc, m2, mt, ls, F, rF, lane);
                } else {
                    D::template step_bf16<2>(st, vv, a.qk_scale_log2, qf, acc, m2, mt, ls, lane);
                }
            } else {
                const uint32_t st[1] = {a0};
                const int vv[1] = {v0};
                if constexpr (TQ) {
                    const __half* const sc[1] = {reinterpret_cast<const __half*>(c0)};
                    D::template step_tq<1>(st, sc, vv, cq, tq_lut, qf, acc, m2, mt, ls, zs, F, rF, lane);
                } else if constexpr (FP8) {
                    const float* const sc[1] = {reinterpret_cast<const float*>(c0)};
                    D::template step_fp8<1>(st, sc, vv, cq, qf, acc, m2, mt, ls, F, rF, lane);
                } else {
                    D::template step_bf16<1>(st, vv, a.qk_scale_log2, qf, acc, m2, mt, ls, lane);
                }
            }
            __syncwarp();
            if (next < t1) issue(next++, s0);
            if (two && next < t1) issue(next++, s1);
            t += two ? 2 : 1;
            cs = two ? (s1 + 1 == S ? 0 : s1 + 1) : s1;
            cph = two ? (s1 + 1 == S ? ph1 ^ 1u : ph1) : ph1;
        }
        if (ok) {
            // o = acc * F / l (+ z / l), the rows' m (log2 units) and l, as the head-warp kernel's epilogue
            float* stg = reinterpret_cast<float*>(ring);
#pragma unroll
            for (int m = 0; m < NT; ++m)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float l = ls[m][j], M = m2[m][j], ref = m2[m][j];
                    l += __shfl_xor_sync(kFull, l, 4);
                    l += __shfl_xor_sync(kFull, l, 8);
                    l += __shfl_xor_sync(kFull, l, 16);
                    if constexpr (D::kLazy) {
                        M = mt[m][j];
                        M = fmaxf(M, __shfl_xor_sync(kFull, M, 4));
                        M = fmaxf(M, __shfl_xor_sync(kFull, M, 8));
                        M = fmaxf(M, __shfl_xor_sync(kFull, M, 16));
                    }
                    const float il = l > 0.f ? 1.f / l : 0.f;
                    const float inv = il * (FP8 ? F : TQ ? F * 16777216.f : 1.f);
                    float zq = 0.f;
                    if constexpr (TQ) {
                        float z = zs[m][j];
                        z += __shfl_xor_sync(kFull, z, 4);
                        z += __shfl_xor_sync(kFull, z, 8);
                        z += __shfl_xor_sync(kFull, z, 16);
                        zq = z * il;
                    }
                    const int q = m * 8 + 2 * tig + j;
                    if (gid == 0) {
                        stats[warp * 2 * kSelRows + q] = M;
                        stats[(warp * 2 + 1) * kSelRows + q] = M == -INFINITY ? l : l * ex2(ref - M);
                    }
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        if constexpr (F16) {
                            const int d = TQ ? (32 * (c >> 1) + 4 * gid + 2 * (c & 1)) : (16 * gid + 2 * c);
                            float2 v;
                            if constexpr (TQ) {
                                v.x = fmaf(acc[m][c][j], inv, zq);
                                v.y = fmaf(acc[m][c][j + 2], inv * 0.0625f, zq);
                            } else {
                                v.x = acc[m][c][j] * inv;
                                v.y = acc[m][c][j + 2] * inv;
                            }
                            *reinterpret_cast<float2*>(stg + q * kHeadDim + (((d >> 2) ^ (q & 6)) << 2) + (d & 3)) = v;
                        } else {
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const int d = 16 * c + gid + 8 * k;
                                stg[q * kHeadDim + (((d >> 2) ^ (q & 6)) << 2) + (d & 3)] = acc[m][c][j + 2 * k] * inv;
                            }
                        }
                    }
                }
        } else if (lane == 0) {
            if (a.err_word) atomicOr(a.err_word, PDA_ERRW_PIPELINE_TIMEOUT);
            // no copy may land in this CTA's memory after it leaves (bounded by the default limit)
            for (int s = 0; s < S; ++s) {
                if (issued <= s) continue;
                const int j = s + ((issued - 1 - s) / S) * S;
                (void)mbar_wait(bar0 + 8 * s, (uint32_t)((j / S) & 1), kDefaultTimeoutNs);
            }
        }
    }
    if ((t0 >= t1 || !ok) && lane < kSelRows) {   // this warp has nothing to say
        stats[warp * 2 * kSelRows + lane] = -INFINITY;
        stats[(warp * 2 + 1) * kSelRows + lane] = 0.f;
    }
    __syncthreads();
    // The CTA's rows: a weight of exactly zero leaves its warp out (its memory holds no rows then).  The joined
    // rows take the place of the first warp's: each four values are read and written by one thread.
    float* joined = reinterpret_cast<float*>(smem);
    auto place = [](int q, int c) { return q * kHeadDim + ((c ^ (q & 6)) << 2); };
    for (int i = threadIdx.x; i < a.QG * 32; i += blockDim.x) {
        const int q = i >> 5, c = i & 31;
        float M = -INFINITY;
        for (int w = 0; w < nw; ++w) M = fmaxf(M, stats[w * 2 * kSelRows + q]);
        float L = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < nw; ++w) {
            const float l = stats[(w * 2 + 1) * kSelRows + q];
            if (l == 0.f) continue;
            const float f = l * ex2(stats[w * 2 * kSelRows + q] - M);
            const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + w * Sel::kRing) + place(q, c));
            L += f;
            o.x = fmaf(f, v.x, o.x);
            o.y = fmaf(f, v.y, o.y);
            o.z = fmaf(f, v.z, o.z);
            o.w = fmaf(f, v.w, o.w);
        }
        if (C == 1) {
            store_joined<OWN>(a, (long long)rows_of * a.QG + q, c, o, M, L);
        } else {
            *reinterpret_cast<float4*>(joined + place(q, c)) = o;
            if (c == 0) {
                jm[q] = M;
                jl[q] = L;
            }
        }
    }
    if (C == 1) return leave();
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    for (int i = rank * blockDim.x + threadIdx.x; i < a.QG * 32; i += C * blockDim.x) {
        const int q = i >> 5, c = i & 31;
        float M = -INFINITY;
        for (int r = 0; r < C; ++r) M = fmaxf(M, *cl.map_shared_rank(jm + q, r));
        float L = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int r = 0; r < C; ++r) {
            const float l = *cl.map_shared_rank(jl + q, r);
            if (l == 0.f) continue;
            const float f = ex2(*cl.map_shared_rank(jm + q, r) - M);
            const float4 v = *reinterpret_cast<const float4*>(cl.map_shared_rank(joined + place(q, c), r));
            L += l * f;
            o.x = fmaf(f, v.x, o.x);
            o.y = fmaf(f, v.y, o.y);
            o.z = fmaf(f, v.z, o.z);
            o.w = fmaf(f, v.w, o.w);
        }
        store_joined<OWN>(a, (long long)rows_of * a.QG + q, c, o, M, L);
    }
    cl.sync();   // nobody leaves while its rows are read
    leave();
}

}  // namespace pda
