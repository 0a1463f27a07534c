// pda_sparse.cu -- choosing the cache blocks a decode step attends to: pda_summarize_blocks,
// pda_score_blocks, pda_select_blocks.  (pda_decode_selected, the attention over them, has its kernel in
// pda_selected.cuh and its checks in pda_api.cu.)
//
// A block's summary is, per KV head, the largest and smallest value of each key dimension over the
// block's tokens.  For a query row q every key k of the block satisfies
//   q.k = sum_d q_d k_d <= sum_d max(q_d, 0) kmax_d + min(q_d, 0) kmin_d,
// so the right side, the block's score, bounds every logit in the block; the score of a KV head is
// the largest over its query rows.  The two terms are one inner product of length 256, [q+ | q-]
// with [kmax | kmin], which is a matrix product of the blocks' summaries with the query rows.
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "pda.h"
#include "pda_internal.h"
#include "pda_ptx.cuh"

namespace pda {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kSumBytes = 512;   // one summary: 128 maxima, 128 minima, bf16

__device__ __forceinline__ int clean_ctx(int c, int max_ctx, int* err_word, bool report) {
    if (c >= 0 && c <= max_ctx) return c;
    if (report && err_word) atomicOr(err_word, PDA_ERRW_BAD_CONTEXT_LEN);
    return 0;
}

// ------------------------------------------------------------------------- summaries
struct SumArgs {
    const uint8_t* cache;
    const int* block_table;
    const int* context_lens;
    const int* since;        // may be null: all blocks
    const float* centroids;  // TQ4
    uint8_t* summaries;      // [NB][Hk][2][128] bf16
    int* err_word;
    long long NB, block_bytes, meta_offset;
    int Hk, MB, BS;
    int ctas;                // CTAs per sequence
};

// fp32 to bf16 away from the interior: up for a maximum, down for a minimum, so that the rounded
// value still bounds what it stands for (bf16 keys are exact; fp8 and TQ4 products need it).
__device__ __forceinline__ uint32_t bf16_up(float x) {
    const uint32_t u = __float_as_uint(x);
    uint32_t t = u >> 16;
    if ((u & 0xFFFFu) && !(u >> 31)) ++t;   // truncation moved a positive value down
    return t;
}
__device__ __forceinline__ uint32_t bf16_down(float x) { return bf16_up(-x) ^ 0x8000u; }

// One warp per (block, KV head).  A key row is R16 16-byte words (16 bf16, 8 fp8, 4 TQ4), so 32/R16
// tokens are loaded by one instruction and a lane keeps the words of its dimensions; the lanes that
// hold the same dimensions of other tokens are joined by shuffles at the end.  All of a block's
// loads (BS / (32/R16) per lane) are requested before the first is used.  Bound by HBM: the keys are
// read once (a 256-byte run per bf16 row), 512 bytes are written (whole contexts, 390146 tokens of 8 heads: 152 us, 5.6
// TB/s); by latency where only the newest blocks are renewed (16 sequences of 8 heads: 3.7 us).
template <int KV, int BS>
__global__ void __launch_bounds__(256) pda_summarize_kernel(const SumArgs a) {
    allow_dependent_launch();
    grid_dependency_wait();
    constexpr int R16 = KV == PDA_KV_BF16 ? 16 : KV == PDA_KV_FP8_E4M3 ? 8 : 4;
    constexpr int TOK = 32 / R16, LOADS = BS / TOK, E = 128 / R16;   // E elements per word
    constexpr int kTokenBytes = KV == PDA_KV_BF16 ? 512 : KV == PDA_KV_FP8_E4M3 ? 256 : 128;
    const int b = blockIdx.x / a.ctas, cta = blockIdx.x - b * a.ctas;
    const int lane = threadIdx.x & 31, part = lane % R16, tok0 = lane / R16;
    const int max_ctx = a.MB * a.BS;
    const int ctx = clean_ctx(__ldg(a.context_lens + b), max_ctx, a.err_word, cta == 0 && threadIdx.x == 0);
    const int first = a.since ? max(0, __ldg(a.since + b)) / BS : 0;
    const int n = (ctx + BS - 1) / BS - first;
    if (n <= 0) return;
    const long long items = (long long)n * a.Hk, step = (long long)a.ctas * (blockDim.x >> 5);
    for (long long it = (long long)cta * (blockDim.x >> 5) + (threadIdx.x >> 5); it < items; it += step) {
        const int j = first + (int)(it / a.Hk), h = (int)(it % a.Hk);
        const int id = __ldg(a.block_table + (long long)b * a.MB + j);
        if (id < 0 || id >= a.NB) {
            if (h == 0 && lane == 0 && a.err_word) atomicOr(a.err_word, PDA_ERRW_BAD_BLOCK_ID);
            continue;
        }
        const int valid = min(BS, ctx - j * BS);
        const uint8_t* block = a.cache + (long long)id * a.block_bytes;
        const uint8_t* row = block + (long long)h * kTokenBytes + part * 16;
        uint4 w[LOADS];
        float sc[LOADS];
#pragma unroll
        for (int l = 0; l < LOADS; ++l) {
            const int t = min(l * TOK + tok0, valid - 1);   // past the context: the last token again
            w[l] = __ldg(reinterpret_cast<const uint4*>(row + (long long)t * a.Hk * kTokenBytes));
            if constexpr (KV == PDA_KV_FP8_E4M3)
                sc[l] = __ldg(reinterpret_cast<const float*>(block + a.meta_offset) + (long long)h * 2 * BS + t);
            if constexpr (KV == PDA_KV_TQ4)
                sc[l] = __half2float(__ushort_as_half(
                    __ldg(reinterpret_cast<const unsigned short*>(block + a.meta_offset) + (long long)h * 3 * BS + t)));
        }
        float mx[E], mn[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            mx[e] = -INFINITY;
            mn[e] = INFINITY;
        }
#pragma unroll
        for (int l = 0; l < LOADS; ++l) {
            const uint32_t x[4] = {w[l].x, w[l].y, w[l].z, w[l].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float v[E / 4];
                if constexpr (KV == PDA_KV_BF16) {
                    v[0] = bf16_lo(x[i]);
                    v[1] = bf16_hi(x[i]);
                } else if constexpr (KV == PDA_KV_FP8_E4M3) {
                    uint32_t lo, hi;
                    e4m3x4_to_f16x2x2(x[i], lo, hi);
                    const float2 p = __half22float2(*reinterpret_cast<__half2*>(&lo));
                    const float2 q = __half22float2(*reinterpret_cast<__half2*>(&hi));
                    v[0] = __fmul_rn(p.x, sc[l]);
                    v[1] = __fmul_rn(p.y, sc[l]);
                    v[2] = __fmul_rn(q.x, sc[l]);
                    v[3] = __fmul_rn(q.y, sc[l]);
                } else {
#pragma unroll
                    for (int c = 0; c < 8; ++c) v[c] = __fmul_rn(__ldg(a.centroids + ((x[i] >> (4 * c)) & 15u)), sc[l]);
                }
#pragma unroll
                for (int c = 0; c < E / 4; ++c) {
                    mx[i * (E / 4) + c] = fmaxf(mx[i * (E / 4) + c], v[c]);
                    mn[i * (E / 4) + c] = fminf(mn[i * (E / 4) + c], v[c]);
                }
            }
        }
#pragma unroll
        for (int o = R16; o < 32; o <<= 1)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                mx[e] = fmaxf(mx[e], __shfl_xor_sync(kAll, mx[e], o));
                mn[e] = fminf(mn[e], __shfl_xor_sync(kAll, mn[e], o));
            }
        // the first R16 lanes store the maxima, the next R16 the minima
        if (lane < 2 * R16) {
            uint32_t out[E / 2];
#pragma unroll
            for (int e = 0; e < E / 2; ++e)
                out[e] = lane < R16 ? bf16_up(mx[2 * e]) | (bf16_up(mx[2 * e + 1]) << 16)
                                    : bf16_down(mn[2 * e]) | (bf16_down(mn[2 * e + 1]) << 16);
            uint4* dst = reinterpret_cast<uint4*>(a.summaries + ((long long)id * a.Hk + h) * kSumBytes +
                                                  (lane < R16 ? 0 : 256) + part * (E * 2));
#pragma unroll
            for (int c = 0; c < E / 8; ++c) dst[c] = make_uint4(out[4 * c], out[4 * c + 1], out[4 * c + 2], out[4 * c + 3]);
        }
    }
}

// ------------------------------------------------------------------------- scores
struct ScoreArgs {
    const uint16_t* query;      // bf16 [B][Hk*QG][128]
    const uint8_t* summaries;   // [NB][Hk][2][128] bf16
    const int* block_table;
    const int* context_lens;
    float* scores;              // [B][Hk][MB]
    int* err_word;
    long long NB;
    int Hk, QG, MB, BS;
    int ctas;                   // CTAs per (sequence, KV head)
    float scale;
};

constexpr int kScoreWarps = 4;

// A warp takes 16 blocks of one (sequence, KV head) at a time: m16n8k16 with the blocks as M, the
// query rows as N (NT tiles of 8) and the 256 products as K.  Any order of K serves as long as both
// operands use it: lane (gid, tig) takes the 16-byte words tig, tig + 4, ... of the summary rows gid
// and gid + 8 as they lie in memory (16 independent loads, 8 KB per warp in flight), and its B
// fragments hold the same dimensions of [q+ | q-]; a bf16 value's part is itself or zero, so both
// operands are exact and the sums are fp32.  Bound by HBM: 512 bytes per block and head, read once
// (52 MB of them, 16 sequences of up to 32768 tokens: 10.1 us, 5.1 TB/s; three CTAs per SM and as many as are
// resident at once, against 12.2 us with six and 1.4 waves; two tiles of words in flight per warp: 12 us;
// 32-byte loads: 11.2 us).
__device__ __forceinline__ uint4 load_once(const uint4* p) {   // in program order: every load before the first use
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
template <int NT>
__global__ void __launch_bounds__(kScoreWarps * 32, 3) pda_score_kernel(const ScoreArgs a) {
    allow_dependent_launch();
    grid_dependency_wait();
    const int unit = blockIdx.x / a.ctas, cta = blockIdx.x - unit * a.ctas;
    const int b = unit / a.Hk, h = unit - b * a.Hk;
    const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
    const int ctx = clean_ctx(__ldg(a.context_lens + b), a.MB * a.BS, a.err_word,
                              h == 0 && cta == 0 && threadIdx.x == 0);
    const int nb = (ctx + a.BS - 1) / a.BS, tiles = (nb + 15) >> 4;
    int tile = cta * kScoreWarps + (threadIdx.x >> 5);
    if (tile >= tiles) return;
    // word tig + 4i of a summary row: dimensions 8(tig + 4i) .. +7 of kmax (i < 4) or kmin
    uint32_t qf[NT][8][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = n * 8 + gid;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (r < a.QG)
                v = __ldg(reinterpret_cast<const uint4*>(a.query + (((long long)b * a.Hk + h) * a.QG + r) * kHeadDim) +
                          tig + 4 * i);
            const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t neg = ((x[c] >> 15) & 0x00010001u) * 0xFFFFu;   // halves with the sign bit
                qf[n][i][c] = x[c] & ~neg;
                qf[n][i + 4][c] = x[c] & neg;
            }
        }
    }
    const int* table = a.block_table + (long long)b * a.MB;
    float* out = a.scores + (long long)unit * a.MB;
    for (; tile < tiles; tile += a.ctas * kScoreWarps) {
        const int j0 = tile * 16 + gid, j1 = j0 + 8;
        int id0 = j0 < nb ? __ldg(table + j0) : 0, id1 = j1 < nb ? __ldg(table + j1) : 0;
        const bool bad0 = id0 < 0 || id0 >= a.NB, bad1 = id1 < 0 || id1 >= a.NB;
        if ((bad0 || bad1) && h == 0 && tig == 0 && a.err_word) atomicOr(a.err_word, PDA_ERRW_BAD_BLOCK_ID);
        if (bad0) id0 = 0;
        if (bad1) id1 = 0;
        const uint4* r0 = reinterpret_cast<const uint4*>(a.summaries + ((long long)id0 * a.Hk + h) * kSumBytes) + tig;
        const uint4* r1 = reinterpret_cast<const uint4*>(a.summaries + ((long long)id1 * a.Hk + h) * kSumBytes) + tig;
        uint4 v0[8], v1[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v0[i] = load_once(r0 + 4 * i);
            v1[i] = load_once(r1 + 4 * i);
        }
        float d[NT][2][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) d[n][0][c] = d[n][1][c] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mma_bf16(d[n][0], v0[i].x, v1[i].x, v0[i].y, v1[i].y, qf[n][i][0], qf[n][i][1]);
                mma_bf16(d[n][1], v0[i].z, v1[i].z, v0[i].w, v1[i].w, qf[n][i][2], qf[n][i][3]);
            }
        float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c)
                if (n * 8 + 2 * tig + c < a.QG) {
                    m0 = fmaxf(m0, d[n][0][c] + d[n][1][c]);
                    m1 = fmaxf(m1, d[n][0][c + 2] + d[n][1][c + 2]);
                }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            m0 = fmaxf(m0, __shfl_xor_sync(kAll, m0, o));
            m1 = fmaxf(m1, __shfl_xor_sync(kAll, m1, o));
        }
        if (tig == 0 && j0 < nb) out[j0] = bad0 ? -INFINITY : m0 * a.scale;
        if (tig == 1 && j1 < nb) out[j1] = bad1 ? -INFINITY : m1 * a.scale;
    }
}

// ------------------------------------------------------------------------- selection
struct SelectArgs {
    const float* scores;   // [B][Hk][MB]
    const int* block_table;
    const int* context_lens;
    int* sel_table;        // [B][Hk][K] physical ids, ascending in the sequence, then -1
    int* sel_lens;         // [B][Hk] tokens
    int* sel_blocks;       // [B][Hk][K] logical indices or null
    int* err_word;
    int Hk, MB, BS, K, first, last;
    int staged;            // keys that fit the launch's shared memory
};

// An unsigned key in the order of the scores: NaN lowest, -0 as +0.
__device__ __forceinline__ uint32_t score_key(float x) {
    if (x != x) return 0u;
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u >> 31) ? ~u : u | 0x80000000u;
}

constexpr int kSelThreads = 256;

// One CTA per (sequence, KV head).  The forced blocks apart, the need-th largest key is found by passes
// over 8-bit digits of its distance from the least key, from the highest bit that differs on (the scores of
// one row lie close together: their own leading digits would tell nothing apart), with a histogram in shared
// memory, until a digit's whole bin is wanted or its keys are few enough to be ranked one by one.  Then every
// thread takes a run of consecutive blocks, counts its larger and its equal ones, and one scan gives each
// selected block its place in ascending order; of the equal ones the first in the sequence are taken.
// Bound by latency: a row's scores are a few KB (128 rows of up to 1024 blocks: 6.6 us; 9.1 us with four passes
// over the keys' own digits whose equal ones the lanes matched, 7.7 us without the ranking).
__global__ void __launch_bounds__(kSelThreads) pda_select_kernel(const SelectArgs a) {
    extern __shared__ uint32_t keys[];
    __shared__ uint32_t hist[256];
    __shared__ uint32_t sums[kSelThreads / 32], tops[kSelThreads / 32];
    __shared__ unsigned long long sums64[kSelThreads / 32];
    __shared__ uint32_t pick, left, count;
    allow_dependent_launch();
    grid_dependency_wait();
    const int b = blockIdx.x / a.Hk, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool lead = blockIdx.x == (unsigned)(b * a.Hk) && tid == 0;
    const int ctx = clean_ctx(__ldg(a.context_lens + b), a.MB * a.BS, a.err_word, lead);
    const int nb = (ctx + a.BS - 1) / a.BS, c = min(a.K, nb);
    const int lo = min(a.first, nb), hi = max(lo, nb - a.last);   // blocks [lo, hi) compete
    const float* row = a.scores + (long long)blockIdx.x * a.MB;
    const int* table = a.block_table + (long long)b * a.MB;
    int* out = a.sel_table + (long long)blockIdx.x * a.K;
    int* outb = a.sel_blocks ? a.sel_blocks + (long long)blockIdx.x * a.K : nullptr;
    const int n = hi - lo;
    const bool all = c == nb, staged = n <= a.staged;
    const uint32_t need0 = (uint32_t)(c - (nb - n));   // of the competing blocks (c >= the forced ones)

    uint32_t T = 0, mask = 0, need = need0, base = 0;
    auto key_of = [&](int i) { return (staged ? keys[i] : score_key(__ldg(row + lo + i))) - base; };
    if (!all && need0 > 0) {
        uint32_t least = 0xFFFFFFFFu, most = 0u;
        for (int i = tid; i < n; i += kSelThreads) {
            const uint32_t k = score_key(__ldg(row + lo + i));
            if (staged) keys[i] = k;
            least = min(least, k);
            most = max(most, k);
        }
        least = __reduce_min_sync(kAll, least);
        most = __reduce_max_sync(kAll, most);
        if (lane == 0) {
            sums[warp] = least;
            tops[warp] = most;
        }
        __syncthreads();
        for (int w = 0; w < kSelThreads / 32; ++w) {
            least = min(least, sums[w]);
            most = max(most, tops[w]);
        }
        base = least;
        const int bits = 32 - __clz(most - least);   // 0: every key is the same
        for (int shift = max(0, bits - 8); bits > 0; shift = max(0, shift - 8)) {
            hist[tid] = 0u;
            __syncthreads();
            for (int i = tid; i < n; i += kSelThreads) {
                const uint32_t k = key_of(i);
                if ((k & mask) == T) atomicAdd(hist + ((k >> shift) & 255u), 1u);
            }
            __syncthreads();
            // from the top: thread t holds digit 255 - t
            const uint32_t mine = hist[255 - tid];
            uint32_t v = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t x = __shfl_up_sync(kAll, v, o);
                if (lane >= o) v += x;
            }
            if (lane == 31) sums[warp] = v;
            __syncthreads();
            for (int w = 0; w < warp; ++w) v += sums[w];
            if (v >= need && v - mine < need) {
                pick = (uint32_t)(255 - tid);
                left = need - (v - mine);
            }
            __syncthreads();
            T |= pick << shift;
            mask |= 255u << shift;
            need = left;
            const uint32_t bin = hist[pick];
            if (tid == 0) count = 0u;
            __syncthreads();
            if (need == bin || shift == 0) break;   // every key with these digits is wanted, or no digit is left
            if (bin <= kSelThreads) {               // few enough for a thread each: they rank themselves
                for (int i = tid; i < n; i += kSelThreads) {
                    const uint32_t k = key_of(i);
                    if ((k & mask) == T) hist[atomicAdd(&count, 1u)] = k;
                }
                __syncthreads();
                if (tid < (int)bin) {
                    const uint32_t k = hist[tid];
                    uint32_t above = 0, same = 0;
                    for (uint32_t i = 0; i < bin; ++i) {
                        above += hist[i] > k;
                        same += hist[i] == k;
                    }
                    if (above < need && need <= above + same) {   // threads with this key all write the same
                        pick = k;
                        left = need - above;
                    }
                }
                __syncthreads();
                T = pick;
                mask = 0xFFFFFFFFu;
                need = left;
                break;
            }
        }
    }
    // larger: (key & mask) > T; equal: (key & mask) == T, the first `need` of them
    const int per = (nb + kSelThreads - 1) / kSelThreads;
    const int j0 = min(nb, tid * per), j1 = min(nb, j0 + per);
    auto kind = [&](int j) -> int {   // 2 taken, 1 equal, 0 not
        if (all || j < lo || j >= hi) return 2;
        if (need0 == 0) return 0;
        const uint32_t k = key_of(j - lo) & mask;
        return k > T ? 2 : k == T ? 1 : 0;
    };
    unsigned long long mine = 0;   // taken in the high half, equal in the low one
    for (int j = j0; j < j1; ++j) {
        const int k = kind(j);
        mine += k == 2 ? 1ull << 32 : (unsigned long long)k;
    }
    unsigned long long v = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long x = __shfl_up_sync(kAll, v, o);
        if (lane >= o) v += x;
    }
    if (lane == 31) sums64[warp] = v;
    __syncthreads();
    for (int w = 0; w < warp; ++w) v += sums64[w];
    v -= mine;
    uint32_t taken = (uint32_t)(v >> 32), equal = (uint32_t)v;
    int tokens = 0;
    for (int j = j0; j < j1; ++j) {
        const int k = kind(j);
        if (k == 2 || (k == 1 && equal < need)) {
            const uint32_t at = taken + min(equal, need);
            out[at] = __ldg(table + j);
            if (outb) outb[at] = j;
            tokens += min(a.BS, ctx - j * a.BS);
        }
        if (k == 2) ++taken;
        if (k == 1) ++equal;
    }
    for (int i = c + tid; i < a.K; i += kSelThreads) {
        out[i] = -1;
        if (outb) outb[i] = -1;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) tokens += __shfl_xor_sync(kAll, tokens, o);
    if (lane == 0) sums[warp] = (uint32_t)tokens;
    __syncthreads();
    if (tid == 0) {
        int t = 0;
        for (int w = 0; w < kSelThreads / 32; ++w) t += (int)sums[w];
        a.sel_lens[blockIdx.x] = t;
    }
}

// ------------------------------------------------------------------------- host side
template <class K, class A>
static int launch_pdl(K kernel, const A& args, dim3 grid, int threads, int smem, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args) == cudaSuccess ? PDA_OK : PDA_ERR_LAUNCH;
}

static bool off(const void* p, unsigned a) { return ((uintptr_t)p & (a - 1)) != 0; }
static bool bad_pool(long long nb) { return nb < 1 || nb > (1ll << 31) - 1; }

}  // namespace pda

using namespace pda;

extern "C" {

long long pda_summary_size(const pda_plan_t* plan, long long num_cache_blocks) {
    if (!plan || pda_workspace_size(plan) < 0 || bad_pool(num_cache_blocks)) return -1;
    return num_cache_blocks * plan->num_kv_heads * kSumBytes;
}

int pda_summarize_blocks(const pda_plan_t* plan, const void* kv_cache, long long num_cache_blocks,
                         const int* block_table, const int* context_lens, const int* since, const float* centroids,
                         void* summaries, int* err_word, void* stream) {
    if (!plan || pda_workspace_size(plan) < 0) return PDA_ERR_INVALID_ARG;
    const bool tq = plan->kv_dtype == PDA_KV_TQ4;
    if (tq != (centroids != nullptr)) return PDA_ERR_INVALID_ARG;
    if (plan->num_seqs == 0) return PDA_OK;
    if (!kv_cache || !block_table || !context_lens || !summaries || bad_pool(num_cache_blocks)) return PDA_ERR_INVALID_ARG;
    if (off(kv_cache, 16) || off(summaries, 16) || off(block_table, 4) || off(context_lens, 4) || off(since, 4) ||
        off(centroids, 4) || off(err_word, 4))
        return PDA_ERR_INVALID_ARG;
    const int sms = device_sm_count();
    if (sms <= 0) return PDA_ERR_CUDA;
    // how many blocks are new is known on the device only: about one wave of CTAs, shared by the sequences
    const long long want = ((long long)plan->max_blocks_per_seq * plan->num_kv_heads + 7) / 8;
    const long long cap = (4ll * sms + plan->num_seqs - 1) / plan->num_seqs;
    const int ctas = (int)(want < cap ? want : cap);
    const SumArgs a{static_cast<const uint8_t*>(kv_cache), block_table, context_lens, since, centroids,
                    static_cast<uint8_t*>(summaries), err_word, num_cache_blocks, plan->cache_block_bytes,
                    plan->meta_offset_bytes, plan->num_kv_heads, plan->max_blocks_per_seq, plan->kv_block_size, ctas};
    const long long total = (long long)ctas * plan->num_seqs;
    if (total > (1ll << 31) - 1) return PDA_ERR_INVALID_ARG;
    const dim3 grid((unsigned)total);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool big = plan->kv_block_size == 32;
    if (plan->kv_dtype == PDA_KV_BF16)
        return big ? launch_pdl(pda_summarize_kernel<PDA_KV_BF16, 32>, a, grid, 256, 0, s)
                   : launch_pdl(pda_summarize_kernel<PDA_KV_BF16, 16>, a, grid, 256, 0, s);
    if (tq)
        return big ? launch_pdl(pda_summarize_kernel<PDA_KV_TQ4, 32>, a, grid, 256, 0, s)
                   : launch_pdl(pda_summarize_kernel<PDA_KV_TQ4, 16>, a, grid, 256, 0, s);
    return big ? launch_pdl(pda_summarize_kernel<PDA_KV_FP8_E4M3, 32>, a, grid, 256, 0, s)
               : launch_pdl(pda_summarize_kernel<PDA_KV_FP8_E4M3, 16>, a, grid, 256, 0, s);
}

int pda_score_blocks(const pda_plan_t* plan, const void* query, const void* summaries, long long num_cache_blocks,
                     const int* block_table, const int* context_lens, float* scores, int* err_word, void* stream) {
    if (!plan || pda_workspace_size(plan) < 0) return PDA_ERR_INVALID_ARG;
    if (plan->num_seqs == 0) return PDA_OK;
    if (!query || !summaries || !block_table || !context_lens || !scores || bad_pool(num_cache_blocks))
        return PDA_ERR_INVALID_ARG;
    if (off(query, 16) || off(summaries, 16) || off(block_table, 4) || off(context_lens, 4) || off(scores, 4) ||
        off(err_word, 4))
        return PDA_ERR_INVALID_ARG;
    const long long units = (long long)plan->num_seqs * plan->num_kv_heads;
    const int sms = device_sm_count();
    if (sms <= 0) return PDA_ERR_CUDA;
    const long long want = (plan->max_blocks_per_seq + 16 * kScoreWarps - 1) / (16 * kScoreWarps);
    const long long cap = (3ll * sms + units - 1) / units;
    const int ctas = (int)(want < cap ? want : cap);
    if (ctas * units > (1ll << 31) - 1) return PDA_ERR_INVALID_ARG;
    const dim3 grid((unsigned)(ctas * units));
    const ScoreArgs a{static_cast<const uint16_t*>(query), static_cast<const uint8_t*>(summaries), block_table,
                      context_lens, scores, err_word, num_cache_blocks, plan->num_kv_heads, plan->query_group_size,
                      plan->max_blocks_per_seq, plan->kv_block_size, ctas, plan->resolved_softmax_scale};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return plan->query_group_size <= 8 ? launch_pdl(pda_score_kernel<1>, a, grid, kScoreWarps * 32, 0, s)
                                       : launch_pdl(pda_score_kernel<2>, a, grid, kScoreWarps * 32, 0, s);
}

int pda_select_blocks(const pda_plan_t* plan, const float* scores, const int* block_table, const int* context_lens,
                      int num_select, int num_first, int num_last, int* sel_table, int* sel_lens, int* sel_blocks,
                      int* err_word, void* stream) {
    if (!plan || pda_workspace_size(plan) < 0) return PDA_ERR_INVALID_ARG;
    if (num_select < 1 || num_first < 0 || num_last < 0 || (long long)num_first + num_last > num_select ||
        (long long)num_select * plan->kv_block_size > (1ll << 30))
        return PDA_ERR_INVALID_ARG;
    if (plan->num_seqs == 0) return PDA_OK;
    if (!scores || !block_table || !context_lens || !sel_table || !sel_lens) return PDA_ERR_INVALID_ARG;
    if (off(scores, 4) || off(block_table, 4) || off(context_lens, 4) || off(sel_table, 4) || off(sel_lens, 4) ||
        off(sel_blocks, 4) || off(err_word, 4))
        return PDA_ERR_INVALID_ARG;
    constexpr int kMaxStaged = 40960 / 4;   // keys kept in shared memory: 40 KB, no opt-in needed
    const int staged = plan->max_blocks_per_seq <= kMaxStaged ? plan->max_blocks_per_seq : 0;
    const SelectArgs a{scores, block_table, context_lens, sel_table, sel_lens, sel_blocks, err_word, plan->num_kv_heads,
                       plan->max_blocks_per_seq, plan->kv_block_size, num_select, num_first, num_last, staged};
    const long long units = (long long)plan->num_seqs * plan->num_kv_heads;
    return launch_pdl(pda_select_kernel, a, dim3((unsigned)units), kSelThreads, staged * 4,
                      static_cast<cudaStream_t>(stream));
}

}  // extern "C"
