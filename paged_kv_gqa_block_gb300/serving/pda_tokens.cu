// pda_tokens.cu -- tokens of the cache, many at a time: pda_write_kv (stored in the cache's format), pda_read_kv (gathered
// and dequantised) and pda_accept_tokens (the accepted path of drafted tokens moves to consecutive positions).
//
// The formats, per token and KV head, K and V apart:
//   bf16   as given
//   e4m3   scale = max |x| / 448 (1 for a row of zeros), code = e4m3(x / scale): pda_append_kv's arithmetic, division by
//          division, so that a token has the same bytes whichever call wrote it
//   TQ4    K: k_norm = f16(|k|), code = the number of midpoints of neighbouring centroids below fp32(k_d / k_norm)
//          V: v_zero = f16(min v), v_scale = f16((max v - min v) / 15), code = rint((v_d - v_zero) / v_scale) in 0 .. 15
// Every quotient is that of an IEEE division and |k| is rounded once, from 64 bits where 32 cannot tell to which f16 value, so
// that the codes are a function of the values alone: two writes of one token, on any grid, give the same bytes.
//
// A warp takes up to four KV heads of one token at a time, whose loads are asked for together: addresses are computed once per token
// (a search of token_starts and the block table's entry, by one thread), and a whole row leaves in one or two store instructions.
// Measured, 131072 tokens of 8 heads: written in bf16 160 us (6.7 TB/s: HBM), fp8 164 us (5.0 TB/s), TQ4 288 us (2.4 TB/s: 276
// instructions per row, 71 % of the issue slots used); read back from bf16 159 us, fp8 124 us (6.6 TB/s), TQ4 138 us (4.9 TB/s: a conversion per code).
// 16 prompts of up to 4096 tokens into fp8 22 us, 16 contexts of up to 8192 fp8 tokens back 42 us (6.1 TB/s), up to nine tokens of
// 8 sequences 2.8 us.
#include <cuda_runtime.h>

#include <cstdint>

#include "pda.h"
#include "pda_internal.h"
#include "pda_ptx.cuh"

namespace pda {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kTokThreads = 256;
constexpr int kTokWarps = kTokThreads / 32;
constexpr int kMaxTokensPerCta = 32, kManyReads = 16;
constexpr int kHeadsAhead = 4;            // KV heads of one token that a warp takes together, at most, loads first

struct TokenArgs {
    uint8_t* cache;              // read_kv does not write it
    const int* block_table;      // [B][MB]
    const int* token_starts;     // [B + 1]
    const int* positions;        // [B]
    const float* centroids;      // TQ4: [16]
    int* err_word;
    const uint16_t* k_new;       // write: rows k_stride elements apart
    const uint16_t* v_new;
    void* k_out;                 // read: [N][Hk][128]
    void* v_out;
    long long k_stride, v_stride;
    long long num_cache_blocks, cache_block_bytes, meta_offset_bytes;
    int num_tokens, B, Hk, MB, BS, bs_shift, per_cta;
    int ahead, groups;           // KV heads of an item, and items of a token
    unsigned long long by_groups; // 2^32 / groups, rounded up (0 where a CTA has one token)
};

// Where the CTA's tokens lie in the pool: byte offset of the token's row (head 0) and of its first field, or a negative
// offset for a token that is no sequence's or has no place.  False (in every thread) where token_starts do not ascend within [0, num_tokens].
struct Places {
    long long row[kMaxTokensPerCta], field[kMaxTokensPerCta];
};
__device__ __forceinline__ bool find_places(const TokenArgs& a, Places& at, int first, int n, int row_bytes,
                                            int field_bytes) {
    bool bad = false;
    for (int b = threadIdx.x; b <= a.B; b += kTokThreads) {
        const int s = __ldg(a.token_starts + b);
        bad |= s < 0 || s > a.num_tokens || (b < a.B && __ldg(a.token_starts + b + 1) < s);
    }
    if (__syncthreads_or(bad)) {
        if (blockIdx.x == 0 && threadIdx.x == 0 && a.err_word) atomicOr(a.err_word, PDA_ERRW_BAD_TOKENS);
        return false;
    }
    if ((int)threadIdx.x < n) {
        const int i = first + threadIdx.x;
        int lo = 0, hi = a.B + 1;   // the number of starts that are not above i
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (__ldg(a.token_starts + mid) <= i)
                lo = mid + 1;
            else
                hi = mid;
        }
        const int b = lo - 1;
        long long row = -1, field = 0;
        if (b >= 0 && b < a.B) {
            const int p0 = __ldg(a.positions + b);
            const long long pos = (long long)p0 + (i - __ldg(a.token_starts + b));
            if (p0 >= 0) {
                if (pos >= (long long)a.MB * a.BS) {
                    if (a.err_word) atomicOr(a.err_word, PDA_ERRW_BAD_POSITION);
                } else {
                    const int id = __ldg(a.block_table + (long long)b * a.MB + (pos >> a.bs_shift));
                    if (id < 0 || id >= a.num_cache_blocks) {
                        if (a.err_word) atomicOr(a.err_word, PDA_ERRW_BAD_BLOCK_ID);
                    } else {
                        const int slot = (int)pos & (a.BS - 1);
                        row = id * a.cache_block_bytes + (long long)slot * a.Hk * row_bytes;
                        field = id * a.cache_block_bytes + a.meta_offset_bytes + slot * field_bytes;
                    }
                }
            }
        }
        at.row[threadIdx.x] = row;
        at.field[threadIdx.x] = field;
    }
    __syncthreads();
    return true;
}

// What a warp takes at a time: up to kHeadsAhead KV heads of one token.  Their rows lie a fixed number of bytes apart, so that one
// address serves all; item x of a CTA is group x % groups of its token x / groups (x < 32 groups, and groups <= 4096 where a CTA has
// more than one token, so the rounded-up inverse is exact).
struct Item {
    int t, h, n;   // token of the CTA, first KV head, KV heads
    __device__ __forceinline__ Item(const TokenArgs& a, int x)
        : t((int)(x * a.by_groups >> 32)), h((x - t * a.groups) * a.ahead), n(min(a.ahead, a.Hk - h)) {}
};

// ------------------------------------------------------------------------- writing
// x / b rounded to the nearest fp32 value, for many x: r is 1 / b rounded.  Each step adds the remainder over b, which an fma
// gives exactly; with r correctly rounded and a quotient within one unit in its last place the result is correctly rounded
// (Markstein), and the first step takes x * r, off by two half units, there.  Holds while no remainder underflows; where
// the quotient is too small for that, what it is used for does not depend on its last place (see the callers).
__device__ __forceinline__ float quotient(float x, float b, float r) {
    float q = __fmul_rn(x, r);
    q = __fmaf_rn(__fmaf_rn(-q, b, x), r, q);
    return __fmaf_rn(__fmaf_rn(-q, b, x), r, q);
}
// The sorted codebook: midpoints of neighbours (15, then +inf) and the code of each rank.
struct __align__(16) Codebook {
    float mid[16];
    uint32_t code[16];
    int plain;   // no midpoint but 0 is below 2^-60
    int ascending;   // the codes are the ranks
};
__device__ __forceinline__ void sort_codebook(const float* centroids, Codebook& book, float* sorted) {
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        const float c = __ldg(centroids + (lane & 15));   // lanes 16 .. 31: not looked at
        int rank = 0;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float o = __shfl_sync(kAll, c, j);
            rank += o < c || (o == c && j < lane);
        }
        if (lane < 16) {
            sorted[rank] = c;
            book.code[rank] = lane;
        }
        __syncwarp();
        const float mid = lane < 15 ? __fmul_rn(__fadd_rn(sorted[lane], sorted[lane + 1]), 0.5f) : INFINITY;
        if (lane < 16) book.mid[lane] = mid;
        const bool plain = __all_sync(kAll, lane >= 15 || mid == 0.f || fabsf(mid) >= 8.6736174e-19f);
        const bool ascending = __all_sync(kAll, lane >= 16 || rank == lane);
        if (lane == 0) {
            book.plain = plain;
            book.ascending = ascending;
        }
    }
}

// The smaller of two bf16 values each, of zeros the negative one.
__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float f16_saturated(float x) {
    return __half2float(__float2half_rn(fminf(fmaxf(x, -65504.f), 65504.f)));
}

// fp8: lane l < 16 holds K's dimensions 8l .. 8l+7, lane 16 + l V's.  Bound by instructions (HBM would take two thirds of the time),
// so a value is divided by its row's inverse and two exact remainders, five instructions: a quotient whose remainder underflows is far
// below e4m3's smallest.  (Codes from products a little too small and a little too large, and quotients only where the two differ, were
// slower: bf16 values have few mantissas, their quotients meet e4m3's ties often, and a row of four was left open; 16 prompts of up to 4096
// tokens 26 us and not 22.)  Rows that are tiny or hold infinities or NaN are divided.
__device__ __forceinline__ void write_fp8(uint8_t* row, float* scales, uint4 raw, int lane, int BS) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    // magnitudes of bf16 values are ordered like their bits
    const uint32_t mx = __vmaxs2(__vmaxs2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu), __vmaxs2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
    int top = max(mx & 0xFFFFu, mx >> 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(kAll, top, o));
    const float most = __uint_as_float((uint32_t)top << 16);
    float scale = top > 0 ? quotient(most, 448.f, 1.f / 448.f) : 1.f;   // of a normal number that counts
    uint32_t a, b;
    const bool odd = !(most > 1e-25f && top < 0x7F80);   // the same in the half warp
    if (odd) {   // pda_append_kv's maximum and division; fmaxf passes NaN by
        const uint32_t mine = 0xFFFFu << (lane & 16);
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(mine, m, o));
        scale = m > 0.f ? __fdiv_rn(m, 448.f) : 1.f;
        auto code = [&](uint32_t v) { return f32x2_to_e4m3x2(__fdiv_rn(bf16_lo(v), scale), __fdiv_rn(bf16_hi(v), scale)); };
        a = code(w[0]) | code(w[1]) << 16;
        b = code(w[2]) | code(w[3]) << 16;
    } else {
        const float by = __frcp_rn(scale);
        auto code = [&](uint32_t v) { return f32x2_to_e4m3x2(quotient(bf16_lo(v), scale, by), quotient(bf16_hi(v), scale, by)); };
        // the sign of a zero does not outlive its remainder, so signs are those of the values
        a = code(w[0]) | code(w[1]) << 16 | (__byte_perm(w[0], w[1], 0x7531) & 0x80808080u);
        b = code(w[2]) | code(w[3]) << 16 | (__byte_perm(w[2], w[3], 0x7531) & 0x80808080u);
    }
    *reinterpret_cast<uint2*>(row + 8 * lane) = make_uint2(a, b);
    if ((lane & 15) == 0) scales[(lane >> 4) * BS] = scale;
}

// TQ4: a half warp writes a row, lane l of it dimensions 8l .. 8l+7 of K and of V; the other half another row, so that what is done
// once per row (reductions, roots, inverses) is shared by two.  Bound by instructions.
__device__ __forceinline__ void write_tq4(uint8_t* row, uint16_t* fields, bool live, uint4 kraw, uint4 vraw, const Codebook& book, int l,
                                          int BS) {
    const uint32_t kw[4] = {kraw.x, kraw.y, kraw.z, kraw.w}, vw[4] = {vraw.x, vraw.y, vraw.z, vraw.w};
    float sum, part[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) part[i] = fmaf(bf16_hi(kw[i]), bf16_hi(kw[i]), bf16_lo(kw[i]) * bf16_lo(kw[i]));
    sum = (part[0] + part[1]) + (part[2] + part[3]);
    // the smallest V, and the smallest of -V, as bf16 pairs: both exact
    uint32_t low = min_bf16x2(min_bf16x2(vw[0], vw[1]), min_bf16x2(vw[2], vw[3]));
    uint32_t high = min_bf16x2(min_bf16x2(vw[0] ^ 0x80008000u, vw[1] ^ 0x80008000u), min_bf16x2(vw[2] ^ 0x80008000u, vw[3] ^ 0x80008000u));
    uint32_t both = min_bf16x2(__byte_perm(low, high, 0x5410), __byte_perm(low, high, 0x7632));   // low halves, high halves
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(kAll, sum, o);
        both = min_bf16x2(both, __shfl_xor_sync(kAll, both, o));
    }
    const float lo = bf16_lo(both), hi = -bf16_hi(both);
    // |k| is rounded to f16 once: eight fp32 roundings of positive terms and the root are off by less than 2^-20, and where
    // that does not decide the f16 value (one row in a thousand) the sum is taken again in 64 bits.  The sum is the same in
    // every lane of the row (a butterfly adds the same pairs).
    const float root = sqrtf(sum);
    uint16_t norm_bits = __half_as_ushort(__float2half_rn(fminf(root, 65504.f)));
    const float up = fminf(__fmul_rn(root, 1.f + 9.5367431640625e-7f), 65504.f);
    const float down = fminf(__fmul_rn(root, 1.f - 9.5367431640625e-7f), 65504.f);
    const bool open = __half_as_ushort(__float2half_rn(up)) != __half_as_ushort(__float2half_rn(down));
    if (__any_sync(kAll, open)) {
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < 4; ++i) s += (double)bf16_lo(kw[i]) * (double)bf16_lo(kw[i]) + (double)bf16_hi(kw[i]) * (double)bf16_hi(kw[i]);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
        // by way of fp32 without rounding twice: cut, and odd where something was cut off
        const double exact = fmin(sqrt(s), 65504.0);
        float cut = __double2float_rz(exact);
        if ((double)cut != exact) cut = __uint_as_float(__float_as_uint(cut) | 1u);
        if (open) norm_bits = __half_as_ushort(__float2half_rn(cut));
    }
    const float norm = __half2float(__ushort_as_half(norm_bits));
    const float by = norm > 0.f ? norm : 1.f, rk = __frcp_rn(by);
    uint32_t kc = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // |k| is at most the norm, or the norm is 65504: nothing overflows; a quotient below 2^-61 lies between the same midpoints
        // whatever its last places
        const float k = i & 1 ? bf16_hi(kw[i >> 1]) : bf16_lo(kw[i >> 1]), x = book.plain ? quotient(k, by, rk) : __fdiv_rn(k, by);
        // midpoints 7, then 3 or 11, then the three of one quarter at once
        const bool upper = book.mid[7] < x;
        const int q = (upper ? 2 : 0) + ((upper ? book.mid[11] : book.mid[3]) < x ? 1 : 0);
        const float4 m = *reinterpret_cast<const float4*>(book.mid + 4 * q);
        const int rank = 4 * q + (m.x < x ? 1 : 0) + (m.y < x ? 1 : 0) + (m.z < x ? 1 : 0);
        kc |= (book.ascending ? (uint32_t)rank : book.code[rank]) << (4 * i);
    }
    const float zero = f16_saturated(lo), step = f16_saturated(__fdiv_rn(__fsub_rn(hi, lo), 15.f));
    const float vby = step > 0.f ? step : 1.f, rv = __frcp_rn(vby);   // at least f16's smallest, 2^-24
    uint32_t vc = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // brought into 0 .. 15, then rounded by the sum with 1.5 * 2^23, whose last bits are the integer
        const float v = i & 1 ? bf16_hi(vw[i >> 1]) : bf16_lo(vw[i >> 1]);
        const float c = fminf(fmaxf(quotient(__fsub_rn(v, zero), vby, rv), 0.f), 15.f);
        vc |= (__float_as_uint(__fadd_rn(c, 12582912.f)) & 15u) << (4 * i);
    }
    if (!live) return;
    *reinterpret_cast<uint32_t*>(row + 4 * l) = kc;
    *reinterpret_cast<uint32_t*>(row + 64 + 4 * l) = vc;
    if (l < 3) {
        const uint16_t f = l == 0 ? norm_bits : __half_as_ushort(__float2half_rn(l == 1 ? step : zero));
        fields[l * BS] = f;
    }
}

template <int KV>
__global__ void __launch_bounds__(kTokThreads) pda_write_kernel(const TokenArgs a) {
    __shared__ Places at;
    __shared__ Codebook book;
    __shared__ float sorted[16];
    constexpr int kRow = KV == PDA_KV_BF16 ? 512 : KV == PDA_KV_FP8_E4M3 ? 256 : 128;   // K and V of one head
    const int first = blockIdx.x * a.per_cta, n = min(a.per_cta, a.num_tokens - first);
    if constexpr (KV == PDA_KV_TQ4) sort_codebook(a.centroids, book, sorted);
    if (!find_places(a, at, first, n, kRow, KV == PDA_KV_FP8_E4M3 ? 4 : 2)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int item = warp; item < n * a.groups; item += kTokWarps) {
        const Item x(a, item);
        if (at.row[x.t] < 0) continue;
        const uint16_t* k = a.k_new + (first + x.t) * a.k_stride + x.h * kHeadDim;
        const uint16_t* v = a.v_new + (first + x.t) * a.v_stride + x.h * kHeadDim;
        uint4 raw[kHeadsAhead];   // eight dimensions of K or V; TQ4: of K and V of every other head
        const int half = lane >> 4, l = lane & 15;
#pragma unroll
        for (int i = 0; i < kHeadsAhead; ++i) {
            if constexpr (KV == PDA_KV_TQ4) {
                const int head = min((i & ~1) + half, x.n - 1);   // an odd last one is taken twice, and written once
                if ((i & ~1) < x.n) raw[i] = __ldg(reinterpret_cast<const uint4*>((i & 1 ? v : k) + head * kHeadDim) + l);
            } else if (i < x.n) {
                raw[i] = __ldg(reinterpret_cast<const uint4*>((lane < 16 ? k : v) + i * kHeadDim) + l);
            }
        }
        uint8_t* row = a.cache + at.row[x.t] + (long long)x.h * kRow;
        uint8_t* field = a.cache + at.field[x.t];
#pragma unroll
        for (int i = 0; i < kHeadsAhead; ++i)
            if (i < x.n) {
                if constexpr (KV == PDA_KV_TQ4) {
                    if (i & 1) continue;
                    const int head = i + half;
                    write_tq4(row + head * kRow, reinterpret_cast<uint16_t*>(field) + (x.h + head) * 3 * a.BS, head < x.n, raw[i], raw[i + 1],
                              book, l, a.BS);
                } else if constexpr (KV == PDA_KV_BF16)
                    *reinterpret_cast<uint4*>(row + i * kRow + 16 * lane) = raw[i];
                else
                    write_fp8(row + i * kRow, reinterpret_cast<float*>(field) + (x.h + i) * 2 * a.BS, raw[i], lane, a.BS);
            }
    }
}

// ------------------------------------------------------------------------- reading
// Lane l < 16 reads dimensions 8l .. 8l+7 of K, lane 16 + l those of V.
template <int KV, bool F32>
__global__ void __launch_bounds__(kTokThreads) pda_read_kernel(const TokenArgs a) {
    __shared__ Places at;
    __shared__ float book[16];
    constexpr int kRow = KV == PDA_KV_BF16 ? 512 : KV == PDA_KV_FP8_E4M3 ? 256 : 128;
    const int first = blockIdx.x * a.per_cta, n = min(a.per_cta, a.num_tokens - first);
    if (KV == PDA_KV_TQ4 && threadIdx.x < 16) book[threadIdx.x] = __ldg(a.centroids + threadIdx.x);
    if (!find_places(a, at, first, n, kRow, KV == PDA_KV_FP8_E4M3 ? 4 : 2)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = lane >> 4, l = lane & 15;
    void* const out = half ? a.v_out : a.k_out;
    for (int item = warp; item < n * a.groups; item += kTokWarps) {
        const Item at_heads(a, item);
        if (at.row[at_heads.t] < 0 || !out) continue;
        const uint8_t* row = a.cache + at.row[at_heads.t] + (long long)at_heads.h * kRow;
        const uint8_t* field = a.cache + at.field[at_heads.t];
        uint4 raw[kHeadsAhead];                // fp8: x, y, TQ4: x
        float m[kHeadsAhead], z[kHeadsAhead];  // fp8: the scale; TQ4: k_norm, or v_scale and v_zero
#pragma unroll
        for (int i = 0; i < kHeadsAhead; ++i)
            if (i < at_heads.n) {
                if constexpr (KV == PDA_KV_BF16) {
                    raw[i] = __ldg(reinterpret_cast<const uint4*>(row + i * kRow) + lane);
                } else if constexpr (KV == PDA_KV_FP8_E4M3) {
                    const uint2 c = __ldg(reinterpret_cast<const uint2*>(row + i * kRow) + lane);
                    raw[i].x = c.x;
                    raw[i].y = c.y;
                    m[i] = __ldg(reinterpret_cast<const float*>(field) + ((at_heads.h + i) * 2 + half) * a.BS);
                } else {
                    const __half* f = reinterpret_cast<const __half*>(field) + (at_heads.h + i) * 3 * a.BS;
                    raw[i].x = __ldg(reinterpret_cast<const uint32_t*>(row + i * kRow) + lane);
                    m[i] = __half2float(__ldg(f + half * a.BS));
                    z[i] = half ? __half2float(__ldg(f + 2 * a.BS)) : 0.f;
                }
            }
        const long long o = ((long long)(first + at_heads.t) * a.Hk + at_heads.h) * kHeadDim + 8 * l;
#pragma unroll
        for (int i = 0; i < kHeadsAhead; ++i)
            if (i < at_heads.n) {
                float x[8];
                if constexpr (KV == PDA_KV_BF16) {
                    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        x[2 * k] = bf16_lo(w[k]);
                        x[2 * k + 1] = bf16_hi(w[k]);
                    }
                } else if constexpr (KV == PDA_KV_FP8_E4M3) {
                    uint32_t p[4];
                    e4m3x4_to_f16x2x2(raw[i].x, p[0], p[1]);
                    e4m3x4_to_f16x2x2(raw[i].y, p[2], p[3]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p[k]));
                        x[2 * k] = f.x * m[i];
                        x[2 * k + 1] = f.y * m[i];
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t code = raw[i].x >> (4 * k) & 15u;
                        x[k] = half ? fmaf((float)code, m[i], z[i]) : book[code] * m[i];   // code * v_scale is exact
                    }
                }
                if constexpr (F32) {
                    float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + o + i * kHeadDim);
                    p[0] = make_float4(x[0], x[1], x[2], x[3]);
                    p[1] = make_float4(x[4], x[5], x[6], x[7]);
                } else {
                    uint4 w = raw[i];
                    if constexpr (KV != PDA_KV_BF16)
                        w = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
                    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + o + i * kHeadDim) = w;
                }
            }
    }
}

// ------------------------------------------------------------------------- accepting
struct AcceptArgs {
    uint8_t* cache;
    const int* block_table;
    const int* context_lens;
    const int* path;             // [B][A]
    const int* path_lens;        // [B]
    int* out_lens;               // [B]
    int* err_word;
    long long num_cache_blocks, cache_block_bytes, meta_offset_bytes;
    int B, MB, BS, bs_shift, A;
    int row_bytes;               // a token's data, all heads
    int fields, field_bytes;     // its metadata: [heads * fields][BS]
};
constexpr int kPathChunk = 128;

// A CTA moves a share of the bytes of one sequence's tokens.  Token k of the path goes from drafted index path[k] >= k to k, in
// the path's order, and every byte is one thread's: a place is read no later than it is overwritten (it is a source only of
// path[k'] = k, k' <= k), so reads may run ahead of the writes and nothing else has to be ordered.  Bound by latency (lengths, path,
// table, tokens): 8 paths 2.7 us, 128 paths out of trees of up to 64 fp8 tokens 3.8 us.
__global__ void __launch_bounds__(kTokThreads) pda_accept_kernel(const AcceptArgs a) {
    __shared__ long long src_block[kPathChunk], dst_block[kPathChunk];
    __shared__ int src_slot[kPathChunk], dst_slot[kPathChunk];
    const int b = blockIdx.x;
    const int* path = a.path + (long long)b * a.A;
    const int ctx = __ldg(a.context_lens + b), n = __ldg(a.path_lens + b);
    const long long room = (long long)a.MB * a.BS;
    int bad = 0;
    if (ctx < 0 || ctx > room) bad |= PDA_ERRW_BAD_CONTEXT_LEN;
    if (n < 0 || n > a.A) bad |= PDA_ERRW_BAD_TOKENS;
    if (!bad)
        for (int k = threadIdx.x; k < n; k += kTokThreads) {
            const int p = __ldg(path + k), before = k ? __ldg(path + k - 1) : -1;
            if (p <= before) bad |= PDA_ERRW_BAD_TOKENS;
            if (p >= room - ctx) bad |= PDA_ERRW_BAD_POSITION;
        }
    const bool refused = __syncthreads_or(bad);
    if (bad && a.err_word) atomicOr(a.err_word, bad);
    if (blockIdx.y == 0 && threadIdx.x == 0) a.out_lens[b] = refused ? ctx : ctx + n;
    if (refused) return;
    const int* table = a.block_table + (long long)b * a.MB;
    const int words = a.row_bytes / 16, metas = a.fields, stride = gridDim.y * kTokThreads;
    const int me = blockIdx.y * kTokThreads + threadIdx.x;
    for (int k0 = 0; k0 < n; k0 += kPathChunk) {
        const int m = min(kPathChunk, n - k0);
        __syncthreads();
        for (int k = threadIdx.x; k < m; k += kTokThreads) {
            const int from = ctx + __ldg(path + k0 + k), to = ctx + k0 + k;
            const int f = __ldg(table + (from >> a.bs_shift)), t = __ldg(table + (to >> a.bs_shift));
            const bool out = f < 0 || f >= a.num_cache_blocks || t < 0 || t >= a.num_cache_blocks;
            if (out && from != to && a.err_word) atomicOr(a.err_word, PDA_ERRW_BAD_BLOCK_ID);
            src_block[k] = out || from == to ? -1 : f * a.cache_block_bytes;
            dst_block[k] = t * a.cache_block_bytes;
            src_slot[k] = from & (a.BS - 1);
            dst_slot[k] = to & (a.BS - 1);
        }
        __syncthreads();
        for (int u = me; u < words + metas; u += stride) {
            if (u < words) {
                for (int k = 0; k < m; k += 8) {
                    uint4 v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (k + i < m && src_block[k + i] >= 0)
                            v[i] = *reinterpret_cast<const uint4*>(a.cache + src_block[k + i] + (long long)src_slot[k + i] * a.row_bytes + 16 * u);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (k + i < m && src_block[k + i] >= 0)
                            *reinterpret_cast<uint4*>(a.cache + dst_block[k + i] + (long long)dst_slot[k + i] * a.row_bytes + 16 * u) = v[i];
                }
            } else {
                const long long base = a.meta_offset_bytes + (long long)(u - words) * a.BS * a.field_bytes;
                for (int k = 0; k < m; k += 8) {
                    uint32_t v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (k + i < m && src_block[k + i] >= 0) {
                            const uint8_t* p = a.cache + src_block[k + i] + base + src_slot[k + i] * a.field_bytes;
                            v[i] = a.field_bytes == 4 ? *reinterpret_cast<const uint32_t*>(p) : *reinterpret_cast<const uint16_t*>(p);
                        }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (k + i < m && src_block[k + i] >= 0) {
                            uint8_t* p = a.cache + dst_block[k + i] + base + dst_slot[k + i] * a.field_bytes;
                            if (a.field_bytes == 4)
                                *reinterpret_cast<uint32_t*>(p) = v[i];
                            else
                                *reinterpret_cast<uint16_t*>(p) = (uint16_t)v[i];
                        }
                }
            }
        }
    }
}

// ------------------------------------------------------------------------- host side
static bool off(const void* p, unsigned a) { return ((uintptr_t)p & (a - 1)) != 0; }
static bool bad_pool(long long nb) { return nb < 1 || nb > (1ll << 31) - 1; }

// What both directions check and fill in.  A status other than OK ends the call; *nothing: there is no token to move.
static int token_args(const pda_plan_t* plan, const void* kv_cache, long long num_cache_blocks, const float* centroids,
                      const int* block_table, const int* token_starts, const int* positions, long long num_tokens,
                      int* err_word, bool reading, TokenArgs& a, unsigned& grid) {
    if (!plan || pda_workspace_size(plan) < 0) return PDA_ERR_INVALID_ARG;
    if ((plan->kv_dtype == PDA_KV_TQ4) != (centroids != nullptr)) return PDA_ERR_INVALID_ARG;
    if (num_tokens < 0 || num_tokens > (1ll << 31) - 1 - kMaxTokensPerCta || bad_pool(num_cache_blocks)) return PDA_ERR_INVALID_ARG;
    grid = 0;
    if (plan->num_seqs == 0 || num_tokens == 0) return PDA_OK;
    if (!kv_cache || !block_table || !token_starts || !positions) return PDA_ERR_INVALID_ARG;
    if (off(kv_cache, 16) || off(block_table, 4) || off(token_starts, 4) || off(positions, 4) || off(centroids, 4) || off(err_word, 4))
        return PDA_ERR_INVALID_ARG;
    a.cache = static_cast<uint8_t*>(const_cast<void*>(kv_cache));
    a.block_table = block_table;
    a.token_starts = token_starts;
    a.positions = positions;
    a.centroids = centroids;
    a.err_word = err_word;
    a.num_cache_blocks = num_cache_blocks;
    a.cache_block_bytes = plan->cache_block_bytes;
    a.meta_offset_bytes = plan->meta_offset_bytes;
    a.num_tokens = (int)num_tokens;
    a.B = plan->num_seqs;
    a.Hk = plan->num_kv_heads;
    a.MB = plan->max_blocks_per_seq;
    a.BS = plan->kv_block_size;
    a.bs_shift = a.BS == 32 ? 5 : 4;
    // Few rows: one per warp, for the sake of the latency (35 tokens of 8 heads 4.2 -> 2.8 us).  Else four CTAs per SM where that
    // is one wave, in whole rounds of a CTA's warps.
    a.ahead = num_tokens * a.Hk <= 4 * 152 * kTokWarps ? 1 : kHeadsAhead;
    a.groups = (a.Hk + a.ahead - 1) / a.ahead;
    // More than one wave: 32 tokens per CTA (64 left the last wave uneven: 60000 fp8 tokens of 8 heads back 70 -> 62 us, into TQ4 157 -> 145;
    // 24 and 16 are slower in writes of one wave), and 16 in reads, whose CTAs are twice as many per SM (62 -> 60 us).
    const long long even = (num_tokens + 4 * 152 - 1) / (4 * 152);
    const long long most = a.groups > 4096 ? 1 : reading && even > kMaxTokensPerCta ? kManyReads : kMaxTokensPerCta;
    const long long step = a.groups % 8 == 0 ? 1 : a.groups % 4 == 0 ? 2 : a.groups % 2 == 0 ? 4 : 8;   // tokens of whole rounds
    const long long round = a.ahead == 1 ? even : (even + step - 1) / step * step;
    a.per_cta = (int)(round > most ? most : round);
    a.by_groups = a.per_cta == 1 ? 0 : ((1ull << 32) + a.groups - 1) / a.groups;
    grid = (unsigned)((num_tokens + a.per_cta - 1) / a.per_cta);
    return PDA_OK;
}

}  // namespace pda

using namespace pda;

extern "C" {

int pda_write_kv(const pda_plan_t* plan, const void* k_new, const void* v_new, long long k_stride, long long v_stride,
                 long long num_tokens, void* kv_cache, long long num_cache_blocks, const float* centroids,
                 const int* block_table, const int* token_starts, const int* positions, int* err_word, void* stream) {
    TokenArgs a = {};
    unsigned grid;
    const int rc = token_args(plan, kv_cache, num_cache_blocks, centroids, block_table, token_starts, positions, num_tokens,
                              err_word, false, a, grid);
    if (rc != PDA_OK) return rc;
    const long long row = (long long)plan->num_kv_heads * kHeadDim;
    if (k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8) return PDA_ERR_INVALID_ARG;
    if (grid == 0) return PDA_OK;
    if (!k_new || !v_new || off(k_new, 16) || off(v_new, 16)) return PDA_ERR_INVALID_ARG;
    a.k_new = static_cast<const uint16_t*>(k_new);
    a.v_new = static_cast<const uint16_t*>(v_new);
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (plan->kv_dtype == PDA_KV_BF16)
        pda_write_kernel<PDA_KV_BF16><<<grid, kTokThreads, 0, s>>>(a);
    else if (plan->kv_dtype == PDA_KV_FP8_E4M3)
        pda_write_kernel<PDA_KV_FP8_E4M3><<<grid, kTokThreads, 0, s>>>(a);
    else
        pda_write_kernel<PDA_KV_TQ4><<<grid, kTokThreads, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? PDA_OK : PDA_ERR_LAUNCH;
}

int pda_read_kv(const pda_plan_t* plan, const void* kv_cache, long long num_cache_blocks, const float* centroids,
                const int* block_table, const int* token_starts, const int* positions, long long num_tokens, void* k_out,
                void* v_out, int out_dtype, int* err_word, void* stream) {
    if (out_dtype != PDA_OUT_BF16 && out_dtype != PDA_OUT_F32) return PDA_ERR_INVALID_ARG;
    TokenArgs a = {};
    unsigned grid;
    const int rc = token_args(plan, kv_cache, num_cache_blocks, centroids, block_table, token_starts, positions, num_tokens,
                              err_word, true, a, grid);
    if (rc != PDA_OK || grid == 0) return rc;
    if ((!k_out && !v_out) || off(k_out, 16) || off(v_out, 16)) return PDA_ERR_INVALID_ARG;
    a.k_out = k_out;
    a.v_out = v_out;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool f32 = out_dtype == PDA_OUT_F32;
    auto launch = [&](auto kernel) { kernel<<<grid, kTokThreads, 0, s>>>(a); };
    if (plan->kv_dtype == PDA_KV_BF16)
        f32 ? launch(pda_read_kernel<PDA_KV_BF16, true>) : launch(pda_read_kernel<PDA_KV_BF16, false>);
    else if (plan->kv_dtype == PDA_KV_FP8_E4M3)
        f32 ? launch(pda_read_kernel<PDA_KV_FP8_E4M3, true>) : launch(pda_read_kernel<PDA_KV_FP8_E4M3, false>);
    else
        f32 ? launch(pda_read_kernel<PDA_KV_TQ4, true>) : launch(pda_read_kernel<PDA_KV_TQ4, false>);
    return cudaGetLastError() == cudaSuccess ? PDA_OK : PDA_ERR_LAUNCH;
}

int pda_accept_tokens(const pda_plan_t* plan, void* kv_cache, long long num_cache_blocks, const int* block_table,
                      const int* context_lens, const int* path, const int* path_lens, int max_path, int* out_lens,
                      int* err_word, void* stream) {
    if (!plan || pda_workspace_size(plan) < 0 || bad_pool(num_cache_blocks) || max_path < 0) return PDA_ERR_INVALID_ARG;
    if (plan->num_seqs == 0) return PDA_OK;
    if (!kv_cache || !block_table || !context_lens || (!path && max_path > 0) || !path_lens || !out_lens)
        return PDA_ERR_INVALID_ARG;
    if (off(kv_cache, 16) || off(block_table, 4) || off(context_lens, 4) || off(path, 4) || off(path_lens, 4) ||
        off(out_lens, 4) || off(err_word, 4))
        return PDA_ERR_INVALID_ARG;
    auto overlap = [&](const int* p, long long n) {   // CTAs of a sequence read what one of them would have written
        const uintptr_t x = (uintptr_t)p, y = (uintptr_t)out_lens;
        return x < y + 4ull * plan->num_seqs && y < x + 4ull * n;
    };
    const long long seqs = plan->num_seqs;
    if (overlap(context_lens, seqs) || overlap(path_lens, seqs) || overlap(path, seqs * max_path) ||
        overlap(block_table, seqs * plan->max_blocks_per_seq))
        return PDA_ERR_INVALID_ARG;
    AcceptArgs a = {};
    a.cache = static_cast<uint8_t*>(kv_cache);
    a.block_table = block_table;
    a.context_lens = context_lens;
    a.path = path;
    a.path_lens = path_lens;
    a.out_lens = out_lens;
    a.err_word = err_word;
    a.num_cache_blocks = num_cache_blocks;
    a.cache_block_bytes = plan->cache_block_bytes;
    a.meta_offset_bytes = plan->meta_offset_bytes;
    a.B = plan->num_seqs;
    a.MB = plan->max_blocks_per_seq;
    a.BS = plan->kv_block_size;
    a.bs_shift = a.BS == 32 ? 5 : 4;
    a.A = max_path;
    const int kv = plan->kv_dtype, Hk = plan->num_kv_heads;
    const long long row = (long long)Hk * (kv == PDA_KV_BF16 ? 512 : kv == PDA_KV_FP8_E4M3 ? 256 : 128);
    if (row > (1ll << 31) - 1) return PDA_ERR_INVALID_ARG;
    a.row_bytes = (int)row;
    a.fields = kv == PDA_KV_BF16 ? 0 : kv == PDA_KV_FP8_E4M3 ? 2 * Hk : 3 * Hk;
    a.field_bytes = kv == PDA_KV_FP8_E4M3 ? 4 : 2;
    const long long units = row / 16 + a.fields;
    const dim3 grid((unsigned)a.B, (unsigned)((units + kTokThreads - 1) / kTokThreads < 64 ? (units + kTokThreads - 1) / kTokThreads : 64));
    pda_accept_kernel<<<grid, kTokThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
    return cudaGetLastError() == cudaSuccess ? PDA_OK : PDA_ERR_LAUNCH;
}

}  // extern "C"
