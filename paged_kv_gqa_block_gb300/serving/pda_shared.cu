// pda_shared.cu -- pda_decode_shared: a decode step for sequences that share prefixes in groups.  The prefix pass
// (pda_prefix.cuh), the own tokens' pass (pda_selected.cuh) and, here, the join of their partials and the host side.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pda_prefix.cuh"

namespace pda {

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
