// pda_tree.cu -- pda_decode_tree: a step for drafted tokens, several per sequence, over their cache.
//
// For drafted token i of a sequence with ctx cached tokens and KV head h, its QG query rows
//   out = softmax(scale [q.K ; mask]) V
// over the cached tokens t < ctx (of a window, those with ctx + before(i) - t < window and the first num_first) and over the
// drafted tokens j that the row of its mask names; before(i) is the number of drafted tokens other than i that it sees.  The
// drafted tokens' K and V lie in the cache behind the cached ones (pda_write_kv).
//
// The rows of all drafted tokens of a sequence and KV head are one matrix product with its cache, so K and V are read once per
// 256 rows and not once per drafted token: pda_prefix.cuh, where a sequence takes the place of a group.  Its pieces are joined
// here.
//
// Measured, replays of a graph (a call from Python by itself is longer, see the table of cases): 4 trees of 64 tokens over 32768
// bf16 tokens 192 us (1.43 PFLOP/s: the tensor cores); 32 trees of 9 to 33 over contexts of 2048 to 8192 128 us (sequences of
// more than 256 rows have further row tiles, which read K and V again: 487 MB of 352; the join 12); 64 trees of up to 6 in a
// window of 4096 fp8 tokens 98 us (2.0 TB/s: 1.1 to 1.3 us per step and CTA, and some 5 us where a CTA goes on to the next
// sequence and head, most of it the first fetch of the code); 64 of 4 over 4096 bf16 tokens 175 us (6.2 TB/s: HBM), fp8 156 us,
// TQ4 258 us (four warps convert K, then V, in short loops: 2.3 us per step); one of 4 over 250 10.3 us (latency of two launches).
// Chains: every row tile walks all steps of its sequence, also those behind its own tokens; 512 tokens of 64 heads behind nothing
// 23 us (bf16), 2048 196 us, in a window of 128 210 us (16 steps per row tile where its tokens see 3).
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pda_maps.h"
#include "pda_prefix.cuh"

namespace pda {

// CTAs per SM of the join: its rows wait for their loads.  With eight pieces at a time in place of four (and three CTAs) 32 sequences of up
// to 33 drafted tokens took 140 us and not 130; six CTAs spill.
constexpr int kJoinCtas = 4;

struct TreeJoinArgs {
    const int* refused;
    const float* part_o;   // [N][Hk][slots][QG][D]
    const float* part_l;   // [N][Hk][slots][QG]
    const float* part_m;
    const int* pieces;     // [N][Hk][QG]
    void* out;
    long long rows;        // N * Hk * QG
    int QG, slots, out_f32;
};

// One warp per row of more than one piece; the rows of a warp lie as far apart as there are warps, and their numbers of pieces
// are read 32 at a time, so that rows of one piece, which are whole already, cost next to nothing.  Lane i holds (m, l) of
// pieces i, i + 32, ..; each lane sums four dimensions over the pieces in order.
__global__ void __launch_bounds__(256, kJoinCtas) pda_tree_join_kernel(const TreeJoinArgs a) {
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const long long warps = (long long)gridDim.x * 8, first = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int refused = __ldcg(a.refused);
    for (long long k0 = 0; first + k0 * warps < a.rows; k0 += 32) {
        const long long mine = first + (k0 + lane) * warps;
        const int pieces = mine < a.rows ? __ldcg(a.pieces + mine) : 1;
        if (refused) return;
        unsigned todo = __ballot_sync(kLanes, pieces > 1);
        while (todo) {
            const int src = __ffs(todo) - 1;
            todo &= todo - 1;
            const long long row = first + (k0 + src) * warps, unit = row / a.QG;
            const int total = min(a.slots, __shfl_sync(kLanes, pieces, src));
            const long long row0 = unit * a.slots * a.QG + (row - unit * a.QG);
            auto stats = [&](int i, float& m, float& l) {
                m = -INFINITY;
                l = 0.f;
                if (i < total) {
                    m = __ldcg(a.part_m + row0 + (long long)i * a.QG);
                    l = __ldcg(a.part_l + row0 + (long long)i * a.QG);
                    if (l == 0.f) m = -INFINITY;   // a piece of which the row sees nothing
                }
            };
            float4 o[4];   // four pieces at a time, the first asked for with the statistics
            auto ask = [&](int i) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    o[j] = __ldcg(reinterpret_cast<const float4*>(a.part_o + (row0 + (long long)min(i + j, total - 1) * a.QG) * kHeadDim) + lane);
            };
            ask(0);
            float m0, l0;
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
                const float w = l0 != 0.f ? partition_weight(l0, m0, M) : 0.f;   // 0 past the last piece
                sum += w;
                for (int j0 = i0; j0 < min(total, i0 + 32); j0 += 4) {
                    if (j0 > 0) ask(j0);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float f = __shfl_sync(kLanes, w, (j0 + j) & 31);
                        if (j0 + j < total) {
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
            const float inv = sum == 0.f ? 0.f : 1.f / sum;   // a row that sees nothing gives zeros
            if (a.out_f32) {
                *reinterpret_cast<float4*>(static_cast<float*>(a.out) + row * kHeadDim + 4 * lane) =
                    make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
            } else {
                uint2 v;
                v.x = pack_bf16(acc.x * inv, acc.y * inv);
                v.y = pack_bf16(acc.z * inv, acc.w * inv);
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * kHeadDim + 4 * lane) = v;
            }
        }
    }
}

// ------------------------------------------------------------------------- host side
static long long up256(long long x) { return (x + 255) & ~255ll; }
static bool odd(const void* p, unsigned a) { return ((uintptr_t)p & (a - 1)) != 0; }

static long long steps_of(const pda_plan_t* p) { return ((long long)p->max_blocks_per_seq * p->kv_block_size + kStep - 1) / kStep; }
// The most row tiles (times steps) that the drafted tokens can have.
static long long most_tree_tiles(const pda_plan_t* p, long long tokens) {
    const long long seqs = p->num_seqs < tokens ? p->num_seqs : tokens;
    return (tokens * p->query_group_size / kUnitRows + seqs) * p->num_kv_heads;
}
// Pieces of the longest sequence: four times as many as give every SM one, since lengths differ, and of two steps at least.
static long long wanted_tiles() {
    const int sms = device_sm_count();
    return 4ll * (sms > 0 ? sms : 152);
}
static int tree_pieces(const pda_plan_t* p, long long tokens) {
    const long long rows = (tokens * p->query_group_size + kUnitRows - 1) / kUnitRows;
    const long long seqs = p->num_seqs < tokens ? p->num_seqs : tokens;
    const long long tiles = (rows > seqs ? rows : seqs) * p->num_kv_heads;
    const long long want = (wanted_tiles() + tiles - 1) / tiles, most = (steps_of(p) + 1) / 2;
    return (int)(want < most ? want : most);
}
static bool tree_fits(const pda_plan_t* p, long long tokens) {
    constexpr long long kPlaces = 2000000000ll;   // places are ints
    if (tokens < 0 || tokens > (1ll << 30) / p->query_group_size) return false;
    const long long tiles = most_tree_tiles(p, tokens);
    return tiles <= kPlaces && tiles * (steps_of(p) + TreeArgs::kSwitchSteps) <= kPlaces;
}
struct TreeLayout {
    long long o, l, m, pieces, seen, refused, bytes;
    int slots;
};
static TreeLayout tree_layout(const pda_plan_t* p, long long tokens) {
    TreeLayout w;
    w.slots = tree_pieces(p, tokens) + 1;
    const long long rows = tokens * p->num_kv_heads * p->query_group_size;
    w.o = 0;
    w.l = w.o + up256(rows * w.slots * kHeadDim * 4);
    w.m = w.l + up256(rows * w.slots * 4);
    w.pieces = w.m + up256(rows * w.slots * 4);
    w.seen = w.pieces + up256(rows * 4);
    w.refused = w.seen + up256(tokens);
    w.bytes = w.refused + 256;
    return w;
}

}  // namespace pda

using namespace pda;

extern "C" {

long long pda_tree_workspace_size(const pda_plan_t* plan, long long num_tokens) {
    if (!plan || pda_workspace_size(plan) < 0 || !tree_fits(plan, num_tokens)) return -1;
    if (num_tokens == 0 || plan->num_seqs == 0) return 0;
    // Fewer tokens may be cut into more pieces, and take more.  A workspace serves those too: the largest of the calls with so few
    // tiles that they are cut into `pieces` or more are the ones with the most tokens.
    long long bytes = tree_layout(plan, num_tokens).bytes;
    for (int pieces = tree_pieces(plan, num_tokens) + 1, last = tree_pieces(plan, 1); pieces <= last; ++pieces) {
        const long long x = (wanted_tiles() - 1) / ((pieces - 1ll) * plan->num_kv_heads);   // row tiles of a head
        const long long fewer = plan->num_seqs <= x ? x * kUnitRows / plan->query_group_size : x;
        const long long b = tree_layout(plan, fewer < num_tokens ? fewer : num_tokens).bytes;
        if (b > bytes) bytes = b;
    }
    return bytes;
}

int pda_decode_tree(const pda_plan_t* plan, const void* query, long long num_tokens, const void* kv_cache,
                    long long num_cache_blocks, const float* centroids, const int* block_table, const int* context_lens,
                    const int* token_starts, const unsigned long long* tree_masks, int mask_words, int window, int num_first,
                    void* workspace, long long workspace_bytes, void* out, int out_dtype, int* err_word, void* stream) {
    if (!plan || pda_workspace_size(plan) < 0 || !tree_fits(plan, num_tokens)) return PDA_ERR_INVALID_ARG;
    if ((plan->kv_dtype == PDA_KV_TQ4) != (centroids != nullptr) || (out_dtype != PDA_OUT_BF16 && out_dtype != PDA_OUT_F32))
        return PDA_ERR_INVALID_ARG;
    if (window < 0 || num_first < 0 || (tree_masks && (mask_words < 1 || mask_words > 1 << 20)) || (!tree_masks && mask_words != 0))
        return PDA_ERR_INVALID_ARG;
    if (num_cache_blocks < 1 || num_cache_blocks > (1ll << 31) - 1) return PDA_ERR_INVALID_ARG;
    if (plan->num_seqs == 0 || num_tokens == 0) return PDA_OK;
    if (!query || !kv_cache || !block_table || !context_lens || !token_starts || !workspace || !out) return PDA_ERR_INVALID_ARG;
    if (odd(query, 16) || odd(kv_cache, 16) || odd(centroids, 4) || odd(block_table, 4) || odd(context_lens, 4) ||
        odd(token_starts, 4) || odd(tree_masks, 8) || odd(workspace, 32) || odd(err_word, 4) ||
        odd(out, 16))
        return PDA_ERR_INVALID_ARG;
    const TreeLayout w = tree_layout(plan, num_tokens);
    if (workspace_bytes < w.bytes) return PDA_ERR_WORKSPACE_TOO_SMALL;
    const int sms = device_sm_count();
    if (sms <= 0) return PDA_ERR_CUDA;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    auto f32 = [&](long long at) { return reinterpret_cast<float*>(ws + at); };
    TreeArgs a = {};
    a.query = static_cast<const uint16_t*>(query);
    a.group_starts = token_starts;
    a.prefix_table = block_table;
    a.prefix_lens = context_lens;
    a.part_o = f32(w.o);
    a.part_l = f32(w.l);
    a.part_m = f32(w.m);
    a.pieces = reinterpret_cast<int*>(ws + w.pieces);
    a.err_word = err_word;
    a.num_cache_blocks = num_cache_blocks;
    a.B = (int)num_tokens;
    a.NG = plan->num_seqs;
    a.Hk = plan->num_kv_heads;
    a.QG = plan->query_group_size;
    a.MP = plan->max_blocks_per_seq;
    a.BS = plan->kv_block_size;
    a.P = w.slots - 1;
    a.slots = w.slots;
    a.first = 1;
    a.qk_scale_log2 = plan->resolved_softmax_scale * kLog2eS;
    a.timeout_ns = plan->wait_timeout_ns > 0 ? (unsigned long long)plan->wait_timeout_ns : kDefaultTimeoutNs;
    a.masks = reinterpret_cast<const uint32_t*>(tree_masks);
    a.centroids = centroids;
    a.refused = reinterpret_cast<int*>(ws + w.refused);
    a.seen = ws + w.seen;
    a.words = 2 * mask_words;
    a.window = window;
    a.num_first = num_first;
    a.cache = static_cast<const uint8_t*>(kv_cache);
    a.block_bytes = plan->cache_block_bytes;
    a.meta_bytes = plan->meta_offset_bytes;
    a.out = out;
    a.out_f32 = out_dtype == PDA_OUT_F32;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    CUtensorMap kv_map, sc_map;
    if (!encode_tokens_map(&kv_map, kv_cache, plan, num_cache_blocks, a.BS, 1)) return PDA_ERR_LAUNCH;
    sc_map = kv_map;
    if (plan->kv_dtype != PDA_KV_BF16 && !encode_fields_map(&sc_map, kv_cache, plan, num_cache_blocks, a.BS)) return PDA_ERR_LAUNCH;
    const long long most = most_tree_tiles(plan, num_tokens) * steps_of(plan);   // no more CTAs than there can be steps
    const int ctas = (int)(most < sms ? most : sms);
    int rc;
    if (plan->kv_dtype == PDA_KV_BF16)
        rc = launch_prefix<PDA_KV_BF16>(a, kv_map, sc_map, ctas, s);
    else if (plan->kv_dtype == PDA_KV_FP8_E4M3)
        rc = launch_prefix<PDA_KV_FP8_E4M3>(a, kv_map, sc_map, ctas, s);
    else
        rc = launch_prefix<PDA_KV_TQ4>(a, kv_map, sc_map, ctas, s);
    if (rc != PDA_OK) return rc;
    TreeJoinArgs j = {};
    j.refused = a.refused;
    j.part_o = a.part_o;
    j.part_l = a.part_l;
    j.part_m = a.part_m;
    j.pieces = a.pieces;
    j.out = out;
    j.rows = num_tokens * a.Hk * a.QG;
    j.QG = a.QG;
    j.slots = a.slots;
    j.out_f32 = a.out_f32;
    const long long join = (j.rows + 7) / 8;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(join < (long long)kJoinCtas * sms ? join : (long long)kJoinCtas * sms));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, pda_tree_join_kernel, j) == cudaSuccess ? PDA_OK : PDA_ERR_LAUNCH;
}

}  // extern "C"
