// pda_window.cu -- pda_decode_window: a decode step over a sliding window and a few first tokens.
//
// The query of a sequence of ctx tokens stands at position ctx - 1 and sees token t where ctx - 1 - t < window or
// t < num_first.  What it does not see is not read: the kernel is the cluster kernel over short lists (pda_selected.cuh),
// whose list here is a run of tiles computed from the length (WindowTiles).
//
// Measured: 64 sequences of 500 to 16384 fp8 tokens in a window of 4096 68 us (5.3 TB/s: HBM, and the uneven end), bf16 109 us, TQ4
// 74 us (2.5 TB/s: the decoding of its codes); 4 of 32768 bf16 tokens in one of 1024 9.0 us (latency: table, copies, joins in
// the cluster).
#include <cuda_runtime.h>

#include <cstdint>

#include "pda.h"
#include "pda_internal.h"
#include "pda_maps.h"

namespace pda {

int launch_window_clusters(int kv_dtype, const DecodeArgs& a, const CUtensorMap& kv_map, const CUtensorMap& sc_map, int window,
                           int num_first, cudaStream_t stream);

static bool off(const void* p, unsigned a) { return ((uintptr_t)p & (a - 1)) != 0; }

}  // namespace pda

using namespace pda;

extern "C" int pda_decode_window(const pda_plan_t* plan, const void* query, const void* kv_cache, long long num_cache_blocks,
                                 const float* centroids, const int* block_table, const int* context_lens, int window,
                                 int num_first, void* out, int out_dtype, int* err_word, void* stream) {
    if (!plan || pda_workspace_size(plan) < 0) return PDA_ERR_INVALID_ARG;
    if ((plan->kv_dtype == PDA_KV_TQ4) != (centroids != nullptr) || (out_dtype != PDA_OUT_BF16 && out_dtype != PDA_OUT_F32))
        return PDA_ERR_INVALID_ARG;
    if (window < 1 || num_first < 0) return PDA_ERR_INVALID_ARG;
    if (plan->kernel_variant != PDA_VARIANT_AUTO) return PDA_ERR_UNSUPPORTED;   // one layout
    if (num_cache_blocks < 1 || num_cache_blocks > (1ll << 31) - 1) return PDA_ERR_INVALID_ARG;
    if (plan->num_seqs == 0) return PDA_OK;
    if (!query || !kv_cache || !block_table || !context_lens || !out) return PDA_ERR_INVALID_ARG;
    if (off(query, 16) || off(kv_cache, 16) || off(centroids, 4) || off(block_table, 4) || off(context_lens, 4) ||
        off(err_word, 4) || off(out, out_dtype == PDA_OUT_F32 ? 16 : 8))
        return PDA_ERR_INVALID_ARG;
    DecodeArgs a = {};
    a.query = static_cast<const uint16_t*>(query);
    a.block_table = block_table;
    a.context_lens = context_lens;
    a.centroids = centroids;
    a.err_word = err_word;
    a.num_cache_blocks = num_cache_blocks;
    a.B = plan->num_seqs * plan->num_kv_heads;   // units of one KV head each: query rows and output have the same layout
    a.Hk = 1;
    a.sel_heads = plan->num_kv_heads;
    a.QG = plan->query_group_size;
    a.MB = plan->max_blocks_per_seq;
    a.BS = plan->kv_block_size;
    a.P = plan->num_partitions;
    a.W = plan->partition_tokens;
    a.bs_shift = a.BS == 32 ? 5 : 4;
    a.HG = 1;
    a.qk_scale_log2 = plan->resolved_softmax_scale * 1.4426950408889634f;
    a.timeout_ns = plan->wait_timeout_ns > 0 ? (unsigned long long)plan->wait_timeout_ns : kDefaultTimeoutNs;
    a.out = out;
    a.out_f32 = out_dtype == PDA_OUT_F32;
    CUtensorMap kv_map, sc_map;
    if (!encode_tokens_map(&kv_map, kv_cache, plan, num_cache_blocks, kTileTokens, 0)) return PDA_ERR_LAUNCH;
    sc_map = kv_map;
    if (plan->kv_dtype != PDA_KV_BF16 && !encode_fields_map(&sc_map, kv_cache, plan, num_cache_blocks, kTileTokens))
        return PDA_ERR_LAUNCH;
    return launch_window_clusters(plan->kv_dtype, a, kv_map, sc_map, window, num_first, static_cast<cudaStream_t>(stream));
}
