// pda_maps.cu -- see pda_maps.h.
#include "pda_maps.h"

#include <cuda_runtime.h>

#include <mutex>

#include "pda_internal.h"

namespace pda {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiled encoder() {
    static EncodeTiled fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiled>(p);
    });
    return fn;
}
static cuuint64_t row_bytes(const pda_plan_t* p) {   // K and V of one token and head
    return p->kv_dtype == PDA_KV_BF16 ? 4 * kHeadDim : p->kv_dtype == PDA_KV_FP8_E4M3 ? 2 * kHeadDim : kHeadDim;
}

bool encode_tokens_map(CUtensorMap* m, const void* cache, const pda_plan_t* p, long long nb, int tokens, int chunks) {
    const EncodeTiled fn = encoder();
    if (!fn) return false;
    const cuuint64_t row = row_bytes(p), all = row / 128;
    const cuuint64_t dims[5] = {128, (cuuint64_t)p->kv_block_size, all, (cuuint64_t)p->num_kv_heads, (cuuint64_t)nb};
    const cuuint64_t strides[4] = {(cuuint64_t)p->num_kv_heads * row, 128, row, (cuuint64_t)p->cache_block_bytes};
    const cuuint32_t box[5] = {128, (cuuint32_t)tokens, chunks ? (cuuint32_t)chunks : (cuuint32_t)all, 1, 1};
    const cuuint32_t each[5] = {1, 1, 1, 1, 1};
    // a TQ4 row is 128 bytes: wider fetches would bring the next head's
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void*>(cache), dims, strides, box, each, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, row >= 256 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_fields_map(CUtensorMap* m, const void* cache, const pda_plan_t* p, long long nb, int tokens) {
    const EncodeTiled fn = encoder();
    if (!fn || p->kv_dtype == PDA_KV_BF16) return false;
    const bool tq = p->kv_dtype == PDA_KV_TQ4;
    const cuuint64_t bs = (cuuint64_t)p->kv_block_size, fields = tq ? 3 : 2, size = tq ? 2 : 4;
    char* base = static_cast<char*>(const_cast<void*>(cache)) + p->meta_offset_bytes;
    const cuuint64_t dims[4] = {bs, fields, (cuuint64_t)p->num_kv_heads, (cuuint64_t)nb};
    const cuuint64_t strides[3] = {bs * size, bs * size * fields, (cuuint64_t)p->cache_block_bytes};
    const cuuint32_t box[4] = {(cuuint32_t)tokens, (cuuint32_t)fields, 1, 1};
    const cuuint32_t each[4] = {1, 1, 1, 1};
    return fn(m, tq ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, base, dims, strides, box, each,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace pda
