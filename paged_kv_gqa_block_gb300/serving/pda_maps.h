// pda_maps.h -- tensor maps of the paged cache for the serving operators: the tiled copies (TMA) of the tokens of one block.
#pragma once

#include <cuda.h>

#include "pda.h"

namespace pda {

// K and V of `tokens` tokens of one block and KV head: dimensions {128 bytes of a chunk, BS slots, chunks per token and head,
// Hk heads, NB blocks}; `chunks` 128-byte chunks per copy (0: all).  The box lands as [chunk][token][128 bytes], swizzled.
bool encode_tokens_map(CUtensorMap* m, const void* cache, const pda_plan_t* p, long long num_cache_blocks, int tokens, int chunks);
// Their metadata: {BS slots, fields, Hk heads, NB blocks}, landing as [field][token] (fp8: K scale, V scale in fp32; TQ4:
// k_norm, v_scale, v_zero in fp16).  `tokens` divides BS and copies start at a multiple of it.
bool encode_fields_map(CUtensorMap* m, const void* cache, const pda_plan_t* p, long long num_cache_blocks, int tokens);

}  // namespace pda
