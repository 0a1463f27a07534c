// pda_decode_selected.cu -- instantiation and launch of the partition kernel for attention over
// selected blocks: one block table and one length per (sequence, KV head).
#include "pda_decode.cuh"
#include "pda_launch.cuh"

namespace pda {

// Head warps in every format (a head group's copies span heads, whose blocks differ here), with the
// stages and CTAs per SM of the same kernels over whole contexts.
int launch_decode_selected(int kv_dtype, const DecodeArgs& a, const CUtensorMap& kv_map, const CUtensorMap& sc_map,
                           cudaStream_t stream) {
    if (kv_dtype == PDA_KV_BF16) {
        if (a.QG <= 8) return launch_partition<PDA_KV_BF16, 1, 4, 6, false, true>(a, kv_map, kv_map, stream);
        return launch_partition<PDA_KV_BF16, 2, 4, 1, false, true>(a, kv_map, kv_map, stream);
    }
    if (kv_dtype == PDA_KV_TQ4) {
        if (a.QG <= 8) return launch_partition<PDA_KV_TQ4, 1, 6, 12, false, true>(a, kv_map, sc_map, stream);
        return launch_partition<PDA_KV_TQ4, 2, 6, 8, false, true>(a, kv_map, sc_map, stream);
    }
    if (a.QG <= 8) return launch_partition<PDA_KV_FP8_E4M3, 1, 3, 12, false, true>(a, kv_map, sc_map, stream);
    return launch_partition<PDA_KV_FP8_E4M3, 2, 4, 8, false, true>(a, kv_map, sc_map, stream);
}

}  // namespace pda
