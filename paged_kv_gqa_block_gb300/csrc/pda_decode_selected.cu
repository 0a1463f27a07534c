// pda_decode_selected.cu -- instantiations and launches of the partition kernel inside other steps: over
// selected blocks (one block table and one length per (sequence, KV head)), and over the sequences' own
// tokens beside a shared prefix.
#include "pda_decode.cuh"
#include "pda_launch.cuh"

namespace pda {

// Head warps in every format (a head group's copies span heads, whose blocks differ here), with the
// stages and CTAs per SM of the same kernels over whole contexts.
int launch_decode_selected(int kv_dtype, const DecodeArgs& a, const CUtensorMap& kv_map, const CUtensorMap& sc_map,
                           cudaStream_t stream) {
    if (kv_dtype == PDA_KV_BF16) {
        if (a.QG <= 8) return launch_partition<PDA_KV_BF16, 1, 4, 6, false, kSelected>(a, kv_map, kv_map, stream);
        return launch_partition<PDA_KV_BF16, 2, 4, 1, false, kSelected>(a, kv_map, kv_map, stream);
    }
    if (kv_dtype == PDA_KV_TQ4) {
        if (a.QG <= 8) return launch_partition<PDA_KV_TQ4, 1, 6, 12, false, kSelected>(a, kv_map, sc_map, stream);
        return launch_partition<PDA_KV_TQ4, 2, 6, 8, false, kSelected>(a, kv_map, sc_map, stream);
    }
    if (a.QG <= 8) return launch_partition<PDA_KV_FP8_E4M3, 1, 3, 12, false, kSelected>(a, kv_map, sc_map, stream);
    return launch_partition<PDA_KV_FP8_E4M3, 2, 4, 8, false, kSelected>(a, kv_map, sc_map, stream);
}

int launch_decode_own(int kv_dtype, const DecodeArgs& a, const CUtensorMap& kv_map, const CUtensorMap& sc_map,
                      cudaStream_t stream) {
    if (kv_dtype == PDA_KV_BF16) {
        if (a.QG <= 8) return launch_partition<PDA_KV_BF16, 1, 4, 6, false, kOwnTokens>(a, kv_map, kv_map, stream);
        return launch_partition<PDA_KV_BF16, 2, 4, 1, false, kOwnTokens>(a, kv_map, kv_map, stream);
    }
    if (a.QG <= 8) return launch_partition<PDA_KV_FP8_E4M3, 1, 3, 12, false, kOwnTokens>(a, kv_map, sc_map, stream);
    return launch_partition<PDA_KV_FP8_E4M3, 2, 4, 8, false, kOwnTokens>(a, kv_map, sc_map, stream);
}

}  // namespace pda
