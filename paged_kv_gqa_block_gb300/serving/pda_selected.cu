// pda_selected.cu -- launches of the one-launch kernel over short lists (pda_selected.cuh): selected blocks,
// own tokens beside a shared prefix, and the window of pda_decode_window.
#include <mutex>

#include "pda.h"
#include "pda_selected.cuh"

namespace pda {

// The cluster of a unit: C CTAs of nw warps.  `wps` warps fit an SM, in CTAs of at most `nwmax`; a unit has
// `tiles` tiles (the table's capacity; the lengths are on the device).  Counted in a warp's tiles, a
// round of CTAs takes a warp's run, and 6 for its start and its join, 3 more for a cluster's join; the rounds
// that the units need are what the choice weighs against it.  A cluster lies within one group of SMs, so of 152
// SMs clusters of four CTAs reach 144, and of eight 120 with one CTA per SM (144, 136 with two, three): 16
// units of 2048 bf16 tokens took 13.7 us in two rounds of eight, and 8.7 us by this rule.  Measured against the partition
// pass and reduce (kernel_variant head warps), every list of blocks of its own and none in L2: 8 units of 2048 bf16
// tokens 7.7 us against 15.7, 32 units 11.5 against 16.4, 256 units of 2048 fp8 tokens 26.7 against 43.6, 512 units 47.8
// against 64.5, 1024 units of 8192 347 against 392, 800 of 4096 bf16 tokens 245 against 295, 512 of 2048 TQ4 tokens 53
// against 74; only few units of long lists were slower (8 of 65536 fp8 tokens 66 against 61 us, one of them 64 against
// 60: a unit is one cluster, and eight clusters of eight CTAs are less than half of the SMs).
struct Shape {
    int C, nw;
};
static Shape selected_shape(long long units, int tiles, int sms, int wps, int nwmax) {
    long long best = 0;
    Shape s = {1, 1};
    for (int C = 1; C <= 8; C *= 2)
        for (int nw = 1; nw <= nwmax; ++nw) {
            const int per = wps / nw, part = C <= 2 ? 19 : C == 4 || per == 2 || per > 3 ? 18 : per == 3 ? 17 : 15;
            const long long slots = (long long)sms * per * part / 19, rounds = (units * C + slots - 1) / slots;
            const int pairs = (tiles + 1) / 2;
            const long long t = rounds * (2 * ((pairs + C * nw - 1) / (C * nw)) + 6 + (C > 1 ? 3 : 0));
            if (best == 0 || t < best) {
                best = t;
                s = Shape{C, nw};
            }
        }
    return s;
}

// Windows are of unlike length: contexts shorter than the window are the rule for a part of a batch.  A shape whose clusters
// all fit at once takes as long as the longest one's warps; more and wider ones, the long ones first, share the GPU evenly but
// for about a third of the longest one's time at the end.  Counted as above, with six tenths of the longest list on average: 512 units
// of 500 to 4100 fp8 tokens 88 -> 68 us, of as many bf16 tokens 116 -> 107, 1600 of 10 to 1028 fp8 tokens 72 -> 43 (where all are
// of 4100 tokens, 512 take 101 us in place of 94).
static Shape window_shape(long long units, int tiles, int sms, int wps, int nwmax) {
    double best = 0;
    Shape s = {1, 1};
    for (int C = 1; C <= 8; C *= 2)
        for (int nw = 1; nw <= nwmax; ++nw) {
            const int per = wps / nw, part = C <= 2 ? 19 : C == 4 || per == 2 || per > 3 ? 18 : per == 3 ? 17 : 15;
            const long long slots = (long long)sms * per * part / 19;
            const int pairs = (tiles + 1) / 2, start = 6 + (C > 1 ? 3 : 0);
            const double longest = 2 * ((pairs + C * nw - 1) / (C * nw)) + start;
            const double even = (double)units * C * (1.2 * pairs / (C * nw) + start) / (double)slots;
            const double t = units * C <= slots ? longest : (even > longest ? even : longest) + 0.35 * longest;
            if (best == 0 || t < best) {
                best = t;
                s = Shape{C, nw};
            }
        }
    return s;
}
// The long ones first where that is two or three rounds: with more the order costs its 0.5 us per cluster more often than it
// saves the end (1600 units of up to 1028 bf16 tokens in five rounds 57 -> 70 us).
static bool sorted_window(long long units, Shape s, int sms, int wps) {
    const long long slots = (long long)sms * (wps / s.nw);
    return units * s.C > slots && units * s.C <= 3 * slots;
}

template <int KV, int NT, int S, int NWMAX, int MINB, int LIST>
static int launch_clusters(bool behind, const DecodeArgs& a, const CUtensorMap& kv_map, const CUtensorMap& sc_map, Shape shape,
                           int window, int num_first, int most, cudaStream_t stream) {
    auto kernel = pda_selected_kernel<KV, NT, S, NWMAX, MINB, LIST>;
    static bool attr_set[64] = {false};
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PDA_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!attr_set[dev]) {
            if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SelectedCfg<KV, S>::bytes(NWMAX)) !=
                cudaSuccess)
                return PDA_ERR_LAUNCH;
            attr_set[dev] = true;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.B * shape.C));
    cfg.blockDim = dim3(32 * shape.nw);
    cfg.dynamicSmemBytes = SelectedCfg<KV, S>::bytes(shape.nw);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = shape.C;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, kv_map, sc_map, a, shape.C, (int)behind, window, num_first, most);
    return e == cudaSuccess ? PDA_OK : PDA_ERR_LAUNCH;
}

template <int LIST, int KV, int NT, int S, int NWMAX, int WPS>
static int launch_clusters_of(bool behind, const DecodeArgs& a, const CUtensorMap& kv_map, const CUtensorMap& sc_map,
                              cudaStream_t stream, int window = 0, int num_first = 0) {
    const int sms = device_sm_count();
    if (sms <= 0) return PDA_ERR_CUDA;
    int tiles = (a.MB * a.BS + 15) / 16;
    if (LIST == kListWindow) {   // at most: the window may begin and end within a tile
        const long long seen = ((long long)num_first + 15) / 16 + ((long long)window + 30) / 16;
        tiles = (int)(seen < tiles ? seen : tiles);
    }
    const Shape shape = (LIST == kListWindow ? window_shape : selected_shape)(a.B, tiles, sms, WPS, NWMAX);
    if ((long long)a.B * shape.C > 0x7FFFFFFFll) return PDA_ERR_INVALID_ARG;
    const bool sorted = LIST == kListWindow && a.B / a.sel_heads <= 1024 && sorted_window(a.B, shape, sms, WPS);
    return launch_clusters<KV, NT, S, NWMAX, WPS / NWMAX, LIST>(behind, a, kv_map, sc_map, shape, window, num_first,
                                                                sorted ? tiles : 0, stream);
}

// bf16: eight warps per SM with rings of three tiles, where six with four took longer: 512 units of 512 tokens at 16
// rows 33.5 -> 26.3 us, 16 of 8192 26.0 -> 23.3, 128 sequences of 64 heads with 100 tokens of their own beside a
// prefix of 32768 104.3 -> 101.9; 800 units of 2048 98.1 -> 99.8 us the other way (lists drawn from one pool, whose
// blocks units share in L2; of their own blocks the 800 take 128.5 us).
int launch_selected_clusters(int kv_dtype, const DecodeArgs& a, const CUtensorMap& kv_map, const CUtensorMap& sc_map,
                             cudaStream_t stream) {
    if (kv_dtype == PDA_KV_BF16) {
        if (a.QG <= 8) return launch_clusters_of<kListSelected, PDA_KV_BF16, 1, 3, 8, 8>(false, a, kv_map, kv_map, stream);
        return launch_clusters_of<kListSelected, PDA_KV_BF16, 2, 3, 8, 8>(false, a, kv_map, kv_map, stream);
    }
    if (kv_dtype == PDA_KV_TQ4) {
        if (a.QG <= 8) return launch_clusters_of<kListSelected, PDA_KV_TQ4, 1, 6, 6, 12>(false, a, kv_map, sc_map, stream);
        return launch_clusters_of<kListSelected, PDA_KV_TQ4, 2, 6, 4, 8>(false, a, kv_map, sc_map, stream);
    }
    if (a.QG <= 8) return launch_clusters_of<kListSelected, PDA_KV_FP8_E4M3, 1, 3, 6, 12>(false, a, kv_map, sc_map, stream);
    return launch_clusters_of<kListSelected, PDA_KV_FP8_E4M3, 2, 4, 4, 8>(false, a, kv_map, sc_map, stream);
}

long long own_clusters_ctas(const pda_plan_t* p, int sms) {
    const long long units = (long long)p->num_seqs * p->num_kv_heads;
    const bool bf16 = p->kv_dtype == PDA_KV_BF16, wide = p->query_group_size > 8;   // as below
    return units * selected_shape(units, (p->max_blocks_per_seq * p->kv_block_size + 15) / 16, sms, bf16 || wide ? 8 : 12,
                                  bf16 ? 8 : wide ? 4 : 6).C;
}

int launch_own_clusters(int kv_dtype, bool behind, const DecodeArgs& a, const CUtensorMap& kv_map, const CUtensorMap& sc_map,
                        cudaStream_t stream) {
    if (kv_dtype == PDA_KV_BF16) {
        if (a.QG <= 8) return launch_clusters_of<kListOwn, PDA_KV_BF16, 1, 3, 8, 8>(behind, a, kv_map, kv_map, stream);
        return launch_clusters_of<kListOwn, PDA_KV_BF16, 2, 3, 8, 8>(behind, a, kv_map, kv_map, stream);
    }
    if (a.QG <= 8) return launch_clusters_of<kListOwn, PDA_KV_FP8_E4M3, 1, 4, 6, 12>(behind, a, kv_map, sc_map, stream);
    return launch_clusters_of<kListOwn, PDA_KV_FP8_E4M3, 2, 4, 4, 8>(behind, a, kv_map, sc_map, stream);
}

int launch_window_clusters(int kv_dtype, const DecodeArgs& a, const CUtensorMap& kv_map, const CUtensorMap& sc_map, int window,
                           int num_first, cudaStream_t stream) {
    auto of = [&](auto launch) { return launch(false, a, kv_map, sc_map, stream, window, num_first); };
    const bool narrow = a.QG <= 8;
    if (kv_dtype == PDA_KV_BF16)
        return narrow ? of(launch_clusters_of<kListWindow, PDA_KV_BF16, 1, 3, 8, 8>)
                      : of(launch_clusters_of<kListWindow, PDA_KV_BF16, 2, 3, 8, 8>);
    if (kv_dtype == PDA_KV_TQ4)
        return narrow ? of(launch_clusters_of<kListWindow, PDA_KV_TQ4, 1, 6, 6, 12>)
                      : of(launch_clusters_of<kListWindow, PDA_KV_TQ4, 2, 6, 4, 8>);
    return narrow ? of(launch_clusters_of<kListWindow, PDA_KV_FP8_E4M3, 1, 3, 6, 12>)
                  : of(launch_clusters_of<kListWindow, PDA_KV_FP8_E4M3, 2, 4, 4, 8>);
}

}  // namespace pda
