// pda_pages.cu -- moving and sharing the blocks of a paged cache: pda_copy_blocks,
// pda_fork_sequences, pda_compact_blocks.
//
// All three move whole cache blocks (cache_block_bytes of any format) and otherwise only integers,
// so their results are exact.  A block's count is the number of block-table entries that hold it;
// a block with count 0 is free.  The fork and the compaction read one set of tables and counts and
// write another: nothing that is read is changed (blocks are copied into free blocks only), so the
// old batch stays valid until the caller drops it, and a call that fails can be repeated.
//
// Both are two launches, the second a programmatic dependent of the first:
//   1. a scan by one thread-block cluster (kScanCtas CTAs of 1024 threads; one CTA for a small
//      pool): every CTA counts its slice of the counts, the totals are exchanged through
//      distributed shared memory, and each free or used block gets its rank (slices of up to 4096 counts
//      from the registers, longer ones in a second sweep, now in L1: 6.1 -> 5.7 and 9.5 -> 9.2 us for the forks
//      below).  One launch in place of count / prefix / write;
//   2. a grid over the table segments and the 4 KB chunks of the blocks to copy.
// What bounds them: the copies HBM (read + write), everything else launch and load latency.  Measured: 2048
// blocks of 64 KB copied in 44.4 us (6.0 TB/s, read and written; under counters 39 us), to pinned host memory in 695 and
// from it in 638 us (193 and 210 GB/s, what one plain copy of as many bytes takes); 4 sequences forked from two
// parents 5.7 us, 64 from 16 parents of up to 16000 tokens in a pool of 16384 blocks 9.3 us (the second launch 7.5
// us under counters); a pool of 8192 blocks of 64 KB compacted in 49.5 us, of which the copies are 39 us (246 MB
// read and written, 6.3 TB/s) and the rest the scan in front of them.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "pda.h"
#include "pda_internal.h"
#include "pda_ptx.cuh"

namespace pda {

namespace cg = cooperative_groups;

constexpr int kScanThreads = 1024;
constexpr int kScanCtas = 8;              // the portable cluster size
constexpr int kScanTile = 4 * kScanThreads;
constexpr long long kScanOneCta = kScanTile;   // pools up to here are scanned by one CTA, in one tile
constexpr int kPageThreads = 256;
constexpr int kRowInts = 8;

// ------------------------------------------------------------------------- copies
// One chunk of a block: every thread moves U 16-byte words, all loads before the first store.
template <int U>
__device__ __forceinline__ void copy_chunk(const uint8_t* src, uint8_t* dst, long long bytes, long long chunk) {
    const long long base = chunk * (kPageThreads * 16 * U) + threadIdx.x * 16;
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const long long o = base + u * (kPageThreads * 16);
        if (o < bytes) v[u] = __ldcs(reinterpret_cast<const uint4*>(src + o));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const long long o = base + u * (kPageThreads * 16);
        if (o < bytes) __stcs(reinterpret_cast<uint4*>(dst + o), v[u]);
    }
}
template <int U>
__host__ __device__ constexpr long long chunks_of(long long bytes) {
    return (bytes + kPageThreads * 16 * U - 1) / (kPageThreads * 16 * U);
}

struct CopyArgs {
    const uint8_t* src;
    uint8_t* dst;
    const int* pairs;   // [n][2]
    int* err_word;
    long long src_blocks, dst_blocks, block_bytes, n;
};

template <int U>
__global__ void __launch_bounds__(kPageThreads) pda_copy_kernel(const CopyArgs a) {
    grid_dependency_wait();
    const long long cpb = chunks_of<U>(a.block_bytes), items = a.n * cpb;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const long long i = it / cpb, c = it - i * cpb;
        const int s = __ldg(a.pairs + 2 * i), d = __ldg(a.pairs + 2 * i + 1);
        if (s < 0 || d < 0) continue;
        if (s >= a.src_blocks || d >= a.dst_blocks) {
            if (c == 0 && threadIdx.x == 0 && a.err_word) atomicOr(a.err_word, PDA_ERRW_BAD_BLOCK_ID);
            continue;
        }
        const uint8_t* from = a.src + s * a.block_bytes;
        uint8_t* to = a.dst + d * a.block_bytes;
        if (from != to) copy_chunk<U>(from, to, a.block_bytes, c);
    }
}

// ------------------------------------------------------------------------- scans
// Inclusive sum over the block's threads (1024), `total` to all.  `tmp` holds 32 values.
template <class T>
__device__ __forceinline__ T block_scan(T x, T* tmp, T& total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    T v = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T n = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += n;
    }
    if (lane == 31) tmp[w] = v;
    __syncthreads();
    if (w == 0) {
        T t = tmp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const T n = __shfl_up_sync(0xFFFFFFFFu, t, o);
            if (lane >= o) t += n;
        }
        tmp[lane] = t;
    }
    __syncthreads();
    total = tmp[31];
    const T r = v + (w ? tmp[w - 1] : T(0));
    __syncthreads();
    return r;
}

struct ScanArgs {
    const int* refs;       // [NB]
    long long NB;
    int* out_refs;
    int* err_word;
    // fork: the new rows
    const int* block_table;
    const int* context_lens;
    const int* parents;
    const int* new_tokens;
    int* out_lens;
    int* free_ids;         // workspace [NB]
    int* first;            // workspace [B]: the first new row of each old one (INT_MAX: none, -1: it got no blocks)
    int* rows;             // workspace [R][kRowInts]
    int B, R, MB, BS;
    // compaction
    int* used_ids;         // workspace [NB]: at r, the id of the used block of rank r, where it moves
    int* holes;            // workspace [NB]
    int* scalars;          // workspace: {moved, used below U}
    int* remap;
    int* num_used;
};

// A new row's record: {parent, length, new length, its first place in free_ids}, {flags, last block's id}
enum { kRowCopy = 1, kRowFirst = 2 };

// The slice of the pool that this CTA of the cluster scans.
__device__ __forceinline__ void slice_of(const cg::cluster_group& cl, long long NB, long long& lo, long long& hi) {
    const long long per = (NB + cl.num_blocks() - 1) / cl.num_blocks();
    lo = min(NB, per * cl.block_rank());
    hi = min(NB, lo + per);
}

// The entries of this CTA's slice for which `f` holds are counted: `before` are those ahead of the slice, `total` those of
// the pool.  A slice of one tile is not read again: the thread keeps its four entries, their count and the
// inclusive sum over the threads.  The caller syncs the cluster once more (the totals are read from the other CTAs).
struct Count {
    int before, total, r[4], n, incl;
};
template <class F>
__device__ __forceinline__ Count count_slice(const cg::cluster_group& cl, const int* refs, long long lo, long long hi,
                                             int none, int* tmp, int* share, F f) {
    Count c = {0, 0, {none, none, none, none}, 0, 0};
    for (long long t0 = lo + 4 * threadIdx.x; t0 < hi; t0 += kScanTile)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            c.r[u] = t0 + u < hi ? __ldg(refs + t0 + u) : none;
            c.n += f(c.r[u]);
        }
    c.incl = block_scan(c.n, tmp, c.total);
    if (cl.num_blocks() == 1) return c;
    if (threadIdx.x == 0) *share = c.total;
    cl.sync();
    c.total = 0;
    for (unsigned r = 0; r < cl.num_blocks(); ++r) {
        const int v = *cl.map_shared_rank(share, r);
        if (r < cl.block_rank()) c.before += v;
        c.total += v;
    }
    return c;
}

// What a new row asks for.
struct NewRow {
    int p, L, nl, tail_id, tail_ref;
    bool live;
};
__device__ __forceinline__ NewRow new_row(const ScanArgs& a, int i) {
    NewRow r = {-1, 0, 0, -1, 0, false};
    if (i >= a.R) return r;
    r.p = __ldg(a.parents + i);
    const int g = a.new_tokens ? __ldg(a.new_tokens + i) : 0;
    if (r.p < 0) return r;
    if (r.p >= a.B) {
        if (a.err_word) atomicOr(a.err_word, PDA_ERRW_BAD_SEQUENCE);
        return r;
    }
    const long long max_ctx = (long long)a.MB * a.BS;
    r.L = __ldg(a.context_lens + r.p);
    if (r.L < 0 || r.L > max_ctx) {
        if (a.err_word) atomicOr(a.err_word, PDA_ERRW_BAD_CONTEXT_LEN);
        r.L = 0;
    }
    if (g < 0 || (long long)r.L + g > max_ctx) {
        if (a.err_word) atomicOr(a.err_word, PDA_ERRW_BAD_POSITION);
        return r;
    }
    r.nl = r.L + g;
    r.live = true;
    if (r.L % a.BS) {
        r.tail_id = __ldg(a.block_table + (long long)r.p * a.MB + r.L / a.BS);
        if (r.tail_id < 0 || r.tail_id >= a.NB) {
            if (a.err_word) atomicOr(a.err_word, PDA_ERRW_BAD_BLOCK_ID);   // carried along as it is
        } else {
            r.tail_ref = __ldg(a.refs + r.tail_id);
        }
    }
    return r;
}

__global__ void __launch_bounds__(kScanThreads) pda_fork_scan_kernel(const ScanArgs a) {
    __shared__ int tmp[32], share, first_s[kScanThreads];
    __shared__ long long tmp64[32];
    allow_dependent_launch();
    grid_dependency_wait();
    cg::cluster_group cl = cg::this_cluster();
    // The last CTA lays out the rows.  What the first 1024 ask for is a chain of four loads, requested
    // before the scan of the pool so that the two overlap.
    const bool rows_here = cl.block_rank() == cl.num_blocks() - 1;
    int* const first = a.B <= kScanThreads ? first_s : a.first;
    NewRow row0 = {-1, 0, 0, -1, 0, false};
    if (rows_here) {
        for (int b = threadIdx.x; b < a.B; b += kScanThreads) first[b] = INT_MAX;
        row0 = new_row(a, threadIdx.x);
    }
    long long lo, hi;
    slice_of(cl, a.NB, lo, hi);
    const bool one = hi - lo <= kScanTile;
    Count q = count_slice(cl, a.refs, lo, hi, 1, tmp, &share, [](int r) { return r == 0 ? 1 : 0; });
    const int nfree = q.total;
    int at = q.before;
    for (long long t0 = lo; t0 < hi; t0 += kScanTile) {
        const long long i = t0 + 4 * threadIdx.x;
        int (&r)[4] = q.r;
        int n = 0;
        if (!one) {
            q.n = 0;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                r[u] = i + u < hi ? __ldg(a.refs + i + u) : 1;
                q.n += r[u] == 0;
            }
            q.incl = block_scan(q.n, tmp, n);
        }
        int k = at + q.incl - q.n;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (i + u < hi) a.out_refs[i + u] = r[u];
            if (r[u] == 0) a.free_ids[k++] = (int)(i + u);
        }
        at += n;
    }
    if (cl.num_blocks() > 1) cl.sync();   // nobody leaves with a total still to be read
    if (!rows_here) return;
    // which row is the first of its parent, what each has to get, and where its blocks start in the
    // list of free ones
    __syncthreads();
    for (int i = threadIdx.x; i < a.R; i += kScanThreads) {
        const NewRow r = i < kScanThreads ? row0 : new_row(a, i);
        if (r.live) atomicMin(first + r.p, i);
    }
    __threadfence_block();
    __syncthreads();
    long long used = 0;   // 64 bits: the rows may ask for more than any pool has
    for (int i0 = 0; i0 < a.R; i0 += kScanThreads) {
        const int i = i0 + threadIdx.x;
        const NewRow r = i0 == 0 ? row0 : new_row(a, i);
        int need = 0, flags = 0;
        if (r.live) {
            if (*(volatile int*)(first + r.p) == i) flags |= kRowFirst;
            const bool in_pool = r.tail_id >= 0 && r.tail_id < a.NB;
            if (in_pool && !((flags & kRowFirst) && r.tail_ref == 1)) flags |= kRowCopy;
            need = (flags & kRowCopy) + (r.nl + a.BS - 1) / a.BS - (r.L + a.BS - 1) / a.BS;
        }
        long long n;
        const long long off = used + block_scan((long long)need, tmp64, n) - need;
        used += n;
        if (i < a.R) {
            const bool ok = r.live && (need == 0 || off + need <= nfree);
            if (r.live && !ok && a.err_word) atomicOr(a.err_word, PDA_ERRW_OUT_OF_BLOCKS);
            if (r.live && !ok && (flags & kRowFirst)) first[r.p] = -1;
            int4* rec = reinterpret_cast<int4*>(a.rows + (long long)i * kRowInts);
            rec[0] = make_int4(ok ? r.p : -1, ok ? r.L : 0, ok ? r.nl : 0, ok ? (int)off : 0);
            rec[1] = make_int4(ok ? flags : 0, r.tail_id, 0, 0);
            a.out_lens[i] = ok ? r.nl : 0;
        }
    }
    if (first == first_s) {
        __syncthreads();
        for (int b = threadIdx.x; b < a.B; b += kScanThreads) a.first[b] = first_s[b];
    }
}

struct ForkArgs {
    uint8_t* cache;
    const int* block_table;
    const int* context_lens;
    const int* free_ids;
    const int* first;
    const int* rows;
    int* out_table;
    int* out_refs;
    int* err_word;
    long long NB, block_bytes;
    int B, R, MB, BS, segs;
};

constexpr int kSegEntries = 4 * kPageThreads;   // table entries of one item

// Items: new rows x (table segments, then chunks of the block to copy), then old rows x segments.
// Counts move only where they change: the first child of a row takes over the row's full blocks as
// they are, so a batch that only grows touches the counts of its new blocks alone.
__global__ void __launch_bounds__(kPageThreads) pda_fork_apply_kernel(const ForkArgs a) {
    grid_dependency_wait();
    const long long cpb = chunks_of<1>(a.block_bytes), per = a.segs + cpb;
    const long long rows_items = a.R * per, items = rows_items + (long long)a.B * a.segs;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        if (it < rows_items) {
            const int i = (int)(it / per);
            const long long k = it - i * per;
            const int4* rec = reinterpret_cast<const int4*>(a.rows + (long long)i * kRowInts);
            const int4 r0 = __ldcg(rec), r1 = __ldcg(rec + 1);
            const int p = r0.x, L = r0.y, nl = r0.z, off = r0.w, flags = r1.x, tail_id = r1.y;
            const bool copy = flags & kRowCopy;
            if (k >= a.segs) {
                if (copy)
                    copy_chunk<1>(a.cache + tail_id * a.block_bytes,
                                  a.cache + (long long)__ldcg(a.free_ids + off) * a.block_bytes, a.block_bytes, k - a.segs);
                continue;
            }
            const int full = L / a.BS, h0 = (L + a.BS - 1) / a.BS, h1 = (nl + a.BS - 1) / a.BS;
            const int j0 = (int)k * kSegEntries + threadIdx.x;
            for (int u = 0; u < 4; ++u) {
                const int j = j0 + u * kPageThreads;
                if (j >= a.MB) break;
                int id = -1;
                if (j < full) {
                    id = __ldg(a.block_table + (long long)p * a.MB + j);
                    if (id < 0 || id >= a.NB) {
                        if (a.err_word) atomicOr(a.err_word, PDA_ERRW_BAD_BLOCK_ID);
                    } else if (!(flags & kRowFirst)) {
                        atomicAdd(a.out_refs + id, 1);
                    }
                } else if (j < h0 && !copy) {
                    id = tail_id;
                } else if (j < h1) {
                    id = __ldcg(a.free_ids + off + (j < h0 ? 0 : (copy ? 1 : 0) + j - h0));
                    atomicAdd(a.out_refs + id, 1);
                }
                a.out_table[(long long)i * a.MB + j] = id;
            }
        } else {
            const long long r = it - rows_items;
            const int b = (int)(r / a.segs), seg = (int)(r - (long long)b * a.segs);
            int L = __ldg(a.context_lens + b);
            if (L < 0 || L > a.MB * a.BS) {
                if (seg == 0 && threadIdx.x == 0 && a.err_word) atomicOr(a.err_word, PDA_ERRW_BAD_CONTEXT_LEN);
                L = 0;
            }
            const int held = (L + a.BS - 1) / a.BS, full = L / a.BS;
            const int f = __ldcg(a.first + b);
            const bool heir = f >= 0 && f != INT_MAX;
            bool tail_gone = true;
            if (heir) tail_gone = __ldcg(a.rows + (long long)f * kRowInts + 4) & kRowCopy;
            for (int u = 0; u < 4; ++u) {
                const int j = seg * kSegEntries + u * kPageThreads + threadIdx.x;
                if (j >= held) break;
                if (heir && (j < full || !tail_gone)) continue;
                const int id = __ldg(a.block_table + (long long)b * a.MB + j);
                if (id < 0 || id >= a.NB) {
                    if (a.err_word) atomicOr(a.err_word, PDA_ERRW_BAD_BLOCK_ID);
                } else {
                    atomicSub(a.out_refs + id, 1);
                }
            }
        }
    }
}

// U = blocks in use, of which V have ids below U.  The used block of rank r >= V (its id is at or above U)
// moves to the free block below U of rank r - V.  One scan gives both ranks: a block's rank among the
// used ones, and, as the rest of its id, among the free ones.
__global__ void __launch_bounds__(kScanThreads) pda_compact_scan_kernel(const ScanArgs a) {
    __shared__ int tmp[32], share;
    allow_dependent_launch();
    grid_dependency_wait();
    cg::cluster_group cl = cg::this_cluster();
    long long lo, hi;
    slice_of(cl, a.NB, lo, hi);
    const bool one = hi - lo <= kScanTile;
    Count q = count_slice(cl, a.refs, lo, hi, 0, tmp, &share, [](int r) { return r > 0 ? 1 : 0; });
    const int U = q.total;
    int at = q.before;
    if (U == 0 && cl.block_rank() == 0 && threadIdx.x == 0) a.scalars[0] = a.scalars[1] = 0;
    for (long long t0 = lo; t0 < hi; t0 += kScanTile) {
        const long long i = t0 + 4 * threadIdx.x;
        int (&r)[4] = q.r;
        int n = 0;
        if (!one) {
            q.n = 0;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                r[u] = i + u < hi ? __ldg(a.refs + i + u) : 0;
                q.n += r[u] > 0;
            }
            q.incl = block_scan(q.n, tmp, n);
        }
        int k = at + q.incl - q.n;   // used blocks before this one
        at += n;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const long long id = i + u;
            if (id >= hi) break;
            const bool used = r[u] > 0, low = id < U;
            if (used && !low) a.used_ids[k] = (int)id;
            if (!used && low) a.holes[id - k] = (int)id;
            if (!used || low) a.remap[id] = used ? (int)id : -1;
            if (used || !low) a.out_refs[id] = low ? r[u] : 0;
            k += used;
            if (id == U - 1) {
                a.scalars[0] = U - k;
                a.scalars[1] = k;
            }
        }
    }
    __threadfence();
    cl.sync();   // both lists are complete
    const int M = __ldcg(a.scalars), V = __ldcg(a.scalars + 1);
    for (int k = cl.block_rank() * kScanThreads + threadIdx.x; k < M; k += cl.num_blocks() * kScanThreads) {
        const int from = __ldcg(a.used_ids + V + k), to = __ldcg(a.holes + k);
        a.remap[from] = to;
        a.out_refs[to] = __ldg(a.refs + from);
    }
    if (cl.block_rank() == 0 && threadIdx.x == 0) *a.num_used = U;
}

struct CompactArgs {
    uint8_t* cache;
    const int* block_table;
    const int* context_lens;
    const int* used_ids;
    const int* holes;
    const int* scalars;
    const int* remap;
    int* out_table;
    int* err_word;
    long long NB, block_bytes;
    int B, MB, BS, segs;
};

template <int U>
__global__ void __launch_bounds__(kPageThreads) pda_compact_apply_kernel(const CompactArgs a) {
    grid_dependency_wait();
    const long long cpb = chunks_of<U>(a.block_bytes), tables = (long long)a.B * a.segs;
    const long long items = tables + (long long)__ldcg(a.scalars) * cpb;
    const int* movers = a.used_ids + __ldcg(a.scalars + 1);
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        if (it < tables) {
            const int b = (int)(it / a.segs), seg = (int)(it - (long long)b * a.segs);
            int L = __ldg(a.context_lens + b);
            if (L < 0 || L > a.MB * a.BS) {
                if (seg == 0 && threadIdx.x == 0 && a.err_word) atomicOr(a.err_word, PDA_ERRW_BAD_CONTEXT_LEN);
                L = 0;
            }
            const int held = (L + a.BS - 1) / a.BS;
            for (int u = 0; u < 4; ++u) {
                const int j = seg * kSegEntries + u * kPageThreads + threadIdx.x;
                if (j >= a.MB) break;
                int id = -1;
                if (j < held) {
                    const int old = __ldg(a.block_table + (long long)b * a.MB + j);
                    if (old >= 0 && old < a.NB) id = __ldcg(a.remap + old);
                    if (id < 0 && a.err_word) atomicOr(a.err_word, PDA_ERRW_BAD_BLOCK_ID);
                }
                a.out_table[(long long)b * a.MB + j] = id;
            }
        } else {
            const long long r = it - tables, k = r / cpb;
            copy_chunk<U>(a.cache + (long long)__ldcg(movers + k) * a.block_bytes,
                          a.cache + (long long)__ldcg(a.holes + k) * a.block_bytes, a.block_bytes, r - k * cpb);
        }
    }
}

// ------------------------------------------------------------------------- host side
template <class K, class A>
static int launch_pages(K kernel, const A& args, long long grid, int threads, int cluster, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 0 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args) == cudaSuccess ? PDA_OK : PDA_ERR_LAUNCH;
}

static bool misaligned(const void* p, unsigned a) { return ((uintptr_t)p & (a - 1)) != 0; }

// Whether two buffers share a byte.
static bool overlap(const void* p, long long n, const void* q, long long m) {
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
    return a < b + (uintptr_t)m && b < a + (uintptr_t)n;
}

// Workspace, in ints: [NB] + [NB] lists, [4] scalars, [R][kRowInts] rows, [B] first rows.
static long long workspace_ints(long long B, long long R, long long NB) {
    const long long lists = (2 * NB + 3) & ~3ll;
    return lists + 4 + R * kRowInts + B;
}

}  // namespace pda

using namespace pda;

extern "C" {

long long pda_page_workspace_size(const pda_plan_t* plan, int num_rows, long long num_cache_blocks) {
    if (!plan || pda_workspace_size(plan) < 0 || num_rows < 0 || num_cache_blocks < 1 ||
        num_cache_blocks > (1ll << 31) - 1)
        return -1;
    return 4 * workspace_ints(plan->num_seqs, num_rows, num_cache_blocks);
}

int pda_copy_blocks(const pda_plan_t* plan, const void* src_cache, long long src_blocks, void* dst_cache,
                    long long dst_blocks, const int* pairs, long long num_pairs, int* err_word, void* stream) {
    if (!plan || pda_workspace_size(plan) < 0) return PDA_ERR_INVALID_ARG;
    if (num_pairs < 0 || num_pairs > (1ll << 31) - 1) return PDA_ERR_INVALID_ARG;
    if (src_blocks < 1 || src_blocks > (1ll << 31) - 1 || dst_blocks < 1 || dst_blocks > (1ll << 31) - 1)
        return PDA_ERR_INVALID_ARG;
    if (num_pairs == 0) return PDA_OK;
    if (!src_cache || !dst_cache || !pairs) return PDA_ERR_INVALID_ARG;
    if (misaligned(src_cache, 16) || misaligned(dst_cache, 16) || misaligned(pairs, 4) || misaligned(err_word, 4))
        return PDA_ERR_INVALID_ARG;
    const long long bytes = plan->cache_block_bytes;
    // two pools that overlap without being the same would not be copied block by block
    if (src_cache != dst_cache && overlap(src_cache, src_blocks * bytes, dst_cache, dst_blocks * bytes))
        return PDA_ERR_INVALID_ARG;
    const int sms = device_sm_count();
    if (sms <= 0) return PDA_ERR_CUDA;
    const CopyArgs a{static_cast<const uint8_t*>(src_cache), static_cast<uint8_t*>(dst_cache), pairs, err_word, src_blocks,
                     dst_blocks, bytes, num_pairs};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const long long resident = 8ll * sms;   // 2048 threads per SM
    // one 16-byte word per thread while that still fits one wave (a few blocks: latency), else four
    const long long small = num_pairs * chunks_of<1>(bytes);
    if (small <= resident) return launch_pages(pda_copy_kernel<1>, a, small, kPageThreads, 0, s);
    const long long items = num_pairs * chunks_of<4>(bytes);
    return launch_pages(pda_copy_kernel<4>, a, items < resident ? items : resident, kPageThreads, 0, s);
}

int pda_fork_sequences(const pda_plan_t* plan, void* kv_cache, long long num_cache_blocks, const int* block_table,
                       const int* context_lens, const int* refcounts, int num_rows, const int* parents,
                       const int* new_tokens, int* out_table, int* out_lens, int* out_refcounts, void* workspace,
                       long long workspace_bytes, int* err_word, void* stream) {
    const long long need = pda_page_workspace_size(plan, num_rows, num_cache_blocks);
    if (need < 0) return PDA_ERR_INVALID_ARG;
    const long long NB = num_cache_blocks, B = plan->num_seqs, R = num_rows, MB = plan->max_blocks_per_seq;
    if (!kv_cache || !refcounts || !out_refcounts || !workspace || (B > 0 && (!block_table || !context_lens)) ||
        (R > 0 && (!parents || !out_table || !out_lens)))
        return PDA_ERR_INVALID_ARG;
    if (misaligned(kv_cache, 16) || misaligned(workspace, 16) || misaligned(block_table, 4) ||
        misaligned(context_lens, 4) || misaligned(refcounts, 4) || misaligned(parents, 4) || misaligned(new_tokens, 4) ||
        misaligned(out_table, 4) || misaligned(out_lens, 4) || misaligned(out_refcounts, 4) || misaligned(err_word, 4))
        return PDA_ERR_INVALID_ARG;
    if (workspace_bytes < need) return PDA_ERR_WORKSPACE_TOO_SMALL;
    if (overlap(block_table, 4 * B * MB, out_table, 4 * R * MB) || overlap(context_lens, 4 * B, out_lens, 4 * R) ||
        overlap(refcounts, 4 * NB, out_refcounts, 4 * NB))
        return PDA_ERR_INVALID_ARG;
    const int sms = device_sm_count();
    if (sms <= 0) return PDA_ERR_CUDA;
    int* ws = static_cast<int*>(workspace);
    int* rows = ws + ((2 * NB + 3) & ~3ll) + 4;
    ScanArgs s = {};
    s.refs = refcounts;
    s.NB = NB;
    s.out_refs = out_refcounts;
    s.err_word = err_word;
    s.block_table = block_table;
    s.context_lens = context_lens;
    s.parents = parents;
    s.new_tokens = new_tokens;
    s.out_lens = out_lens;
    s.free_ids = ws;
    s.rows = rows;
    s.first = rows + R * kRowInts;
    s.B = (int)B;
    s.R = num_rows;
    s.MB = (int)MB;
    s.BS = plan->kv_block_size;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int ctas = NB <= kScanOneCta ? 1 : kScanCtas;
    int rc = launch_pages(pda_fork_scan_kernel, s, ctas, kScanThreads, ctas, st);
    if (rc != PDA_OK) return rc;
    ForkArgs f = {};
    f.cache = static_cast<uint8_t*>(kv_cache);
    f.block_table = block_table;
    f.context_lens = context_lens;
    f.free_ids = s.free_ids;
    f.first = s.first;
    f.rows = s.rows;
    f.out_table = out_table;
    f.out_refs = out_refcounts;
    f.err_word = err_word;
    f.NB = NB;
    f.block_bytes = plan->cache_block_bytes;
    f.B = s.B;
    f.R = s.R;
    f.MB = s.MB;
    f.BS = s.BS;
    f.segs = (int)((MB + kSegEntries - 1) / kSegEntries);
    const long long items = R * (f.segs + chunks_of<1>(f.block_bytes)) + B * f.segs;
    if (items == 0) return PDA_OK;
    return launch_pages(pda_fork_apply_kernel, f, items < 8ll * sms ? items : 8ll * sms, kPageThreads, 0, st);
}

int pda_compact_blocks(const pda_plan_t* plan, void* kv_cache, long long num_cache_blocks, const int* block_table,
                       const int* context_lens, const int* refcounts, int* out_table, int* out_refcounts, int* remap,
                       int* num_used, void* workspace, long long workspace_bytes, int* err_word, void* stream) {
    const long long need = pda_page_workspace_size(plan, 0, num_cache_blocks);
    if (need < 0) return PDA_ERR_INVALID_ARG;
    const long long NB = num_cache_blocks, B = plan->num_seqs, MB = plan->max_blocks_per_seq;
    if (!kv_cache || !refcounts || !out_refcounts || !remap || !num_used || !workspace ||
        (B > 0 && (!block_table || !context_lens || !out_table)))
        return PDA_ERR_INVALID_ARG;
    if (misaligned(kv_cache, 16) || misaligned(workspace, 16) || misaligned(block_table, 4) ||
        misaligned(context_lens, 4) || misaligned(refcounts, 4) || misaligned(out_table, 4) ||
        misaligned(out_refcounts, 4) || misaligned(remap, 4) || misaligned(num_used, 4) || misaligned(err_word, 4))
        return PDA_ERR_INVALID_ARG;
    if (workspace_bytes < need) return PDA_ERR_WORKSPACE_TOO_SMALL;
    if (overlap(block_table, 4 * B * MB, out_table, 4 * B * MB) || overlap(refcounts, 4 * NB, out_refcounts, 4 * NB) ||
        overlap(refcounts, 4 * NB, remap, 4 * NB) || overlap(out_refcounts, 4 * NB, remap, 4 * NB))
        return PDA_ERR_INVALID_ARG;
    const int sms = device_sm_count();
    if (sms <= 0) return PDA_ERR_CUDA;
    int* ws = static_cast<int*>(workspace);
    ScanArgs s = {};
    s.refs = refcounts;
    s.NB = NB;
    s.out_refs = out_refcounts;
    s.err_word = err_word;
    s.used_ids = ws;
    s.holes = ws + NB;
    s.scalars = ws + ((2 * NB + 3) & ~3ll);
    s.remap = remap;
    s.num_used = num_used;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int ctas = NB <= kScanOneCta ? 1 : kScanCtas;
    int rc = launch_pages(pda_compact_scan_kernel, s, ctas, kScanThreads, ctas, st);
    if (rc != PDA_OK) return rc;
    CompactArgs c = {};
    c.cache = static_cast<uint8_t*>(kv_cache);
    c.block_table = block_table;
    c.context_lens = context_lens;
    c.used_ids = s.used_ids;
    c.holes = s.holes;
    c.scalars = s.scalars;
    c.remap = remap;
    c.out_table = out_table;
    c.err_word = err_word;
    c.NB = NB;
    c.block_bytes = plan->cache_block_bytes;
    c.B = (int)B;
    c.MB = (int)MB;
    c.BS = plan->kv_block_size;
    c.segs = (int)((MB + kSegEntries - 1) / kSegEntries);
    // how many blocks move is known on the device only: at most half of the pool
    const long long items = B * c.segs + NB / 2 * chunks_of<4>(c.block_bytes);
    if (items == 0) return PDA_OK;
    return launch_pages(pda_compact_apply_kernel<4>, c, items < 8ll * sms ? items : 8ll * sms, kPageThreads, 0, st);
}

}  // extern "C"
