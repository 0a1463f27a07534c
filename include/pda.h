/*
 * pda.h -- C ABI of libpda: single-token decode attention over a paged KV cache with GQA
 * grouping ("paged decode attention"), for NVIDIA GB300 (sm_103a).
 *
 * One decode step, for every sequence b and KV head h: the query_group_size (QG) query rows
 * of head group h (query heads h*QG .. h*QG+QG-1) attend over the sequence's context
 * (context_lens[b] tokens), gathered through the block table in kv_block_size-token blocks.
 * The context is split FA-2 style into partitions of G*256 tokens; pda_decode computes one
 * partial per non-empty partition (normalised output, running max, sum of exponentials) and
 * pda_reduce combines the partials into the softmax-weighted sum of V.
 *
 * Source of the method: the vLLM "tq_decode" page (build_tq_decode_module and the kernel body
 * tq_decode_kernel): argument list, grid (sequence, KV head, partition), block-table walk,
 * partition split with tile_groups_per_partition, mask, online softmax and partial epilogue.
 * The KV element formats here are bf16, fp8 e4m3 with one fp32 scale per token per KV head, and
 * the page's own 4-bit format (TQ4: K codes into 16 centroids times a per-token norm, V codes
 * with a per-token scale and zero point; pda_decode_tq4).
 *
 * Conventions for every call
 *   - Pointers named "device" are device pointers owned by the caller; the library allocates
 *     nothing, frees nothing and keeps no per-call state.  Process-wide state: a cache of the
 *     driver's tensor-map encoder and of per-device occupancy figures, and, in every GPU that
 *     loads the library, two static arrays: 256 slots of per-launch counters, used by the fp8
 *     head-group kernel and by the fused step's grid barrier (each such launch takes the next
 *     slot in turn; the launch's last CTA returns it to zero, so a captured launch can be
 *     replayed; two launches whose slots coincide, one taken 256 such launches after the other,
 *     must not overlap on the GPU, and a graph replay keeps the slot taken at capture), and the
 *     64 MiB array of pda_decode_step_noalloc.  The first such launch on a device looks up the
 *     slots' address; make it before any stream capture, and make no launch on a device after
 *     cudaDeviceReset in the same process.
 *   - Launches are asynchronous on the caller's stream (a cudaStream_t passed as void*;
 *     NULL = the legacy default stream).  Calls that share output or workspace buffers race
 *     if they overlap on the GPU.
 *   - Every call returns a pda_status.  Argument errors are reported before anything is
 *     launched.  Errors found in the data on the device (a context length or a block id out
 *     of range, a pipeline wait that timed out) never fault or trap: the kernel sets a bit
 *     in the optional device word *err_word (atomicOr) and carries on with the rule stated
 *     at pda_decode; the caller reads the word after synchronising.
 */
#ifndef PDA_H
#define PDA_H

#if defined(__GNUC__)
#define PDA_API __attribute__((visibility("default")))
#else
#define PDA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum pda_status {
    PDA_OK = 0,
    PDA_ERR_INVALID_ARG = -1,         /* null pointer, bad size, misaligned buffer, edited plan */
    PDA_ERR_UNSUPPORTED = -2,         /* QG not in {6,8,16}, BS not in {16,32}, head_dim != 128 */
    PDA_ERR_WORKSPACE_TOO_SMALL = -3, /* a size passed with a buffer is below the plan's need */
    PDA_ERR_LAUNCH = -4,              /* the CUDA launch (or tensor-map encode) failed */
    PDA_ERR_NOT_IMPLEMENTED = -5,
    PDA_ERR_CUDA = -6                 /* a CUDA runtime query failed (no device, ...) */
} pda_status;

enum { PDA_KV_BF16 = 0, PDA_KV_FP8_E4M3 = 1, PDA_KV_TQ4 = 2 };
enum { PDA_OUT_BF16 = 0, PDA_OUT_F32 = 1 };
enum { PDA_VARIANT_AUTO = 0, PDA_VARIANT_HEAD_WARPS = 1, PDA_VARIANT_HEAD_GROUPS = 2, PDA_VARIANT_ROW_HALVES = 3 };

/* Bits of the device error word. */
enum {
    PDA_ERRW_BAD_CONTEXT_LEN = 1,   /* context_lens[b] < 0 or > max_blocks_per_seq*kv_block_size */
    PDA_ERRW_BAD_BLOCK_ID = 2,      /* a block-table entry used by the context is outside [0, NB) */
    PDA_ERRW_PIPELINE_TIMEOUT = 4,  /* a bounded wait inside the kernel gave up */
    PDA_ERRW_BAD_POSITION = 8,      /* pda_append_kv: a position >= max_blocks_per_seq*kv_block_size;
                                       pda_fork_sequences: a row that would grow past it, or by < 0;
                                       the token operators: a token that would lie past it */
    PDA_ERRW_BAD_SEQUENCE = 16,     /* pda_fork_sequences: parents[i] >= num_seqs */
    PDA_ERRW_OUT_OF_BLOCKS = 32,    /* pda_fork_sequences: fewer free blocks than the rows need */
    PDA_ERRW_BAD_GROUP = 64,        /* pda_decode_shared: group_starts not ascending within [0, num_seqs] */
    PDA_ERRW_BAD_TOKENS = 128       /* token_starts not ascending within [0, num_tokens]; pda_accept_tokens: a path not ascending
                                       from an index >= 0, or longer than max_path */
};

/*
 * Problem description.  The caller fills the input fields and calls pda_plan, which checks
 * them and fills the output fields.  The launch calls recompute the outputs from the inputs
 * and reject a plan whose outputs were edited (PDA_ERR_INVALID_ARG).
 * Field names follow build_tq_decode_module's arguments.
 */
typedef struct pda_plan_t {
    /* ---- inputs ---- */
    int num_seqs;                  /* B >= 0 (0 = nothing to do)                                  */
    int num_kv_heads;              /* Hk >= 1                                                      */
    int query_group_size;          /* QG = query heads / KV heads, one of 6, 8, 16                */
    int head_dim;                  /* D, must be 128                                              */
    int kv_block_size;             /* BS tokens per cache block, 16 or 32                         */
    int max_blocks_per_seq;        /* MB, row length of the block table, >= 1                     */
    int tile_groups_per_partition; /* G >= 1, or 0 = smallest G with num_partitions <= max_partitions */
    int max_partitions;            /* cap used when G == 0 (0 = no cap, i.e. G = 1)              */
    int kv_dtype;                  /* PDA_KV_BF16, PDA_KV_FP8_E4M3 or PDA_KV_TQ4                  */
    float softmax_scale;           /* <= 0 selects 1/sqrt(head_dim)                                */
    int wait_timeout_ns;           /* limit of each bounded wait inside pda_decode's kernel, in
                                      nanoseconds; 0 = 1 s.  A wait that gives up sets
                                      PDA_ERRW_PIPELINE_TIMEOUT.  Copies already in flight are
                                      always waited for (up to 1 s) before a warp leaves.  No
                                      counterpart on the pages; small values exist for testing
                                      the timeout path.                                          */
    int kernel_variant;            /* how pda_decode lays out the partition pass on the GPU (the
                                      results agree within the parity tolerances; each variant is
                                      deterministic on its own):
                                        PDA_VARIANT_AUTO (0): chosen at launch from the shape
                                          (head groups for fp8 and row halves for bf16 with
                                          query_group_size 16 when the plan has at least two
                                          units per resident CTA, else head warps),
                                        PDA_VARIANT_HEAD_WARPS (1): one warp per (sequence, KV head,
                                          partition) unit, any format,
                                        PDA_VARIANT_HEAD_GROUPS (2): one CTA per (sequence, group of
                                          up to 4 KV heads, partition) unit, fp8 e4m3 only,
                                        PDA_VARIANT_ROW_HALVES (3): one CTA per (sequence, KV head,
                                          partition) unit, its 16 query rows split between two
                                          warps, bf16 with query_group_size 16 only (the
                                          partials equal head warps' bit for bit).
                                      pda_decode_fused runs head groups where pda_decode would,
                                      else head warps.  No counterpart on the pages.              */
    /* ---- outputs of pda_plan ---- */
    int num_partitions;            /* P = ceil(MB*BS / W)                                          */
    int partition_tokens;          /* W = G * 256                                                 */
    int resolved_tile_groups;      /* G actually used                                              */
    float resolved_softmax_scale;
    long long cache_block_bytes;   /* bytes per cache block (data region + metadata region)       */
    long long meta_offset_bytes;   /* offset of the metadata region inside a block                */
    long long workspace_bytes;     /* bytes of partial_out + exp_sums + max_logits                 */
} pda_plan_t;

/*
 * pda_plan -- host only; launches nothing.
 * Checks the inputs (build_tq_decode_module's asserts: QG in {6,8,16}, BS in {16,32}, G >= 1)
 * and fills the outputs.  G == 0 follows the long-context launcher policy described with
 * tile_groups_per_partition on the same page: the smallest G with ceil(MB*BS / (G*256)) <=
 * max_partitions (the page's example: BS 32, cap 32 partitions -> G = 5, 32*5*256 = 40960
 * tokens).  Also rejects sizes whose index arithmetic would not fit the kernels' int32/int64
 * ranges (PDA_ERR_INVALID_ARG).
 *
 * Cache block layout (the page's stride block; formats of this library):
 *   data region   [BS slots][Hk heads][K: D elements | V: D elements], elements bf16, e4m3, or
 *                 TQ4 4-bit codes (two per byte, dimension 2j in the low nibble of byte j),
 *   meta region   at meta_offset_bytes: fp8: fp32 [Hk][2: K scale, V scale][BS];
 *                 TQ4: fp16 [Hk][3: k_norm, v_scale, v_zero][BS]; bf16: none.
 *   cache_block_bytes = BS*Hk*2*D*elem (+ Hk*2*BS*4 for fp8), or BS*Hk*D + Hk*3*BS*2 for TQ4.
 * Returns PDA_OK, PDA_ERR_INVALID_ARG or PDA_ERR_UNSUPPORTED.
 */
PDA_API int pda_plan(pda_plan_t* plan);

/*
 * pda_decode -- the partition pass (tq_decode_kernel: steps B to G).
 *   query          device, bf16 [B][Hk*QG][D] contiguous, 16-byte aligned.
 *                  query, block_table and context_lens may instead be pinned host memory that
 *                  the device can address (cudaHostAlloc, or cudaHostRegister, under unified
 *                  addressing): the kernels then read them across the host link, with no copy.
 *   kv_cache       device, bytes [num_cache_blocks][cache_block_bytes], 16-byte aligned.
 *   num_cache_blocks  NB >= 1, < 2^31; block ids outside [0, NB) are data errors.
 *   block_table    device, int32 [B][max_blocks_per_seq]; only entries t/BS for t < ctx are read.
 *   context_lens   device, int32 [B], each in [0, MB*BS].
 *   partial_out    device, fp32 [B][Hk][P][QG][D]   (normalised partial o_p)
 *   exp_sums       device, fp32 [B][Hk][P][QG]      (l_p = sum of exp(s - m_p) over the partition)
 *   max_logits     device, fp32 [B][Hk][P][QG]      (m_p = max of s = softmax_scale * q.k)
 *   err_word       device int or NULL.
 *   stream         cudaStream_t or NULL.
 * Only partitions p < ceil(ctx_b / W) are written; rows >= QG do not exist in the layout;
 * other partitions' slots are left untouched.
 * Data errors: a context length out of range is treated as 0 (nothing written for that
 * sequence) and sets PDA_ERRW_BAD_CONTEXT_LEN; a block id out of range is read as zeros
 * (the tensor copy's out-of-bounds fill) and sets PDA_ERRW_BAD_BLOCK_ID.
 * A TQ4 plan is rejected (PDA_ERR_INVALID_ARG): that format needs pda_decode_tq4.
 */
PDA_API int pda_decode(const pda_plan_t* plan, const void* query, const void* kv_cache, long long num_cache_blocks,
               const int* block_table, const int* context_lens, float* partial_out, float* exp_sums,
               float* max_logits, int* err_word, void* stream);

/*
 * pda_decode_tq4 -- the partition pass for a TQ4 cache (plan->kv_dtype == PDA_KV_TQ4): the
 * page's own format, decoded as its STEP F does (tq_decode_kernel):
 *   K[t][d] = centroids[code] * k_norm[t],   V[t][d] = code * v_scale[t] + v_zero[t]
 * with code the 4-bit code of dimension d of token t (K codes: bytes 0..63 of the token-head
 * row, V codes: bytes 64..127; dimension 2j in the low nibble of byte j) and the fp16 fields
 * of the metadata region.  The query is taken as given: on the page it arrives already rotated
 * into the basis the codes were made in (STEP B), so the rotation is the caller's.
 *   centroids      device, fp32 [16], finite (STEP A's codebook).
 * Every other argument, the partial layout and the error rules are those of pda_decode;
 * pda_reduce combines the partials.  A non-TQ4 plan is rejected (PDA_ERR_INVALID_ARG).
 */
PDA_API int pda_decode_tq4(const pda_plan_t* plan, const void* query, const void* kv_cache,
                           long long num_cache_blocks, const float* centroids, const int* block_table,
                           const int* context_lens, float* partial_out, float* exp_sums, float* max_logits,
                           int* err_word, void* stream);

/*
 * pda_reduce -- combines the partials of pda_decode (the reduce that follows the partition
 * pass; the page's per-partition exp_sums / max_logits outputs exist for it):
 *   M = max_p m_p,  w_p = l_p * exp(m_p - M),  out = sum_p (w_p / sum_q w_q) * o_p
 * over p < ceil(ctx_b / W).  One partition is copied bit for bit; ctx 0 gives 0.
 *   out            device, [B][Hk*QG][D], bf16 (PDA_OUT_BF16, round to nearest even) or fp32.
 *                  out and context_lens may be pinned host memory, as for pda_decode's inputs.
 * A context length out of range gives 0 and sets PDA_ERRW_BAD_CONTEXT_LEN.
 */
PDA_API int pda_reduce(const pda_plan_t* plan, const int* context_lens, const float* partial_out,
               const float* exp_sums, const float* max_logits, void* out, int out_dtype, int* err_word,
               void* stream);

/*
 * pda_append_kv -- the write side of the same cache: stores K and V of one new token for every
 * sequence b with positions[b] >= 0, at token index positions[b]: cache block
 * block_table[b][pos / BS], slot pos % BS (the paged slot formula of the KV insert on the
 * DeepSeek attention-front page: block = slot // block_size, offset = slot % block_size, and a
 * negative slot means no write).
 *   k_new, v_new  device, bf16 [B][Hk][D], 8-byte aligned
 *   kv_cache      device, the cache pda_decode reads (16-byte aligned)
 *   positions     device, int32 [B]
 * bf16 caches store the values as given.  fp8 caches store, per (token, KV head) and separately
 * for K and V, scale = absmax / 448 in fp32 (1 when the row is all zero) in the metadata region
 * and codes e4m3(x / scale), both divisions correctly rounded in fp32, the conversion rounding to
 * nearest even and saturating at +-448.  TQ4 caches are not supported (PDA_ERR_UNSUPPORTED): the
 * pages give no encoder for that format (its rotation and codebook are not on them).
 * Data errors (nothing is written for that sequence): a position >= MB*BS sets
 * PDA_ERRW_BAD_POSITION, a block id outside [0, NB) sets PDA_ERRW_BAD_BLOCK_ID.
 * Two sequences whose table entries name the same block and slot race.
 */
PDA_API int pda_append_kv(const pda_plan_t* plan, const void* k_new, const void* v_new, void* kv_cache,
                          long long num_cache_blocks, const int* block_table, const int* positions, int* err_word,
                          void* stream);

/*
 * pda_decode_fused -- one launch for the whole step: the partition pass of pda_decode, then, in
 * the same launch, the reduce of pda_reduce.  The launch is cooperative (every CTA resident): once
 * every CTA has written its partials they meet at a grid barrier (a bounded wait on a counter of
 * the library's per-launch slots; a wait that gives up sets PDA_ERRW_PIPELINE_TIMEOUT), and then
 * all of them merge the output rows, each row in partition order with pda_reduce's arithmetic, so
 * results are deterministic and equal pda_decode + pda_reduce's bit for bit.  On head-warp plans a
 * (sequence, KV head) whose context fits one partition is written to `out` by its partition's
 * epilogue (its partial is not stored).  The rows of a sequence with no tokens (context 0, or an
 * invalid length, which also sets PDA_ERRW_BAD_CONTEXT_LEN) are written as zeros, as pda_reduce
 * writes them.
 *   partial_out, exp_sums, max_logits   as for pda_decode (scratch here)
 *   counters   device int32 [B][Hk], zero: reserved (an earlier form of this step counted arrivals
 *              there); the call leaves them zero.
 *   out, out_dtype                      as for pda_reduce
 * query, block_table, context_lens and out may be pinned host memory, as for pda_decode.
 * Calls that share partials race if they overlap on the GPU; fewer than 256 launches of this
 * library's counter-slot kernels may be in flight on a device at once.
 * A TQ4 plan is rejected (PDA_ERR_INVALID_ARG): that format is read by pda_decode_tq4 only.
 * On GB300 this step measured slower than pda_decode followed by pda_reduce on every workload
 * timed (the reduce launch is already resident when the partition pass ends; the barrier and
 * the merge after it cost more); it exists for callers that want a single launch.
 */
PDA_API int pda_decode_fused(const pda_plan_t* plan, const void* query, const void* kv_cache,
                             long long num_cache_blocks, const int* block_table, const int* context_lens,
                             float* partial_out, float* exp_sums, float* max_logits, int* counters, void* out,
                             int out_dtype, int* err_word, void* stream);

/*
 * pda_decode_step_noalloc -- pda_decode followed by pda_reduce, for callers that cannot
 * allocate device memory when they run a step: for example a plugin inside an engine that owns
 * every byte of device memory, or code that must not call cudaMalloc because it can synchronise
 * the device.  Such callers can pass inputs and outputs but no partials workspace, so this entry
 * point keeps the partials in a fixed array inside the library.  The pages describe no such
 * entry point; it has no counterpart there.
 *   Arguments are those of pda_decode and pda_reduce without the three partial buffers:
 *   query, kv_cache, num_cache_blocks, block_table, context_lens as for pda_decode; out and
 *   out_dtype as for pda_reduce.
 * The array holds PDA_NOALLOC_SCRATCH_BYTES (64 MiB) on every GPU that loads the library, until
 * the process exits.  A plan whose partials (B*Hk*P*QG*(D*4 + 8) bytes, each part rounded up to
 * 256 bytes) do not fit returns PDA_ERR_WORKSPACE_TOO_SMALL and launches nothing.
 * query, block_table, context_lens and out may be pinned host memory, as for pda_decode and
 * pda_reduce.
 * The first call on a device looks up the array's device address (cudaGetSymbolAddress) with
 * that device current; make that first call before any stream capture.  The address is kept for
 * the life of the process: after cudaDeviceReset, or anything else that destroys the device's
 * primary context, do not call this entry point again in the same process.  The call allocates
 * nothing and frees nothing.
 * All calls share the one array and it keeps the last call's contents (nothing in it needs to
 * start at zero); calls that overlap on the GPU, on any streams, race.
 * A TQ4 plan is rejected (PDA_ERR_INVALID_ARG): that format is read by pda_decode_tq4 only.
 */
#define PDA_NOALLOC_SCRATCH_BYTES (64ll << 20)
PDA_API int pda_decode_step_noalloc(const pda_plan_t* plan, const void* query, const void* kv_cache,
                                    long long num_cache_blocks, const int* block_table, const int* context_lens,
                                    void* out, int out_dtype, int* err_word, void* stream);

/*
 * pda_kernel_variant -- host only; launches nothing.  The partition-pass layout pda_decode would
 * launch for this plan on the current device: PDA_VARIANT_HEAD_WARPS, PDA_VARIANT_HEAD_GROUPS or
 * PDA_VARIANT_ROW_HALVES (plan->kernel_variant resolved, PDA_VARIANT_AUTO included).  Returns PDA_ERR_INVALID_ARG for
 * a NULL or edited plan, PDA_ERR_CUDA when the device cannot be queried.  No counterpart on the
 * pages.
 */
PDA_API int pda_kernel_variant(const pda_plan_t* plan);

/* ---------------------------------------------------------------- pages of the cache
 * A pool of num_cache_blocks blocks is shared by the sequences of a batch.  refcounts[id] is the
 * number of block-table entries that hold block id (entries of any batch the caller keeps, of
 * prefixes and so on); a block with count 0 is free.  Sequence b holds the first
 * ceil(context_lens[b] / kv_block_size) entries of its table row.  The plan gives the block size
 * in bytes (any kv_dtype), num_seqs, max_blocks_per_seq and kv_block_size.
 *
 * A call moves the blocks of the pool it is given, and nothing else that block ids index:
 *   - Other pools under the same tables (one per layer of a model).  After a fork they need the same copies: for each
 *     new row i whose parent p's length L is no multiple of kv_block_size, the pair (block_table[p][j],
 *     out_table[i][j]) with j = L / kv_block_size, where the two differ.  After a compaction: the pairs
 *     (id, remap[id]) for every id.  Both by pda_copy_blocks within each pool.
 *   - Block summaries (pda_summarize_blocks).  After a compaction or a copy the rows of moved blocks have to be moved
 *     by the same pairs, or renewed (pda_summarize_blocks with since NULL and the new tables); until then
 *     pda_score_blocks reads what the id stood for before, without an error bit.  After a fork a copied block's row is
 *     renewed by the call that follows the next append; before that, by since[i] = out_lens[i] - 1.
 *
 * pda_copy_blocks: block pairs[2i] of src_cache to block pairs[2i+1] of dst_cache, whole
 * (data and metadata region), for i < num_pairs.
 *   src_cache, dst_cache   device memory, or pinned host memory that the device can address (a
 *                          block swapped out or in); the same pool, or two that do not overlap
 *   pairs                  device, int32 [num_pairs][2]; a pair with a negative id is skipped
 * A source may be named any number of times.  A destination that is also another pair's source or
 * destination races with it (no order is kept).  An id past its pool sets PDA_ERRW_BAD_BLOCK_ID and
 * its pair is skipped.
 */
PDA_API int pda_copy_blocks(const pda_plan_t* plan, const void* src_cache, long long src_blocks, void* dst_cache,
                            long long dst_blocks, const int* pairs, long long num_pairs, int* err_word, void* stream);

/* Bytes of the workspace (16-byte aligned device memory) of pda_fork_sequences with num_rows new rows
 * and of pda_compact_blocks (num_rows = 0); -1 for an invalid plan or size. */
PDA_API long long pda_page_workspace_size(const pda_plan_t* plan, int num_rows, long long num_cache_blocks);

/*
 * pda_fork_sequences -- a batch laid out anew: row i of the new batch is sequence parents[i] of the
 * old one, grown by new_tokens[i] positions.  One call forks (a parent named by several rows),
 * reorders, keeps, grows and frees (a sequence that no row names): the step of a beam search, of
 * parallel sampling, or of continuous batching between two decode steps.
 *   - Full blocks of the parent are shared.  Its partial last block stays with the first row that
 *     names it when nothing else holds that block (count 1); every other row gets a copy of it in a
 *     fresh block, so that rows may append independently.
 *   - Positions past the last block get fresh blocks.  Fresh blocks are the free blocks of
 *     `refcounts`, lowest id first, in row order (a row's copy before its new blocks).
 *   - out_refcounts = refcounts - the entries the old sequences hold + those the new rows hold.
 *   parents        device, int32 [num_rows], negative: an empty row
 *   new_tokens     device, int32 [num_rows], or NULL (no growth)
 *   out_table      device, int32 [num_rows][max_blocks_per_seq]; entries a row does not hold are -1
 *   out_lens       device, int32 [num_rows]
 *   out_refcounts  device, int32 [num_cache_blocks]
 * block_table, context_lens and refcounts are not changed and must not overlap their outputs, and
 * blocks are copied only into blocks that were free: until the caller drops it the old batch stays
 * valid, so a call that set an error bit can be repeated with other rows.
 * Data errors: a parent >= num_seqs (PDA_ERRW_BAD_SEQUENCE), a length past max_blocks_per_seq *
 * kv_block_size or a negative growth (PDA_ERRW_BAD_POSITION), and a row whose fresh blocks lie past
 * the last free one (PDA_ERRW_OUT_OF_BLOCKS; the rows before it have theirs) give an empty row (length
 * 0).  A context length out of range counts as 0 (PDA_ERRW_BAD_CONTEXT_LEN).  A held id outside the
 * pool is carried along and counted nowhere (PDA_ERRW_BAD_BLOCK_ID).
 */
PDA_API int pda_fork_sequences(const pda_plan_t* plan, void* kv_cache, long long num_cache_blocks,
                               const int* block_table, const int* context_lens, const int* refcounts, int num_rows,
                               const int* parents, const int* new_tokens, int* out_table, int* out_lens,
                               int* out_refcounts, void* workspace, long long workspace_bytes, int* err_word,
                               void* stream);

/*
 * pda_compact_blocks -- moves the blocks in use (count > 0) to ids 0 .. U-1, U their number, so that
 * the rest of the pool can be given back.  Blocks below U stay; the k-th block in use at or above U
 * moves to the k-th free id below U.
 *   out_table      device, int32 [num_seqs][max_blocks_per_seq]: the table with the new ids; entries a
 *                  sequence does not hold are -1
 *   out_refcounts  device, int32 [num_cache_blocks]
 *   remap          device, int32 [num_cache_blocks]: the new id of each block, -1 for a free one (for
 *                  tables the caller keeps elsewhere)
 *   num_used       device, int32 [1]: U
 * The inputs are not changed, must not overlap their outputs, and stay valid until a block at or past
 * U is overwritten.  A held id that is outside the pool or free becomes -1 (PDA_ERRW_BAD_BLOCK_ID).
 */
PDA_API int pda_compact_blocks(const pda_plan_t* plan, void* kv_cache, long long num_cache_blocks,
                               const int* block_table, const int* context_lens, const int* refcounts, int* out_table,
                               int* out_refcounts, int* remap, int* num_used, void* workspace,
                               long long workspace_bytes, int* err_word, void* stream);

/* ---------------------------------------------------------------- attention over selected blocks
 * For long contexts: keep a summary of every block, score the blocks of a sequence against the step's
 * query, select some of them per (sequence, KV head), attend to those.
 *
 * A summary holds, per KV head, the largest and the smallest value of each key dimension over the
 * block's tokens: bf16 [num_cache_blocks][num_kv_heads][2: max, min][128], rounded outwards (bf16
 * keys exactly), pda_summary_size bytes, 16-byte aligned.  Keys must be finite.  Rows belong to block ids: the page
 * operators move blocks, not summaries (see there).
 */
PDA_API long long pda_summary_size(const pda_plan_t* plan, long long num_cache_blocks);

/*
 * pda_summarize_blocks -- writes the summaries of the blocks that hold tokens since[b] ..
 * context_lens[b]-1 of each sequence, each over all its tokens below context_lens[b] (call it after
 * pda_append_kv with the position appended, or with since NULL for whole contexts).
 *   since      device, int32 [num_seqs] or NULL
 *   centroids  device, fp32 [16] for a TQ4 plan, else NULL
 * A block id outside the pool is skipped (PDA_ERRW_BAD_BLOCK_ID).  Sequences that share a block must
 * give it the same tokens, or race.
 */
PDA_API int pda_summarize_blocks(const pda_plan_t* plan, const void* kv_cache, long long num_cache_blocks,
                                 const int* block_table, const int* context_lens, const int* since,
                                 const float* centroids, void* summaries, int* err_word, void* stream);

/*
 * pda_score_blocks -- scores[b][h][j] = softmax_scale * max over the query rows r of KV head h of
 *   sum_d max(q_rd, 0) * kmax_d + min(q_rd, 0) * kmin_d,
 * an upper bound of every logit of block j, but for the rounding of the fp32 sums.  scores: device, fp32 [num_seqs][num_kv_heads]
 * [max_blocks_per_seq]; entries past the context are left as they are.  A block id outside the pool
 * scores -inf (PDA_ERRW_BAD_BLOCK_ID).  query as for pda_decode, in device memory.
 */
PDA_API int pda_score_blocks(const pda_plan_t* plan, const void* query, const void* summaries,
                             long long num_cache_blocks, const int* block_table, const int* context_lens,
                             float* scores, int* err_word, void* stream);

/*
 * pda_select_blocks -- per (sequence, KV head): the first num_first blocks, the last num_last, and of
 * the others those with the highest scores (of equal scores the first; NaN lowest), num_select blocks
 * in all, or every block where there are no more.
 *   sel_table   device, int32 [num_seqs][num_kv_heads][num_select]: their block ids in the sequence's
 *               order, then -1
 *   sel_lens    device, int32 [num_seqs][num_kv_heads]: their tokens
 *   sel_blocks  device, int32 like sel_table, or NULL: their indices in the sequence
 * num_first + num_last <= num_select.  With num_last >= 1 the newest block, the only one that may be
 * partly filled, is always among them.
 */
PDA_API int pda_select_blocks(const pda_plan_t* plan, const float* scores, const int* block_table,
                              const int* context_lens, int num_select, int num_first, int num_last, int* sel_table,
                              int* sel_lens, int* sel_blocks, int* err_word, void* stream);

/*
 * pda_decode_selected -- a decode step over selected blocks, with one table row and one length per
 * (sequence, KV head), in one launch: each (sequence, KV head) is split over the warps of a thread-block
 * cluster and joined in its shared memory.  With kernel_variant head warps it is the partition pass and the
 * reduce instead, whose partials are those of pda_decode over the same lists.  That form is slower but for few units
 * of long lists (8 units of 65536 fp8 tokens 61 us against 66): a unit's cluster is at most eight SMs.
 *   plan        as for pda_decode, with max_blocks_per_seq = num_select (kernel_variant automatic or
 *               head warps, else PDA_ERR_UNSUPPORTED)
 *   centroids   device, fp32 [16] for a TQ4 plan, else NULL
 *   sel_table   device, int32 [num_seqs][num_kv_heads][max_blocks_per_seq]
 *   sel_lens    device, int32 [num_seqs][num_kv_heads]: tokens; all blocks but the last are full
 *   partial_out, exp_sums, max_logits   as for pda_decode with kernel_variant head warps; otherwise not
 *               looked at (may be NULL)
 *   out, out_dtype and the data errors as for pda_decode and pda_reduce
 * query may be pinned host memory as for pda_decode, and out as for pda_reduce.
 */
PDA_API int pda_decode_selected(const pda_plan_t* plan, const void* query, const void* kv_cache,
                                long long num_cache_blocks, const float* centroids, const int* sel_table,
                                const int* sel_lens, float* partial_out, float* exp_sums, float* max_logits, void* out,
                                int out_dtype, int* err_word, void* stream);

/* ---------------------------------------------------------------- sequences that share a prefix
 * pda_decode_shared -- a decode step for a batch whose sequences share prefixes in groups: sequences
 * group_starts[g] .. group_starts[g+1]-1 attend over the first prefix_lens[g] tokens of group g's blocks and then
 * over the context_lens[b] tokens of their own.  The prefix is read once for all of a group's query rows
 * (tensor-core products over 256 rows at a time) instead of once per sequence; out equals a decode over
 * the concatenation.  It pays where a prefix is shared and is the larger part.  Own tokens of one (sequence, KV head)
 * run on at most eight SMs, and fp8 prefixes are converted whatever the rows, so groups of one sequence, and few
 * sequences with thousands of tokens of their own, are better served by pda_decode over concatenated tables.
 *   prefix_plan    num_seqs = groups (>= 1), max_blocks_per_seq = row length of prefix_table, and
 *                  tile_groups_per_partition (pda_shared_tile_groups gives a good one): a prefix is cut into at
 *                  most num_partitions + 1 pieces.  kernel_variant is not looked at.
 *   plan           num_seqs = sequences; as for pda_decode over the sequences' own tokens
 *                  (heads, group size, block size, kv_dtype and softmax_scale equal in both plans;
 *                  bf16 and fp8: a TQ4 plan is PDA_ERR_UNSUPPORTED; kernel_variant and the partition length
 *                  are not looked at)
 *   group_starts   device, int32 [groups + 1], ascending; sequences outside [group_starts[0],
 *                  group_starts[groups]) have no prefix
 *   prefix_table   device, int32 [groups][prefix_plan->max_blocks_per_seq]
 *   prefix_lens    device, int32 [groups]; a prefix may end inside a block
 *   block_table, context_lens   device, the sequences' own blocks and lengths (0: prefix only)
 *   workspace      device, pda_shared_workspace_size bytes, 32-byte aligned
 *   query, out, out_dtype as for pda_decode and pda_reduce (query and out may be pinned host memory)
 * The weights of the prefix part are rounded to bf16 (bf16 KV), or they, V's scale and the scaled V to f16 (fp8 KV),
 * before their product, so an fp32 out carries that rounding: at most 2^-8, or 3 * 2^-11, of each term.  With fp8 KV
 * a weight below 2^-21 of its row's largest is off by at most 2^-32 of that one instead; and of the prefix's aligned
 * 128 tokens, with f the largest V scale among them, one whose scale is below 2^-15 f has that scale off by up to
 * 2^-26 f, and an element of V below 2^-15 f is off by up to 2^-26 f.  pda_decode rounds less (bf16 KV: weights to
 * 2^-16; fp8 KV: once to f16): moving a batch here from there changes an fp32 out by this much.
 * Data errors: a prefix length out of range counts as 0 (PDA_ERRW_BAD_CONTEXT_LEN); group_starts that are not
 * ascending within [0, num_seqs] set PDA_ERRW_BAD_GROUP, and the step runs without prefixes; block ids as
 * for pda_decode.
 *
 * pda_shared_tile_groups -- host only: tile_groups_per_partition of a prefix plan for num_groups prefixes of up
 * to prefix_blocks blocks, with which a prefix is cut into as many pieces as the GPU's SMs have room for.
 * pda_shared_workspace_size -- bytes of the workspace; -1 where the plans do not belong together.
 */
PDA_API int pda_shared_tile_groups(const pda_plan_t* plan, int num_groups, int prefix_blocks);
PDA_API long long pda_shared_workspace_size(const pda_plan_t* prefix_plan, const pda_plan_t* plan);
PDA_API int pda_decode_shared(const pda_plan_t* prefix_plan, const pda_plan_t* plan, const void* query,
                              const void* kv_cache, long long num_cache_blocks, const int* group_starts,
                              const int* prefix_table, const int* prefix_lens, const int* block_table,
                              const int* context_lens, void* workspace, long long workspace_bytes, void* out,
                              int out_dtype, int* err_word, void* stream);

/* ---------------------------------------------------------------- many tokens of the cache
 * Tokens of a batch, several per sequence, are rows of packed arrays: rows token_starts[b] .. token_starts[b+1]-1 are
 * sequence b's.
 *   token_starts   device, int32 [num_seqs + 1], ascending within [0, num_tokens]; rows before the first start and from the
 *                  last one on (a padded batch) are not looked at and not written
 * token_starts that do not ascend set PDA_ERRW_BAD_TOKENS, and the call moves or computes nothing.
 *
 * pda_write_kv -- K and V of any number of new tokens per sequence into the cache, in its format: a prompt, a part of one, or
 * drafted tokens.  Row i of sequence b goes to position positions[b] + i - token_starts[b].
 *   k_new, v_new   device, bf16, 16-byte aligned; row i starts k_stride (v_stride) elements after row i-1, a multiple of 8 and
 *                  at least Hk*128, and holds [Hk][128]: rows of a fused projection need no copy
 *   positions      device, int32 [num_seqs]; negative: none of the sequence's rows is written
 *   centroids      device, fp32 [16], finite, in any order, for a TQ4 plan, else NULL
 * bf16 and fp8 caches get the bytes that pda_append_kv would give them.  TQ4 (keys already in the basis of the codebook, as the
 * query; K and V finite): K: k_norm = the norm of the row, taken in 64 bits and rounded once to fp16 (at most 65504),
 * code = how many midpoints of neighbouring centroids, (c + c') / 2 in fp32, lie below k_d / k_norm in fp32 (of the sorted
 * codebook; a row of norm 0 is divided by 1); V: v_zero = fp16(min v), v_scale = fp16((max v - min v) / 15), both kept within
 * +-65504, code =
 * (v_d - v_zero) / v_scale (by 1 where v_scale is 0), rounded to the nearest even integer and brought into 0 .. 15; all
 * quotients and differences correctly rounded in fp32.
 * Data errors: a row past max_blocks_per_seq*kv_block_size (PDA_ERRW_BAD_POSITION) or whose block id is outside the pool
 * (PDA_ERRW_BAD_BLOCK_ID) is not written.  Rows that name the same slot race.
 */
PDA_API int pda_write_kv(const pda_plan_t* plan, const void* k_new, const void* v_new, long long k_stride,
                         long long v_stride, long long num_tokens, void* kv_cache, long long num_cache_blocks,
                         const float* centroids, const int* block_table, const int* token_starts, const int* positions,
                         int* err_word, void* stream);

/*
 * pda_read_kv -- the other direction: tokens of the cache, gathered and dequantised.
 *   k_out, v_out   device, [num_tokens][Hk][128], bf16 (PDA_OUT_BF16, rounded to nearest even) or fp32, 16-byte aligned;
 *                  one of them may be NULL
 *   the others, and the data errors, as for pda_write_kv: rows that it would not write are left as they are
 * Values: bf16 as stored; fp8 code * scale, TQ4 centroids[code] * k_norm and code * v_scale + v_zero, in fp32.
 */
PDA_API int pda_read_kv(const pda_plan_t* plan, const void* kv_cache, long long num_cache_blocks, const float* centroids,
                        const int* block_table, const int* token_starts, const int* positions, long long num_tokens,
                        void* k_out, void* v_out, int out_dtype, int* err_word, void* stream);

/* ---------------------------------------------------------------- drafted tokens
 * pda_decode_tree -- a step for drafted tokens, several per sequence, in a chain or a tree: token i of sequence b attends over
 * the context_lens[b] cached tokens and over those of the sequence's drafted tokens that its mask names.  The drafted tokens'
 * K and V lie in the cache behind the cached ones, token i at position context_lens[b] + i (pda_write_kv with positions =
 * context_lens).
 *   plan          num_seqs, heads, block size and max_blocks_per_seq; any kv_dtype.  kernel_variant and the partition length are
 *                 not looked at.
 *   query         device, bf16 [num_tokens][Hk*QG][128], 16-byte aligned, in device memory or pinned host memory
 *   centroids     device, fp32 [16], finite, for a TQ4 plan, else NULL
 *   block_table, context_lens   device, int32, as for pda_decode; context_lens without the drafted tokens
 *   token_starts  device, int32 [num_seqs + 1] (see above); a sequence may have no drafted token
 *   tree_masks    device, 64-bit words [num_tokens][mask_words], 8-byte aligned: bit j % 64 of word j / 64 of row i says
 *                 whether token i sees drafted token j of its sequence (its own bit too).  Tokens past the words' bits are seen
 *                 by none; bits past the sequence's tokens are not looked at.  NULL (and mask_words 0): a chain, i sees 0 .. i.
 *   window        0: every cached token is seen.  Else a token at position p sees the cached tokens t with p - t < window, and
 *                 t < num_first.  p is context_lens[b] + the number of drafted tokens other than itself that it sees.  Masks
 *                 alone say which drafted tokens are seen; in a chain they count as cached ones.
 *   workspace     device, 32-byte aligned, pda_tree_workspace_size bytes; one made under the same plan for more tokens will do
 *   out           [num_tokens][Hk*QG][128], as for pda_reduce but 16-byte aligned in either type; a row that sees nothing is 0
 * K and V of the tokens that any of the sequence's rows sees must be finite: a row that does not see one of them still has it in
 * its products, with weight 0.  What no row sees (cached tokens before the window of a drafted token at position context_lens[b],
 * drafted tokens that no mask names, what lies behind them) is not read, or not used, whatever it holds; block ids of blocks
 * wholly before that window and behind the first num_first tokens are not looked at.
 * The roundings are those of the prefix in pda_decode_shared; fp8: also the query's, the sum of two e4m3 parts, by at most 2^-17 of
 * the row's largest |q|; TQ4: the weights to f16 as there, V rounded once to f16 (2^-11 of its value, or 2^-33 of the step's
 * largest 15 |v_scale| + |v_zero|) from a sum in fp32 (2^-18 |v_scale| + 2^-21 |v_zero|, which shows where the two cancel),
 * centroids to f16.
 * Data errors: a context length out of range (PDA_ERRW_BAD_CONTEXT_LEN) or drafted tokens that do not fit behind it
 * (PDA_ERRW_BAD_POSITION) give zeros for the sequence's rows; block ids as for pda_decode.
 */
PDA_API long long pda_tree_workspace_size(const pda_plan_t* plan, long long num_tokens);
PDA_API int pda_decode_tree(const pda_plan_t* plan, const void* query, long long num_tokens, const void* kv_cache,
                            long long num_cache_blocks, const float* centroids, const int* block_table,
                            const int* context_lens, const int* token_starts, const unsigned long long* tree_masks,
                            int mask_words, int window, int num_first, void* workspace, long long workspace_bytes, void* out,
                            int out_dtype, int* err_word, void* stream);

/*
 * pda_accept_tokens -- keeps the accepted drafted tokens: token path[b][k] of sequence b moves to position context_lens[b] + k,
 * for k < path_lens[b] (whole tokens, any kv_dtype), and out_lens[b] = context_lens[b] + path_lens[b].  What lies behind is
 * free to be overwritten.
 *   path       device, int32 [num_seqs][max_path]: ascending indices of drafted tokens (an ancestor before its descendants)
 *   path_lens  device, int32 [num_seqs], each in [0, max_path]
 *   out_lens   device, int32 [num_seqs]; must overlap none of context_lens, path, path_lens and block_table
 * The call works within the pool it is given; the pools of a model's other layers need the same call each.  Sequences must not
 * share the blocks that hold drafted tokens.
 * Data errors: a context length out of range (PDA_ERRW_BAD_CONTEXT_LEN), a path that does not ascend or is too long
 * (PDA_ERRW_BAD_TOKENS) or leaves the table (PDA_ERRW_BAD_POSITION): nothing of the sequence moves and its length stays.  A
 * token whose block id, or its place's, is outside the pool does not move (PDA_ERRW_BAD_BLOCK_ID).
 */
PDA_API int pda_accept_tokens(const pda_plan_t* plan, void* kv_cache, long long num_cache_blocks, const int* block_table,
                              const int* context_lens, const int* path, const int* path_lens, int max_path, int* out_lens,
                              int* err_word, void* stream);

/* ---------------------------------------------------------------- sliding window
 * pda_decode_window -- a decode step in which the query of sequence b, at position context_lens[b] - 1, sees the tokens t with
 * context_lens[b] - 1 - t < window and those with t < num_first.  The others are not read, and block ids of blocks that hold
 * none of the seen ones are not looked at.  One launch, no partials.
 *   plan        as for pda_decode; any kv_dtype; kernel_variant automatic (else PDA_ERR_UNSUPPORTED)
 *   centroids   device, fp32 [16] for a TQ4 plan, else NULL
 *   window      >= 1;  num_first >= 0
 *   query, block_table, context_lens, out, out_dtype and the data errors as for pda_decode and pda_reduce
 */
PDA_API int pda_decode_window(const pda_plan_t* plan, const void* query, const void* kv_cache, long long num_cache_blocks,
                              const float* centroids, const int* block_table, const int* context_lens, int window,
                              int num_first, void* out, int out_dtype, int* err_word, void* stream);

/* Human-readable name of a pda_status value (static string; never NULL). */
PDA_API const char* pda_status_string(int status);

/* plan->workspace_bytes after pda_plan (-1 for a NULL or unplanned plan). */
PDA_API long long pda_workspace_size(const pda_plan_t* plan);

/* sizeof(pda_plan_t), for bindings that mirror the structure. */
PDA_API int pda_plan_struct_size(void);

#ifdef __cplusplus
}
#endif
#endif /* PDA_H */
