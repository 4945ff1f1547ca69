/*
 * kvq.h -- C ABI of the quantized K/V cache library (one GB300, sm_103a).
 *
 * The library keeps a transformer's K/V cache in a paged pool, as FP16, as
 * int8 codes with one FP16 scale per 64 head dims, or as K8V4 (int8 K and
 * rotated 4-bit V), and runs the calls that touch it on the decode / verify
 * / prompt paths:
 *
 *   kvq_append       quantize-on-write of new K/V rows into the pool
 *   kvq_decode_attn  GQA attention of 1..W query tokens against the pool,
 *                    as split-K partials merged by a log-sum-exp combine
 *   kvq_compact_f16  the pool copied out to contiguous FP16 staging
 *   kvq_chunk_attn   attention of a prompt chunk over that staging
 *   kvq_gather_cells / kvq_scatter_cells
 *                    a sequence's codes and scales out of / into the pool
 *   kvq_stream_plan / kvq_stream_fetch
 *                    a resident window of device blocks over a host copy
 *   kvq_plan_step    block tables and slot maps of a step from the requests'
 *                    lengths, on the device
 *   kvq_bound_blocks bounds of each block's keys
 *   kvq_select_blocks
 *                    the blocks each query token and KV head attends to,
 *                    ranked by those bounds
 *   kvq_sparse_decode_attn
 *                    decode attention over such lists of blocks
 *   kvq_append_rotary
 *                    norms of each head's q and k, rotary positions, and the
 *                    append of k and v, in one pass
 *   kvq_decode_attn_scored / kvq_chunk_attn_scored
 *                    attention whose scores are capped by a tanh, biased by
 *                    the distance, or kept to a window, document or prefix
 *   kvq_verify_draft drafted tokens accepted or replaced by the target's
 *                    probabilities, from given random numbers
 *   kvq_trim_step    the cells of rejected drafts taken back
 *
 * Sources (page title, section):
 *   [kv-q8 PR]  "#3084 qwen35: FP16 K/V cache by default, int8 with --kv-q8
 *               (262144 fits a 16 GiB card)": "Summary" (the two formats,
 *               one FP16 scale per 64 dims), "What changed" (the formula
 *               scale = fp16(max|x|/127), code = clamp(rint(x/scale),
 *               -127, 127); k_attn_prep / k_attn_part / k_kv_f16 templated on
 *               the cache format; scale arrays carried beside the code
 *               arrays), "Extra Notes" (split-K decode; k_kv_f16 compacts
 *               [kvh][ctx][HD] into [kvh][P][HD] halves for the prompt).
 *   [k8v4 PR]   "#711 kv: --kv k8v4 streams with --kv-resident": "How"
 *               (a block is a list of byte runs -- codes, then scales; the
 *               decode, verify-window and prompt appends; a writer that
 *               tests one pointer and silently skips the other), "Tests"
 *               (the negative control that catches that skip), "What"
 *               (K8V4: INT8 K + rotated Q4_0 V, 816 B per cell).
 *   [Path F v3] "Path F format v3: persist per-head INT8 KV scales for
 *               INT8 + persistent KV interop": "Why", "Scope" (int8 bytes
 *               without their scales are refused, not used).
 *
 * Conventions for every call
 *   - All device arrays are owned and allocated by the caller; the library
 *     allocates nothing and keeps no state between calls beyond one-time
 *     kernel setup (each kernel configuration's shared-memory limit and
 *     occupancy, kept per device and redone when that device's context
 *     changes, so one process may drive several devices) and
 *     kvq_decode_attn_static's scratch.  Pointers marked "device" must be
 *     device (or managed) memory of the current device.
 *   - Every call is asynchronous on `stream` (a cudaStream_t; NULL = the
 *     legacy default stream).  No call reads device memory on the host or
 *     synchronizes.
 *   - Arguments are validated on the host before anything is launched; an
 *     invalid argument returns KVQ_ERR_ARG (or KVQ_ERR_UNSUPPORTED for a
 *     valid but unimplemented shape) and launches nothing.  No call aborts,
 *     exits, throws or traps on the device.  A launch failure reported by
 *     the runtime returns KVQ_ERR_CUDA.
 *   - Device-side preconditions (not checked on the host, since the values
 *     live on the device): block ids in the block table lie in
 *     [0, n_blocks) for every cell that is read or written; token positions
 *     are < max_blocks_per_seq * block_size; 0 <= ctx_lens[b] <= max_ctx (a
 *     query token with no visible cell, as when ctx_lens[b] < W, gets 0).
 *     Breaking them gives unspecified values for the cells involved but no
 *     out-of-bounds access: every kernel checks each block id it reads
 *     against [0, n_blocks) and skips (append, compaction) or reads as
 *     zeros (attention) a cell whose id is out of range; the append kernel
 *     checks tok_seq against [0, n_seq) and tok_pos against the table width;
 *     the attention kernels clamp ctx_lens[b] to [0, max_blocks_per_seq *
 *     block_size].
 */
#ifndef KVQ_H
#define KVQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Cache formats ([kv-q8 PR], "Summary"). */
typedef enum {
    KVQ_F16 = 0, /* K and V stored as IEEE fp16 (round to nearest even)      */
    KVQ_Q8 = 1,  /* int8 codes + one fp16 scale per 64 dims of a row         */
    KVQ_K8V4 = 2 /* K as KVQ_Q8; V rotated (Walsh-Hadamard), then 4-bit      */
                 /* codes + one fp16 scale per 32 rotated dims ([k8v4 PR])  */
} kvq_format;

typedef enum {
    KVQ_OK = 0,
    KVQ_ERR_ARG = 1,         /* null / misaligned pointer, bad size or shape  */
    KVQ_ERR_UNSUPPORTED = 2, /* valid request outside the implemented shapes */
    KVQ_ERR_WORKSPACE = 3,   /* workspace missing or smaller than required   */
    KVQ_ERR_CUDA = 4         /* the CUDA runtime reported a launch error     */
} kvq_status;

/* Group of head dims sharing one fp16 scale in KVQ_Q8 (and K8V4's K). */
#define KVQ_GROUP 64
/* Block of rotated V dims sharing one fp16 scale in KVQ_K8V4. */
#define KVQ_Q4_BLOCK 32

/*
 * One layer's paged K/V pool.  A physical block holds block_size consecutive
 * cells of one sequence for all n_kv_heads KV heads; K and V, codes and
 * scales are four separate arrays ("byte runs", [k8v4 PR] "How"):
 *
 *   k_data, v_data     [n_blocks][n_kv_heads][block_size][head_dim]
 *                      fp16 (KVQ_F16) or int8 (KVQ_Q8)
 *   k_scales, v_scales [n_blocks][n_kv_heads][block_size][head_dim / 64]
 *                      fp16 bits; KVQ_Q8 only (must be NULL-free for Q8,
 *                      ignored for F16)
 *
 * KVQ_K8V4 keeps K as KVQ_Q8 does (k_data int8, k_scales per 64 dims) and V
 * as two other runs:
 *
 *   v_data             [n_blocks][n_kv_heads][block_size][head_dim / 2]
 *                      bytes: two 4-bit codes each, dim 2j in the low
 *                      nibble of byte j, dim 2j + 1 in the high nibble
 *   v_scales           [n_blocks][n_kv_heads][block_size][head_dim / 32]
 *                      fp16 bits, one per 32 dims
 *
 * where the dims are those of the rotated row y = H v (H the Walsh-Hadamard
 * matrix of order head_dim, Sylvester order, entries +-1), so a cell costs
 * 2 * n_kv_heads * (head_dim + head_dim / 32) + n_kv_heads * head_dim * 18 /
 * 32 bytes: 816 at 2 KV heads of 256 dims ([k8v4 PR], "What").
 *
 * Cell p of sequence b is block block_table[b * max_blocks_per_seq +
 * p / block_size], slot p % block_size; its row of KV head h starts at
 * element ((block * n_kv_heads + h) * block_size + slot) * head_dim.
 *
 * Limits: head_dim in {64, 128, 256}; block_size a power of two in
 * [16, 1024]; all four pointers 256-byte aligned (torch allocations are);
 * n_blocks * n_kv_heads * block_size < 2^31.
 */
typedef struct kvq_cache {
    int32_t fmt;        /* kvq_format */
    int32_t n_kv_heads;
    int32_t head_dim;
    int32_t block_size;
    int32_t n_blocks;
    int32_t reserved;   /* must be 0 */
    void *k_data;
    void *v_data;
    void *k_scales;
    void *v_scales;
} kvq_cache;

/*
 * Bytes one physical block occupies in the pool: K and V codes plus, for
 * KVQ_Q8, their scales (2 bytes per 64 dims).  Per element that is 2 bytes
 * (F16) or 1 + 2/64 bytes (Q8) -- the 6.0 GiB and 3.1 GiB of a 262144-cell
 * cache in [kv-q8 PR], "Summary".  KVQ_K8V4: 1 + 2/64 bytes per K element
 * and 18/32 per V element.  Returns 0 for an invalid geometry.
 */
size_t kvq_block_bytes(int fmt, int n_kv_heads, int head_dim, int block_size);

/*
 * Quantize-on-write of n_tok new cells ([kv-q8 PR], "What changed";
 * [k8v4 PR], "How": one call serves the decode step (n_tok = number of
 * sequences), a verify window and a prompt chunk).
 *
 *   k, v        device fp32 [n_tok][n_kv_heads][head_dim], 16-byte aligned
 *   tok_seq     device int32 [n_tok]: sequence of each new cell
 *   tok_pos     device int32 [n_tok]: its position (cell index) in that
 *               sequence
 *   block_table device int32 [n_seq][max_blocks_per_seq]
 *   n_seq       host int: rows of block_table (bounds tok_seq)
 *
 * KVQ_F16 stores fp16_rne(x).  KVQ_Q8 stores, per row and per group of 64
 * dims, s = fp16_rne(max|x| / 127) and codes clamp(rint(x / float(s)), -127,
 * 127): both divisions are IEEE fp32 divisions, rint rounds half to even; a
 * group whose scale is 0 gets zero codes.  The result is bit-identical to
 * that definition.  KVQ_K8V4 writes K that way; V is first rotated, y = H v,
 * in fp32 by butterflies (stages h = 1, 2, ..., head_dim / 2; in each, dims
 * j and j + h, bit h of j clear, become their sum and difference), then
 * each block of 32 dims of y gets d = fp16_rne(m / -8), m the block's
 * element of largest magnitude (the first one on ties), and codes
 * clamp(rint(y / float(d)), -8, 7) + 8 (8 when d is 0), both divisions
 * IEEE fp32.  A cell written twice holds the last write; two tokens of
 * one call must not name the same cell.  n_tok == 0 is a no-op returning
 * KVQ_OK.
 */
kvq_status kvq_append(const kvq_cache *cache, const float *k, const float *v, int n_tok,
                      const int32_t *tok_seq, const int32_t *tok_pos,
                      const int32_t *block_table, int n_seq, int max_blocks_per_seq,
                      void *stream);

/*
 * Workspace bytes kvq_decode_attn needs for these sizes on the current
 * device (the split plan depends on its SM count).  Returns 0 for invalid
 * arguments.
 */
size_t kvq_decode_workspace_bytes(const kvq_cache *cache, int n_seq, int W, int n_q,
                                  int max_ctx);

/*
 * Decode attention of W query tokens per sequence against the cache
 * ([kv-q8 PR], "What changed" and "Extra Notes": the split-K partial kernel
 * k_attn_part and its combine).
 *
 *   q           device fp32 [n_seq][W][n_q][head_dim], 16-byte aligned
 *   ctx_lens    device int32 [n_seq]: cells in each sequence, the W query
 *               tokens' own cells included (they are appended first)
 *   max_ctx     host int: an upper bound of ctx_lens, used to plan splits
 *   block_table device int32 [n_seq][max_blocks_per_seq]
 *   sm_scale    softmax scale (usually 1/sqrt(head_dim))
 *   out         device fp32 [n_seq][W][n_q][head_dim], 16-byte aligned
 *   workspace   device scratch of at least kvq_decode_workspace_bytes(),
 *               256-byte aligned; no initial contents are needed.  It
 *               holds the split-K partials between the partial kernel and
 *               the combine kernel of one call, so calls sharing a
 *               workspace must be ordered (same stream, or events).
 *
 * Query head h reads KV head h / (n_q / n_kv_heads); n_q must be a
 * multiple of n_kv_heads.  Query token w of sequence b is the cell
 * ctx_lens[b] - W + w and attends to cells [0, ctx_lens[b] - W + w]
 * (causal inside the window).  out = softmax(sm_scale * q . K^T) V over the
 * dequantized cache, computed in fp32; a query with no visible cell gets 0.
 * For KVQ_K8V4 the dequantized V is the rotated one, (code - 8) * d, and
 * the result is rotated back, out = H o / head_dim.
 * W in [1, 16], n_q / n_kv_heads * W <= 32.
 */
kvq_status kvq_decode_attn(const kvq_cache *cache, const float *q, int n_seq, int W, int n_q,
                           const int32_t *ctx_lens, int max_ctx, const int32_t *block_table,
                           int max_blocks_per_seq, float sm_scale, float *out,
                           void *workspace, size_t workspace_bytes, void *stream);

/*
 * kvq_decode_attn with the failure path of its copy waits exercised, for
 * tests of that path only.  Every wait of the tensor-core decode for a
 * copy into shared memory is bounded; a wait that runs out marks the
 * split's partial as lost, the combine writes NaN for the affected output
 * rows, and the kernel still waits (bounded) for its own copies before it
 * exits, so the context stays usable.  This call adds extra_tx_bytes
 * (a multiple of 16 in [16, 4096]) to the byte count every copy stage
 * expects, bytes no copy ever delivers, and bounds each wait by
 * wait_limit polls (1 .. 2^25; kvq_decode_attn uses 2^25): every wait runs
 * out, and a correct failure path returns KVQ_OK with NaN in every output
 * row of a sequence with cells.  No fault, trap or unbounded wait is
 * involved.  Other arguments, checks and errors as kvq_decode_attn; shapes
 * that the tensor-core kernel does not serve return KVQ_ERR_UNSUPPORTED.
 */
kvq_status kvq_decode_attn_lost_wait_test(const kvq_cache *cache, const float *q, int n_seq,
                                          int W, int n_q, const int32_t *ctx_lens, int max_ctx,
                                          const int32_t *block_table, int max_blocks_per_seq,
                                          float sm_scale, float *out, void *workspace,
                                          size_t workspace_bytes, uint32_t wait_limit,
                                          uint32_t extra_tx_bytes, void *stream);

/*
 * FP16 compaction of cells [0, n_cells) of one sequence ([kv-q8 PR],
 * "Extra Notes": k_kv_f16 compacts [kvh][ctx][HD] into [kvh][P][HD]
 * halves; on the FP16 cache it is a pure copy).
 *
 *   block_table_row device int32 [ceil(n_cells / block_size)]: the
 *                   sequence's row of the block table
 *   out_k, out_v    device fp16 [n_kv_heads][n_cells][head_dim], 16-byte
 *                   aligned
 *
 * KVQ_F16 copies the stored bits; KVQ_Q8 writes fp16_rne(code * scale)
 * (the product is exact in fp32).  KVQ_K8V4 writes K that way and V as
 * fp16_rne(w / head_dim), w the fp32 butterflies of kvq_append applied to
 * the row of (code - 8) * d (the inverse rotation).  n_cells == 0 is a
 * no-op.
 */
kvq_status kvq_compact_f16(const kvq_cache *cache, const int32_t *block_table_row, int n_cells,
                           void *out_k, void *out_v, void *stream);

/*
 * Attention of a prompt chunk over the FP16 staging ([kv-q8 PR], "Extra
 * Notes": the prompt chunk's Q K^T and P V products read the contiguous
 * [kvh][P][HD] fp16 halves that k_kv_f16 writes).
 *
 *   k16, v16   device fp16 [n_kv_heads][P][head_dim], 16-byte aligned: the
 *              sequence's P cells as kvq_compact_f16 writes them
 *   q          device fp32 [T][n_q][head_dim], 16-byte aligned: the chunk's
 *              T query tokens, which are the sequence's last T cells
 *   out        device fp32 [T][n_q][head_dim], 16-byte aligned
 *
 * Token t attends to cells [0, P - T + t] (causal); query head h reads KV
 * head h / (n_q / n_kv_heads).  out = softmax(sm_scale * q . K^T) V with
 * fp32 accumulation (q enters the tensor cores as an fp16 hi + lo pair, the
 * softmax weights as one fp16 value).  head_dim in {64, 128, 256}; 1 <= T <= P;
 * n_q a multiple of n_kv_heads; n_kv_heads * P < 2^31.  Invalid arguments
 * return KVQ_ERR_ARG / KVQ_ERR_UNSUPPORTED before any launch.  Asynchronous
 * on `stream`; the library allocates nothing.
 */
kvq_status kvq_chunk_attn(const void *k16, const void *v16, int n_kv_heads, int P, int head_dim,
                          const float *q, int T, int n_q, float sm_scale, float *out,
                          void *stream);

/*
 * kvq_chunk_attn with the failure path of its waits exercised, for tests of
 * that path only.  Every mbarrier wait of the chunk kernel is bounded; a
 * wait that runs out turns the CTA's rows into NaN (through the merge too,
 * when a short chunk's key tiles are split over a cluster of CTAs), and
 * each role still waits (bounded) for its own copies and MMAs before the
 * CTA exits, so the context stays usable.  This call adds extra_tx_bytes
 * (a multiple of 16 in [16, 4096]) to the byte count every K and V stage
 * expects, bytes no copy ever delivers, and bounds each wait by wait_limit
 * polls (1 .. 2^25; kvq_chunk_attn uses 2^25): every wait runs out, and a
 * correct failure path returns KVQ_OK with NaN in every output row.  No
 * fault, trap or unbounded wait is involved.  Other arguments, checks and
 * errors as kvq_chunk_attn.
 */
kvq_status kvq_chunk_attn_lost_wait_test(const void *k16, const void *v16, int n_kv_heads, int P,
                                         int head_dim, const float *q, int T, int n_q,
                                         float sm_scale, float *out, uint32_t wait_limit,
                                         uint32_t extra_tx_bytes, void *stream);

/*
 * Persistence of one sequence: cells [0, n_cells) gathered out of the pool
 * into token-major runs, and scattered back into a pool (Path F format v3:
 * persist per-head INT8 KV scales for INT8 + persistent KV interop,
 * "Scope": a saved turn is its used cells' K/V bytes followed by their
 * scales; "Why": int8 bytes without the scales would hydrate to garbage).
 *
 *   block_table_row  device int32 [ceil(n_cells / block_size)]: the
 *                    sequence's row of the block table
 *   codes_k, codes_v device [n_cells][n_kv_heads][head_dim] elements of the
 *                    pool's format (fp16 or int8), 16-byte aligned; K8V4's
 *                    codes_v is [n_cells][n_kv_heads][head_dim / 2] bytes
 *   scales_k, scales_v
 *                    device fp16 [n_cells][n_kv_heads][head_dim / 64], 16-byte
 *                    aligned; required
 *                    for KVQ_Q8 (KVQ_ERR_ARG without them), ignored for
 *                    KVQ_F16; K8V4 requires both, scales_v being
 *                    [n_cells][n_kv_heads][head_dim / 32]
 *
 * Both copy bits unchanged: a gather followed by a scatter into any pool
 * of the same format and geometry, under any block table, restores the
 * cells exactly.  Cells whose block id is out of range are skipped.
 * n_cells == 0 is a no-op.  Asynchronous on `stream`.
 */
kvq_status kvq_gather_cells(const kvq_cache *cache, const int32_t *block_table_row, int n_cells,
                            void *codes_k, void *codes_v, void *scales_k, void *scales_v,
                            void *stream);
kvq_status kvq_scatter_cells(const kvq_cache *cache, const int32_t *block_table_row, int n_cells,
                             const void *codes_k, const void *codes_v, const void *scales_k,
                             const void *scales_v, void *stream);

/*
 * Block streaming with a resident window ([k8v4 PR], "What" and "How": the
 * cache's authoritative copy lives in pinned host memory and a window of
 * N cells' worth of device blocks holds what the GPU reads; a block moves
 * as its list of byte runs, so every format streams the same way; "Tests":
 * attention over the streamed state is bitwise equal to attention over a
 * fully resident pool).
 *
 * The host copy is a kvq_cache whose four arrays are pinned host memory
 * the device can address (cudaHostAlloc'd or registered, mapped; on a
 * Grace-Blackwell node the kernels reach it over NVLink-C2C), n_blocks of
 * them; the window is an ordinary device kvq_cache of n_slots blocks with
 * the same format and geometry.  Appends go to both (the host copy under
 * the sequences' block table, the window under the slot table, where
 * non-resident blocks are -1 and therefore skipped); attention and
 * compaction read the window under the slot table.  One step:
 *
 *   kvq_append(host copy, block_table)        authoritative write
 *   kvq_stream_plan(..., block_table, ctx)    slots, fetch list (host)
 *   kvq_stream_fetch(host copy, window, list) missing blocks -> slots
 *   kvq_append(window, slot_table)            resident blocks' new cells
 *   kvq_decode_attn(window, slot_table)
 */

/*
 * Residency plan for one call, host only (no device access, nothing
 * launched).  The residency state is three caller-owned host arrays and a
 * counter, initialised by the caller to -1 / -1 / 0 / 0:
 *
 *   slot_of_block [n_host_blocks]  int32: window slot of a host block, -1
 *   block_of_slot [n_slots]        int32: host block in a slot, -1 if free
 *   last_use      [n_slots]        int64: the counter value of the slot's
 *                                  last plan
 *   clock                          int64: advanced by one per plan
 *
 * Inputs (host int32): block_table [n_seq][max_blocks_per_seq] of host
 * block ids, ctx_lens [n_seq] (cells each sequence's call reads, its new
 * cells included), block_size.  The call reads blocks [0, ceil(ctx_lens[b]
 * / block_size)) of each row; ids outside [0, n_host_blocks) are ignored.
 * Every distinct block read gets a slot: a resident one keeps its slot (a
 * hit); the others take, in order of first use, free slots in index
 * order, then the slots this call does not read, least recently used first
 * (ties: lower index).  Outputs (host): slot_table [n_seq][max_blocks_per_seq]
 * (the slot of each entry's block, -1 where it is not resident),
 * fetch_src / fetch_dst [capacity n_slots] the (host block, slot) pairs
 * to fetch, *n_fetch their count, *n_hits (may be NULL) the hits.  A call
 * that reads more distinct blocks than n_slots returns KVQ_ERR_UNSUPPORTED
 * and changes nothing; invalid sizes or NULL arrays return KVQ_ERR_ARG.
 * The function uses temporary host memory and keeps no state of its own.
 */
kvq_status kvq_stream_plan(int n_host_blocks, int n_slots, int32_t *slot_of_block,
                           int32_t *block_of_slot, int64_t *last_use, int64_t *clock,
                           const int32_t *block_table, int n_seq, int max_blocks_per_seq,
                           const int32_t *ctx_lens, int block_size, int32_t *slot_table,
                           int32_t *fetch_src, int32_t *fetch_dst, int *n_fetch, int *n_hits);

/*
 * Copy n_fetch blocks from the host copy into window slots: block
 * fetch_src[i] of every run of host_copy goes to block fetch_dst[i] of the
 * same run of window, bits unchanged (two runs for KVQ_F16, four
 * otherwise).  One kernel reads the host memory directly (16-byte loads,
 * several in flight per thread) and writes the window; no copy engine is
 * involved.  fetch_src / fetch_dst: int32 [n_fetch] that the device can
 * read (device memory or mapped pinned host memory, e.g. the plan's
 * outputs in pinned memory).  Both caches must pass the kvq_append checks
 * and agree in format, n_kv_heads, head_dim and block_size (else
 * KVQ_ERR_ARG); every array of the host copy must be device-addressable
 * at its own address (the runtime's pointer attributes give it that device
 * address: pinned memory under unified addressing, device or managed
 * memory), so that kvq_append can write it too, else KVQ_ERR_ARG -- checked
 * even when n_fetch is 0, so a call with n_fetch 0 validates a host copy
 * before anything writes to it.  Ids out of range skip their fetch.  Two
 * fetches must not name the same slot.  Asynchronous on `stream`.
 */
kvq_status kvq_stream_fetch(const kvq_cache *host_copy, const kvq_cache *window,
                            const int32_t *fetch_src, const int32_t *fetch_dst, int n_fetch,
                            void *stream);

/*
 * Bytes of device scratch that kvq_decode_attn_static keeps in the library
 * (one array per device that loads the library, held until the process
 * exits).
 */
#define KVQ_STATIC_SCRATCH_BYTES (8u << 20)

/*
 * kvq_decode_attn without a workspace argument, for callers that cannot
 * allocate device memory: code running during CUDA graph capture (where
 * cudaMalloc is not allowed), plugins inside a framework whose allocator
 * owns the device memory, real-time loops whose memory is fixed at
 * start-up.  The paper has no counterpart to this call; it exists for
 * such callers only.
 *
 * Arguments, results and errors are those of kvq_decode_attn.  The scratch
 * is a file-scope device array of KVQ_STATIC_SCRATCH_BYTES inside the
 * library; when the split plan kvq_decode_workspace_bytes describes needs
 * more, the context is cut into fewer splits until it fits, and a request
 * that does not fit even with one split per (sequence, KV head) returns
 * KVQ_ERR_WORKSPACE and launches nothing.  The first call on a device
 * looks up the array's address and caches it for that device's context
 * (looked up again after the context changes, e.g. after cudaDeviceReset):
 * make that first call before any stream capture.
 * Every call uses the same array, so calls whose kernels may overlap on
 * the GPU (unordered streams) race on it; order them.  The array needs no
 * clearing between calls.
 */
kvq_status kvq_decode_attn_static(const kvq_cache *cache, const float *q, int n_seq, int W,
                                  int n_q, const int32_t *ctx_lens, int max_ctx,
                                  const int32_t *block_table, int max_blocks_per_seq,
                                  float sm_scale, float *out, void *stream);

/*
 * One serving step's block tables and slot maps, built on the device from
 * the requests' lengths: what kvq_append (tok_seq, tok_pos, the table) and
 * the attention calls (the lengths) take, without a copy to the host.
 *
 *   ctx_in        device int32 [n_seq]: cells each sequence holds
 *   n_new         device int32 [n_seq]: tokens it gets this step (0: none);
 *                 negative: the sequence ends and gives its blocks back
 *   block_table   device int32 [n_seq][max_blocks_per_seq], updated in
 *                 place: new entries follow the old ones (a released row
 *                 keeps its entries, which its length of 0 leaves unread)
 *   free_list     device int32 [n_blocks], updated in place: a stack of
 *                 free block ids, its top at index *free_count_in - 1
 *   free_count_in device int32 [1]
 *   max_tok       host int: capacity of the token arrays
 *   ctx_out       device int32 [n_seq]: ctx_in + n_new, 0 for a released one
 *   tok_start     device int32 [n_seq + 1]: each sequence's first token
 *   tok_seq, tok_pos, slots
 *                 device int32 [max_tok], 16-byte aligned: each token's
 *                 sequence, its position, and its cell in the pool (block *
 *                 block_size + offset; slots may be NULL), the sequences in
 *                 order; -1 past the last token, which kvq_append skips, so a
 *                 captured graph can append all max_tok rows
 *   free_count_out device int32 [1]
 *   info          device int32 [4], 16-byte aligned: tokens, blocks handed
 *                 out, blocks given back, status
 *
 * Blocks given back are pushed in (sequence, column) order, then the new
 * ones are popped in (sequence, column) order, so a step may hand out what
 * it got back.  A step that cannot be placed leaves lengths, tables, list
 * and count as they were, places no token (tok_start 0, the token arrays
 * -1, info 0, 0, 0, status) and says why in status, a sum of:
 */
#define KVQ_PLAN_TOKENS 1 /* more than max_tok tokens                        */
#define KVQ_PLAN_ROW 2    /* a sequence longer than its row, or ctx_in < 0   */
#define KVQ_PLAN_BLOCKS 4 /* not enough free blocks                          */
#define KVQ_PLAN_LIST 8   /* free_count_in outside [0, n_blocks], or more    */
                          /* blocks given back than the list holds           */
/*
 * Output arrays must not overlap one another or an input (KVQ_ERR_ARG): a
 * step reads one set of lengths and count and writes another.  n_seq <=
 * 16384 and max_tok <= 2^30, else KVQ_ERR_UNSUPPORTED; n_blocks * block_size
 * and max_blocks_per_seq * block_size < 2^31; block_size as in kvq_cache.
 * Table and list entries read must be block ids the caller owns; they are
 * copied, not followed.  One launch, no workspace.
 */
kvq_status kvq_plan_step(const int32_t *ctx_in, const int32_t *n_new, int n_seq, int block_size,
                         int n_blocks, int32_t *block_table, int max_blocks_per_seq,
                         int32_t *free_list, const int32_t *free_count_in, int max_tok,
                         int32_t *ctx_out, int32_t *tok_start, int32_t *tok_seq, int32_t *tok_pos,
                         int32_t *slots, int32_t *free_count_out, int32_t *info, void *stream);

/*
 * Bounds of the keys of every block that cells [ctx_start[b], ctx_lens[b])
 * touch (after the append that wrote them): per KV head and dim the smallest
 * and largest dequantised K over the block's cells below ctx_lens[b], as
 * int8 codes rounded outwards.
 *
 *   ctx_start    device int32 [n_seq]: first cell that changed (NULL: 0,
 *                all blocks)
 *   ctx_lens     device int32 [n_seq]
 *   max_new      host int: an upper bound of ctx_lens - ctx_start, at most
 *                what a row holds (max_blocks_per_seq * block_size, else
 *                KVQ_ERR_ARG); blocks beyond what it covers keep their old
 *                bounds
 *   bounds       device int8 [n_blocks][n_kv_heads][2][head_dim], 256-byte
 *                aligned: lo codes, then hi codes
 *   bound_scales device fp32 [n_blocks][n_kv_heads][head_dim / 64]
 *
 * Per 64 dims the scale is 2^e, e in [-24, 16] the smallest with 127 * 2^e
 * >= max(|lo|, |hi|); the codes are floor(lo / 2^e) and ceil(hi / 2^e).  The
 * result is bit-identical to that definition for finite keys; NaN keys and
 * int8 keys whose scale is not finite are passed over (a dim with nothing
 * else gets 0), infinite FP16 keys give codes of +-127 at e = 16.  Bounds
 * belong to the physical block: a block that several rows share needs one of
 * them bounded, and a block that is refilled needs a new call.  (Rows of one
 * call that end at different cells of a block they share leave the bounds of
 * either.)
 * Sequences with ctx_start >= ctx_lens and blocks with an id out of range
 * are skipped.  max_new == 0 is a no-op.
 */
kvq_status kvq_bound_blocks(const kvq_cache *cache, const int32_t *block_table, int n_seq,
                            int max_blocks_per_seq, const int32_t *ctx_start,
                            const int32_t *ctx_lens, int max_new, void *bounds,
                            float *bound_scales, void *stream);

/*
 * The blocks each query token attends to, chosen per KV head by an estimate
 * of the largest q . k over each block: the bound that kvq_bound_blocks's
 * codes give for q rounded to 8 bits.  It is not a bound for q itself: the
 * rounding moves it up or down by at most half a code step of every dim
 * times that dim's larger bound, and infinite FP16 keys have finite bounds.
 *
 *   q          device fp32 [n_seq][W][n_q][head_dim], 16-byte aligned, as
 *              kvq_decode_attn takes it (token w sees cells [0, ctx_lens[b]
 *              - W + w]); any W >= 1
 *   max_ctx    host int: an upper bound of ctx_lens, at most
 *              max_blocks_per_seq * block_size (KVQ_ERR_ARG)
 *   n_sel      blocks per list, of which the first n_first and the last
 *              n_last visible blocks are always kept (n_first + n_last <=
 *              n_sel)
 *   sel_blocks device int32 [n_seq][W][n_kv_heads][n_sel]: pool block ids, in
 *              ascending order of the blocks' place in the sequence, -1 past
 *              the list's end
 *   sel_index  the same entries as indexes into the sequence's row, or NULL
 *   sel_lens   device int32 [n_seq][W][n_kv_heads]: cells the list holds (the
 *              last visible block, if chosen, counts its visible cells)
 *
 * Only cache's geometry is read.  Score of a block: per 64 dims of a query
 * row, the scale 2^f is the smallest (f in [-60, 60]) with 127 * 2^f >=
 * max|q| and the codes are c = rint(q / 2^f), half to even (NaN: 0); S =
 * sum over the dims of max(c, 0) hi + min(c, 0) lo over the bounds' codes, a
 * whole number; t = S * 2^f * bound_scale, exact in fp32 for the scales
 * kvq_bound_blocks writes; the score is t0, t0 + t1, or (t0 + t1) + (t2 +
 * t3) in fp32, and the largest over the KV head's n_q / n_kv_heads query
 * heads counts.  The n_sel highest visible blocks are taken, ties to the
 * lower index; blocks whose id is out of range never are.  The result is
 * bit-identical to that definition.
 *
 * n_q / n_kv_heads <= 32, ceil(max_ctx / block_size) <= 32768, n_seq * W *
 * n_kv_heads <= 2^24, n_sel * block_size < 2^30, else KVQ_ERR_UNSUPPORTED.
 * One launch, no workspace.
 */
kvq_status kvq_select_blocks(const kvq_cache *cache, const void *bounds, const float *bound_scales,
                             const float *q, int n_seq, int W, int n_q, const int32_t *ctx_lens,
                             int max_ctx, const int32_t *block_table, int max_blocks_per_seq,
                             int n_sel, int n_first, int n_last, int32_t *sel_blocks,
                             int32_t *sel_index, int32_t *sel_lens, void *stream);

/*
 * kvq_decode_attn over a list of blocks for each (sequence, query token, KV
 * head), as kvq_select_blocks writes them (any lists will do).
 *
 *   q, out     device fp32 [n_seq][W][n_q][head_dim], 16-byte aligned; any
 *              W >= 1
 *   sel_blocks device int32 [n_seq][W][n_kv_heads][n_sel]: pool block ids
 *   sel_lens   device int32 [n_seq][W][n_kv_heads]: cells of each list: the
 *              first sel_lens of its blocks' cells, block by block, are
 *              attended to (clamped to [0, n_sel * block_size]; 0 gives 0)
 *   workspace  256-byte aligned, under kvq_decode_attn's rules: at least 256
 *              bytes, else KVQ_ERR_WORKSPACE.  The splits of few lists meet
 *              through kvq_sparse_workspace_bytes() of it; in a smaller one
 *              they meet in thread-block clusters (8 lists of 4096 cells 8.9
 *              -> 12.3 us in FP16, 7.9 -> 14.0 in int8; 32 lists alike).  That
 *              size is 256 once the lists fill the GPU, so a workspace
 *              sized for a batch may be smaller than what a part of the
 *              batch would use; it serves both.
 *
 * Cells of a block whose id is out of range are masked.  Precision, formats,
 * checks and errors as kvq_decode_attn; n_q / n_kv_heads <= 32, n_seq * W *
 * n_kv_heads <= 2^24 and n_sel * block_size < 2^30, else
 * KVQ_ERR_UNSUPPORTED.  kvq_sparse_workspace_bytes returns 0 for invalid
 * arguments.
 */
size_t kvq_sparse_workspace_bytes(const kvq_cache *cache, int n_seq, int W, int n_q, int n_sel);
kvq_status kvq_sparse_decode_attn(const kvq_cache *cache, const float *q, int n_seq, int W, int n_q,
                                  const int32_t *sel_blocks, const int32_t *sel_lens, int n_sel,
                                  float sm_scale, float *out, void *workspace,
                                  size_t workspace_bytes, void *stream);

/*
 * kvq_sparse_decode_attn with the failure path of its copy waits exercised,
 * for tests of that path only, as kvq_decode_attn_lost_wait_test does: every
 * wait runs out, and a correct failure path returns KVQ_OK with NaN in
 * every output row of a list with cells, whether its splits meet through
 * the workspace or in a cluster.
 */
kvq_status kvq_sparse_decode_attn_lost_wait_test(const kvq_cache *cache, const float *q, int n_seq,
                                                 int W, int n_q, const int32_t *sel_blocks,
                                                 const int32_t *sel_lens, int n_sel, float sm_scale,
                                                 float *out, void *workspace,
                                                 size_t workspace_bytes, uint32_t wait_limit,
                                                 uint32_t extra_tx_bytes, void *stream);

/* Element types of the calls below. */
typedef enum {
    KVQ_T_F32 = 0,
    KVQ_T_F16 = 1,
    KVQ_T_BF16 = 2
} kvq_type;

/*
 * How kvq_append_rotary treats each head of q and k:
 *
 *   norm      x <- x * rsqrt(mean(x^2) + eps) * w over the head's head_dim
 *             values (w = q_norm or k_norm, fp32 [head_dim]; NULL: no norm of
 *             that input.  A model that stores w - 1 passes w)
 *   rotation  of the head's first rot_dim dims, pairs i = 0 .. rot_dim / 2 - 1
 *             of dims (2i, 2i + 1) if interleaved, else (i, i + rot_dim / 2):
 *             (a, b) <- (a cos t - b sin t, b cos t + a sin t) * gain with the
 *             angle t = position * inv_freq[i], the position taken on axis
 *             pair_axis[i] (NULL: axis 0).  Dims from rot_dim on stay.
 *
 * Arrays are device memory; inv_freq, q_norm and k_norm 16-byte aligned.
 */
typedef struct kvq_rotary {
    int32_t type;        /* kvq_type of q, k and v                            */
    int32_t rot_dim;     /* a multiple of 16 in [0, head_dim]                 */
    int32_t interleaved; /* 0 or 1                                            */
    int32_t n_axes;      /* axes of `positions`, 1 .. 8                       */
    float eps;           /* >= 0                                              */
    float gain;          /* 1, or a factor on cos and sin                     */
    const float *inv_freq;    /* [rot_dim / 2], radians a position            */
    const int32_t *pair_axis; /* [rot_dim / 2] or NULL; clamped to the axes   */
    const float *q_norm;      /* [head_dim] or NULL                           */
    const float *k_norm;      /* [head_dim] or NULL                           */
} kvq_rotary;

/*
 * kvq_append of k and v as a projection leaves them: q and k of each token
 * are normed and rotated, q is written out for the attention calls, k and v
 * go into the pool in its format (kvq_append's, of the fp32 values the norm
 * and rotation give; v is only converted).
 *
 *   q, k, v    device [n_tok] rows of n_q, n_kv_heads, n_kv_heads heads, of
 *              rotary->type, 16-byte aligned; row t starts at element t *
 *              q_stride (k_stride, v_stride), so they may be parts of one
 *              [n_tok][(n_q + 2 n_kv_heads) head_dim] array.  Strides are at
 *              least a row and a multiple of 16 bytes (KVQ_ERR_ARG)
 *   n_q        query heads, any number >= 0 (0: q and q_out unread)
 *   positions  device int32 [n_axes][n_tok] or NULL: tok_pos on every axis
 *              (then n_axes is 1)
 *   tok_seq, tok_pos, block_table, n_seq, max_blocks_per_seq
 *              as kvq_append takes them
 *   q_out      device fp32 [n_tok][n_q][head_dim], 16-byte aligned, not
 *              overlapping an input
 *
 * Two tokens of one call must not name the same cell.  A token whose tok_seq
 * is outside [0, n_seq) or whose tok_pos is negative (padding) is skipped: its
 * row of q_out stays as it was, nothing is
 * appended.  Where only its block is out of range its q is written still.
 * Sums, angles and rotation are fp32 or better: an angle of up to 2^22
 * radians is reduced to within 2^-22 before its sine and cosine are taken, a
 * larger one to within the fp64 rounding of the product (negative positions
 * on an axis alike).  Nothing is rounded to 16 bits in between.
 * n_tok == 0 is a no-op.  n_tok * (n_q + 2 n_kv_heads) < 2^31, else
 * KVQ_ERR_UNSUPPORTED.  One launch, no workspace.
 */
kvq_status kvq_append_rotary(const kvq_cache *cache, const kvq_rotary *rotary, const void *q,
                             const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                             int64_t v_stride, int n_tok, int n_q, const int32_t *tok_seq,
                             const int32_t *tok_pos, const int32_t *positions,
                             const int32_t *block_table, int n_seq, int max_blocks_per_seq,
                             float *q_out, void *stream);

/*
 * Scores of the attention calls below.  Query head h at position i gives cell
 * j the score
 *
 *   s = (q . k_j) * sm_scale
 *   s = softcap * tanh(s / softcap)          if softcap > 0
 *   s = s - slopes[h] * |i - j|              if slopes
 *
 * and sees the cells j with
 *
 *   max(first, i - window + 1) <= j <= max(i, last)
 *
 * (first 0 and last i where NULL, no window where 0), below the context's
 * length.  A token that sees no cell gets 0.
 */
typedef struct kvq_scores {
    float softcap;         /* 0: none, else in [1e-3, 1e6]                     */
    int32_t window;        /* >= 0; 0: none                                    */
    const float *slopes;   /* device fp32 [n_q] or NULL                        */
    const int32_t *first;  /* device int32 or NULL: decode [n_seq], chunk [T]  */
    const int32_t *last;   /* device int32 or NULL: chunk [T]; decode: NULL    */
} kvq_scores;

/*
 * kvq_decode_attn with such scores: arguments, formats, limits, workspace
 * rules and errors as there, `first` per sequence (the first cell of a
 * request behind padding, or of its document).  Token w of the window is at
 * position ctx_lens[b] - W + w.  Only tiles that some token of the sequence
 * sees are read, and a window bounds the workspace too.
 * kvq_scored_workspace_bytes returns 0 for invalid arguments.
 *
 * Cells that no token of the sequence sees may hold anything; the values of
 * cells that some of its tokens see and others do not (the edges of a verify
 * window) must be finite.  Scores, softmax and sums are fp32, q and the
 * weights enter the tensor cores as fp16 hi + lo pairs.
 */
size_t kvq_scored_workspace_bytes(const kvq_cache *cache, const kvq_scores *scores, int n_seq, int W,
                                  int n_q, int max_ctx);
kvq_status kvq_decode_attn_scored(const kvq_cache *cache, const kvq_scores *scores, const float *q,
                                  int n_seq, int W, int n_q, const int32_t *ctx_lens, int max_ctx,
                                  const int32_t *block_table, int max_blocks_per_seq,
                                  float sm_scale, float *out, void *workspace,
                                  size_t workspace_bytes, void *stream);

/*
 * kvq_decode_attn_scored with the failure path of its copy waits exercised,
 * for tests of that path only, as kvq_decode_attn_lost_wait_test does.
 */
kvq_status kvq_decode_attn_scored_lost_wait_test(
    const kvq_cache *cache, const kvq_scores *scores, const float *q, int n_seq, int W, int n_q,
    const int32_t *ctx_lens, int max_ctx, const int32_t *block_table, int max_blocks_per_seq,
    float sm_scale, float *out, void *workspace, size_t workspace_bytes, uint32_t wait_limit,
    uint32_t extra_tx_bytes, void *stream);

/*
 * kvq_chunk_attn with such scores: token t of the chunk is at position P - T
 * + t; `first` [T] keeps it to its document, `last` [T] lets a token of a
 * bidirectional prefix see the prefix's later tokens (up to P - 1).
 *
 *   out        device [T][n_q][head_dim] of out_type (kvq_type), 16-byte
 *              aligned
 *
 * Keys no row of a 128-row tile sees are not read.  The values of the whole
 * staging must be finite.  Everything else as kvq_chunk_attn; the weights
 * enter the tensor cores as one fp16 value each.
 */
kvq_status kvq_chunk_attn_scored(const void *k16, const void *v16, int n_kv_heads, int P,
                                 int head_dim, const kvq_scores *scores, const float *q, int T,
                                 int n_q, float sm_scale, void *out, int out_type, void *stream);

/*
 * kvq_chunk_attn_scored with the failure path of its waits exercised, for
 * tests of that path only, as kvq_chunk_attn_lost_wait_test does.
 */
kvq_status kvq_chunk_attn_scored_lost_wait_test(const void *k16, const void *v16, int n_kv_heads,
                                                int P, int head_dim, const kvq_scores *scores,
                                                const float *q, int T, int n_q, float sm_scale,
                                                void *out, int out_type, uint32_t wait_limit,
                                                uint32_t extra_tx_bytes, void *stream);

/*
 * Drafted tokens against the target's probabilities, by rejection sampling
 * from given random numbers.  A verify window of W tokens (the last sampled
 * one and up to W - 1 drafts) gives W rows of target probabilities, row i
 * those of the token after window token i, which draft i proposes.
 *
 *   target       device [n_seq][W] rows of `vocab` probabilities
 *   draft        device [n_seq][W - 1] rows, what each draft was sampled
 *                from; NULL: drafts are certain (a lookup's, an argmax), each
 *                with probability 1
 *   type         kvq_type of both; aligned to it
 *   target_stride, draft_stride
 *                elements from row to row, >= vocab
 *   draft_tokens device int32 [n_seq][W - 1]
 *   n_draft      device int32 [n_seq] or NULL (W - 1): drafts of each
 *                sequence, at most W - 1 (more count as W - 1); negative: the
 *                sequence takes no part: 0 accepted, tokens -1, 0 dropped
 *                (a sequence the step gave no token, or whose plan was
 *                refused, has to take no part: its drafts are in no cell).
 *                Fewer drafts: a sequence's rows are the first of its W,
 *                where the attention calls have its tokens in the last
 *   u            device fp32 [n_seq][W - 1], u_sample device fp32 [n_seq]:
 *                uniform in [0, 1)
 *   n_accepted   device int32 [n_seq]
 *   tokens       device int32 [n_seq][W]: the accepted drafts, one sampled
 *                token, -1 behind it
 *   n_dropped    device int32 [n_seq] or NULL: drafts not accepted, whose
 *                cells kvq_trim_step takes back
 *
 * Draft x at place i is accepted if all before it were and u_i * draft_i(x) <
 * target_i(x), compared exactly; a token outside [0, vocab) never is.  Behind
 * the accepted ones (a of them) one token is sampled: from max(target_a -
 * draft_a, 0) if a draft was rejected there (certain drafts: from target_a
 * without x), from target_a if none was left, and from target_a too where
 * that difference is nowhere above 0.  Sampling is by the inverse of the
 * cumulated weights in whole numbers: a weight r (in fp32; NaN and negative
 * ones 0, above 1 one) counts floor(r * 2^40); with S their sum and U =
 * floor(u_sample * 2^24) (held in [0, 2^24 - 1]) the token is the first whose
 * cumulated count is above floor(S * U / 2^24); -1 if S is 0.  The result is
 * bit-identical to that definition.
 *
 * 1 <= W <= 32, n_seq <= 65535 * 8, vocab <= 2^20, else KVQ_ERR_UNSUPPORTED.
 * One launch, no workspace.
 */
kvq_status kvq_verify_draft(const void *target, const void *draft, int type, int64_t target_stride,
                            int64_t draft_stride, int n_seq, int W, int vocab,
                            const int32_t *draft_tokens, const int32_t *n_draft, const float *u,
                            const float *u_sample, int32_t *n_accepted, int32_t *tokens,
                            int32_t *n_dropped, void *stream);

/*
 * The last cells of sequences taken back (rejected drafts, a rollback): the
 * lengths shrink, blocks no longer needed go back to the free list, in
 * (sequence, column) order.  Table entries stay as they are, unread.
 *
 *   ctx_in        device int32 [n_seq]: cells each sequence holds
 *   n_drop        device int32 [n_seq]: cells to take back, 0 .. ctx_in
 *   block_table   device int32 [n_seq][max_blocks_per_seq], read
 *   free_list     device int32 [n_blocks], updated in place above its top
 *   free_count_in device int32 [1]
 *   ctx_out       device int32 [n_seq]: ctx_in - n_drop
 *   free_count_out device int32 [1]
 *   info          device int32 [4], 16-byte aligned: cells taken back (held at
 *                 2^31 - 1), 0, blocks given back, status
 *
 * A step with a broken argument changes nothing (ctx_out = ctx_in, info 0, 0,
 * 0, status): KVQ_PLAN_ROW for a length below 0 or beyond its row or an
 * n_drop outside [0, ctx_in], KVQ_PLAN_LIST as in kvq_plan_step.  The call
 * knows nothing of the plan before it: the tokens of a refused plan are in no
 * cell, and n_drop has to be 0 for them (kvq_verify_draft's n_dropped is, with
 * n_draft negative).  Limits, overlap rules and errors as there.  One launch, no
 * workspace.
 */
kvq_status kvq_trim_step(const int32_t *ctx_in, const int32_t *n_drop, int n_seq, int block_size,
                         int n_blocks, const int32_t *block_table, int max_blocks_per_seq,
                         int32_t *free_list, const int32_t *free_count_in, int32_t *ctx_out,
                         int32_t *free_count_out, int32_t *info, void *stream);

/* Static, human-readable name of a status code. */
const char *kvq_status_string(int status);

#ifdef __cplusplus
}
#endif
#endif /* KVQ_H */
