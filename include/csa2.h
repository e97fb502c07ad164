/*
 * csa2.h -- C ABI of the CSA2 global-attention decode path on GB300 (sm_103a).
 *
 * The path (DeepSeek-V4.1-Flash, "An infra-oriented diagram of the
 * DeepSeek-V4.1-Flash architecture", reading notes; perchy.ai card
 * "Full. Reindex. Reuse."):
 *   1. lightning-indexer score of every visible cache entry      csa2_index_score
 *   2. top-512 selection (or a 2,048-block candidate pool first)  csa2_topk
 *   3. dequantisation of the selected FP4 latents + 64-head MQA
 *      attention over them and the 128-token FP8 window          csa2_sparse_attn
 *   0. cache write: FP4 / FP8 packing (m=1 or gated m=2)          csa2_fp4_pack
 * and around it, for caches kept in pages: the plan of a step from the
 * sequences' lengths (csa2_page_plan), the norm, rotation and cache write of its
 * tokens (csa2_qk_norm_rope), reading records back (csa2_cache_read), and
 * attention over paged latents, all visible ones or a selection
 * (csa2_paged_attn); and what such a cache keeps: the attention weight that its
 * entries get (csa2_attn_weight), eviction by it (csa2_evict), the verification
 * of drafted tokens (csa2_verify_drafts), pages given back (csa2_page_trim).
 *
 * Conventions (every entry point):
 *   - Returns a csa2_status.  Nothing aborts, prints or allocates device memory.
 *   - Pointers marked (device) are caller-owned device buffers; the library
 *     never frees or retains them.  Scratch space is passed in by the caller;
 *     csa2_workspace_size() says how much.
 *   - All work is enqueued on `stream` and is asynchronous.  Host-side argument
 *     checks happen before anything is launched; on a failed check nothing is
 *     launched and CSA2_ERR_INVALID_ARG / CSA2_ERR_UNSUPPORTED is returned.
 *   - Values held in device arrays (sequence ids, lengths, selected indices,
 *     pool block ids) are checked by the kernels: an out-of-range value is
 *     skipped and records CSA2_ERR_BOUNDS in a sticky device status word, read
 *     (and cleared) with csa2_get_device_status().  No kernel traps or spins
 *     without a bound.
 *   - Errors from the CUDA runtime (launch failures) return CSA2_ERR_CUDA.
 *
 * Cache record formats (logical bytes per record are fixed by the pages; the
 * physical arrangement below is this library's choice):
 *   KV  (S1) 288 B per entry, array of records [n_seq][n_max][288]: bytes 0..255
 *            hold 512 FP4 E2M1 codes (low nibble = even channel), bytes
 *            256..287 hold 32 E4M3 scales, one per 16 channels (the study's
 *            section "The KV cache" sizes a main-cache entry at 288 bytes: 512
 *            FP4 codes and one E4M3 scale for each 16 channels).
 *   IDX (S2) 68 B per entry as two planes, so that every row is 16-B aligned:
 *            nibbles [rows][64] (128 E2M1 codes) and scales [rows][4] (E8M0, one
 *            per 32 channels) (the same section sizes an indexer key at 68
 *            bytes: 128 FP4 codes, an E8M0 scale for each 32).  The nibble plane is stored in the
 *            64-byte swizzled order of the tensor cores: the 16-byte chunk c
 *            (channels 32c .. 32c+31) of a row at byte address A is stored at
 *            chunk c ^ ((A >> 7) & 3) of that row; with a 512-B aligned plane
 *            that is c ^ ((row >> 1) & 3).  csa2_fp4_pack writes this order, so
 *            any 8-row-aligned range can be packed independently.  The indexer
 *            query heads (S4) use the same format with rows = n_q * 32.
 *   SWA (S3) 528 B per entry [n_seq][swa_cap][528]: 512 E4M3 values then 16
 *            E8M0 scales, one per 32 channels (a reading of the same section,
 *            which gives the window as 128 FP8 entries of 528 bytes).
 *
 * Rounding (shared by every packer): round to nearest, ties to even, saturating
 * at the format's largest finite value; the sign of x is kept when the magnitude
 * rounds to zero.  E4M3 latent scale = E4M3(amax/6); a group whose scale is zero
 * stores zero codes.  E8M0 scale = the smallest power of two >= amax/6 (FP4) or
 * >= amax/448 (FP8), exponent clamped to [-127, 127]; amax = 0 stores byte 0 and
 * zero codes.
 */
#ifndef CSA2_H
#define CSA2_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *csa2_stream_t;   /* == cudaStream_t; NULL = legacy default stream */

typedef enum {
  CSA2_OK = 0,
  CSA2_ERR_INVALID_ARG = 1,   /* a null pointer, a negative or misaligned size, an unknown kind */
  CSA2_ERR_UNSUPPORTED = 2,   /* parameters other than the pages' constants, k above the limit */
  CSA2_ERR_CUDA = 3,          /* the CUDA runtime reported an error                           */
  CSA2_ERR_BOUNDS = 4,        /* (device) an index or length in a device array was out of range */
  CSA2_ERR_TIMEOUT = 5,       /* (device) a bounded wait ran out                               */
  CSA2_ERR_WORKSPACE = 6      /* the workspace passed in is smaller than required             */
} csa2_status;

/* Record kinds for csa2_entry_bytes / csa2_fp4_pack. */
enum { CSA2_KV_NVFP4 = 0, CSA2_IDX_MXFP4 = 1, CSA2_SWA_MXFP8 = 2 };
/* Output dtypes for csa2_sparse_attn. */
enum { CSA2_OUT_BF16 = 0, CSA2_OUT_F32 = 1 };
/* Operations for csa2_workspace_size. */
enum { CSA2_OP_TOPK = 0, CSA2_OP_SPARSE_ATTN = 1, CSA2_OP_DECODE = 2, CSA2_OP_DECODE_HOST = 3, CSA2_OP_DECODE_MQ = 4,
       CSA2_OP_BUILD_CACHE = 5, CSA2_OP_DECODE_REINDEX = 6, CSA2_OP_PAGED_ATTN = 7, CSA2_OP_ATTN_WEIGHT = 8,
       CSA2_OP_EVICT = 9, CSA2_OP_VERIFY = 10 };
/* Modes and types of csa2_verify_drafts. */
enum { CSA2_VERIFY_SAMPLE = 0, CSA2_VERIFY_GREEDY = 1 };
enum { CSA2_PROB_BF16 = 0, CSA2_PROB_F32 = 1, CSA2_PROB_F16 = 2 };

/* Model constants.  The kernels are built for the pages' values only
 * (study, reading notes: 64 heads, 512-wide latent, RoPE on 64 of the 512
 * dims; lightning indexer 32 x 128, top-512; pool of 2,048 blocks of 8;
 * helix.ml: 128-token window).  rope_base and sm_scale are free. */
typedef struct {
  int heads;        /* 64                      */
  int dim;          /* 512                     */
  int rope_dim;     /* 64                      */
  int rope_off;     /* 448 (dims 448..511)     */
  double rope_base; /* 10000                   */
  float sm_scale;   /* 1/sqrt(512)             */
  int idx_heads;    /* 32                      */
  int idx_dim;      /* 128                     */
  int topk;         /* 512                     */
  int swa;          /* 128                     */
  int block;        /* 8                       */
  int pool_blocks;  /* 2048                    */
} csa2_params;

/* Fills *p with the pages' constants.  Never fails for a non-null p. */
csa2_status csa2_default_params(csa2_params *p);

/* Bytes per logical record: KV 288, IDX 68, SWA 528; 0 for an unknown kind. */
size_t csa2_entry_bytes(int kind);

/* Human-readable name of a status code (static string). */
const char *csa2_status_string(csa2_status s);

/*
 * csa2_fp4_pack -- cache write: quantise bf16 rows into cache records.
 * (An infra-oriented diagram of the DeepSeek-V4.1-Flash architecture, reading
 * notes and section "The KV cache": the encoder pools each pair of tokens into
 * one entry through a learned softmax gate, and the latent cache holds E2M1
 * values with an E4M3 scale for every 16 channels.)
 *
 *   kind         CSA2_KV_NVFP4 (src rows of 512), CSA2_IDX_MXFP4 (rows of 128),
 *                CSA2_SWA_MXFP8 (rows of 512).
 *   src          (device) bf16 [rows][width], row-major, 16-B aligned.
 *   rows         number of source rows (tokens); >= 0.  0 launches nothing.
 *   m            1, or 2 (KV only): rows must be even; output row r pools
 *                source rows 2r and 2r+1 per channel with weights
 *                softmax(gate_logits[2r][c], gate_logits[2r+1][c]), computed
 *                in fp64 and rounded to bf16 before packing.
 *   gate_logits  (device) fp32 [rows][512] when m == 2, else must be NULL.
 *   dst          (device) KV/SWA: rows/m records of 288/528 B; IDX: the nibble
 *                plane [rows][64].  16-B aligned.
 *   dst_scales   (device) IDX only: the scale plane [rows][4]; NULL otherwise.
 */
csa2_status csa2_fp4_pack(int kind, const void *src, int64_t rows, int m, const float *gate_logits,
                          void *dst, void *dst_scales, csa2_stream_t stream);

/*
 * csa2_index_score -- lightning-indexer scores.
 * (An infra-oriented diagram of the DeepSeek-V4.1-Flash architecture, reading
 * notes: the indexer compares 32 FP4 query heads of width 128 with the single
 * key of each entry, clamps each head's dot product at zero and adds them up
 * with one weight per head):
 *     s_j = sum_{h<32} w_h * max(0, qhat_h . khat_j)
 * with qhat, khat the dequantised FP4 values (E2M1 x E8M0), fp32 accumulation.
 *
 *   key_nib, key_scale  (device) IDX cache planes of n_seq * n_max entries;
 *                       entry j of sequence b is row b*n_max + j.  key_nib
 *                       512-B aligned, key_scale 16-B aligned.
 *   n_max               entries per sequence; a positive multiple of 128.
 *   n_seq               number of sequences (>= 1).
 *   q_nib, q_scale      (device) indexer queries, IDX format, rows = n_q*32;
 *                       q_nib 512-B aligned, q_scale 16-B aligned.
 *   w                   (device) fp32 [n_q][32] per-head weights, 16-B aligned.
 *   q_seq               (device) int32 [n_q] sequence of each query.
 *   n_vis               (device) int32 [n_q]: entries [0, n_vis) are visible.
 *   n_q                 number of queries (0 launches nothing).
 *   pool_blocks         NULL: Full mode, scores[q][j] for j < n_vis[q] (other
 *                       columns untouched).  Non-NULL (device) int32 [n_q][2048]
 *                       block ids (-1 = none): Reindex mode, scores[q][s] for the
 *                       16,384 pool slots s (entry 8*pool_blocks[q][s/8] + s%8),
 *                       -inf for a slot whose block is -1 or whose entry is not
 *                       visible (same page, lightning-indexer note: decoder
 *                       Reindex layers score only the 16,384 positions of the
 *                       pool an earlier layer picked as 2,048 blocks of 8).
 *   scores              (device) fp32, row stride score_stride (>= n_max in Full
 *                       mode, >= 16384 in Reindex mode).
 */
csa2_status csa2_index_score(const void *key_nib, const void *key_scale, int64_t n_max, int n_seq,
                             const void *q_nib, const void *q_scale, const float *w,
                             const int32_t *q_seq, const int32_t *n_vis, int n_q,
                             const int32_t *pool_blocks, float *scores, int64_t score_stride,
                             const csa2_params *params, csa2_stream_t stream);

/*
 * csa2_topk -- top-k selection by (score descending, index ascending): the lower
 * index wins ties; -0.0 equals +0.0.  Output indices ascending, padded with -1
 * when fewer than k items are valid.
 * (perchy.ai/models/deepseek, card "Full. Reindex. Reuse.": the main selection
 * keeps 512 entries and later decoder indexers look at no more than 16,384
 * candidates; An infra-oriented diagram of the DeepSeek-V4.1-Flash architecture,
 * lightning-indexer note: those candidates are 2,048 blocks of 8 entries.)
 *
 *   scores        (device) fp32 [n_q][score_stride].
 *   n_valid       (device) int32 [n_q]: number of visible entries.
 *   n_max         entries per row considered (Full mode: columns [0, n_max);
 *                 <= score_stride).
 *   k             1 .. 2048.
 *   block         1: items are entries j < n_valid.
 *                 8: items are blocks b of 8 entries (b*8 < n_valid), scored by
 *                    the max over their visible entries (a reading of the
 *                    card's selection in 8-entry blocks); the output holds block
 *                    ids.  pool_blocks must be NULL.
 *   pool_blocks   NULL, or (device) int32 [n_q][2048] when the scores are Reindex
 *                 pool slots (row length 16384): item s is entry
 *                 8*pool_blocks[q][s/8] + s%8, valid if the block id is >= 0 and
 *                 the entry < n_valid; the output holds those entry indices.
 *   out           (device) int32 [n_q][k].
 *   workspace     (device) scratch of at least csa2_workspace_size(CSA2_OP_TOPK,..)
 *                 bytes, 256-B aligned; contents need no initialisation.
 */
csa2_status csa2_topk(const float *scores, int64_t score_stride, int n_q, const int32_t *n_valid,
                      int64_t n_max, int k, int block, const int32_t *pool_blocks, int32_t *out,
                      void *workspace, size_t workspace_bytes, csa2_stream_t stream);

/*
 * csa2_sparse_attn -- 64-head MQA attention over the selected entries plus the
 * sliding window, k = v.
 * (An infra-oriented diagram of the DeepSeek-V4.1-Flash architecture, reading
 * notes: each token has one 512-wide latent serving as both key and value for
 * all 64 query heads; attention covers the selected 512 entries plus the
 * window; RoPE acts on 64 of the 512 dimensions and is undone on the output.
 * DeepSeek V4.1 Flash: Why Its Encoder, Engram and KV Cache Matter, section
 * "CSA2 makes long context cheaper to retain": the window is the last 128
 * tokens.)  For each query and head h:
 *     l_i = sm_scale * q_h . khat_i  over i in {selected} + {window}
 *     o_h = sum_i softmax(l)_i khat_i
 * then the pairs (rope_off + 2i, rope_off + 2i + 1), i < 32, are rotated by
 * -pos:  (a, b) <- (a cos t + b sin t, -a sin t + b cos t),
 * t = pos * rope_base^(-2i/64).  A query with no entry at all gets zeros.
 * Arithmetic: dequantised latents are exact (f16 for chunks of selected
 * entries only, bf16 for chunks holding window entries), products accumulate
 * in fp32, and the softmax numerators are rounded to f16 (11 bits) or kept as
 * bf16 hi + lo parts; the row-normalised error against an fp64 evaluation is
 * about 2e-4 (under 2e-3).  A query's heads share one power of two in f16, so this
 * holds for heads within about 2^24 of its largest (csa2_paged_attn scales each).
 *
 *   q            (device) bf16 [n_q][64][512] (already rotated by upstream).
 *   kv_cache     (device) KV records [n_seq][n_max][288].
 *   sel          (device) int32 [n_q][sel_stride]: entry indices (< n_max) or -1;
 *                sel_stride in 1 .. 512.
 *   swa_cache    (device) SWA records [n_seq][swa_cap][528]; may be NULL when
 *                swa_cap == 0.
 *   q_seq, pos   (device) int32 [n_q]: sequence id, RoPE position of the query.
 *   swa_first, swa_cnt  (device) int32 [n_q]: the window is ring slots
 *                (swa_first + t) % swa_cap, t < swa_cnt, with
 *                0 <= swa_cnt <= min(128, swa_cap) and 0 <= swa_first < swa_cap
 *                when swa_cnt > 0; a query breaking this (or with q_seq out of
 *                range) records CSA2_ERR_BOUNDS and gets zeros.
 *   out          (device) [n_q][64][512], bf16 or fp32 per out_dtype.
 *   workspace    (device) >= csa2_workspace_size(CSA2_OP_SPARSE_ATTN, ..) bytes.
 */
csa2_status csa2_sparse_attn(const void *q, const void *kv_cache, int64_t n_max, int n_seq,
                             const int32_t *sel, int sel_stride, const void *swa_cache, int swa_cap,
                             const int32_t *q_seq, const int32_t *pos, const int32_t *swa_first,
                             const int32_t *swa_cnt, int n_q, void *out, int out_dtype,
                             const csa2_params *params, void *workspace, size_t workspace_bytes,
                             csa2_stream_t stream);

/*
 * csa2_decode -- one Full-layer decode step: csa2_index_score over every
 * visible entry, top-512 selection, csa2_sparse_attn over the selection and
 * the window, issued as one call.  The pages give no such call; it composes
 * the three steps above (same arguments, same meaning, the same selection as
 * the chain csa2_index_score -> csa2_topk(k = 512, block = 1) ->
 * csa2_sparse_attn(sel_stride = 512)), and lets the indexer's epilogue also
 * write the maxima the selection starts from, which saves the selection's
 * first pass over the scores.  For small batches (up to about 30 queries on
 * 152 SMs) over long rows, the selection also hands its candidates (a superset
 * of the selected entries, at most 640, in index order) to the attention before
 * its exact pass, and the attention masks those below the smallest selected
 * key: the output then attends to exactly the selected entries and the window,
 * but groups them into other chunks than csa2_sparse_attn does, so it agrees
 * with the chain's to rounding (relative 1e-3) rather than bit for bit; the
 * same holds for batches (about 39 to 76 queries on 152 SMs) where the
 * attention runs a query's window chunk first in its last split, while the
 * selection finishes.  The same inputs give the same bits on every call.
 *
 *   key_nib .. n_q      as csa2_index_score (Full mode; scores are kept in the
 *                       workspace).
 *   q .. swa_cnt, out, out_dtype, params   as csa2_sparse_attn.
 *   sel                 (device) int32 [n_q][512]: the selected entries
 *                       (ascending, -1 padding), as csa2_topk writes them.
 *   workspace           (device) >= csa2_workspace_size(CSA2_OP_DECODE, n_q,
 *                       n_max, 512) bytes, 256-B aligned; no initialisation.
 */
csa2_status csa2_decode(const void *key_nib, const void *key_scale, int64_t n_max, int n_seq, const void *q_nib,
                        const void *q_scale, const float *w, const int32_t *q_seq, const int32_t *n_vis, int n_q,
                        const void *q, const void *kv_cache, const void *swa_cache, int swa_cap, const int32_t *pos,
                        const int32_t *swa_first, const int32_t *swa_cnt, int32_t *sel, void *out, int out_dtype,
                        const csa2_params *params, void *workspace, size_t workspace_bytes, csa2_stream_t stream);

/*
 * csa2_decode_reindex -- the decode step of a Reindex layer ("An
 * infra-oriented diagram of the DeepSeek-V4.1-Flash architecture", reading
 * notes on the Full / Reindex / Reuse roles; perchy.ai card "Full. Reindex.
 * Reuse."): the layer's own indexer query scores the 16,384 positions of the
 * candidate pool the Full layer chose (2,048 blocks of 8), the top-512 of the
 * pool is selected, and the attention runs over it and the window, as one
 * call.  The results are those of the chain csa2_index_score (pool mode) ->
 * csa2_topk(k = 512, block = 1, pool_blocks) -> csa2_sparse_attn(sel_stride =
 * 512): the selection bit for bit, the output bit for bit where the attention
 * splits a query's chunks as csa2_sparse_attn does, else to rounding (relative
 * 1e-3; for some batch sizes the call runs a query's window chunk first in its
 * last split, while the selection finishes).  Inside the call the indexer also
 * writes the largest order key of every 8-entry block of the pool, so that
 * the selection reads only the blocks that can hold one of the 512, and the
 * attention, whose inputs are final before the call starts, stages them while
 * the selection runs.
 *
 *   key_nib .. n_q      as csa2_index_score; q_nib, q_scale, w are the
 *                       Reindex layer's indexer query and weights.
 *   pool_blocks         (device) int32 [n_q][2048]: the pool's block ids, as
 *                       csa2_topk(block = 8) writes them (-1: none).
 *   q .. swa_cnt, out, out_dtype, params   as csa2_sparse_attn.
 *   sel                 (device) int32 [n_q][512]: the selected entries
 *                       (ascending, -1 padding), as csa2_topk writes them.
 *   workspace           (device) >= csa2_workspace_size(CSA2_OP_DECODE_REINDEX,
 *                       n_q, n_max, 512) bytes, 256-B aligned; no initialisation.
 */
csa2_status csa2_decode_reindex(const void *key_nib, const void *key_scale, int64_t n_max, int n_seq,
                                const void *q_nib, const void *q_scale, const float *w, const int32_t *q_seq,
                                const int32_t *n_vis, int n_q, const int32_t *pool_blocks, const void *q,
                                const void *kv_cache, const void *swa_cache, int swa_cap, const int32_t *pos,
                                const int32_t *swa_first, const int32_t *swa_cnt, int32_t *sel, void *out,
                                int out_dtype, const csa2_params *params, void *workspace, size_t workspace_bytes,
                                csa2_stream_t stream);

/*
 * csa2_index_score_mq -- csa2_index_score (Full mode) for groups of queries
 * that share a sequence, such as several draft positions of one sequence
 * decoded in the same step (DeepSeek V4.1 Flash: Why Its Encoder, Engram and
 * KV Cache Matter, section on DSpark: five future positions per step).  The
 * queries [g * q_group, g * q_group + q_group) must all name the same
 * sequence; each of its key units is read once for the whole group and
 * multiplied with all 32 x q_group query heads at once.  Results as
 * csa2_index_score for every query (scores[q][j] for j < n_vis[q]).
 *
 *   q_group    1 .. 6; n_q a multiple of q_group.  A group whose queries name
 *              different sequences (or an out-of-range sequence or length) is
 *              skipped and records CSA2_ERR_BOUNDS.
 *   the rest   as csa2_index_score (no pool mode).
 */
csa2_status csa2_index_score_mq(const void *key_nib, const void *key_scale, int64_t n_max, int n_seq,
                                const void *q_nib, const void *q_scale, const float *w, const int32_t *q_seq,
                                const int32_t *n_vis, int n_q, int q_group, float *scores, int64_t score_stride,
                                const csa2_params *params, csa2_stream_t stream);

/*
 * csa2_decode_mq -- the decode step of csa2_decode for groups of q_group
 * queries per sequence: csa2_index_score_mq, then the top-512 of every query
 * (csa2_topk), then csa2_sparse_attn of every query; the results are those of
 * that chain.  Arguments as csa2_decode, with q_group as in
 * csa2_index_score_mq; workspace >= csa2_workspace_size(CSA2_OP_DECODE_MQ,
 * n_q, n_max, 512) bytes, 256-B aligned, no initialisation.
 */
csa2_status csa2_decode_mq(const void *key_nib, const void *key_scale, int64_t n_max, int n_seq, const void *q_nib,
                           const void *q_scale, const float *w, const int32_t *q_seq, const int32_t *n_vis, int n_q,
                           int q_group, const void *q, const void *kv_cache, const void *swa_cache, int swa_cap,
                           const int32_t *pos, const int32_t *swa_first, const int32_t *swa_cnt, int32_t *sel,
                           void *out, int out_dtype, const csa2_params *params, void *workspace,
                           size_t workspace_bytes, csa2_stream_t stream);

/*
 * csa2_decode_host -- csa2_decode with the step's inputs and outputs in host
 * memory: the end-to-end call of a decode step.  The caches (indexer keys,
 * latents, window) stay resident in device memory; the per-step tensors
 * travel with the call.  On `stream`, in order: the inputs into the
 * workspace -- where all four input buffers are page-locked (cudaHostAlloc,
 * cudaMallocHost, cudaHostRegister: device-accessible under unified
 * addressing), one kernel reads them in place and packs the indexer query;
 * otherwise one cudaMemcpyAsync per buffer and csa2_fp4_pack --, then
 * csa2_decode, whose last grid writes the output straight into h_out where
 * that is page-locked (else into the workspace, then one cudaMemcpyAsync),
 * then one cudaMemcpyAsync into h_sel, if given.  Either way the results are
 * the same.  Asynchronous: the host buffers must stay valid
 * and unchanged (and the outputs unread) until the stream has passed the
 * call; pageable memory works but serialises the copies.
 *
 *   key_nib .. n_seq, kv_cache, swa_cache, swa_cap   (device) as csa2_decode.
 *   h_q        (host) bf16 [n_q][64][512], the attention query (rotated).
 *   h_qidx     (host) bf16 [n_q][32][128], the indexer query before packing.
 *   h_w        (host) fp32 [n_q][32], the indexer head weights.
 *   h_desc     (host) int32 [5][n_q]: rows q_seq, n_vis, pos, swa_first,
 *              swa_cnt (meanings as csa2_decode).
 *   h_sel      (host, may be NULL) int32 [n_q][512]: receives the selection.
 *   h_out      (host) [n_q][64][512], bf16 or fp32 per out_dtype.
 *   workspace  (device) >= csa2_workspace_size(CSA2_OP_DECODE_HOST, n_q,
 *              n_max, 512) bytes, 256-B aligned; no initialisation.
 * Argument checks and errors as csa2_decode; a failed copy returns
 * CSA2_ERR_CUDA.
 */
csa2_status csa2_decode_host(const void *key_nib, const void *key_scale, int64_t n_max, int n_seq, const void *kv_cache,
                             const void *swa_cache, int swa_cap, const void *h_q, const void *h_qidx, const float *h_w,
                             const int32_t *h_desc, int n_q, int32_t *h_sel, void *h_out, int out_dtype,
                             const csa2_params *params, void *workspace, size_t workspace_bytes, csa2_stream_t stream);

/*
 * csa2_index_key_proj -- the indexer keys of cache entries: the 512 -> 128
 * projection of each entry's latent ("An infra-oriented diagram of the
 * DeepSeek-V4.1-Flash architecture", reading notes on the Full layer's global
 * KV: the indexer's key is a 512 -> 128 projection of the same latent).  The
 * pages give no weights; the caller supplies them.
 *   keys[r][n] = bf16( sum_c latent[r][c] * w_idx[n][c] ), fp32 accumulation on
 *   the tensor cores, rounded to nearest even.
 *   latent  (device) bf16 [rows][512], 16-B aligned.
 *   w_idx   (device) bf16 [128][512], 16-B aligned.
 *   keys    (device) bf16 [rows][128], 16-B aligned; the input of
 *           csa2_fp4_pack(CSA2_IDX_MXFP4, ...).
 */
csa2_status csa2_index_key_proj(const void *latent, int64_t rows, const void *w_idx, void *keys,
                                csa2_stream_t stream);

/*
 * csa2_build_cache -- the cache entries of a prompt (the study's reading
 * notes: encoder caches pool two tokens into one entry with a learned softmax
 * gate, m = 2; the decoder's Full layer keeps one entry per token, m = 1; the
 * indexer's key is a 512 -> 128 projection of the entry's latent): per entry,
 * the latent (gated pooling for m = 2), its 288-B main-cache record, its key
 * (csa2_index_key_proj) and the key's two-plane 68-B record -- the same bytes
 * as csa2_fp4_pack(CSA2_KV_NVFP4, m), csa2_index_key_proj and
 * csa2_fp4_pack(CSA2_IDX_MXFP4) on the pooled latents.  Prompts of any length
 * (1,048,576 tokens and more) are built in chunks of 131,072 entries, so the
 * scratch stays bounded (168 MB for m = 2, 34 MB for m = 1).
 *   tokens       (device) bf16 [n_tokens][512], 16-B aligned.
 *   n_tokens     a multiple of 8 m (so that chunks start on 8-row boundaries
 *                of the key plane).
 *   m, gate_logits   as csa2_fp4_pack (gate_logits [n_tokens][512] for m = 2,
 *                NULL for m = 1).
 *   w_idx        (device) bf16 [128][512].
 *   kv           (device) [n_tokens / m][288]; idx_nib [n_tokens / m][64]
 *                (512-B aligned, the swizzled key plane); idx_scale
 *                [n_tokens / m][4].  Entry e of the prompt is row e of each.
 *   workspace    (device) >= csa2_workspace_size(CSA2_OP_BUILD_CACHE, 0,
 *                n_tokens, m) bytes, 256-B aligned; no initialisation.
 */
csa2_status csa2_build_cache(const void *tokens, int64_t n_tokens, int m, const float *gate_logits,
                             const void *w_idx, void *kv, void *idx_nib, void *idx_scale, void *workspace,
                             size_t workspace_bytes, csa2_stream_t stream);

/*
 * csa2_profile_events -- measurement hook: while set, csa2_decode and
 * csa2_decode_reindex record `begin` on their stream just before they launch
 * the indexer and `end` just after it, so that the indexer kernel of the step
 * itself (the instantiation that also writes the selection's maxima) can be
 * timed with cudaEventElapsedTime.  Recording between the step's kernels keeps
 * the next kernel from starting early beside the indexer, so a step timed this
 * way runs a little slower than one that is not.  Both null: off.  The setting
 * is per host thread.
 *
 *   begin, end   cudaEvent_t (created by the caller), or both null.
 */
csa2_status csa2_profile_events(void *begin, void *end);

/*
 * Paged caches.  The main cache is n_pages pages of page_size KV records,
 * [n_pages][page_size][288], 32-B aligned; page_size is any positive number.
 * Row b of a block table (int32 [n_seq][table_stride]) names the pages of
 * sequence b in order: its entry j is record j % page_size of page
 * block_table[b][j / page_size], and the entry's slot is its place in the whole
 * cache, page * page_size + j % page_size (csa2_sparse_attn and csa2_decode keep
 * their contiguous caches).  The window stays a ring of swa_cap records per
 * sequence, [n_seq][swa_cap][528], position p of sequence b in slot
 * b * swa_cap + p % swa_cap.  All pointers belong to the current device.
 *
 * csa2_page_plan -- block tables, slots and descriptors of a step from the
 * sequences' lengths.  Sequence b holds seq_len[b] entries and gets new_len[b]
 * tokens, at positions seq_len[b], seq_len[b] + 1, ...  The step's tokens are
 * numbered in sequence order, and so are the pages it needs: columns
 * ceil(seq_len / page_size) .. ceil((seq_len + new_len) / page_size) - 1 of row b
 * of the block table are written with the next pages of the free list; no other
 * column is written.  One launch; the host reads nothing.  An entry is a token
 * (m = 1): caches that pool two tokens into an entry need descriptors of their own.
 *
 *   seq_len, new_len  (device) int32 [n_seq]; n_seq in 0 .. 16384.  A sequence
 *                with a negative length, or with more entries than its row of
 *                the block table can hold, records CSA2_ERR_BOUNDS and gets no
 *                tokens.
 *   free_pages   (device) int32 [n_free] page ids; free_head (device) int32 [1]
 *                or NULL (0): the first one to take.  Where the list ends, or
 *                names no page, CSA2_ERR_BOUNDS is recorded, the column gets -1
 *                and the tokens on it get slot -1 (so do tokens on an earlier
 *                column that names no page).
 *   desc         (device) int32 [7][max_tokens], per token: its sequence
 *                (q_seq); the entries it sees, itself included (n_vis = pos + 1);
 *                pos; the window's first ring slot and length (swa_first,
 *                swa_cnt = min(128, swa_cap, pos + 1)); its slot in the main
 *                cache; its slot in the window cache, or -1 where a later token
 *                of the same step (one below max_tokens) takes the same ring slot.  Rows 0 .. 4 are
 *                csa2_decode_host's h_desc rows.  Columns behind the last token
 *                get 0, 0, 0, 0, 0, -1, -1: queries that attend to nothing and
 *                write nothing.  Tokens from max_tokens on are dropped and record
 *                CSA2_ERR_BOUNDS.  The windows are those of tokens whose window
 *                records are written one after another; a caller that writes all of
 *                a step's records before it attends needs a ring that holds them
 *                beside the first token's window, new_len + min(seq_len, w - 1) <=
 *                swa_cap for w = min(128, swa_cap), or the first tokens see later
 *                ones.  The plan does not know the order and reports nothing;
 *                decode.PagedCache gives such a sequence no tokens.
 *   first        (device) int32 [n_seq + 1]: the first token of each sequence,
 *                then the number of tokens (sums beyond 2^31 - 1 stay there).
 *   totals       (device) int32 [2]: the tokens, and the pages the step needs
 *                (advance free_head by as many).
 *   Limits: n_pages * page_size and n_seq * swa_cap below 2^31.  (A step of more
 *   tokens than csa2_paged_attn's 65,535 is attended to in parts: rows of desc from
 *   a column on.)
 */
csa2_status csa2_page_plan(const int32_t *seq_len, const int32_t *new_len, int n_seq, int page_size, int n_pages,
                           const int32_t *free_pages, int n_free, const int32_t *free_head, int32_t *block_table,
                           int64_t table_stride, int swa_cap, int32_t *desc, int max_tokens, int32_t *first,
                           int32_t *totals, csa2_stream_t stream);

/*
 * csa2_qk_norm_rope -- the norm of every query head and of the latent, the
 * rotation of their last 64 dims, and the latent's cache write, in one pass:
 * what csa2_sparse_attn and csa2_paged_attn expect "already rotated by
 * upstream".  ("An infra-oriented diagram of the DeepSeek-V4.1-Flash
 * architecture", reading notes: RoPE acts on 64 of the 512 dims, and the cache
 * stays in one rotated form.)  Per 512-wide row x with gain g:
 *     y_c = g_c x_c / sqrt(mean_c(x_c^2) + eps)
 * then the pairs (rope_off + 2i, rope_off + 2i + 1), i < 32, are rotated by
 * +pos:  (a, b) <- (a cos t - b sin t, a sin t + b cos t),
 * t = pos * rope_base^(-2i/64).  Queries are computed in fp32 (rows that fp32
 * squares do not hold in fp64) and rounded once; the latent is the exact value
 * rounded once to bf16 (to 2^-30 of it, or of the pair that it was rotated from, at
 * any position), and its records are those csa2_fp4_pack makes of that bf16 row,
 * byte for byte.
 *
 *   q            (device) bf16, token t's 64 heads at q + t * q_stride elements
 *                ([64][512] each; q_stride >= 32768, a multiple of 8); NULL: no
 *                queries.  q_out (device) bf16 [n][64][512]; it may be q itself
 *                where q_stride is 32768, and must not overlap q otherwise (nor may
 *                any output overlap another input).
 *   latent       (device) bf16, row t at latent + t * latent_stride elements
 *                (>= 512, a multiple of 8); NULL: none.  latent_out (device) bf16
 *                [n][512] or NULL: the normed, rotated latents (the input of
 *                csa2_index_key_proj); in place as q_out.
 *   q_gain, latent_gain   (device) fp32 [512], 16-B aligned, or NULL: all ones.
 *   pos          (device) int32 [n].
 *   slot         (device) int32 [n]: the KV record of kv_cache (kv_slots records)
 *                that row t is written to, -1: none; kv_cache NULL: no records.
 *   swa_slot     the same for the window cache (swa_slots records of 528 B).
 *                A slot at or above kv_slots / swa_slots is skipped and records
 *                CSA2_ERR_BOUNDS.  Each slot may be named once per call (the
 *                bytes of a record named twice are unspecified).
 *   n            tokens; 0 launches nothing.  eps > 0.
 */
csa2_status csa2_qk_norm_rope(const void *q, int64_t q_stride, const float *q_gain, void *q_out, const void *latent,
                              int64_t latent_stride, const float *latent_gain, void *latent_out, const int32_t *pos,
                              const int32_t *slot, const int32_t *swa_slot, int n, double eps, void *kv_cache,
                              int64_t kv_slots, void *swa_cache, int64_t swa_slots, const csa2_params *params,
                              csa2_stream_t stream);

/*
 * csa2_cache_read -- records back to 512-wide latents: out[i] is the dequantised
 * record slots[i], exact in fp32 and rounded once for bf16 (exact there too for
 * KV records, and for window records down to bf16's smallest value).
 *   kind      CSA2_KV_NVFP4 or CSA2_SWA_MXFP8 (indexer keys: unsupported).
 *   cache     (device) n_slots records, 16-B aligned.
 *   slots     (device) int32 [n]; a negative slot gives zeros, one at or above
 *             n_slots zeros and CSA2_ERR_BOUNDS.
 *   out       (device) [n][512], bf16 or fp32 per out_dtype, 16-B aligned.
 * Codes that no packer writes are not read alike: a KV scale of 0x7F is 480 here and
 * NaN in the attention, a window scale of byte 0 with codes other than zero counts
 * as 2^-127 here and as zero there.
 */
csa2_status csa2_cache_read(int kind, const void *cache, int64_t n_slots, const int32_t *slots, int64_t n, void *out,
                            int out_dtype, csa2_stream_t stream);

/*
 * csa2_paged_attn -- csa2_sparse_attn's attention (64 heads, k = v, window, RoPE
 * undone on the output) over a paged main cache, for every visible entry or for
 * a selection, with the log-sum-exp of the logits.  A query q of sequence b
 * attends to the entries [0, n_vis[q]) of b -- or, with sel, to the entries
 * sel[q] -- and to its window; one new token or several of a sequence, each
 * with its own n_vis.  A long row is split over the SMs and joined, whatever the
 * rows' lengths; the same inputs give the same bits on every call.
 * Arithmetic as csa2_sparse_attn on FP4 latents (f16 products of exact
 * dequantised latents, fp32 sums, numerators rounded to 11 bits): row-normalised
 * error against an fp64 evaluation about 2e-4 (under 2e-3); lse to about 1e-6
 * where the logits are of unit size (and within 1e-4: fp32 sums of 512 products).
 * out and lse must not overlap any input.
 *
 *   q            (device) bf16 [n_q][64][512], rotated (csa2_qk_norm_rope).
 *   pages .. n_seq   the paged cache and its block table (above).  A table entry
 *                outside [0, n_pages) in a row's visible part: its entries are
 *                skipped and CSA2_ERR_BOUNDS is recorded.
 *   sel          NULL, or (device) int32 [n_q][sel_stride], sel_stride in 1 ..
 *                512: entry indices below n_vis[q], or negative (none); an index at
 *                or above n_vis[q] is skipped and records CSA2_ERR_BOUNDS.
 *   swa_cache .. swa_cnt, pos, out, out_dtype, params   as csa2_sparse_attn.
 *   n_vis        (device) int32 [n_q], at most table_stride * page_size; a query
 *                with q_seq, n_vis or the window out of range records
 *                CSA2_ERR_BOUNDS and gets zeros.  A query with no entry at all
 *                gets zeros and an lse of -inf.
 *   lse          NULL, or (device) fp32 [n_q][64]: log sum_i exp(l_i), which joins
 *                outputs over disjoint sets of entries (the un-rotation is linear).
 *   workspace    (device) >= csa2_workspace_size(CSA2_OP_PAGED_ATTN, 0, 0, 0)
 *                bytes, 256-B aligned; no initialisation.  Calls that may run at
 *                the same time need one each.
 *   Limits: n_q <= 65535; n_pages * page_size below 2^31; n_q * (row / 128 + 1) up to 2^30, row = sel_stride or
 *   table_stride * page_size.  Each head of a query has its own scale: whatever it
 *   holds, an infinity or NaN among it, the query's other heads stay as they are.
 */
csa2_status csa2_paged_attn(const void *q, const void *pages, int n_pages, int page_size, const int32_t *block_table,
                            int64_t table_stride, int n_seq, const int32_t *sel, int sel_stride, const void *swa_cache,
                            int swa_cap, const int32_t *q_seq, const int32_t *n_vis, const int32_t *pos,
                            const int32_t *swa_first, const int32_t *swa_cnt, int n_q, void *out, int out_dtype,
                            float *lse, const csa2_params *params, void *workspace, size_t workspace_bytes,
                            csa2_stream_t stream);

/*
 * What a paged cache keeps.  A cache that loses entries has places that are no
 * positions any more: entry j of a sequence is its j-th one still there, and
 * gone[b] counts those that were lost.  (A latent carries its position's rotation,
 * and attention does not depend on the entries' order.)
 *
 * csa2_page_plan_at -- csa2_page_plan for such caches: the new tokens of sequence
 * b take places seq_len[b], seq_len[b] + 1, .. (block tables, slots, n_vis = place +
 * 1) at positions gone[b] + seq_len[b], .. (pos, the window and its ring).
 *
 *   gone         NULL (none: csa2_page_plan), or (device) int32 [n_seq].  A
 *                negative one, or positions beyond 2^31 - 1, record
 *                CSA2_ERR_BOUNDS, and the sequence gets no tokens.
 */
csa2_status csa2_page_plan_at(const int32_t *seq_len, const int32_t *new_len, const int32_t *gone, int n_seq,
                              int page_size, int n_pages, const int32_t *free_pages, int n_free,
                              const int32_t *free_head, int32_t *block_table, int64_t table_stride, int swa_cap,
                              int32_t *desc, int max_tokens, int32_t *first, int32_t *totals, csa2_stream_t stream);

/*
 * csa2_attn_weight -- the attention weight that the main cache's entries get from
 * a step's queries, added to what they had:
 *     weight[s] = decay * prior[s] + sum_q sum_h exp(sm_scale q_h . k_j - lse[q][h])
 * for the slot s of every entry j that a query of its sequence sees (j below the
 * largest n_vis), the sum over the sequence's queries that see j and their 64
 * heads.  With the lse of csa2_paged_attn over the same entries these are the
 * softmax weights with which the queries attended to j (the window's entries have
 * the rest).  Queries of one sequence are neighbours.  fp32 sums in a fixed order:
 * the same inputs give the same bits.  A head whose lse or query is not finite adds
 * nothing (and one that attended to nothing, with an lse of -inf).
 *
 *   q            (device) bf16 [n_q][64][512], as csa2_paged_attn's.
 *   pages .. table_stride   the paged cache and its block table.  A table entry
 *                outside [0, n_pages): its entries are skipped and CSA2_ERR_BOUNDS
 *                is recorded.  Sequences may not share pages here.
 *   first        (device) int32 [n_seq + 1]: sequence b's queries are first[b] ..
 *                first[b + 1] - 1 (csa2_page_plan's); out of range of n_q: recorded, the
 *                sequence is skipped (and all, where ranges cross so often that their work
 *                passes 32 bits; with sel a query that several ranges have counts for
 *                one of them).  A sequence without queries is left as it is.
 *   sel          NULL, or (device) int32 [n_q][sel_stride], as csa2_paged_attn's: a
 *                query sees the entries sel[q] only; one named twice counts twice.
 *                decay still takes all entries below the largest n_vis.  (An entry
 *                without a page is recorded where it is selected.)  Of a query
 *                with an n_vis of 0 it is not read.
 *   n_vis        (device) int32 [n_q]; outside [0, table_stride * page_size]:
 *                recorded, the query adds nothing.
 *   lse          (device) fp32 [n_q][64].
 *   prior        NULL (zeros), or (device) fp32 [n_pages * page_size], by slot; it
 *                may be weight itself, and may not overlap it otherwise.
 *   weight       (device) fp32 [n_pages * page_size].  Slots of other entries are
 *                left as they are.
 *   workspace    (device) >= csa2_workspace_size(CSA2_OP_ATTN_WEIGHT, n_q, n_seq,
 *                sel_stride or 0) bytes, 256-B aligned; no initialisation.  Calls
 *                that may run at the same time need one each.
 *   Limits: n_q <= 65535; n_seq <= 16384; n_pages * page_size below 2^31, table_stride *
 *   page_size up to 2^31 - 256; n_q * (row / 128 + 1) up to 2^30, row = sel_stride or table_stride * page_size.
 */
csa2_status csa2_attn_weight(const void *q, const void *pages, int n_pages, int page_size, const int32_t *block_table,
                             int64_t table_stride, const int32_t *first, int n_seq, const int32_t *sel, int sel_stride,
                             const int32_t *n_vis, const float *lse, int n_q, float decay, const float *prior,
                             float *weight, const csa2_params *params, void *workspace, size_t workspace_bytes,
                             csa2_stream_t stream);

/*
 * csa2_evict -- cuts sequences down to their heaviest entries.  Of the seq_len[b]
 * entries of sequence b, k = min(keep[b], seq_len[b]) stay: the last min(recent, k),
 * and of the others those of largest weight (of equal ones those at the lowest
 * places; -0 equals 0; NaN is lighter than everything).  They keep their order, and
 * their records and weights go to places 0 .. k - 1 of row b of the destination.
 * In place, the weights of the places behind become 0.  Nothing else is written.
 *
 *   pages .. table_stride, seq_len   the paged cache; weight (device) fp32
 *                [n_pages * page_size] by slot, 16-B aligned.  An entry on a column
 *                that names no page is taken for the lightest, recorded as
 *                CSA2_ERR_BOUNDS and, where it stays all the same, not copied.
 *                Sequences may not share pages here.
 *   keep         (device) int32 [n_seq].  recent >= 0.
 *   dst_pages .. dst_stride   the destination, of the same page_size: other pages, of
 *                the same cache (another table) or of another one, none of which is
 *                read here or named twice, with their weights; or the source itself (the same
 *                pointers): then the entries move in place.  (The pages behind
 *                them: csa2_page_trim.)
 *   new_len      (device) int32 [n_seq]: k.  May be seq_len itself.
 *   from         NULL, or (device) int32 [n_seq][from_stride]: the places that the
 *                kept entries come from, in order; what is behind them is left as
 *                it is.  (For what else a caller keeps of an entry.)
 *   A negative length or keep, a length that the block table cannot hold, or more
 *   kept entries than the destination or from can: CSA2_ERR_BOUNDS is recorded,
 *   nothing of the sequence moves, and new_len is seq_len in place, else 0.
 *   In place the kernel's blocks wait for one another's reads.  A wait that runs
 *   out (2 s) is recorded as CSA2_ERR_TIMEOUT: places that had not been written by
 *   then keep what they held, and the sequences are not whole any more.
 *   workspace    (device) >= csa2_workspace_size(CSA2_OP_EVICT, n_seq, table_stride
 *                * page_size, 0) bytes, 256-B aligned; no initialisation.  Calls
 *                that may run at the same time need one each.
 *   Limits: n_seq <= 16384; caches of fewer than 2^31 entries, rows of up to 2^31 - 256.
 */
csa2_status csa2_evict(const void *pages, const float *weight, int n_pages, int page_size, const int32_t *block_table,
                       int64_t table_stride, const int32_t *seq_len, const int32_t *keep, int n_seq, int recent,
                       void *dst_pages, float *dst_weight, int n_dst_pages, const int32_t *dst_table,
                       int64_t dst_stride, int32_t *new_len, int32_t *from, int64_t from_stride, void *workspace,
                       size_t workspace_bytes, csa2_stream_t stream);

/*
 * csa2_page_trim -- gives the pages behind new lengths back to the free list:
 * columns ceil(new_len / page_size) .. ceil(len / page_size) - 1 of every sequence's
 * row of the block table go to the places ahead of free_head, in sequence order,
 * and get -1 in the table; free_head moves back by as many.
 *
 *   len, new_len (device) int32 [n_seq], 0 <= new_len <= len, len within its row:
 *                else CSA2_ERR_BOUNDS is recorded and the sequence's pages stay.
 *   free_pages, n_free, free_head   as csa2_page_plan's, here written.  More pages
 *                than were taken (free_head), or a free_head outside the list: recorded,
 *                and nothing is given back.  A column that names no page goes to the
 *                list as it is, and is recorded.
 */
csa2_status csa2_page_trim(const int32_t *len, const int32_t *new_len, int n_seq, int page_size, int n_pages,
                           int32_t *free_pages, int n_free, int32_t *free_head, int32_t *block_table,
                           int64_t table_stride, csa2_stream_t stream);

/*
 * csa2_verify_drafts -- which drafted tokens stay, and the token that follows.
 * Rows first[b] .. first[b + 1] - 1 are the tokens of sequence b's step: the last
 * sampled one, then drafts.  Row r of target is the target model's distribution of
 * the token after tokens[r], so draft tokens[r + 1] is judged by row r.
 *   CSA2_VERIFY_SAMPLE: in order, draft x = tokens[r + 1] stays while
 *     u[r] * draft[r][x] < target[r][x].  At the first one that does not, next is
 *     drawn from max(target[r] - draft[r], 0); if all stay, from the last row of
 *     target: the lowest index whose running sum is above v[b] times the total (where
 *     rounding leaves none, the last index of any weight).  If nothing is above zero
 *     there, next is drawn from target[r].  Decided as by exact arithmetic (sums to
 *     about 2^-46 of the total for a vocab of up to 2^20, 2^-42 for 2^28).
 *   draft NULL: the drafts were not drawn (a lookup): draft[r] is 1 at x, 0 elsewhere.
 *   CSA2_VERIFY_GREEDY: x stays while it is the index of row r's largest entry (the
 *     lowest of equal ones; -0 equals 0; NaN is none), which is next otherwise;
 *     target may hold logits; draft NULL; u and v are not read.
 *
 *   target       (device) [n_rows][target_stride] of type dtype, vocab entries a row;
 *                draft likewise.  Element alignment will do; 16-B aligned rows are
 *                read faster.  An entry that is negative, NaN or above 2^96 is
 *                no probability and counts as 0 (SAMPLE).
 *   tokens       (device) int32 [n_rows].  A draft outside [0, vocab) is refused and
 *                recorded as CSA2_ERR_BOUNDS.
 *   first        (device) int32 [n_seq + 1], as csa2_page_plan's; out of range of
 *                n_rows (GREEDY: or of first[n_seq]): recorded, the sequence gets 0 and
 *                -1.  Rows from first[n_seq] on belong to no sequence.
 *   u, v         (device) fp32 [n_rows], [n_seq]: random numbers in [0, 1).
 *   kept         (device) int32 [n_seq]: the step's tokens that stay, the accepted
 *                drafts and the one before them; 0 for a sequence without rows.
 *   next         (device) int32 [n_seq]; -1 for a sequence without rows, and, recorded,
 *                where target[r] has no entry above zero (GREEDY: nothing but NaN).
 *   workspace    GREEDY: (device) >= csa2_workspace_size(CSA2_OP_VERIFY, n_rows, 0, 0)
 *                bytes, 256-B aligned; no initialisation.  Calls that may run at the
 *                same time need one each.  SAMPLE: NULL will do.
 *   Limits: n_seq <= 16384; n_rows <= 65535; vocab <= 2^28.
 */
csa2_status csa2_verify_drafts(int mode, const void *target, int64_t target_stride, const void *draft,
                               int64_t draft_stride, int dtype, int vocab, const int32_t *tokens, const int32_t *first,
                               int n_seq, int n_rows, const float *u, const float *v, int32_t *kept, int32_t *next,
                               void *workspace, size_t workspace_bytes, csa2_stream_t stream);

/*
 * csa2_workspace_size -- scratch bytes needed by an operation.
 *   op = CSA2_OP_TOPK:        n_q queries, n_items = items per row (entries,
 *                             blocks, or 16384 pool slots), k.
 *   op = CSA2_OP_SPARSE_ATTN: n_q queries, n_items = sel_stride + 128, k unused.
 *   op = CSA2_OP_DECODE:      n_q queries, n_items = n_max, k unused (512).
 *   op = CSA2_OP_DECODE_HOST: as CSA2_OP_DECODE (the device copies of the
 *                             step's inputs and outputs are included).
 *   op = CSA2_OP_DECODE_MQ:   n_q queries, n_items = n_max, k unused (512).
 *   op = CSA2_OP_BUILD_CACHE: n_q unused, n_items = tokens, k = m (1 or 2).
 *   op = CSA2_OP_DECODE_REINDEX: n_q queries, n_items = n_max, k unused (512).
 *   op = CSA2_OP_PAGED_ATTN:  n_q, n_items and k unused: the same for every call
 *                             (two partial outputs per SM, 40 MB).
 *   op = CSA2_OP_ATTN_WEIGHT: n_q queries, n_items = n_seq, k = sel_stride (0 without sel).
 *   op = CSA2_OP_EVICT:       n_q = n_seq, n_items = entries of a row (table_stride *
 *                             page_size), k unused.
 *   op = CSA2_OP_VERIFY:      n_q = n_rows, n_items and k unused.
 * Sizes are for the current device (the attention's split plan follows its
 * SM count).
 */
csa2_status csa2_workspace_size(int op, int n_q, int64_t n_items, int k, size_t *bytes);

/*
 * csa2_topk_noalloc -- csa2_topk for callers that cannot allocate device
 * memory: code running where cudaMalloc is not available or not allowed (inside
 * a host callback or another library's allocation-free region, a plugin whose
 * host owns all device memory, a process that must not grow its footprint after
 * start-up).  The pages have no counterpart of this call: it exists only for
 * the library's users.
 *
 * Same arguments, results and errors as csa2_topk, without the workspace.  The
 * scratch it needs (rows longer than 16,384 items only: 4 bytes per group of
 * scores, 2,048 to 16,384 groups per row; for 1,048,576-entry rows and k = 512
 * that is 8 KiB per query) lives in one fixed device array of
 * CSA2_TOPK_NOALLOC_SCRATCH_BYTES (4 MiB), held on each GPU until the process
 * exits.  With CUDA's default lazy module loading the array is mapped on a
 * device only when its module is first loaded there, i.e. by the first call
 * of this function on that device: that first call grows the device
 * footprint by the 4 MiB.  Callers that need a fixed footprint after start-up
 * make one call on each device (any size) during start-up.  A call whose
 * scratch would exceed it returns CSA2_ERR_WORKSPACE and launches nothing (use
 * csa2_topk with a workspace instead).  The call allocates nothing and calls no
 * allocating routine.  The first call on a device looks up the array's device
 * address on that device; make that first call before any stream capture.
 * All calls share the one array: calls that can run at the same time on the
 * GPU (other streams, other host threads) race and must be serialised by the
 * caller.  Nothing has to be cleared between calls: every scratch value a call
 * reads is written (or cleared) earlier in that same call.
 */
#define CSA2_TOPK_NOALLOC_SCRATCH_BYTES (4u << 20)
csa2_status csa2_topk_noalloc(const float *scores, int64_t score_stride, int n_q, const int32_t *n_valid,
                              int64_t n_max, int k, int block, const int32_t *pool_blocks, int32_t *out,
                              csa2_stream_t stream);

/*
 * csa2_check_bounded_wait -- self-test of the library's bounded waits (the
 * pages have no counterpart).  Launches one warp that takes tensor memory,
 * waits on a barrier that nothing will complete, gives up after limit_us
 * microseconds (1 .. 2,000,000), records CSA2_ERR_TIMEOUT in the device
 * status word, returns the tensor memory and exits: the path every kernel of
 * this library takes when one of its waits runs out (each of them bounded by
 * 2 s of wall time), with nothing asynchronous in flight.  Read the outcome
 * with csa2_get_device_status; the context stays usable.
 */
csa2_status csa2_check_bounded_wait(unsigned limit_us, csa2_stream_t stream);

/*
 * csa2_get_device_status -- synchronises `stream`, returns in *out the first
 * device-side error recorded by any kernel of this library on the current
 * device since the last call (CSA2_OK if none), and clears it.
 */
csa2_status csa2_get_device_status(csa2_stream_t stream, csa2_status *out);

#ifdef __cplusplus
}
#endif
#endif /* CSA2_H */
