/*
 * csa2.h -- C ABI of the CSA2 decode hot-path library (libcsa2.so) for
 * NVIDIA GB300 (sm_103a).
 *
 * The library implements the decode-time path of Compressed Sparse
 * Attention 2 as the pages describe it:
 *   - FP4 main-KV write: E2M1 values with one E4M3 scale per 16 channels
 *     (foosynaptic atlas "DeepSeek-V4.1-Flash 梗概", section 3.2, "FP4 main
 *     KV"; newsaint.id "DeepSeek-V4.1-Flash 2026: ...", section 4 and the
 *     FP4Quantizer of section 8);
 *   - the decoder's Hierarchical Sparse Indexer: a Full-mode scan of every
 *     visible position keeps the Top-2048 blocks of 8 as a candidate pool and
 *     Reindex layers score only inside the pool to take Top-512 (atlas,
 *     section 3.2, "Hierarchical Sparse Indexer (decoder)"; newsaint.id,
 *     section 3);
 *   - sparse MLA-style core attention over the selected FP4 main-KV entries
 *     plus an exact bf16 SWA window under one query, for the Full / Reindex /
 *     Reuse layer modes (atlas, section 3.2 mode table and figure "异构 KV";
 *     stamatios.com "DeepSeek-V4.1 Flash comprime cache KV para 890 bytes por
 *     token", section "CSA2: compressão em três dimensões").
 *
 * Conventions for every call
 *   - Pointers named as device pointers are caller-owned GPU memory; the
 *     library never allocates, frees or synchronises (except
 *     csa2_get_device_status, which reads back one word).
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  All work is enqueued on it, in order.
 *   - Argument errors are detected on the host, return a status code and
 *     launch nothing.
 *   - Violations that only the device can see (a context length above the
 *     capacity, a page id or a Top-K index out of range, an SWA length above
 *     the window) set bits in an error word inside the caller's workspace;
 *     the offending entry is skipped.  csa2_get_device_status reads it.
 *     No kernel traps or spins without a bound.
 *   - bf16 tensors are passed as uint16_t bit patterns.
 *   - Index sets are int32 logical positions, sorted ascending; -1 pads.
 *   - Ties in every ranking go to the lower index.
 *   - Inputs must be finite; NaN / Inf inputs give unspecified results.
 *
 * KV layout (main KV planes and indexer K), "rows" being cache slots:
 *   codes   uint8  [rows][256]   packed E2M1, channel 2j low nibble of byte j
 *   scales  uint8  [rows][32]    E4M3 scale of channels 16g..16g+15
 *   rope    bf16   [rows][64]    high-precision key part
 *   idx_k   E4M3   [rows][128], or fp32 [rows][64], or FP4 in two planes:
 *           codes uint8 [rows][64] (E2M1, channel 2j low nibble of byte j)
 *           followed by scales uint8 [rows][8] (E4M3, channels 16g..16g+15),
 *           the scales plane starting at idx_k + rows * 64, where rows =
 *           batch * max_ctx (contiguous) or num_pages * 64 (paged)
 * Logical position t of sequence b lives in row
 *   page_table == NULL : b * dims.max_ctx + t
 *   page_table != NULL : page_table[b * dims.max_pages + t / 64] * 64 + t % 64
 * with 64-position pages and page ids in [0, dims.num_pages).
 */
#ifndef CSA2_H
#define CSA2_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define CSA2_LATENT 512      /* shared latent channels per main-KV entry   */
#define CSA2_ROPE 64         /* bf16 high-precision key channels           */
#define CSA2_DQK 576         /* key / query channels: latent + rope        */
#define CSA2_PAGE 64         /* positions per KV page                      */
#define CSA2_BLOCK 8         /* positions per indexer block                */

typedef enum {
  CSA2_OK = 0,
  CSA2_ERR_INVALID_ARG = 1,        /* null pointer, negative size, bad enum   */
  CSA2_ERR_UNSUPPORTED_SHAPE = 2,  /* dims outside what the kernels support   */
  CSA2_ERR_WORKSPACE_TOO_SMALL = 3,
  CSA2_ERR_CUDA = 4,               /* a CUDA runtime call failed               */
  CSA2_ERR_DEVICE_ASSERT = 5,      /* the device error word is non-zero        */
  CSA2_ERR_TIMEOUT = 6             /* a bounded device wait ran out            */
} csa2_status;

/* Bits of the device error word. */
#define CSA2_DEV_CTX_LEN   0x01  /* ctx_len[b] < 0 or > max_ctx              */
#define CSA2_DEV_PAGE_ID   0x02  /* page id outside [0, num_pages)           */
#define CSA2_DEV_TOPK_IDX  0x04  /* Top-K index outside [-1, ctx_len[b])     */
#define CSA2_DEV_SWA_LEN   0x08  /* swa_len[b] outside [0, dims.swa]         */
#define CSA2_DEV_POOL      0x10  /* pool id / pool_len out of range          */
#define CSA2_DEV_TIMEOUT   0x20  /* a bounded wait gave up                   */
#define CSA2_DEV_Q_START   0x40  /* q_start falls back or leaves [0, total_q] */

typedef enum {
  CSA2_IDXK_E4M3 = 0,   /* indexer K E4M3 [rows][idx_dim], query bf16 */
  CSA2_IDXK_F32 = 1,    /* indexer K fp32 [rows][idx_dim], query fp32 */
  CSA2_IDXK_FP4 = 2     /* indexer K FP4 (two planes, idx_dim 128), query bf16,
                           quantized by the call to the same FP4 format; the
                           score is that of the dequantized query and keys */
} csa2_idxk_dtype;

typedef enum { CSA2_MODE_FULL = 0, CSA2_MODE_REINDEX = 1, CSA2_MODE_REUSE = 2 } csa2_mode;

/* Problem dimensions, shared by every call of a decode step. */
typedef struct {
  int32_t idx_heads;    /* indexer heads Hi, 1..16                            */
  int32_t idx_dim;      /* indexer dim Di: 128 (E4M3, FP4) or 64 (fp32)       */
  int32_t idx_k_dtype;  /* csa2_idxk_dtype                                    */
  int32_t pool_blocks;  /* candidate-pool blocks P, 1..2048 (pages: 2048)     */
  int32_t topk;         /* Top-K, 1..2048 (the pages use 512)                 */
  int32_t heads;        /* attention heads H, 1..64                           */
  int32_t swa;          /* SWA window rows W, 0..128                          */
  int32_t max_pages;    /* row stride of page_table (paged layout)            */
  int64_t num_pages;    /* number of physical pages (paged layout)            */
  int64_t max_ctx;      /* capacity per sequence in positions, 1..2^20;
                           also the row stride between sequences when
                           page_table == NULL                                 */
} csa2_dims;

/* Library version (major * 10000 + minor * 100 + patch). */
int32_t csa2_version(void);

/* Human-readable name of a status code (static string). */
const char* csa2_status_string(csa2_status st);

/* Bytes of workspace that indexer_full_topk, indexer_reindex_topk and
 * csa2_sparse_attn_decode need for `batch` sequences under `d`.  One
 * workspace can serve all three (calls on one stream run in order).  The
 * first 256 bytes hold the device error word; clear the whole workspace
 * (or call csa2_clear_device_status) once before first use.
 * Errors: CSA2_ERR_INVALID_ARG, CSA2_ERR_UNSUPPORTED_SHAPE. */
csa2_status csa2_workspace_size(const csa2_dims* d, int32_t batch, size_t* bytes);

/* FP4 main-KV write (atlas 3.2 "FP4 main KV"; newsaint.id section 8,
 * FP4Quantizer.quantize_and_pack).  For each row of x (bf16 [n][512],
 * device) and each group of 16 channels:
 *   s_code = E4M3(amax/6), round-to-nearest-even, saturating at 448;
 *   element nibble = sign bit << 3 | E2M1 magnitude code of |x|/s, rounded
 *   to nearest with ties to the even code (0 when s == 0).
 * Writes codes (uint8 [n][256], device) and scales (uint8 [n][32], device).
 * Errors: CSA2_ERR_INVALID_ARG (null pointer with n > 0, n < 0),
 *         CSA2_ERR_CUDA (launch failure). */
csa2_status fp4_kv_quantize(const uint16_t* x, int64_t n, uint8_t* codes,
                            uint8_t* scales, void* stream);

/* As fp4_kv_quantize, but row i of x is written to cache row dst_rows[i]
 * (int64 [n], device) -- the decode-time append of new tokens into a paged
 * or strided cache.  Rows with dst_rows[i] < 0 are skipped.  The caller
 * guarantees dst_rows[i] < rows of the cache planes. */
csa2_status fp4_kv_quantize_scatter(const uint16_t* x, int64_t n,
                                    const int64_t* dst_rows, uint8_t* codes,
                                    uint8_t* scales, void* stream);

/* fp4_kv_quantize_scatter with flags (0: the plain call).
 * CSA2_KV_EARLY_INPUTS: the operation enqueued just before this call on the
 * stream writes neither x nor dst_rows and reads or writes none of the
 * destination rows, so the rows may be written while it is still running;
 * the call still completes only after that operation has completed, so
 * later work on the stream sees the results of both.  In a decode step this
 * holds for the newest token's append enqueued after the Full layer's
 * indexer call (which reads no main-KV rows).  Other bits:
 * CSA2_ERR_INVALID_ARG. */
#define CSA2_KV_EARLY_INPUTS 1
csa2_status fp4_kv_quantize_scatter_ex(const uint16_t* x, int64_t n,
                                       const int64_t* dst_rows, uint8_t* codes,
                                       uint8_t* scales, int32_t flags, void* stream);

/* FP4 indexer-key write (the main-KV format of fp4_kv_quantize applied to
 * the indexer keys: foosynaptic atlas 3.2 "FP4 main KV" and the FP4-trained
 * indexer of newsaint.id section 4).  Row i of x (bf16 [n][128], device,
 * 16-byte aligned) is quantized per 16 channels exactly as fp4_kv_quantize
 * does and written to row dst_rows[i] (int64 [n], device; NULL: row i) of
 * the two-plane FP4 indexer-K buffer idx_k (device, 16-byte aligned) of
 * cache_rows rows: codes at idx_k + row * 64, scales at
 * idx_k + cache_rows * 64 + row * 8.  Rows whose destination is negative or
 * not below cache_rows are skipped.
 * Errors: CSA2_ERR_INVALID_ARG (null pointer with n > 0, n < 0,
 *         cache_rows < 0, misalignment, n > cache_rows without dst_rows),
 *         CSA2_ERR_CUDA. */
csa2_status fp4_idx_k_quantize_scatter(const uint16_t* x, int64_t n, const int64_t* dst_rows,
                                       uint8_t* idx_k, int64_t cache_rows, void* stream);

/* Inverse of fp4_kv_quantize: y (bf16 [n][512], device) = sign * E2M1 level
 * * E4M3 scale, which bf16 holds exactly (newsaint.id section 4: FP4 values
 * are dequantized just before attention).
 * Errors: CSA2_ERR_INVALID_ARG, CSA2_ERR_CUDA. */
csa2_status fp4_kv_dequantize(const uint8_t* codes, const uint8_t* scales,
                              int64_t n, uint16_t* y, void* stream);

/* Full-mode indexer (atlas 3.2 "Hierarchical Sparse Indexer (decoder)";
 * newsaint.id section 3 and the Full branch of HierarchicalSparseIndexer in
 * section 8).  For every sequence b (ctx_len[b] = N_b, device int32 [B]):
 *   s_t  = sum_h w_h * ReLU(q_h . k_t)           for every t < N_b,
 *   bs_j = max of s_t over block j = [8j, 8j+8),
 *   pool = Top-min(P, ceil(N_b/8)) blocks by (bs desc, j asc), ascending,
 *   topk = Top-min(K, |pool positions|) pool positions by (s desc, t asc),
 *          ascending, -1 padded.
 * Scores are ranked as if computed exactly: head dots are the exact sums
 * rounded once to fp64 and the head sum is fp64 in head order; the kernels
 * use fp32 / tensor-core scores with a rigorous error bound and re-score in
 * exact arithmetic every candidate the bound cannot decide.
 *   idx_k:   device, layout above (dtype per d->idx_k_dtype)
 *   idx_q:   device, bf16 (E4M3 and FP4 keys; 16-byte aligned for FP4) or
 *            fp32 [B][Hi][Di]
 *   w:       device, fp32 [B][Hi]
 *   pool_blocks_out: device int32 [B][P], ascending, -1 padded
 *   pool_len_out:    device int32 [B]
 *   topk_out:        device int32 [B][K]
 * The indexer-K cache may hold at most 2^31 - 1 rows (B * max_ctx
 * contiguous, num_pages * 64 paged): its tiles are addressed by 32-bit row
 * coordinates.  A larger cache is CSA2_ERR_UNSUPPORTED_SHAPE.
 * Errors: CSA2_ERR_INVALID_ARG, CSA2_ERR_UNSUPPORTED_SHAPE,
 *         CSA2_ERR_WORKSPACE_TOO_SMALL, CSA2_ERR_CUDA. */
csa2_status indexer_full_topk(const csa2_dims* d, int32_t batch,
                              const void* idx_k, const int32_t* page_table,
                              const int32_t* ctx_len, const void* idx_q,
                              const float* w, int32_t* pool_blocks_out,
                              int32_t* pool_len_out, int32_t* topk_out,
                              void* ws, size_t ws_bytes, void* stream);

/* Reindex mode (atlas 3.2: re-score with this layer's indexer query over
 * the latest Full layer's main KV / indexer K; newsaint.id section 8,
 * re-indexing branch: gather the pool's keys, score only those).  Scores
 * the positions of pool_blocks[b][0 .. pool_len[b]) with (idx_q, w) and
 * writes their Top-min(K, |pool positions|), ascending, -1 padded, with the
 * same exact ranking as indexer_full_topk.  Arguments as there; pool_blocks
 * (device int32 [B][P]) and pool_len (device int32 [B]) are the Full
 * layer's outputs. */
csa2_status indexer_reindex_topk(const csa2_dims* d, int32_t batch,
                                 const void* idx_k, const int32_t* page_table,
                                 const int32_t* ctx_len, const void* idx_q,
                                 const float* w, const int32_t* pool_blocks,
                                 const int32_t* pool_len, int32_t* topk_out,
                                 void* ws, size_t ws_bytes, void* stream);

/* indexer_full_topk / indexer_reindex_topk with flags (0: the plain calls).
 * CSA2_IDX_EARLY_INPUTS: idx_k, page_table and ctx_len (and, for Reindex,
 * pool_blocks and pool_len) are not written by the operation enqueued just
 * before this call on the stream (they were written by earlier work, before
 * that operation began), so the call may start reading them -- the scan
 * streams its first key tiles -- while that operation is still running.
 * idx_q, w, the outputs and the workspace are accessed only after it has
 * finished.  In a decode step this holds for a Full layer that follows an
 * attention call or the latent append (not the indexer-key write) and for a
 * Reindex layer that follows an attention call.  Other bits:
 * CSA2_ERR_INVALID_ARG. */
#define CSA2_IDX_EARLY_INPUTS 1
csa2_status indexer_full_topk_ex(const csa2_dims* d, int32_t batch, int32_t flags,
                                 const void* idx_k, const int32_t* page_table,
                                 const int32_t* ctx_len, const void* idx_q, const float* w,
                                 int32_t* pool_blocks_out, int32_t* pool_len_out,
                                 int32_t* topk_out, void* ws, size_t ws_bytes, void* stream);
csa2_status indexer_reindex_topk_ex(const csa2_dims* d, int32_t batch, int32_t flags,
                                    const void* idx_k, const int32_t* page_table,
                                    const int32_t* ctx_len, const void* idx_q, const float* w,
                                    const int32_t* pool_blocks, const int32_t* pool_len,
                                    int32_t* topk_out, void* ws, size_t ws_bytes, void* stream);

/* Sparse MLA-style decode attention, all layer modes (atlas 3.2 mode table
 * and figure "异构 KV": main Q reads the Top-K main-KV entries and the
 * exact SWA KV, merged; Reuse keeps KV and indices and changes only Q).
 * For every sequence b and head h, over E = {valid topk[b][i]} + {SWA rows
 * 0 .. swa_len[b]):
 *   key(e) = [dq(latent) ; rope] (576), value(e) = dq(latent) (512) for main
 *   entries, the SWA row (576) / its first 512 channels for SWA entries;
 *   logit = scale * q[b][h] . key(e);  out = softmax-weighted sum of values;
 *   lse = max logit + ln(sum exp(logit - max)); empty E: out 0, lse -inf.
 *   out is the sum of the parts of up to 8 chunks of 128 entries: for few
 *   (sequence, 32-head group) pairs each chunk runs on its own SM and the
 *   parts are added in the order the chunks finish, so repeated calls can
 *   differ in the last bits of out (lse does not); for many pairs one CTA
 *   accumulates the chunks in order and out is reproducible.
 *   mode: csa2_mode.  Indices are always supplied.  CSA2_MODE_REUSE (the
 *     layer keeps the KV and indices an earlier layer used) lets the call
 *     start reading topk, ctx_len, page_table and the main-KV planes
 *     (kv_codes, kv_scales, kv_rope) while the operation enqueued just before
 *     it on the stream is still running: in this mode those buffers must not
 *     be written by that operation (they were written by earlier work on the
 *     stream, before it began).  q, swa_kv, swa_len, out and lse are always
 *     accessed only after it has finished.  CSA2_MODE_FULL and
 *     CSA2_MODE_REINDEX read nothing before it has finished.
 *   q:        device bf16 [B][H][576], 16-byte aligned
 *   kv_codes, kv_scales, kv_rope: device, layout above (16-, 2- and
 *             16-byte aligned)
 *   topk:     device int32 [B][K], -1 = padding
 *   swa_kv:   device bf16 [B][W][576];  swa_len: device int32 [B]
 *   out:      device fp32 [B][H][512];  lse: device fp32 [B][H]
 * Errors: CSA2_ERR_INVALID_ARG, CSA2_ERR_UNSUPPORTED_SHAPE,
 *         CSA2_ERR_WORKSPACE_TOO_SMALL, CSA2_ERR_CUDA. */
csa2_status csa2_sparse_attn_decode(const csa2_dims* d, int32_t batch, int32_t mode,
                                    const uint16_t* q, const uint8_t* kv_codes,
                                    const uint8_t* kv_scales, const uint16_t* kv_rope,
                                    const int32_t* page_table, const int32_t* ctx_len,
                                    const int32_t* topk, const uint16_t* swa_kv,
                                    const int32_t* swa_len, float scale, float* out,
                                    float* lse, void* ws, size_t ws_bytes, void* stream);

/* Multi-query decode attention: q_len (1 .. CSA2_MAX_QLEN) consecutive new
 * tokens per sequence, e.g. the draft tokens a speculative step verifies
 * (stamatios.com "DeepSeek-V4.1 Flash comprime cache KV para 890 bytes por
 * token", DSpark paragraph: draft blocks over the SWA-128 window; foosynaptic
 * atlas, section 3 component table, DSpark row).  The q_len tokens are the
 * newest rows of each sequence's SWA window and share the layer's Top-K set:
 * query i (0-based, oldest first) of sequence b attends to the valid topk
 * entries and to SWA rows 0 .. swa_len[b] - (q_len - 1 - i) - 1 (its own row
 * and the older ones), with the rules of csa2_sparse_attn_decode otherwise.
 * q_len == 1 is exactly csa2_sparse_attn_decode.
 *   q:   device bf16 [B][q_len][H][576], 16-byte aligned
 *   out: device fp32 [B][q_len][H][512];  lse: device fp32 [B][q_len][H]
 *   other arguments as for csa2_sparse_attn_decode (one Top-K set, one SWA
 *   window and one swa_len per sequence).
 * Limit: for q_len > 1, topk + swa <= 1024 (at most 8 chunks of 128
 * entries, merged inside one thread-block cluster); larger shapes return
 * CSA2_ERR_UNSUPPORTED_SHAPE.
 * Errors: as csa2_sparse_attn_decode; q_len outside 1 .. CSA2_MAX_QLEN is
 *         CSA2_ERR_UNSUPPORTED_SHAPE. */
#define CSA2_MAX_QLEN 4
csa2_status csa2_sparse_attn_decode_mq(const csa2_dims* d, int32_t batch, int32_t q_len, int32_t mode,
                                       const uint16_t* q, const uint8_t* kv_codes,
                                       const uint8_t* kv_scales, const uint16_t* kv_rope,
                                       const int32_t* page_table, const int32_t* ctx_len,
                                       const int32_t* topk, const uint16_t* swa_kv,
                                       const int32_t* swa_len, float scale, float* out, float* lse,
                                       void* ws, size_t ws_bytes, void* stream);

/* Allocation-free variant of csa2_sparse_attn_decode.  The pages describe
 * no counterpart of this call; it exists for callers that must not allocate
 * GPU memory on their hot path -- e.g. a plugin running inside another
 * engine's execution step, or a serving loop whose memory budget is fixed
 * before it starts -- and so cannot provide the workspace the other calls
 * take.  The split-KV scratch lives instead in a fixed device array of
 * CSA2_NOALLOC_SCRATCH_BYTES inside the library, held on every GPU that
 * loads the library until the process exits.
 *   Limit: with S = ceil((topk + swa) / 128) chunks of entries, up to 8
 *   chunks are merged inside one thread-block cluster (or accumulated by one
 *   CTA) and need only the 256-byte error word (any batch).  Above 8 chunks the per-chunk partial
 *   outputs live in the array: 256 + B*S*H*2048 + B*S*H*8 bytes (each part
 *   rounded up to 256) must fit it -- up to batch 5 at Top-2048, SWA-128,
 *   64 heads; larger shapes return CSA2_ERR_WORKSPACE_TOO_SMALL and launch
 *   nothing.
 *   Arguments and results are those of csa2_sparse_attn_decode without
 *   ws / ws_bytes; err_word (device int32, may be NULL) receives the device
 *   error bits of this call, ORed in.
 *   The first call on a device looks up the array's device address (once
 *   per device, with that device current); make that first call before any
 *   stream capture.  The call allocates nothing (no cudaMalloc / cudaFree).
 *   All calls share the one array and it keeps the last call's contents:
 *   calls whose GPU work can overlap (e.g. on unsynchronised streams) race
 *   on it and must be serialised by the caller. */
#define CSA2_NOALLOC_SCRATCH_BYTES (12u << 20)
csa2_status csa2_sparse_attn_decode_noalloc(const csa2_dims* d, int32_t batch, int32_t mode,
                                            const uint16_t* q, const uint8_t* kv_codes,
                                            const uint8_t* kv_scales, const uint16_t* kv_rope,
                                            const int32_t* page_table, const int32_t* ctx_len,
                                            const int32_t* topk, const uint16_t* swa_kv,
                                            const int32_t* swa_len, float scale, float* out,
                                            float* lse, int32_t* err_word, void* stream);

/* Rotary positions (the pages apply them to the 64 bf16 key channels and the
 * matching query channels before this library's cache and attention are
 * reached: foosynaptic atlas, section 3.2; the layouts and scalings are the
 * published ones).  Pair i of the `rot` rotated channels, i = 0 .. rot/2 - 1,
 * turns by the angle pos * f_i:
 *   (u, v) -> mscale * (u cos - v sin, u sin + v cos),   f_i = theta^(-2 i / rot)
 * with the pair's channels
 *   CSA2_ROPE_INTERLEAVED: 2 i and 2 i + 1;   CSA2_ROPE_HALF: i and rot/2 + i
 * and, for contexts longer than the original one, f_i scaled by
 *   CSA2_ROPE_LINEAR: f_i / factor (position interpolation);
 *   CSA2_ROPE_PARTS:  by the turns n_i = orig_ctx * f_i / (2 pi) that the pair makes
 *     over the original context (the by-parts rule of YaRN): with k = (n_i - turns_lo)
 *     / (turns_hi - turns_lo) limited to [0, 1], f_i * k + f_i / factor * (1 - k);
 *   CSA2_ROPE_BASE:   theta replaced by theta * factor^(rot / (rot - 2)) (rot > 2).
 * Angles are right modulo one turn for every int32 position, to 2^-31 turns. */
typedef enum { CSA2_ROPE_INTERLEAVED = 0, CSA2_ROPE_HALF = 1 } csa2_rope_layout;
typedef enum {
  CSA2_ROPE_PLAIN = 0,
  CSA2_ROPE_LINEAR = 1,
  CSA2_ROPE_PARTS = 2,
  CSA2_ROPE_BASE = 3
} csa2_rope_scaling;
typedef struct {
  int32_t rot;        /* rotated channels, even, 2..256                        */
  int32_t layout;     /* csa2_rope_layout                                      */
  int32_t scaling;    /* csa2_rope_scaling                                     */
  float mscale;       /* multiplies cosine and sine (1: a rotation), finite    */
  double theta;       /* base, > 1                                             */
  double factor;      /* context factor, >= 1 (not PLAIN)                      */
  double orig_ctx;    /* original context, > 0 (PARTS)                         */
  double turns_lo;    /* >= 0 (PARTS; usually 1)                               */
  double turns_hi;    /* > turns_lo (PARTS; usually 32)                        */
} csa2_rope;

/* y = rotary(x) on channels [offset, offset + rot) of every head; the other
 * channels are copied, or left alone when y == x (in place, equal strides).
 *   dtype:  CSA2_ROPE_BF16 or CSA2_ROPE_F32, of x and y (device)
 *   pos:    device int32 [tokens]: the position of each token (any value)
 *   x[t][h][c] at x + t * x_token + h * x_head + c (strides in elements; x may
 *   repeat rows with stride 0); y likewise, without overlap of its rows.
 *   inverse: 0, or 1 for the transpose mscale * R(-angle): the gradient with
 *     respect to x of a forward call, applied to the gradient of y.
 * x and y must be the same buffer with the same strides, or blocks (first to last
 * element) that do not overlap.
 * Errors: CSA2_ERR_INVALID_ARG (also: y's rows overlap), CSA2_ERR_UNSUPPORTED_SHAPE
 * (rot outside 2..256 or odd, offset + rot > dim, sizes below 0, more than 2^31
 * positions, heads > 65535, heads * dim > 2^27), CSA2_ERR_CUDA.  The same values give
 * the same bits whatever the strides and the alignment. */
#define CSA2_ROPE_BF16 0
#define CSA2_ROPE_F32 1
csa2_status csa2_rope_apply(const csa2_rope* r, int32_t dtype, const void* x, void* y, const int32_t* pos,
                            int64_t tokens, int32_t heads, int32_t dim, int32_t offset, int64_t x_token,
                            int64_t x_head, int64_t y_token, int64_t y_head, int32_t inverse, void* stream);

/* Cache append from a layer's projection: row i of x (bf16, x + i * x_stride, 576
 * channels: 512 latent, then 64 rotary) is normed, rotated, quantized and written
 * to cache row dst_rows[i] in one pass:
 *   latent = bf16(x w / sqrt(mean(x^2) + eps)), rounded once from the exact value
 *            (x itself when norm_w is NULL); in a row that holds an infinity or a NaN
 *            the square root is infinite or NaN: 0 or NaN throughout;
 *   codes, scales of the latent exactly as fp4_kv_quantize forms them;
 *   rope   = bf16(rotary(x[512..575], pos[i])) with r (r->rot must be 64).
 * A row whose destination is negative or not below cache_rows writes no cache row.
 * Destinations must differ from each other (of two rows with the same one, which
 * bytes of which row remain is not specified).
 *   norm_w:   device bf16 [512] of magnitudes below 2^127, or NULL;  0 < eps <= 1
 *   pos:      device int32 [n];  dst_rows: device int64 [n]
 *   codes, scales, rope: the cache planes (layout above; 16-, 2- and 16-byte aligned)
 *   entry:    device bf16 [n][576], or NULL: also receives every row i as
 *             [latent ; rope] in bf16 (an SWA window row), whatever dst_rows[i] is;
 *             no part of it within x
 *   x: 16-byte aligned, x_stride a multiple of 8, at least 576 for n > 1
 * Errors: CSA2_ERR_INVALID_ARG, CSA2_ERR_UNSUPPORTED_SHAPE (rot != 64), CSA2_ERR_CUDA. */
csa2_status csa2_kv_append(const csa2_rope* r, const uint16_t* x, int64_t n, int64_t x_stride,
                           const uint16_t* norm_w, float eps, const int32_t* pos, const int64_t* dst_rows,
                           uint8_t* codes, uint8_t* scales, uint16_t* rope, int64_t cache_rows, uint16_t* entry,
                           void* stream);

/* Dense attention of a chunk of new tokens over the main-KV cache: every visible
 * position of the cache takes part (no Top-K set, no separate window; the new
 * tokens' own rows have been appended before).  The queries of `batch` sequences
 * are packed: sequence b owns tokens q_start[b] .. q_start[b + 1] of q.  Its token i
 * (0-based, of n) stands at position ctx_len[b] - n + i and sees
 *   the positions 0 .. ctx_len[b] - n + i (causal; with window > 0 only the last
 *   `window` of them), or, with CSA2_DENSE_ALL_POSITIONS, 0 .. ctx_len[b] - 1.
 * For each of its heads h:
 *   logit_t = scale * q . [dq(latent_t) ; rope_t],  out = sum_t softmax(logit)_t dq(latent_t),
 *   lse = ln sum_t exp(logit_t);  a token that sees nothing: out 0, lse -inf.
 * Any number of tokens per sequence, none included: one (a decode step), a few
 * (drafts), a prompt's chunk, a whole prompt.  Tokens of q before q_start[0] or
 * from q_start[batch] on are not touched.  Results do not change from call to call.
 * An infinity or a NaN at a position (rope keys, a NaN scale) or in a query reaches only
 * the outputs of the tokens that see that position, or of that token and head.
 *   Dimensions read: heads, max_ctx, max_pages, num_pages (the others must be valid
 *   only for the calls that use them).
 *   q:        device bf16 [total_q][H][576], 16-byte aligned
 *   q_start:  device int32 [batch + 1], not decreasing, within 0 .. total_q
 *   kv_codes, kv_scales, kv_rope, page_table, ctx_len: as csa2_sparse_attn_decode, all
 *             three planes 16-byte aligned;
 *             a block of positions whose page id is out of range is skipped and reported
 *   out:      device bf16 [total_q][H][512], 16-byte aligned;  lse: device fp32 [total_q][H]
 *   ws:       workspace of csa2_dense_attn_workspace_size(d, batch, total_q) bytes, its
 *             first 256 the error word as elsewhere.  Calls that may run at the same
 *             time need a workspace each.
 *   P is rounded to fp16 (2^-11) and the output to bf16; everything between is fp32.
 *   The product of a row of q, scaled by the power of two that brings its largest value
 *   to 2^14, with a key has to stay within fp32 (rope keys below 2^100 do).
 * A CSA2 layer with a window (dims.swa > 0) joins the FP4 entries with exact bf16 rows in
 * one softmax (csa2_sparse_attn_decode); this call has no such operand and reads FP4 rows
 * alone, as that one does with swa 0 and every position in its Top-K set.
 * Limits: total_q * H <= 2^30, batch <= 2^20, cache rows (batch * max_ctx, or num_pages *
 * 64) < 2^31.
 * Make the first call on a device before any stream capture.
 * Errors: CSA2_ERR_INVALID_ARG (window < 0, window with CSA2_DENSE_ALL_POSITIONS,
 *         unknown flags, pointers, a scale that is not finite), CSA2_ERR_UNSUPPORTED_SHAPE,
 *         CSA2_ERR_WORKSPACE_TOO_SMALL, CSA2_ERR_CUDA. */
#define CSA2_DENSE_ALL_POSITIONS 1
csa2_status csa2_dense_attn_workspace_size(const csa2_dims* d, int32_t batch, int64_t total_q, size_t* bytes);
csa2_status csa2_dense_attn_chunk(const csa2_dims* d, int32_t batch, int64_t total_q, const uint16_t* q,
                                  const int32_t* q_start, const uint8_t* kv_codes, const uint8_t* kv_scales,
                                  const uint16_t* kv_rope, const int32_t* page_table, const int32_t* ctx_len,
                                  float scale, int32_t window, int32_t flags, uint16_t* out, float* lse, void* ws,
                                  size_t ws_bytes, void* stream);

/* Kernel timing, a tracing aid.  While enabled, the library brackets every
 * kernel it launches with a pair of CUDA events on the launching stream
 * (not for use during stream capture).  Enabling (or disabling) clears the
 * records.  csa2_profile_read waits for the recorded events and returns per
 * kernel name the number of launches and their summed milliseconds in
 * out[0 .. min(*n_entries, max_entries)), *n_entries = number of kernels. */
typedef struct {
  char name[32];
  int32_t launches;
  double total_ms;
} csa2_kernel_time;
csa2_status csa2_profile_enable(int32_t on);
csa2_status csa2_profile_read(csa2_kernel_time* out, int32_t max_entries, int32_t* n_entries);

/* Copies the device error word of `ws` to *word (synchronising `stream`)
 * and returns CSA2_OK if it is zero, CSA2_ERR_DEVICE_ASSERT otherwise. */
csa2_status csa2_get_device_status(const void* ws, void* stream, int32_t* word);

/* Zeroes the device error word of `ws` (enqueued on `stream`). */
csa2_status csa2_clear_device_status(void* ws, void* stream);

/* Self-test of the device timeout path.  Enqueues one small kernel whose
 * thread waits, with the bounded mbarrier wait every library kernel uses, on
 * an mbarrier that nothing arrives at; after limit_us microseconds
 * (1 .. 1,000,000) the wait gives up, CSA2_DEV_TIMEOUT is set in the error
 * word of ws (device, 256-byte aligned, ws_bytes >= 256) and the kernel
 * returns: no fault, no trap, the context stays usable.
 * Errors: CSA2_ERR_INVALID_ARG, CSA2_ERR_CUDA. */
csa2_status csa2_selftest_wait_timeout(void* ws, size_t ws_bytes, uint32_t limit_us, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CSA2_H */
