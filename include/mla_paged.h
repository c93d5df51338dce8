/*
 * mla_paged.h -- C ABI of the GB300 (sm_103a) paged Multi-head Latent Attention library.
 *
 * What the calls compute (flashinfer-bench "MLA Paged", sections "decode" and
 * "prefill"): for every query row r and query head h,
 *
 *   s_t      = sm_scale * (q_nope[r,h,:] . ckv[t,:] + q_pe[r,h,:] . kpe[t,:])
 *   lse[r,h] = log(sum_t exp(s_t))                       (natural log)
 *   out[r,h] = sum_t exp(s_t - lse[r,h]) * ckv[t,:]      (V is the 512-wide latent itself,
 *                                                         Modular MAX "mla_decoding_single_batch")
 *
 * where t runs over the key slots kv_indices[kv_indptr[b] .. kv_indptr[b+1]) of the
 * row's request b (decode), or over the first kv_len_b - q_len_b + i + 1 of them for
 * query i of request b (prefill: causal, bottom-right aligned).  One KV head is shared
 * by all query heads.
 *
 * Conventions shared by every call:
 *  - All tensor pointers are DEVICE pointers to contiguous row-major arrays; the
 *    caller owns every buffer (inputs, outputs, workspace).  The library allocates
 *    nothing on the device and keeps only a host-side cache of TMA descriptors keyed
 *    by pointer and shape.
 *  - bf16 tensors (q_nope, q_pe, ckv_cache, kpe_cache, out) must start on a 16-byte
 *    boundary (TMA requirement) or the call returns MLA_ERR_ALIGN.
 *  - kv_indices holds token slots: slot = page * page_size + offset, an index into the
 *    caches viewed as [num_pages * page_size, 512] and [.., 64] (the physical-index
 *    mapping of FlashMLA's abs_indices2indices_in_kvcache).  kv_indptr counts keys, so
 *    a request's kv length is kv_indptr[b+1] - kv_indptr[b].
 *  - Calls only enqueue work on `stream` (a cudaStream_t; NULL = legacy default
 *    stream).  They never synchronise and never read device memory on the host, so
 *    they may be captured in a CUDA graph.  Launch errors are returned; faults
 *    inside a kernel surface at the caller's next synchronisation.
 *  - Slots outside kv_indices are never read into the result: NaN or Inf there does
 *    not change the output.  An index outside [0, num_pages*page_size) is skipped (it
 *    is not a key of the row) instead of faulting; MLA_VALIDATE reports it.
 *  - A request with no keys gets out = 0 and lse = -inf.
 */
#ifndef MLA_PAGED_H
#define MLA_PAGED_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes (0 = success, negative = error). */
enum mla_status {
  MLA_OK = 0,
  MLA_ERR_NULL = -1,       /* a required pointer is NULL                                  */
  MLA_ERR_DIMS = -2,       /* head dims != 512/64, heads not in 1..128, bad sizes          */
  MLA_ERR_ALIGN = -3,      /* a bf16 tensor pointer is not 16-byte aligned                 */
  MLA_ERR_WORKSPACE = -4,  /* workspace NULL or smaller than mla_workspace_bytes()         */
  MLA_ERR_LAUNCH = -5,     /* a kernel launch failed (cudaGetLastError after the launch)   */
  MLA_ERR_BAD_INDEX = -6,  /* (device status) MLA_VALIDATE found bad indptr/indices        */
  MLA_ERR_TIMEOUT = -7,    /* (device status) a bounded wait inside a kernel gave up       */
  MLA_ERR_CUDA = -8,       /* a CUDA runtime/driver call failed (device query, TMA encode) */
  MLA_ERR_UNSUPPORTED = -9, /* no sm_103a-class device is current                          */
  MLA_ERR_INTERNAL = -10,  /* (device status) a kernel found an internal invariant broken  */
  MLA_ERR_NO_PAGES = -11   /* (result of a pool entry) the pool has too few free pages      */
};

/* Flags (bitwise OR). */
enum mla_flags {
  MLA_VALIDATE = 1 /* run an index-validation kernel first; it records MLA_ERR_BAD_INDEX in
                      the workspace status word (read it with mla_read_device_status) */
};

/* Problem sizes.  All fields are host-side values. */
typedef struct mla_dims {
  int32_t batch;          /* decode: number of requests (= query rows); prefill: requests   */
  int32_t num_qo_heads;   /* query heads, 1..128 (one shared KV head)                       */
  int32_t head_dim_ckv;   /* must be 512                                                     */
  int32_t head_dim_kpe;   /* must be 64                                                      */
  int32_t num_pages;      /* pages in ckv_cache / kpe_cache                                  */
  int32_t page_size;      /* slots per page (>= 1); num_pages * page_size < 2^31             */
  int32_t total_q;        /* prefill: qo_indptr[batch] (query rows); decode: ignored         */
  int32_t num_kv_indices; /* kv_indptr[batch]: length of kv_indices                          */
  int32_t num_workers;    /* split-KV workers (CTA pairs); 0 = one per SM pair of the device */
} mla_dims;

/*
 * Paged MLA decode: flashinfer-bench "MLA Paged", section "decode".
 *   q_nope     [batch, H, 512] bf16      q_pe      [batch, H, 64] bf16
 *   ckv_cache  [num_pages, page_size, 512] bf16
 *   kpe_cache  [num_pages, page_size, 64]  bf16
 *   kv_indptr  [batch + 1] int32 (non-decreasing, kv_indptr[0] = 0)
 *   kv_indices [num_kv_indices] int32 token slots
 *   sm_scale   softmax scale multiplying the q.k dot product
 *   out        [batch, H, 512] bf16 (written)   lse [batch, H] fp32, natural log (written)
 *   workspace  device scratch of at least mla_workspace_bytes(dims, 0) bytes, caller-owned;
 *              it holds split-KV partial results, merge counters and the device status
 *              word.  Zero-fill it once before its first use (the status word, its first
 *              4 bytes, only accumulates error bits until mla_read_device_status clears
 *              it); everything else is rewritten by every call, so one workspace may serve
 *              calls with different sizes, worker counts or head counts.  Calls that share
 *              a workspace must not overlap on the GPU.
 *   flags      MLA_VALIDATE or 0;  stream: cudaStream_t
 * Returns MLA_OK or a negative mla_status; nothing is launched on an argument error.
 */
int mla_paged_decode(const void* q_nope, const void* q_pe, const void* ckv_cache,
                     const void* kpe_cache, const int32_t* kv_indptr, const int32_t* kv_indices,
                     float sm_scale, void* out, float* lse, const mla_dims* dims,
                     void* workspace, size_t workspace_bytes, int flags, void* stream);

/*
 * Paged MLA causal prefill: flashinfer-bench "MLA Paged", section "prefill"; the
 * causal mask is bottom-right aligned: query i of request b sees its first
 * kv_len_b - q_len_b + i + 1 keys (kv_len_b >= q_len_b is required; rows that
 * would see no key get out = 0, lse = -inf, and MLA_VALIDATE flags them).
 *   q_nope [total_q, H, 512], q_pe [total_q, H, 64], out [total_q, H, 512], lse [total_q, H]
 *   qo_indptr [batch + 1] int32 query offsets (qo_indptr[batch] = total_q)
 *   other arguments as for mla_paged_decode; workspace >= mla_workspace_bytes(dims, 1).
 */
int mla_paged_prefill(const void* q_nope, const void* q_pe, const void* ckv_cache,
                      const void* kpe_cache, const int32_t* qo_indptr, const int32_t* kv_indptr,
                      const int32_t* kv_indices, float sm_scale, void* out, float* lse,
                      const mla_dims* dims, void* workspace, size_t workspace_bytes, int flags,
                      void* stream);

/*
 * Packed multi-token decode (speculative / MTP decode): every request has the same
 * number q_len >= 1 of new query tokens, causal within the request: token i of request
 * b sees the first kv_len_b - q_len + i + 1 of its keys (kv_len_b >= q_len is required;
 * MLA_VALIDATE flags shorter requests).  This is the fixed-Q form of the packed-query
 * decode in flashinfer's prims_ts wrapper (batch_mla_decode_with_paged_kv_cache,
 * parameters qo_indptr / max_seq_len_q, mask_type "causal"), and FlashMLA's
 * flash_mla_with_kvcache with seq_len_q > 1: the q_len tokens of a request share each
 * KV tile, q_len * H rows per tile.
 *   q_nope [batch, q_len, H, 512], q_pe [batch, q_len, H, 64] bf16
 *   out    [batch, q_len, H, 512] bf16, lse [batch, q_len, H] fp32 (natural log)
 *   q_len * num_qo_heads must be <= 128 (else MLA_ERR_DIMS; use mla_paged_prefill with
 *   qo_indptr for more rows per request).
 *   workspace >= mla_workspace_bytes_mtp(dims, q_len); other arguments as for
 *   mla_paged_decode (dims->total_q is ignored).
 */
int mla_paged_decode_mtp(const void* q_nope, const void* q_pe, const void* ckv_cache,
                         const void* kpe_cache, const int32_t* kv_indptr, const int32_t* kv_indices,
                         float sm_scale, void* out, float* lse, const mla_dims* dims, int q_len,
                         void* workspace, size_t workspace_bytes, int flags, void* stream);

/*
 * Sparse (top-k) paged MLA decode: FlashMLA notes, "flash_mla_with_kvcache (Sparse
 * Attention with FP8 KV Cache)" and "Sparse Attention Decoding with KV Cache" (bf16
 * caches here).  Every query row attends only to the token slots listed for it, with no
 * causal mask.
 *   q_nope [rows, H, 512], q_pe [rows, H, 64] bf16: one row per (request, query token),
 *          e.g. [batch, s_q, H, 512] viewed as [batch * s_q, H, 512]
 *   indices [rows, topk] int32 token slots (slot = page * page_size + offset); an entry
 *          that is negative or >= num_pages * page_size is padding and is skipped; a
 *          row without a valid entry gets out = 0, lse = -inf
 *   out [rows, H, 512] bf16, lse [rows, H] fp32 (natural log)
 *   dims->batch = rows; dims->num_kv_indices is ignored (rows * topk); other fields as
 *   for mla_paged_decode; workspace >= mla_workspace_bytes(dims, 0).  MLA_VALIDATE
 *   checks nothing here (any index may be padding).
 */
int mla_paged_decode_sparse(const void* q_nope, const void* q_pe, const void* ckv_cache,
                            const void* kpe_cache, const int32_t* indices, int topk, float sm_scale,
                            void* out, float* lse, const mla_dims* dims, void* workspace,
                            size_t workspace_bytes, int flags, void* stream);

/*
 * Paged MLA decode over an FP8 KV cache (FlashMLA notes, "FP8 KV Cache Quantization
 * and Dequantization", layout V32_FP8Sparse; "flash_mla_with_kvcache" with
 * is_fp8_kvcache).  kv_fp8 [num_pages * page_size][656] bytes, 16-byte aligned: per
 * token, bytes 0-511 the 512 latent values as E4M3, bytes 512-527 four float32 scales
 * (one per 128 latent values), bytes 528-655 the 64 rope values as bf16.  Latent value
 * i of a token is read as bf16(float32(e4m3_i) * scale[i / 128]) (product in float32,
 * both roundings to nearest even), the BF16 that the page's dequantisation returns;
 * the attention is then exactly mla_paged_decode's over those values.  Other arguments
 * as for mla_paged_decode (same workspace size).  MLA_ERR_ALIGN if kv_fp8 is not
 * 16-byte aligned.  Codes 0x7F / 0xFF (E4M3 NaN) propagate as NaN.
 */
int mla_paged_decode_fp8(const void* q_nope, const void* q_pe, const void* kv_fp8, const int32_t* kv_indptr,
                         const int32_t* kv_indices, float sm_scale, void* out, float* lse, const mla_dims* dims,
                         void* workspace, size_t workspace_bytes, int flags, void* stream);

/*
 * Sparse (top-k) decode over an FP8 KV cache (FlashMLA notes, "flash_mla_with_kvcache
 * (Sparse Attention with FP8 KV Cache)"): mla_paged_decode_sparse's arguments with the
 * cache of mla_paged_decode_fp8.
 */
int mla_paged_decode_sparse_fp8(const void* q_nope, const void* q_pe, const void* kv_fp8, const int32_t* indices,
                                int topk, float sm_scale, void* out, float* lse, const mla_dims* dims,
                                void* workspace, size_t workspace_bytes, int flags, void* stream);

/*
 * Block-table adapter.  The prims_ts wrapper ("batch_mla_decode_with_paged_kv_cache":
 * block_tables [batch, max_num_blocks], seq_lens) and FlashMLA's flash_mla_with_kvcache
 * (block_table, cache_seqlens) name a request's keys as the first seq_len slots of its
 * pages, in block-table order.  This writes the token-slot CSR the decode calls take:
 *   len_b = clamp(seq_lens[b], 0, max_blocks * page_size)
 *   kv_indptr[b] = len_0 + ... + len_{b-1}  (kv_indptr[batch] = the total)
 *   kv_indices[kv_indptr[b] + k] = block_table[b * max_blocks + k / page_size] * page_size
 *                                  + k % page_size
 *   block_table [batch, max_blocks] int32 page ids (row-major; entries past a request's
 *               last needed block are not read), seq_lens [batch] int32
 *   kv_indptr [batch + 1] int32 (written), kv_indices [capacity] int32 (written)
 * A slot that is negative or does not fit in int32 is written as -1, and any slot
 * outside the cache is skipped by the decode (not a key).  Positions at or past
 * `capacity` are not written (kv_indptr still counts them; pass capacity as
 * num_kv_indices and the decode reads no further).  batch * max_blocks * page_size is
 * always enough.  Two kernel launches on `stream`, no synchronisation; graph-capturable.
 * Returns MLA_ERR_DIMS (negative sizes, page_size < 1, max_blocks * page_size or
 * capacity above INT32_MAX), MLA_ERR_NULL, MLA_ERR_LAUNCH, or MLA_OK.
 */
int mla_block_table_to_csr(const int32_t* block_table, const int32_t* seq_lens, int batch, int max_blocks,
                           int page_size, int32_t* kv_indptr, int32_t* kv_indices, long long capacity,
                           void* stream);

/*
 * Paged MLA decode from a block table: mla_block_table_to_csr into the workspace, then
 * mla_paged_decode on that CSR, on `stream`.  Arguments as for mla_paged_decode, with
 * block_table [batch, max_blocks] and seq_lens [batch] in place of kv_indptr and
 * kv_indices; dims->num_kv_indices is ignored (the CSR's capacity,
 * batch * max_blocks * page_size, is used and must fit int32, else MLA_ERR_DIMS).
 * workspace >= mla_workspace_bytes_block_table(dims, max_blocks) bytes, zero-filled
 * before first use like the decode's; flags must be 0 (MLA_ERR_DIMS otherwise: the
 * CSR ends short of its capacity, which MLA_VALIDATE would report).
 */
size_t mla_workspace_bytes_block_table(const mla_dims* dims, int max_blocks);
int mla_paged_decode_block_table(const void* q_nope, const void* q_pe, const void* ckv_cache,
                                 const void* kpe_cache, const int32_t* block_table, const int32_t* seq_lens,
                                 int max_blocks, float sm_scale, void* out, float* lse, const mla_dims* dims,
                                 void* workspace, size_t workspace_bytes, int flags, void* stream);

/*
 * Paged MLA decode for callers that cannot allocate device memory (a plugin that runs
 * inside another framework's memory pool, code that must not call cudaMalloc after
 * start-up, or a context where an allocation would synchronise the device).  This entry
 * point has no counterpart in the pages the library follows; it computes exactly what
 * mla_paged_decode computes, with the same arguments except the workspace.
 *
 * The split-KV scratch lives in one static device array of 32 MiB inside the library,
 * held by every GPU that loads the library until the process exits.  With
 * dims->num_workers == 0 the call uses one worker per SM pair, or fewer if their
 * partial results would not fit in the 32 MiB; an explicit num_workers whose scratch
 * needs more returns MLA_ERR_WORKSPACE.  flags must be 0 (the device status word is not
 * read through the status call below instead), else MLA_ERR_DIMS.  All calls share the
 * array and it keeps the last call's contents: calls that overlap on the GPU race.
 * Nothing else carries over between calls (each call clears the status word and zeroes
 * the merge counters it uses).  The first call on each device looks up the array's
 * address (with that device current); make it before any stream capture.  The call
 * itself allocates nothing.
 */
int mla_paged_decode_noalloc(const void* q_nope, const void* q_pe, const void* ckv_cache,
                             const void* kpe_cache, const int32_t* kv_indptr, const int32_t* kv_indices,
                             float sm_scale, void* out, float* lse, const mla_dims* dims, int flags,
                             void* stream);

/* Device status of the most recent mla_paged_decode_noalloc call on the current device:
 * synchronises `stream`, reads and clears the status word in the library's static
 * scratch and returns MLA_OK, MLA_ERR_TIMEOUT or MLA_ERR_INTERNAL (as
 * mla_read_device_status does for a caller's workspace).  No counterpart on the pages. */
int mla_noalloc_read_status(void* stream);

/*
 * Causal prefill of a chunk of new tokens with staged keys: mla_paged_prefill's arguments,
 * mask and definition (the results differ in rounding).  The call first copies the keys it
 * needs into its workspace, so every page size and slot order runs at the same rate, and
 * attends in blocks of 128 (token, head) rows, so few heads cost no more than many: on four
 * prompts with 128 heads and bf16 caches it takes half of mla_paged_prefill's time.  (For a
 * token or a few per request over bf16 caches the decode calls, which read every key once,
 * are faster.)  Chunks
 * may be ragged, down to one token or none per request; rows that see no key get out = 0,
 * lse = -inf.  dims->total_q may be larger than qo_indptr[batch], and num_kv_indices than
 * kv_indptr[batch]: the rows behind the last request are left as they were.  (MLA_VALIDATE
 * reports both, as for mla_paged_prefill.)  A listed slot outside the cache is not a key.
 * A key that holds a value that is not finite makes out and lse NaN in the rows that see
 * it and changes no other row.  (mla_paged_prefill lets such a value run through its
 * arithmetic: in the rows that see it some columns of out, and lse, may stay finite.)
 *   workspace >= mla_workspace_bytes_prefill_staged(dims) bytes, zero-filled before its first
 *   use; it holds the staged keys (1152 bytes for each of dims->num_kv_indices, plus up to
 *   128 keys per request) and two fragments of 256 KB (513 KB with their lse) per worker.  Calls whose staged keys
 *   number 2^31 or more are refused (MLA_ERR_DIMS; their workspace size reads 0).
 * mla_paged_prefill_fp8 is the same over the FP8 cache of mla_paged_decode_fp8 (every latent
 * value read as the same BF16 number), with the same workspace size.
 */
size_t mla_workspace_bytes_prefill_staged(const mla_dims* dims);
int mla_paged_prefill_staged(const void* q_nope, const void* q_pe, const void* ckv_cache, const void* kpe_cache,
                             const int32_t* qo_indptr, const int32_t* kv_indptr, const int32_t* kv_indices,
                             float sm_scale, void* out, float* lse, const mla_dims* dims, void* workspace,
                             size_t workspace_bytes, int flags, void* stream);
size_t mla_workspace_bytes_prefill_fp8(const mla_dims* dims);
int mla_paged_prefill_fp8(const void* q_nope, const void* q_pe, const void* kv_fp8, const int32_t* qo_indptr,
                          const int32_t* kv_indptr, const int32_t* kv_indices, float sm_scale, void* out,
                          float* lse, const mla_dims* dims, void* workspace, size_t workspace_bytes, int flags,
                          void* stream);

/*
 * Rotary positions and the cache write, for the new tokens of a step.  With 32 pairs of
 * elements (interleaved: elements 2i and 2i + 1; else elements i and i + 32) and
 * angle = positions[axis(i)][t] * inv_freq[i], pair (a, b) of every query head of token t
 * and of its key becomes (a cos - b sin, a sin + b cos), computed in float32 and rounded to
 * bf16 once; angles keep their precision at any int32 position.  Pairs 0 .. section[0] - 1
 * follow axis 0, the next section[1] axis 1, the rest axis 2 (text: one axis; images and
 * video: time, height, width).
 *   q_pe  [tokens, H, 64] bf16 with strides (H may be 0: no queries, q_pe and q_out unused)
 *   ckv   [tokens, 512] bf16 latents, written as they are;  k_pe [tokens, 64] bf16, rotated
 *   positions [num_axes, tokens] int32;  inv_freq [32] float32 (device)
 *   slots [tokens] int32 token slots; a token whose slot is outside the cache is not
 *         written (its query is rotated all the same).  Slots named by several tokens end
 *         up with a mixture of those tokens' values: name a slot once.
 *   q_out [tokens, H, 64] bf16, contiguous; may be q_pe itself if q_pe is contiguous
 *         (MLA_ERR_DIMS otherwise), and must not overlap it in any other way
 * Strides are in elements and multiples of 8; all tensor pointers 16-byte aligned
 * (MLA_ERR_ALIGN).  MLA_ERR_DIMS if the sections do not add up to 32 pairs over num_axes
 * axes.  One launch.
 *
 * The _fp8 form writes the 656-byte token of mla_paged_decode_fp8: per 128 latent values
 * scale = amax / 448 over the finite ones (1 for a tile of zeros) and the E4M3 number
 * nearest to the float32 quotient value / scale; a value that is not finite is written
 * as E4M3's NaN.  The rope part stays bf16.
 */
typedef struct mla_rope_dims {
  int32_t tokens;
  int32_t num_qo_heads;  /* 0..128 */
  int32_t num_axes;      /* 1..3 */
  int32_t section[3];    /* pairs of each axis; the used ones sum to 32 */
  int32_t interleaved;   /* 1: pairs (2i, 2i + 1); 0: pairs (i, i + 32) */
  int32_t num_pages;
  int32_t page_size;
  int64_t q_stride_token, q_stride_head; /* elements */
  int64_t ckv_stride, kpe_stride;        /* elements between tokens */
} mla_rope_dims;

int mla_rope_append(const void* q_pe, const void* ckv, const void* k_pe, const int32_t* positions,
                    const float* inv_freq, const int32_t* slots, void* q_out, void* ckv_cache, void* kpe_cache,
                    const mla_rope_dims* dims, void* stream);
int mla_rope_append_fp8(const void* q_pe, const void* ckv, const void* k_pe, const int32_t* positions,
                        const float* inv_freq, const int32_t* slots, void* q_out, void* kv_fp8,
                        const mla_rope_dims* dims, void* stream);

/*
 * Cached tokens as contiguous bf16 rows: row i of ckv_out [n, 512] and kpe_out [n, 64] is
 * the token in slots[i] (FP8: dequantised as mla_paged_decode_fp8 reads it); zeros where
 * slots[i] is outside the cache.  count: optional device scalar (for instance
 * kv_indptr + batch); rows at or past it are left as they were.  One launch.
 */
int mla_cache_gather(const void* ckv_cache, const void* kpe_cache, const int32_t* slots, int n,
                     const int32_t* count, int num_pages, int page_size, void* ckv_out, void* kpe_out,
                     void* stream);
int mla_cache_gather_fp8(const void* kv_fp8, const int32_t* slots, int n, const int32_t* count, int num_pages,
                         int page_size, void* ckv_out, void* kpe_out, void* stream);

/*
 * Page copies within a cache: for e < n the first tokens[e] slots (tokens NULL: the whole
 * page) of page src[e] are copied to page dst[e].  An entry with a page outside the cache
 * (the pool's lists are padded with -1) copies nothing.  count: optional device scalar;
 * entries at or past it are not read.  No page may be the dst of two entries, or the dst
 * of one and the src of another (the pool's lists never have that; such pages end up with
 * a mixture).  Run it once for every layer's cache.  One launch.
 */
int mla_cache_copy_pages(void* ckv_cache, void* kpe_cache, const int32_t* src, const int32_t* dst,
                         const int32_t* tokens, int n, const int32_t* count, int num_pages, int page_size,
                         void* stream);
int mla_cache_copy_pages_fp8(void* kv_fp8, const int32_t* src, const int32_t* dst, const int32_t* tokens, int n,
                             const int32_t* count, int num_pages, int page_size, void* stream);

/*
 * The page pool: which pages belong to which sequence.  Three device arrays of the caller:
 *   block_table [max_rows, max_blocks] int32 page ids in sequence order
 *   seq_lens    [max_rows] int32 (0: an empty row)
 *   ref_count   [num_pages] int32: how many rows hold the page; 0 = free
 * A row's entries past its last page in use are neither read nor changed.  A new pool has
 * seq_lens and ref_count zero.  A caller may hold pages of its own (a prefix kept for later)
 * by adding to their ref_count.  A row's length changes through these calls only (a length
 * lowered by hand would leave the pages behind it counted).  The arrays are what
 * mla_block_table_to_csr and mla_paged_decode_block_table take.  The calls are deterministic: pages are taken lowest
 * id first in the order of the entries.
 *
 * mla_pages_extend: row rows[i] grows by new_tokens[i] >= 0 tokens.
 *   results [n]: MLA_OK; MLA_ERR_BAD_INDEX (nothing changes) if the row is out of range or
 *     named by an earlier entry, the count negative, the new length over max_blocks *
 *     page_size, or the row's last, partly filled page held by anyone else too;
 *     MLA_ERR_NO_PAGES (nothing changes) if the entry needs pages and the free pages do not
 *     cover it together with all earlier valid entries
 *   new_indptr [n + 1]: offsets of the granted tokens (refused entries add none), packed in
 *     list order (the qo_indptr of a prefill).  Behind a refused entry the offsets are not
 *     those of the requested counts: inputs that were packed by the requested counts have to
 *     be repacked by new_indptr before they are written to the slots or attended
 *   slots [capacity]: their token slots (the slots of mla_rope_append); positions past
 *     the last granted token get -1, tokens past the capacity are counted but not written
 * mla_pages_fork: row children[i] (empty) becomes a copy of row parents[i]: full pages are
 *   shared (ref_count + 1), a partly filled last page gets a page of its own, whose first
 *   copy_tokens[i] slots are to be copied from page src[i] to dst[i] by
 *   mla_cache_copy_pages for every cache (-1, -1, 0 where nothing is to be copied).
 *   results [n]: as above; MLA_ERR_BAD_INDEX also for a child that is not empty, is its own
 *   parent or is named by an earlier entry.  Lengths are read as they were before the call.
 * mla_pages_free: rows[i] gives up its pages (ref_count - 1; its entries become -1) and is
 *   empty.  Rows that are empty, out of range or listed twice are no error.  ref_count
 *   never goes below 0.
 * mla_pages_compact: with L live pages, the live pages with ids >= L move, in id order, to
 *   the free ids < L, ascending; block_table and ref_count are updated.
 *   counts [2]: L and the number of moves; src, dst [num_pages / 2]: the moves, for
 *   mla_cache_copy_pages (and for renaming page ids kept elsewhere), padded with -1.
 *
 * n entries, all arrays int32 on the device, outputs as described.  workspace >=
 * mla_workspace_bytes_pages(pool, n) bytes (compact: n = 0), 16-byte aligned; nothing in
 * it carries over between calls, and its first 256 bytes are left as they are, so it may be
 * the workspace of an attention call, whose status word stays what it was.  Calls on the
 * same pool or workspace must be ordered.
 * MLA_ERR_DIMS: negative sizes, page_size < 1, max_blocks * page_size or num_pages *
 * page_size over INT32_MAX.
 */
typedef struct mla_pool {
  int32_t* block_table;
  int32_t* seq_lens;
  int32_t* ref_count;
  int32_t max_rows;
  int32_t max_blocks;
  int32_t num_pages;
  int32_t page_size;
} mla_pool;

size_t mla_workspace_bytes_pages(const mla_pool* pool, int n);
int mla_pages_extend(const mla_pool* pool, const int32_t* rows, const int32_t* new_tokens, int n,
                     int32_t* new_indptr, int32_t* slots, long long capacity, int32_t* results, void* workspace,
                     size_t workspace_bytes, void* stream);
int mla_pages_fork(const mla_pool* pool, const int32_t* parents, const int32_t* children, int n, int32_t* src,
                   int32_t* dst, int32_t* copy_tokens, int32_t* results, void* workspace, size_t workspace_bytes,
                   void* stream);
int mla_pages_free(const mla_pool* pool, const int32_t* rows, int n, void* stream);
int mla_pages_compact(const mla_pool* pool, int32_t* counts, int32_t* src, int32_t* dst, void* workspace,
                      size_t workspace_bytes, void* stream);

/* Workspace bytes a call with these dims needs (0 on invalid dims).  With
 * dims->num_workers == 0 it queries the current device's SM count. */
size_t mla_workspace_bytes(const mla_dims* dims, int is_prefill);

/* Workspace bytes of mla_paged_decode_mtp with q_len tokens per request (0 on invalid
 * dims or q_len * num_qo_heads > 128). */
size_t mla_workspace_bytes_mtp(const mla_dims* dims, int q_len);

/* Number of split-KV workers (CTA pairs) used when dims->num_workers == 0, for the
 * current device; negative mla_status on failure. */
int mla_default_num_workers(void);

/* Human-readable name of a status code (static string). */
const char* mla_status_string(int status);

/* Synchronises `stream`, reads the device status word kept in `workspace` (MLA_OK,
 * MLA_ERR_BAD_INDEX, MLA_ERR_TIMEOUT or MLA_ERR_INTERNAL), clears it, and returns it.
 * Returns MLA_ERR_CUDA if the synchronisation itself reports an error. */
int mla_read_device_status(void* workspace, void* stream);

/* Test hook of the kernels' bounded waits (off by default; not for production use).
 * With skip_tile >= 1, the attention kernel's producer for split-KV worker 0 (first CTA
 * of the pair) skips the loads and the arrival of that tile of its range in every call
 * that follows, so the waits on it run out; wait_ns sets the limit of every bounded wait
 * (0 = the default of 4 s).  The kernel then gives up, unwinds (drains its copies and
 * matrix operations, frees tensor memory) and records MLA_ERR_TIMEOUT in the status
 * word, where mla_read_device_status finds it; outputs of that call are undefined.
 * skip_tile = -1 restores normal calls.  Returns MLA_ERR_DIMS for skip_tile 0 or < -1.
 * Not thread-safe with respect to calls in flight on other threads. */
int mla_debug_inject_timeout(int skip_tile, unsigned long long wait_ns);

/* Kernel timing for benchmarks.  When enabled, every attention call records CUDA events on
 * its stream around its main attention kernel (for the staged prefill: staging and
 * attention) and its combine kernel;
 * mla_profile_read synchronises on the last events, returns the summed milliseconds
 * and the number of timed calls since the last read, and resets the sums. */
int mla_profile_enable(int on);
int mla_profile_read(double* main_ms, double* combine_ms, int* calls);

#ifdef __cplusplus
}
#endif

#endif /* MLA_PAGED_H */
