// launch.h -- host-side launchers, one per kernel translation unit.
#pragma once
#include <cuda_runtime.h>

#include "common.cuh"

namespace mla {

// Merge of split rows' fragments (one warp per worker record and head).
cudaError_t launch_combine(const MlaParams& p, cudaStream_t stream);
// Optional index validation (sets the status word; never traps).
cudaError_t launch_validate(const MlaParams& p, cudaStream_t stream);
// Block table + sequence lengths -> token-slot CSR (two kernels on `stream`).
cudaError_t launch_block_table_csr(const int32_t* block_table, const int32_t* seq_lens, int batch, int max_blocks,
                                   int page_size, int32_t* kv_indptr, int32_t* kv_indices, long long capacity,
                                   cudaStream_t stream);

// Block table + sequence lengths -> groups that share leading pages, prefix lists and own lists.
struct SharedTableParams {
  const int32_t* block_table;  // [batch, max_blocks]
  const int32_t* seq_lens;     // [batch]
  int batch, max_blocks, page_size, min_shared;
  int32_t* group_indptr;       // [batch + 1]
  int32_t* prefix_indptr;      // [batch + 1]
  int32_t* prefix_indices;     // [prefix_capacity]
  int32_t* kv_indptr;          // [batch + 1]
  int32_t* kv_indices;         // [capacity]
  long long prefix_capacity, capacity;
};
cudaError_t launch_shared_tables(const SharedTableParams& p, cudaStream_t stream);

// ---------------------------------------------------------------- the cache's writers and readers
struct RopeParams {
  const __nv_bfloat16* q;    // [tokens, H, 64], strides in elements
  const __nv_bfloat16* ckv;  // [tokens, 512], row stride ckv_stride
  const __nv_bfloat16* kpe;  // [tokens, 64], row stride kpe_stride
  const int32_t* positions;  // [axes, tokens]
  const float* inv_freq;     // [32] radians per position of every pair
  const int32_t* slots;      // [tokens]; outside the cache: the token is not written
  __nv_bfloat16* q_out;      // [tokens, H, 64] contiguous
  __nv_bfloat16* ckv_cache;  // [num_slots, 512] (bf16 cache)
  __nv_bfloat16* kpe_cache;  // [num_slots, 64]
  uint8_t* kv_fp8;           // [num_slots, 656] (FP8 cache)
  long long q_stride_t, q_stride_h, ckv_stride, kpe_stride;
  int tokens, heads, num_slots;
  int section0, section1;    // pairs of axis 0 and 1; the rest are axis 2's
  bool interleaved;
};

struct GatherParams {
  const __nv_bfloat16* ckv;
  const __nv_bfloat16* kpe;
  const uint8_t* kv_fp8;     // FP8 cache
  const int32_t* slots;      // [n]
  const int32_t* count;      // device scalar: rows past it are left as they are (nullptr: n)
  __nv_bfloat16* ckv_out;    // [n, 512]
  __nv_bfloat16* kpe_out;    // [n, 64]
  int n, num_slots;
};

struct CopyParams {
  uint8_t* a;                // page bytes: page_size * bytes_a each
  uint8_t* b;                // second part (rope cache), or unused with bytes_b = 0
  const int32_t* src;
  const int32_t* dst;
  const int32_t* tokens;     // slots of the page to copy (nullptr: all)
  const int32_t* count;      // device scalar: entries in use (nullptr: n)
  int n, num_pages, page_size, bytes_a, bytes_b;
};

cudaError_t launch_rope_append(const RopeParams& p, bool fp8, cudaStream_t stream);
cudaError_t launch_gather(const GatherParams& p, bool fp8, cudaStream_t stream);
cudaError_t launch_copy_pages(const CopyParams& p, cudaStream_t stream);

// ---------------------------------------------------------------- the page pool
struct PoolParams {
  int32_t* block_table;      // [max_rows, max_blocks]
  int32_t* seq_lens;         // [max_rows]
  int32_t* ref_count;        // [num_pages]
  int max_rows, max_blocks, num_pages, page_size;
  int n;                     // entries of the call
  const int32_t* rows;       // extend, free
  const int32_t* new_tokens; // extend
  const int32_t* parents;    // fork
  const int32_t* children;
  int32_t* results;          // [n] status of every entry
  int32_t* new_indptr;       // extend: [n + 1]
  int32_t* slots;            // extend: [capacity]
  long long capacity;
  int32_t* src;              // fork [n], compact [num_pages / 2]: pages to copy
  int32_t* dst;
  int32_t* copy_tokens;      // fork [n]
  int32_t* counts;           // compact: {live pages, moves}
};

// Scratch of one call; nothing in it outlives the call.
struct PoolWork {
  uint32_t* bits;            // free pages, 32 a word
  int32_t* before;           // free pages before a word (in a large pool: within its span)
  int32_t* base;             // free pages before a span of words (large pools)
  int32_t* claim;            // [max_rows] first entry that names the row
  int32_t* pages;            // [num_pages] the free pages that the call takes
  int32_t* old_len;          // [n] length that a granted entry starts from, else -1
  int32_t* first;            // [n] an entry's first place in pages
};

cudaError_t launch_pages_extend(const PoolParams& p, const PoolWork& w, cudaStream_t stream);
cudaError_t launch_pages_fork(const PoolParams& p, const PoolWork& w, cudaStream_t stream);
cudaError_t launch_pages_free(const PoolParams& p, cudaStream_t stream);
cudaError_t launch_pages_compact(const PoolParams& p, const PoolWork& w, cudaStream_t stream);

}  // namespace mla
