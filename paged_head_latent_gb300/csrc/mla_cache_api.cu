// mla_cache_api.cu -- C entry points of the cache's writers, readers and page pool: argument
// checks and workspace layout.  Like the attention calls they only enqueue work on the
// caller's stream and read no device memory on the host.
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "launch.h"
#include "mla_paged.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool cache_dims(int num_pages, int page_size) {
  return num_pages >= 0 && page_size >= 1 && (long long)num_pages * page_size < (1LL << 31);
}

int launched(cudaError_t e) { return e == cudaSuccess ? MLA_OK : MLA_ERR_LAUNCH; }

cudaStream_t stream_of(void* stream) {
  cudaGetLastError();  // clear stale errors so the checks after the launches see only ours
  return static_cast<cudaStream_t>(stream);
}

int rope_append(const void* q_pe, const void* ckv, const void* k_pe, const int32_t* positions, const float* inv_freq,
                const int32_t* slots, void* q_out, void* ckv_cache, void* kpe_cache, void* kv_fp8, bool fp8,
                const mla_rope_dims* d, void* stream) {
  if (!d) return MLA_ERR_NULL;
  if (d->tokens < 0 || d->num_qo_heads < 0 || d->num_qo_heads > mla::kMaxHeads) return MLA_ERR_DIMS;
  if (d->num_axes < 1 || d->num_axes > 3 || !cache_dims(d->num_pages, d->page_size)) return MLA_ERR_DIMS;
  long long pairs = 0;
  for (int a = 0; a < d->num_axes; ++a) {
    if (d->section[a] < 0) return MLA_ERR_DIMS;
    pairs += d->section[a];
  }
  if (pairs != mla::kDimKpe / 2) return MLA_ERR_DIMS;
  if (d->q_stride_token < 0 || d->q_stride_head < 0 || d->ckv_stride < 0 || d->kpe_stride < 0) return MLA_ERR_DIMS;
  if (d->tokens == 0) return MLA_OK;
  if (!ckv || !k_pe || !positions || !inv_freq || !slots) return MLA_ERR_NULL;
  if (d->num_qo_heads > 0 && (!q_pe || !q_out)) return MLA_ERR_NULL;
  if (d->num_pages > 0 && (fp8 ? !kv_fp8 : !ckv_cache || !kpe_cache)) return MLA_ERR_NULL;
  if (!aligned16(ckv) || !aligned16(k_pe) || !aligned16(ckv_cache) || !aligned16(kpe_cache) || !aligned16(kv_fp8))
    return MLA_ERR_ALIGN;
  if (d->num_qo_heads > 0 && (!aligned16(q_pe) || !aligned16(q_out))) return MLA_ERR_ALIGN;
  if (d->ckv_stride % 8 || d->kpe_stride % 8) return MLA_ERR_ALIGN;
  if (d->num_qo_heads > 0 && (d->q_stride_token % 8 || d->q_stride_head % 8)) return MLA_ERR_ALIGN;
  // In place, a warp writes where it read only if the queries lie as the output does.
  if (d->num_qo_heads > 0 && q_out == q_pe &&
      ((d->num_qo_heads > 1 && d->q_stride_head != mla::kDimKpe) ||
       (d->tokens > 1 && d->q_stride_token != (int64_t)d->num_qo_heads * mla::kDimKpe)))
    return MLA_ERR_DIMS;
  mla::RopeParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q_pe);
  p.ckv = static_cast<const __nv_bfloat16*>(ckv);
  p.kpe = static_cast<const __nv_bfloat16*>(k_pe);
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.slots = slots;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.ckv_cache = static_cast<__nv_bfloat16*>(ckv_cache);
  p.kpe_cache = static_cast<__nv_bfloat16*>(kpe_cache);
  p.kv_fp8 = static_cast<uint8_t*>(kv_fp8);
  p.q_stride_t = d->q_stride_token;
  p.q_stride_h = d->q_stride_head;
  p.ckv_stride = d->ckv_stride;
  p.kpe_stride = d->kpe_stride;
  p.tokens = d->tokens;
  p.heads = d->num_qo_heads;
  p.num_slots = d->num_pages * d->page_size;
  p.section0 = d->section[0];
  p.section1 = d->num_axes > 1 ? d->section[1] : 0;
  p.interleaved = d->interleaved != 0;
  return launched(mla::launch_rope_append(p, fp8, stream_of(stream)));
}

int gather(const void* ckv, const void* kpe, const void* kv_fp8, bool fp8, const int32_t* slots, int n,
           const int32_t* count, int num_pages, int page_size, void* ckv_out, void* kpe_out, void* stream) {
  if (n < 0 || !cache_dims(num_pages, page_size)) return MLA_ERR_DIMS;
  if (n == 0) return MLA_OK;
  if (!slots || !ckv_out || !kpe_out) return MLA_ERR_NULL;
  if (num_pages > 0 && (fp8 ? !kv_fp8 : !ckv || !kpe)) return MLA_ERR_NULL;
  if (!aligned16(ckv) || !aligned16(kpe) || !aligned16(kv_fp8) || !aligned16(ckv_out) || !aligned16(kpe_out))
    return MLA_ERR_ALIGN;
  mla::GatherParams p{};
  p.ckv = static_cast<const __nv_bfloat16*>(ckv);
  p.kpe = static_cast<const __nv_bfloat16*>(kpe);
  p.kv_fp8 = static_cast<const uint8_t*>(kv_fp8);
  p.slots = slots;
  p.count = count;
  p.ckv_out = static_cast<__nv_bfloat16*>(ckv_out);
  p.kpe_out = static_cast<__nv_bfloat16*>(kpe_out);
  p.n = n;
  p.num_slots = num_pages * page_size;
  return launched(mla::launch_gather(p, fp8, stream_of(stream)));
}

int copy_pages(void* a, void* b, int bytes_a, int bytes_b, const int32_t* src, const int32_t* dst,
               const int32_t* tokens, int n, const int32_t* count, int num_pages, int page_size, void* stream) {
  if (n < 0 || !cache_dims(num_pages, page_size)) return MLA_ERR_DIMS;
  if (n == 0 || num_pages == 0) return MLA_OK;
  if (!src || !dst || !a || (bytes_b && !b)) return MLA_ERR_NULL;
  if (!aligned16(a) || !aligned16(b)) return MLA_ERR_ALIGN;
  mla::CopyParams p{};
  p.a = static_cast<uint8_t*>(a);
  p.b = static_cast<uint8_t*>(b);
  p.src = src;
  p.dst = dst;
  p.tokens = tokens;
  p.count = count;
  p.n = n;
  p.num_pages = num_pages;
  p.page_size = page_size;
  p.bytes_a = bytes_a;
  p.bytes_b = bytes_b;
  return launched(mla::launch_copy_pages(p, stream_of(stream)));
}

int check_pool(const mla_pool* pool) {
  if (!pool) return MLA_ERR_NULL;
  if (pool->max_rows < 0 || pool->max_blocks < 0 || !cache_dims(pool->num_pages, pool->page_size)) return MLA_ERR_DIMS;
  if ((long long)pool->max_blocks * pool->page_size > 0x7fffffffLL) return MLA_ERR_DIMS;
  return MLA_OK;
}

// The pool's arrays may be NULL only where they hold nothing.
int check_arrays(const mla_pool* pool) {
  if (pool->max_rows > 0 && (!pool->seq_lens || (pool->max_blocks > 0 && !pool->block_table))) return MLA_ERR_NULL;
  if (pool->num_pages > 0 && !pool->ref_count) return MLA_ERR_NULL;
  return MLA_OK;
}

mla::PoolParams params_of(const mla_pool* pool, int n) {
  mla::PoolParams p{};
  p.block_table = pool->block_table;
  p.seq_lens = pool->seq_lens;
  p.ref_count = pool->ref_count;
  p.max_rows = pool->max_rows;
  p.max_blocks = pool->max_blocks;
  p.num_pages = pool->num_pages;
  p.page_size = pool->page_size;
  p.n = n;
  return p;
}

// Workspace: 256 bytes left alone (the attention calls' status word, where the workspace serves them
// too), free-page bitmap, free pages before each of its words and spans, claims, pages taken, then
// the entries' decisions.
struct PoolLayout {
  size_t bits, before, base, claim, pages, old_len, first, total;
  PoolLayout(const mla_pool* pool, int n) {
    const size_t words = ((size_t)pool->num_pages + 31) / 32;
    bits = 256;
    before = bits + mla::align_up(words * 4, 256);
    base = before + mla::align_up(words * 4, 256);
    claim = base + mla::align_up(words / 256 * 4 + 4, 256);
    pages = claim + mla::align_up((size_t)pool->max_rows * 4, 256);
    old_len = pages + mla::align_up((size_t)pool->num_pages * 4, 256);
    first = old_len + mla::align_up((size_t)n * 4, 256);
    total = first + mla::align_up((size_t)n * 4, 256) + 256;
  }
};

int work_of(const mla_pool* pool, int n, void* workspace, size_t bytes, mla::PoolWork* w) {
  const PoolLayout lay(pool, n);
  if (!workspace || bytes < lay.total) return MLA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return MLA_ERR_ALIGN;
  auto* ws = static_cast<uint8_t*>(workspace);
  w->bits = reinterpret_cast<uint32_t*>(ws + lay.bits);
  w->before = reinterpret_cast<int32_t*>(ws + lay.before);
  w->base = reinterpret_cast<int32_t*>(ws + lay.base);
  w->claim = reinterpret_cast<int32_t*>(ws + lay.claim);
  w->pages = reinterpret_cast<int32_t*>(ws + lay.pages);
  w->old_len = reinterpret_cast<int32_t*>(ws + lay.old_len);
  w->first = reinterpret_cast<int32_t*>(ws + lay.first);
  return MLA_OK;
}

}  // namespace

extern "C" {

int mla_rope_append(const void* q_pe, const void* ckv, const void* k_pe, const int32_t* positions,
                    const float* inv_freq, const int32_t* slots, void* q_out, void* ckv_cache, void* kpe_cache,
                    const mla_rope_dims* dims, void* stream) {
  return rope_append(q_pe, ckv, k_pe, positions, inv_freq, slots, q_out, ckv_cache, kpe_cache, nullptr, false, dims,
                     stream);
}

int mla_rope_append_fp8(const void* q_pe, const void* ckv, const void* k_pe, const int32_t* positions,
                        const float* inv_freq, const int32_t* slots, void* q_out, void* kv_fp8,
                        const mla_rope_dims* dims, void* stream) {
  return rope_append(q_pe, ckv, k_pe, positions, inv_freq, slots, q_out, nullptr, nullptr, kv_fp8, true, dims, stream);
}

int mla_cache_gather(const void* ckv_cache, const void* kpe_cache, const int32_t* slots, int n, const int32_t* count,
                     int num_pages, int page_size, void* ckv_out, void* kpe_out, void* stream) {
  return gather(ckv_cache, kpe_cache, nullptr, false, slots, n, count, num_pages, page_size, ckv_out, kpe_out, stream);
}

int mla_cache_gather_fp8(const void* kv_fp8, const int32_t* slots, int n, const int32_t* count, int num_pages,
                         int page_size, void* ckv_out, void* kpe_out, void* stream) {
  return gather(nullptr, nullptr, kv_fp8, true, slots, n, count, num_pages, page_size, ckv_out, kpe_out, stream);
}

int mla_cache_copy_pages(void* ckv_cache, void* kpe_cache, const int32_t* src, const int32_t* dst,
                         const int32_t* tokens, int n, const int32_t* count, int num_pages, int page_size,
                         void* stream) {
  return copy_pages(ckv_cache, kpe_cache, 2 * mla::kDimCkv, 2 * mla::kDimKpe, src, dst, tokens, n, count, num_pages,
                    page_size, stream);
}

int mla_cache_copy_pages_fp8(void* kv_fp8, const int32_t* src, const int32_t* dst, const int32_t* tokens, int n,
                             const int32_t* count, int num_pages, int page_size, void* stream) {
  return copy_pages(kv_fp8, nullptr, mla::kFp8TokenBytes, 0, src, dst, tokens, n, count, num_pages, page_size, stream);
}

size_t mla_workspace_bytes_pages(const mla_pool* pool, int n) {
  if (n < 0 || check_pool(pool) != MLA_OK) return 0;
  return PoolLayout(pool, n).total;
}

int mla_pages_extend(const mla_pool* pool, const int32_t* rows, const int32_t* new_tokens, int n, int32_t* new_indptr,
                     int32_t* slots, long long capacity, int32_t* results, void* workspace, size_t workspace_bytes,
                     void* stream) {
  int st = check_pool(pool);
  if (st != MLA_OK) return st;
  if (n < 0 || capacity < 0 || capacity > 0x7fffffffLL) return MLA_ERR_DIMS;
  if ((st = check_arrays(pool)) != MLA_OK) return st;
  if (!new_indptr || (n > 0 && (!rows || !new_tokens || !results)) || (capacity > 0 && !slots)) return MLA_ERR_NULL;
  mla::PoolWork w;
  if ((st = work_of(pool, n, workspace, workspace_bytes, &w)) != MLA_OK) return st;
  mla::PoolParams p = params_of(pool, n);
  p.rows = rows;
  p.new_tokens = new_tokens;
  p.new_indptr = new_indptr;
  p.slots = slots;
  p.capacity = capacity;
  p.results = results;
  return launched(mla::launch_pages_extend(p, w, stream_of(stream)));
}

int mla_pages_fork(const mla_pool* pool, const int32_t* parents, const int32_t* children, int n, int32_t* src,
                   int32_t* dst, int32_t* copy_tokens, int32_t* results, void* workspace, size_t workspace_bytes,
                   void* stream) {
  int st = check_pool(pool);
  if (st != MLA_OK) return st;
  if (n < 0) return MLA_ERR_DIMS;
  if ((st = check_arrays(pool)) != MLA_OK) return st;
  if (n == 0) return MLA_OK;
  if (!parents || !children || !src || !dst || !copy_tokens || !results) return MLA_ERR_NULL;
  mla::PoolWork w;
  if ((st = work_of(pool, n, workspace, workspace_bytes, &w)) != MLA_OK) return st;
  mla::PoolParams p = params_of(pool, n);
  p.parents = parents;
  p.children = children;
  p.src = src;
  p.dst = dst;
  p.copy_tokens = copy_tokens;
  p.results = results;
  return launched(mla::launch_pages_fork(p, w, stream_of(stream)));
}

int mla_pages_free(const mla_pool* pool, const int32_t* rows, int n, void* stream) {
  int st = check_pool(pool);
  if (st != MLA_OK) return st;
  if (n < 0) return MLA_ERR_DIMS;
  if ((st = check_arrays(pool)) != MLA_OK) return st;
  if (n == 0) return MLA_OK;
  if (!rows) return MLA_ERR_NULL;
  mla::PoolParams p = params_of(pool, n);
  p.rows = rows;
  return launched(mla::launch_pages_free(p, stream_of(stream)));
}

int mla_pages_compact(const mla_pool* pool, int32_t* counts, int32_t* src, int32_t* dst, void* workspace,
                      size_t workspace_bytes, void* stream) {
  int st = check_pool(pool);
  if (st != MLA_OK) return st;
  if ((st = check_arrays(pool)) != MLA_OK) return st;
  if (!counts || (pool->num_pages > 1 && (!src || !dst))) return MLA_ERR_NULL;
  mla::PoolWork w;
  if ((st = work_of(pool, 0, workspace, workspace_bytes, &w)) != MLA_OK) return st;
  mla::PoolParams p = params_of(pool, 0);
  p.counts = counts;
  p.src = src;
  p.dst = dst;
  return launched(mla::launch_pages_compact(p, w, stream_of(stream)));
}

}  // extern "C"
