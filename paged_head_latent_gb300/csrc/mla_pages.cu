// mla_pages.cu -- the page pool: which pages of the cache belong to which sequence.
//
// The pool is three device arrays that the caller owns: block_table [max_rows, max_blocks]
// (page ids in sequence order), seq_lens [max_rows] and ref_count [num_pages] (how many
// sequences hold a page; 0 = free).  There is no free list to keep consistent: a call that
// needs pages takes the free pages with the lowest ids, in the order of its entries, so its
// outcome is unique whatever the order of the kernels' threads, and the pages it fills lie
// at the front of the cache.
//
// A call is two launches on one stream: one block that makes a bitmap of the free pages (one
// pass over ref_count, 4 bytes a page), numbers them and decides every entry, and a grid that
// applies the decisions.  For a pool of more than 16,384 pages a grid makes the bitmap first.
// Nothing but integers is computed; the counters that several threads change are changed by
// integer atomics, whose order does not matter.  What bounds these calls is latency: the
// plan is a chain of dependent loads (row, length, last page, its count) and block scans.
#include "launch.h"
#include "mla_paged.h"

namespace mla {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kApplyThreads = 128;

__device__ __forceinline__ int blocks_of(int len, int page_size) {
  return len <= 0 ? 0 : (len - 1) / page_size + 1;
}

// A row's blocks in use, clamped to the table.
__device__ __forceinline__ int used_blocks(const PoolParams& p, int len) {
  return min(blocks_of(len, p.page_size), p.max_blocks);
}

__device__ __forceinline__ bool is_page(const PoolParams& p, int page) { return page >= 0 && page < p.num_pages; }

// Bit i of word w: page 32 w + i is free; before[w]: free pages in the earlier words of the
// word's span.  One block a span; totals[span] = its free pages.
constexpr int kSpan = 256;

__global__ void __launch_bounds__(kSpan) free_bitmap_kernel(PoolParams p, PoolWork w) {
  __shared__ int warps[kSpan / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int words = (p.num_pages + 31) / 32, w0 = blockIdx.x * kSpan + 32 * warp;
  int32_t ref[32];  // the counts of the warp's 32 words
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    const long long page = 32LL * (w0 + k) + lane;
    ref[k] = page < p.num_pages ? p.ref_count[page] : 1;
  }
  uint32_t mine = 0;  // lane k keeps word w0 + k
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    const unsigned b = __ballot_sync(0xffffffffu, ref[k] <= 0);
    if (lane == k) mine = b;
  }
  const int c = __popc(mine);
  int incl = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) warps[warp] = incl;
  __syncthreads();
  int at = incl - c, all = 0;
#pragma unroll
  for (int i = 0; i < kSpan / 32; ++i) {
    if (i < warp) at += warps[i];
    all += warps[i];
  }
  if (w0 + lane < words) {
    w.bits[w0 + lane] = mine;
    w.before[w0 + lane] = at;
  }
  if (threadIdx.x == 0) w.base[blockIdx.x] = all;
}

// Exclusive sum of v over the block; *total = the block's sum.
__device__ __forceinline__ long long block_scan(long long v, long long* part, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    long long s = part[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += x;
    }
    part[lane] = s;
  }
  __syncthreads();
  const long long before = warp ? part[warp - 1] : 0;
  *total = part[kPlanThreads / 32 - 1];
  __syncthreads();
  return before + incl - v;
}

// The numbered free pages: base (nullptr: zeros) has the free pages before each span.
struct FreeView {
  const uint32_t* bits;
  const int32_t* before;
  const int32_t* base;
  __device__ int before_word(int i) const { return before[i] + (base ? base[i / kSpan] : 0); }
  __device__ int before_page(int page) const {
    return before_word(page >> 5) + __popc(bits[page >> 5] & ((1u << (page & 31)) - 1u));
  }
  __device__ bool is_free(int page) const { return (bits[page >> 5] >> (page & 31)) & 1u; }
  // The j-th free page (j < the number of free pages).
  __device__ int page(int words, int j) const {
    int lo = 0, hi = words - 1;  // last word with at most j free pages before it
    while (lo < hi) {
      const int mid = lo + (hi - lo + 1) / 2;
      if (before_word(mid) <= j) lo = mid; else hi = mid - 1;
    }
    uint32_t b = bits[lo];
    for (int k = j - before_word(lo); k > 0; --k) b &= b - 1;
    return 32 * lo + __ffs(b) - 1;
  }
};

// The plan's numbering.  kNear: the block makes the bitmap itself, in shared memory;
// otherwise the grid before it did, span by span, and the block adds up the spans.  A fork
// that is refused takes (warm) 5.0 us near and 7.2 by the grid for 4096 pages, 5.2 and 6.9 for
// 16,384; for 65,536 pages a bitmap of the block's own took 12.7 us, the grid's 7.0.
constexpr int kNearWords = 512;

template <bool kNear>
struct FreePages {
  const PoolParams& p;
  const PoolWork& w;
  uint32_t* near_bits;
  int32_t* near_before;
  __device__ FreePages(const PoolParams& pool, const PoolWork& work, uint32_t* bits, int32_t* before)
      : p(pool), w(work), near_bits(bits), near_before(before) {}
  __device__ int words() const { return (p.num_pages + 31) / 32; }
  __device__ FreeView view() const {
    return kNear ? FreeView{near_bits, near_before, nullptr} : FreeView{w.bits, w.before, w.base};
  }

  // Numbers the free pages and returns how many there are (called by the whole block).
  __device__ long long number(long long* part) {
    long long run = 0, total;
    if constexpr (kNear) {
      const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
      constexpr int kFlight = kNearWords / (kPlanThreads / 32);  // words of a warp, all in flight
      const int w0 = kFlight * warp;
      int32_t ref[kFlight];
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        const int page = 32 * (w0 + k) + lane;
        ref[k] = page < p.num_pages ? p.ref_count[page] : 1;
      }
      uint32_t mine = 0;  // lane k keeps word w0 + k
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        const unsigned b = __ballot_sync(0xffffffffu, ref[k] <= 0);
        if (lane == k) mine = b;
      }
      if (lane < kFlight) near_bits[w0 + lane] = mine;
      __syncthreads();
      const int i = threadIdx.x;
      const long long at = block_scan(i < kNearWords ? __popc(near_bits[i]) : 0, part, &run);
      if (i < kNearWords) near_before[i] = (int32_t)at;
    } else {
      const int spans = (words() + kSpan - 1) / kSpan;
      for (int base = 0; base < spans; base += kPlanThreads) {
        const int i = base + threadIdx.x;
        const long long at = run + block_scan(i < spans ? w.base[i] : 0, part, &total);
        if (i < spans) w.base[i] = (int32_t)at;
        run += total;
      }
    }
    __syncthreads();
    return run;
  }

  // The ids of the first `need` free pages, in order.
  __device__ void list(long long need) {
    const FreeView v = view();
    for (int base = 0; base < words() && v.before_word(base) < need; base += kPlanThreads) {
      const int i = base + threadIdx.x;
      if (i >= words()) break;
      uint32_t b = v.bits[i];
      for (long long r = v.before_word(i); b && r < need; ++r, b &= b - 1) w.pages[r] = 32 * i + __ffs(b) - 1;
    }
  }
};

// One block: decides every entry in list order.  Entry i is valid if its indices are and no
// earlier entry names its row; a valid entry is granted if it needs no page, or if the
// pages that the valid entries up to and including it need are there.
template <bool kFork, bool kNear>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PoolParams p, PoolWork w) {
  __shared__ long long part[32];
  __shared__ uint32_t near_bits[kNear ? kNearWords : 1];
  __shared__ int32_t near_before[kNear ? kNearWords : 1];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ int taken;
  const int32_t* rows = kFork ? p.children : p.rows;
  auto good_row = [&](int r) { return r >= 0 && r < p.max_rows; };
  const long long room = (long long)p.max_blocks * p.page_size;
  struct Entry {
    int row, len, add, need;
    bool ok;
  };
  auto examine = [&](int i) {  // all but whether an earlier entry names the row
    Entry e{-1, 0, 0, 0, false};
    if (i >= p.n) return e;
    e.row = rows[i];
    if (!good_row(e.row)) return e;
    if constexpr (kFork) {
      const int parent = p.parents[i];
      e.ok = good_row(parent) && parent != e.row && p.seq_lens[e.row] == 0;
      if (e.ok) {
        e.len = p.seq_lens[parent];
        e.ok = e.len >= 0 && e.len <= room;
      }
      if (e.ok && e.len % p.page_size != 0) {
        e.ok = is_page(p, p.block_table[(size_t)parent * p.max_blocks + e.len / p.page_size]);
        e.need = 1;
      }
    } else {
      e.len = p.seq_lens[e.row];
      e.add = p.new_tokens[i];
      e.ok = e.len >= 0 && e.add >= 0 && (long long)e.len + e.add <= room;
      if (e.ok && e.add > 0 && e.len % p.page_size != 0) {
        // The new tokens go on in the row's last page, which has to be its own.
        const int page = p.block_table[(size_t)e.row * p.max_blocks + e.len / p.page_size];
        e.ok = is_page(p, page) && p.ref_count[page] == 1;
      }
      if (e.ok) e.need = blocks_of(e.len + e.add, p.page_size) - blocks_of(e.len, p.page_size);
    }
    return e;
  };
  if (threadIdx.x == 0) taken = 0;
  for (int i = threadIdx.x; i < p.n; i += kPlanThreads)
    if (good_row(rows[i])) w.claim[rows[i]] = 0x7fffffff;
  __syncthreads();
  for (int i = threadIdx.x; i < p.n; i += kPlanThreads)
    if (good_row(rows[i])) atomicMin(&w.claim[rows[i]], i);
  const Entry early = examine(threadIdx.x);  // (its chain of loads overlaps the claims' round trip)
  FreePages<kNear> free(p, w, near_bits, near_before);
  const long long free_pages = free.number(part);
  __syncthreads();
  long long need_run = 0, new_run = 0, total;
  for (int base = 0; base < p.n; base += kPlanThreads) {
    const int i = base + threadIdx.x;
    const Entry e = base == 0 ? early : examine(i);
    const bool ok = e.ok && __ldcg(&w.claim[e.row]) == i;
    const int need = ok ? e.need : 0;
    const long long first = need_run + block_scan(need, part, &total);
    need_run += total;
    const bool granted = ok && (need == 0 || first + need <= free_pages);
    long long at = 0;
    if constexpr (!kFork) {
      at = new_run + block_scan(granted ? e.add : 0, part, &total);
      new_run += total;
    }
    // Granted entries that need pages are a prefix of those that need any.
    if (granted && need > 0) atomicMax(&taken, (int)(first + need));
    if (i < p.n) {
      p.results[i] = granted ? MLA_OK : ok ? MLA_ERR_NO_PAGES : MLA_ERR_BAD_INDEX;
      w.old_len[i] = granted ? e.len : -1;
      w.first[i] = (int32_t)first;
      if (!kFork) p.new_indptr[i] = (int32_t)min(at, 0x7fffffffLL);
    }
  }
  // Rows that share a partly filled page that is counted once (no call of the pool makes such) could
  // be granted more tokens than an int holds; no slot is written past the capacity, so none there.
  if (!kFork && threadIdx.x == 0) p.new_indptr[p.n] = (int32_t)min(new_run, 0x7fffffffLL);
  __syncthreads();
  free.list(taken);
}

// One block per entry: the row's new blocks, their counts, and the new tokens' slots.
__global__ void __launch_bounds__(kApplyThreads) extend_kernel(PoolParams p, PoolWork w) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int i = blockIdx.x; i < p.n; i += gridDim.x) {
    const int len = w.old_len[i];
    if (len < 0) continue;
    const int row = p.rows[i], add = p.new_tokens[i];
    int32_t* table = p.block_table + (size_t)row * p.max_blocks;
    const int have = blocks_of(len, p.page_size), want = blocks_of(len + add, p.page_size);
    const int32_t* pages = w.pages + w.first[i];
    for (int k = have + threadIdx.x; k < want; k += kApplyThreads) {
      const int page = pages[k - have];
      table[k] = page;
      p.ref_count[page] = 1;
    }
    const int last = have > 0 && len % p.page_size != 0 ? table[have - 1] : 0;
    const long long at = p.new_indptr[i];
    for (int k = threadIdx.x; k < add && at + k < p.capacity; k += kApplyThreads) {
      const int pos = len + k, block = pos / p.page_size;
      const int page = block < have ? last : pages[block - have];
      p.slots[at + k] = page * p.page_size + pos % p.page_size;
    }
    if (threadIdx.x == 0) p.seq_lens[row] = len + add;
  }
  // Slots past the granted tokens name no slot, so a write of that many tokens skips them.
  for (long long k = (long long)p.new_indptr[p.n] + blockIdx.x * kApplyThreads + threadIdx.x; k < p.capacity;
       k += (long long)gridDim.x * kApplyThreads)
    p.slots[k] = -1;
}

// One block per pair: the parent's full pages are shared, its partial page is listed for copying.
__global__ void __launch_bounds__(kApplyThreads) fork_kernel(PoolParams p, PoolWork w) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (the page copies)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int i = blockIdx.x; i < p.n; i += gridDim.x) {
    const int len = w.old_len[i];
    int src = -1, dst = -1, tokens = 0;
    if (len >= 0) {
      const int32_t* from = p.block_table + (size_t)p.parents[i] * p.max_blocks;
      int32_t* to = p.block_table + (size_t)p.children[i] * p.max_blocks;
      const int full = len / p.page_size;
      for (int k = threadIdx.x; k < full; k += kApplyThreads) {
        const int page = from[k];
        to[k] = page;
        if (is_page(p, page)) atomicAdd(&p.ref_count[page], 1);
      }
      tokens = len - full * p.page_size;
      if (tokens > 0) {
        src = from[full];
        dst = w.pages[w.first[i]];
        if (threadIdx.x == 0) {
          to[full] = dst;
          p.ref_count[dst] = 1;
        }
      }
      if (threadIdx.x == 0) p.seq_lens[p.children[i]] = len;
    }
    if (threadIdx.x == 0) {
      p.src[i] = src;
      p.dst[i] = dst;
      p.copy_tokens[i] = tokens;
    }
  }
}

// One block per listed row.  The row's length is taken by an exchange, so a row that is
// listed twice is freed once.
__global__ void __launch_bounds__(kApplyThreads) free_kernel(PoolParams p) {
  __shared__ int taken;
  for (int i = blockIdx.x; i < p.n; i += gridDim.x) {
    const int row = p.rows[i];
    if (row < 0 || row >= p.max_rows) continue;
    __syncthreads();
    if (threadIdx.x == 0) taken = atomicExch(&p.seq_lens[row], 0);
    __syncthreads();
    const int used = used_blocks(p, taken);
    int32_t* table = p.block_table + (size_t)row * p.max_blocks;
    for (int k = threadIdx.x; k < used; k += kApplyThreads) {
      const int page = table[k];
      table[k] = -1;
      if (is_page(p, page) && atomicSub(&p.ref_count[page], 1) <= 0) atomicAdd(&p.ref_count[page], 1);
    }
  }
}

// Compaction.  With L live pages, the live pages with ids >= L move, in order, to the free
// pages with ids < L: as many of the one as of the other.
template <bool kNear>
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(PoolParams p, PoolWork w) {
  __shared__ long long part[32];
  __shared__ uint32_t near_bits[kNear ? kNearWords : 1];
  __shared__ int32_t near_before[kNear ? kNearWords : 1];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  FreePages<kNear> free(p, w, near_bits, near_before);
  const int live = p.num_pages - (int)free.number(part);
  if constexpr (kNear)
    for (int i = threadIdx.x; i < free.words(); i += kPlanThreads) {
      w.bits[i] = near_bits[i];
      w.before[i] = near_before[i];
    }
  if (threadIdx.x == 0) {
    p.counts[0] = live;
    p.counts[1] = live < p.num_pages ? free.view().before_page(live) : 0;  // no page is free: none moves
  }
}

template <bool kNear>
__global__ void __launch_bounds__(256) compact_apply_kernel(PoolParams p, PoolWork w) {
  __shared__ uint32_t near_bits[kNear ? kNearWords : 1];
  __shared__ int32_t near_before[kNear ? kNearWords : 1];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (the page copies)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int live = p.counts[0], moves = p.counts[1], words = (p.num_pages + 31) / 32;
  if constexpr (kNear) {  // the searches below are chains of dependent reads
    for (int i = threadIdx.x; i < words; i += blockDim.x) {
      near_bits[i] = w.bits[i];
      near_before[i] = w.before[i];
    }
    __syncthreads();
  }
  const FreeView v = kNear ? FreeView{near_bits, near_before, nullptr} : FreeView{w.bits, w.before, w.base};
  const long long tid = blockIdx.x * blockDim.x + threadIdx.x, step = (long long)gridDim.x * blockDim.x;
  auto move_of = [&](int page) { return page - v.before_page(page) - (live - moves); };  // of a live page >= live
  for (long long page = live + tid; page < p.num_pages; page += step) {
    if (v.is_free((int)page)) continue;
    const int j = move_of((int)page), to = v.page(words, j);
    p.src[j] = (int)page;
    p.dst[j] = to;
    p.ref_count[to] = p.ref_count[page];
    p.ref_count[page] = 0;
  }
  for (long long k = moves + tid; k < p.num_pages / 2; k += step) p.src[k] = p.dst[k] = -1;
  const long long cells = (long long)p.max_rows * p.max_blocks;
  for (long long c = tid; c < cells; c += step) {
    const int row = (int)(c / p.max_blocks), k = (int)(c - (long long)row * p.max_blocks);
    if (k >= blocks_of(p.seq_lens[row], p.page_size)) continue;
    const int page = p.block_table[c];
    if (page < live || page >= p.num_pages || v.is_free(page)) continue;
    p.block_table[c] = v.page(words, move_of(page));
  }
}

int grid_of(long long threads, int block, int most) {
  const long long g = (threads + block - 1) / block;
  return (int)(g < 1 ? 1 : g > most ? most : g);
}

bool near_pool(const PoolParams& p) { return p.num_pages <= 32 * kNearWords; }

// The bitmap of a large pool.
cudaError_t launch_bitmap(const PoolParams& p, const PoolWork& w, cudaStream_t stream) {
  if (near_pool(p)) return cudaSuccess;
  free_bitmap_kernel<<<(p.num_pages - 1) / (32 * kSpan) + 1, kSpan, 0, stream>>>(p, w);
  return cudaGetLastError();
}

// A programmatic dependent of the plan: its launch overlaps the plan.
template <typename K>
cudaError_t launch_apply(K kernel, int grid, int threads, const PoolParams& p, const PoolWork& w, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p, w);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool kFork>
cudaError_t launch_plan(const PoolParams& p, const PoolWork& w, cudaStream_t stream) {
  const cudaError_t e = launch_bitmap(p, w, stream);
  if (e != cudaSuccess) return e;
  if (near_pool(p)) plan_kernel<kFork, true><<<1, kPlanThreads, 0, stream>>>(p, w);
  else plan_kernel<kFork, false><<<1, kPlanThreads, 0, stream>>>(p, w);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_pages_extend(const PoolParams& p, const PoolWork& w, cudaStream_t stream) {
  const cudaError_t e = launch_plan<false>(p, w, stream);
  return e != cudaSuccess ? e : launch_apply(extend_kernel, p.n < 1 ? 1 : p.n < 4096 ? p.n : 4096, kApplyThreads, p, w, stream);
}

cudaError_t launch_pages_fork(const PoolParams& p, const PoolWork& w, cudaStream_t stream) {
  const cudaError_t e = launch_plan<true>(p, w, stream);
  return e != cudaSuccess ? e : launch_apply(fork_kernel, p.n < 4096 ? p.n : 4096, kApplyThreads, p, w, stream);
}

cudaError_t launch_pages_free(const PoolParams& p, cudaStream_t stream) {
  free_kernel<<<p.n < 4096 ? p.n : 4096, kApplyThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_pages_compact(const PoolParams& p, const PoolWork& w, cudaStream_t stream) {
  cudaError_t e = launch_bitmap(p, w, stream);
  if (e != cudaSuccess) return e;
  if (near_pool(p)) compact_plan_kernel<true><<<1, kPlanThreads, 0, stream>>>(p, w);
  else compact_plan_kernel<false><<<1, kPlanThreads, 0, stream>>>(p, w);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const long long threads = (long long)p.max_rows * p.max_blocks > p.num_pages ? (long long)p.max_rows * p.max_blocks : p.num_pages;
  const int grid = grid_of(threads, 256, 1216);
  return near_pool(p) ? launch_apply(compact_apply_kernel<true>, grid, 256, p, w, stream)
                      : launch_apply(compact_apply_kernel<false>, grid, 256, p, w, stream);
}

}  // namespace mla
