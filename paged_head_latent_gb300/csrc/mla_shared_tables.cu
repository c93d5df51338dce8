// mla_shared_tables.cu -- block table + sequence lengths -> the groups of neighbouring rows that
// share leading pages, with the key lists that the shared attention takes.
//
//   len_i   = clamp(seq_lens[i], 0, max_blocks * page_size)
//   pages_i = number of leading page ids that rows i - 1 and i have in common, of those that are full
//             in both (a partly filled page belongs to one row)
//   row i opens a group if i = 0 or pages_i * page_size < max(1, min_shared), else it joins row i - 1's
//   shared_g = page_size * min pages_i over the rows that joined group g; 0 if none did
// As the leading pages of a row are compared with those of its neighbour, the least of a group is
// what all its rows share.  prefix list g: the first shared_g slots of the group's first row; own
// list i: the slots behind them of row i.  Integer work, whose outcome is unique.
//
// What bounds it: latency.  The first launch reads the table once (a block a row), the second is
// one block's three scans (groups, prefix offsets, own offsets), the third writes the lists: 4, 5
// and 10 us by themselves for 500 rows of up to 290 pages.  A small table takes one block and one
// launch: 8 us for 16 rows of 60 pages.
#include "launch.h"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kScanThreads = 1024;
constexpr int kFillBlocks = 4;  // blocks of threads for a row's lists

__device__ __forceinline__ long long length_of(const SharedTableParams& p, int i) {
  const long long v = __ldg(p.seq_lens + i), most = (long long)p.max_blocks * p.page_size;
  return v < 0 ? 0 : v > most ? most : v;
}

// pages_i into kv_indptr[i], which the next launch overwrites.
__global__ void __launch_bounds__(kThreads) common_pages_kernel(const SharedTableParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ int first[kThreads / 32];
  for (int i = blockIdx.x; i < p.batch; i += gridDim.x) {
    int most = 0;
    if (i > 0) most = (int)(min(length_of(p, i - 1), length_of(p, i)) / p.page_size);
    const int32_t* a = p.block_table + (size_t)i * p.max_blocks;
    const int32_t* b = a - p.max_blocks;
    int differ = most;
    // (unsigned: a step behind the last of 2^31 - 1 pages is not in front of the first)
#pragma unroll 4
    for (unsigned k = threadIdx.x; k < (unsigned)most; k += kThreads)
      if (__ldg(a + k) != __ldg(b + k)) differ = min(differ, (int)k);
    differ = __reduce_min_sync(0xffffffffu, differ);
    if ((threadIdx.x & 31) == 0) first[threadIdx.x >> 5] = differ;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
      for (int k = 1; k < kThreads / 32; ++k) differ = min(differ, first[k]);
      p.kv_indptr[i] = differ;
    }
    __syncthreads();
  }
}

// Inclusive sum over the block's threads.
__device__ __forceinline__ long long scan_block(long long v, long long* part, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  if (lane == 31) part[warp] = v;
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
  v += warp > 0 ? part[warp - 1] : 0;
  *total = part[kScanThreads / 32 - 1];
  __syncthreads();
  return v;
}

__device__ __forceinline__ int32_t offset32(long long v) { return (int32_t)min(v, 0x7fffffffLL); }

// One block: the groups and all offsets.  prefix_indptr[g + 1] holds the least pages_i of group g
// and kv_indptr[i] the group of row i in between.
__global__ void __launch_bounds__(kScanThreads) groups_kernel(const SharedTableParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ long long part[kScanThreads / 32];
  const int n = p.batch;
  for (int g = threadIdx.x; g <= n; g += kScanThreads) {
    p.group_indptr[g] = n;
    p.prefix_indptr[g] = g == 0 ? 0 : 0x7fffffff;
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");  // pages_i
  const long long least = p.min_shared > 1 ? p.min_shared : 1;
  long long run = 0, total;
  for (int base = 0; base < n; base += kScanThreads) {
    const int i = base + threadIdx.x;
    int pages = 0;
    bool opens = false;
    if (i < n) {
      pages = __ldcg(p.kv_indptr + i);
      opens = i == 0 || (long long)pages * p.page_size < least;
    }
    const int g = (int)(run + scan_block(opens, part, &total)) - 1;
    if (i < n) {
      if (opens) p.group_indptr[g] = i;
      else atomicMin(p.prefix_indptr + g + 1, pages);
      p.kv_indptr[i] = g;
    }
    run += total;
  }
  __threadfence_block();
  __syncthreads();
  run = 0;
  for (int base = 0; base < n; base += kScanThreads) {
    const int g = base + threadIdx.x;
    long long keys = 0;
    if (g < n) {
      const int pages = __ldcg(p.prefix_indptr + g + 1);
      keys = pages == 0x7fffffff ? 0 : (long long)pages * p.page_size;
    }
    // (the offsets stay at the largest int once they have reached it)
    const long long end = run + scan_block(keys, part, &total);
    if (g < n) p.prefix_indptr[g + 1] = offset32(end);
    run += total;
  }
  // A row's group was written by another warp, after that warp's last meeting in the sum.
  __threadfence_block();
  __syncthreads();
  run = 0;
  for (int base = 0; base < n; base += kScanThreads) {
    const int i = base + threadIdx.x;
    long long keys = 0;
    if (i < n) {
      const int g = p.kv_indptr[i];
      // (a length that was rewritten since the pages were counted may be the less: offsets never fall,
      // so no list is written in front of its buffer)
      keys = max(0LL, length_of(p, i) - (__ldcg(p.prefix_indptr + g + 1) - __ldcg(p.prefix_indptr + g)));
    }
    const long long end = run + scan_block(keys, part, &total);
    if (i < n) p.kv_indptr[i] = offset32(end - keys);
    run += total;
  }
  if (threadIdx.x == 0) p.kv_indptr[n] = offset32(run);
}

// Blocks (i, y): every kFillBlocks-th run of keys of row i's own list, and of group i's prefix.  The
// offsets are read from L2, as this kernel may have begun before they were written, and by one warp
// for its block: 500 rows of up to 290 pages take 10 us, 21 if every warp asks for the same few lines.
__global__ void __launch_bounds__(kThreads) lists_kernel(const SharedTableParams p) {
  __shared__ int own_skip, own_at, group_row, prefix_at, prefix_keys;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the offsets
  const int lane = threadIdx.x & 31;
  const int first = blockIdx.y * kThreads + threadIdx.x;
  auto fill = [&](const int32_t* row, int skip, long long n, int at, int32_t* list, long long room) {
    n = min(n, room - at);
    for (long long k = first; k < n; k += kThreads * kFillBlocks) {  // (a step behind 2^31 - 1 keys is behind them)
      const int key = skip + (int)k;
      const long long slot = (long long)__ldg(row + key / p.page_size) * p.page_size + key % p.page_size;
      list[at + k] = slot < 0 || slot > 0x7fffffffLL ? -1 : (int32_t)slot;
    }
  };
  for (int i = blockIdx.x; i < p.batch; i += gridDim.x) {
    if (threadIdx.x < 32) {
      // The row's group: the last one that opens at or before it (32 probes at a time).
      int g = 0;
      for (int n = p.batch; n > 1;) {
        const int s = (n + 31) / 32;
        const bool below = lane * s < n && __ldcg(p.group_indptr + g + lane * s) <= i;
        const int k = __popc(__ballot_sync(0xffffffffu, below));
        const int at = max(k - 1, 0) * s;
        g += at;
        n = min(s, n - at);
      }
      if (lane == 0) {
        own_skip = __ldcg(p.prefix_indptr + g + 1) - __ldcg(p.prefix_indptr + g);
        own_at = __ldcg(p.kv_indptr + i);
        group_row = __ldcg(p.group_indptr + i);
        prefix_at = __ldcg(p.prefix_indptr + i);
        prefix_keys = __ldcg(p.prefix_indptr + i + 1) - prefix_at;
      }
    }
    __syncthreads();
    fill(p.block_table + (size_t)i * p.max_blocks, own_skip, length_of(p, i) - own_skip, own_at, p.kv_indices, p.capacity);
    if (group_row < p.batch)
      fill(p.block_table + (size_t)group_row * p.max_blocks, 0, prefix_keys, prefix_at, p.prefix_indices,
           p.prefix_capacity);
    __syncthreads();  // (before the next row's)
  }
}

// A small table in one block: a warp a row.  16 rows of 60 pages take 16 us a call instead of 24, two
// launches less of the host's time; lists of more than 64K entries would take one block longer than that.
constexpr int kSmallRows = 64;
constexpr long long kSmallKeys = 1 << 16;

__global__ void __launch_bounds__(kScanThreads) small_tables_kernel(const SharedTableParams p) {
  __shared__ int pages[kSmallRows], group[kSmallRows], opens[kSmallRows + 1], prefix[kSmallRows + 1], own[kSmallRows + 1];
  const int n = p.batch, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kWarps = kScanThreads / 32;
  for (int i = warp; i < n; i += kWarps) {
    int differ = i > 0 ? (int)(min(length_of(p, i - 1), length_of(p, i)) / p.page_size) : 0;
    const int32_t* a = p.block_table + (size_t)i * p.max_blocks;
    const int most = differ;
    for (int k = lane; k < most; k += 32)
      if (__ldg(a + k) != __ldg(a + k - p.max_blocks)) differ = min(differ, k);
    differ = __reduce_min_sync(0xffffffffu, differ);
    if (lane == 0) {
      pages[i] = differ;
      own[i] = (int)length_of(p, i);  // (at most kSmallKeys)
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    const long long least = p.min_shared > 1 ? p.min_shared : 1;
    int g = -1;
    for (int i = 0; i < n; ++i) {
      if (i == 0 || (long long)pages[i] * p.page_size < least) {
        opens[++g] = i;
        prefix[g] = -1;
      } else {
        prefix[g] = prefix[g] < 0 ? pages[i] : min(prefix[g], pages[i]);
      }
      group[i] = g;
    }
    int at = 0, next = 0;
    for (int i = 0; i <= g; ++i) {  // (the least pages become the offsets of the prefixes)
      const int keys = max(prefix[i], 0) * p.page_size;
      prefix[i] = at;
      at += keys;
    }
    for (int i = g + 1; i <= n; ++i) opens[i] = n, prefix[i] = at;
    for (int i = 0; i < n; ++i) {
      const int keys = max(0, own[i] - (prefix[group[i] + 1] - prefix[group[i]]));  // (as in groups_kernel)
      own[i] = next;
      next += keys;
    }
    own[n] = next;
  }
  __syncthreads();
  if (threadIdx.x <= n) {
    p.group_indptr[threadIdx.x] = opens[threadIdx.x];
    p.prefix_indptr[threadIdx.x] = prefix[threadIdx.x];
    p.kv_indptr[threadIdx.x] = own[threadIdx.x];
  }
  auto fill = [&](const int32_t* row, int skip, int from, int to, int32_t* list, long long room) {
    for (int at = from + lane; at < min((long long)to, room); at += 32) {
      const int key = skip + at - from;
      const long long slot = (long long)__ldg(row + key / p.page_size) * p.page_size + key % p.page_size;
      list[at] = slot < 0 || slot > 0x7fffffffLL ? -1 : (int32_t)slot;
    }
  };
  for (int i = warp; i < 2 * n; i += kWarps) {
    if (i < n) {
      const int shared = prefix[group[i] + 1] - prefix[group[i]];
      fill(p.block_table + (size_t)i * p.max_blocks, shared, own[i], own[i + 1], p.kv_indices, p.capacity);
    } else if (opens[i - n] < n) {
      fill(p.block_table + (size_t)opens[i - n] * p.max_blocks, 0, prefix[i - n], prefix[i - n + 1], p.prefix_indices,
           p.prefix_capacity);
    }
  }
}

template <typename Kernel>
cudaError_t launch_after(Kernel kernel, dim3 grid, int threads, const SharedTableParams& p, cudaStream_t stream) {
  // A programmatic dependent: its launch overlaps the tail of the one before.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_shared_tables(const SharedTableParams& p, cudaStream_t stream) {
  if (p.batch <= kSmallRows && (long long)p.batch * p.max_blocks * p.page_size <= kSmallKeys) {
    small_tables_kernel<<<1, kScanThreads, 0, stream>>>(p);
    return cudaGetLastError();
  }
  const int rows = p.batch < 65535 ? (p.batch > 0 ? p.batch : 1) : 65535;
  common_pages_kernel<<<rows, kThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = launch_after(groups_kernel, dim3(1), kScanThreads, p, stream);
  if (e == cudaSuccess && p.batch > 0) e = launch_after(lists_kernel, dim3(rows, kFillBlocks), kThreads, p, stream);
  return e;
}

}  // namespace mla
