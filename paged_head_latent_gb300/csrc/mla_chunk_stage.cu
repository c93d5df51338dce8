// mla_chunk_stage.cu -- what runs before and after the chunk attention: the call's keys as
// bf16 tiles, the plan, and the merge of split blocks.
#include "chunk.h"
#include "ptx.cuh"

namespace mla {
namespace {

constexpr int kStageThreads = 512;
constexpr int kNear = 1024;  // entries of the plan's tables that are kept in shared memory too
constexpr int kBlockCost = 2;  // cost units (tiles) of starting a block: its Q load and its output

struct ChunkReq {
  int q0, q_len, k0, kv_len;
  int tile0;  // first staged tile
};

// Offsets are clamped, so corrupt ones lead to no access outside the buffers.  Request b's
// keys start at staged tile ceil(k0 / 128) + b: since ceil(k1 / 128) - ceil(k0 / 128) + 1
// is at least ceil((k1 - k0) / 128), requests do not overlap, and no prefix sum is needed.
__device__ __forceinline__ ChunkReq load_request(const ChunkParams& p, int b) {
  ChunkReq r;
  const int k0 = min(max(__ldg(p.kv_indptr + b), 0), p.num_kv_indices);
  const int k1 = min(max(__ldg(p.kv_indptr + b + 1), k0), p.num_kv_indices);
  r.k0 = k0;
  r.kv_len = k1 - k0;
  r.q0 = min(max(__ldg(p.qo_indptr + b), 0), p.total_q);
  r.q_len = min(max(__ldg(p.qo_indptr + b + 1), r.q0), p.total_q) - r.q0;
  r.tile0 = (k0 + kChunkKeys - 1) / kChunkKeys + b;
  return r;
}

// One block: the list of row blocks with their running cost, and every worker's start.
// Blocks follow one another in row order; a block costs kBlockCost + its tiles, and worker
// w takes the tiles whose cost units lie in [w C / G, (w + 1) C / G).
__device__ void plan(const ChunkParams& p) {
  __shared__ long long part[kStageThreads / 32];
  __shared__ int near_first[kNear];
  __shared__ long long near_cost[kNear];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto scan = [&](long long v, long long* total) {  // exclusive sum over the block
    long long incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kStageThreads / 32; ++i) {
      if (i < warp) before += part[i];
      all += part[i];
    }
    __syncthreads();
    *total = all;
    return before + incl - v;
  };
  auto first_of = [&](int b) { return b < kNear ? near_first[b] : p.first_block[b]; };
  auto cost_of = [&](int i) { return i < kNear ? near_cost[i] : p.blocks[i].cost0; };
  long long run = 0, total;
  for (int base = 0; base < p.batch; base += kStageThreads) {
    const int b = base + threadIdx.x;
    long long n = 0;
    if (b < p.batch) n = ((long long)load_request(p, b).q_len * p.heads + kChunkRows - 1) / kChunkRows;
    const int at = (int)(run + scan(n, &total));
    if (b < p.batch) {
      if (b < kNear) near_first[b] = at;
      else p.first_block[b] = at;
    }
    run += total;
  }
  const int nblocks = (int)min(run, (long long)p.max_blocks);  // (offsets that overlap could name more)
  __syncthreads();
  long long cost = 0;
  for (int base = 0; base < nblocks; base += kStageThreads) {
    const int i = base + threadIdx.x;
    ChunkBlock blk{};
    if (i < nblocks) {
      int lo = 0, hi = p.batch - 1;  // last request whose first block is <= i
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first_of(mid) <= i) lo = mid; else hi = mid - 1;
      }
      const ChunkReq r = load_request(p, lo);
      blk.local0 = (i - first_of(lo)) * kChunkRows;
      blk.row0 = r.q0 * p.heads + blk.local0;
      blk.rows = min(kChunkRows, r.q_len * p.heads - blk.local0);
      blk.tile0 = r.tile0;
      blk.seen = r.kv_len - r.q_len + 1;
      const int last = blk.seen + (blk.local0 + blk.rows - 1) / p.heads;  // keys of the last row
      blk.tiles = last > 0 ? (last + kChunkKeys - 1) / kChunkKeys : 1;
    }
    blk.cost0 = cost + scan(i < nblocks ? blk.tiles + kBlockCost : 0, &total);
    if (i < nblocks) {
      p.blocks[i] = blk;
      if (i < kNear) near_cost[i] = blk.cost0;
    }
    cost += total;
  }
  __syncthreads();
  for (int w = threadIdx.x; w <= p.workers; w += kStageThreads) {
    ChunkStart s{nblocks, 0};
    const long long x = (long long)w * cost / p.workers;
    if (w < p.workers && x < cost) {
      int lo = 0, hi = nblocks - 1;  // last block whose cost0 is <= x
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cost_of(mid) <= x) lo = mid; else hi = mid - 1;
      }
      s.i = lo;
      s.t = (int)max(0LL, x - cost_of(lo) - kBlockCost);
    }
    p.starts[w] = s;
  }
}

// One block per staged tile (and one more for the plan): 128 keys of one request, read
// through their slots, dequantised to the bf16 numbers that the cache stands for.  Rows past
// the request's keys, slots outside the cache and keys with a value that is not finite
// are written as zeros, so that a weight of zero always makes a zero product; the tile's
// flags tell which rows are keys and which of them were not finite.
__global__ void __launch_bounds__(kStageThreads) chunk_stage_kernel(const ChunkParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x == 0) {
    plan(p);
    return;
  }
  __shared__ uint32_t flags[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tile = blockIdx.x - 1;
  // The request: the last one whose first tile is <= tile (32 probes at a time).
  int lo = 0, n = p.batch;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int b = lo + lane * step;
    const bool below = lane * step < n &&
        (min(max(__ldg(p.kv_indptr + b), 0), p.num_kv_indices) + kChunkKeys - 1) / kChunkKeys + b <= tile;
    const int k = __popc(__ballot_sync(0xffffffffu, below));
    const int at = max(k - 1, 0) * step;
    lo += at;
    n = min(step, n - at);
  }
  const ChunkReq r = load_request(p, lo);
  const int key0 = (tile - r.tile0) * kChunkKeys;
  const int here = min(kChunkKeys, r.kv_len - key0);
  // (a request without keys has one tile of zeros: its rows' weights are zero)
  if ((here <= 0 && key0 != 0) || key0 < 0 || r.q_len == 0) return;
  constexpr int kTok = kChunkKeys * 32 / kStageThreads;  // a warp's tokens, all in flight
  const int k0 = warp * kTok;
  int mine = -1;
  if (lane < kTok && k0 + lane < here) mine = __ldg(p.kv_indices + r.k0 + key0 + k0 + lane);
  if (threadIdx.x < 8) flags[threadIdx.x] = 0;
  __syncthreads();
  if (mine >= p.num_slots) mine = -1;
  uint4 code[kTok], rope[kTok];
  float sc[kTok];
#pragma unroll
  for (int k = 0; k < kTok; ++k) {
    const int slot = __shfl_sync(0xffffffffu, mine, k);
    code[k] = rope[k] = make_uint4(0, 0, 0, 0);
    sc[k] = 0.f;
    if (slot < 0) continue;
    const uint8_t* tok = p.kv_fp8 + (size_t)slot * kFp8TokenBytes;
    code[k] = *reinterpret_cast<const uint4*>(tok + 16 * lane);
    sc[k] = *reinterpret_cast<const float*>(tok + kDimCkv + 4 * (lane >> 3));
    if (lane < 8) rope[k] = *reinterpret_cast<const uint4*>(tok + kDimCkv + 16 + 16 * lane);
  }
#pragma unroll
  for (int k = 0; k < kTok; ++k) {
    uint4 a = ptx::e4m3x8_scaled_to_bf16x8(make_uint2(code[k].x, code[k].y), sc[k]);
    uint4 b = ptx::e4m3x8_scaled_to_bf16x8(make_uint2(code[k].z, code[k].w), sc[k]);
    const uint32_t w[12] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, rope[k].x, rope[k].y, rope[k].z, rope[k].w};
    uint32_t odd = 0;
#pragma unroll
    for (int i = 0; i < 12; ++i) odd |= __vcmpeq2(w[i] & 0x7f807f80u, 0x7f807f80u);  // exponent all ones
    const bool bad = __any_sync(0xffffffffu, odd != 0);
    if (bad) a = b = rope[k] = make_uint4(0, 0, 0, 0);
    const size_t row = (size_t)tile * kChunkKeys + k0 + k;
    uint4* dst = reinterpret_cast<uint4*>(p.ckv + row * kDimCkv + 16 * lane);
    dst[0] = a;
    dst[1] = b;
    if (lane < 8) *reinterpret_cast<uint4*>(p.kpe + row * kDimKpe + 8 * lane) = rope[k];
    if (lane == 0 && bad) atomicOr(&flags[4 + ((k0 + k) >> 5)], 1u << ((k0 + k) & 31));
  }
  const unsigned keys = __ballot_sync(0xffffffffu, mine >= 0);
  if (lane == 0 && keys) atomicOr(&flags[k0 >> 5], keys << (k0 & 31));
  __syncthreads();
  if (threadIdx.x < 8) p.flags[(size_t)tile * 8 + threadIdx.x] = flags[threadIdx.x];
}

// Merge of split blocks.  Block (w, y): if worker w starts inside a block and holds its last
// tile, rows 8 y .. 8 y + 7 of that block, one warp a row: lse = log2 of the sum of the
// fragments' 2^lse, out = their average with those weights, in worker order.
constexpr int kMergeRows = 8;

__global__ void __launch_bounds__(32 * kMergeRows) chunk_merge_kernel(const ChunkParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int w = blockIdx.x, lane = threadIdx.x & 31;
  const ChunkStart s = p.starts[w], e = p.starts[w + 1];
  if (s.t == 0 || e.i == s.i) return;  // starts a block, or the block goes on in the next worker
  const ChunkBlock blk = p.blocks[s.i];
  const int row = blockIdx.y * kMergeRows + (threadIdx.x >> 5);
  if (row >= blk.rows) return;
  // The block's first worker: the last one that starts before the block or at its tile 0.
  int first = w;
  for (bool found = false; !found;) {
    const int v = first - 1 - lane;
    const bool before = v < 0 || p.starts[v].i < s.i || p.starts[v].t == 0;
    const unsigned hit = __ballot_sync(0xffffffffu, before);
    found = hit != 0;
    first = found ? max(first - __ffs(hit), 0) : first - 32;
  }
  // Lane f has the f-th fragment's place and lse (-inf: no fragment) of 32 at a time.
  float top = -INFINITY, sum = 0.f, acc[16];
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  for (int v0 = first; v0 <= w; v0 += 32) {
    const int v = v0 + lane;
    size_t frag = 0;
    float l = -INFINITY;
    if (v <= w) {
      const ChunkStart a = p.starts[v], b = p.starts[v + 1];
      frag = ((size_t)v * 2 + (a.i == s.i ? 0 : 1)) * kChunkRows;
      if (a.i != b.i || a.t != b.t) l = p.part_lse[frag + row];
    }
    nan |= __any_sync(0xffffffffu, l != l);
    float m = l;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (m > top) {  // (uniform) the earlier fragments' share shrinks
      const float shrink = exp2f(top - m);
      sum *= shrink;
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[i] *= shrink;
      top = m;
    }
    const float weight = l > -INFINITY ? exp2f(l - top) : 0.f;
    unsigned todo = __ballot_sync(0xffffffffu, weight > 0.f);
    while (todo) {  // two fragments in flight
      const int f0 = __ffs(todo) - 1;
      todo &= todo - 1;
      const bool two = todo != 0;
      const int f1 = two ? __ffs(todo) - 1 : f0;
      const float w0 = __shfl_sync(0xffffffffu, weight, f0), w1 = __shfl_sync(0xffffffffu, weight, f1);
      todo &= todo - 1;
      const float4* o0 = reinterpret_cast<const float4*>(p.part_o + __shfl_sync(0xffffffffu, frag, f0) * kDimCkv) + row;
      const float4* o1 = reinterpret_cast<const float4*>(p.part_o + __shfl_sync(0xffffffffu, frag, f1) * kDimCkv) + row;
      float4 x[4], y[4];  // [column / 4][row]
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        x[q] = o0[(lane + 32 * q) * kChunkRows];
        y[q] = two ? o1[(lane + 32 * q) * kChunkRows] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      sum += w0;
      if (two) sum += w1;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        acc[4 * q] = fmaf(w1, y[q].x, fmaf(w0, x[q].x, acc[4 * q]));
        acc[4 * q + 1] = fmaf(w1, y[q].y, fmaf(w0, x[q].y, acc[4 * q + 1]));
        acc[4 * q + 2] = fmaf(w1, y[q].z, fmaf(w0, x[q].z, acc[4 * q + 2]));
        acc[4 * q + 3] = fmaf(w1, y[q].w, fmaf(w0, x[q].w, acc[4 * q + 3]));
      }
    }
  }
  const float inv = nan ? __int_as_float(0x7fc00000) : sum > 0.f ? 1.f / sum : 0.f;
  __nv_bfloat16* out = p.out + ((size_t)blk.row0 + row) * kDimCkv;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(acc[4 * q] * inv, acc[4 * q + 1] * inv);
    const __nv_bfloat162 b = __floats2bfloat162_rn(acc[4 * q + 2] * inv, acc[4 * q + 3] * inv);
    reinterpret_cast<uint2*>(out)[lane + 32 * q] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
  if (lane == 0)
    p.lse[(size_t)blk.row0 + row] = nan ? __int_as_float(0x7fc00000)
                                        : sum > 0.f ? 0.69314718055994531f * top + logf(sum) : -INFINITY;
}

}  // namespace

cudaError_t launch_chunk_stage(const ChunkParams& p, cudaStream_t stream) {
  chunk_stage_kernel<<<p.tiles + 1, kStageThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_chunk_merge(const ChunkParams& p, cudaStream_t stream) {
  // A programmatic dependent of the attention kernel: its launch overlaps that kernel's tail.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.workers, kChunkRows / kMergeRows);
  cfg.blockDim = dim3(32 * kMergeRows);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, chunk_merge_kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mla
