// mla_chunk_stage.cu -- what runs before and after the chunk attention: the call's keys as
// bf16 tiles, the plan, and the merge of split blocks.
#include "chunk.h"
#include "ptx.cuh"

namespace mla {
namespace {

constexpr int kStageThreads = 256;
constexpr int kStageKeys = 32;  // keys of a staging block: one word of the tile's flags
constexpr int kNear = 1024;  // entries of the plan's tables that are kept in shared memory too

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
// w takes the tiles whose cost units lie in [w C / G, (w + 1) C / G); a start in a block's
// leading units is the block's first tile.
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
    const int at = (int)min(run + scan(n, &total), 0x7fffffffLL);  // (overlapping offsets: see nblocks)
    if (b < p.batch) {
      if (b < kNear) near_first[b] = at;
      else p.first_block[b] = at;
    }
    run += total;
  }
  // Offsets that overlap could name more blocks than there is room for, even more than an int holds.
  const int nblocks = (int)min(run, (long long)p.max_blocks);
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
  // At most one worker for each cost unit, so that two starts inside a block are never the same.
  const long long G = min((long long)p.workers, max(cost, 1LL));
  auto start_of = [&](long long w) { return w < G ? w * cost / G : cost; };
  for (int w = threadIdx.x; w <= p.workers; w += kStageThreads) {
    ChunkStart s{nblocks, 0, ChunkBlock{}};
    ChunkMerge m{0, 0, 0, 0};
    const long long x = start_of(w);
    if (x < cost) {
      int lo = 0, hi = nblocks - 1;  // last block whose cost0 is <= x
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cost_of(mid) <= x) lo = mid; else hi = mid - 1;
      }
      const long long c0 = cost_of(lo);
      s.i = lo;
      s.t = (int)max(0LL, x - c0 - kBlockCost);
      s.blk = p.blocks[lo];
      if (s.t > 0 && start_of(w + 1) >= c0 + kBlockCost + s.blk.tiles) {  // a split block's last tile
        m.row0 = s.blk.row0;
        m.rows = s.blk.rows;
        m.first = (int)(((c0 + kBlockCost + 1) * G - 1) / cost);  // the worker of the block's first tile
        m.slot = start_of(m.first) >= c0 ? 0 : 1;  // its own first block, or one after others
      }
    }
    p.starts[w] = s;
    if (w < p.workers) p.merges[w] = m;
  }
}

// Block 0 makes the plan.  The others take parts of staged tiles: 32 keys of one request, read
// through their slots, as the bf16 numbers that the cache holds or (kFp8) stands for.  Rows past
// the request's keys, slots outside the cache and keys with a value that is not finite
// are written as zeros, so that a weight of zero always makes a zero product; the tile's
// flags tell which rows are keys and which of them were not finite.  301K FP8 keys (545 MB) take
// 95 us, 5.7 TB/s (with one block of 128 keys a tile 115 us: one block an SM, nothing to cover its
// waits); 16K keys of short requests 7 us, four dependent round trips (offsets, slots, tokens,
// the store) and the launch; a buffer of 524K indices for 32K keys costs 1 us more.  The plan of
// 2059 blocks takes about 13 us beside it.
template <bool kFp8>
__global__ void __launch_bounds__(kStageThreads) chunk_stage_kernel(const ChunkParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x == 0) {
    plan(p);
    return;
  }
  __shared__ uint32_t is_key, is_odd;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kParts = kChunkKeys / kStageKeys;
  // The list of keys may be shorter than its buffer: only the tiles in use are walked.
  const int used = min(max(__ldg(p.kv_indptr + p.batch), 0), p.num_kv_indices);
  const int parts = min(p.tiles, (used + kChunkKeys - 1) / kChunkKeys + p.batch) * kParts;
  for (int at_part = blockIdx.x - 1; at_part < parts; at_part += gridDim.x - 1) {
    const int tile = at_part / kParts, first = at_part % kParts * kStageKeys;
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
    if ((here <= 0 && key0 != 0) || key0 < 0 || r.q_len == 0) continue;
    constexpr int kTok = kStageKeys * 32 / kStageThreads;  // a warp's tokens, all in flight
    const int k0 = first + warp * kTok;
    int mine = -1;
    if (lane < kTok && k0 + lane < here) mine = __ldg(p.kv_indices + r.k0 + key0 + k0 + lane);
    __syncthreads();  // (the flags of the last round are written)
    if (threadIdx.x == 0) is_key = is_odd = 0;
    __syncthreads();
    if (mine >= p.num_slots) mine = -1;
    uint4 lat[kTok][kFp8 ? 1 : 2], rope[kTok];  // lane: latent values 16 lane .. + 15, rope values 8 lane .. + 7
    float sc[kTok];
#pragma unroll
    for (int k = 0; k < kTok; ++k) {
      const int slot = __shfl_sync(0xffffffffu, mine, k);
      lat[k][0] = lat[k][kFp8 ? 0 : 1] = rope[k] = make_uint4(0, 0, 0, 0);
      sc[k] = 0.f;
      if (slot < 0) continue;
      if constexpr (kFp8) {
        const uint8_t* tok = p.kv_fp8 + (size_t)slot * kFp8TokenBytes;
        lat[k][0] = *reinterpret_cast<const uint4*>(tok + 16 * lane);
        sc[k] = *reinterpret_cast<const float*>(tok + kDimCkv + 4 * (lane >> 3));
        if (lane < 8) rope[k] = *reinterpret_cast<const uint4*>(tok + kDimCkv + 16 + 16 * lane);
      } else {
        const uint4* tok = reinterpret_cast<const uint4*>(p.ckv_cache + (size_t)slot * kDimCkv + 16 * lane);
        lat[k][0] = tok[0];
        lat[k][1] = tok[1];
        if (lane < 8) rope[k] = *reinterpret_cast<const uint4*>(p.kpe_cache + (size_t)slot * kDimKpe + 8 * lane);
      }
    }
#pragma unroll
    for (int k = 0; k < kTok; ++k) {
      uint4 a, b;
      if constexpr (kFp8) {
        a = ptx::e4m3x8_scaled_to_bf16x8(make_uint2(lat[k][0].x, lat[k][0].y), sc[k]);
        b = ptx::e4m3x8_scaled_to_bf16x8(make_uint2(lat[k][0].z, lat[k][0].w), sc[k]);
      } else {
        a = lat[k][0];
        b = lat[k][1];
      }
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
      if (lane == 0 && bad) atomicOr(&is_odd, 1u << ((k0 + k) & 31));
    }
    const unsigned keys = __ballot_sync(0xffffffffu, mine >= 0);
    if (lane == 0 && keys) atomicOr(&is_key, keys << (k0 & 31));
    __syncthreads();
    if (threadIdx.x == 0) {
      p.flags[(size_t)tile * 8 + first / 32] = is_key;
      p.flags[(size_t)tile * 8 + 4 + first / 32] = is_odd;
    }
  }
}

// Merge of split blocks.  Block (w, y): of the split block that worker w ends, if any, rows
// 32 (y / 4) .. + 31 and columns 128 (y % 4) .. + 127.  A lane has a row and 16 columns, so a
// fragment ([column / 4][row][4]) is read 512 contiguous bytes at a time and an output sector is
// written whole, and a row's running maximum and sum need no other lane.  Fragments are added
// in worker order, the next two under way.  It adds 4 us to 32 blocks of drafted tokens and 9 us
// to two long chunks (40 MB of fragments); a row to a warp, with the same reads 16 bytes at a
// time, added 13 and 17.
constexpr int kMergeThreads = 256, kMergeParts = 16;
static_assert(sizeof(ChunkMerge) == 16, "read as one word");

__global__ void __launch_bounds__(kMergeThreads) chunk_merge_kernel(const ChunkParams p) {
  const int w = blockIdx.x;
  // (the plan is older than the attention kernel, whose end the wait is for)
  const int4 plan = __ldcg(reinterpret_cast<const int4*>(p.merges + w));
  const ChunkMerge blk{plan.x, plan.y, plan.z, plan.w};
  const int row = 32 * (blockIdx.y >> 2) + (threadIdx.x & 31);
  const int col = 128 * (blockIdx.y & 3) + 16 * (threadIdx.x >> 5);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (row >= blk.rows) return;
  const int n = w - blk.first + 1;
  float top = -INFINITY, sum = 0.f, acc[16], l[2];
  float4 x[2][4];
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  auto fetch = [&](int f, int k) {
    if (f >= n) return;
    const size_t frag = ((size_t)(blk.first + f) * 2 + (f == 0 ? blk.slot : 0)) * kChunkRows;
    l[k] = p.part_lse[frag + row];
    const float4* o = reinterpret_cast<const float4*>(p.part_o + frag * kDimCkv) + (col / 4) * kChunkRows + row;
#pragma unroll
    for (int q = 0; q < 4; ++q) x[k][q] = o[q * kChunkRows];
  };
  auto add = [&](int f, int k) {
    if (f >= n) return;
    nan |= l[k] != l[k];
    if (!(l[k] > -INFINITY)) return;
    const float m = fmaxf(top, l[k]), shrink = exp2f(top - m), g = exp2f(l[k] - m);
    top = m;
    sum = fmaf(sum, shrink, g);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      acc[4 * q] = fmaf(acc[4 * q], shrink, g * x[k][q].x);
      acc[4 * q + 1] = fmaf(acc[4 * q + 1], shrink, g * x[k][q].y);
      acc[4 * q + 2] = fmaf(acc[4 * q + 2], shrink, g * x[k][q].z);
      acc[4 * q + 3] = fmaf(acc[4 * q + 3], shrink, g * x[k][q].w);
    }
  };
  fetch(0, 0);
  fetch(1, 1);
  for (int f = 0; f < n; f += 2) {
    add(f, 0);
    fetch(f + 2, 0);
    add(f + 1, 1);
    fetch(f + 3, 1);
  }
  const float inv = nan ? __int_as_float(0x7fc00000) : sum > 0.f ? 1.f / sum : 0.f;
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    o[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  uint4* out = reinterpret_cast<uint4*>(p.out + ((size_t)blk.row0 + row) * kDimCkv + col);
  out[0] = make_uint4(o[0], o[1], o[2], o[3]);
  out[1] = make_uint4(o[4], o[5], o[6], o[7]);
  if (col == 0)
    p.lse[(size_t)blk.row0 + row] = nan ? __int_as_float(0x7fc00000)
                                        : sum > 0.f ? fmaf(top, 0.69314718055994531f, logf(sum)) : -INFINITY;
}

}  // namespace

cudaError_t launch_chunk_stage(const ChunkParams& p, bool fp8, cudaStream_t stream) {
  // Blocks walk the parts in use, so a buffer longer than its list costs little.  With a block for
  // every part of the buffer and no loop the whole call takes 170 us instead of 172 for 301K keys and
  // 980 instead of 988 for 2.1 million, but 47 instead of 34 for 32K keys in a buffer of 524K, and
  // 93 instead of 34 in one of 2 million (one token a request, 16 heads); caps of 64 and 128
  // blocks an SM gain nothing on the full lists and take 40 and 47 on the third.
  const int parts = p.tiles * (kChunkKeys / kStageKeys);  // (tiles * 128 is below 2^31)
  const int grid = 1 + (parts < 152 * 32 ? parts : 152 * 32);
  if (fp8) chunk_stage_kernel<true><<<grid, kStageThreads, 0, stream>>>(p);
  else chunk_stage_kernel<false><<<grid, kStageThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_chunk_merge(const ChunkParams& p, cudaStream_t stream) {
  // A programmatic dependent of the attention kernel: its launch overlaps that kernel's tail.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.workers, kMergeParts);
  cfg.blockDim = dim3(kMergeThreads);
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
