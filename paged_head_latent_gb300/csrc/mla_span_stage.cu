// mla_span_stage.cu -- what runs before the window and the shared attention: their keys as
// bf16 tiles of 128, and the plan.  (The attention is mla_chunk.cu's, the merge
// mla_chunk_stage.cu's.)
#include "chunk.h"
#include "ptx.cuh"

namespace mla {
namespace {

constexpr int kStageThreads = 256;
constexpr int kStageKeys = 32;  // keys of a staging block: one word of the tile's flags
constexpr int kNear = 1024;     // entries of the plan's tables that are kept in shared memory too
constexpr int kBlockCost = 3;   // cost units (tiles) of starting a block, as in the staged prefill

__device__ __forceinline__ int key_tiles(int keys) { return (keys + kChunkKeys - 1) / kChunkKeys; }

// Offsets are clamped, so corrupt ones lead to no access outside the buffers.
__device__ __forceinline__ int clamped(const int32_t* ptr, int i, int most) { return min(max(__ldg(ptr + i), 0), most); }

// Requests: their new tokens [q0, q0 + q_len) and their (own) keys [k0, k0 + kv_len).
struct SpanReq {
  int q0, q_len, k0, kv_len;
};
__device__ __forceinline__ SpanReq load_request(const ChunkParams& p, int b) {
  SpanReq r;
  r.k0 = clamped(p.kv_indptr, b, p.num_kv_indices);
  r.kv_len = max(clamped(p.kv_indptr, b + 1, p.num_kv_indices), r.k0) - r.k0;
  if (p.qo_indptr) {
    r.q0 = clamped(p.qo_indptr, b, p.total_q);
    r.q_len = max(clamped(p.qo_indptr, b + 1, p.total_q), r.q0) - r.q0;
  } else {
    r.q0 = b;
    r.q_len = 1;
  }
  return r;
}

// First staged tile of request b (kWindow: of its keys that any token sees), of group g's
// prefix.  As ceil(k1 / 128) - ceil(k0 / 128) + 1 >= ceil((k1 - k0) / 128), lists do not overlap.
__device__ __forceinline__ int request_tile0(const ChunkParams& p, int b) {
  if (p.per_request) return b * p.per_request + key_tiles(p.qo_indptr ? clamped(p.qo_indptr, b, p.total_q) : b);
  return p.prefix_tiles + key_tiles(clamped(p.kv_indptr, b, p.num_kv_indices)) + b;
}
__device__ __forceinline__ int prefix_tile0(const ChunkParams& p, int g) {
  return key_tiles(clamped(p.prefix_indptr, g, p.num_prefix)) + g;
}

// kWindow: the key tiles of a request that its tokens see: the first `head`, and from `rest` on.
struct SeenTiles {
  int low;   // first key of the first token's window
  int head, rest;
};
__device__ __forceinline__ SeenTiles seen_tiles(const ChunkParams& p, int seen_first, int seen_last) {
  SeenTiles s;
  s.low = max(0, max(seen_first, 0) - p.window);
  s.rest = s.low / kChunkKeys;
  s.head = min(key_tiles(min(p.sinks, max(seen_last, 0))), s.rest);
  return s;
}

// Exclusive sum over the block's threads.
struct Scan {
  long long* part;  // [kStageThreads / 32] shared
  __device__ long long operator()(long long v, long long* total) const {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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
  }
};

// Last i < n for which at(i) <= x, at ascending with at(0) <= x.
template <typename At, typename T>
__device__ __forceinline__ int last_at_most(int n, T x, At at) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (at(mid) <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// One block of threads: the list of row blocks with their running cost, and every worker's start,
// cut as in the staged prefill: a block costs kBlockCost + its tiles, and worker w takes the tiles
// whose cost units lie in [w C / G, (w + 1) C / G); a start in a block's leading units is the
// block's first tile.
template <int kSpan>
__device__ void plan(const ChunkParams& p) {
  __shared__ long long part[kStageThreads / 32];
  __shared__ int near_first[kNear], near_own[kNear];
  __shared__ long long near_cost[kNear];
  const Scan scan{part};
  const int lists = kSpan == kShared ? p.groups : p.batch;
  auto first_of = [&](int b) { return b < kNear ? near_first[b] : p.first_block[b]; };
  auto own_before = [&](int b) { return b < kNear ? near_own[b] : p.own_tiles[b]; };
  auto cost_of = [&](int i) { return i < kNear ? near_cost[i] : p.blocks[i].cost0; };
  // The first token of request b (kShared: its place among the queries).
  auto token_of = [&](int b) { return p.qo_indptr ? clamped(p.qo_indptr, b, p.total_q) : b; };
  long long run = 0, total;
  if constexpr (kSpan == kShared) {  // own tiles of the requests before each
    for (int base = 0; base < p.batch; base += kStageThreads) {
      const int b = base + threadIdx.x;
      int n = 0;
      if (b < p.batch) {
        const SpanReq r = load_request(p, b);
        n = r.q_len > 0 ? key_tiles(r.kv_len) : 0;
      }
      const int at = (int)min(run + scan(n, &total), 0x7fffffffLL);
      if (b < kNear) near_own[b] = at;
      else if (b < p.batch) p.own_tiles[b] = at;
      run += total;
    }
    run = 0;
  }
  // A list's rows: a request's tokens, or a group's.
  auto rows_of = [&](int b, int* row0) {
    long long t0, t1;
    if constexpr (kSpan == kShared) {
      const int g0 = clamped(p.group_indptr, b, p.batch), g1 = max(g0, clamped(p.group_indptr, b + 1, p.batch));
      t0 = token_of(g0);
      t1 = g1 > g0 ? max((int)t0, token_of(g1)) : (int)t0;
    } else {
      const SpanReq r = load_request(p, b);
      t0 = r.q0;
      t1 = r.q0 + r.q_len;
    }
    *row0 = (int)t0 * p.heads;
    return (t1 - t0) * p.heads;
  };
  for (int base = 0; base < lists; base += kStageThreads) {
    const int b = base + threadIdx.x;
    long long n = 0;
    int row0;
    if (b < lists) n = (rows_of(b, &row0) + kChunkRows - 1) / kChunkRows;
    const int at = (int)min(run + scan(n, &total), 0x7fffffffLL);  // (overlapping offsets: see nblocks)
    if (b < lists) {
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
      const int b = last_at_most(lists, i, first_of);
      blk.local0 = (i - first_of(b)) * kChunkRows;
      int row0;
      const long long rows = rows_of(b, &row0);
      blk.row0 = row0 + blk.local0;
      blk.rows = (int)min((long long)kChunkRows, rows - blk.local0);
      if constexpr (kSpan == kShared) {
        const int t0 = blk.row0 / p.heads, t1 = (blk.row0 + blk.rows - 1) / p.heads;  // first and last token
        auto request_of = [&](int t) { return p.qo_indptr ? last_at_most(p.batch, t, token_of) : t; };
        const int lo = request_of(t0), hi = max(lo, request_of(t1));
        const SpanReq r = load_request(p, hi);
        const int seen = min(r.kv_len, r.kv_len - r.q_len + 1 + t1 - r.q0);
        const int k0 = clamped(p.prefix_indptr, b, p.num_prefix);
        blk.head = key_tiles(max(clamped(p.prefix_indptr, b + 1, p.num_prefix), k0) - k0);
        blk.tile0 = prefix_tile0(p, b);
        blk.req = lo;
        blk.seen = 0x7fffffff;
        blk.tiles = blk.head + max(0, own_before(hi) - own_before(lo)) + key_tiles(max(seen, 0));
        if (blk.tiles == 0) {  // no row sees a key: the request's tile of zeros
          blk.head = blk.tiles = 1;
          blk.seen = 0;
          blk.tile0 = request_tile0(p, lo);
        }
      } else {
        const SpanReq r = load_request(p, b);
        blk.seen = r.kv_len - r.q_len + 1;
        const int first = blk.seen + blk.local0 / p.heads, last = blk.seen + (blk.local0 + blk.rows - 1) / p.heads;
        const SeenTiles all = seen_tiles(p, blk.seen, r.kv_len), s = seen_tiles(p, first, last);
        blk.tile0 = request_tile0(p, b);
        blk.head = s.head;
        blk.rest_key = s.rest;
        blk.rest0 = blk.tile0 + (p.per_request ? all.head + s.rest - all.rest : s.rest);
        blk.tiles = max(1, s.head + max(0, key_tiles(max(last, 0)) - s.rest));
      }
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
      const int lo = last_at_most(nblocks, x, cost_of);
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

// Where a staged tile's keys come from: entries [from, from + kChunkKeys) of a list, of which
// those in [low, end) and below `sinks` are keys that a row may see (numbers within the list).
struct TileSource {
  const int32_t* list;
  int from, low, sinks, end;
};

// The request or group that staged tile `tile` belongs to: the last one whose first tile is <= it
// (32 probes at a time; all lanes of the warp).
template <typename Tile0>
__device__ __forceinline__ int owner_of(int n, int tile, Tile0 tile0) {
  const int lane = threadIdx.x & 31;
  int lo = 0;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const bool below = lane * step < n && tile0(lo + lane * step) <= tile;
    const int k = __popc(__ballot_sync(0xffffffffu, below));
    const int at = max(k - 1, 0) * step;
    lo += at;
    n = min(step, n - at);
  }
  return lo;
}

// False if no block reads the tile.
template <int kSpan>
__device__ __forceinline__ bool tile_source(const ChunkParams& p, int tile, TileSource* s) {
  if (kSpan == kShared && tile < p.prefix_tiles) {
    const int g = owner_of(p.groups, tile, [&](int i) { return prefix_tile0(p, i); });
    const int k0 = clamped(p.prefix_indptr, g, p.num_prefix);
    s->list = p.prefix_indices + k0;
    s->from = (tile - prefix_tile0(p, g)) * kChunkKeys;
    s->low = s->sinks = 0;
    s->end = max(clamped(p.prefix_indptr, g + 1, p.num_prefix), k0) - k0;
    return s->from >= 0 && s->from < s->end && clamped(p.group_indptr, g + 1, p.batch) > clamped(p.group_indptr, g, p.batch);
  }
  const int b = owner_of(p.batch, tile, [&](int i) { return request_tile0(p, i); });
  const SpanReq r = load_request(p, b);
  const int at = tile - request_tile0(p, b);
  if (at < 0 || r.q_len == 0) return false;
  s->list = p.kv_indices + r.k0;
  s->end = r.kv_len;
  s->low = s->sinks = 0;
  int key_tile = at;
  if constexpr (kSpan == kWindow) {
    const SeenTiles t = seen_tiles(p, r.kv_len - r.q_len + 1, r.kv_len);
    if (p.per_request) key_tile = at < t.head ? at : at - t.head + t.rest;
    else if (at >= t.head && at < t.rest) return false;
    s->low = t.low;
    s->sinks = p.sinks;
  }
  s->from = (int)min((long long)key_tile * kChunkKeys, 0x7fffff80LL);
  // (a request without keys has one tile of zeros: its rows' weights are zero)
  return s->from < s->end || at == 0;
}

// Block 0 makes the plan.  The others take parts of staged tiles: 32 keys of one list, read
// through their slots, as the bf16 numbers that the cache holds or (kFp8) stands for.  Entries that
// are no keys, slots outside the cache and keys with a value that is not finite are written as
// zeros, so that a weight of zero always makes a zero product; the tile's flags tell which rows
// are keys and which of them were not finite.
template <bool kFp8, int kSpan>
__global__ void __launch_bounds__(kStageThreads) span_stage_kernel(const ChunkParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x == 0) {
    plan<kSpan>(p);
    return;
  }
  __shared__ uint32_t is_key, is_odd;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kParts = kChunkKeys / kStageKeys;
  // The lists may be shorter than their buffers: only the tiles in use are walked.
  int prefixes = 0;
  if constexpr (kSpan == kShared) prefixes = min(p.prefix_tiles, key_tiles(clamped(p.prefix_indptr, p.groups, p.num_prefix)) + p.groups);
  const int used = min(p.tiles, request_tile0(p, p.batch)) - p.prefix_tiles + prefixes;
  for (int at_part = blockIdx.x - 1; at_part < used * kParts; at_part += gridDim.x - 1) {
    const int nth = at_part / kParts, first = at_part % kParts * kStageKeys;
    const int tile = nth < prefixes ? nth : nth - prefixes + p.prefix_tiles;
    TileSource src;
    if (!tile_source<kSpan>(p, tile, &src)) continue;
    constexpr int kTok = kStageKeys * 32 / kStageThreads;  // a warp's tokens, all in flight
    const int k0 = first + warp * kTok;
    int mine = -1;
    if (lane < kTok) {
      const int key = src.from + k0 + lane;
      if (key < src.end && (key >= src.low || key < src.sinks)) mine = __ldg(src.list + key);
    }
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

// MLA_VALIDATE for the groups: group_indptr runs from 0 to the batch and prefix_indptr from 0 to the
// number of prefix indices, both without falling, and every prefix index is a slot of the cache.
__global__ void validate_groups_kernel(const ChunkParams p) {
  const int tid = blockIdx.x * blockDim.x + threadIdx.x, threads = gridDim.x * blockDim.x;
  bool bad = false;
  for (int g = tid; g <= p.groups; g += threads) {
    const int b = p.group_indptr[g], k = p.prefix_indptr[g];
    if (g == 0) bad |= b != 0 || k != 0;
    if (g == p.groups) bad |= b != p.batch || k != p.num_prefix;
    else bad |= p.group_indptr[g + 1] < b || p.prefix_indptr[g + 1] < k;
  }
  for (int i = tid; i < p.num_prefix; i += threads) {
    const int s = p.prefix_indices[i];
    bad |= s < 0 || s >= p.num_slots;
  }
  if (bad) atomicOr(p.status, kStatusBadIndex);
}

}  // namespace

cudaError_t launch_validate_groups(const ChunkParams& p, cudaStream_t stream) {
  validate_groups_kernel<<<64, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_span_stage(const ChunkParams& p, int span, bool fp8, cudaStream_t stream) {
  const int parts = p.tiles * (kChunkKeys / kStageKeys);  // (tiles * 128 is below 2^31)
  const int grid = 1 + (parts < 152 * 32 ? parts : 152 * 32);
  if (span == kWindow) {
    if (fp8) span_stage_kernel<true, kWindow><<<grid, kStageThreads, 0, stream>>>(p);
    else span_stage_kernel<false, kWindow><<<grid, kStageThreads, 0, stream>>>(p);
  } else {
    if (fp8) span_stage_kernel<true, kShared><<<grid, kStageThreads, 0, stream>>>(p);
    else span_stage_kernel<false, kShared><<<grid, kStageThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace mla
