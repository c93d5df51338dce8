// mla_span_stage.cu -- what runs before the window and the shared attention: their keys as
// bf16 rows, or where in the cache they are, and the plan.  (The attention is mla_chunk.cu's, the
// merge mla_chunk_stage.cu's.)
//
// A block of 128 query rows walks halves of 64 keys, two to a tile.  A half is 64 consecutive rows,
// staged ones or cache slots.  kShared: every list has halves of its own from its first key on.
// kWindow: a block's halves are those of the sinks in front of its first row's window, and those
// from that window's first key on (or, with p.aligned, from the multiple of 64 before it).
#include "chunk.h"
#include "ptx.cuh"

namespace mla {
namespace {

constexpr int kStageThreads = 256;
constexpr int kStageRows = 8;   // staged rows that a warp takes at a time: one byte of the flags
// Blocks of threads that run at a time.
constexpr int kStageBlocks = 152 * 2, kFp8Blocks = 152 * 3, kSourceBlocks = 152 * 4;
constexpr int kNear = 1024;     // entries of the plan's tables of lists that are kept in shared memory too
constexpr int kNearCost = 4096; // ... and of blocks

__device__ __forceinline__ int key_tiles(int keys) { return (keys + kChunkKeys - 1) / kChunkKeys; }
__device__ __forceinline__ int key_halves(int keys) { return (keys + kHalfKeys - 1) / kHalfKeys; }

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

// kShared: halves of a request's own keys.
__device__ __forceinline__ int own_halves(const SpanReq& r) { return r.q_len > 0 ? key_halves(r.kv_len) : 0; }
// ... and room for all of them.
__device__ __forceinline__ int own_room(const ChunkParams& p) { return (p.zero_row - p.prefix_tiles * kChunkKeys) / kHalfKeys; }

// First staged tile of request b's keys (kWindow: of those that any of its tokens sees), of group g's
// prefix.  As ceil(k1 / 128) - ceil(k0 / 128) + 1 >= ceil((k1 - k0) / 128), lists do not overlap.
__device__ __forceinline__ int request_tile0(const ChunkParams& p, int b) {
  if (p.per_request) return b * p.per_request + key_tiles(p.qo_indptr ? clamped(p.qo_indptr, b, p.total_q) : b);
  return key_tiles(clamped(p.kv_indptr, b, p.num_kv_indices)) + b;
}
__device__ __forceinline__ int prefix_tile0(const ChunkParams& p, int g) {
  return key_tiles(clamped(p.prefix_indptr, g, p.num_prefix)) + g;
}

// kWindow: the first key of the window of a token that sees `seen` keys (as halves begin there).
__device__ __forceinline__ int window_key(const ChunkParams& p, int seen) {
  const int low = max(0, max(seen, 0) - p.window);
  return p.aligned ? low & ~(kHalfKeys - 1) : low;
}
// kWindow: how a request's keys are staged, from its first token's count of keys: `head` halves of
// sinks, then the keys from `low` on; or, where sinks and window meet and in a layout with room for
// all keys, the keys from 0 on.
struct StagedKeys {
  int head, low;
};
__device__ __forceinline__ StagedKeys staged_keys(const ChunkParams& p, int seen) {
  const int low = window_key(p, seen);
  return low < p.sinks || !p.per_request ? StagedKeys{0, 0} : StagedKeys{key_halves(p.sinks), low};
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
  __shared__ long long near_cost[kNearCost];
  const Scan scan{part};
  const int lists = kSpan == kShared ? p.groups : p.batch;
  auto first_of = [&](int b) { return b < kNear ? near_first[b] : p.first_block[b]; };
  auto own_before = [&](int b) { return b < kNear ? near_own[b] : p.own_halves[b]; };
  auto cost_of = [&](int i) { return i < kNearCost ? near_cost[i] : p.blocks[i].cost0; };
  // The first token of request b (kShared: its place among the queries).
  auto token_of = [&](int b) { return p.qo_indptr ? clamped(p.qo_indptr, b, p.total_q) : b; };
  long long run = 0, total;
  if constexpr (kSpan == kShared) {  // own halves of the requests before each
    for (int base = 0; base < p.batch; base += kStageThreads) {
      const int b = base + threadIdx.x;
      int n = 0;
      if (b < p.batch) {
        const SpanReq r = load_request(p, b);
        n = own_halves(r);
      }
      const int at = (int)min(run + scan(n, &total), 0x7fffffffLL);
      if (b < kNear) near_own[b] = at;
      else if (b < p.batch) p.own_halves[b] = at;
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
  auto block_of = [&](int i) {
    ChunkBlock blk{};
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
      blk.head = key_halves(max(clamped(p.prefix_indptr, b + 1, p.num_prefix), k0) - k0);
      blk.tile0 = prefix_tile0(p, b) * kChunkKeys;
      // (offsets that overlap could name more halves than there is room for)
      const int before = min(own_before(lo), own_room(p)), own = max(0, own_before(hi) - own_before(lo));
      blk.rest0 = p.prefix_tiles * kChunkKeys + before * kHalfKeys;
      blk.halves = blk.head + min(own + min(key_halves(max(seen, 0)), own_halves(r)), own_room(p) - before);
    } else {
      const SpanReq r = load_request(p, b);
      blk.seen = r.kv_len - r.q_len + 1;
      const int first = blk.seen + blk.local0 / p.heads, last = blk.seen + (blk.local0 + blk.rows - 1) / p.heads;
      const StagedKeys all = staged_keys(p, blk.seen);
      blk.rest_key = window_key(p, first);
      blk.head = key_halves(min(p.sinks, blk.rest_key));
      blk.tile0 = request_tile0(p, b) * kChunkKeys;
      blk.rest0 = blk.tile0 + all.head * kHalfKeys + blk.rest_key - all.low;
      blk.halves = blk.head + key_halves(max(0, last - blk.rest_key));
    }
    blk.tiles = max(1, (blk.halves + 1) / 2);
    return blk;
  };
  long long cost = 0;
  int largest = 0;
  constexpr int kEach = 4;  // blocks of a thread between two sums
  for (int base = 0; base < nblocks; base += kStageThreads * kEach) {
    ChunkBlock blk[kEach];
    long long own = 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int i = base + threadIdx.x * kEach + e;
      if (i >= nblocks) continue;
      blk[e] = block_of(i);
      blk[e].cost0 = own;
      own += blk[e].tiles + kBlockCost;
      largest = max(largest, blk[e].tiles + kBlockCost);
    }
    const long long before = cost + scan(own, &total);
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int i = base + threadIdx.x * kEach + e;
      if (i >= nblocks) continue;
      blk[e].cost0 += before;
      p.blocks[i] = blk[e];
      if (i < kNearCost) near_cost[i] = blk[e].cost0;
    }
    cost += total;
  }
  // At most one worker for each cost unit, so that two starts inside a block are never the same.
  const long long G = min((long long)p.workers, max(cost, 1LL));
  // A worker to each block, if there are enough and the largest block is not far above a worker's share:
  // then no block is cut, and none has to be merged.
  const bool uncut = __syncthreads_and(nblocks <= G && (p.uncut || largest <= cost / G + kMergeCost));
  auto start_of = [&](long long w) { return uncut ? (w < nblocks ? cost_of((int)w) : cost) : w < G ? w * cost / G : cost; };
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

// Where staged rows from a multiple of 32 on (and to the next multiple of 64) come from: entries
// `from` .. of a list, of which those in [low, end) and those below `sinks` are keys that a row may see.
struct RowSource {
  const int32_t* list;
  int from, low, sinks, end;
  bool zero;    // the half of zeros: no list
  bool direct;  // every row that reads this half of 64 keys sees all of them
  HalfInfo info;  // kShared: of the half that begins here
  __device__ bool holds(int key) const { return key < end && (key >= low || key < sinks); }
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

// kShared: where every request's own halves begin.  Each block of threads makes the sums for itself,
// for up to kNear runs of requests.
struct OwnTable {
  int before[kNear + 1];  // halves before a run; all of them behind the last
  long long part[kStageThreads / 32];
  __device__ static int run_length(int batch) { return (batch + kNear - 1) / kNear; }
  __device__ void make(const ChunkParams& p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, each = run_length(p.batch);
    constexpr int kRuns = kNear / kStageThreads;
    long long n[kRuns], sum = 0;
#pragma unroll
    for (int i = 0; i < kRuns; ++i) {
      n[i] = sum;
      const int run = threadIdx.x * kRuns + i;
      for (int b = run * each; b < min((run + 1) * each, p.batch); ++b) sum += own_halves(load_request(p, b));
    }
    long long incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    long long base = incl - sum;
    for (int i = 0; i < warp; ++i) base += part[i];
    // (offsets that overlap could name more halves than there is room for)
    const long long room = own_room(p);
#pragma unroll
    for (int i = 0; i < kRuns; ++i) before[threadIdx.x * kRuns + i] = (int)min(base + n[i], room);
    if (threadIdx.x == kStageThreads - 1) before[kNear] = (int)min(base + sum, room);
    __syncthreads();
  }
  __device__ int total() const { return before[kNear]; }
  // The request that own half x belongs to; x becomes the number of the half among the request's.
  __device__ int find(const ChunkParams& p, int* x) const {
    const int run = last_at_most(kNear, *x, [&](int i) { return before[i]; }), each = run_length(p.batch);
    *x -= before[run];
    int b = run * each;
    for (; b < p.batch - 1; ++b) {
      const int n = own_halves(load_request(p, b));
      if (*x < n) break;
      *x -= n;
    }
    return b;
  }
};

// kShared: the source of rows of the prefixes' tiles, of the own halves or of the half of zeros.
// False if no block reads these rows.
__device__ __forceinline__ bool shared_source(const ChunkParams& p, const OwnTable& own, int row, RowSource* s) {
  s->low = s->sinks = 0;
  s->info = HalfInfo{0, 0, 0, 0};
  s->zero = false;
  const int prefix_rows = p.prefix_tiles * kChunkKeys;
  if (row < prefix_rows) {
    const int g = owner_of(p.groups, row / kChunkKeys, [&](int i) { return prefix_tile0(p, i); });
    const int k0 = clamped(p.prefix_indptr, g, p.num_prefix);
    s->list = p.prefix_indices + k0;
    s->from = row - prefix_tile0(p, g) * kChunkKeys;
    s->end = max(clamped(p.prefix_indptr, g + 1, p.num_prefix), k0) - k0;
    s->direct = true;  // (a block has rows of one group)
    s->info = HalfInfo{0, kMany, kMany, 0};
    return s->from >= 0 && s->from < key_halves(s->end) * kHalfKeys &&
           clamped(p.group_indptr, g + 1, p.batch) > clamped(p.group_indptr, g, p.batch);
  }
  int at = (row - prefix_rows) / kHalfKeys;
  if (at >= own.total()) {
    s->zero = true;
    s->from = s->end = 0;
    s->direct = false;
    return true;
  }
  const int b = own.find(p, &at);
  const SpanReq r = load_request(p, b);
  const int seen = r.kv_len - r.q_len + 1;  // keys that the first token sees
  s->list = p.kv_indices + r.k0;
  s->end = r.kv_len;
  s->from = at * kHalfKeys + row % kHalfKeys;
  s->info = HalfInfo{r.q0, r.q0 + r.q_len, seen - r.q0 - at * kHalfKeys, 0};
  // A block may have rows of several requests, if it is not filled by a token: then their own keys are
  // staged, as a key that is not finite must not reach the others' rows.  (64 requests of 4000 own
  // keys behind prefixes of 64, in 64-key pages: 173 us with 16 heads, 87 with 128, read in place.)
  s->direct = (at + 1) * kHalfKeys <= seen;
  if (s->direct && p.sources && p.heads != kChunkRows) {
    const int g = owner_of(p.groups, b, [&](int i) { return clamped(p.group_indptr, i, p.batch); });
    s->direct = clamped(p.group_indptr, g + 1, p.batch) - clamped(p.group_indptr, g, p.batch) == 1;
  }
  return true;
}

// kWindow: the source of rows of a request's keys.  False if no block reads these rows.
__device__ __forceinline__ bool window_source(const ChunkParams& p, int row, RowSource* s) {
  const int b = owner_of(p.batch, row / kChunkKeys, [&](int i) { return request_tile0(p, i); });
  const SpanReq r = load_request(p, b);
  const int at = row - request_tile0(p, b) * kChunkKeys;
  if (at < 0 || r.q_len == 0) return false;
  const int seen = r.kv_len - r.q_len + 1;  // keys that the first token sees
  s->list = p.kv_indices + r.k0;
  s->end = r.kv_len;
  s->from = at;
  s->low = max(0, max(seen, 0) - p.window);
  s->sinks = p.sinks;
  s->direct = r.q_len == 1;  // (a block has rows of one request)
  if (p.per_request) {
    const StagedKeys k = staged_keys(p, seen);
    if (at < k.head * kHalfKeys) return true;
    s->from = min(at - k.head * kHalfKeys, 0x7fffffff - k.low) + k.low;
    // (a half may start at any key and reach 63 rows past the last; without keys, one of zeros)
    return s->from < s->end || s->from - s->end < kHalfKeys - 1;
  }
  const int half = at & ~(kHalfKeys - 1);  // (halves of this layout start at multiples of 64 keys)
  if (half >= p.sinks && half + kHalfKeys <= s->low) return false;
  return s->from < max(key_halves(s->end), 1) * kHalfKeys;
}

// The staged rows in use, 32 or 64 at a time (the lists may be shorter than their buffers).
template <int kSpan>
struct StagedRows {
  int prefixes = 0, rows;  // rows in use, of the prefixes and in all
  __device__ StagedRows(const ChunkParams& p, OwnTable* own) {
    if constexpr (kSpan == kShared) {
      own->make(p);
      prefixes = min(p.prefix_tiles, key_tiles(clamped(p.prefix_indptr, p.groups, p.num_prefix)) + p.groups) * kChunkKeys;
      rows = prefixes + (own->total() + 1) * kHalfKeys;
    } else {
      rows = min(p.tiles, request_tile0(p, p.batch)) * kChunkKeys;
    }
  }
  // The staged row of the i-th row in use, and its source.
  __device__ bool source(const ChunkParams& p, const OwnTable* own, int i, int* row, RowSource* s) const {
    if constexpr (kSpan == kShared) {
      *row = i < prefixes ? i : i - prefixes + p.prefix_tiles * kChunkKeys;
      const bool used = shared_source(p, *own, *row, s);
      if (s->zero) *row = p.zero_row + *row % kHalfKeys;
      return used;
    } else {
      *row = i;
      return window_source(p, i, s);
    }
  }
};

// kTok (4 or 8) tokens of a warp on their way from the cache.  A lane has latent values 8 lane .. + 7 and
// 256 + 8 lane .. + 7 of each, and rope values 8 (lane % 8) .. + 7 of token lane / 8 of each four.
template <bool kFp8, int kTok>
struct Tokens {
  uint4 lat[kFp8 ? 1 : kTok][2], rope[kTok / 4];
  uint2 code[kFp8 ? kTok : 1][2];
  float scale[kFp8 ? kTok : 1][2];

  // Ask for the tokens in slots `mine` of lanes first .. first + kTok - 1 (outside the cache: zeros).
  __device__ __forceinline__ void ask(const ChunkParams& p, int mine, int first) {
    const int lane = threadIdx.x & 31;
    auto slot_of = [&](int k) {
      const int s = __shfl_sync(0xffffffffu, mine, first + k);
      return s < p.num_slots ? s : -1;
    };
#pragma unroll
    for (int k = 0; k < kTok; ++k) {
      const int slot = slot_of(k);
      if constexpr (kFp8) code[k][0] = code[k][1] = make_uint2(0, 0), scale[k][0] = scale[k][1] = 0.f;
      else lat[k][0] = lat[k][1] = make_uint4(0, 0, 0, 0);
      if (slot < 0) continue;
      if constexpr (kFp8) {
        const uint8_t* tok = p.kv_fp8 + (size_t)slot * kFp8TokenBytes;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          code[k][h] = *reinterpret_cast<const uint2*>(tok + 256 * h + 8 * lane);
          scale[k][h] = *reinterpret_cast<const float*>(tok + kDimCkv + 8 * h + 4 * (lane >> 4));
        }
      } else {
        const uint4* tok = reinterpret_cast<const uint4*>(p.ckv_cache + (size_t)slot * kDimCkv);
        lat[k][0] = tok[lane];
        lat[k][1] = tok[32 + lane];
      }
    }
#pragma unroll
    for (int i = 0; i < kTok / 4; ++i) {
      const int slot = slot_of(4 * i + (lane >> 3));
      rope[i] = make_uint4(0, 0, 0, 0);
      if (slot < 0) continue;
      const uint8_t* part;
      if constexpr (kFp8) part = p.kv_fp8 + (size_t)slot * kFp8TokenBytes + kDimCkv + 16;
      else part = reinterpret_cast<const uint8_t*>(p.kpe_cache + (size_t)slot * kDimKpe);
      rope[i] = reinterpret_cast<const uint4*>(part)[lane & 7];
    }
  }
  // Exponents of all ones among eight bf16 numbers.
  static __device__ __forceinline__ uint32_t odd_of(uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t odd = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) odd |= __vcmpeq2(w[i] & 0x7f807f80u, 0x7f807f80u);
    return odd;
  }
  // Write them to staged rows `row` .. + kTok - 1.  Returns, to all lanes, which of them hold a value that
  // is not finite (their values are written as zeros, so that a weight of zero always makes a
  // zero product).
  __device__ __forceinline__ uint32_t write(const ChunkParams& p, size_t row) {
    const int lane = threadIdx.x & 31;
    uint32_t rope_odd[kTok / 4], bad = 0;
#pragma unroll
    for (int i = 0; i < kTok / 4; ++i) rope_odd[i] = __ballot_sync(0xffffffffu, odd_of(rope[i]) != 0);
#pragma unroll
    for (int k = 0; k < kTok; ++k) {
      uint4 a, b;
      if constexpr (kFp8) {
        a = ptx::e4m3x8_scaled_to_bf16x8(code[k][0], scale[k][0]);
        b = ptx::e4m3x8_scaled_to_bf16x8(code[k][1], scale[k][1]);
      } else {
        a = lat[k][0];
        b = lat[k][1];
      }
      if (__any_sync(0xffffffffu, (odd_of(a) | odd_of(b)) != 0) || (rope_odd[k / 4] >> (8 * (k & 3)) & 0xffu)) {
        a = b = make_uint4(0, 0, 0, 0);
        bad |= 1u << k;
      }
      uint4* dst = reinterpret_cast<uint4*>(p.ckv + (row + k) * kDimCkv);
      dst[lane] = a;
      dst[32 + lane] = b;
    }
#pragma unroll
    for (int i = 0; i < kTok / 4; ++i)
      reinterpret_cast<uint4*>(p.kpe + (row + 4 * i) * kDimKpe)[lane] =
          bad >> (4 * i + (lane >> 3)) & 1u ? make_uint4(0, 0, 0, 0) : rope[i];
    return bad;
  }
};

// Block 0 makes the plan.  The others' warps take 8 staged rows at a time, of one list, read through
// their slots as the bf16 numbers that the cache holds or (kFp8) stands for.  Entries that are no
// keys and slots outside the cache are written as zeros; the flags tell which rows are keys and
// which of them were not finite.
//
// What bounds it: few keys, the chain of round trips (offsets, slots, tokens, the store): a warp asks
// for its next rows' slots while its tokens are on their way.  Many keys, memory: 158K FP8 keys
// (285 MB read and written) take 46 us, 6.2 TB/s.  (FP8 tokens eight at a time instead of four: 2 us
// more, by registers.)
template <bool kFp8, int kSpan>
__global__ void __launch_bounds__(kStageThreads, kFp8 ? 3 : 2) span_stage_kernel(const ChunkParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x == 0) {
    plan<kSpan>(p);
    return;
  }
  __shared__ OwnTable own;
  const int lane = threadIdx.x & 31, warps = (gridDim.x - 1) * (kStageThreads / 32);
  const StagedRows<kSpan> staged(p, &own);
  const int units = staged.rows / kStageRows;
  int row, next_row, mine, next_mine = -1;
  bool used, next_used;
  auto look = [&](int unit) {  // the unit's rows, and its slots in the first lanes
    RowSource src;
    next_used = staged.source(p, &own, unit * kStageRows, &next_row, &src);
    next_mine = -1;
    if (next_used) {
      const int key = src.from + lane;
      if (lane < kStageRows && src.holds(key)) next_mine = __ldg(src.list + key);
      if (kSpan == kShared && next_row % kHalfKeys == 0 && lane == 0) p.infos[next_row / kHalfKeys] = src.info;
    }
  };
  int unit = (blockIdx.x - 1) * (kStageThreads / 32) + (threadIdx.x >> 5);
  if (unit < units) look(unit);
  for (; unit < units; unit += warps) {
    row = next_row, mine = next_mine, used = next_used;
    constexpr int kTok = kFp8 ? kStageRows / 2 : kStageRows;
    Tokens<kFp8, kTok> x;
    if (used) x.ask(p, mine, 0);
    if (unit + warps < units) look(unit + warps);
    if (!used) continue;
    uint32_t bad = x.write(p, row);
    if (kTok < kStageRows) {
      x.ask(p, mine, kTok);
      bad |= x.write(p, (size_t)row + kTok) << kTok;
    }
    const uint32_t keys = __ballot_sync(0xffffffffu, mine >= 0 && mine < p.num_slots);
    if (lane == 0) {  // (a byte has the flags of 8 rows)
      reinterpret_cast<uint8_t*>(p.flags)[row / kStageRows] = (uint8_t)keys;
      reinterpret_cast<uint8_t*>(p.flags + (size_t)p.tiles * 4)[row / kStageRows] = (uint8_t)bad;
    }
  }
}

// The same where whole halves may be read from the cache (p.sources): a warp looks at a half's 64
// slots; if they are all keys of all rows that read it and follow one another, it notes the
// first.  The block's warps then copy the others together, eight rows each.
template <int kSpan>
__global__ void __launch_bounds__(kStageThreads, 4) span_source_kernel(const ChunkParams p, int halves_per_block) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x == 0) {
    plan<kSpan>(p);
    return;
  }
  constexpr int kWarps = kStageThreads / 32, kTok = kHalfKeys / kWarps;
  __shared__ int slots[kWarps][kHalfKeys], rows[kWarps];
  __shared__ uint32_t is_odd[kWarps][2];
  __shared__ OwnTable own;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const StagedRows<kSpan> staged(p, &own);
  const int halves = staged.rows / kHalfKeys;
  // A block's halves lie far from one another: those to be copied, at a list's ends, are neighbours.
  const int blocks = gridDim.x - 1;
  for (int first = blockIdx.x - 1; first < halves; first += blocks * halves_per_block) {
    int copy_row = -1;
    const int nth = first + warp * blocks;
    if (warp < halves_per_block && nth < halves) {
      int row;
      RowSource src;
      if (staged.source(p, &own, nth * kHalfKeys, &row, &src)) {
        if (kSpan == kShared && lane == 0) p.infos[row / kHalfKeys] = src.info;
        int s[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int key = src.from + 32 * h + lane;
          s[h] = src.holds(key) ? __ldg(src.list + key) : -1;
        }
        const int slot = __shfl_sync(0xffffffffu, s[0], 0);
        const bool run = src.direct && slot >= 0 && slot <= p.num_slots - kHalfKeys && s[0] == slot + lane &&
                         s[1] == slot + 32 + lane;
        if (__all_sync(0xffffffffu, run)) {
          if (lane == 0) p.sources[row / kHalfKeys] = slot;
        } else {
          copy_row = row;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            slots[warp][32 * h + lane] = s[h];
            const uint32_t keys = __ballot_sync(0xffffffffu, s[h] >= 0 && s[h] < p.num_slots);
            if (lane == 0) p.flags[row / 32 + h] = keys;
          }
          if (lane == 0) p.sources[row / kHalfKeys] = -1;
        }
      }
    }
    if (lane == 0) {
      rows[warp] = copy_row;
      is_odd[warp][0] = is_odd[warp][1] = 0;
    }
    __syncthreads();
    for (int i = 0; i < halves_per_block; ++i) {
      const int row = rows[i];
      if (row < 0) continue;
      const int mine = slots[i][warp * kTok + (lane & (kTok - 1))];
      Tokens<false, kTok / 2> x;
      x.ask(p, mine, 0);
      uint32_t bad = x.write(p, (size_t)row + warp * kTok);
      x.ask(p, mine, kTok / 2);
      bad |= x.write(p, (size_t)row + warp * kTok + kTok / 2) << (kTok / 2);
      if (lane == 0 && bad) atomicOr(&is_odd[i][warp / 4], bad << (warp % 4 * kTok));
    }
    __syncthreads();
    if (warp < halves_per_block && copy_row >= 0 && lane < 2)
      p.flags[(size_t)p.tiles * 4 + copy_row / 32 + lane] = is_odd[warp][lane];
    __syncthreads();  // (before the next round's rows)
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
  if (p.sources) {
    // As few halves to a block as fill the GPU, and a warp each at most.
    const int halves = p.tiles * 2, most = kStageThreads / 32;
    const int each = (int)min(((long long)halves + kSourceBlocks - 1) / kSourceBlocks, (long long)most);
    const int blocks = (halves + each - 1) / each, grid = 1 + (blocks < kSourceBlocks ? blocks : kSourceBlocks);
    if (span == kWindow) span_source_kernel<kWindow><<<grid, kStageThreads, 0, stream>>>(p, each);
    else span_source_kernel<kShared><<<grid, kStageThreads, 0, stream>>>(p, each);
    return cudaGetLastError();
  }
  const int blocks = (p.tiles * (kChunkKeys / kStageRows) + kStageThreads / 32 - 1) / (kStageThreads / 32);
  const int most = fp8 ? kFp8Blocks : kStageBlocks, grid = 1 + (blocks < most ? blocks : most);
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
