// chunk.h -- parameters of the chunk attention (mla_chunk.cu) and its staging pass.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "common.cuh"

namespace mla {

constexpr int kChunkKeys = 128;  // keys of a tile
constexpr int kChunkRows = 128;  // query rows (token, head) of a block
// Cost units (tiles) of starting a block: its Q load and its output.  Four prompts with 128 heads
// took 935, 881, 871 and 886 us at 1 to 4, 32 blocks of drafted tokens 24.7, 22.9, 22.7 and 23.9.
constexpr int kBlockCost = 3;
// ... and, in the window and the shared attention's plan, of writing and merging the fragments of cut
// blocks; tiles of a block that never pay a cut.
constexpr int kMergeCost = 6, kUncutTiles = kMergeCost - kBlockCost;

// Which keys a row sees.  kCausal: all of its request's keys up to its own token.  kWindow: of
// those the last `window` and the first `sinks`.  kShared: all keys of its group's prefix list,
// and of its request's own list those up to its own token.
enum { kCausal = 0, kWindow = 1, kShared = 2 };

// 128 consecutive query rows of one request (kShared: of one group); row 0 of request b is (token
// 0, head 0).  kCausal: its keys are tiles of 128 of the request's.  Else they are halves of 64,
// two to a tile, in two runs: kWindow, those with sinks and those from the first row's window
// on; kShared, the prefix's, then those of its requests' own keys (each list in halves of its own).
struct ChunkBlock {
  int row0;      // first row of the block in [total_q * H]
  int local0;    // ... and within its request (kShared: unused)
  int rows;      // rows in use, 1..128
  int tiles;     // key tiles that its rows see (at least 1)
  int tile0;     // kCausal: first staged tile of the request; else the staged row of the first run
  int seen;      // keys that token 0 of the request sees (may be <= 0; kShared: unused)
  // Halves: at most 2 * tiles, at least one less; but 0 for rows that see no key, which walk a tile all
  // the same (kWindow: the request's first half, masked; kShared: the half of zeros).  Causal: unused,
  // as what follows.
  int halves;
  int head;      // ... of the first run
  int rest0;     // staged row of the second run
  int rest_key;  // kWindow: ... and its first key's number in the request
  long long cost0;  // cost units before this block
};

// kShared: what a staged half is.  Token i of the call sees its keys below i + more if i is in [from, to).
struct HalfInfo {
  int from, to, more, pad;
};
constexpr int kMany = 1 << 30;  // more tokens or keys than there are

// Where a worker's range starts: tile t of block i (a copy of which saves a load's latency).
struct ChunkStart {
  int i, t;
  ChunkBlock blk;
};

// A split block that a worker holds the last tile of: its rows, the worker that holds its
// first tile (fragment slot 0 or 1 there, 0 everywhere else).
struct ChunkMerge {
  int row0, rows;  // rows = 0: none
  int first, slot;
};

struct ChunkParams {
  // the call
  const int32_t* qo_indptr;
  const int32_t* kv_indptr;
  const int32_t* kv_indices;
  const uint8_t* kv_fp8;            // FP8 cache, or
  const __nv_bfloat16* ckv_cache;   // bf16 caches
  const __nv_bfloat16* kpe_cache;
  __nv_bfloat16* out;  // [total_q * H, 512]
  float* lse;          // [total_q * H]
  int batch, heads, total_q, num_slots, num_kv_indices, workers;
  float scale_log2;
  // workspace
  uint32_t* status;
  ChunkStart* starts;   // [workers + 1]
  ChunkMerge* merges;   // [workers]
  int32_t* first_block; // [batch + 1]
  ChunkBlock* blocks;
  // kCausal: [tiles][8], a tile's 128 bits "is a key" and 128 bits "holds a value that is not finite";
  // else the first bits of all rows, [tiles * 4], then the second
  uint32_t* flags;
  // Half a tile's keys: the first of 64 consecutive cache slots that hold them, or -1: they are staged
  int32_t* sources;     // [tiles * 2], or null: all are staged
  __nv_bfloat16* ckv;   // [tiles * 128, 512] staged keys
  __nv_bfloat16* kpe;   // [tiles * 128, 64]
  float* part_lse;      // [workers][2][128] base-2 lse of partial fragments
  float* part_o;        // [workers][2][512 / 4][128 rows][4]
  int tiles;            // staged tiles (an upper bound from the host's sizes)
  // kWindow; kShared (qo_indptr may be null in both: a token per request)
  int window, sinks;
  int per_request;      // kWindow: tiles set aside for a request, or 0: for all of its keys
  int aligned;          // kWindow: the second run starts at a multiple of 64 keys (sources, or per_request = 0)
  bool uncut;           // known to the host: at most as many blocks as workers, of up to kUncutTiles; no merge
  const int32_t* group_indptr;   // [groups + 1] requests
  const int32_t* prefix_indptr;  // [groups + 1] prefix keys
  const int32_t* prefix_indices;
  int groups, num_prefix, prefix_tiles;  // prefix_tiles: staged tiles of the prefixes, before the own keys'
  int32_t* own_halves;  // [batch] own halves of the requests before each
  HalfInfo* infos;      // kShared: [tiles * 2]
  // kShared: the staged rows are the prefixes' tiles, the requests' own halves one after another, and
  // a half of zeros, for what is behind a block's last half or sees no key
  int zero_row;
  int max_blocks;       // room in blocks
  unsigned long long wait_ns;
  int fault_skip_tile;
};

// ---- where the staged keys of the window and the shared attention lie (host and device)
constexpr int kHalfKeys = 64;

// kWindow.  A request's keys that any of its tokens sees are at most `sinks` and window + q_len - 1
// more.  With tiles set aside for them, request b starts at staged tile b * per + ceil(q0 / 128),
// which needs no prefix sum: as 128 (ceil(q1 / 128) - ceil(q0 / 128)) >= q_len - 127, it has at least
// sinks + window + q_len + 129 rows; it needs the sinks in whole halves, the others from any key
// on, and 63 rows behind them that a half may reach into.
__host__ __device__ inline long long window_tiles_per_request(int window, int sinks) {
  return ((long long)sinks + kChunkKeys - 1) / kChunkKeys + ((long long)window + kChunkKeys - 1) / kChunkKeys + 2;
}

struct ChunkMaps {
  CUtensorMap q_nope, q_pe, ckv, kpe;  // boxes of 64 rows x 64 columns, 128-byte swizzle
  CUtensorMap cache_ckv, cache_kpe;    // ... of the caches, where p.sources is not null
};

struct ChunkLayout {
  size_t starts, merges, first_block, own_halves, blocks, flags, sources, infos, part_lse, part_o, ckv, kpe, total;
  long long tiles, max_blocks;
  ChunkLayout(int workers, int heads, int batch, int total_q, int num_kv_indices) {
    tiles = ((long long)num_kv_indices + kChunkKeys - 1) / kChunkKeys + batch;
    max_blocks = ((long long)total_q * heads + kChunkRows - 1) / kChunkRows + batch;
    place(workers, batch, 0, false);
  }
  void place(int workers, int lists, long long requests, bool spans) {
    starts = 256;
    merges = align_up(starts + ((size_t)workers + 1) * sizeof(ChunkStart), 256);
    first_block = align_up(merges + (size_t)workers * sizeof(ChunkMerge), 256);
    own_halves = align_up(first_block + ((size_t)lists + 1) * sizeof(int32_t), 256);
    blocks = align_up(own_halves + (size_t)requests * sizeof(int32_t), 256);
    flags = align_up(blocks + (size_t)max_blocks * sizeof(ChunkBlock), 256);
    sources = align_up(flags + (size_t)tiles * 32, 256);
    infos = align_up(sources + (spans ? (size_t)tiles * 8 : 0), 256);
    part_lse = align_up(infos + (requests ? (size_t)tiles * 2 * sizeof(HalfInfo) : 0), 256);
    part_o = align_up(part_lse + (size_t)workers * 2 * kChunkRows * sizeof(float), 256);
    ckv = align_up(part_o + (size_t)workers * 2 * kChunkRows * kDimCkv * sizeof(float), 256);
    kpe = ckv + (size_t)tiles * kChunkKeys * kDimCkv * 2;
    total = align_up(kpe + (size_t)tiles * kChunkKeys * kDimKpe * 2, 256);
  }
  // The window and the shared attention: their own tiles, and room for blocks and own_halves.
  ChunkLayout(int workers, int heads, int lists, int total_q, long long staged_tiles, long long batch)
      : tiles(staged_tiles) {
    max_blocks = ((long long)total_q * heads + kChunkRows - 1) / kChunkRows + lists;
    place(workers, lists, batch, true);
  }
  bool addressable() const { return tiles * kChunkKeys < (1LL << 31); }  // a staged row is a tensor-map coordinate
};

// The three launches of a call: stage the keys and plan, attend, merge split blocks.
cudaError_t launch_chunk_stage(const ChunkParams& p, bool fp8, cudaStream_t stream);
cudaError_t launch_span_stage(const ChunkParams& p, int span, bool fp8, cudaStream_t stream);  // kWindow, kShared
cudaError_t launch_chunk(const ChunkMaps& maps, const ChunkParams& p, int span, cudaStream_t stream);
cudaError_t launch_validate_groups(const ChunkParams& p, cudaStream_t stream);
cudaError_t launch_chunk_merge(const ChunkParams& p, cudaStream_t stream);

}  // namespace mla
