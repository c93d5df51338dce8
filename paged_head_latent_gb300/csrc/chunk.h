// chunk.h -- parameters of the chunk attention (mla_chunk.cu) and its staging pass.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "common.cuh"

namespace mla {

constexpr int kChunkKeys = 128;  // keys of a tile
constexpr int kChunkRows = 128;  // query rows (token, head) of a block

// 128 consecutive query rows of one request; row 0 of request b is (token 0, head 0).
struct ChunkBlock {
  int row0;      // first row of the block in [total_q * H]
  int local0;    // ... and within its request
  int rows;      // rows in use, 1..128
  int tiles;     // key tiles that its last row sees (at least 1)
  int tile0;     // first staged tile of the request
  int seen;      // keys that token 0 of the request sees (may be <= 0)
  long long cost0;  // cost units before this block
};

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
  uint32_t* flags;      // [tiles][8]: 128 bits "is a key", 128 bits "holds a value that is not finite"
  __nv_bfloat16* ckv;   // [tiles * 128, 512] staged keys
  __nv_bfloat16* kpe;   // [tiles * 128, 64]
  float* part_lse;      // [workers][2][128] base-2 lse of partial fragments
  float* part_o;        // [workers][2][512 / 4][128 rows][4]
  int tiles;            // staged tiles (an upper bound from the host's sizes)
  int max_blocks;       // room in blocks
  unsigned long long wait_ns;
  int fault_skip_tile;
};

struct ChunkMaps {
  CUtensorMap q_nope, q_pe, ckv, kpe;  // boxes of 64 rows x 64 columns, 128-byte swizzle
};

struct ChunkLayout {
  size_t starts, merges, first_block, blocks, flags, part_lse, part_o, ckv, kpe, total;
  long long tiles, max_blocks;
  ChunkLayout(int workers, int heads, int batch, int total_q, int num_kv_indices) {
    tiles = ((long long)num_kv_indices + kChunkKeys - 1) / kChunkKeys + batch;
    max_blocks = ((long long)total_q * heads + kChunkRows - 1) / kChunkRows + batch;
    starts = 256;
    merges = align_up(starts + ((size_t)workers + 1) * sizeof(ChunkStart), 256);
    first_block = align_up(merges + (size_t)workers * sizeof(ChunkMerge), 256);
    blocks = align_up(first_block + ((size_t)batch + 1) * sizeof(int32_t), 256);
    flags = align_up(blocks + (size_t)max_blocks * sizeof(ChunkBlock), 256);
    part_lse = align_up(flags + (size_t)tiles * 32, 256);
    part_o = align_up(part_lse + (size_t)workers * 2 * kChunkRows * sizeof(float), 256);
    ckv = align_up(part_o + (size_t)workers * 2 * kChunkRows * kDimCkv * sizeof(float), 256);
    kpe = ckv + (size_t)tiles * kChunkKeys * kDimCkv * 2;
    total = align_up(kpe + (size_t)tiles * kChunkKeys * kDimKpe * 2, 256);
  }
  bool addressable() const { return tiles * kChunkKeys < (1LL << 31); }  // a staged row is a tensor-map coordinate
};

// The three launches of a call: stage the keys and plan, attend, merge split blocks.
cudaError_t launch_chunk_stage(const ChunkParams& p, bool fp8, cudaStream_t stream);
cudaError_t launch_chunk(const ChunkMaps& maps, const ChunkParams& p, cudaStream_t stream);
cudaError_t launch_chunk_merge(const ChunkParams& p, cudaStream_t stream);

}  // namespace mla
