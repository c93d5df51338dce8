// mla_chunk.cu -- attention of blocks of 128 query rows against 128-key tiles on the
// 5th-generation tensor cores, one pair of SMs per worker: a causal chunk of new tokens, a sliding
// window with sinks, and requests that share a prefix.
//
// A request's queries are q_len * H rows of 576 values (token-major, as they lie in memory),
// cut into blocks of 128 rows whatever H is, so a head-sharded model with 16 heads fills a
// block with eight tokens.  Row r of a request belongs to token r / H and sees the first
// kv_len - q_len + r / H + 1 keys; the mask is applied row by row, so a block may cut a token's
// heads.  Per tile: S = Q K^T, online softmax, O += P V with V = the latent part of K.
//
// Why a pair.  O of 128 rows x 512 fp32 would fill an SM's tensor memory.  With
// tcgen05.mma.cta_group::2 and M = 128 each SM of the pair keeps 64 of the rows: its O takes
// 256 columns (lanes 0-63 hold the first half of the product's columns, lanes 64-127 the
// second), two S tiles 64 columns each, and the softmax of a row never leaves its SM.  The
// B operand is split instead: SM c stages 64 of a tile's 128 keys (all 576 columns) for S and
// all 128 keys of its 256 latent columns for O.  Measured on this part: a 16-deep step takes
// 32.2 cycles for S (N = 128) and 64.3 for O (N = 256), the full rate, so a tile costs 36 x 32 +
// 16 x 64 = 2176 cycles of the tensor pipe; one SM alone (cta_group::1) has half the rate at M =
// 64, and a split of the depth needs partial scores to cross between the SMs (the decode
// kernel's way; its prefill runs at 0.45 of this rate).
//
// Shared memory (224 KB): Q (64 rows x 576, 72 KB), one K tile (9 chunks of 64 keys x 64
// columns, 8 KB each), one V tile (8 such chunks) and P (16 KB).  Nothing is double-buffered:
// K is reloaded in three parts and V in two, each as soon as the products that read it are
// done, which leaves a load most of a tile's time.  The loads are 136 KB per SM and tile; L2
// sustained 62 bytes a cycle and SM for these boxes, which is 2250 cycles a tile.
//
// What bounds it.  A tile takes 2470 cycles with its share of the blocks' starts and ends (four
// prompts, 128 heads, 22 tiles a block: 850 to 870 us with staging and merge, 1.72 to 1.76 PFLOP/s,
// 0.90 to 0.92 of the measured bf16 burst rate, at the 1.6 GHz that the power limit leaves; one
// prompt of 256 tokens over 4096 keys: tensor pipe 80 % active).  What writes shared memory, the
// loads and P, is 152 KB a tile, 1216 cycles at 128 bytes a cycle; the products read their operands
// besides, at a rate that was not measured.
//
// The window and the shared attention (kSpan; decode calls of theirs too) take the same tiles as
// pairs of halves of 64 keys, each from one of two runs (chunk.h), so that a window begins and a
// list ends where it likes; a half of which every row that reads it sees all keys is loaded from the
// bf16 cache (kDirect), and an odd block's last half costs no P V product.  A tile takes as long as a
// causal one; what else a call costs is starts of blocks (about three tiles each, which short
// windows and lists have many of).  Measured at the power limit, with staging: 2710 tokens of 128
// heads with windows of 1024 keys 583 us (1.29 PFLOP/s), 1374 tokens of 128 heads behind two prefixes of
// 1408 keys 448 us (1.42).  64 requests x 128 heads, windows of 4096 keys in 64-key pages: 82 us, DRAM at
// 5.0 TB/s in the kernel, which starts and ends with no load in flight.
//
// The tensor pipe's order is S(j+1), then O += P(j) V(j): the softmax of tile j runs while S(j+1)
// is computed.
//
// Warps: 0-7 softmax and output (a thread has a row, a quarter of a tile's keys and a quarter of
// the output's columns), 8 loads Q and K, 9 loads V, 10 issues the products (leader SM only), 11
// tensor memory.
//
// Two rules of the waits.  The warp that issues the products waits as a whole and stays converged.
// And a wait by parity may be one phase behind its barrier at most (the phase before has the parity
// of the one to come), so a warp waits for every phase of a barrier that it uses, needed or not.
#include <mutex>

#include "chunk.h"
#include "ptx.cuh"

namespace mla {

using namespace ptx;

namespace {

constexpr int kThreads = 384;
constexpr int kSoftmax = 8;  // softmax warps
constexpr int kKWarp = 8, kVWarp = 9, kMmaWarp = 10, kTmemWarp = 11;
constexpr uint32_t kBox = 64 * 128;  // 64 rows x 64 bf16, 128-byte swizzle
constexpr int kKBoxes = 9, kVBoxes = 8;
constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffK = kOffQ + kKBoxes * kBox;
constexpr uint32_t kOffV = kOffK + kKBoxes * kBox;
constexpr uint32_t kOffP = kOffV + kVBoxes * kBox;
constexpr uint32_t kOffRed = kOffP + 2 * kBox;        // [2][4][64] row maxima
constexpr uint32_t kOffBar = kOffRed + 2 * 4 * 64 * 4;
constexpr uint32_t kOffMisc = kOffBar + 256;
constexpr uint32_t kSmem = kOffMisc + 16;
constexpr uint32_t kColO = 0, kColS = 256, kTmemCols = 512;
constexpr float kRescaleLog2 = 8.0f;  // O is rescaled only when a row's maximum grows by more than 2^8

// K is handed over in groups of chunks and V in its two key halves; the last group of a product
// is free when the product is done, which S_FULL and PV_DONE tell already.
constexpr uint32_t kGroup = 3, kKGroups = kKBoxes / kGroup;
enum Bar : uint32_t {
  K_FULL, K_EMPTY = K_FULL + kKGroups, V_FULL = K_EMPTY + kKGroups - 1, V_EMPTY = V_FULL + 2, Q_FULL, S_FULL,
  P_FULL = S_FULL + 2, PV_DONE, O_EMPTY, DRAIN, NUM_BARS
};
static_assert(NUM_BARS * 8 <= 256, "barrier area");
static_assert(kSmem <= 232448, "shared memory");

struct Misc {
  uint32_t tmem;
  int abort;
};

// ---- pair forms of the tensor-core instructions
__device__ __forceinline__ void tmem_alloc2(uint32_t dst, uint32_t n) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(n) : "memory");
}
__device__ __forceinline__ void tmem_relinquish2() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t t, uint32_t n) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(t), "r"(n) : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(r));
  return r;
}
// The operands' descriptors are given by their low words (address and leading offset): the
// high word (stride 1024, 128-byte swizzle) is the same for all.
__device__ __forceinline__ void mma2(uint32_t issue, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                     uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %6};\n\t"
      "mov.b64 db, {%2, %6};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(issue), "n"((1024 >> 4) | (1 << 14) | (2 << 29))
      : "memory");
}
// Arrive on the barrier at this offset in both SMs when the products issued so far are done.
__device__ __forceinline__ void commit2(uint32_t issue, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.b32 e, %2, 0;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
          bar),
      "h"(static_cast<uint16_t>(3)), "r"(issue)
      : "memory");
}
// Load a box into this SM's shared memory; the bytes complete on a barrier of the pair.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
// Arrive on the leader's barrier.  What the arrival announces is complete before it is issued
// (tcgen05.wait for tensor-memory accesses, fence.proxy.async for P, which only this SM's own
// tensor core reads), so no cluster-wide release is needed: that form took 1250 cycles here.
__device__ __forceinline__ void arrive_leader(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// The four warps that share rows meet here; a warp that leaves the loop early has seen (or
// raised) the abort flag and arrives once more, which helps to release the others, each of
// which then sees the flag and does the same.
__device__ __forceinline__ void rows_sync(int warp) { asm volatile("bar.sync %0, 128;" ::"r"(1 + (warp & 1)) : "memory"); }
__device__ __forceinline__ void rows_release(int warp) {
  asm volatile("bar.arrive %0, 128;" ::"r"(1 + (warp & 1)) : "memory");
}

// A worker's tiles in order, segment by segment (a segment: tiles of one block).
struct Walk {
  const ChunkParams& p;
  int i, end_i, end_t;
  ChunkBlock blk;
  int t, t0, t_end, seg;
  bool live;
  __device__ Walk(const ChunkParams& params, int w) : p(params), seg(0) {
    const ChunkStart& start = p.starts[w];
    const ChunkStart& end = p.starts[w + 1];
    i = start.i;
    t0 = start.t;
    blk = start.blk;
    end_i = end.i;
    end_t = end.t;
    open();
  }
  __device__ void open() {
    live = i < end_i || (i == end_i && t0 < end_t);
    t = t0;
    t_end = i < end_i ? blk.tiles : end_t;
  }
  __device__ bool first() const { return t == t0; }
  __device__ bool last() const { return t == t_end - 1; }
  __device__ void next_segment() {
    ++i;
    ++seg;
    t0 = 0;
    if (i < end_i || (i == end_i && end_t > 0)) blk = p.blocks[i];
    open();
  }
  __device__ void advance() {
    if (++t == t_end) next_segment();
  }
};

// ---- the window and the shared attention: a tile's two halves of 64 keys
// Staged row of half h of the tile that a walk stands at.  An odd block's last tile has one half, but
// loads two and takes S of both (kWindow: its last half again, kShared: the half of zeros); only
// their P V is left out.
template <int kSpan>
__device__ __forceinline__ int half_row(const ChunkParams& p, const Walk& it, int h) {
  int u = 2 * it.t + h;
  if (kSpan == kShared && u >= it.blk.halves) return p.zero_row;
  if (kSpan == kWindow) u = max(min(u, it.blk.halves - 1), 0);
  return u < it.blk.head ? it.blk.tile0 + kHalfKeys * u : it.blk.rest0 + kHalfKeys * (u - it.blk.head);
}

// kDirect: p.sources says which halves are read from the caches.
template <int kSpan, bool kDirect>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ ChunkMaps maps, const __grid_constant__ ChunkParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  Misc& misc = *reinterpret_cast<Misc*>(smem + kOffMisc);
  const uint32_t rank = cluster_ctarank();
  const int w = blockIdx.x >> 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &misc.abort;
  auto bar = [&](uint32_t i) { return base + kOffBar + 8 * i; };
  auto leader = [&](uint32_t i) { return mapa(bar(i), 0); };

  if (threadIdx.x == 0) {
    misc.abort = (base & 1023u) ? 1 : 0;  // swizzled tiles need 1 KB alignment
    if (misc.abort) atomicOr(p.status, kStatusInternal);
    for (uint32_t i = 0; i < NUM_BARS; ++i)
      mbar_init(bar(i), i == P_FULL || i == O_EMPTY ? 2 * kSoftmax : 1);  // (both SMs' softmax warps)
    fence_mbar_init();
  }
  if (warp == kTmemWarp) {
    tmem_alloc2(base + kOffMisc, kTmemCols);
    tmem_relinquish2();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan and the staged keys
  // All 512 columns are ours, so they start at 0, and the products' addresses are constants.
  const uint32_t tmem = 0;
  if (misc.tmem != 0 && threadIdx.x == 0) {
    atomicOr(p.status, kStatusInternal);
    *abort = 1;
  }
  __syncthreads();
  const bool sound = misc.abort == 0;

  if (warp == kKWarp || warp == kVWarp) {
    // ------------------------------------------------------------ loads
    // A lane has a box of its own (K's and Q's nine chunks, V's four for each half), so that a group
    // of them leaves in one instruction: a product waits for its operands as long as they are
    // reloaded, and a thread that issued them one after another cost 5 to 10 % of a tile.
    if (sound) {
      const bool is_k = warp == kKWarp;
      const bool fault = is_k && p.fault_skip_tile >= 1 && w == 0 && rank == 0;
      bool ok = true;
      // (the whole warp waits, and leaves together)
      auto wait = [&](uint32_t i, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(bar(i), parity, abort, p.status, kStatusTimeout, p.wait_ns));
      };
      const int half = is_k ? (int)rank : lane >> 2 & 1;  // of the tile's keys
      const int chunk = is_k ? lane : 4 * (int)rank + (lane & 3);
      const uint32_t dst = base + (is_k ? kOffK : kOffV) + lane * kBox;
      const int column = chunk < 8 ? 64 * chunk : 0;
      const CUtensorMap* const staged = chunk < 8 ? &maps.ckv : &maps.kpe;
      const CUtensorMap* const cached = chunk < 8 ? &maps.cache_ckv : &maps.cache_kpe;
      const uint32_t group = is_k ? lane / kGroup : lane >> 2;  // (lanes without a box have one past the last)
      const uint32_t full = leader((is_k ? K_FULL : V_FULL) + min(group, is_k ? kKGroups - 1 : 1)), q_full = leader(Q_FULL);
      uint32_t j = 0;
      // Where the lane's half of the next tile is: its staged row, or the cache slot.
      int next_row = 0, next_slot = -1;
      Walk ahead(p, w);
      auto look = [&]() {
        if (!ahead.live) return;
        if constexpr (kSpan == kCausal) {
          next_row = (ahead.blk.tile0 + ahead.t) * kChunkKeys + kHalfKeys * half;
        } else {
          next_row = half_row<kSpan>(p, ahead, half);
          if (kDirect) next_slot = __ldcg(p.sources + next_row / kHalfKeys);
        }
      };
      look();
      for (; ahead.live && ok; ++j) {
        const bool first = ahead.first();
        const int q_row = ahead.blk.row0;
        const bool direct = kDirect && next_slot >= 0;
        const int row = direct ? next_slot : next_row;
        const CUtensorMap* map = direct ? cached : staged;
        ahead.advance();
        look();
        const uint32_t again = (j - 1) & 1;  // phase of the previous use of a buffer
        if (is_k) {
          if (fault && (int)j == p.fault_skip_tile) break;  // (test of the give-up path: no more loads)
#pragma unroll
          for (uint32_t g = 0; g < kKGroups; ++g) {
            if (j > 0 && !(ok = g < kKGroups - 1 ? wait(K_EMPTY + g, again)
                                                 : wait(S_FULL + again, ((j - 1) >> 1) & 1)))
              break;
            if (rank == 0 && lane == 0) mbar_arrive_expect_tx(bar(K_FULL + g), 2 * kGroup * kBox);
            if (group == g) tma_load_pair(dst, map, column, row, full);
          }
          if (first && ok) {  // (the previous block's last S is done, so Q is free)
            if (rank == 0 && lane == 0) mbar_arrive_expect_tx(bar(Q_FULL), 2 * kKBoxes * kBox);
            if (lane < kKBoxes)
              tma_load_pair(base + kOffQ + lane * kBox, lane < 8 ? &maps.q_nope : &maps.q_pe, column, q_row + 64 * rank, q_full);
          }
        } else {
#pragma unroll
          for (uint32_t h = 0; h < 2; ++h) {  // keys 64 h .. + 63, this SM's 256 columns
            if (j > 0 && !(ok = wait(h ? PV_DONE : V_EMPTY, again))) break;
            if (rank == 0 && lane == 0) mbar_arrive_expect_tx(bar(V_FULL + h), 8 * kBox);
            if (group == h) tma_load_pair(dst, map, column, row, full);
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ products (leader SM)
    // The whole warp runs this, with one elected thread issuing, and the loop is short enough
    // straight-line code with operands that are constants plus warp-uniform values, so that an
    // issue costs less than its product (32 cycles for S, 64 for O).  Measured on four prompts
    // with 128 heads: from one thread of a divergent warp 1299 us, with 64-bit descriptors and
    // a copy of S's products for each buffer 1114, as it is 907, with the loops rolled 1012-1324.
    // A failed wait does not branch before the tile's end.
    if (rank == 0 && sound) {
      constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, false, false);
      constexpr uint32_t kIdescO = idesc_bf16_f32(128, 256, false, true);
      auto low = [&](uint32_t off, uint32_t lead) { return ((base + off) >> 4) | (lead >> 4) << 16; };
      const uint32_t q0 = low(kOffQ, 16), k0 = low(kOffK, 16), p0 = low(kOffP, 16), v0 = low(kOffV, kBox);
      const uint32_t issue = elect_one();
      bool good = true;
      auto wait = [&](uint32_t i, uint32_t parity) {
        good &= mbar_wait(bar(i), parity, abort, p.status, kStatusTimeout, p.wait_ns);
        __syncwarp();
        tc_fence_after();
      };
      auto scores = [&](uint32_t j) {  // S of tile j
        const uint32_t dst = kColS + 64 * (j & 1);
#pragma unroll
        for (uint32_t g = 0; g < kKGroups; ++g) {
          wait(K_FULL + g, j & 1);
#pragma unroll
          for (uint32_t c = kGroup * g; c < kGroup * (g + 1); ++c)
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k)
              mma2(issue, dst, q0 + c * (kBox / 16) + 2 * k, k0 + c * (kBox / 16) + 2 * k, kIdescS, c + k > 0);
          commit2(issue, bar(g < kKGroups - 1 ? K_EMPTY + g : S_FULL + (j & 1)));
        }
      };
      auto output = [&](uint32_t j, bool first, uint32_t seg, bool lone) {  // O += P V of tile j (lone: of its first half)
        wait(P_FULL, j & 1);
        if (first && seg > 0) wait(O_EMPTY, (seg - 1) & 1);
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
          wait(V_FULL + h, j & 1);
#pragma unroll
          for (uint32_t n = 0; n < 2; ++n)
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k)
              mma2(kSpan != kCausal && h > 0 && lone ? 0u : issue, kColO + 128 * n, p0 + h * (kBox / 16) + 2 * k,
                   v0 + (2 * h + n) * (2 * kBox / 16) + 128 * k, kIdescO, h > 0 || k > 0 ? 1u : first ? 0u : 1u);
          commit2(issue, bar(h ? PV_DONE : V_EMPTY));
        }
      };
      // Within a segment S(j + 1) goes before O(j); at its end O comes first, so that the output
      // does not wait for the next block's Q.
      uint32_t j = 0;
      for (Walk it(p, w); it.live && __all_sync(0xffffffffu, good); it.next_segment()) {
        const uint32_t n = it.t_end - it.t;
        const bool odd = kSpan != kCausal && it.t_end == it.blk.tiles && (it.blk.halves & 1);
        wait(Q_FULL, it.seg & 1);
        for (uint32_t i = 0; i <= n; ++i) {
          if (i < n) scores(j + i);
          if (i > 0) output(j + i - 1, i == 1, it.seg, odd && i == n);
          if (!__all_sync(0xffffffffu, good)) break;
        }
        j += n;
      }
      // Everything issued is done once this arrives.
      commit2(issue, bar(DRAIN));
      volatile int no_abort = 0;
      mbar_wait(bar(DRAIN), 0, &no_abort, p.status, kStatusTimeout, p.wait_ns);
    }
    __syncwarp();
  } else if (warp < kSoftmax && sound) {
    // ------------------------------------------------------------ softmax and output
    // This thread: row r of the SM's 64, keys 64 half + 32 part .. + 31 of a tile, and output
    // columns 256 half + 128 part .. + 127.
    const int half = (warp >> 1) & 1, part = warp >> 2, r = 32 * (warp & 1) + lane;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    float* red = reinterpret_cast<float*>(smem + kOffRed);
    const int quarter = 2 * half + part;
    const uint32_t mine = base + kOffP + half * kBox + r * 128;  // this thread's row of P
    const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
    const uint32_t col_s = tmem + lanes + kColS + 32 * part, col_o = tmem + lanes + kColO + 128 * part;
    const uint32_t p_full = leader(P_FULL), o_empty = leader(O_EMPTY);
    const float scale = p.scale_log2;
    float m_ref = 0.f, l = 0.f;
    int seen = 0;   // keys that this row sees (kCausal)
    int token = 0;  // the row's token (kWindow: of its request)
    // The whole warp waits, and leaves together.
    auto wait = [&](uint32_t i, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar(i), parity, abort, p.status, kStatusTimeout, p.wait_ns));
    };
    auto aborted = [&]() -> bool { return __any_sync(0xffffffffu, *abort != 0); };
    auto below = [](int x) { return x >= 32 ? 0xffffffffu : x <= 0 ? 0u : (1u << x) - 1u; };
    // kWindow, kShared: which of the next tile's keys the row sees, asked for a tile ahead, as each
    // instruction and each load between a tile's scores and its weights counts.
    struct {
      int row, u, slot;
      uint32_t keys[2], odd[2];
      int4 info;
    } next;
    Walk ahead(p, w);
    auto look = [&]() {
      if constexpr (kSpan != kCausal) {
        if (!ahead.live) return;
        next.u = 2 * ahead.t + half;
        const int row = half_row<kSpan>(p, ahead, half), at = row + 32 * part;
        next.row = row;
        // (from L2: this kernel may have begun before the staging pass wrote them)
        const uint32_t* fl = p.flags + (at >> 5);
        const size_t to_odd = (size_t)p.tiles * 4;
        next.keys[0] = __ldcg(fl), next.odd[0] = __ldcg(fl + to_odd);
        if (kSpan == kWindow && !kDirect && (at & 31)) next.keys[1] = __ldcg(fl + 1), next.odd[1] = __ldcg(fl + to_odd + 1);
        if constexpr (kDirect) next.slot = __ldcg(p.sources + row / kHalfKeys);
        if constexpr (kSpan == kShared) next.info = __ldcg(reinterpret_cast<const int4*>(p.infos + row / kHalfKeys));
      }
    };
    look();
    bool ok = true;
    uint32_t j = 0;
    for (Walk it(p, w); it.live; it.advance(), ++j) {
      const bool first = it.first();
      uint32_t keys, odd;
      int n;                // keys of this thread's part that the row sees
      uint32_t hidden = 0;  // ... but for these
      bool cached = false;  // all are keys then, but any may not be finite
      if constexpr (kSpan == kCausal) {
        const int local = it.blk.local0 + 64 * rank + r;  // row within its request
        if (first) seen = it.blk.seen + local / p.heads;
        n = seen - it.t * kChunkKeys - 32 * quarter;
        const uint32_t* fl = p.flags + (size_t)(it.blk.tile0 + it.t) * 8 + quarter;
        // (from L2: this kernel may have begun before the staging pass wrote them)
        keys = __ldcg(fl), odd = __ldcg(fl + 4);
      } else {
        if (first) token = ((kSpan == kShared ? it.blk.row0 : it.blk.local0) + 64 * (int)rank + r) / p.heads;
        keys = next.keys[0], odd = next.odd[0];
        if constexpr (kSpan == kShared) {
          n = token >= next.info.x && token < next.info.y ? token + next.info.z - 32 * part : 0;
        } else {
          const int shift = next.row & 31, over = next.u - it.blk.head;
          if (!kDirect && shift) {
            keys = __funnelshift_r(keys, next.keys[1], shift);
            odd = __funnelshift_r(odd, next.odd[1], shift);
          }
          const int key = (over < 0 ? kHalfKeys * next.u : it.blk.rest_key + kHalfKeys * over) + 32 * part;
          const int sinks = p.sinks - key;
          if (over < 0) {
            n = min(sinks, it.blk.rest_key - key);
          } else {
            n = it.blk.seen + token - key;
            if (n > p.window) hidden = below(n - p.window) & ~below(sinks);
          }
          if (next.u >= it.blk.halves) n = 0;
        }
        if (kDirect) cached = next.slot >= 0;
        if (cached) keys = 0xffffffffu, odd = 0;
      }
      if (!wait(S_FULL + (j & 1), (j >> 1) & 1)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t raw[32];
      tmem_ld32(col_s + 64 * (j & 1), raw);
      if constexpr (kSpan != kCausal) {
        ahead.advance();
        look();
      }
      tmem_ld_wait();
      float s[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) s[k] = __uint_as_float(raw[k]);
      if constexpr (kDirect) {
        if (cached) {
          // A key that is not finite makes a score that is not (an infinite weightless key would
          // otherwise pass): the row is NaN, as with staged keys.
          float z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < 32; ++k) z[k & 3] = fmaf(s[k], 0.f, z[k & 3]);
          z[0] = (z[0] + z[1]) + (z[2] + z[3]);
          if (z[0] != z[0]) l = z[0];
        }
      }
      const bool full = n >= 32 && keys == 0xffffffffu && odd == 0 && scale >= 0.f && hidden == 0;
      if (!full) {
        const uint32_t see = keys & below(n) & ~hidden;
        // (a staged key that is not finite is all zeros: its scores are finite, the row is NaN below)
        if (odd & see) l = __int_as_float(0x7fc00000);
#pragma unroll
        for (int k = 0; k < 32; ++k) s[k] = (see >> k) & 1u ? s[k] * scale : -INFINITY;
      }
      float mx;
      {
        float m8[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) m8[k] = fmaxf(fmaxf(s[k], s[k + 8]), fmaxf(s[k + 16], s[k + 24]));
#pragma unroll
        for (int k = 0; k < 4; ++k) m8[k] = fmaxf(m8[k], m8[k + 4]);
        mx = fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3]));
      }
      if (full) mx *= scale;
      float* red_j = red + (j & 1) * 256 + r;
      red_j[64 * quarter] = mx;
      rows_sync(warp);
      if (aborted()) {
        ok = false;
        break;
      }
      mx = fmaxf(fmaxf(red_j[0], red_j[64]), fmaxf(red_j[128], red_j[192]));
      bool rescale = false;
      float alpha = 1.f;
      if (first) {
        m_ref = mx;
        l = l != l ? l : 0.f;  // (NaN: this tile holds a key that is not finite)
      } else if (mx > m_ref + kRescaleLog2) {
        alpha = fast_exp2(m_ref - mx);  // (0 when no key was seen before)
        m_ref = mx;
        l *= alpha;
        rescale = true;
      }
      const float m = m_ref == -INFINITY ? 0.f : m_ref;
      uint32_t pk[16];
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      const float mul = full ? scale : 1.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float a = fast_exp2(fmaf(s[2 * k], mul, -m)), b = fast_exp2(fmaf(s[2 * k + 1], mul, -m));
        sum[k & 3] += a + b;
        // The operand type beside a bf16 V: a weight is off by 2^-8 of itself at most, its sum keeps
        // all bits.  On the measured chunks the output is within 2.0e-3 of 64 bits, 1.7e-3 with float32
        // weights; weights in two bf16 parts would double the product.
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        pk[k] = *reinterpret_cast<const uint32_t*>(&h);
      }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      // P is single-buffered: the previous tile's product has to be done (it also settles O).
      if (j > 0 && !wait(PV_DONE, (j - 1) & 1)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          tmem_ld32(col_o + 32 * c, o);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
          tmem_st32(col_o + 32 * c, o);
        }
        tmem_st_wait();
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(mine + (((4 * part + u) ^ (r & 7)) << 4)), "r"(pk[4 * u]),
                     "r"(pk[4 * u + 1]), "r"(pk[4 * u + 2]), "r"(pk[4 * u + 3])
                     : "memory");
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_leader(p_full);

      if (it.last()) {
        // Output: O / l to out, or a fragment to the workspace.
        red_j = red + ((j + 1) & 1) * 256 + r;  // (the maxima there were read before the last meeting)
        red_j[64 * quarter] = l;
        rows_sync(warp);
        if (aborted()) {
          ok = false;
          break;
        }
        const float total = (red_j[0] + red_j[64]) + (red_j[128] + red_j[192]);
        rows_sync(warp);  // the next tile writes its maxima there
        if (!wait(PV_DONE, j & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const bool whole = it.t_end == it.blk.tiles && it.t0 == 0;
        const float inv = total > 0.f ? 1.f / total : total != total ? total : 0.f;  // (no key: out 0, lse -inf)
        const int in_block = 64 * rank + 32 * (warp & 1);  // first of this warp's rows
        const int slot = it.seg == 0 ? 0 : 1;
        const size_t frag = ((size_t)w * 2 + slot) * kChunkRows;
        if (quarter == 0 && in_block + lane < it.blk.rows) {
          if (whole)
            p.lse[(size_t)it.blk.row0 + in_block + lane] =
                total == 0.f ? -INFINITY : fmaf(m_ref, 0.69314718055994531f, logf(total));
          else
            p.part_lse[frag + in_block + lane] = total == 0.f ? -INFINITY : m_ref + log2f(total);
        }
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {  // (rolled: its code must not push the tiles' code out of the instruction cache)
          uint32_t x[32];
          tmem_ld32(col_o + 32 * c, x);
          tmem_ld_wait();
          if (c == 3) {  // O is in registers: the next block's products may begin
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_leader(o_empty);
          }
          float y[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) y[k] = __uint_as_float(x[k]) * inv;
          if (whole) {
            uint32_t h[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * k], y[2 * k + 1]);
              h[k] = *reinterpret_cast<const uint32_t*>(&b);
            }
            // Two lanes write 64 bytes of a row together, then of the other's row: half the lines to a store.
            // (Windows of 1024 keys with 128 heads 596 -> 586 us; four lanes and 128 bytes take more
            // code and registers: 653.)
            const bool upper = lane & 1;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? h[k] : h[8 + k], 1);
              if (upper) h[k] = got; else h[8 + k] = got;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int rr = in_block + (lane & ~1) + i;
              if (rr >= it.blk.rows) continue;
              __nv_bfloat16* dst =
                  p.out + ((size_t)it.blk.row0 + rr) * kDimCkv + 256 * half + 128 * part + 32 * c + 16 * (lane & 1);
              if (wide) {
                st_global_v8(dst, h + 8 * i);
              } else {
                reinterpret_cast<uint4*>(dst)[0] = make_uint4(h[8 * i], h[8 * i + 1], h[8 * i + 2], h[8 * i + 3]);
                reinterpret_cast<uint4*>(dst)[1] = make_uint4(h[8 * i + 4], h[8 * i + 5], h[8 * i + 6], h[8 * i + 7]);
              }
            }
          } else if (in_block + lane < it.blk.rows) {
            // A fragment lies as [column / 4][row][4], so a store is 512 contiguous bytes.
            float4* dst = reinterpret_cast<float4*>(p.part_o + frag * kDimCkv) + (64 * half + 32 * part + 8 * c) * kChunkRows +
                          in_block + lane;
#pragma unroll
            for (int u = 0; u < 8; ++u) dst[u * kChunkRows] = make_float4(y[4 * u], y[4 * u + 1], y[4 * u + 2], y[4 * u + 3]);
          }
        }
        l = 0.f;
      }
    }
    if (!ok) rows_release(warp);
  }

  // The merge may be scheduled; it waits for this grid's end before it reads anything.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __syncwarp();
  __syncthreads();
  if (*abort && threadIdx.x == 0) {
    // A wait gave up, so loads may be in flight that nobody waited for: their barriers are the
    // leader's and may never complete.  Loads take microseconds; give them a millisecond.
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 1000000ull) {
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == kTmemWarp) {
    tc_fence_after();
    tmem_dealloc2(tmem, kTmemCols);
  }
}

template <int kSpan, bool kDirect>
cudaError_t launch_instance(const ChunkMaps& maps, const ChunkParams& p, cudaStream_t stream) {
  // The shared-memory attribute is set once per device; calls may come from any host thread.
  static std::mutex mu;
  static bool configured[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!configured[dev]) {
      const cudaError_t e =
          cudaFuncSetAttribute(chunk_kernel<kSpan, kDirect>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
      if (e != cudaSuccess) return e;
      configured[dev] = true;
    }
  }
  // A programmatic dependent of the staging pass: this kernel's start overlaps that one's tail.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * p.workers);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, chunk_kernel<kSpan, kDirect>, maps, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_chunk(const ChunkMaps& maps, const ChunkParams& p, int span, cudaStream_t stream) {
  const bool direct = p.sources != nullptr;
  if (span == kWindow)
    return direct ? launch_instance<kWindow, true>(maps, p, stream) : launch_instance<kWindow, false>(maps, p, stream);
  if (span == kShared)
    return direct ? launch_instance<kShared, true>(maps, p, stream) : launch_instance<kShared, false>(maps, p, stream);
  return launch_instance<kCausal, false>(maps, p, stream);
}

}  // namespace mla
