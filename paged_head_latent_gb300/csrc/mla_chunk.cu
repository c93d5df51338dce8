// mla_chunk.cu -- causal attention of a chunk of new tokens on the 5th-generation tensor
// cores: blocks of 128 query rows against staged 128-key tiles, one pair of SMs per worker.
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
// 0.90 to 0.92 of the measured bf16 burst rate, at the 1.6 GHz that the power limit leaves; one prompt of 256 tokens over 4096 keys: tensor pipe
// 80 % active).  What writes shared memory, the loads and P, is 152 KB a tile, 1216 cycles at 128
// bytes a cycle; the products read their operands besides, at a rate that was not measured.
//
// The tensor pipe's order is S(j+1), then O += P(j) V(j): the softmax of tile j runs while S(j+1)
// is computed.
//
// Warps: 0-7 softmax and output (a thread has a row, a quarter of a tile's keys and a quarter of
// the output's columns), 8 loads Q and K, 9 loads V, 10 issues the products (leader SM only), 11
// tensor memory.
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
    if (lane == 0 && sound) {
      const bool is_k = warp == kKWarp;
      const bool fault = is_k && p.fault_skip_tile >= 1 && w == 0 && rank == 0;
      bool ok = true;
      uint32_t j = 0;
      for (Walk it(p, w); it.live && ok; it.advance(), ++j) {
        const int row = (it.blk.tile0 + it.t) * kChunkKeys;
        const uint32_t again = (j - 1) & 1;  // phase of the previous use of a buffer
        if (is_k) {
          if (fault && (int)j == p.fault_skip_tile) break;  // (test of the give-up path: no more loads)
#pragma unroll
          for (uint32_t g = 0; g < kKGroups && ok; ++g) {
            if (j > 0)
              ok = g < kKGroups - 1 ? mbar_wait(bar(K_EMPTY + g), again, abort, p.status, kStatusTimeout, p.wait_ns)
                                    : mbar_wait(bar(S_FULL + again), ((j - 1) >> 1) & 1, abort, p.status, kStatusTimeout, p.wait_ns);
            if (!ok) break;
            if (rank == 0) mbar_arrive_expect_tx(bar(K_FULL + g), 2 * kGroup * kBox);
#pragma unroll
            for (int c = kGroup * g; c < (int)(kGroup * (g + 1)); ++c)
              tma_load_pair(base + kOffK + c * kBox, c < 8 ? &maps.ckv : &maps.kpe, c < 8 ? 64 * c : 0, row + 64 * rank,
                            leader(K_FULL + g));
          }
          if (it.first() && ok) {  // (the previous block's last S is done, so Q is free)
            if (rank == 0) mbar_arrive_expect_tx(bar(Q_FULL), 2 * kKBoxes * kBox);
            for (int c = 0; c < kKBoxes; ++c)
              tma_load_pair(base + kOffQ + c * kBox, c < 8 ? &maps.q_nope : &maps.q_pe, c < 8 ? 64 * c : 0,
                            it.blk.row0 + 64 * rank, leader(Q_FULL));
          }
        } else {
#pragma unroll
          for (uint32_t h = 0; h < 2 && ok; ++h) {  // keys 64 h .. + 63, this SM's 256 columns
            if (j > 0) ok = mbar_wait(bar(h ? PV_DONE : V_EMPTY), again, abort, p.status, kStatusTimeout, p.wait_ns);
            if (!ok) break;
            if (rank == 0) mbar_arrive_expect_tx(bar(V_FULL + h), 8 * kBox);
#pragma unroll
            for (int c = 0; c < 4; ++c)
              tma_load_pair(base + kOffV + (4 * h + c) * kBox, &maps.ckv, 256 * rank + 64 * c, row + 64 * h,
                            leader(V_FULL + h));
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
      auto output = [&](uint32_t j, bool first, uint32_t seg) {  // O += P V of tile j
        wait(P_FULL, j & 1);
        if (first && seg > 0) wait(O_EMPTY, (seg - 1) & 1);
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
          wait(V_FULL + h, j & 1);
#pragma unroll
          for (uint32_t n = 0; n < 2; ++n)
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k)
              mma2(issue, kColO + 128 * n, p0 + h * (kBox / 16) + 2 * k, v0 + (2 * h + n) * (2 * kBox / 16) + 128 * k,
                   kIdescO, h > 0 || k > 0 ? 1u : first ? 0u : 1u);
          commit2(issue, bar(h ? PV_DONE : V_EMPTY));
        }
      };
      // Within a segment S(j + 1) goes before O(j); at its end O comes first, so that the output
      // does not wait for the next block's Q.
      uint32_t j = 0;
      for (Walk it(p, w); it.live && __all_sync(0xffffffffu, good); it.next_segment()) {
        const uint32_t n = it.t_end - it.t;
        wait(Q_FULL, it.seg & 1);
        for (uint32_t i = 0; i <= n; ++i) {
          if (i < n) scores(j + i);
          if (i > 0) output(j + i - 1, i == 1, it.seg);
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
    const uint32_t piece = base + kOffP + half * kBox + (warp & 1) * 4096 + part * 2048;  // 2 KB of P for the output
    const uint32_t col_s = tmem + lanes + kColS + 32 * part, col_o = tmem + lanes + kColO + 128 * part;
    const uint32_t p_full = leader(P_FULL), o_empty = leader(O_EMPTY);
    const float scale = p.scale_log2;
    float m_ref = 0.f, l = 0.f;
    int seen = 0;  // keys that this row sees
    // The whole warp waits, and leaves together.
    auto wait = [&](uint32_t i, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar(i), parity, abort, p.status, kStatusTimeout, p.wait_ns));
    };
    auto aborted = [&]() -> bool { return __any_sync(0xffffffffu, *abort != 0); };
    bool ok = true;
    uint32_t j = 0;
    for (Walk it(p, w); it.live; it.advance(), ++j) {
      const bool first = it.first();
      const int local = it.blk.local0 + 64 * rank + r;  // row within its request
      if (first) seen = it.blk.seen + local / p.heads;
      const uint32_t* fl = p.flags + (size_t)(it.blk.tile0 + it.t) * 8 + quarter;
      // (from L2: this kernel may have begun before the staging pass wrote them)
      const uint32_t keys = __ldcg(fl), odd = __ldcg(fl + 4);
      if (!wait(S_FULL + (j & 1), (j >> 1) & 1)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t raw[32];
      tmem_ld32(col_s + 64 * (j & 1), raw);
      tmem_ld_wait();
      float s[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) s[k] = __uint_as_float(raw[k]);
      const int n = seen - it.t * kChunkKeys - 32 * quarter;  // keys of this thread's part that the row sees
      const bool full = n >= 32 && keys == 0xffffffffu && odd == 0 && scale >= 0.f;
      if (!full) {
        const uint32_t see = keys & (n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u);
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
        uint32_t o[2][32];
        tmem_ld32(col_o, o[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {  // 32 columns at a time, the next ones under way
          uint32_t(&x)[32] = o[c & 1];
          tmem_ld_wait();
          if (c < 3) {
            tmem_ld32(col_o + 32 * (c + 1), o[(c + 1) & 1]);
          } else {  // O is in registers: the next block's products may begin
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_leader(o_empty);
          }
          if (whole) {
            // Through this warp's part of P, so that a store writes 64 contiguous bytes of 8 rows.
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              uint32_t y[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float a = __uint_as_float(x[8 * u + 2 * e]), b = __uint_as_float(x[8 * u + 2 * e + 1]);
                const __nv_bfloat162 h = __floats2bfloat162_rn(a * inv, b * inv);
                y[e] = *reinterpret_cast<const uint32_t*>(&h);
              }
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(piece + lane * 64 + ((u ^ ((lane >> 1) & 3)) << 4)),
                           "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3])
                           : "memory");
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int rr = 8 * i + (lane >> 2), u = lane & 3;
              uint4 v;
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                           : "r"(piece + rr * 64 + ((u ^ ((rr >> 1) & 3)) << 4))
                           : "memory");
              if (in_block + rr < it.blk.rows)
                *reinterpret_cast<uint4*>(p.out + ((size_t)it.blk.row0 + in_block + rr) * kDimCkv + 256 * half + 128 * part +
                                          32 * c + 8 * u) = v;
            }
            __syncwarp();
          } else {
            // A fragment lies as [column / 4][row][4], so a store is 512 contiguous bytes.
            float4* dst = reinterpret_cast<float4*>(p.part_o + frag * kDimCkv) + (64 * half + 32 * part + 8 * c) * kChunkRows +
                          in_block + lane;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              float4 y;
              y.x = __uint_as_float(x[4 * u]) * inv;
              y.y = __uint_as_float(x[4 * u + 1]) * inv;
              y.z = __uint_as_float(x[4 * u + 2]) * inv;
              y.w = __uint_as_float(x[4 * u + 3]) * inv;
              dst[u * kChunkRows] = y;
            }
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

}  // namespace

cudaError_t launch_chunk(const ChunkMaps& maps, const ChunkParams& p, cudaStream_t stream) {
  // The shared-memory attribute is set once per device; calls may come from any host thread.
  static std::mutex mu;
  static bool configured[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!configured[dev]) {
      const cudaError_t e = cudaFuncSetAttribute(chunk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, chunk_kernel, maps, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mla
