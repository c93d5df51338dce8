// mla_cache.cu -- writers and readers of the paged latent cache: rotary positions with the
// write of new tokens, tokens read back by slot, and page copies.  All three are bound by
// HBM (a few operations per byte) or, for a few tokens, by the launch.
//
// The unit of work is a warp with its whole piece in registers, and every global access is
// 16 bytes per lane over contiguous rows.  No shared-memory staging: the warps of an SM cover
// one another's latency.
#include "launch.h"
#include "ptx.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kHeadsPerUnit = 16;  // query heads that one warp rotates

__device__ __forceinline__ uint4 ld16(const void* p) { return *static_cast<const uint4*>(p); }
__device__ __forceinline__ void st16(void* p, uint4 v) { *static_cast<uint4*>(p) = v; }

__device__ __forceinline__ float2 bf2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t to_bf2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Turns per position of a frequency (radians per position), as a 64-bit binary fraction
// of a turn.  position * turns wraps exactly in integer arithmetic, so the angle of a far
// position keeps its fraction: the error is the 2^-53 of the double product times the
// position (2^-33 turns at position 10^6), where a float32 product of position and
// frequency would be off by whole radians at 10^8.
__device__ __forceinline__ uint64_t turns_of(float freq) {
  double r = static_cast<double>(freq) * 0.15915494309189533577;  // 1 / (2 pi)
  r -= floor(r);
  return static_cast<uint64_t>(r * 18446744073709551616.0);  // r < 1 (or NaN: handled by the caller)
}

__device__ __forceinline__ void angle(uint64_t turns, int pos, bool finite, float* c, float* s) {
  const uint64_t t = turns * static_cast<uint64_t>(static_cast<int64_t>(pos));
  // The top 32 bits as a signed fraction of a turn, in half turns for sincospi.
  sincospif(static_cast<float>(static_cast<int32_t>(t >> 32)) * 4.656612873077393e-10f, s, c);
  if (!finite) *c = *s = __int_as_float(0x7fc00000);
}

// E4M3 codes of 16 latent values of one 128-value tile shared by 8 lanes, and the tile's
// scale.  amax is over the finite values; scale = amax / 448 (1 for a tile of zeros); a
// code is the E4M3 number nearest to the float32 quotient x / scale (IEEE division), and
// a value that is not finite becomes E4M3's NaN.
__device__ __forceinline__ uint4 quantise16(const uint4 (&raw)[2], float* scale) {
  float x[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint4& r = raw[i >> 2];
    const uint32_t w = (i & 3) == 0 ? r.x : (i & 3) == 1 ? r.y : (i & 3) == 2 ? r.z : r.w;
    const float2 f = bf2(w);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float a = fabsf(x[i]);
    m = fmaxf(m, a < INFINITY ? a : 0.f);
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float sc = m > 0.f ? __fdiv_rn(m, 448.f) : 1.f;
  *scale = sc;
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t w = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float a = __fdiv_rn(x[4 * i + 2 * h], sc), b = __fdiv_rn(x[4 * i + 2 * h + 1], sc);
      if (fabsf(x[4 * i + 2 * h]) == INFINITY) a = __int_as_float(0x7fc00000);
      if (fabsf(x[4 * i + 2 * h + 1]) == INFINITY) b = __int_as_float(0x7fc00000);
      uint16_t p;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(p) : "f"(b), "f"(a));
      w |= static_cast<uint32_t>(p) << (16 * h);
    }
    out[i] = w;
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// Rotary positions and the cache write.  A token is units - 1 query units (16 heads each)
// and one cache unit; a warp takes units grid-stride.  Lane i holds pair i's turns for the
// whole kernel and its cosine and sine for the current token.
//   interleaved: pair i = elements 2i, 2i + 1; a warp rotates 4 heads per instruction, lane
//                l the pairs 4(l % 8) .. + 3 of head l / 8;
//   half-split:  pair i = elements i, i + 32; 8 heads per instruction pair, lane l the pairs
//                8(l % 4) .. + 7 of head l / 4.
// Bound by HBM: 8192 tokens of 128 heads (287 MB) take 47.1 us, 6.1 TB/s, 0.91 of the measured
// copy rate; 8000 into an FP8 cache 45.3 us, where the bytes take 41.3; 8000 of one head, whose cache
// rows are most of it, 6.4 us (bf16, bytes 3.1) and 10 (FP8, bytes 2.5).  64 tokens take 2.5 us, 2.9
// into an FP8 cache (calls back to back in a graph): a launch and two round trips to memory.
template <bool kInterleaved, bool kFp8>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const RopeParams p) {
  // One warp does the block's double-precision work: with every warp doing it, 8000 tokens of
  // one head took 8.1 us.
  __shared__ uint64_t all_turns[32];
  const int lane = threadIdx.x & 31;
  const bool finite = fabsf(p.inv_freq[lane]) < INFINITY;
  if (threadIdx.x < 32) all_turns[lane] = finite ? turns_of(p.inv_freq[lane]) : 0;
  __syncthreads();
  const uint64_t turns = all_turns[lane];
  const int axis = lane < p.section0 ? 0 : lane < p.section0 + p.section1 ? 1 : 2;
  const int units = (p.heads + kHeadsPerUnit - 1) / kHeadsPerUnit + 1;
  const long long total = (long long)p.tokens * units;
  for (long long u = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); u < total; u += (long long)gridDim.x * kWarps) {
    const int t = (int)(u / units), j = (int)(u - (long long)t * units);
    float c, s;
    if (j < units - 1) {
      const int h0 = j * kHeadsPerUnit;
      const __nv_bfloat16* src = p.q + (long long)t * p.q_stride_t;
      __nv_bfloat16* dst = p.q_out + ((size_t)t * p.heads) * kDimKpe;
      if constexpr (kInterleaved) {
        uint4 v[4];
        const int h = h0 + (lane >> 3), ch = lane & 7;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (h + 4 * i < p.heads) v[i] = ld16(src + (long long)(h + 4 * i) * p.q_stride_h + 8 * ch);
        angle(turns, p.positions[(size_t)axis * p.tokens + t], finite, &c, &s);
        float cc[4], ss[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          cc[k] = __shfl_sync(0xffffffffu, c, 4 * ch + k);
          ss[k] = __shfl_sync(0xffffffffu, s, 4 * ch + k);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (h + 4 * i >= p.heads) continue;
          const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = bf2(w[k]);
            o[k] = to_bf2(f.x * cc[k] - f.y * ss[k], f.x * ss[k] + f.y * cc[k]);
          }
          st16(dst + (size_t)(h + 4 * i) * kDimKpe + 8 * ch, make_uint4(o[0], o[1], o[2], o[3]));
        }
      } else {
        uint4 lo[2], hi[2];
        const int h = h0 + (lane >> 2), ch = lane & 3;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (h + 8 * i < p.heads) {
            lo[i] = ld16(src + (long long)(h + 8 * i) * p.q_stride_h + 8 * ch);
            hi[i] = ld16(src + (long long)(h + 8 * i) * p.q_stride_h + 32 + 8 * ch);
          }
        angle(turns, p.positions[(size_t)axis * p.tokens + t], finite, &c, &s);
        float cc[8], ss[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          cc[k] = __shfl_sync(0xffffffffu, c, 8 * ch + k);
          ss[k] = __shfl_sync(0xffffffffu, s, 8 * ch + k);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (h + 8 * i >= p.heads) continue;
          const uint32_t a[4] = {lo[i].x, lo[i].y, lo[i].z, lo[i].w}, b[4] = {hi[i].x, hi[i].y, hi[i].z, hi[i].w};
          uint32_t oa[4], ob[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 x = bf2(a[k]), y = bf2(b[k]);
            oa[k] = to_bf2(x.x * cc[2 * k] - y.x * ss[2 * k], x.y * cc[2 * k + 1] - y.y * ss[2 * k + 1]);
            ob[k] = to_bf2(x.x * ss[2 * k] + y.x * cc[2 * k], x.y * ss[2 * k + 1] + y.y * cc[2 * k + 1]);
          }
          st16(dst + (size_t)(h + 8 * i) * kDimKpe + 8 * ch, make_uint4(oa[0], oa[1], oa[2], oa[3]));
          st16(dst + (size_t)(h + 8 * i) * kDimKpe + 32 + 8 * ch, make_uint4(ob[0], ob[1], ob[2], ob[3]));
        }
      }
      continue;
    }
    // The cache unit: latent copied (or quantised), rope part rotated, both to the token's slot.
    const int slot = p.slots[t];
    if (slot < 0 || slot >= p.num_slots) continue;
    const __nv_bfloat16* lat = p.ckv + (long long)t * p.ckv_stride;
    const __nv_bfloat16* kp = p.kpe + (long long)t * p.kpe_stride;
    uint4 raw[2];
    if constexpr (kFp8) {
      raw[0] = ld16(lat + 16 * lane);
      raw[1] = ld16(lat + 16 * lane + 8);
    } else {
      raw[0] = ld16(lat + 8 * lane);
      raw[1] = ld16(lat + 256 + 8 * lane);
    }
    const int i0 = kInterleaved ? 2 * lane : lane, i1 = kInterleaved ? 2 * lane + 1 : lane + 32;
    const float a = __bfloat162float(kp[i0]), b = __bfloat162float(kp[i1]);
    angle(turns, p.positions[(size_t)axis * p.tokens + t], finite, &c, &s);
    __nv_bfloat16* ko;
    if constexpr (kFp8) {
      uint8_t* tok = p.kv_fp8 + (size_t)slot * kFp8TokenBytes;
      float scale;
      const uint4 codes = quantise16(raw, &scale);
      st16(tok + 16 * lane, codes);
      if ((lane & 7) == 0) *reinterpret_cast<float*>(tok + kDimCkv + 4 * (lane >> 3)) = scale;
      ko = reinterpret_cast<__nv_bfloat16*>(tok + kDimCkv + 16);
    } else {
      __nv_bfloat16* o = p.ckv_cache + (size_t)slot * kDimCkv;
      st16(o + 8 * lane, raw[0]);
      st16(o + 256 + 8 * lane, raw[1]);
      ko = p.kpe_cache + (size_t)slot * kDimKpe;
    }
    ko[i0] = __float2bfloat16_rn(a * c - b * s);
    ko[i1] = __float2bfloat16_rn(a * s + b * c);
  }
}

// Tokens read by slot into contiguous bf16 rows, kTok tokens of a warp in flight.  Tokens whose
// slot is outside the cache become zero rows.  Bound by HBM: 263K FP8 tokens on 64-slot pages
// (477 MB) take 74.5 us, 6.4 TB/s, 0.96 of the measured copy rate (two tokens in flight 97 us,
// eight 78; with a grid of resident blocks 84), 263K bf16 tokens (607 MB) 88 us, the copy rate.
template <bool kFp8, int kTok>
__global__ void __launch_bounds__(kThreads) gather_kernel(const GatherParams p) {
  const int lane = threadIdx.x & 31;
  int n = p.n;
  if (p.count) n = min(n, max(*p.count, 0));
  const long long stride = (long long)gridDim.x * kWarps * kTok;
  for (long long i0 = ((long long)blockIdx.x * kWarps + (threadIdx.x >> 5)) * kTok; i0 < n; i0 += stride) {
    int mine = -1;
    if (lane < kTok && i0 + lane < n) mine = p.slots[i0 + lane];
    if (mine >= p.num_slots) mine = -1;
    uint4 a[kTok], b[kTok], r[kTok];
    float sc[kTok];
#pragma unroll
    for (int k = 0; k < kTok; ++k) {
      const int slot = __shfl_sync(0xffffffffu, mine, k);
      a[k] = b[k] = r[k] = make_uint4(0, 0, 0, 0);
      sc[k] = 0.f;
      if (slot < 0) continue;
      if constexpr (kFp8) {
        const uint8_t* tok = p.kv_fp8 + (size_t)slot * kFp8TokenBytes;
        a[k] = ld16(tok + 16 * lane);
        sc[k] = *reinterpret_cast<const float*>(tok + kDimCkv + 4 * (lane >> 3));
        if (lane < 8) r[k] = ld16(tok + kDimCkv + 16 + 16 * lane);
      } else {
        const __nv_bfloat16* lat = p.ckv + (size_t)slot * kDimCkv;
        a[k] = ld16(lat + 8 * lane);
        b[k] = ld16(lat + 256 + 8 * lane);
        if (lane < 8) r[k] = ld16(p.kpe + (size_t)slot * kDimKpe + 8 * lane);
      }
    }
#pragma unroll
    for (int k = 0; k < kTok; ++k) {
      if (i0 + k >= n) break;
      __nv_bfloat16* o = p.ckv_out + (size_t)(i0 + k) * kDimCkv;
      if constexpr (kFp8) {
        const uint4 lo = ptx::e4m3x8_scaled_to_bf16x8(make_uint2(a[k].x, a[k].y), sc[k]);
        const uint4 hi = ptx::e4m3x8_scaled_to_bf16x8(make_uint2(a[k].z, a[k].w), sc[k]);
        st16(o + 16 * lane, lo);
        st16(o + 16 * lane + 8, hi);
      } else {
        st16(o + 8 * lane, a[k]);
        st16(o + 256 + 8 * lane, b[k]);
      }
      if (lane < 8) st16(p.kpe_out + (size_t)(i0 + k) * kDimKpe + 8 * lane, r[k]);
    }
  }
}

// Page copies: entry e copies the first tokens[e] slots of page src[e] to page dst[e].  A
// unit is 2 KB of one page's bytes (latent, then rope part; or FP8 tokens), one warp.  Bound by
// HBM: 4500 pages of 64 bf16 tokens (332 MB read, as much written) take 96 us, 6.9 TB/s.
constexpr int kCopyBytes = 2048;

__global__ void __launch_bounds__(kThreads) copy_pages_kernel(const CopyParams p) {
  const int lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // (what came before on the stream: the lists)
  int n = p.n;
  if (p.count) n = min(n, max(*p.count, 0));
  const long long page_a = (long long)p.page_size * p.bytes_a, page_b = (long long)p.page_size * p.bytes_b;
  const long long units_a = (page_a + kCopyBytes - 1) / kCopyBytes, units_b = (page_b + kCopyBytes - 1) / kCopyBytes;
  const long long per = units_a + units_b, total = per * n;
  for (long long u = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); u < total; u += (long long)gridDim.x * kWarps) {
    const int e = (int)(u / per);
    const long long q = u - e * per;
    const int src = p.src[e], dst = p.dst[e];
    if (src < 0 || dst < 0 || src >= p.num_pages || dst >= p.num_pages || src == dst) continue;
    const int tokens = p.tokens ? min(max(p.tokens[e], 0), p.page_size) : p.page_size;
    const bool second = q >= units_a;
    const long long off = (second ? q - units_a : q) * kCopyBytes;
    const long long end = (long long)tokens * (second ? p.bytes_b : p.bytes_a), page = second ? page_b : page_a;
    uint8_t* base = second ? p.b : p.a;
    const uint8_t* from = base + (size_t)src * page;
    uint8_t* to = base + (size_t)dst * page;
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long o = off + 512 * i + 16 * lane;
      if (o < end) v[i] = ld16(from + o);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long o = off + 512 * i + 16 * lane;
      if (o < end) st16(to + o, v[i]);
    }
  }
}

int blocks_for(long long warps, int most) {
  const long long b = (warps + kWarps - 1) / kWarps;
  return (int)(b < 1 ? 1 : b > most ? most : b);
}

// Blocks of a grid-stride kernel.  Four to eight of them fill an SM; several rounds of blocks
// keep reads and writes mixed (8192 tokens of 128 heads: 47.5 us at 32 a SM, 48.9 at 8, 51.2
// with a block for every eight units; 354 MB of pages moved: 124.6, 131.0, 132.6 us).
constexpr int kMostBlocks = 152 * 32;

}  // namespace

cudaError_t launch_rope_append(const RopeParams& p, bool fp8, cudaStream_t stream) {
  const long long units = (long long)p.tokens * ((p.heads + kHeadsPerUnit - 1) / kHeadsPerUnit + 1);
  const int grid = blocks_for(units, kMostBlocks);
  if (fp8) {
    if (p.interleaved) rope_append_kernel<true, true><<<grid, kThreads, 0, stream>>>(p);
    else rope_append_kernel<false, true><<<grid, kThreads, 0, stream>>>(p);
  } else {
    if (p.interleaved) rope_append_kernel<true, false><<<grid, kThreads, 0, stream>>>(p);
    else rope_append_kernel<false, false><<<grid, kThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_gather(const GatherParams& p, bool fp8, cudaStream_t stream) {
  // A warp's tokens are one pass of its block (up to 311K tokens): blocks that end and begin at
  // different times keep reads and writes mixed.
  constexpr int kTok = 4;
  const int grid = blocks_for(((long long)p.n + kTok - 1) / kTok, 152 * 64);
  if (fp8) gather_kernel<true, kTok><<<grid, kThreads, 0, stream>>>(p);
  else gather_kernel<false, kTok><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_copy_pages(const CopyParams& p, cudaStream_t stream) {
  const long long per = ((long long)p.page_size * p.bytes_a + kCopyBytes - 1) / kCopyBytes +
                        ((long long)p.page_size * p.bytes_b + kCopyBytes - 1) / kCopyBytes;
  // A programmatic dependent: its launch overlaps the pool's kernel that writes the lists.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks_for(per * p.n, kMostBlocks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, copy_pages_kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mla
