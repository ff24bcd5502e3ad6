// k_int8.cuh -- products of 8-bit integers with a scale for every token and every output channel.
//
//   scale_r = fp32(amax_r / 127),  code = x / scale_r rounded to nearest even  (per row of x and of W)
//   y[m][n] = (sum_k a[m][k] w[n][k]) * (sa[m] sw[n]) + bias[n]
// The sum is an exact 32-bit integer (K < 2^17 keeps 128 * 128 * K below 2^31), so no split or
// order of it changes a result; it is rounded to fp32 once, then scaled, and the output rounded
// once to its type.
//
// Codes are stored in rows of Kp = K rounded up to 16 bytes, zeros behind K, so that every row
// is addressable by TMA whatever K is.
#pragma once

#include <cuda_fp16.h>

#include "k_attn.cuh"     // attn::warp_wait_abort
#include "k_rotary.cuh"   // rotary::Vec
#include "veda_ptx.cuh"

namespace veda {
namespace int8 {

// ------------------------------------------------------------------------------------
// Row quantisation: HBM bound (one read of the row, one write of its codes). A row of up to 8,192
// values belongs to a group of threads -- a warp up to 1,024 values, a CTA above -- whose thread i
// owns the 8-value vectors i, i + threads, ...: rows run through a ring of kQuantStages rows in
// shared memory that each thread fills for itself with asynchronous copies, so the next rows are
// on their way while one is rounded.
// The division is exact: x * (1 / scale) is rounded, and where that product lies next to a half the
// sign of the exactly rounded x - scale (q +- 1/2) decides, ties to even.
// A row with a NaN or an infinity gets scale NaN (and codes 0), so its outputs are NaN; a row
// whose largest value is below 2^-100 counts as zero (scale 1, codes 0).
// ------------------------------------------------------------------------------------
struct QuantArgs {
  const void* x;
  int64_t x_stride;      // elements between rows
  int8_t* codes;         // [rows][kp]
  float* scale;          // [rows]
  int64_t rows;
  int32_t K, kp;
  int32_t vec;           // rows start on 16-byte boundaries
  int32_t dtype;         // of x (few-token product)
};

constexpr int kQuantWarpK = 1024;
constexpr int kQuantMaxK = 8192;      // ring kernels
constexpr int kQuantVecs = 4;         // vectors a thread (a CTA per row with 8: 109 us where 4 take 86)
constexpr int kQuantThreads = 256;    // most threads of a CTA
constexpr int kQuantStages = 3;

// Eight codes. Adding 1.5 * 2^23 to x * inv rounds it to an integer, ties to even, whose low byte
// is the float's; d is what was rounded away. x * inv is off by less than 2^-15, so only where |d| is
// within 2^-14 of a half can the integer be the wrong neighbour (16-bit inputs meet such borders, most
// of them exact ties, once in 900 values): there fma rounds x - s (q +- 1/2) once, so its sign is exact.
__device__ __forceinline__ uint2 codes8(const float* f, float s, float inv, bool live) {
  if (!live) return make_uint2(0u, 0u);
  constexpr float kRound = 12582912.0f, kNear = 0.5f - 0x1p-14f;
  const uint64_t inv2 = f2_splat(inv), round2 = f2_splat(kRound), minus2 = f2_splat(-1.0f);
  float t[8], d[8];
  float worst = 0.f;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const uint64_t x = f2_pack(__float_as_uint(f[i]), __float_as_uint(f[i + 1]));
    const uint64_t r = f2_fma(x, inv2, round2);
    f2_unpack(r, t[i], t[i + 1]);
    f2_unpack(f2_fma(x, inv2, f2_fma(r, minus2, round2)), d[i], d[i + 1]);
    worst = fmax3(worst, fabsf(d[i]), fabsf(d[i + 1]));
  }
  if (worst > kNear) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (fabsf(d[i]) <= kNear) continue;
      const float h = copysignf(0.5f, d[i]);
      const float z = fmaf(-s, (t[i] - kRound) + h, f[i]);            // x past the border q + h?
      const bool odd = (__float_as_uint(t[i]) & 1u) != 0;
      if ((h > 0.f ? z > 0.f : z < 0.f) || (z == 0.f && odd)) t[i] += 2.f * h;
    }
  }
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __byte_perm(__float_as_uint(t[4 * h]), __float_as_uint(t[4 * h + 1]), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(t[4 * h + 2]), __float_as_uint(t[4 * h + 3]), 0x0040);
    w[h] = __byte_perm(lo, hi, 0x5410);
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The row's scale from the largest |x| (as bits: a NaN or an infinity is the largest).
__device__ __forceinline__ float row_scale(uint32_t amax_bits, bool& live) {
  live = false;
  if (amax_bits >= 0x7f800000u) return __uint_as_float(0x7fffffffu);   // NaN
  const float amax = __uint_as_float(amax_bits);
  if (amax < 0x1p-100f) return 1.0f;
  live = true;
  return __fdiv_rn(amax, 127.0f);
}

// Largest |x| of the vectors added, as fp32 bits, NaN above all.
template <typename T> struct AbsMax;
template <> struct AbsMax<__nv_bfloat16> {
  __nv_bfloat162 m = __nv_bfloat162(__ushort_as_bfloat16(0), __ushort_as_bfloat16(0));
  __device__ __forceinline__ void add(const uint4& v) {
    const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __hmax2_nan(m, __habs2(p[i]));
  }
  __device__ __forceinline__ uint32_t bits() const {
    return __float_as_uint(__bfloat162float(__hmax_nan(m.x, m.y))) & 0x7fffffffu;
  }
};
template <> struct AbsMax<__half> {
  __half2 m = __half2(__ushort_as_half(0), __ushort_as_half(0));
  __device__ __forceinline__ void add(const uint4& v) {
    const __half2* p = reinterpret_cast<const __half2*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __hmax2_nan(m, __habs2(p[i]));
  }
  __device__ __forceinline__ uint32_t bits() const {
    return __float_as_uint(__half2float(__hmax_nan(m.x, m.y))) & 0x7fffffffu;
  }
};
template <> struct AbsMax<float> {
  uint32_t m = 0u;
  __device__ __forceinline__ void add(const uint4& v) {
    const uint32_t mask = 0x7fffffffu;
    m = max(m, max(max(v.x & mask, v.y & mask), max(v.z & mask, v.w & mask)));
  }
  __device__ __forceinline__ uint32_t bits() const { return m; }
};

// kWarp: a row per warp, else a row per CTA. Rows start on 16-byte boundaries.
template <typename T, bool kWarp>
__global__ void __launch_bounds__(kQuantThreads, sizeof(T) == 4 ? 2 : kWarp ? 3 : 4) quant_ring_kernel(const QuantArgs a) {
  constexpr int kWarps = kQuantThreads / 32;
  using V = rotary::Vec<T>;
  constexpr int U = 8 / V::E;                                  // 16-byte units a vector
  constexpr int kStage = kQuantVecs * U;                       // units a thread and row
  extern __shared__ __align__(16) uint8_t quant_smem[];
  __shared__ uint32_t red[2][kWarps];
  const int32_t threads = kWarp ? 32 : static_cast<int32_t>(blockDim.x);
  const int32_t me = kWarp ? (threadIdx.x & 31) : threadIdx.x, warps = blockDim.x >> 5;
  uint4* ring = reinterpret_cast<uint4*>(quant_smem) + (kWarp ? (threadIdx.x >> 5) * kQuantStages * kStage * 32 : 0) + me;
  if (!kWarp) {
    if (threadIdx.x < 2 * kWarps) (&red[0][0])[threadIdx.x] = 0u;
    __syncthreads();
  }
  const int64_t step = kWarp ? static_cast<int64_t>(gridDim.x) * warps : gridDim.x;
  const int64_t first = kWarp ? static_cast<int64_t>(blockIdx.x) * warps + (threadIdx.x >> 5) : blockIdx.x;

  // first value of 16-byte unit u of vector j: a vector is 8 neighbouring values of a 16-bit type, or two
  // fp32 units `threads` apart, so that a warp's accesses are contiguous
  const auto unit = [&](int j, int u) { return (me + (j * U + u) * threads) * V::E; };
  const T* x = static_cast<const T*>(a.x) + first * a.x_stride;     // the next row to fetch
  const int64_t x_step = step * a.x_stride;
  int64_t next = first;
  const auto fetch = [&](uint4* slot) {
    if (next < a.rows) {
#pragma unroll
      for (int j = 0; j < kQuantVecs; ++j)
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int32_t k0 = unit(j, u);
          uint4* const to = slot + (j * U + u) * threads;
          if (k0 + V::E <= a.K) {
            rotary::copy16_async(smem_u32(to), x + k0);
          } else if (k0 < a.kp) {                              // the row's end: zeros behind K
            uint4 tmp;
            T* t = reinterpret_cast<T*>(&tmp);
#pragma unroll
            for (int i = 0; i < V::E; ++i) t[i] = k0 + i < a.K ? x[k0 + i] : V::to(0.f);
            *to = tmp;
          }
        }
    }
    rotary::copies_commit();
    x += x_step;
    next += step;
  };
  const int32_t row_units = kStage * threads;
  uint4* const ring_end = ring + kQuantStages * row_units;
  uint4* free_slot = ring;
  for (int i = 0; i < kQuantStages - 1; ++i, free_slot += row_units) fetch(free_slot);
  uint4* slot = ring;
  int flip = 0;
  int8_t* out = a.codes + first * a.kp;
  const int64_t out_step = step * a.kp;
  for (int64_t row = first; row < a.rows; row += step, out += out_step) {
    rotary::copies_wait<kQuantStages - 2>();
    uint4 raw[kQuantVecs][U];
    AbsMax<T> big;
#pragma unroll
    for (int j = 0; j < kQuantVecs; ++j)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        raw[j][u] = unit(j, u) < a.kp ? slot[(j * U + u) * threads] : make_uint4(0, 0, 0, 0);
        big.add(raw[j][u]);
      }
    fetch(free_slot);                                          // read in the previous round
    uint32_t m = __reduce_max_sync(0xffffffffu, big.bits());
    if (!kWarp) {
      if ((threadIdx.x & 31) == 0) red[flip][threadIdx.x >> 5] = m;
      __syncthreads();
#pragma unroll
      for (int32_t w = 0; w < kWarps; ++w) m = max(m, red[flip][w]);      // zeros past the last warp
      flip ^= 1;
    }
    bool live;
    const float s = row_scale(m, live);
    const float inv = 1.0f / s;
#pragma unroll
    for (int j = 0; j < kQuantVecs; ++j) {
      if (unit(j, 0) >= a.kp) continue;
      float f[8];
#pragma unroll
      for (int u = 0; u < U; ++u) V::get(raw[j][u], f + u * V::E);
      const uint2 q = codes8(f, s, inv, live);
      if constexpr (U == 1) {
        *reinterpret_cast<uint2*>(out + unit(j, 0)) = q;
      } else {
        *reinterpret_cast<uint32_t*>(out + unit(j, 0)) = q.x;
        if (unit(j, 1) < a.kp) *reinterpret_cast<uint32_t*>(out + unit(j, 1)) = q.y;
      }
    }
    if (me == 0) a.scale[row] = s;
    free_slot = slot;
    slot = slot + row_units == ring_end ? ring : slot + row_units;
  }
  rotary::copies_wait<0>();
}

// Rows without 16-byte boundaries, and long ones: a CTA per row, a thread's elements 256 apart, so
// that every access of a warp is one contiguous piece; the first kQuantHeld of a thread's elements
// stay in registers between the maximum and the rounding, the rest are read again.
constexpr int kQuantHeld = 32;
template <typename T>
__global__ void __launch_bounds__(kQuantThreads) quant_row_kernel(const QuantArgs a) {
  using V = rotary::Vec<T>;
  __shared__ uint32_t red[kQuantThreads / 32];
  const int32_t me = threadIdx.x;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    T held[kQuantHeld];
#pragma unroll
    for (int i = 0; i < kQuantHeld; ++i) {
      const int32_t k = me + i * kQuantThreads;
      held[i] = k < a.K ? x[k] : V::to(0.f);
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kQuantHeld; ++i) m = max(m, abs_bits(V::one(held[i])));
#pragma unroll 4
    for (int32_t k = me + kQuantHeld * kQuantThreads; k < a.K; k += kQuantThreads) m = max(m, abs_bits(V::one(x[k])));
    m = __reduce_max_sync(0xffffffffu, m);
    if ((me & 31) == 0) red[me >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int32_t w = 0; w < kQuantThreads / 32; ++w) m = max(m, red[w]);
    bool live;
    const float s = row_scale(m, live);
    const float inv = 1.0f / s;
    int8_t* out = a.codes + row * a.kp;
    const auto put8 = [&](const float* f, int32_t k0) {
      const uint2 q = codes8(f, s, inv, live);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int32_t k = k0 + i * kQuantThreads;
        if (k < a.kp) out[k] = static_cast<int8_t>((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
      }
    };
#pragma unroll
    for (int j = 0; j < kQuantHeld; j += 8) {
      if (me + j * kQuantThreads >= a.kp) break;
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = V::one(held[j + i]);
      put8(f, me + j * kQuantThreads);
    }
    for (int32_t k0 = me + kQuantHeld * kQuantThreads; k0 < a.kp; k0 += 8 * kQuantThreads) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = k0 + i * kQuantThreads < a.K ? V::one(x[k0 + i * kQuantThreads]) : 0.f;
      put8(f, k0);
    }
    if (me == 0) a.scale[row] = s;
    __syncthreads();                                           // red is read before the next row's maxima
  }
}

// ------------------------------------------------------------------------------------
// Epilogue arithmetic shared by the products.
// ------------------------------------------------------------------------------------
struct MatArgs {
  const int8_t* a;       // [M][kp] (few-token kernel)
  const int8_t* w;       // [N][kp]
  const float* sa;       // [M]
  const float* sw;       // [N]
  const float* bias;     // null or [N]
  void* out;             // [M][ldo]
  int64_t ldo;           // elements
  int32_t M, N, kp;
  int32_t chunks;        // K chunks of 128 codes
  int32_t tiles_n;
  int64_t tiles;
  int32_t out_vec;       // rows of out start on 16-byte boundaries
};

__device__ __forceinline__ float scaled(int32_t acc, float sa, float sw, float bias) {
  return fmaf(static_cast<float>(acc), sa * sw, bias);
}

// Eight values of row m of x from k0, zeros behind K.
template <typename T>
__device__ __forceinline__ void few_load_as(const QuantArgs& q, int32_t m, int32_t k0, float* f) {
  using V = rotary::Vec<T>;
  const T* x = static_cast<const T*>(q.x) + m * q.x_stride;
  if (q.vec && k0 + 8 <= q.K) {
#pragma unroll
    for (int u = 0; u < 8 / V::E; ++u) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(x + k0) + u);
      V::get(v, f + u * V::E);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = k0 + i < q.K ? V::one(x[k0 + i]) : 0.f;
  }
}
__device__ __forceinline__ void few_load(const QuantArgs& q, int32_t m, int32_t k0, float* f) {
  if (q.dtype == 0) few_load_as<__nv_bfloat16>(q, m, k0, f);        // VEDA_BF16
  else if (q.dtype == 1) few_load_as<__half>(q, m, k0, f);          // VEDA_FP16
  else few_load_as<float>(q, m, k0, f);
}

// ------------------------------------------------------------------------------------
// Few tokens (M <= kFewMax, kFewMaxFused): the weights are read once and that is the whole cost, so a warp
// takes one output channel's row at a time, 16 bytes a lane with several loads in flight, and forms
// the products of all tokens with four-way integer dot products. The tokens' codes come from global
// memory (through L1) or, kFused, are made here: every CTA rounds the few rows of x into its shared
// memory, while its first weights are already on their way. For one token of 5,120 values that is
// 10 KB a CTA and saves the separate launch; M x K is bounded (kFewFused) so that it stays small
// beside the weights.
// ------------------------------------------------------------------------------------
// Weights from HBM, us of 5,120 x 5,120 (1,024 x 1,024): 2 tokens 9.3 (3.1) here, 3 tokens 9.7 (4.4) on the
// tensor cores (int8_tokens_kernel), whose time hardly grows up to 16. The fused form against
// rounding and product in two launches: 1 token 8.7 / 10.6 (2.6 / 4.3), 2 tokens 12.4 / 13.7 (4.1 / 5.4), 3 tokens
// 14.2 / 12.4 (4.8 / 6.7), 4 tokens of 4,096 13.3 / 11.2 (5.8 / 6.9): 3 and 4 tokens gain by it up to about
// 2,000 values and lose above, up to kFewFused, where the call still needs no workspace.
constexpr int kFewMax = 2, kFewMaxFused = 4;
constexpr int kSomeMax = 128;
constexpr int kFewThreads = 256;
constexpr int kFewFused = 16384;      // M * kp of the fused form
// CTAs an SM, by the registers of MT tokens; the grid is that many, so that a warp's next channel
// follows its last and its loads never pause
template <int MT> constexpr int few_ctas() { return MT <= 2 ? 5 : 4; }

template <typename T, int MT, bool kFused>
__global__ void __launch_bounds__(kFewThreads, few_ctas<MT>()) few_tokens_kernel(const __grid_constant__ MatArgs p,
                                                                const __grid_constant__ QuantArgs q) {
  using V = rotary::Vec<T>;
  extern __shared__ __align__(16) int8_t few_codes[];          // kFused: [M][kp]
  __shared__ uint32_t few_max[MT];
  const int32_t lane = threadIdx.x & 31;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kFewThreads / 32);
  int64_t n = static_cast<int64_t>(blockIdx.x) * (kFewThreads / 32) + (threadIdx.x >> 5);
  const int32_t vecs = p.kp / 16;
  constexpr int U = 4;
  int4 wv[U];
  const auto load = [&](int64_t channel, int32_t v0) {
    const int4* w = reinterpret_cast<const int4*>(p.w + channel * p.kp);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      wv[u] = make_int4(0, 0, 0, 0);
      if (channel < p.N && v0 + 32 * u < vecs) wv[u] = __ldcs(w + v0 + 32 * u);
    }
  };
  load(n, lane);
  float sa[MT];
  if constexpr (kFused) {
    if (threadIdx.x < MT) few_max[threadIdx.x] = 0u;
    __syncthreads();
    for (int32_t m = 0; m < p.M; ++m) {
      uint32_t big = 0;
      for (int32_t k0 = threadIdx.x * 8; k0 < p.kp; k0 += kFewThreads * 8) {
        float f[8];
        few_load(q, m, k0, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) big = max(big, abs_bits(f[i]));
      }
      big = __reduce_max_sync(0xffffffffu, big);
      if (lane == 0) atomicMax(&few_max[m], big);
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (m >= p.M) continue;
      bool live;
      sa[m] = row_scale(few_max[m], live);
      const float inv = 1.0f / sa[m];
      for (int32_t k0 = threadIdx.x * 8; k0 < p.kp; k0 += kFewThreads * 8) {
        float f[8];
        few_load(q, m, k0, f);
        *reinterpret_cast<uint2*>(few_codes + m * p.kp + k0) = codes8(f, sa[m], inv, live);
      }
    }
    __syncthreads();
  } else {
#pragma unroll
    for (int m = 0; m < MT; ++m) sa[m] = m < p.M ? __ldg(p.sa + m) : 0.f;
  }
  for (; n < p.N; n += step) {
    const float sw = __ldg(p.sw + n), bias = p.bias ? __ldg(p.bias + n) : 0.f;
    int32_t acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m] = 0;
    for (int32_t v0 = lane; v0 < vecs; v0 += 32 * U) {
      int4 cur[U];
#pragma unroll
      for (int u = 0; u < U; ++u) cur[u] = wv[u];
      // the next weights of this channel, or the first of the warp's next one
      if (v0 + 32 * U < vecs) load(n, v0 + 32 * U);
      else load(n + step, lane);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (v0 + 32 * u >= vecs) continue;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          if (m >= p.M) continue;
          const int4 av = kFused ? *(reinterpret_cast<const int4*>(few_codes + m * p.kp) + v0 + 32 * u)
                                 : __ldg(reinterpret_cast<const int4*>(p.a + static_cast<int64_t>(m) * p.kp) + v0 + 32 * u);
          acc[m] = __dp4a(cur[u].x, av.x, acc[m]);
          acc[m] = __dp4a(cur[u].y, av.y, acc[m]);
          acc[m] = __dp4a(cur[u].z, av.z, acc[m]);
          acc[m] = __dp4a(cur[u].w, av.w, acc[m]);
        }
      }
    }
    if (lane >= vecs) load(n + step, lane);      // a lane that owns no vector of a short row
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (m >= p.M) continue;
      const int32_t s = __reduce_add_sync(0xffffffffu, acc[m]);
      if (lane == m) static_cast<T*>(p.out)[m * p.ldo + n] = V::to(scaled(s, sa[m], sw, bias));
    }
  }
}

// ------------------------------------------------------------------------------------
// The tensor-core product: persistent pairs of CTAs (clusters of two), 256 tokens x kBN channels a
// tile. tcgen05.mma with cta_group::2 runs on both SMs of a pair: each CTA loads 128 rows of A and
// kBN / 2 rows of W a chunk, half of what two separate 128 x kBN tiles would fetch. That is what
// the pair is for: at kBN = 256 a chunk of 512 tensor cycles needs 64 bytes a cycle and SM from L2
// (about what 148 SMs get); one CTA alone at 128 x 256 needs 96, and measured 933 us at
// 50,220 x 5,120 x 5,120.
//   warp 4 (both CTAs)  TMA producer: per 128-deep K chunk its rows of A and W (128-byte swizzle)
//            into a kStages-deep ring; the bytes of both CTAs are counted on the leader's barrier
//   warp 5 (leader)     MMA issuer (one thread): four kind::i8 MMAs (M 256, N kBN, K 32) a chunk into
//            one of two accumulators; its commits free the stage in both CTAs
//   warps 0..3 (both)   epilogue of the CTA's 128 rows, 128 bytes of output a row at a time: a thread
//            scales and rounds its own row (the channels' scales and biases as broadcasts from shared
//            memory), stages it, and the warp writes the staged rows in contiguous pieces whatever
//            their alignment; overlaps the next tile's main loop, which hides it (tensor pipe 85.5% busy
//            at K = 5,120). (Scaling after the staging, a row at a time with a lane on two columns, is a
//            chain of dependent steps, as long as a main loop.)
// Tiles run channel-fastest, so the pairs of one wave share a few rows of A and all of W from L2.
// Every wait is bounded; on a timeout a CTA raises its abort flag, its roles leave their loops, the
// other CTA's waits run out in turn, in-flight copies and MMAs are drained, and both meet at the
// cluster barrier before the tensor memory is freed.
// ------------------------------------------------------------------------------------
constexpr int kThreads = 192;
constexpr int kBM = 256;                                      // rows per pair
constexpr uint32_t kStageTotal = 6 * 32768;                   // ring bytes a CTA
template <int BN> constexpr uint32_t stage_bytes() { return 16384u + static_cast<uint32_t>(BN) * 64u; }
template <int BN> constexpr int stages() { return static_cast<int>(kStageTotal / stage_bytes<BN>()); }
constexpr int kMaxStages = 9;
constexpr uint32_t kEpiStride = 128 + 16;                     // bytes a staged row: 16-byte accesses free of conflicts
constexpr uint32_t kEpiWarpBytes = 32 * kEpiStride;
constexpr uint32_t kOffScales = kStageTotal + 4 * kEpiWarpBytes;    // [2][2][256]: channel scales and biases
constexpr uint32_t kSmemBytes = kOffScales + 2 * 2 * 256 * 4 + 1024;
constexpr uint32_t kTmemCols = 512;
static_assert(stages<64>() <= kMaxStages && stages<128>() <= kMaxStages, "barriers for every stage");

// Instruction descriptor of kind::i8: signed A and B, both K-major, s32 accumulator.
__host__ __device__ constexpr uint32_t idesc_s8_s32(int M, int N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// D[tmem of both CTAs] (+)= A B^T over a pair of CTAs; descriptors of the leader's shared memory, the
// other CTA's operands at the same offsets.
__device__ __forceinline__ void mma2_ss_i8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on `bar` of both CTAs when every MMA issued so far by this thread has completed.
__device__ __forceinline__ void commit2(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
// This CTA's box of a tensor map into its own shared memory, counted on a barrier of the pair.
__device__ __forceinline__ void tma2_load(uint32_t dst, const CUtensorMap* map, uint32_t cluster_bar, int32_t x, int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
      "[%2];" ::"r"(dst),
      "l"(map), "r"(cluster_bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ uint32_t map_to_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void arrive_cluster(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// mbar_wait with cluster scope (arrivals of the other CTA's threads).
__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity, volatile int* abort, uint32_t site) {
  if (try_wait_cluster(bar, parity)) return true;
  if (!mbar_wait_slow(bar, parity, abort, site, kWaitLimitNs)) return false;
  return try_wait_cluster(bar, parity);            // the phase is complete: this one acquires it
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void tmem_alloc2(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

struct Bars {
  uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drain;
  uint32_t tmem_base;
  int abort;
};

// 128 bytes a row (W = 128 / sizeof(T) columns from n0) of 32 rows from m0: accumulators at `taddr` to
// the output. `w`, `b`: the W columns' scales and biases in shared memory; sa: this lane's row's scale.
template <typename T>
__device__ __forceinline__ void store_columns(const MatArgs& p, uint32_t taddr, uint8_t* staged, const float* w,
                                              const float* b, int32_t m0, int32_t n0, uint32_t lane, float sa) {
  using V = rotary::Vec<T>;
  constexpr int W = 128 / static_cast<int>(sizeof(T));
#pragma unroll
  for (int h = 0; h < W; h += 32) {
    uint32_t r[32];
    tmem_ld32_sync(taddr + h, r);
#pragma unroll
    for (int j = 0; j < 32; j += V::E) {
      float y[V::E];
#pragma unroll
      for (int i = 0; i < V::E; i += 4) {
        const float4 cw = *reinterpret_cast<const float4*>(w + h + j + i), cb = *reinterpret_cast<const float4*>(b + h + j + i);
        y[i] = scaled(static_cast<int32_t>(r[j + i]), sa, cw.x, cb.x);
        y[i + 1] = scaled(static_cast<int32_t>(r[j + i + 1]), sa, cw.y, cb.y);
        y[i + 2] = scaled(static_cast<int32_t>(r[j + i + 2]), sa, cw.z, cb.z);
        y[i + 3] = scaled(static_cast<int32_t>(r[j + i + 3]), sa, cw.w, cb.w);
      }
      *reinterpret_cast<uint4*>(staged + lane * kEpiStride + (h + j) * sizeof(T)) = V::put(y);
    }
  }
  __syncwarp();
  const int32_t rows = min(32, p.M - m0), cols = min(W, p.N - n0);
  T* out = static_cast<T*>(p.out) + static_cast<int64_t>(m0) * p.ldo + n0;
  if (p.out_vec && cols == W) {              // 8 lanes a row, 4 rows an instruction
    const int32_t c = static_cast<int32_t>(lane & 7);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int32_t row = 4 * i + static_cast<int32_t>(lane >> 3);
      const uint4 v = *reinterpret_cast<const uint4*>(staged + row * kEpiStride + c * 16);
      if (row < rows) *reinterpret_cast<uint4*>(out + row * p.ldo + c * V::E) = v;
    }
  } else {
#pragma unroll 1
    for (int32_t row = 0; row < rows; row += 8) {          // eight rows out of shared memory, then to the output
      T v[8][W / 32];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int h = 0; h < W / 32; ++h)
          v[i][h] = reinterpret_cast<const T*>(staged + (row + i) * kEpiStride)[32 * h + static_cast<int32_t>(lane)];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int h = 0; h < W / 32; ++h) {
          const int32_t c = 32 * h + static_cast<int32_t>(lane);
          if (row + i < rows && c < cols) out[(row + i) * p.ldo + c] = v[i][h];
        }
    }
  }
  __syncwarp();
}

template <typename T, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
int8_gemm_kernel(const __grid_constant__ CUtensorMap mA, const __grid_constant__ CUtensorMap mB,
                 const __grid_constant__ MatArgs p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(8) Bars bars;
  constexpr int kStages = stages<BN>();
  constexpr uint32_t kStageB = stage_bytes<BN>();
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  volatile int* abort = &bars.abort;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&bars.full[i]), 1);
      mbar_init(smem_u32(&bars.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars.acc_full[i]), 1);
      mbar_init(smem_u32(&bars.acc_empty[i]), 8);      // the epilogue warps of both CTAs
    }
    mbar_init(smem_u32(&bars.drain), 1);
    bars.abort = 0;
    fence_mbar_init();
  }
  if (warp == 5) tmem_alloc2(smem_u32(&bars.tmem_base), kTmemCols);
  if (warp == 4 && lane == 0) {
    prefetch_tensormap(&mA);
    prefetch_tensormap(&mB);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                                      // both CTAs' barriers and tensor memory exist
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;
  const int64_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (warp < 4) {
    uint8_t* staged = smem + kStageTotal + warp * kEpiWarpBytes;
    uint32_t it = 0;
    for (int64_t t = pair; t < p.tiles; t += pairs, ++it) {
      const int32_t m0 = static_cast<int32_t>(t / p.tiles_n) * kBM + static_cast<int32_t>(rank * 128 + warp * 32);
      const int32_t n0 = static_cast<int32_t>(t % p.tiles_n) * BN;
      const uint32_t ab = it & 1;
      const int32_t m = m0 + static_cast<int32_t>(lane);
      const float sa = m < p.M ? __ldg(p.sa + m) : 0.f;
      float* w = reinterpret_cast<float*>(smem + kOffScales) + ab * 512;
      float* b = w + 256;
      for (int32_t c = static_cast<int32_t>(tid); c < BN; c += 128) {
        const bool have = n0 + c < p.N;
        w[c] = have ? __ldg(p.sw + n0 + c) : 0.f;
        b[c] = have && p.bias ? __ldg(p.bias + n0 + c) : 0.f;
      }
      // the epilogue's four warps; one barrier a tile: the buffers alternate
      asm volatile("bar.sync 1, 128;" ::: "memory");
      const bool ok = attn::warp_wait_abort(smem_u32(&bars.acc_full[ab]), (it >> 1) & 1, abort, 70);
      tc_fence_after();
      constexpr int W = 128 / static_cast<int>(sizeof(T));
      const uint32_t taddr = tmem + ((warp * 32) << 16) + ab * 256;
#pragma unroll 1
      for (int cc = 0; cc < BN && ok; cc += W) {
        if (n0 + cc >= p.N || m0 >= p.M) break;
        store_columns<T>(p, taddr + cc, staged, w + cc, b + cc, m0, n0 + cc, lane, sa);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_cluster(map_to_cta(smem_u32(&bars.acc_empty[ab]), 0));
    }
  } else if (warp == 4 && lane == 0) {
    uint32_t g = 0;
    for (int64_t t = pair; t < p.tiles && !*abort; t += pairs) {
      const int32_t m0 = static_cast<int32_t>(t / p.tiles_n) * kBM + static_cast<int32_t>(rank) * 128;
      const int32_t n0 = static_cast<int32_t>(t % p.tiles_n) * BN + static_cast<int32_t>(rank) * (BN / 2);
      for (int32_t c = 0; c < p.chunks; ++c, ++g) {
        const uint32_t s = g % kStages;
        if (g >= kStages && !mbar_wait(smem_u32(&bars.empty[s]), (g / kStages - 1) & 1, abort, 71)) {
          t = p.tiles;
          break;
        }
        const uint32_t st = sb + s * kStageB, full = smem_u32(&bars.full[s]);
        if (rank == 0) mbar_arrive_expect_tx(full, 2 * kStageB);       // both CTAs' bytes
        const uint32_t leader_full = map_to_cta(full, 0);
        tma2_load(st, &mA, leader_full, c * 128, m0);
        tma2_load(st + 16384u, &mB, leader_full, c * 128, n0);
      }
    }
    // the leader's barriers count both CTAs' copies: none is in flight when it reaches the cluster barrier
    if (rank == 0)
      for (uint32_t i = g > kStages ? g - kStages : 0; i < g; ++i)
        mbar_wait(smem_u32(&bars.full[i % kStages]), (i / kStages) & 1, nullptr, 72);
  } else if (warp == 5 && lane == 0 && rank == 0) {
    constexpr uint32_t kIdesc = idesc_s8_s32(kBM, BN);
    uint32_t g = 0, it = 0;
    for (int64_t t = pair; t < p.tiles; t += pairs, ++it) {
      const uint32_t ab = it & 1;
      if (it >= 2 && !wait_cluster(smem_u32(&bars.acc_empty[ab]), ((it >> 1) - 1) & 1, abort, 73)) break;
      tc_fence_after();
      bool ok = true;
      for (int32_t c = 0; c < p.chunks; ++c, ++g) {
        const uint32_t s = g % kStages;
        if (!mbar_wait(smem_u32(&bars.full[s]), (g / kStages) & 1, abort, 74)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t dA = smem_desc_sw128(sb + s * kStageB, 16, 1024);
        const uint64_t dB = smem_desc_sw128(sb + s * kStageB + 16384u, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)   // 32 codes = 32 bytes per k-step: +2 in 16-byte units
          mma2_ss_i8(tmem + ab * 256, dA + kk * 2, dB + kk * 2, kIdesc, (c > 0 || kk > 0) ? 1u : 0u);
        commit2(smem_u32(&bars.empty[s]));
      }
      if (!ok) break;
      commit2(smem_u32(&bars.acc_full[ab]));
    }
    commit2(smem_u32(&bars.drain));
    mbar_wait(smem_u32(&bars.drain), 0, nullptr, 75);
  } else if (warp == 5 && lane == 0) {
    mbar_wait(smem_u32(&bars.drain), 0, nullptr, 76);  // the leader's last commit has reached this CTA too
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();                                      // neither CTA's memory is used by the other any more
  tc_fence_after();
  if (warp == 5) tmem_dealloc2(tmem, kTmemCols);
}

// ------------------------------------------------------------------------------------
// Some tokens (kFewMax < M <= 128): still bound by reading the weights, so the weights are the M side
// of the MMAs (128 channels a tile, BN >= M tokens as columns) and K is split over the CTAs of a
// cluster, so that a small N still fills the SMs; two CTAs share an SM, and one's set-up and reduction
// hide behind the other's loads. The integer partial sums meet through distributed shared memory:
// CTA r adds up and writes tokens r, r + S, ... Any split gives the same bits.
// ------------------------------------------------------------------------------------
namespace tokens {
constexpr int kThreads = 192;
constexpr int kMaxSplit = 8;
constexpr uint32_t kRing = 110592;                            // 108 KB: two CTAs an SM
template <int BN> constexpr uint32_t stage_bytes() { return 16384u + static_cast<uint32_t>(BN) * 128u; }
template <int BN> constexpr int stages() { return static_cast<int>(kRing / stage_bytes<BN>()); }
constexpr int kMaxStages = 6;
constexpr uint32_t kSmemBytes = kRing + 1024;
static_assert(stages<16>() <= kMaxStages && 128u * 128u * 4u <= kRing, "barriers; partial sums fit the ring");

struct Bars {
  uint64_t full[kMaxStages], empty[kMaxStages], acc_full, drain;
  uint32_t tmem_base;
  int abort;
};

__device__ __forceinline__ void mma_ss_i8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ int4 ld_cluster(uint32_t cluster_addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(cluster_addr) : "memory");
  return v;
}

// This CTA's tokens (rank, rank + split, ...; a warp every fourth of them): sums over the cluster, scaled
// and written. A lane has four channels; U tokens' loads from up to S CTAs are in flight together, as a
// load from another CTA's shared memory takes as long as one from L2.
template <typename T, int U, int S>
__device__ __forceinline__ void write_tokens(const MatArgs& p, uint32_t sb, int32_t n0, int32_t rank, int32_t split,
                                             uint32_t warp, uint32_t lane) {
  using V = rotary::Vec<T>;
  const int32_t n = n0 + 4 * static_cast<int32_t>(lane), step = 4 * split;
  float sw[4], bias[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sw[i] = n + i < p.N ? __ldg(p.sw + n + i) : 0.f;
    bias[i] = n + i < p.N && p.bias ? __ldg(p.bias + n + i) : 0.f;
  }
  uint32_t peer[S];
#pragma unroll
  for (int i = 0; i < S; ++i) peer[i] = map_to_cta(sb + lane * 16u, static_cast<uint32_t>(i < split ? i : 0));
  for (int32_t m0 = rank + static_cast<int32_t>(warp) * split; m0 < p.M; m0 += U * step) {
    int4 part[U][S];
    float sa[U];
#pragma unroll
    for (int t = 0; t < U; ++t) {
      const int32_t m = m0 + t * step;
      sa[t] = m < p.M ? __ldg(p.sa + m) : 0.f;
#pragma unroll
      for (int i = 0; i < S; ++i)
        part[t][i] = i < split && m < p.M ? ld_cluster(peer[i] + static_cast<uint32_t>(m) * 512u) : make_int4(0, 0, 0, 0);
    }
#pragma unroll
    for (int t = 0; t < U; ++t) {
      const int32_t m = m0 + t * step;
      if (m >= p.M) continue;
      int32_t acc[4] = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < S; ++i) {
        acc[0] += part[t][i].x;
        acc[1] += part[t][i].y;
        acc[2] += part[t][i].z;
        acc[3] += part[t][i].w;
      }
      T y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = V::to(scaled(acc[i], sa[t], sw[i], bias[i]));
      T* out = static_cast<T*>(p.out) + m * p.ldo + n;
      if (p.out_vec && n + 4 <= p.N) {
        if constexpr (sizeof(T) == 2) *reinterpret_cast<uint2*>(out) = *reinterpret_cast<const uint2*>(y);
        else *reinterpret_cast<uint4*>(out) = *reinterpret_cast<const uint4*>(y);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n + i < p.N) out[i] = y[i];
      }
    }
  }
}

template <typename T, int BN>
__global__ void __launch_bounds__(kThreads, 2)
int8_tokens_kernel(const __grid_constant__ CUtensorMap mW, const __grid_constant__ CUtensorMap mX,
                   const __grid_constant__ MatArgs p, const int32_t split) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(8) Bars bars;
  constexpr int kStages = stages<BN>();
  constexpr uint32_t kStageB = stage_bytes<BN>();
  constexpr uint32_t kCols = BN < 32 ? 32 : BN;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int32_t rank = static_cast<int32_t>(cluster_rank());
  const int32_t n0 = static_cast<int32_t>(blockIdx.x / split) * 128;
  const int32_t c0 = static_cast<int32_t>(static_cast<int64_t>(p.chunks) * rank / split);
  const int32_t c1 = static_cast<int32_t>(static_cast<int64_t>(p.chunks) * (rank + 1) / split);   // > c0: split <= chunks
  volatile int* abort = &bars.abort;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&bars.full[i]), 1);
      mbar_init(smem_u32(&bars.empty[i]), 1);
    }
    mbar_init(smem_u32(&bars.acc_full), 1);
    mbar_init(smem_u32(&bars.drain), 1);
    bars.abort = 0;
    fence_mbar_init();
  }
  if (warp == 5) {
    tmem_alloc(smem_u32(&bars.tmem_base), kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;

  if (warp == 4 && lane == 0) {
    uint32_t g = 0;
    for (int32_t c = c0; c < c1; ++c, ++g) {
      const uint32_t s = g % kStages;
      if (g >= kStages && !mbar_wait(smem_u32(&bars.empty[s]), (g / kStages - 1) & 1, abort, 80)) break;
      mbar_arrive_expect_tx(smem_u32(&bars.full[s]), kStageB);
      tma_load_2d(sb + s * kStageB, &mW, smem_u32(&bars.full[s]), c * 128, n0);
      tma_load_2d(sb + s * kStageB + 16384u, &mX, smem_u32(&bars.full[s]), c * 128, 0);
    }
    for (uint32_t i = g > kStages ? g - kStages : 0; i < g; ++i)
      mbar_wait(smem_u32(&bars.full[i % kStages]), (i / kStages) & 1, nullptr, 81);
  } else if (warp == 5 && lane == 0) {
    constexpr uint32_t kIdesc = idesc_s8_s32(128, BN);
    uint32_t g = 0;
    for (int32_t c = c0; c < c1; ++c, ++g) {
      const uint32_t s = g % kStages;
      if (!mbar_wait(smem_u32(&bars.full[s]), (g / kStages) & 1, abort, 82)) break;
      tc_fence_after();
      const uint64_t dW = smem_desc_sw128(sb + s * kStageB, 16, 1024);
      const uint64_t dX = smem_desc_sw128(sb + s * kStageB + 16384u, 16, 1024);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) mma_ss_i8(tmem, dW + kk * 2, dX + kk * 2, kIdesc, (c > c0 || kk > 0) ? 1u : 0u);
      tc_commit(smem_u32(&bars.empty[s]));
    }
    tc_commit(smem_u32(&bars.acc_full));
    tc_commit(smem_u32(&bars.drain));
    mbar_wait(smem_u32(&bars.drain), 0, nullptr, 83);
  }
  // partial sums [token][channel] over the ring, whose last stage the MMAs have read
  int32_t* partial = reinterpret_cast<int32_t*>(smem);
  if (warp < 4) {
    if (attn::warp_wait_abort(smem_u32(&bars.acc_full), 0, abort, 84)) {
      tc_fence_after();
      const uint32_t taddr = tmem + ((warp * 32) << 16);
#pragma unroll
      for (int cc = 0; cc < static_cast<int>(kCols); cc += 32) {
        uint32_t r[32];
        tmem_ld32_sync(taddr + cc, r);
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (cc + j < BN && cc + j < p.M) partial[(cc + j) * 128 + static_cast<int32_t>(warp * 32 + lane)] = static_cast<int32_t>(r[j]);
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  cluster_sync();                                             // every CTA's partial sums are written
  if (warp < 4) {
    if (split <= 2) write_tokens<T, 8, 2>(p, sb, n0, rank, split, warp, lane);
    else if (split <= 4) write_tokens<T, 4, 4>(p, sb, n0, rank, split, warp, lane);
    else write_tokens<T, 2, 8>(p, sb, n0, rank, split, warp, lane);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                                             // no CTA's sums are read any more
  tc_fence_after();
  if (warp == 5) tmem_dealloc(tmem, kCols);
}
}  // namespace tokens

}  // namespace int8
}  // namespace veda
