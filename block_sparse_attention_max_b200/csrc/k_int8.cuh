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
// on their way while one is rounded. Longer rows, and rows that start on no 16-byte boundary, are
// read twice with plain loads.
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
};

constexpr int kQuantWarpK = 1024;
constexpr int kQuantMaxK = 8192;      // ring kernels
constexpr int kQuantVecs = 4;         // vectors a thread
constexpr int kQuantThreads = 256;    // most threads of a CTA
constexpr int kQuantStages = 3;

template <typename T>
__device__ __forceinline__ void load8(const T* row, int32_t k0, int32_t K, bool vec, float* f) {
  using V = rotary::Vec<T>;
  if (vec && k0 + 8 <= K) {
#pragma unroll
    for (int u = 0; u < 8 / V::E; ++u) {
      uint4 v = *reinterpret_cast<const uint4*>(row + k0 + u * V::E);
      V::get(v, f + u * V::E);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = k0 + i < K ? V::one(row[k0 + i]) : 0.f;
  }
}

// x / s to the nearest integer, ties to even, |x| <= 127.5 s, for a quotient near a half-integer
// (x * inv is off by less than 2^-15): fma rounds x - s (q +- 1/2) once, so its sign is exact.
__device__ __forceinline__ int32_t div_round(float x, float s, float inv) {
  float q = rintf(x * inv);
  const float up = fmaf(-s, q + 0.5f, x), dn = fmaf(-s, q - 0.5f, x);
  const bool odd = (static_cast<int32_t>(q) & 1) != 0;
  if (up > 0.f || (up == 0.f && odd)) q += 1.f;
  else if (dn < 0.f || (dn == 0.f && odd)) q -= 1.f;
  return static_cast<int32_t>(q);
}

// The eight codes of a vector by the exact test (out of line: it runs rarely).
__device__ __noinline__ uint2 codes8_exact(float4 a, float4 b, float s, float inv) {
  const float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i >> 2] |= (static_cast<uint32_t>(div_round(f[i], s, inv)) & 0xffu) << (8 * (i & 3));
  return make_uint2(w[0], w[1]);
}

// Eight codes. Adding 1.5 * 2^23 to x * inv rounds it to an integer, ties to even, whose low byte
// is the float's; d is what was rounded away. Only where some |d| is within 2^-14 of a half can an
// integer be the wrong neighbour, and only then (1 vector in 500 or so) is the exact test run.
__device__ __forceinline__ uint2 codes8(const float* f, float s, float inv, bool live) {
  if (!live) return make_uint2(0u, 0u);
  constexpr float kRound = 12582912.0f;
  float t[8];
  float worst = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t[i] = fmaf(f[i], inv, kRound);
    worst = fmaxf(worst, fabsf(fmaf(f[i], inv, kRound - t[i])));
  }
  if (worst > 0.5f - 0x1p-14f)
    return codes8_exact(make_float4(f[0], f[1], f[2], f[3]), make_float4(f[4], f[5], f[6], f[7]), s, inv);
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

// Largest |x| of a vector, as bits (packed for the 16-bit types, whose order is their bits').
template <typename T> struct AbsMax {
  uint32_t m = 0u;
  __device__ __forceinline__ void add(const uint4& v) {
    const uint32_t mask = 0x7fff7fffu;
    m = __vmaxu2(m, __vmaxu2(__vmaxu2(v.x & mask, v.y & mask), __vmaxu2(v.z & mask, v.w & mask)));
  }
  __device__ __forceinline__ uint32_t bits() const {
    const uint16_t b = static_cast<uint16_t>(max(m & 0xffffu, m >> 16));
    return __float_as_uint(rotary::Vec<T>::one(*reinterpret_cast<const T*>(&b))) & 0x7fffffffu;
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
__global__ void __launch_bounds__(kQuantThreads) quant_ring_kernel(const QuantArgs a) {
  using V = rotary::Vec<T>;
  constexpr int U = 8 / V::E;                                  // 16-byte units a vector
  constexpr int kStage = kQuantVecs * U;                       // units a thread and row
  extern __shared__ __align__(16) uint8_t quant_smem[];
  __shared__ uint32_t red[2][kQuantThreads / 32];
  const int32_t threads = kWarp ? 32 : static_cast<int32_t>(blockDim.x);
  const int32_t me = kWarp ? (threadIdx.x & 31) : threadIdx.x, warps = blockDim.x >> 5;
  uint4* ring = reinterpret_cast<uint4*>(quant_smem) + (kWarp ? (threadIdx.x >> 5) * kQuantStages * kStage * 32 : 0) + me;
  const int64_t step = kWarp ? static_cast<int64_t>(gridDim.x) * warps : gridDim.x;
  const int64_t first = kWarp ? static_cast<int64_t>(blockIdx.x) * warps + (threadIdx.x >> 5) : blockIdx.x;

  const auto fetch = [&](int64_t row, int st) {
    if (row < a.rows) {
      const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
      uint4* slot = ring + st * kStage * threads;
#pragma unroll
      for (int j = 0; j < kQuantVecs; ++j) {
        const int32_t k0 = (me + j * threads) * 8;
        if (k0 + 8 <= a.K) {
#pragma unroll
          for (int u = 0; u < U; ++u)
            rotary::copy16_async(smem_u32(slot + (j * U + u) * threads), reinterpret_cast<const uint4*>(x + k0) + u);
        } else if (k0 < a.kp) {                                // the row's end: zeros behind K
          uint4 tmp[U];
          T* t = reinterpret_cast<T*>(tmp);
#pragma unroll
          for (int i = 0; i < 8; ++i) t[i] = k0 + i < a.K ? x[k0 + i] : V::to(0.f);
#pragma unroll
          for (int u = 0; u < U; ++u) slot[(j * U + u) * threads] = tmp[u];
        }
      }
    }
    rotary::copies_commit();
  };
  for (int i = 0; i < kQuantStages - 1; ++i) fetch(first + i * step, i);
  int st = 0, flip = 0;
  for (int64_t row = first; row < a.rows; row += step) {
    rotary::copies_wait<kQuantStages - 2>();
    const uint4* slot = ring + st * kStage * threads;
    uint4 raw[kQuantVecs][U];
    AbsMax<T> big;
#pragma unroll
    for (int j = 0; j < kQuantVecs; ++j) {
      const bool own = (me + j * threads) * 8 < a.kp;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        raw[j][u] = own ? slot[(j * U + u) * threads] : make_uint4(0, 0, 0, 0);
        big.add(raw[j][u]);
      }
    }
    fetch(row + (kQuantStages - 1) * step, st == 0 ? kQuantStages - 1 : st - 1);   // read last round
    uint32_t m = __reduce_max_sync(0xffffffffu, big.bits());
    if (!kWarp) {
      if ((threadIdx.x & 31) == 0) red[flip][threadIdx.x >> 5] = m;
      __syncthreads();
      for (int32_t w = 0; w < warps; ++w) m = max(m, red[flip][w]);
      flip ^= 1;
    }
    bool live;
    const float s = row_scale(m, live);
    const float inv = 1.0f / s;
    int8_t* out = a.codes + row * a.kp;
#pragma unroll
    for (int j = 0; j < kQuantVecs; ++j) {
      const int32_t k0 = (me + j * threads) * 8;
      if (k0 >= a.kp) continue;
      float f[8];
#pragma unroll
      for (int u = 0; u < U; ++u) V::get(raw[j][u], f + u * V::E);
      *reinterpret_cast<uint2*>(out + k0) = codes8(f, s, inv, live);
    }
    if (me == 0) a.scale[row] = s;
    st = st == kQuantStages - 1 ? 0 : st + 1;
  }
  rotary::copies_wait<0>();
}

// Any row: a CTA reads it twice.
template <typename T>
__global__ void __launch_bounds__(kQuantThreads) quant_row_kernel(const QuantArgs a) {
  __shared__ uint32_t red[kQuantThreads / 32];
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    uint32_t m = 0;
    for (int32_t k = threadIdx.x; k < a.K; k += blockDim.x) m = max(m, abs_bits(rotary::Vec<T>::one(x[k])));
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
    for (int32_t w = 0; w < static_cast<int32_t>(blockDim.x >> 5); ++w) m = max(m, red[w]);
    bool live;
    const float s = row_scale(m, live);
    const float inv = 1.0f / s;
    int8_t* out = a.codes + row * a.kp;
    for (int32_t k0 = threadIdx.x * 8; k0 < a.kp; k0 += blockDim.x * 8) {
      float f[8];
      load8<T>(x, k0, a.K, a.vec != 0, f);
      *reinterpret_cast<uint2*>(out + k0) = codes8(f, s, inv, live);
    }
    if (threadIdx.x == 0) a.scale[row] = s;
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
  int32_t tiles_m, tiles_n;
  int64_t tiles;
  int32_t out_vec;       // rows of out start on 16-byte boundaries
};

__device__ __forceinline__ float scaled(int32_t acc, float sa, float sw, float bias) {
  return fmaf(static_cast<float>(acc), sa * sw, bias);
}

// ------------------------------------------------------------------------------------
// Few tokens (M <= kFewMax): the weights are read once and that is the whole cost, so a warp
// takes one output channel's row, 16 bytes a lane with several loads in flight, and forms the
// products of all tokens with four-way integer dot products (tokens' codes come through L1).
// ------------------------------------------------------------------------------------
constexpr int kFewMax = 8;
constexpr int kFewThreads = 256;

template <typename T, int MT>
__global__ void __launch_bounds__(kFewThreads) few_tokens_kernel(const MatArgs p) {
  using V = rotary::Vec<T>;
  const int32_t lane = threadIdx.x & 31;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * (kFewThreads / 32) + (threadIdx.x >> 5);
  if (n >= p.N) return;
  const int4* w = reinterpret_cast<const int4*>(p.w + n * p.kp);
  const int32_t vecs = p.kp / 16;
  int32_t acc[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) acc[m] = 0;
  constexpr int U = 4;
  for (int32_t v0 = lane; v0 < vecs; v0 += 32 * U) {
    int4 wv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      wv[u] = make_int4(0, 0, 0, 0);
      if (v0 + 32 * u < vecs) wv[u] = __ldcs(w + v0 + 32 * u);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (v0 + 32 * u >= vecs) continue;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (m >= p.M) continue;
        const int4 av = __ldg(reinterpret_cast<const int4*>(p.a + static_cast<int64_t>(m) * p.kp) + v0 + 32 * u);
        acc[m] = __dp4a(wv[u].x, av.x, acc[m]);
        acc[m] = __dp4a(wv[u].y, av.y, acc[m]);
        acc[m] = __dp4a(wv[u].z, av.z, acc[m]);
        acc[m] = __dp4a(wv[u].w, av.w, acc[m]);
      }
    }
  }
  const float sw = p.sw[n], bias = p.bias ? p.bias[n] : 0.f;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    if (m >= p.M) continue;
    const int32_t s = __reduce_add_sync(0xffffffffu, acc[m]);
    if (lane == m) static_cast<T*>(p.out)[m * p.ldo + n] = V::to(scaled(s, p.sa[m], sw, bias));
  }
}

// ------------------------------------------------------------------------------------
// The tensor-core product: persistent, one CTA per SM, 128 tokens x 256 channels per tile.
//   warp 4   TMA producer: per 128-deep K chunk, 128 rows of A and 256 rows of W (128-byte
//            swizzle) into a kStages-deep ring
//   warp 5   MMA issuer (one thread): four kind::i8 MMAs (M 128, N 256, K 32) a chunk into one of
//            two accumulators of 256 TMEM columns
//   warps 0..3  epilogue: 32 columns at a time, one output row per thread; overlaps the next
//            tile's main loop
// Tiles run channel-fastest, so the CTAs of one wave share a few rows of A and all of W from L2.
// Every wait is bounded; on a timeout the CTA raises its abort flag, the roles leave their loops,
// in-flight copies and MMAs are drained and the tensor memory is freed.
// ------------------------------------------------------------------------------------
constexpr int kThreads = 192;
constexpr int kStages = 4;
constexpr int kBM = 128, kBN = 256;
constexpr uint32_t kABytes = kBM * 128, kBBytes = kBN * 128;
constexpr uint32_t kStageB = kABytes + kBBytes;
constexpr uint32_t kSmemBytes = kStages * kStageB + 1024;
constexpr uint32_t kTmemCols = 512;

// Instruction descriptor of kind::i8: signed A and B, both K-major, s32 accumulator.
__host__ __device__ constexpr uint32_t idesc_s8_s32(int M, int N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ void mma_ss_i8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

struct Bars {
  uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], drain;
  uint32_t tmem_base;
  int abort;
};

// 32 accumulator columns of one output row: scale, bias, store.
template <typename T>
__device__ __forceinline__ void store32(const MatArgs& p, const uint32_t (&r)[32], int64_t m, int32_t n0, float sa) {
  using V = rotary::Vec<T>;
  T* row = static_cast<T*>(p.out) + m * p.ldo;
  if (p.out_vec && n0 + 32 <= p.N) {
#pragma unroll
    for (int j = 0; j < 32; j += V::E) {
      float f[V::E];
#pragma unroll
      for (int i = 0; i < V::E; ++i)
        f[i] = scaled(static_cast<int32_t>(r[j + i]), sa, __ldg(p.sw + n0 + j + i),
                      p.bias ? __ldg(p.bias + n0 + j + i) : 0.f);
      *reinterpret_cast<uint4*>(row + n0 + j) = V::put(f);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (n0 + j < p.N)
        row[n0 + j] = V::to(scaled(static_cast<int32_t>(r[j]), sa, __ldg(p.sw + n0 + j),
                                   p.bias ? __ldg(p.bias + n0 + j) : 0.f));
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
int8_gemm_kernel(const __grid_constant__ CUtensorMap mA, const __grid_constant__ CUtensorMap mB,
                 const __grid_constant__ MatArgs p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ Bars bars;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort = &bars.abort;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&bars.full[i]), 1);
      mbar_init(smem_u32(&bars.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars.acc_full[i]), 1);
      mbar_init(smem_u32(&bars.acc_empty[i]), 4);
    }
    mbar_init(smem_u32(&bars.drain), 1);
    bars.abort = 0;
    fence_mbar_init();
  }
  if (warp == 5) {
    tmem_alloc(smem_u32(&bars.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  if (warp == 4 && lane == 0) {
    prefetch_tensormap(&mA);
    prefetch_tensormap(&mB);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;

  if (warp < 4) {
    uint32_t it = 0;
    for (int64_t t = blockIdx.x; t < p.tiles; t += gridDim.x, ++it) {
      const int32_t m0 = static_cast<int32_t>(t / p.tiles_n) * kBM, n0 = static_cast<int32_t>(t % p.tiles_n) * kBN;
      const uint32_t ab = it & 1;
      if (!attn::warp_wait_abort(smem_u32(&bars.acc_full[ab]), (it >> 1) & 1, abort, 70)) break;
      tc_fence_after();
      const int32_t m = m0 + static_cast<int32_t>(warp * 32 + lane);
      const float sa = m < p.M ? p.sa[m] : 0.f;
      const uint32_t taddr = tmem + ((warp * 32) << 16) + ab * kBN;
#pragma unroll 1
      for (int cc = 0; cc < kBN / 32; ++cc) {
        if (n0 + cc * 32 >= p.N) break;
        uint32_t r[32];
        tmem_ld32_sync(taddr + cc * 32, r);
        if (m < p.M) store32<T>(p, r, m, n0 + cc * 32, sa);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.acc_empty[ab]));
    }
  } else if (warp == 4 && lane == 0) {
    uint32_t g = 0;
    for (int64_t t = blockIdx.x; t < p.tiles && !*abort; t += gridDim.x) {
      const int32_t m0 = static_cast<int32_t>(t / p.tiles_n) * kBM, n0 = static_cast<int32_t>(t % p.tiles_n) * kBN;
      for (int32_t c = 0; c < p.chunks; ++c, ++g) {
        const uint32_t s = g % kStages;
        if (g >= kStages && !mbar_wait(smem_u32(&bars.empty[s]), (g / kStages - 1) & 1, abort, 71)) {
          t = p.tiles;
          break;
        }
        const uint32_t st = sb + s * kStageB;
        mbar_arrive_expect_tx(smem_u32(&bars.full[s]), kStageB);
        tma_load_2d(st, &mA, smem_u32(&bars.full[s]), c * 128, m0);
        tma_load_2d(st + kABytes, &mB, smem_u32(&bars.full[s]), c * 128, n0);
      }
    }
    for (uint32_t i = g > kStages ? g - kStages : 0; i < g; ++i)
      mbar_wait(smem_u32(&bars.full[i % kStages]), (i / kStages) & 1, nullptr, 72);
  } else if (warp == 5 && lane == 0) {
    constexpr uint32_t kIdesc = idesc_s8_s32(kBM, kBN);
    uint32_t g = 0, it = 0;
    for (int64_t t = blockIdx.x; t < p.tiles; t += gridDim.x, ++it) {
      const uint32_t ab = it & 1;
      if (it >= 2 && !mbar_wait(smem_u32(&bars.acc_empty[ab]), ((it >> 1) - 1) & 1, abort, 73)) break;
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
        const uint64_t dB = smem_desc_sw128(sb + s * kStageB + kABytes, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)   // 32 codes = 32 bytes per k-step: +2 in 16-byte units
          mma_ss_i8(tmem + ab * kBN, dA + kk * 2, dB + kk * 2, kIdesc, (c > 0 || kk > 0) ? 1u : 0u);
        tc_commit(smem_u32(&bars.empty[s]));
      }
      if (!ok) break;
      tc_commit(smem_u32(&bars.acc_full[ab]));
    }
    tc_commit(smem_u32(&bars.drain));
    mbar_wait(smem_u32(&bars.drain), 0, nullptr, 75);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 5) tmem_dealloc(tmem, kTmemCols);
}

}  // namespace int8
}  // namespace veda
