// k_norm.cuh -- the norms before and after a transformer block, fused with what stands around
// them: scale and shift of the conditioning before the block, gate and residual sum after it,
// and their backward.
//
//   xh = (x - mean) rstd                (layer), x rstd (rms), x (none)
//   before:  y = (xh w + b) (1 + scale_B) + shift_B
//   after:   y = residual_scale * residual + gate_B (xh w + b)
// Both are y = r * residual + xh * A_B + S_B with A_B = G_B w, S_B = G_B b + shift_B and
// G = 1 + scale or gate, so one kernel serves both.
//
// Backward, for dy, with g = dy A_B:
//   dx = rstd (g - mean(g) - xh mean(g xh))   (rms: no mean(g); none: dx = g)
//        + r * d_residual                     (the gradient that flows around the block)
// and every parameter's gradient follows from two sums over a sequence's tokens,
// P1_B = sum dy xh and P2_B = sum dy:
//   dG_B = w P1_B + b P2_B,  dshift_B = P2_B,  dw = sum_B G_B P1_B,  db = sum_B G_B P2_B.
//
// All of it is HBM bound: a row is read once and written once, everything between is registers.
// A row belongs to a group of threads -- a warp for up to 1,024 channels, a CTA above -- whose
// thread i owns the 8-channel vectors i, i + threads, ...; it therefore keeps A, S (forward) or
// A, P1, P2 (backward) of its channels in registers for all the rows of its slice of one
// sequence. Rows come through a ring of 2 to 4 rows in shared memory that each thread fills
// for itself with 16-byte asynchronous copies (it reads back only what it copied, so no barrier
// guards the ring); the only barriers are the row reductions'. Statistics and sums are fp32: the
// variance is the mean square of the centred values (two passes over registers, not E[x^2] -
// mean^2), the sums over tokens are fp32 per slice, then over the slices in a fixed order, so
// results do not change from run to run.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace veda {
namespace norm {

enum : int32_t { kLayer = 0, kRms = 1, kNone = 2 };
enum : int32_t { kBf16 = 0, kFp16 = 1, kFp32 = 2 };

constexpr int kVec = 8;            // channels per vector
constexpr int kWarpCols = 1024;    // widest row of the warp-per-row kernels
constexpr int kMaxCols = 8192;
constexpr int kMaxThreads = 512;
constexpr int kWarpsPerCta = 8;    // warp-per-row kernels

struct Param {                     // a parameter vector of C values, with a batch stride
  const void* p;
  int64_t bs;
  int32_t dtype;
};

struct Args {
  const void* x;
  const void* res;                 // forward: residual; backward: gradient around the block; or null
  const void* dy;                  // backward
  void* y;                         // forward: y; backward: dx
  int64_t xb, xn, rb, rn, db, dn, yb, yn;   // element strides (batch, token)
  Param w, b, g, t;
  float gain_off, res_scale, eps, inv_c;
  float* mean;                     // forward: out or null; backward: in
  float* rstd;
  float* part;                     // backward: [B * slices][2][C] partial P1, P2
  int32_t B, N, C, kind, slices;
  int32_t stages;                  // rows in the ring: 2 to 4
  int32_t vec;                     // every row starts on a 16-byte boundary and C % 8 == 0
};

__device__ __forceinline__ float load_param(const Param& q, int32_t b, int32_t c) {
  const int64_t i = b * q.bs + c;
  if (q.dtype == kBf16) return __bfloat162float(static_cast<const __nv_bfloat16*>(q.p)[i]);
  if (q.dtype == kFp16) return __half2float(static_cast<const __half*>(q.p)[i]);
  return static_cast<const float*>(q.p)[i];
}

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }

// One 8-channel vector of T in 16-byte units: 1 (16-bit types) or 2 (fp32).
template <typename T> constexpr int units_of() { return sizeof(T) * kVec / 16; }

template <typename T>
__device__ __forceinline__ void unpack(const uint4* u, float* f) {
  const T* p = reinterpret_cast<const T*>(u);
#pragma unroll
  for (int i = 0; i < kVec; ++i) f[i] = to_f<T>(p[i]);
}

__device__ __forceinline__ uint32_t shared_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(shared_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// The oldest row of a ring of `stages` rows has landed (the count is an immediate).
__device__ __forceinline__ void wait_oldest(int32_t stages) {
  if (stages == 4) cp_async_wait<2>();
  else if (stages == 3) cp_async_wait<1>();
  else cp_async_wait<0>();
}

// This thread's share of a row of T into its own ring slots (slot stride: `threads` units).
template <typename T, int NV>
__device__ __forceinline__ void fetch_row(uint4* ring, const T* row, int32_t me, int32_t threads, int32_t C,
                                          bool vec) {
  constexpr int U = units_of<T>();
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int32_t c0 = (me + j * threads) * kVec;
    if (c0 >= C) continue;
    if (vec) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        cp_async16(ring + (j * U + u) * threads, reinterpret_cast<const uint4*>(row + c0) + u);
    } else {
      uint4 tmp[U];
      T* p = reinterpret_cast<T*>(tmp);
#pragma unroll
      for (int i = 0; i < kVec; ++i) p[i] = c0 + i < C ? row[c0 + i] : from_f<T>(0.f);
#pragma unroll
      for (int u = 0; u < U; ++u) ring[(j * U + u) * threads] = tmp[u];
    }
  }
}

template <typename T>
__device__ __forceinline__ void read_vec(const uint4* ring, int j, int32_t threads, float* f) {
  constexpr int U = units_of<T>();
  uint4 tmp[U];
#pragma unroll
  for (int u = 0; u < U; ++u) tmp[u] = ring[(j * U + u) * threads];
  unpack<T>(tmp, f);
}

template <typename T>
__device__ __forceinline__ void store_vec(T* row, int32_t c0, int32_t C, bool vec, const float* f) {
  constexpr int U = units_of<T>();
  uint4 tmp[U];
  T* p = reinterpret_cast<T*>(tmp);
#pragma unroll
  for (int i = 0; i < kVec; ++i) p[i] = from_f<T>(f[i]);
  if (vec) {
#pragma unroll
    for (int u = 0; u < U; ++u) reinterpret_cast<uint4*>(row + c0)[u] = tmp[u];
  } else {
    for (int i = 0; i < kVec && c0 + i < C; ++i) row[c0 + i] = p[i];
  }
}

// Sum of V values over the group. Warp groups: butterflies, every lane gets the sum in the same
// order. CTA groups: one butterfly, one shared row per warp, one barrier; `buf` alternates so
// that a slow warp's reads are separated from the next writes by a barrier.
template <bool kWarp, int V>
__device__ __forceinline__ void group_sum(float (&v)[V], float (*buf)[V], int32_t warps) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (kWarp) return;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) buf[threadIdx.x >> 5][i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = 0.f;
  for (int32_t w = 0; w < warps; ++w)
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] += buf[w][i];
}

struct Slice { int32_t b, lo, hi; };
__device__ __forceinline__ Slice slice_of(const Args& a) {
  Slice s;
  s.b = blockIdx.x / a.slices;
  const int32_t i = blockIdx.x - s.b * a.slices;
  s.lo = static_cast<int32_t>(static_cast<int64_t>(a.N) * i / a.slices);
  s.hi = static_cast<int32_t>(static_cast<int64_t>(a.N) * (i + 1) / a.slices);
  return s;
}

// ------------------------------------------------------------------------------------
// Forward. TI: type of x; TO: type of y and of the residual.
// ------------------------------------------------------------------------------------
template <typename TI, typename TO, int NV, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 32 * kWarpsPerCta : kMaxThreads) norm_fwd_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(16) uint4 ring_base[];
  __shared__ float red[2][kMaxThreads / 32][1];
  constexpr int UI = units_of<TI>(), UO = units_of<TO>();
  const int32_t threads = kWarp ? 32 : static_cast<int32_t>(blockDim.x);
  const int32_t me = kWarp ? (threadIdx.x & 31) : threadIdx.x;
  const int32_t warps = threads / 32;
  const bool has_res = a.res != nullptr;
  const int stage_units = NV * (UI + (has_res ? UO : 0));
  uint4* ring = ring_base + (kWarp ? (threadIdx.x >> 5) * a.stages * stage_units * 32 : 0) + me;
  const Slice s = slice_of(a);
  const int32_t step = kWarp ? kWarpsPerCta : 1;
  const int32_t first = s.lo + (kWarp ? static_cast<int32_t>(threadIdx.x >> 5) : 0);
  const TI* x = static_cast<const TI*>(a.x) + s.b * a.xb;
  const TO* res = has_res ? static_cast<const TO*>(a.res) + s.b * a.rb : nullptr;
  TO* y = static_cast<TO*>(a.y) + s.b * a.yb;
  const bool vec = a.vec != 0;

  auto fetch = [&](int32_t row, int st) {
    if (row < s.hi) {
      uint4* slot = ring + st * stage_units * threads;
      fetch_row<TI, NV>(slot, x + row * a.xn, me, threads, a.C, vec);
      if (has_res) fetch_row<TO, NV>(slot + NV * UI * threads, res + row * a.rn, me, threads, a.C, vec);
    }
    cp_async_commit();
  };
  const int32_t stages = a.stages;
  for (int i = 0; i < stages - 1; ++i) fetch(first + i * step, i);

  // A and S of this thread's channels
  float A[NV][kVec], S[NV][kVec];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int32_t c = (me + j * threads) * kVec + i;
      float w = 0.f, sh = 0.f;
      if (c < a.C) {
        const float gain = a.g.p ? a.gain_off + load_param(a.g, s.b, c) : 1.f;
        w = a.w.p ? gain * load_param(a.w, 0, c) : gain;
        sh = a.t.p ? load_param(a.t, s.b, c) : 0.f;
        if (a.b.p) sh = fmaf(gain, load_param(a.b, 0, c), sh);
      }
      A[j][i] = w;
      S[j][i] = sh;
    }
  }

  int st = 0;
  int32_t flip = 0;
  for (int32_t row = first; row < s.hi; row += step) {
    wait_oldest(stages);
    const uint4* slot = ring + st * stage_units * threads;
    float v[NV][kVec];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int32_t c0 = (me + j * threads) * kVec;
      if (c0 < a.C) {
        read_vec<TI>(slot, j, threads, v[j]);
      } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[j][i] = 0.f;
      }
    }
    // the row that will use the slot read in the previous round
    fetch(row + (stages - 1) * step, st == 0 ? stages - 1 : st - 1);
    float mean = 0.f, rstd = 1.f;
    if (a.kind == kLayer) {
      float m[1] = {0.f};
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < kVec; ++i) m[0] += v[j][i];
      group_sum<kWarp, 1>(m, red[flip], warps);
      flip ^= 1;
      mean = m[0] * a.inv_c;
    }
    if (a.kind != kNone) {
      float q[1] = {0.f};
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int32_t c0 = (me + j * threads) * kVec;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          v[j][i] = c0 + i < a.C ? v[j][i] - mean : 0.f;
          q[0] = fmaf(v[j][i], v[j][i], q[0]);
        }
      }
      group_sum<kWarp, 1>(q, red[flip], warps);
      flip ^= 1;
      rstd = 1.0f / sqrtf(fmaf(q[0], a.inv_c, a.eps));
    }
    if (a.rstd != nullptr && me == 0) {
      const int64_t r = static_cast<int64_t>(s.b) * a.N + row;
      if (a.mean != nullptr) a.mean[r] = mean;
      a.rstd[r] = rstd;
    }
    TO* out = y + row * a.yn;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int32_t c0 = (me + j * threads) * kVec;
      if (c0 >= a.C) continue;
      float o[kVec];
#pragma unroll
      for (int i = 0; i < kVec; ++i) o[i] = fmaf(v[j][i] * rstd, A[j][i], S[j][i]);
      if (has_res) {
        float r[kVec];
        read_vec<TO>(slot + NV * UI * threads, j, threads, r);
#pragma unroll
        for (int i = 0; i < kVec; ++i) o[i] = fmaf(r[i], a.res_scale, o[i]);
      }
      store_vec<TO>(out, c0, a.C, vec, o);
    }
    st = st == stages - 1 ? 0 : st + 1;
  }
  cp_async_wait<0>();
}

// ------------------------------------------------------------------------------------
// Backward. TI: type of x, dx and of the gradient around the block; TO: type of dy.
// ------------------------------------------------------------------------------------
template <typename TI, typename TO, int NV, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 32 * kWarpsPerCta : kMaxThreads) norm_bwd_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(16) uint4 ring_base[];
  __shared__ float red[2][kMaxThreads / 32][2];
  constexpr int UI = units_of<TI>(), UO = units_of<TO>();
  const int32_t threads = kWarp ? 32 : static_cast<int32_t>(blockDim.x);
  const int32_t me = kWarp ? (threadIdx.x & 31) : threadIdx.x;
  const int32_t warps = threads / 32;
  const bool has_res = a.res != nullptr;
  const int stage_units = NV * (UI + UO + (has_res ? UI : 0));
  uint4* ring = ring_base + (kWarp ? (threadIdx.x >> 5) * a.stages * stage_units * 32 : 0) + me;
  const Slice s = slice_of(a);
  const int32_t step = kWarp ? kWarpsPerCta : 1;
  const int32_t first = s.lo + (kWarp ? static_cast<int32_t>(threadIdx.x >> 5) : 0);
  const TI* x = static_cast<const TI*>(a.x) + s.b * a.xb;
  const TO* dy = static_cast<const TO*>(a.dy) + s.b * a.db;
  const TI* res = has_res ? static_cast<const TI*>(a.res) + s.b * a.rb : nullptr;
  TI* dx = static_cast<TI*>(a.y) + s.b * a.yb;
  const bool vec = a.vec != 0;

  auto fetch = [&](int32_t row, int st) {
    if (row < s.hi) {
      uint4* slot = ring + st * stage_units * threads;
      fetch_row<TI, NV>(slot, x + row * a.xn, me, threads, a.C, vec);
      fetch_row<TO, NV>(slot + NV * UI * threads, dy + row * a.dn, me, threads, a.C, vec);
      if (has_res)
        fetch_row<TI, NV>(slot + NV * (UI + UO) * threads, res + row * a.rn, me, threads, a.C, vec);
    }
    cp_async_commit();
  };
  const int32_t stages = a.stages;
  for (int i = 0; i < stages - 1; ++i) fetch(first + i * step, i);

  float A[NV][kVec], P1[NV][kVec], P2[NV][kVec];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int32_t c = (me + j * threads) * kVec + i;
      float w = 0.f;
      if (c < a.C) {
        w = a.g.p ? a.gain_off + load_param(a.g, s.b, c) : 1.f;
        if (a.w.p) w *= load_param(a.w, 0, c);
      }
      A[j][i] = w;
      P1[j][i] = P2[j][i] = 0.f;
    }
  }

  int st = 0;
  int32_t flip = 0;
  for (int32_t row = first; row < s.hi; row += step) {
    const int64_t r = static_cast<int64_t>(s.b) * a.N + row;
    const float mean = a.kind == kLayer ? __ldg(a.mean + r) : 0.f;
    const float rstd = a.kind != kNone ? __ldg(a.rstd + r) : 1.f;
    wait_oldest(stages);
    const uint4* slot = ring + st * stage_units * threads;
    float xh[NV][kVec], g[NV][kVec];
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int32_t c0 = (me + j * threads) * kVec;
      if (c0 < a.C) {
        read_vec<TI>(slot, j, threads, xh[j]);
        read_vec<TO>(slot + NV * UI * threads, j, threads, g[j]);
      } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) xh[j][i] = g[j][i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        xh[j][i] = (xh[j][i] - mean) * rstd;
        P1[j][i] = fmaf(g[j][i], xh[j][i], P1[j][i]);
        P2[j][i] += g[j][i];
        g[j][i] *= A[j][i];                       // 0 past the last channel
        sum[0] += g[j][i];
        sum[1] = fmaf(g[j][i], xh[j][i], sum[1]);
      }
    }
    fetch(row + (stages - 1) * step, st == 0 ? stages - 1 : st - 1);
    float c1 = 0.f, c2 = 0.f;
    if (a.kind != kNone) {
      group_sum<kWarp, 2>(sum, red[flip], warps);
      flip ^= 1;
      c1 = a.kind == kLayer ? sum[0] * a.inv_c : 0.f;
      c2 = sum[1] * a.inv_c;
    }
    TI* out = dx + row * a.yn;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int32_t c0 = (me + j * threads) * kVec;
      if (c0 >= a.C) continue;
      float o[kVec];
#pragma unroll
      for (int i = 0; i < kVec; ++i) o[i] = (fmaf(-xh[j][i], c2, g[j][i]) - c1) * rstd;
      if (has_res) {
        float q[kVec];
        read_vec<TI>(slot + NV * (UI + UO) * threads, j, threads, q);
#pragma unroll
        for (int i = 0; i < kVec; ++i) o[i] = fmaf(q[i], a.res_scale, o[i]);
      }
      store_vec<TI>(out, c0, a.C, vec, o);
    }
    st = st == stages - 1 ? 0 : st + 1;
  }
  cp_async_wait<0>();

  // this CTA's partial sums (warp groups: added up in shared memory, in warp order)
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.C;
  if (!kWarp) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const int32_t c = (me + j * threads) * kVec + i;
        if (c < a.C) {
          part[c] = P1[j][i];
          part[a.C + c] = P2[j][i];
        }
      }
    }
    return;
  }
  float* acc = reinterpret_cast<float*>(ring_base);      // [2][NV * 256]: the ring is drained
  constexpr int32_t W = NV * 32 * kVec;
  for (int32_t w = 0; w < kWarpsPerCta; ++w) {
    __syncthreads();
    if (static_cast<int32_t>(threadIdx.x >> 5) != w) continue;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const int32_t c = (me + j * 32) * kVec + i;
        acc[c] = w ? acc[c] + P1[j][i] : P1[j][i];
        acc[W + c] = w ? acc[W + c] + P2[j][i] : P2[j][i];
      }
    }
  }
  __syncthreads();
  for (int32_t c = threadIdx.x; c < a.C; c += 32 * kWarpsPerCta) {
    part[c] = acc[c];
    part[a.C + c] = acc[W + c];
  }
}

// ------------------------------------------------------------------------------------
// Parameter gradients from the slices' sums. One CTA per 32 channels and sequence: 8 rows of
// threads add up the slices (a fixed assignment and order), then
//   dG = w P1 + b P2, dshift = P2, and the sequence's G P1, G P2 for dw, db.
// ------------------------------------------------------------------------------------
struct GradArgs {
  const float* part;       // [B * slices][2][C]
  Param w, b, g;
  float gain_off;
  float* dgain;            // null or [B][C]
  float* dshift;           // null or [B][C]
  float* gp;               // [B][2][C]: G P1, G P2 (null when neither dw nor db is asked for)
  int32_t B, C, slices;
};
constexpr int kGradRows = 8;

__global__ void __launch_bounds__(32 * kGradRows) norm_grad_kernel(const __grid_constant__ GradArgs a) {
  __shared__ float s1[kGradRows][32], s2[kGradRows][32];
  const int32_t col = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int32_t c = blockIdx.x * 32 + col, b = blockIdx.y;
  float p1 = 0.f, p2 = 0.f;
  if (c < a.C) {
    const float* part = a.part + static_cast<int64_t>(b) * a.slices * 2 * a.C + c;
#pragma unroll 4
    for (int32_t i = r; i < a.slices; i += kGradRows) {
      p1 += part[static_cast<int64_t>(i) * 2 * a.C];
      p2 += part[static_cast<int64_t>(i) * 2 * a.C + a.C];
    }
  }
  s1[r][col] = p1;
  s2[r][col] = p2;
  __syncthreads();
  if (r != 0 || c >= a.C) return;
#pragma unroll
  for (int i = 1; i < kGradRows; ++i) {
    p1 += s1[i][col];
    p2 += s2[i][col];
  }
  const int64_t o = static_cast<int64_t>(b) * a.C + c;
  if (a.dgain) {
    const float w = a.w.p ? load_param(a.w, 0, c) : 1.f;
    a.dgain[o] = a.b.p ? fmaf(w, p1, load_param(a.b, 0, c) * p2) : w * p1;
  }
  if (a.dshift) a.dshift[o] = p2;
  if (a.gp) {
    const float G = a.g.p ? a.gain_off + load_param(a.g, b, c) : 1.f;
    a.gp[static_cast<int64_t>(b) * 2 * a.C + c] = G * p1;
    a.gp[static_cast<int64_t>(b) * 2 * a.C + a.C + c] = G * p2;
  }
}

// dw, db: the sequences' G P1, G P2 added up in order.
__global__ void __launch_bounds__(256) norm_weight_grad_kernel(const float* gp, float* dw, float* db, int32_t B,
                                                               int32_t C) {
  const int32_t c = blockIdx.x * 256 + threadIdx.x;
  if (c >= C) return;
  float a = 0.f, b = 0.f;
  for (int32_t i = 0; i < B; ++i) {
    a += gp[static_cast<int64_t>(i) * 2 * C + c];
    b += gp[static_cast<int64_t>(i) * 2 * C + C + c];
  }
  if (dw) dw[c] = a;
  if (db) db[c] = b;
}

}  // namespace norm
}  // namespace veda
