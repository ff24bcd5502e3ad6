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
// A row belongs to a group of threads -- a warp for up to 1,024 channels (256 where rows have no
// 16-byte boundaries), a CTA above -- whose thread i owns the 8-channel vectors i, i + threads, ...;
// it therefore keeps A, S (forward) or A, P1, P2 (backward) of its channels in registers for all the
// rows of its slice of one sequence. Rows come through a ring of 2 to 4 rows in shared memory that
// each thread fills for itself, with 16-byte asynchronous copies where rows have those boundaries
// (it reads back only what it copied, so no barrier guards the ring); the only barriers are the row
// reductions'. Statistics and sums are fp32: the
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
  int32_t vec;                     // its rows start on 16-byte boundaries and C % 8 == 0
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
  int32_t* done;                   // backward: null, or norm_grad_kernel's counters to clear
  int32_t B, N, C, kind, slices;
  int32_t stages;                  // rows in the ring: 2 to 4
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

__device__ __forceinline__ uint32_t shared_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(shared_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(shared_addr(dst)), "l"(src) : "memory");
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

// Pairs of fp32 values in one 64-bit register: one instruction for two channels.
typedef unsigned long long f2;
__device__ __forceinline__ f2 pair(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 split(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
constexpr int kPairs = kVec / 2;

// One 8-channel vector as four pairs.
template <typename T>
__device__ __forceinline__ void unpack(const uint4* u, f2* f) {
  const T* p = reinterpret_cast<const T*>(u);
#pragma unroll
  for (int i = 0; i < kPairs; ++i) f[i] = pair(to_f<T>(p[2 * i]), to_f<T>(p[2 * i + 1]));
}
template <> __device__ __forceinline__ void unpack<__nv_bfloat16>(const uint4* u, f2* f) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(u);
#pragma unroll
  for (int i = 0; i < kPairs; ++i) f[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}

// Four pairs as one 8-channel vector, each value rounded once.
template <typename T> __device__ __forceinline__ void pack(const f2* f, uint4* u);
template <> __device__ __forceinline__ void pack<__nv_bfloat16>(const f2* f, uint4* u) {
  __nv_bfloat162* p = reinterpret_cast<__nv_bfloat162*>(u);
#pragma unroll
  for (int i = 0; i < kPairs; ++i) p[i] = __float22bfloat162_rn(split(f[i]));
}
template <> __device__ __forceinline__ void pack<__half>(const f2* f, uint4* u) {
  __half2* p = reinterpret_cast<__half2*>(u);
#pragma unroll
  for (int i = 0; i < kPairs; ++i) p[i] = __float22half2_rn(split(f[i]));
}
template <> __device__ __forceinline__ void pack<float>(const f2* f, uint4* u) {
  float2* p = reinterpret_cast<float2*>(u);
#pragma unroll
  for (int i = 0; i < kPairs; ++i) p[i] = split(f[i]);
}

// 1 / sqrt(v): the hardware's approximation and one Newton step (within an fp32 step or two).
__device__ __forceinline__ float inv_sqrt(float v) {
  const float r = rsqrtf(v);
  const float n = fmaf(0.5f * r, fmaf(-v * r, r, 1.0f), r);
  return v > 0x1p-120f && v < 0x1p120f ? n : r;     // the step itself would leave fp32's range
}

// Which channels thread `me` of `threads` owns: NV vectors of two halves of four channels.
//   kVectors: a vector is eight neighbouring channels, vectors `threads` apart (16-byte accesses of
//     16-bit types);
//   kHalves: every half is on its own, halves `threads` apart, so that the accesses of a warp to fp32
//     rows are contiguous too (two 16-byte accesses a vector 32 bytes apart fetch every sector twice:
//     58% of the HBM copy rate where this has 80%); 16-bit rows beside them move in 8-byte pieces;
//   kSingle: rows without 16-byte boundaries: every channel on its own, channels `threads` apart; the
//     CTA's size is a constant there (kFixed), as a channel's address would otherwise cost more than the
//     channel's arithmetic (backward of 6,147 rows of 1,023: 33 us with a run-time size, 24 with this).
enum : int { kSingle = 0, kVectors = 1, kHalves = 2 };
template <int kMode>
struct Own {
  static constexpr int mode = kMode;
  static constexpr bool vec = kMode != kSingle;
  int32_t me, threads, C;
  // first channel of half u of vector j (aligned rows)
  __device__ __forceinline__ int32_t first(int j, int u) const {
    return kMode == kVectors ? (me + j * threads) * kVec + 4 * u : (me + (2 * j + u) * threads) * 4;
  }
  __device__ __forceinline__ bool has(int j, int u) const { return first(j, u) < C; }
  __device__ __forceinline__ int32_t one(int j, int i) const {
    return vec ? first(j, i / 4) + i % 4 : me + (j * kVec + i) * threads;
  }
  // some channel of vector j exists
  __device__ __forceinline__ bool any(int j) const { return (vec ? first(j, 0) : me + j * kVec * threads) < C; }
};

// This thread's share of a row of T on its way into its own ring slots (slot stride: `threads`
// units). Aligned rows go there by asynchronous copies. Other rows are read one channel at a time by plain
// loads (the smallest asynchronous copy has 4 bytes, which 16-bit rows at an odd channel cannot use; fp32
// rows, which could, go the same way): start() issues them into registers, finish() -- a row's work
// later -- writes the ring.
template <typename T, int NV, typename O>
struct Fetch {
  static constexpr int U = units_of<T>();
  uint4 held[O::vec ? 1 : NV][O::vec ? 1 : U];
  __device__ __forceinline__ void start(uint4* ring, const T* row, const O& o) {
    if constexpr (O::vec) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if constexpr (O::mode == kVectors && U == 1) {
          if (o.has(j, 0)) cp_async16(ring + j * o.threads, row + o.first(j, 0));
        } else {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if (!o.has(j, u)) continue;
            if constexpr (U == 2) cp_async16(ring + (2 * j + u) * o.threads, row + o.first(j, u));
            else cp_async8(reinterpret_cast<uint2*>(ring + j * o.threads) + u, row + o.first(j, u));
          }
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        T* p = reinterpret_cast<T*>(held[j]);
#pragma unroll
        for (int i = 0; i < kVec; ++i) p[i] = o.one(j, i) < o.C ? row[o.one(j, i)] : from_f<T>(0.f);
      }
    }
  }
  __device__ __forceinline__ void finish(uint4* ring, const O& o) const {
    if constexpr (!O::vec) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int u = 0; u < U; ++u) ring[(j * U + u) * o.threads] = held[j][u];
    }
  }
};

// Vector j of a ring row (zeros where the thread owns nothing).
template <typename T, typename O>
__device__ __forceinline__ void read_vec(const uint4* ring, int j, const O& o, f2* f) {
  constexpr int U = units_of<T>();
  if (o.any(j)) {
    uint4 tmp[U];
#pragma unroll
    for (int u = 0; u < U; ++u) tmp[u] = ring[(j * U + u) * o.threads];
    unpack<T>(tmp, f);
  } else {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) f[i] = 0ull;
  }
  if (O::mode == kHalves && !o.has(j, 1)) f[2] = f[3] = 0ull;
}

template <typename T, typename O>
__device__ __forceinline__ void store_vec(T* row, int j, const O& o, const f2* f) {
  constexpr int U = units_of<T>();
  uint4 tmp[U];
  pack<T>(f, tmp);
  const T* p = reinterpret_cast<const T*>(tmp);
  if constexpr (O::mode == kVectors && U == 1) {
    *reinterpret_cast<uint4*>(row + o.first(j, 0)) = tmp[0];
  } else if constexpr (O::vec) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (!o.has(j, u)) continue;
      if constexpr (U == 2) *reinterpret_cast<uint4*>(row + o.first(j, u)) = tmp[u];
      else *reinterpret_cast<uint2*>(row + o.first(j, u)) = reinterpret_cast<const uint2*>(tmp)[u];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (o.one(j, i) < o.C) row[o.one(j, i)] = p[i];
  }
}

// A parameter's values of this thread's channels (0 where it owns nothing), in 16-byte loads that
// are all in flight together where its rows allow.
template <typename T, int NV, typename O>
__device__ __forceinline__ void param_values(const T* p, bool vec, const O& o, float (*f)[kVec]) {
  constexpr int U = units_of<T>();
  if (vec && O::vec) {
    uint4 raw[NV][U];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int u = 0; u < U; ++u) raw[j][u] = make_uint4(0, 0, 0, 0);
      if constexpr (O::mode == kVectors && U == 1) {
        if (o.has(j, 0)) raw[j][0] = __ldg(reinterpret_cast<const uint4*>(p + o.first(j, 0)));
      } else {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (!o.has(j, u)) continue;
          if constexpr (U == 2) raw[j][u] = __ldg(reinterpret_cast<const uint4*>(p + o.first(j, u)));
          else reinterpret_cast<uint2*>(raw[j])[u] = __ldg(reinterpret_cast<const uint2*>(p + o.first(j, u)));
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const T* t = reinterpret_cast<const T*>(raw[j]);
#pragma unroll
      for (int i = 0; i < kVec; ++i) f[j][i] = to_f<T>(t[i]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < kVec; ++i) f[j][i] = o.one(j, i) < o.C ? to_f<T>(p[o.one(j, i)]) : 0.f;
  }
}
template <int NV, typename O>
__device__ __forceinline__ void load_params(const Param& q, int32_t b, const O& o, float (*f)[kVec]) {
  if (q.dtype == kBf16)
    param_values<__nv_bfloat16, NV>(static_cast<const __nv_bfloat16*>(q.p) + b * q.bs, q.vec != 0, o, f);
  else if (q.dtype == kFp16)
    param_values<__half, NV>(static_cast<const __half*>(q.p) + b * q.bs, q.vec != 0, o, f);
  else
    param_values<float, NV>(static_cast<const float*>(q.p) + b * q.bs, q.vec != 0, o, f);
}

// Sum of V values over the group. Warp groups: butterflies, every lane gets the sum in the same
// order. CTA groups: one butterfly, one shared value per warp, one barrier; `buf` (zero past the
// last warp) alternates so that a slow warp's reads are separated from the next writes by a
// barrier.
constexpr int kMaxWarps = kMaxThreads / 32;
template <bool kWarp, int V>
__device__ __forceinline__ void group_sum(float (&v)[V], float (*buf)[kMaxWarps]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (kWarp) return;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) buf[i][threadIdx.x >> 5] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float4 q[kMaxWarps / 4];
#pragma unroll
    for (int w = 0; w < kMaxWarps / 4; ++w) q[w] = reinterpret_cast<const float4*>(buf[i])[w];
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kMaxWarps / 4; ++w) {
      t.x += q[w].x;
      t.y += q[w].y;
      t.z += q[w].z;
      t.w += q[w].w;
    }
    v[i] = (t.x + t.y) + (t.z + t.w);
  }
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
// Forward. TI: type of x; TO: type of y and of the residual. Registers leave room for two CTAs an SM (64
// at 512 threads, 128 at 256), so that one's barriers hide behind the other's work; rings of wide fp32
// rows do not (with a residual one CTA runs from 4,096 channels on, where four rows in flight are worth more).
// ------------------------------------------------------------------------------------
template <typename TI, typename TO, int NV, bool kWarp, int kMode, int kFixed>
__global__ void __launch_bounds__(kWarp ? 32 * kWarpsPerCta : NV == 4 ? 256 : kMaxThreads, 2)
norm_fwd_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(16) uint4 ring_base[];
  __shared__ __align__(16) float red[2][1][kMaxWarps];
  constexpr int UI = units_of<TI>(), UO = units_of<TO>();
  const int32_t threads = kWarp ? 32 : kFixed ? kFixed : static_cast<int32_t>(blockDim.x);
  const Own<kMode> o{kWarp ? static_cast<int32_t>(threadIdx.x & 31) : static_cast<int32_t>(threadIdx.x), threads, a.C};
  const bool has_res = a.res != nullptr;
  const int stage_units = NV * (UI + (has_res ? UO : 0)) * threads;
  uint4* ring = ring_base + (kWarp ? (threadIdx.x >> 5) * a.stages * stage_units : 0) + o.me;
  const Slice s = slice_of(a);
  const int32_t step = kWarp ? kWarpsPerCta : 1;
  const int32_t first = s.lo + (kWarp ? static_cast<int32_t>(threadIdx.x >> 5) : 0);
  const TI* x = static_cast<const TI*>(a.x) + s.b * a.xb;
  const TO* res = has_res ? static_cast<const TO*>(a.res) + s.b * a.rb : nullptr;
  TO* y = static_cast<TO*>(a.y) + s.b * a.yb;
  if (!kWarp && threadIdx.x < 2 * kMaxWarps) (&red[0][0][0])[threadIdx.x] = 0.f;

  // rows are fetched one after the other: the next one's addresses
  x += first * a.xn;
  if (has_res) res += first * a.rn;
  y += first * a.yn;
  const int64_t xstep = step * a.xn, rstep = step * a.rn, ystep = step * a.yn;
  int32_t next = first;
  Fetch<TI, NV, Own<kMode>> fx;
  Fetch<TO, NV, Own<kMode>> fr;
  auto start = [&](uint4* slot) {
    if (next < s.hi) {
      fx.start(slot, x, o);
      if (has_res) fr.start(slot + NV * UI * threads, res, o);
    }
    cp_async_commit();
    x += xstep;
    res += rstep;
    next += step;
  };
  auto finish = [&](uint4* slot) {           // of a row past the slice: stale values that no one reads
    fx.finish(slot, o);
    if (has_res) fr.finish(slot + NV * UI * threads, o);
  };
  const int32_t stages = a.stages;
  uint4* const ring_end = ring + stages * stage_units;
  uint4* free_slot = ring;
  for (int i = 0; i < stages - 1; ++i, free_slot += stage_units) {
    start(free_slot);
    finish(free_slot);
  }

  // A and S of this thread's channels
  f2 A[NV][kPairs], S[NV][kPairs];
  {
    float g[NV][kVec], w[NV][kVec], sh[NV][kVec];
    if (a.g.p) load_params<NV>(a.g, s.b, o, g);
    if (a.w.p) load_params<NV>(a.w, 0, o, w);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        g[j][i] = a.g.p ? a.gain_off + g[j][i] : 1.f;
        w[j][i] = a.w.p ? g[j][i] * w[j][i] : g[j][i];
        sh[j][i] = 0.f;
      }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < kPairs; ++i) A[j][i] = pair(w[j][2 * i], w[j][2 * i + 1]);
    if (a.t.p) load_params<NV>(a.t, s.b, o, sh);
    if (a.b.p) {
      load_params<NV>(a.b, 0, o, w);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < kVec; ++i) sh[j][i] = fmaf(g[j][i], w[j][i], sh[j][i]);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < kPairs; ++i) S[j][i] = pair(sh[j][2 * i], sh[j][2 * i + 1]);
  }
  if (!kWarp) __syncthreads();                     // red is zero

  uint4* slot = ring;
  int32_t flip = 0;
  for (int32_t row = first; row < s.hi; row += step) {
    wait_oldest(stages);
    f2 v[NV][kPairs];
#pragma unroll
    for (int j = 0; j < NV; ++j) read_vec<TI>(slot, j, o, v[j]);
    start(free_slot);                              // the slot read in the previous round
    float mean = 0.f, rstd = 1.f;
    if (a.kind == kLayer) {
      f2 t = 0ull;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < kPairs; ++i) t = add2(t, v[j][i]);
      float m[1] = {split(t).x + split(t).y};
      group_sum<kWarp, 1>(m, red[flip]);
      flip ^= 1;
      mean = m[0] * a.inv_c;
      const f2 sub = pair(-mean, -mean);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!o.any(j)) continue;                   // what the thread does not own stays 0
#pragma unroll
        for (int i = 0; i < kPairs; ++i)
          if (o.mode != kHalves || i < 2 || o.has(j, 1)) v[j][i] = add2(v[j][i], sub);
        if (!o.vec) {
#pragma unroll
          for (int i = 0; i < kPairs; ++i) {
            const float2 q = split(v[j][i]);
            v[j][i] = pair(o.one(j, 2 * i) < a.C ? q.x : 0.f, o.one(j, 2 * i + 1) < a.C ? q.y : 0.f);
          }
        }
      }
    }
    if (a.kind != kNone) {
      f2 t = 0ull;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < kPairs; ++i) t = fma2(v[j][i], v[j][i], t);
      float q[1] = {split(t).x + split(t).y};
      group_sum<kWarp, 1>(q, red[flip]);
      flip ^= 1;
      rstd = inv_sqrt(fmaf(q[0], a.inv_c, a.eps));
    }
    if (a.rstd != nullptr && o.me == 0) {
      const int64_t r = static_cast<int64_t>(s.b) * a.N + row;
      if (a.mean != nullptr) a.mean[r] = mean;
      a.rstd[r] = rstd;
    }
    const f2 rs = pair(rstd, rstd), scale = pair(a.res_scale, a.res_scale);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!o.any(j)) continue;
#pragma unroll
      for (int i = 0; i < kPairs; ++i) v[j][i] = fma2(mul2(v[j][i], rs), A[j][i], S[j][i]);
      if (has_res) {
        f2 r[kPairs];
        read_vec<TO>(slot + NV * UI * threads, j, o, r);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) v[j][i] = fma2(r[i], scale, v[j][i]);
      }
      store_vec<TO>(y, j, o, v[j]);
    }
    y += ystep;
    finish(free_slot);
    free_slot = slot;
    slot = slot + stage_units == ring_end ? ring : slot + stage_units;
  }
  cp_async_wait<0>();
}

// ------------------------------------------------------------------------------------
// Backward. TI: type of x, dx and of the gradient around the block; TO: type of dy. A, P1 and P2
// take 24 registers a vector; xh and g are therefore formed twice, before and after the row's
// sums, from the ring (whose slot is not refilled before the next row) instead of being held.
// kBound: most threads of the CTA; 320 (up to 5,120 channels) leaves room for two CTAs an SM.
// ------------------------------------------------------------------------------------
template <typename TI, typename TO, int NV, bool kWarp, int kBound, int kMode, int kFixed>
__global__ void __launch_bounds__(kWarp ? 32 * kWarpsPerCta : kFixed ? kFixed : kBound,
                                  kFixed == 128 ? 5 : kBound == kMaxThreads || (kWarp && NV == 4) ? 1 : 2)
norm_bwd_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(16) uint4 ring_base[];
  __shared__ __align__(16) float red[2][2][kMaxWarps];
  constexpr int UI = units_of<TI>(), UO = units_of<TO>();
  const int32_t threads = kWarp ? 32 : kFixed ? kFixed : static_cast<int32_t>(blockDim.x);
  const Own<kMode> o{kWarp ? static_cast<int32_t>(threadIdx.x & 31) : static_cast<int32_t>(threadIdx.x), threads, a.C};
  const bool has_res = a.res != nullptr;
  const int stage_units = NV * (UI + UO + (has_res ? UI : 0)) * threads;
  uint4* ring = ring_base + (kWarp ? (threadIdx.x >> 5) * a.stages * stage_units : 0) + o.me;
  const Slice s = slice_of(a);
  const int32_t step = kWarp ? kWarpsPerCta : 1;
  const int32_t first = s.lo + (kWarp ? static_cast<int32_t>(threadIdx.x >> 5) : 0);
  const TI* x = static_cast<const TI*>(a.x) + s.b * a.xb;
  const TO* dy = static_cast<const TO*>(a.dy) + s.b * a.db;
  const TI* res = has_res ? static_cast<const TI*>(a.res) + s.b * a.rb : nullptr;
  TI* dx = static_cast<TI*>(a.y) + s.b * a.yb;
  if (!kWarp && threadIdx.x < 4 * kMaxWarps) (&red[0][0][0])[threadIdx.x] = 0.f;
  if (a.done != nullptr && blockIdx.x == 0)
    for (int32_t i = threadIdx.x; i < (a.C + 31) / 32; i += blockDim.x) a.done[i] = 0;

  // rows are fetched one after the other: the next one's addresses
  x += first * a.xn;
  dy += first * a.dn;
  if (has_res) res += first * a.rn;
  dx += first * a.yn;
  const int64_t xstep = step * a.xn, dstep = step * a.dn, rstep = step * a.rn, ystep = step * a.yn;
  int32_t next = first;
  Fetch<TI, NV, Own<kMode>> fx, fr;
  Fetch<TO, NV, Own<kMode>> fd;
  auto start = [&](uint4* slot) {
    if (next < s.hi) {
      fx.start(slot, x, o);
      fd.start(slot + NV * UI * threads, dy, o);
      if (has_res) fr.start(slot + NV * (UI + UO) * threads, res, o);
    }
    cp_async_commit();
    x += xstep;
    dy += dstep;
    res += rstep;
    next += step;
  };
  auto finish = [&](uint4* slot) {           // of a row past the slice: stale values that no one reads
    fx.finish(slot, o);
    fd.finish(slot + NV * UI * threads, o);
    if (has_res) fr.finish(slot + NV * (UI + UO) * threads, o);
  };
  const int32_t stages = a.stages;
  uint4* const ring_end = ring + stages * stage_units;
  uint4* free_slot = ring;
  for (int i = 0; i < stages - 1; ++i, free_slot += stage_units) {
    start(free_slot);
    finish(free_slot);
  }

  f2 A[NV][kPairs], P1[NV][kPairs], P2[NV][kPairs];
  {
    float g[NV][kVec], w[NV][kVec];
    if (a.g.p) load_params<NV>(a.g, s.b, o, g);
    if (a.w.p) load_params<NV>(a.w, 0, o, w);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        g[j][i] = a.g.p ? a.gain_off + g[j][i] : 1.f;
        if (a.w.p) g[j][i] *= w[j][i];
      }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        A[j][i] = pair(g[j][2 * i], g[j][2 * i + 1]);
        P1[j][i] = P2[j][i] = 0ull;
      }
  }
  if (!kWarp) __syncthreads();                     // red is zero

  uint4* slot = ring;
  int32_t flip = 0;
  const float* means = a.mean + static_cast<int64_t>(s.b) * a.N;
  const float* rstds = a.rstd + static_cast<int64_t>(s.b) * a.N;
  for (int32_t row = first; row < s.hi; row += step) {
    const float mean = a.kind == kLayer ? __ldg(means + row) : 0.f;
    const float rstd = a.kind != kNone ? __ldg(rstds + row) : 1.f;
    wait_oldest(stages);
    const f2 sub = pair(-mean, -mean), rs = pair(rstd, rstd);
    // xh of vector j: 0 where the thread owns nothing is not needed, dy is 0 there
    auto normed = [&](int j, f2* xh) {
      read_vec<TI>(slot, j, o, xh);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) xh[i] = mul2(add2(xh[i], sub), rs);
    };
    f2 t1 = 0ull, t2 = 0ull;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      f2 xh[kPairs], g[kPairs];
      normed(j, xh);
      read_vec<TO>(slot + NV * UI * threads, j, o, g);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        P1[j][i] = fma2(g[i], xh[i], P1[j][i]);
        P2[j][i] = add2(P2[j][i], g[i]);
        const f2 q = mul2(g[i], A[j][i]);
        t1 = add2(t1, q);
        t2 = fma2(q, xh[i], t2);
      }
    }
    start(free_slot);                              // the slot read in the previous round
    float c1 = 0.f, c2 = 0.f;
    if (a.kind != kNone) {
      float sum[2] = {split(t1).x + split(t1).y, split(t2).x + split(t2).y};
      group_sum<kWarp, 2>(sum, red[flip]);
      flip ^= 1;
      c1 = a.kind == kLayer ? -sum[0] * a.inv_c : 0.f;
      c2 = -sum[1] * a.inv_c;
    }
    const f2 k1 = pair(c1, c1), k2 = pair(c2, c2), scale = pair(a.res_scale, a.res_scale);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!o.any(j)) continue;
      f2 xh[kPairs], g[kPairs];
      normed(j, xh);
      read_vec<TO>(slot + NV * UI * threads, j, o, g);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) g[i] = mul2(add2(fma2(xh[i], k2, mul2(g[i], A[j][i])), k1), rs);
      if (has_res) {
        f2 q[kPairs];
        read_vec<TI>(slot + NV * (UI + UO) * threads, j, o, q);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) g[i] = fma2(q[i], scale, g[i]);
      }
      store_vec<TI>(dx, j, o, g);
    }
    dx += ystep;
    finish(free_slot);
    free_slot = slot;
    slot = slot + stage_units == ring_end ? ring : slot + stage_units;
  }
  cp_async_wait<0>();

  // this CTA's partial sums (warp groups: added up in shared memory, in warp order)
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.C;
  if (!kWarp) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const int32_t c = o.one(j, i);
        if (c >= a.C) continue;
        const float2 q1 = split(P1[j][i / 2]), q2 = split(P2[j][i / 2]);
        part[c] = i % 2 ? q1.y : q1.x;
        part[a.C + c] = i % 2 ? q2.y : q2.x;
      }
    return;
  }
  float* acc = reinterpret_cast<float*>(ring_base);      // [2][NV * 256]: the ring is drained
  constexpr int32_t W = NV * 32 * kVec;
  for (int32_t w = 0; w < kWarpsPerCta; ++w) {
    __syncthreads();
    if (static_cast<int32_t>(threadIdx.x >> 5) != w) continue;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const int32_t c = o.one(j, i);                   // < W for both mappings
        const float2 q1 = split(P1[j][i / 2]), q2 = split(P2[j][i / 2]);
        const float p1 = i % 2 ? q1.y : q1.x, p2 = i % 2 ? q2.y : q2.x;
        acc[c] = w ? acc[c] + p1 : p1;
        acc[W + c] = w ? acc[W + c] + p2 : p2;
      }
  }
  __syncthreads();
  for (int32_t c = threadIdx.x; c < a.C; c += 32 * kWarpsPerCta) {
    part[c] = acc[c];
    part[a.C + c] = acc[W + c];
  }
}

// ------------------------------------------------------------------------------------
// Parameter gradients from the slices' sums. One CTA per 32 channels and sequence: 16 rows of
// threads add up the slices (a fixed assignment and order), then
//   dG = w P1 + b P2, dshift = P2, and the sequence's G P1, G P2 for dw, db.
// The CTA of these channels that comes last adds those up over the sequences, in their order: which CTA
// it is changes nothing.
// ------------------------------------------------------------------------------------
struct GradArgs {
  const float* part;       // [B * slices][2][C]
  Param w, b, g;
  float gain_off;
  float* dgain;            // null or [B][C]
  float* dshift;           // null or [B][C]
  float* gp;               // [B][2][C]: G P1, G P2 (several sequences, dw or db asked for), or null
  int32_t* done;           // [C / 32]: sequences whose G P1, G P2 are written (the backward kernel clears it)
  float* dw;               // null or [C]
  float* db;
  int32_t B, C, slices;
};
constexpr int kGradRows = 16;

__global__ void __launch_bounds__(32 * kGradRows) norm_grad_kernel(const __grid_constant__ GradArgs a) {
  __shared__ float s1[kGradRows][32], s2[kGradRows][32];
  __shared__ int last;
  const int32_t col = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int32_t c = blockIdx.x * 32 + col, b = blockIdx.y;
  const bool have = c < a.C;
  float p1 = 0.f, p2 = 0.f;
  if (have) {
    const float* part = a.part + static_cast<int64_t>(b) * a.slices * 2 * a.C + c;
#pragma unroll 8
    for (int32_t i = r; i < a.slices; i += kGradRows) {
      p1 += part[static_cast<int64_t>(i) * 2 * a.C];
      p2 += part[static_cast<int64_t>(i) * 2 * a.C + a.C];
    }
  }
  // the rows' sums, in row 0
  const auto rows_sum = [&]() {
    s1[r][col] = p1;
    s2[r][col] = p2;
    __syncthreads();
    if (r != 0) return;
#pragma unroll
    for (int i = 1; i < kGradRows; ++i) {
      p1 += s1[i][col];
      p2 += s2[i][col];
    }
  };
  rows_sum();
  if (r == 0 && have) {
    const int64_t o = static_cast<int64_t>(b) * a.C + c;
    if (a.dgain) {
      const float w = a.w.p ? load_param(a.w, 0, c) : 1.f;
      a.dgain[o] = a.b.p ? fmaf(w, p1, load_param(a.b, 0, c) * p2) : w * p1;
    }
    if (a.dshift) a.dshift[o] = p2;
    const float G = a.g.p ? a.gain_off + load_param(a.g, b, c) : 1.f;
    p1 *= G;
    p2 *= G;
    if (a.gp) {
      a.gp[static_cast<int64_t>(b) * 2 * a.C + c] = p1;
      a.gp[static_cast<int64_t>(b) * 2 * a.C + a.C + c] = p2;
      __threadfence();
    }
  }
  if (a.gp) {
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(a.done + blockIdx.x, 1) == a.B - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    p1 = p2 = 0.f;
    if (have)
      for (int32_t i = r; i < a.B; i += kGradRows) {
        p1 += __ldcg(a.gp + static_cast<int64_t>(i) * 2 * a.C + c);
        p2 += __ldcg(a.gp + static_cast<int64_t>(i) * 2 * a.C + a.C + c);
      }
    rows_sum();
  }
  if (r == 0 && have) {
    if (a.dw) a.dw[c] = p1;
    if (a.db) a.db[c] = p2;
  }
}

}  // namespace norm
}  // namespace veda
