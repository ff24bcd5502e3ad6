// k_rotary.cuh -- rotary positions of Q and K: the cos / sin table, the rotation of raster
// tensors (any strides, any of three types), and the rotation fused into the tile gather of
// steps 1 + 2 and into the scatter of step 6 (its transpose, for the gradients).
//
// Pair p of token n turns by theta = pos[axis(p)][n] * inv_freq[p]:
//   y1 = x1 cos - x2 sin,   y2 = x2 cos + x1 sin,
// with (x1, x2) = (x[2p], x[2p+1]) (interleaved) or (x[p], x[p + P]) (half layout, P pairs);
// channels from 2P on pass through. The rotation is orthogonal up to the table's amplitude,
// so its transpose -- the backward -- is the same kernel with -sin. All products are fp32 and
// each result is rounded once.
//
// Everything here streams HBM: a pair costs four multiply-adds for the 4 to 8 bytes it reads
// and writes. What matters is that every access is a 16-byte vector, that enough of them are in
// flight, and that the table (rot_dim * 4 bytes a token, read by every head) is taken from the
// caches: the plain kernel loads a token's cos / sin into registers once and loops over heads;
// in the tile kernels the CTAs that run together hold the same tile of different heads, so the
// table's rows come from L2.
#pragma once

#include <cuda_fp16.h>

#include "k_gather.cuh"
#include "veda_ptx.cuh"

namespace veda {
namespace rotary {

constexpr int kMaxPairs = 256;      // head_dim up to 512
constexpr int kMaxAxes = 8;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// ------------------------------------------------------------------------------------
// Table: cos_sin[row][p] = amplitude * (cos, sin)(pos[axis(p)][row] * inv_freq[p]). The angle
// and its sine and cosine are fp64: at a position of 10^6 an fp32 angle is off by 0.03 rad.
// The frequencies travel as a kernel argument, so a call copies nothing to the device.
// ------------------------------------------------------------------------------------
struct TableArgs {
  const int32_t* pos;      // [axes][rows]
  float2* out;             // [rows][pairs]
  int64_t rows;
  int32_t pairs;
  double amplitude;
  double inv_freq[kMaxPairs];
  uint8_t axis[kMaxPairs];
};

__global__ void __launch_bounds__(kThreads) table_kernel(const __grid_constant__ TableArgs a) {
  const int64_t total = a.rows * a.pairs;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t row = i / a.pairs;
    const int32_t p = static_cast<int32_t>(i - row * a.pairs);
    const double angle = static_cast<double>(__ldg(a.pos + a.axis[p] * a.rows + row)) * a.inv_freq[p];
    double s, c;
    sincos(angle, &s, &c);
    a.out[i] = make_float2(static_cast<float>(a.amplitude * c), static_cast<float>(a.amplitude * s));
  }
}

// ------------------------------------------------------------------------------------
// 16-byte vectors of T as fp32 values and back.
// ------------------------------------------------------------------------------------
template <typename T> struct Vec;
template <> struct Vec<__nv_bfloat16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void get(const uint4& v, float* f) {
    const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = __bfloat1622float2(p[i]);
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
  static __device__ __forceinline__ uint4 put(const float* f) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
  static __device__ __forceinline__ float one(const __nv_bfloat16& x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 to(float x) { return __float2bfloat16_rn(x); }
};
template <> struct Vec<__half> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void get(const uint4& v, float* f) {
    const __half2* p = reinterpret_cast<const __half2*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = __half22float2(p[i]);
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
  static __device__ __forceinline__ uint4 put(const float* f) {
    uint4 v;
    __half2* p = reinterpret_cast<__half2*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    return v;
  }
  static __device__ __forceinline__ float one(const __half& x) { return __half2float(x); }
  static __device__ __forceinline__ __half to(float x) { return __float2half_rn(x); }
};
template <> struct Vec<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ void get(const uint4& v, float* f) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 put(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
  static __device__ __forceinline__ float one(const float& x) { return x; }
  static __device__ __forceinline__ float to(float x) { return x; }
};

// ------------------------------------------------------------------------------------
// Raster rotation. x, y: element strides (batch, token, head), channels contiguous; y may be x.
// A head's row is cut into items: one item = VE pairs (kVec: one 16-byte vector of an
// interleaved row, two vectors of a half-layout row; otherwise one pair), then the
// pass-through channels in items of the same width. Lane c of a unit's warp takes item c (and
// c + 32, ...) of every head, so its cos / sin stay in registers while it walks the heads;
// rows of fewer than 32 items put 32 / width heads side by side in the warp.
// ------------------------------------------------------------------------------------
struct Args {
  const void* x;
  void* y;
  int64_t xs[3], ys[3];
  const float2* cs;        // [table_rows][P]
  const int32_t* rows;     // null, or [B * N] table row of every token
  int64_t table_rows;
  int64_t batch_rows;      // rows between two sequences' tables (0: shared), when rows is null
  int64_t units;           // B * N * groups
  int32_t N, H, D, P;
  int32_t groups, hg;      // head groups per token, heads per group
  int32_t width_log2;      // lanes per head row
  int32_t items, rot_items;
  float sign;
};

template <typename T, bool kHalf, bool kVec>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ Args a) {
  using V = Vec<T>;
  constexpr int VE = kVec ? (kHalf ? V::E : V::E / 2) : 1;   // pairs per item
  constexpr int U = 4;                                       // heads in flight per lane
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (unit >= a.units) return;
  const int32_t lane = threadIdx.x & 31;
  const int64_t bn = unit / a.groups;
  const int32_t grp = static_cast<int32_t>(unit - bn * a.groups);
  const int64_t b = bn / a.N, n = bn - b * a.N;
  int64_t row = a.rows ? static_cast<int64_t>(__ldg(a.rows + bn)) : b * a.batch_rows + n;
  const bool bad = row < 0 || row >= a.table_rows;           // only a caller's row can be
  if (bad) {
    flag_status(ST_BAD_MAP);
    row = 0;
  }
  const T* x = static_cast<const T*>(a.x) + b * a.xs[0] + n * a.xs[1];
  T* y = static_cast<T*>(a.y) + b * a.ys[0] + n * a.ys[1];
  const float2* cs = a.cs + row * a.P;
  const int32_t h0 = grp * a.hg, h1 = min(a.H, h0 + a.hg);
  const int32_t width = 1 << a.width_log2, hstep = 32 >> a.width_log2;
  for (int32_t c = lane & (width - 1); c < a.items; c += width) {
    const bool turn = c < a.rot_items;
    float co[VE], si[VE];
    int32_t o1, o2;            // first channels of the item's two parts (kVec interleaved: one)
    bool second = true;
    if (turn) {
      const int32_t p = c * VE;
      o1 = kHalf ? p : 2 * p;
      o2 = kHalf ? p + a.P : 2 * p + 1;
      if constexpr (VE % 2 == 0) {
        const float4* t = reinterpret_cast<const float4*>(cs + p);
#pragma unroll
        for (int i = 0; i < VE / 2; ++i) {
          const float4 v = __ldg(t + i);
          co[2 * i] = v.x; si[2 * i] = v.y * a.sign;
          co[2 * i + 1] = v.z; si[2 * i + 1] = v.w * a.sign;
        }
      } else {
        const float2 v = __ldg(cs + p);
        co[0] = v.x; si[0] = v.y * a.sign;
      }
    } else {
      constexpr int W = kVec ? (kHalf ? 2 * V::E : V::E) : 2;   // channels per item
      o1 = 2 * a.P + (c - a.rot_items) * W;
      o2 = o1 + (kVec ? V::E : 1);
      second = o2 < a.D;
#pragma unroll
      for (int i = 0; i < VE; ++i) { co[i] = 1.f; si[i] = 0.f; }
    }
    if (bad) {                  // a flagged token's channels are written as zeros
#pragma unroll
      for (int i = 0; i < VE; ++i) co[i] = si[i] = 0.f;
    }
    for (int32_t h = h0 + (lane >> a.width_log2); h < h1; h += U * hstep) {
      if constexpr (kVec) {
        uint4 v1[U], v2[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int32_t hh = h + u * hstep;
          if (hh >= h1) continue;
          const T* r = x + hh * a.xs[2];
          v1[u] = *reinterpret_cast<const uint4*>(r + o1);
          if (kHalf && second) v2[u] = *reinterpret_cast<const uint4*>(r + o2);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int32_t hh = h + u * hstep;
          if (hh >= h1) continue;
          T* r = y + hh * a.ys[2];
          if (!turn) {          // pass-through: the bits as they are (zeros where flagged)
            if (bad) v1[u] = v2[u] = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(r + o1) = v1[u];
            if (kHalf && second) *reinterpret_cast<uint4*>(r + o2) = v2[u];
            continue;
          }
          float f[V::E];
          V::get(v1[u], f);
          if constexpr (kHalf) {
            float g[V::E];
            V::get(v2[u], g);
            float p[V::E], q[V::E];
#pragma unroll
            for (int i = 0; i < V::E; ++i) {
              p[i] = bad ? 0.f : fmaf(f[i], co[i], -(g[i] * si[i]));
              q[i] = bad ? 0.f : fmaf(g[i], co[i], f[i] * si[i]);
            }
            *reinterpret_cast<uint4*>(r + o1) = V::put(p);
            *reinterpret_cast<uint4*>(r + o2) = V::put(q);
          } else {
            float p[V::E];
#pragma unroll
            for (int i = 0; i < V::E / 2; ++i) {
              p[2 * i] = bad ? 0.f : fmaf(f[2 * i], co[i], -(f[2 * i + 1] * si[i]));
              p[2 * i + 1] = bad ? 0.f : fmaf(f[2 * i + 1], co[i], f[2 * i] * si[i]);
            }
            *reinterpret_cast<uint4*>(r + o1) = V::put(p);
          }
        }
      } else {
        T t1[U], t2[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int32_t hh = h + u * hstep;
          if (hh >= h1) continue;
          t1[u] = x[hh * a.xs[2] + o1];
          if (second) t2[u] = x[hh * a.xs[2] + o2];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int32_t hh = h + u * hstep;
          if (hh >= h1) continue;
          T* r = y + hh * a.ys[2];
          if (!turn) {
            r[o1] = bad ? V::to(0.f) : t1[u];
            if (second) r[o2] = bad ? V::to(0.f) : t2[u];
            continue;
          }
          const float f = V::one(t1[u]), g = V::one(t2[u]);
          r[o1] = V::to(bad ? 0.f : fmaf(f, co[0], -(g * si[0])));
          r[o2] = V::to(bad ? 0.f : fmaf(g, co[0], f * si[0]));
        }
      }
    }
  }
}

// ------------------------------------------------------------------------------------
// Rotation of one 16-byte chunk (channels 8c .. 8c+7) of a bf16 row whose 16 chunks lie in the
// 16 lanes of a half warp. Interleaved pairs are inside the chunk; in the half layout the
// partner chunk is P / 8 lanes away and comes by shuffle (all 32 lanes take part). `cs` is the
// token's table row; `live` is false for a slot without a token, whose chunk is zero.
// ------------------------------------------------------------------------------------
template <bool kHalf>
struct Turn {
  static constexpr int kPairs = kHalf ? 8 : 4;   // pairs whose cos / sin the chunk needs
  int32_t p0;        // first pair of this chunk
  int32_t partner;   // lane holding the partner chunk (half layout)
  float s_sign;      // sign of the partner's term
  bool turned;       // chunk inside the rotated part

  __device__ __forceinline__ Turn(int32_t c, uint32_t lane, int32_t P, float sign) {
    if (kHalf) {
      const int32_t hc = P / 8;
      turned = c < 2 * hc;
      const bool first = c < hc;
      p0 = (first ? c : c - hc) * 8;
      partner = static_cast<int32_t>(lane) + (first ? hc : -hc);
      if (!turned) { p0 = 0; partner = static_cast<int32_t>(lane); }
      s_sign = first ? -sign : sign;
    } else {
      turned = c < P / 4;
      p0 = turned ? 4 * c : 0;
      partner = static_cast<int32_t>(lane);
      s_sign = sign;
    }
  }

  struct CosSin { float4 v[kPairs / 2]; };
  __device__ __forceinline__ void load(CosSin& t, const float2* row, bool live) const {
    const float4* p = reinterpret_cast<const float4*>(row + p0);
#pragma unroll
    for (int i = 0; i < kPairs / 2; ++i)
      t.v[i] = live && turned ? __ldg(p + i) : make_float4(1.f, 0.f, 1.f, 0.f);
  }

  __device__ __forceinline__ void apply(const uint4& raw, const CosSin& t, float* f) const {
    Vec<__nv_bfloat16>::get(raw, f);
    if (kHalf) {
      uint4 o;
      o.x = __shfl_sync(0xffffffffu, raw.x, partner);
      o.y = __shfl_sync(0xffffffffu, raw.y, partner);
      o.z = __shfl_sync(0xffffffffu, raw.z, partner);
      o.w = __shfl_sync(0xffffffffu, raw.w, partner);
      float g[8];
      Vec<__nv_bfloat16>::get(o, g);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 cs = t.v[kHalf ? i : 0];
        f[2 * i] = fmaf(f[2 * i], cs.x, g[2 * i] * (cs.y * s_sign));
        f[2 * i + 1] = fmaf(f[2 * i + 1], cs.z, g[2 * i + 1] * (cs.w * s_sign));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 cs = t.v[i];
        const float a0 = f[4 * i], a1 = f[4 * i + 1], b0 = f[4 * i + 2], b1 = f[4 * i + 3];
        f[4 * i] = fmaf(a0, cs.x, -(a1 * (cs.y * s_sign)));
        f[4 * i + 1] = fmaf(a1, cs.x, a0 * (cs.y * s_sign));
        f[4 * i + 2] = fmaf(b0, cs.z, -(b1 * (cs.w * s_sign)));
        f[4 * i + 3] = fmaf(b1, cs.z, b0 * (cs.w * s_sign));
      }
    }
  }
};

struct TileArgs {
  GatherArgs g;
  const int32_t* valid;    // [H][nT] (gather only)
  float* pooled;           // [B][H][nT][3][128] (gather only)
  const float2* cs;        // [table_rows][P]
  int64_t batch_rows;      // 0 (table shared by the batch) or N
  int32_t P;
  float sign;
};

// Steps 1 + 2 with the rotation on the way: permute_pool_kernel's work split (one warp per
// tile, 16 rows a pass, partials in registers). The pooled mean / max / min are taken from the
// fp32 values before they are rounded for the tile.
template <bool kHalf>
__global__ void __launch_bounds__(kPoolThreads) rotary_permute_pool_kernel(const __grid_constant__ TileArgs p) {
  const GatherArgs& a = p.g;
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t c = lane & 15, half = lane >> 4;
  const Turn<kHalf> turn(static_cast<int32_t>(c), lane, p.P, p.sign);
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kPoolThreads / 32);
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kPoolThreads / 32) + (threadIdx.x >> 5); u < a.units;
       u += warps) {
    int32_t b, h, t;
    unit_coords(u, a.H, a.nT, b, h, t);
    const int64_t lin = (static_cast<int64_t>(b) * a.H + h) * a.nT + t;
    int32_t nv = p.valid[static_cast<int64_t>(h) * a.nT + t];
    nv = nv < 0 ? 0 : (nv > 128 ? 128 : nv);
    const int32_t* m = a.map + static_cast<int64_t>(h) * a.Npad + static_cast<int64_t>(t) * 128 + half;
    const uint8_t* src = a.src + (static_cast<int64_t>(b) * a.N * a.H + h) * kRowBytes + c * 16;
    const int64_t tok_stride = static_cast<int64_t>(a.H) * kRowBytes;
    const float2* cs = p.cs + b * p.batch_rows * p.P;
    uint8_t* dst = a.dst + lin * kTileBytes + half * kRowBytes + c * 16;
    float sum[8], mx[8], mn[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) { sum[k] = 0.f; mx[k] = -INFINITY; mn[k] = INFINITY; }
#pragma unroll 1
    for (int32_t r0 = 0; r0 < 128; r0 += 16) {
      int32_t tok[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) tok[i] = __ldg(m + r0 + 2 * i);
      uint4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = make_uint4(0, 0, 0, 0);
        if (tok[i] >= a.N) flag_status(ST_BAD_MAP);
        if (tok[i] >= a.N) tok[i] = -1;
        if (tok[i] >= 0) v[i] = ld_stream(src + tok[i] * tok_stride);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        typename Turn<kHalf>::CosSin t4;
        turn.load(t4, cs + static_cast<int64_t>(tok[i] < 0 ? 0 : tok[i]) * p.P, tok[i] >= 0);
        float f[8];
        turn.apply(v[i], t4, f);
        st_v4(dst + (r0 + 2 * i) * kRowBytes, turn.turned ? Vec<__nv_bfloat16>::put(f) : v[i]);
        if (r0 + static_cast<int32_t>(half) + 2 * i < nv) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            sum[k] += f[k];
            mx[k] = fmaxf(mx[k], f[k]);
            mn[k] = fminf(mn[k], f[k]);
          }
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 16);
      mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 16));
      mn[k] = fminf(mn[k], __shfl_xor_sync(0xffffffffu, mn[k], 16));
    }
    if (half == 0) {
      float4* o = reinterpret_cast<float4*>(p.pooled + lin * 384 + c * 8);
      const float inv = nv > 0 ? 1.0f / static_cast<float>(nv) : 0.f;
      if (nv == 0) {
#pragma unroll
        for (int k = 0; k < 8; ++k) mx[k] = mn[k] = 0.f;
      }
      o[0] = make_float4(sum[0] * inv, sum[1] * inv, sum[2] * inv, sum[3] * inv);
      o[1] = make_float4(sum[4] * inv, sum[5] * inv, sum[6] * inv, sum[7] * inv);
      o[32] = make_float4(mx[0], mx[1], mx[2], mx[3]);
      o[33] = make_float4(mx[4], mx[5], mx[6], mx[7]);
      o[64] = make_float4(mn[0], mn[1], mn[2], mn[3]);
      o[65] = make_float4(mn[4], mn[5], mn[6], mn[7]);
    }
  }
}

// Step 6 with a rotation on the way (sign -1: the transpose, which takes dQ and dK in tile
// order to raster order and through the rotary positions in one pass).
template <bool kHalf>
__global__ void __launch_bounds__(kCopyThreads) rotary_unpermute_kernel(const __grid_constant__ TileArgs p) {
  const GatherArgs& a = p.g;
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t c = threadIdx.x & 15, r0 = threadIdx.x >> 4;
  const Turn<kHalf> turn(static_cast<int32_t>(c), lane, p.P, p.sign);
  for (int64_t u = blockIdx.x; u < a.units; u += gridDim.x) {
    int32_t b, h, t;
    unit_coords(u, a.H, a.nT, b, h, t);
    const int32_t* m = a.map + static_cast<int64_t>(h) * a.Npad + static_cast<int64_t>(t) * 128;
    const uint8_t* src = a.src + ((static_cast<int64_t>(b) * a.H + h) * a.Npad + static_cast<int64_t>(t) * 128) * kRowBytes;
    const float2* cs = p.cs + b * p.batch_rows * p.P;
    int32_t tok[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) tok[i] = __ldg(m + r0 + 16 * i);
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = make_uint4(0, 0, 0, 0);
      if (tok[i] >= a.N) flag_status(ST_BAD_MAP);
      if (tok[i] >= a.N) tok[i] = -1;
      if (tok[i] >= 0) v[i] = ld_stream(src + (r0 + 16 * i) * kRowBytes + c * 16);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      typename Turn<kHalf>::CosSin t4;
      turn.load(t4, cs + static_cast<int64_t>(tok[i] < 0 ? 0 : tok[i]) * p.P, tok[i] >= 0);
      float f[8];
      turn.apply(v[i], t4, f);
      if (tok[i] >= 0)
        st_v4(a.dst + ((static_cast<int64_t>(b) * a.N + tok[i]) * a.H + h) * kRowBytes + c * 16,
              turn.turned ? Vec<__nv_bfloat16>::put(f) : v[i]);
    }
  }
}

}  // namespace rotary
}  // namespace veda
