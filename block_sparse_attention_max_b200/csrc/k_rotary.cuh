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
// flight, and that the table (rot_dim * 4 bytes a token, read by every head) is fetched once for
// several heads: the raster kernel loads a token's cos / sin into registers and loops over heads;
// the tile kernels copy the rows of a tile's tokens into shared memory for eight heads.
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
// A head's row is cut into items of vectors of W channels. kTwo: an item is two vectors whose channels
// pair up one by one -- W channels of either half (half layout), or a channel and its neighbour
// (interleaved rows without any vector); the channels behind the turned ones follow in items of two
// vectors. Otherwise (interleaved) an item is one vector, W / 2 pairs, of which the last turned item may
// hold some that are not. W is the widest that lengths, strides and addresses allow.
//
// A warp takes a token (a group of its heads). With many heads lane c takes item c (and c + 32, ...)
// of every head, so its cos / sin stay in registers while it walks the heads, U at a time; rows of
// fewer than 32 items put several heads side by side in the warp. kFlat: with few heads there is
// nothing to keep, and a lane takes U items at a time of all of the token's.
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
  int32_t width_log2;      // lanes per head row (not flat)
  int32_t items, rot_items;
  int32_t apart;           // kTwo: channels between the two vectors of a turned item (P, or 1: interleaved)
  float sign;
};

template <int BYTES> struct Word;
template <> struct Word<16> { typedef uint4 type; };
template <> struct Word<8> { typedef uint2 type; };
template <> struct Word<4> { typedef uint32_t type; };
template <> struct Word<2> { typedef uint16_t type; };

template <typename T, bool kTwo, int W, bool kFlat>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ Args a) {
  using V = Vec<T>;
  using R = typename Word<W * static_cast<int>(sizeof(T))>::type;
  constexpr int NP = kTwo ? W : W / 2;                       // pairs per item
  constexpr int U = kFlat && W * sizeof(T) == 16 ? 2 : 4;    // items in flight per lane
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

  struct Item {
    int32_t o1, o2;          // first channels of its vectors
    int32_t live;            // turned pairs (the first ones)
    bool second;             // the second vector exists (kTwo)
  };
  const auto item_of = [&](int32_t c) {
    Item t;
    if (kTwo) {
      const bool turn = c < a.rot_items;
      t.o1 = turn ? (a.apart == 1 ? 2 * c : c * W) : 2 * a.P + (c - a.rot_items) * 2 * W;
      t.o2 = t.o1 + (turn ? a.apart : W);
      t.live = turn ? NP : 0;
      t.second = t.o2 < a.D;
    } else {
      t.o1 = t.o2 = c * W;
      t.live = min(NP, max(0, a.P - c * NP));
      t.second = false;
    }
    return t;
  };
  struct Turns { float c[NP], s[NP]; };
  const auto load_turns = [&](int32_t c, int32_t live, Turns& t) {
    const float2* p = cs + c * NP;
    if (NP % 2 == 0 && live == NP && a.P % 2 == 0) {          // 16-byte aligned
#pragma unroll
      for (int i = 0; i + 1 < NP; i += 2) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
        t.c[i] = v.x; t.s[i] = v.y * a.sign;
        t.c[i + 1] = v.z; t.s[i + 1] = v.w * a.sign;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const float2 v = i < live ? __ldg(p + i) : make_float2(1.f, 0.f);
        t.c[i] = v.x; t.s[i] = v.y * a.sign;
      }
    }
  };
  const auto load = [&](const Item& t, int32_t h, R& v1, R& v2) {
    const T* r = x + h * a.xs[2];
    v1 = *reinterpret_cast<const R*>(r + t.o1);
    if (kTwo && t.second) v2 = *reinterpret_cast<const R*>(r + t.o2);
  };
  // turns the pairs that are to be turned (the others' bits stay as they are) and stores
  const auto finish = [&](const Item& t, const Turns& w, int32_t h, R v1, R v2) {
    T* r = y + h * a.ys[2];
    if (bad) v1 = v2 = R{};                                   // a flagged token is written as zeros
    T* e1 = reinterpret_cast<T*>(&v1);
    T* e2 = reinterpret_cast<T*>(&v2);
    if (t.live > 0 && !bad) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        T& first = kTwo ? e1[i] : e1[2 * i];
        T& second = kTwo ? e2[i] : e1[2 * i + 1];
        const float f = V::one(first), g = V::one(second);
        const T nf = V::to(fmaf(f, w.c[i], -(g * w.s[i]))), ng = V::to(fmaf(g, w.c[i], f * w.s[i]));
        if (kTwo || i < t.live) {
          first = nf;
          second = ng;
        }
      }
    }
    *reinterpret_cast<R*>(r + t.o1) = v1;
    if (kTwo && t.second) *reinterpret_cast<R*>(r + t.o2) = v2;
  };

  if (kFlat) {
    const int32_t total = (h1 - h0) * a.items;
    for (int32_t q = lane; q < total; q += 32 * U) {
      Item t[U];
      Turns w[U];
      R v1[U], v2[U];
      int32_t h[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int32_t i = q + 32 * u;
        if (i >= total) continue;
        h[u] = i / a.items;
        const int32_t c = i - h[u] * a.items;
        h[u] += h0;
        t[u] = item_of(c);
        load(t[u], h[u], v1[u], v2[u]);
        if (t[u].live > 0) load_turns(c, t[u].live, w[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (q + 32 * u < total) finish(t[u], w[u], h[u], v1[u], v2[u]);
    }
  } else {
    const int32_t width = 1 << a.width_log2, hstep = 32 >> a.width_log2;
    for (int32_t c = lane & (width - 1); c < a.items; c += width) {
      const Item t = item_of(c);
      Turns w;
      if (t.live > 0) load_turns(c, t.live, w);
      for (int32_t h = h0 + (lane >> a.width_log2); h < h1; h += U * hstep) {
        R v1[U], v2[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (h + u * hstep < h1) load(t, h + u * hstep, v1[u], v2[u]);
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (h + u * hstep < h1) finish(t, w, h + u * hstep, v1[u], v2[u]);
      }
    }
  }
}

// ------------------------------------------------------------------------------------
// The tile kernels. A CTA takes one tile of up to 8 neighbouring heads, a warp a head; the tile's
// 128 rows go by in batches of 8, and the batches of a CTA's tiles form one stream: while one is
// turned and written, the next two batches' rows (each warp's own) and their rows of the table (one
// copy for the CTA) are on their way into the other buffers by asynchronous copies, and the token
// indices of the batch after those are on their way into a register.
//
// The table is what decides the speed: a token's row of it has rot_dim * 4 bytes, twice the 256
// bytes of the row it turns. Read by every head from L2, 8 to 16 rows in registers at a time, the
// gather of the 16:9 clip took 378 us a tensor; this one takes 224 (185 at the HBM copy rate; 240 with
// one batch on its way instead of two). Neighbouring heads mostly have the same tile map,
// so the CTA copies the rows of its first head's tokens once; a warp whose head has another token
// in some slot (per-head tile orders) reads its rows of the table from global memory instead.
//
// A half warp turns one token row; a lane holds two pieces of four channels, chosen so that both
// halves of a pair are its own and that a warp's accesses of row and table are contiguous:
// interleaved pairs, channels 4c and 64 + 4c; half layout, channels 4c and P + 4c (the rest of the
// lanes carry the channels behind the turned ones).
// ------------------------------------------------------------------------------------
struct TileArgs {
  GatherArgs g;            // units: B * nT * groups
  const int32_t* valid;    // [H][nT] (gather only)
  float* pooled;           // [B][H][nT][3][128] (gather only)
  const float2* cs;        // [table_rows][P]
  int64_t batch_rows;      // 0 (table shared by the batch) or N
  int32_t P;
  int32_t groups, hg;      // head groups, heads per group (warps per CTA)
  float sign;
};

constexpr int kTileHeads = 8;
constexpr int kBatchRows = 8;
constexpr int kTileBuffers = 3;
// one buffer: hg warps' rows, then the table's rows
__host__ __device__ constexpr uint32_t tile_buffer_bytes(int32_t hg, int32_t P) {
  return static_cast<uint32_t>(hg) * kBatchRows * kRowBytes + kBatchRows * static_cast<uint32_t>(P) * 8u;
}

__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint2 ld_shared8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_shared_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void st_v2(void* p, uint2 v) {
  asm volatile("st.global.v2.u32 [%0], {%1, %2};" ::"l"(p), "r"(v.x), "r"(v.y) : "memory");
}
__device__ __forceinline__ float fmin3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ void unpack4(uint2 v, float* f) {
  f[0] = __uint_as_float(v.x << 16);
  f[1] = __uint_as_float(v.x & 0xffff0000u);
  f[2] = __uint_as_float(v.y << 16);
  f[3] = __uint_as_float(v.y & 0xffff0000u);
}

// Place in a CTA's stream of batches.
struct TileBatch {
  int32_t u, r0, b, h0, t;
  __device__ __forceinline__ void at(int32_t unit, const TileArgs& p) {
    u = unit;
    r0 = 0;
    if (u >= p.g.units) return;
    const int32_t bt = u / p.groups;
    h0 = (u - bt * p.groups) * p.hg;
    b = bt / p.g.nT;
    t = bt - b * p.g.nT;
  }
  __device__ __forceinline__ void advance(const TileArgs& p) {
    r0 += kBatchRows;
    if (r0 == 128) at(u + static_cast<int32_t>(gridDim.x), p);
  }
  // lanes r and 8 + r: token of slot r0 + r of head h0 + warp; lanes 16 + r and 24 + r: of head h0.
  // -1 where there is none (past the stream, past the heads, pad slots).
  __device__ __forceinline__ int32_t token(const TileArgs& p, uint32_t warp, uint32_t lane) const {
    const int32_t h = h0 + (lane < 16 ? static_cast<int32_t>(warp) : 0);
    if (u >= p.g.units || h >= p.g.H) return -1;
    return __ldg(p.g.map + static_cast<int64_t>(h) * p.g.Npad + static_cast<int64_t>(t) * 128 + r0 + (lane & (kBatchRows - 1)));
  }
};

// kGather: steps 1 + 2 with the rotation on the way; the pooled mean / max / min are taken from the
// fp32 values before they are rounded for the tile. Otherwise step 6 with a rotation on the way
// (sign -1: the transpose, which takes dQ and dK in tile order to raster order and through the
// rotary positions in one pass).
// kFull: all 128 channels are turned (P = 64).
template <bool kHalf, bool kGather, bool kFull>
__global__ void __launch_bounds__(32 * kTileHeads, 3) rotary_tiles_kernel(const __grid_constant__ TileArgs p) {
  extern __shared__ __align__(16) uint8_t tile_smem[];
  const GatherArgs& a = p.g;
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t c = static_cast<int32_t>(lane & 15), half = static_cast<int32_t>(lane >> 4);
  // this lane's two pieces: first channels, first pairs, whether turned
  const int32_t P = kFull ? 64 : p.P;
  int32_t o1, o2, p1, p2;
  bool t1, t2;
  if (kHalf) {
    t1 = t2 = 4 * c < P;
    o1 = t1 ? 4 * c : 2 * P + 8 * (c - P / 4);
    o2 = t1 ? P + 4 * c : o1 + 4;
    p1 = t1 ? 4 * c : 0;
    p2 = p1 + 2;
  } else {
    o1 = 4 * c;
    o2 = 64 + 4 * c;
    t1 = o1 < 2 * P;
    t2 = o2 < 2 * P;
    p1 = t1 ? 2 * c : 0;
    p2 = t2 ? 32 + 2 * c : 0;
  }
  const uint32_t buffer = tile_buffer_bytes(p.hg, P);
  const uint32_t table = static_cast<uint32_t>(p.hg) * kBatchRows * kRowBytes;    // offset in a buffer
  const uint32_t sb = smem_u32(tile_smem), mine = sb + warp * kBatchRows * kRowBytes;
  const int64_t token_bytes = static_cast<int64_t>(a.H) * kRowBytes;
  const int32_t row_units = P / 2;                                                // 16-byte units a table row

  const auto checked = [&](int32_t tok) {
    if (tok >= a.N) {
      if (lane < 16) flag_status(ST_BAD_MAP);
      return -1;
    }
    return tok;
  };
  const auto issue = [&](const TileBatch& q, int32_t tok, uint32_t k) {
    if (q.u < a.units) {
      const int32_t h = q.h0 + static_cast<int32_t>(warp);
      const uint8_t* raster = a.src + (static_cast<int64_t>(q.b) * a.N * a.H + h) * kRowBytes + c * 16;
      const uint8_t* tile = a.src + ((static_cast<int64_t>(q.b) * a.H + h) * a.Npad + static_cast<int64_t>(q.t) * 128 + q.r0) * kRowBytes + c * 16;
#pragma unroll
      for (int i = 0; i < kBatchRows / 2; ++i) {
        const int32_t tk = __shfl_sync(0xffffffffu, tok, 2 * i + half);
        if (tk >= 0)
          copy16_async(mine + k * buffer + (2 * i + half) * kRowBytes + c * 16,
                       kGather ? raster + tk * token_bytes : tile + (2 * i + half) * kRowBytes);
      }
      const float2* cs = p.cs + q.b * p.batch_rows * P;
      for (int32_t i = static_cast<int32_t>(threadIdx.x); i < kBatchRows * row_units; i += 32 * p.hg) {   // whole warps
        const int32_t r = i / row_units, o = i - r * row_units;
        const int32_t tk = __shfl_sync(0xffffffffu, tok, 16 + r);
        if (tk >= 0)
          copy16_async(sb + k * buffer + table + static_cast<uint32_t>(i) * 16, reinterpret_cast<const float4*>(cs + static_cast<int64_t>(tk) * P) + o);
      }
    }
    copies_commit();
  };

  // batches: the one at work, the next one (on its way), the one after (its tokens are known), and the
  // one whose tokens are on their way
  TileBatch cur, nxt, far;
  cur.at(static_cast<int32_t>(blockIdx.x), p);
  int32_t tok_cur = checked(cur.token(p, warp, lane));
  issue(cur, tok_cur, 0);
  nxt = cur;
  nxt.advance(p);
  int32_t tok_nxt = checked(nxt.token(p, warp, lane));
  issue(nxt, tok_nxt, 1);
  far = nxt;
  far.advance(p);
  int32_t tok_far = checked(far.token(p, warp, lane));
  uint32_t k = 0;
  float sum[8], mx[8], mn[8];
  int32_t nv = 0;
  while (cur.u < a.units) {
    TileBatch last = far;
    last.advance(p);
    const int32_t tok_last = last.token(p, warp, lane);
    copies_wait<1>();
    __syncthreads();            // the batch is here for the whole CTA, and the previous one's buffer is free
    issue(far, tok_far, k == 0 ? 2 : k - 1);
    const int32_t h = cur.h0 + static_cast<int32_t>(warp);
    if (h < a.H) {
      if (kGather && cur.r0 == 0) {
        nv = __ldg(p.valid + static_cast<int64_t>(h) * a.nT + cur.t);
        nv = nv < 0 ? 0 : (nv > 128 ? 128 : nv);
#pragma unroll
        for (int i = 0; i < 8; ++i) { sum[i] = 0.f; mx[i] = -INFINITY; mn[i] = INFINITY; }
      }
      const int64_t lin = (static_cast<int64_t>(cur.b) * a.H + h) * a.nT + cur.t;
      uint8_t* tile = a.dst + lin * kTileBytes + (cur.r0 + half) * kRowBytes;
      uint8_t* raster = a.dst + (static_cast<int64_t>(cur.b) * a.N * a.H + h) * kRowBytes;
      const float2* cs = p.cs + cur.b * p.batch_rows * P;
      const uint32_t src1 = mine + k * buffer + half * kRowBytes + o1 * 2, src2 = src1 + (o2 - o1) * 2;
      const uint32_t row1 = sb + k * buffer + table + static_cast<uint32_t>(half * P + p1) * 8u, row2 = row1 + (p2 - p1) * 8;
      // row 2 i + half, turned: the pieces as written and, in fp32, g
      const auto turn_row = [&](int i, const float4& ta, const float4& tb, float* g, uint2& v1, uint2& v2) {
        v1 = ld_shared8(src1 + i * 2 * kRowBytes);
        v2 = ld_shared8(src2 + i * 2 * kRowBytes);
        float f[8];
        unpack4(v1, f);
        unpack4(v2, f + 4);
        float4 ca = ta, cb = tb;
        if (!kGather) { ca.y *= p.sign; ca.w *= p.sign; cb.y *= p.sign; cb.w *= p.sign; }   // gather: +1
        if (kHalf) {            // pairs (f[e], f[4 + e]), cos / sin (ca, ca, cb, cb)
          g[0] = fmaf(f[0], ca.x, -(f[4] * ca.y)); g[4] = fmaf(f[4], ca.x, f[0] * ca.y);
          g[1] = fmaf(f[1], ca.z, -(f[5] * ca.w)); g[5] = fmaf(f[5], ca.z, f[1] * ca.w);
          g[2] = fmaf(f[2], cb.x, -(f[6] * cb.y)); g[6] = fmaf(f[6], cb.x, f[2] * cb.y);
          g[3] = fmaf(f[3], cb.z, -(f[7] * cb.w)); g[7] = fmaf(f[7], cb.z, f[3] * cb.w);
        } else {
          g[0] = fmaf(f[0], ca.x, -(f[1] * ca.y)); g[1] = fmaf(f[1], ca.x, f[0] * ca.y);
          g[2] = fmaf(f[2], ca.z, -(f[3] * ca.w)); g[3] = fmaf(f[3], ca.z, f[2] * ca.w);
          g[4] = fmaf(f[4], cb.x, -(f[5] * cb.y)); g[5] = fmaf(f[5], cb.x, f[4] * cb.y);
          g[6] = fmaf(f[6], cb.z, -(f[7] * cb.w)); g[7] = fmaf(f[7], cb.z, f[6] * cb.w);
        }
        if (kFull || t1) {
          v1 = make_uint2(pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3]));
        } else {                // behind the turned channels: the bits as they are
#pragma unroll
          for (int e = 0; e < 4; ++e) g[e] = f[e];
        }
        if (kFull || t2) {
          v2 = make_uint2(pack_bf16x2(g[4], g[5]), pack_bf16x2(g[6], g[7]));
        } else {
#pragma unroll
          for (int e = 4; e < 8; ++e) g[e] = f[e];
        }
      };
      uint8_t* tile1 = tile + o1 * 2;
      uint8_t* tile2 = tile + o2 * 2;
      // three kinds of batch, by one vote: every slot's token is that of the CTA's first head (whose
      // table rows are in shared memory), no slot has a token, and the rest, row by row
      const int32_t first_head = __shfl_sync(0xffffffffu, tok_cur, 16 + c);
      const bool same = __all_sync(0xffffffffu, tok_cur >= 0 && tok_cur == first_head) &&
                        (!kGather || nv >= cur.r0 + kBatchRows);
      if (same) {
#pragma unroll
        for (int i = 0; i < kBatchRows / 2; i += 2) {      // two rows at a time: three-input max / min
          float g[8], q[8];
          uint2 v1, v2;
          turn_row(i, ld_shared_f4(row1 + i * 16 * P), ld_shared_f4(row2 + i * 16 * P), g, v1, v2);
          if (kGather) {
            st_v2(tile1 + 2 * i * kRowBytes, v1);
            st_v2(tile2 + 2 * i * kRowBytes, v2);
          } else {
            uint8_t* dst = raster + __shfl_sync(0xffffffffu, tok_cur, 2 * i + half) * token_bytes;
            st_v2(dst + o1 * 2, v1);
            st_v2(dst + o2 * 2, v2);
          }
          turn_row(i + 1, ld_shared_f4(row1 + (i + 1) * 16 * P), ld_shared_f4(row2 + (i + 1) * 16 * P), q, v1, v2);
          if (kGather) {
            st_v2(tile1 + (2 * i + 2) * kRowBytes, v1);
            st_v2(tile2 + (2 * i + 2) * kRowBytes, v2);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              sum[e] += g[e] + q[e];
              mx[e] = fmax3(mx[e], g[e], q[e]);
              mn[e] = fmin3(mn[e], g[e], q[e]);
            }
          } else {
            uint8_t* dst = raster + __shfl_sync(0xffffffffu, tok_cur, 2 * i + 2 + half) * token_bytes;
            st_v2(dst + o1 * 2, v1);
            st_v2(dst + o2 * 2, v2);
          }
        }
      } else if (__all_sync(0xffffffffu, tok_cur < 0 || lane >= 16) && (!kGather || nv <= cur.r0)) {
        if (kGather) {
#pragma unroll
          for (int i = 0; i < kBatchRows / 2; ++i) {
            st_v2(tile1 + 2 * i * kRowBytes, make_uint2(0, 0));
            st_v2(tile2 + 2 * i * kRowBytes, make_uint2(0, 0));
          }
        }
      } else {
#pragma unroll
        for (int i0 = 0; i0 < kBatchRows / 2; i0 += 2) {   // the table's rows of two slots in flight
          int32_t tk[2];
          float4 ca[2], cb[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            tk[i] = __shfl_sync(0xffffffffu, tok_cur, 2 * (i0 + i) + half);
            const float2* row = cs + static_cast<int64_t>(max(tk[i], 0)) * P;
            ca[i] = __ldg(reinterpret_cast<const float4*>(row + p1));
            cb[i] = __ldg(reinterpret_cast<const float4*>(row + p2));
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int32_t r = 2 * (i0 + i) + half;
            float g[8];
            uint2 v1, v2;
            turn_row(i0 + i, ca[i], cb[i], g, v1, v2);
            if (tk[i] < 0) {               // no token: the buffer holds nothing
#pragma unroll
              for (int e = 0; e < 8; ++e) g[e] = 0.f;
              v1 = v2 = make_uint2(0, 0);
            }
            if (kGather) {
              st_v2(tile1 + 2 * (i0 + i) * kRowBytes, v1);
              st_v2(tile2 + 2 * (i0 + i) * kRowBytes, v2);
              if (cur.r0 + r < nv) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  sum[e] += g[e];
                  mx[e] = fmaxf(mx[e], g[e]);
                  mn[e] = fminf(mn[e], g[e]);
                }
              }
            } else if (tk[i] >= 0) {
              uint8_t* dst = raster + tk[i] * token_bytes;
              st_v2(dst + o1 * 2, v1);
              st_v2(dst + o2 * 2, v2);
            }
          }
        }
      }
      if (kGather && cur.r0 == 128 - kBatchRows) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 16);
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 16));
          mn[e] = fminf(mn[e], __shfl_xor_sync(0xffffffffu, mn[e], 16));
        }
        if (half == 0) {
          float* o = p.pooled + lin * 384;
          const float inv = nv > 0 ? 1.0f / static_cast<float>(nv) : 0.f;
          if (nv == 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) mx[e] = mn[e] = 0.f;
          }
          const auto put = [&](int32_t at, float x, float y, float z, float w) {
            *reinterpret_cast<float4*>(o + at) = make_float4(x, y, z, w);
          };
          put(o1, sum[0] * inv, sum[1] * inv, sum[2] * inv, sum[3] * inv);
          put(o2, sum[4] * inv, sum[5] * inv, sum[6] * inv, sum[7] * inv);
          put(128 + o1, mx[0], mx[1], mx[2], mx[3]);
          put(128 + o2, mx[4], mx[5], mx[6], mx[7]);
          put(256 + o1, mn[0], mn[1], mn[2], mn[3]);
          put(256 + o2, mn[4], mn[5], mn[6], mn[7]);
        }
      }
    }
    cur = nxt;
    tok_cur = tok_nxt;
    nxt = far;
    tok_nxt = tok_far;
    far = last;
    tok_far = checked(tok_last);
    k = k == 2 ? 0 : k + 1;
  }
  copies_wait<0>();
}

}  // namespace rotary
}  // namespace veda
