// veda_norm.cu -- the C ABI of the norms around a block (include/veda.h): argument checks and
// launches. Kernels in k_norm.cuh.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <map>
#include <mutex>
#include <tuple>

#include "k_norm.cuh"
#include "veda_host.h"

namespace veda {
namespace {

using norm::Args;

veda_status fail(veda_status st, const std::string& msg) {
  set_last_error(msg);
  return st;
}
veda_status cuda_fail(cudaError_t e, const char* what) {
  return fail(VEDA_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

bool known(int32_t dtype) { return dtype >= VEDA_BF16 && dtype <= VEDA_FP32; }
int64_t size_of(int32_t dtype) { return dtype == VEDA_FP32 ? 4 : 2; }
bool on(const void* p, int64_t a) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(a) == 0; }

// Rows of this tensor start on 16-byte boundaries.
bool vec_rows(const void* p, int64_t sb, int64_t sn, int32_t dtype) {
  return on(p, 16) && sb * size_of(dtype) % 16 == 0 && sn * size_of(dtype) % 16 == 0;
}

// Rows in the ring: enough bytes in flight for the HBM's latency (Little's law asks for about 45 KB
// an SM), few enough that several CTAs share the SM. Measured as below, of 2 / 3 / 4 rows: forward at
// 5,120 channels, bf16 73 / 79 / 78%, with a residual 93 / 84 / 87% (two tensors: three CTAs an SM
// with 2, two with 4; 256 channels, a row per warp, 77 / 91 / 85%), fp32 to bf16 87 / 88 / 72% (with 4
// one CTA an SM), fp32 residual at 4,096 88 / 92 / 94%; backward 2: 78, 3: 79%.
constexpr int kMaxRing = 224 * 1024;
int ring_rows(bool bwd, bool is_aligned, int32_t ti, int32_t to, bool res, int32_t C) {
  if (!is_aligned) return 2;                     // plain loads: one row ahead
  if (bwd) return 3;
  if (res) return ti != VEDA_FP32 && to != VEDA_FP32 && C > 512 ? 2 : 4;
  return ti == VEDA_FP32 ? 3 : 4;
}

// Who holds a row. Measured on 120 M bf16 values (share of the HBM copy rate; forward without /
// with a residual, backward):
//   a warp, 2 or 4 vectors a lane, up to 1,024 channels: 1,024 channels 79 / 83 / 75%, a CTA of
//     1-vector threads there 58 / 84 / 63%;
//   above, a CTA: the row sums cost a thread the same whatever it holds, so more vectors a thread
//     are faster as long as their registers leave two CTAs an SM: forward without a residual 4
//     (5,120: 78%; 2: 72%), with one 2 (8,192: 93%; 4: 78%), backward 2 (5,120: 80%; 4: 60%).
// Rows without 16-byte boundaries, and all whose channels are no multiple of 8 (also fp32 rows of a
// multiple of 4, which start on such boundaries: 1,004 channels 81 / 71% forward / backward, 1,024 85 /
// 80%), are fetched with plain loads that stall their warp, so there more
// warps with less each are faster: above 256 channels a CTA of 1-vector threads, of 128, 256 or 512
// (backward of 6,147 rows of 1,023, a warp a row 41 us, 64 threads of 2 vectors 54 us).
struct Shape {
  int nv;          // vectors per thread
  bool warp;       // a row per warp
  int threads;     // per CTA
};
Shape shape_of(int32_t C, bool is_aligned, bool bwd, bool res) {
  const int vecs = (C + norm::kVec - 1) / norm::kVec;
  const int warp_threads = 32 * norm::kWarpsPerCta;
  if (C <= 256) return {1, true, warp_threads};
  if (is_aligned && C <= norm::kWarpCols) return {C <= 512 ? 2 : 4, true, warp_threads};
  if (!is_aligned) return {C <= 4096 ? 1 : 2, false, C <= 1024 ? 128 : C <= 2048 ? 256 : norm::kMaxThreads};
  const int nv = bwd || res ? 2 : 4;
  return {nv, false, ((vecs + nv - 1) / nv + 31) / 32 * 32};     // at most kMaxThreads (nv 4: 256)
}

typedef void (*Kernel)(const Args);

// The kernels of one shape for every type pair; null for a pair that is not built.
template <template <typename, typename> class K>
Kernel by_types(int32_t ti, int32_t to) {
  using B = __nv_bfloat16;
  using H = __half;
  if (ti == VEDA_BF16 && to == VEDA_BF16) return K<B, B>::kernel();
  if (ti == VEDA_FP16 && to == VEDA_FP16) return K<H, H>::kernel();
  if (ti == VEDA_FP32 && to == VEDA_FP32) return K<float, float>::kernel();
  if (ti == VEDA_FP32 && to == VEDA_BF16) return K<float, B>::kernel();
  if (ti == VEDA_BF16 && to == VEDA_FP32) return K<B, float>::kernel();
  return nullptr;
}
// A: aligned rows; who owns what there depends on the types
template <typename TI, typename TO, bool A>
constexpr int mode_of() { return !A ? norm::kSingle : sizeof(TI) == 4 || sizeof(TO) == 4 ? norm::kHalves : norm::kVectors; }
template <int NV, bool W, bool A, int FIXED = 0>
struct Fwd {
  template <typename TI, typename TO> struct K {
    static Kernel kernel() { return norm::norm_fwd_kernel<TI, TO, NV, W, mode_of<TI, TO, A>(), FIXED>; }
  };
};
template <int NV, bool W, int BOUND, bool A, int FIXED = 0>
struct Bwd {
  template <typename TI, typename TO> struct K {
    static Kernel kernel() { return norm::norm_bwd_kernel<TI, TO, NV, W, BOUND, mode_of<TI, TO, A>(), FIXED>; }
  };
};
constexpr int kMid = 320, kBig = norm::kMaxThreads;      // thread bounds of the CTA-per-row backward

// is_aligned: every row starts on a 16-byte boundary and C % 8 == 0
Kernel pick(const Shape& s, bool bwd, bool is_aligned, int32_t ti, int32_t to) {
  if (!is_aligned) {
    if (s.warp) return bwd ? by_types<Bwd<1, true, 256, false>::K>(ti, to) : by_types<Fwd<1, true, false>::K>(ti, to);
    if (s.nv == 2) return bwd ? by_types<Bwd<2, false, kBig, false, 512>::K>(ti, to) : by_types<Fwd<2, false, false, 512>::K>(ti, to);
    if (s.threads == 128) return bwd ? by_types<Bwd<1, false, kBig, false, 128>::K>(ti, to) : by_types<Fwd<1, false, false, 128>::K>(ti, to);
    if (s.threads == 256) return bwd ? by_types<Bwd<1, false, kBig, false, 256>::K>(ti, to) : by_types<Fwd<1, false, false, 256>::K>(ti, to);
    return bwd ? by_types<Bwd<1, false, kBig, false, 512>::K>(ti, to) : by_types<Fwd<1, false, false, 512>::K>(ti, to);
  }
  if (s.warp) {
    if (s.nv == 1) return bwd ? by_types<Bwd<1, true, 256, true>::K>(ti, to) : by_types<Fwd<1, true, true>::K>(ti, to);
    if (s.nv == 2) return bwd ? by_types<Bwd<2, true, 256, true>::K>(ti, to) : by_types<Fwd<2, true, true>::K>(ti, to);
    return bwd ? by_types<Bwd<4, true, 256, true>::K>(ti, to) : by_types<Fwd<4, true, true>::K>(ti, to);
  }
  if (!bwd) return s.nv == 4 ? by_types<Fwd<4, false, true>::K>(ti, to) : by_types<Fwd<2, false, true>::K>(ti, to);
  return s.threads <= kMid ? by_types<Bwd<2, false, kMid, true>::K>(ti, to) : by_types<Bwd<2, false, kBig, true>::K>(ti, to);
}

// Ring bytes of a CTA: every row a group has in flight, 16-byte units.
int ring_bytes(const Shape& s, bool bwd, bool is_aligned, int32_t ti, int32_t to, bool res, int32_t C, int32_t& stages) {
  const int ui = ti == VEDA_FP32 ? 2 : 1, uo = to == VEDA_FP32 ? 2 : 1;
  const int units = bwd ? ui + uo + (res ? ui : 0) : ui + (res ? uo : 0);
  const int row = s.nv * units * s.threads * 16;            // <= 96 KB (fp32, 8,192 channels)
  stages = ring_rows(bwd, is_aligned, ti, to, res, C);
  while (stages > 2 && stages * row > kMaxRing) --stages;
  return stages * row;
}

// CTAs of this kernel that fit an SM, asked once per device, kernel and ring. Rings over the
// default limit (48 KB with the static part) are opted into first, always with the same maximum,
// so that calls from two threads cannot take it from one another.
veda_status resident(Kernel k, int threads, int bytes, int& per_sm) {
  static std::mutex mu;
  static std::map<std::tuple<int, Kernel, int, int>, int> known_fits;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  std::lock_guard<std::mutex> lk(mu);
  const auto key = std::make_tuple(dev, k, threads, bytes);
  const auto it = known_fits.find(key);
  if (it != known_fits.end()) {
    per_sm = it->second;
    return VEDA_OK;
  }
  const void* f = reinterpret_cast<const void*>(k);
  if (bytes > 32 * 1024 &&
      (e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxRing)) != cudaSuccess)
    return cuda_fail(e, "cudaFuncSetAttribute");
  if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, f, threads, static_cast<size_t>(bytes))) != cudaSuccess)
    return cuda_fail(e, "cudaOccupancyMaxActiveBlocksPerMultiprocessor");
  known_fits[key] = per_sm;
  return VEDA_OK;
}

// Slices per sequence: together the CTAs that can run at once (so a CTA keeps its channels'
// parameters for as many rows as possible), no more than there are rows; in the backward with a few
// rows each, as every slice also writes two rows of fp32 sums. A sequence has whole slices, so the
// count is rounded down or up, whichever takes fewer rows one after the other (waves of CTAs times the
// rows of one), and up where that is equal: rounded down, some of the SMs' places stay empty, rounded up,
// a few CTAs may run alone behind the others. Measured on 100 M bf16 values, us down / up: 5,120
// channels, 3 sequences, with an fp32 residual 176 / 334, backward 154 / 221; 7 sequences, forward 80 /
// 125; equal counts of rows (150 sequences, backward) 358 / 324.
constexpr int kMaxPerSmFwd = 8, kMaxPerSmBwd = 4, kMaxSms = 160, kMinRowsBwd = 4;
veda_status slices_for(Kernel k, const Shape& s, int bytes, int sms, bool bwd, int32_t B, int32_t N, int32_t& slices) {
  int per_sm = 0;
  const veda_status st = resident(k, s.threads, bytes, per_sm);
  if (st != VEDA_OK) return st;
  per_sm = std::max(1, std::min(per_sm, bwd ? kMaxPerSmBwd : kMaxPerSmFwd));
  const int64_t places = static_cast<int64_t>(std::min(sms, kMaxSms)) * per_sm;
  const int64_t down = std::max<int64_t>(1, places / B), up = (places + B - 1) / B;
  const auto waves = [&](int64_t each) { return (each * B + places - 1) / places; };
  const int64_t want = waves(up) * down <= waves(down) * up ? up : down;
  const int64_t rows = (s.warp ? norm::kWarpsPerCta : 1) * (bwd ? kMinRowsBwd : 1);       // a slice's, at least
  slices = static_cast<int32_t>(std::max<int64_t>(1, std::min(want, N / rows + (bwd ? 0 : N % rows != 0))));
  return VEDA_OK;
}

veda_status check_common(const char* call, int32_t x_dtype, int32_t y_dtype, const veda_norm_params* q, int32_t B,
                         int32_t N, int32_t C, int32_t kind, float eps) {
  const std::string c(call);
  if (B < 0 || N < 0 || N > INT32_MAX - 1024 || C <= 0) return fail(VEDA_ERR_INVALID_ARG, c + ": bad size");
  if (!known(x_dtype) || !known(y_dtype) || !q || !known(q->weight_dtype) || !known(q->mod_dtype))
    return fail(VEDA_ERR_INVALID_ARG, c + ": unknown type");
  if (kind < VEDA_NORM_LAYER || kind > VEDA_NORM_NONE) return fail(VEDA_ERR_INVALID_ARG, c + ": unknown kind of norm");
  if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(VEDA_ERR_INVALID_ARG, c + ": eps must be finite and >= 0");
  if (C > norm::kMaxCols) return fail(VEDA_ERR_UNSUPPORTED, c + ": more than 8192 channels");
  if (!pick({1, true, 0}, false, true, x_dtype, y_dtype))
    return fail(VEDA_ERR_UNSUPPORTED, c + ": input and output types must be equal, or bf16 and fp32");
  const int64_t ws = size_of(q->weight_dtype), ms = size_of(q->mod_dtype);
  if (!on(q->weight, ws) || !on(q->bias, ws) || !on(q->gain, ms) || !on(q->shift, ms))
    return fail(VEDA_ERR_INVALID_ARG, c + ": misaligned parameter");
  return VEDA_OK;
}

void set_params(Args& a, const veda_norm_params* q) {
  const auto param = [&](const void* p, int64_t stride, int32_t dtype) {
    return norm::Param{p, stride, dtype, a.C % norm::kVec == 0 && vec_rows(p, stride, 0, dtype) ? 1 : 0};
  };
  a.w = param(q->weight, 0, q->weight_dtype);
  a.b = param(q->bias, 0, q->weight_dtype);
  a.g = param(q->gain, q->gain_stride, q->mod_dtype);
  a.t = param(q->shift, q->shift_stride, q->mod_dtype);
  a.gain_off = q->gain_offset;
}

}  // namespace
}  // namespace veda

using namespace veda;

extern "C" {

veda_status veda_norm_fwd(const veda_rows* x, const veda_rows* residual, const veda_rows* y,
                          const veda_norm_params* params, float residual_scale, float* mean, float* rstd, int32_t B,
                          int32_t N, int32_t C, int32_t kind, float eps, veda_stream_t stream) {
  return guarded("veda_norm_fwd", [&]() -> veda_status {
    const char* call = "veda_norm_fwd";
    if (!x || !y) return fail(VEDA_ERR_INVALID_ARG, "veda_norm_fwd: no input or output");
    veda_status st = check_common(call, x->dtype, y->dtype, params, B, N, C, kind, eps);
    if (st != VEDA_OK) return st;
    if (residual && residual->dtype != y->dtype)
      return fail(VEDA_ERR_INVALID_ARG, "veda_norm_fwd: the residual has the output's type");
    if ((mean && !rstd)) return fail(VEDA_ERR_INVALID_ARG, "veda_norm_fwd: mean without rstd");
    if (B == 0 || N == 0) return VEDA_OK;
    if (!x->data || !y->data || (residual && !residual->data) || !on(x->data, size_of(x->dtype)) ||
        !on(y->data, size_of(y->dtype)) || (residual && !on(residual->data, size_of(y->dtype))) || !on(mean, 4) ||
        !on(rstd, 4))
      return fail(VEDA_ERR_INVALID_ARG, "veda_norm_fwd: bad pointer");
    int sms;
    if ((st = host_device(sms)) != VEDA_OK) return st;
    Args a{};
    a.x = x->data; a.xb = x->batch_stride; a.xn = x->row_stride;
    a.y = y->data; a.yb = y->batch_stride; a.yn = y->row_stride;
    if (residual) { a.res = residual->data; a.rb = residual->batch_stride; a.rn = residual->row_stride; }
    a.C = C;
    set_params(a, params);
    a.res_scale = residual_scale; a.eps = eps; a.inv_c = 1.0f / static_cast<float>(C);
    a.mean = mean; a.rstd = rstd;
    a.B = B; a.N = N; a.kind = kind;
    const bool vec = C % norm::kVec == 0 && vec_rows(a.x, a.xb, a.xn, x->dtype) && vec_rows(a.y, a.yb, a.yn, y->dtype) &&
            (!residual || vec_rows(a.res, a.rb, a.rn, y->dtype));
    const Shape s = shape_of(C, vec, false, residual != nullptr);
    const int bytes = ring_bytes(s, false, vec, x->dtype, y->dtype, residual != nullptr, C, a.stages);
    const Kernel k = pick(s, false, vec, x->dtype, y->dtype);
    if ((st = slices_for(k, s, bytes, sms, false, B, N, a.slices)) != VEDA_OK) return st;
    k<<<static_cast<unsigned>(B * a.slices), s.threads, bytes, reinterpret_cast<cudaStream_t>(stream)>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? VEDA_OK : cuda_fail(e, "norm_fwd_kernel");
  });
}

size_t veda_norm_bwd_workspace_bytes(int32_t B, int32_t N, int32_t C) {
  if (B <= 0 || N <= 0 || C <= 0 || C > norm::kMaxCols) return 0;
  // partial sums of every slice (slices_for: fewer than kMaxSms * kMaxPerSmBwd + B in all, and at
  // most one a row), then one row pair per sequence, then a counter per 32 channels
  const int64_t slices = std::min<int64_t>(static_cast<int64_t>(B) * N, kMaxSms * kMaxPerSmBwd + B);
  return static_cast<size_t>((slices + B) * 2 * C + (C + 31) / 32) * sizeof(float);
}

veda_status veda_norm_bwd(const veda_rows* dy, const veda_rows* x, const float* mean, const float* rstd,
                          const veda_rows* residual_grad, const veda_rows* dx, const veda_norm_params* params,
                          float residual_scale, float* dgain, float* dshift, float* dweight, float* dbias,
                          void* workspace, size_t workspace_bytes, int32_t B, int32_t N, int32_t C, int32_t kind,
                          veda_stream_t stream) {
  return guarded("veda_norm_bwd", [&]() -> veda_status {
    const char* call = "veda_norm_bwd";
    if (!dy || !x || !dx) return fail(VEDA_ERR_INVALID_ARG, "veda_norm_bwd: no input or output");
    veda_status st = check_common(call, x->dtype, dy->dtype, params, B, N, C, kind, 0.f);
    if (st != VEDA_OK) return st;
    if (dx->dtype != x->dtype || (residual_grad && residual_grad->dtype != x->dtype))
      return fail(VEDA_ERR_INVALID_ARG, "veda_norm_bwd: dx and the gradient around the block have x's type");
    const cudaStream_t s0 = reinterpret_cast<cudaStream_t>(stream);
    if (!on(dgain, 4) || !on(dshift, 4) || !on(dweight, 4) || !on(dbias, 4))
      return fail(VEDA_ERR_INVALID_ARG, "veda_norm_bwd: misaligned gradient");
    int sms;
    if (B == 0 || N == 0) {           // no token: the parameters' gradients are zero
      if ((st = host_device(sms)) != VEDA_OK) return st;
      cudaError_t e = cudaSuccess;
      const size_t row = static_cast<size_t>(C) * sizeof(float);
      if (dgain && B && e == cudaSuccess) e = cudaMemsetAsync(dgain, 0, row * B, s0);
      if (dshift && B && e == cudaSuccess) e = cudaMemsetAsync(dshift, 0, row * B, s0);
      if (dweight && e == cudaSuccess) e = cudaMemsetAsync(dweight, 0, row, s0);
      if (dbias && e == cudaSuccess) e = cudaMemsetAsync(dbias, 0, row, s0);
      return e == cudaSuccess ? VEDA_OK : cuda_fail(e, "cudaMemsetAsync");
    }
    if (!dy->data || !x->data || !dx->data || (residual_grad && !residual_grad->data) ||
        !on(dy->data, size_of(dy->dtype)) || !on(x->data, size_of(x->dtype)) || !on(dx->data, size_of(x->dtype)) ||
        (residual_grad && !on(residual_grad->data, size_of(x->dtype))))
      return fail(VEDA_ERR_INVALID_ARG, "veda_norm_bwd: bad pointer");
    if ((kind != VEDA_NORM_NONE && !rstd) || (kind == VEDA_NORM_LAYER && !mean) || !on(mean, 4) || !on(rstd, 4))
      return fail(VEDA_ERR_INVALID_ARG, "veda_norm_bwd: the forward's statistics are missing");
    if (!workspace || !on(workspace, 16) || workspace_bytes < veda_norm_bwd_workspace_bytes(B, N, C))
      return fail(VEDA_ERR_INVALID_ARG, "veda_norm_bwd: workspace too small or misaligned");
    if (B > 65535) return fail(VEDA_ERR_UNSUPPORTED, "veda_norm_bwd: more than 65535 sequences");
    if ((st = host_device(sms)) != VEDA_OK) return st;
    Args a{};
    a.x = x->data; a.xb = x->batch_stride; a.xn = x->row_stride;
    a.dy = dy->data; a.db = dy->batch_stride; a.dn = dy->row_stride;
    a.y = dx->data; a.yb = dx->batch_stride; a.yn = dx->row_stride;
    if (residual_grad) { a.res = residual_grad->data; a.rb = residual_grad->batch_stride; a.rn = residual_grad->row_stride; }
    a.C = C;
    set_params(a, params);
    a.res_scale = residual_scale; a.inv_c = 1.0f / static_cast<float>(C);
    a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd);
    a.B = B; a.N = N; a.kind = kind;
    const bool vec = C % norm::kVec == 0 && vec_rows(a.x, a.xb, a.xn, x->dtype) && vec_rows(a.dy, a.db, a.dn, dy->dtype) &&
            vec_rows(a.y, a.yb, a.yn, x->dtype) && (!a.res || vec_rows(a.res, a.rb, a.rn, x->dtype));
    const Shape s = shape_of(C, vec, true, a.res != nullptr);
    const int bytes = ring_bytes(s, true, vec, x->dtype, dy->dtype, a.res != nullptr, C, a.stages);
    a.part = static_cast<float*>(workspace);
    const Kernel k = pick(s, true, vec, x->dtype, dy->dtype);
    if ((st = slices_for(k, s, bytes, sms, true, B, N, a.slices)) != VEDA_OK) return st;
    float* const pairs = a.part + static_cast<int64_t>(B) * a.slices * 2 * C;
    const bool over_sequences = B > 1 && (dweight || dbias);
    if (over_sequences) a.done = reinterpret_cast<int32_t*>(pairs + static_cast<int64_t>(B) * 2 * C);
    k<<<static_cast<unsigned>(B * a.slices), s.threads, bytes, s0>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "norm_bwd_kernel");
    if (!dgain && !dshift && !dweight && !dbias) return VEDA_OK;
    norm::GradArgs g{};
    g.part = a.part;
    g.w = a.w; g.b = a.b; g.g = a.g;
    g.gain_off = a.gain_off;
    g.dgain = dgain; g.dshift = dshift;
    g.B = B; g.C = C; g.slices = a.slices;
    g.dw = dweight; g.db = dbias;
    if (over_sequences) {
      g.gp = pairs;
      g.done = a.done;
    }
    norm::norm_grad_kernel<<<dim3((C + 31) / 32, B), 32 * norm::kGradRows, 0, s0>>>(g);
    if ((e = cudaGetLastError()) != cudaSuccess) return cuda_fail(e, "norm_grad_kernel");
    return VEDA_OK;
  });
}

}  // extern "C"
