// api.cpp -- the C ABI (include/sq.h): argument checks, then dispatch to the
// kernel launchers.  Nothing is enqueued when a check fails.
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include "sq_internal.h"

namespace sq {

namespace {
thread_local char g_last_error[512] = "";
constexpr int64_t kMaxK = 133136;  // 127*127*K < 2^31

bool aligned16(const void* p) { return (((uintptr_t)p) & 15u) == 0; }

sq_status check_dtype(sq_dtype t, const char* what) {
  if (t != SQ_F32 && t != SQ_BF16) return fail(SQ_ERR_DTYPE, "%s: unknown dtype %d", what, (int)t);
  return SQ_OK;
}

sq_status check_k(int64_t K, const char* fn) {
  if (K < 16 || K > kMaxK || (K % 16) != 0)
    return fail(SQ_ERR_SHAPE, "%s: K=%lld must be a multiple of 16 in [16, %lld]", fn,
                (long long)K, (long long)kMaxK);
  return SQ_OK;
}

#define SQ_REQ(ptr, fn)                                                                \
  do {                                                                                 \
    if (!(ptr)) return fail(SQ_ERR_INVALID_ARG, "%s: %s must not be NULL", fn, #ptr); \
    if (!aligned16(ptr))                                                               \
      return fail(SQ_ERR_ALIGN, "%s: %s is not 16-byte aligned", fn, #ptr);          \
  } while (0)
#define SQ_OPT(ptr, fn)                                                       \
  do {                                                                        \
    if ((ptr) && !aligned16(ptr))                                             \
      return fail(SQ_ERR_ALIGN, "%s: %s is not 16-byte aligned", fn, #ptr); \
  } while (0)
#define SQ_TRY(expr)                 \
  do {                               \
    sq_status _st = (expr);          \
    if (_st != SQ_OK) return _st;    \
  } while (0)

sq_status cuda_fail(cudaError_t e, const char* fn) {
  return fail(SQ_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
}

}  // namespace

sq_status fail(sq_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof g_last_error, fmt, ap);
  va_end(ap);
  return st;
}

}  // namespace sq

using namespace sq;

extern "C" {

namespace {
sq_status calib_call(const char* fn, const void* x, sq_dtype xt, int64_t T, int64_t K,
                     const float* ln_gamma, const float* ln_beta, float ln_eps, int rms,
                     float* amax, sq_stream stream) {
  g_last_error[0] = 0;
  SQ_TRY(check_dtype(xt, fn));
  if (T < 0) return fail(SQ_ERR_SHAPE, "%s: T=%lld < 0", fn, (long long)T);
  SQ_TRY(check_k(K, fn));
  SQ_REQ(x, fn);
  SQ_REQ(amax, fn);
  if (rms) SQ_REQ(ln_gamma, fn);
  SQ_OPT(ln_gamma, fn);
  SQ_OPT(ln_beta, fn);
  if (ln_beta && !ln_gamma) return fail(SQ_ERR_INVALID_ARG, "%s: ln_beta given without ln_gamma", fn);
  if (ln_gamma && !(ln_eps >= 0.0f && isfinite(ln_eps)))
    return fail(SQ_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", fn);
  if (T == 0) return SQ_OK;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e;
  if (!ln_gamma) {
    e = launch_colmax(x, xt, T, K, amax, st);
  } else {
    RowArgs a{};
    a.x = x; a.T = T; a.K = K; a.g = ln_gamma; a.b = ln_beta; a.eps = ln_eps; a.rms = rms;
    a.colmax = amax;
    e = launch_row(a, xt, ROW_COLMAX, st);
  }
  return e == cudaSuccess ? SQ_OK : cuda_fail(e, fn);
}
}  // namespace

sq_status sq_calib_absmax(const void* x, sq_dtype xt, int64_t T, int64_t K,
                          const float* ln_gamma, const float* ln_beta, float ln_eps,
                          float* amax, sq_stream stream) {
  return calib_call("sq_calib_absmax", x, xt, T, K, ln_gamma, ln_beta, ln_eps, 0, amax, stream);
}

sq_status sq_calib_absmax_rms(const void* x, sq_dtype xt, int64_t T, int64_t K,
                              const float* gamma, float eps, float* amax, sq_stream stream) {
  return calib_call("sq_calib_absmax_rms", x, xt, T, K, gamma, nullptr, eps, 1, amax, stream);
}

sq_status sq_smooth_scales(const float* amax_x, const void* w, sq_dtype wt, int64_t N, int64_t K,
                           float alpha, float* s, float* inv_s, float* act_delta_static,
                           sq_stream stream) {
  const char* fn = "sq_smooth_scales";
  g_last_error[0] = 0;
  SQ_TRY(check_dtype(wt, fn));
  if (N < 0) return fail(SQ_ERR_SHAPE, "%s: N=%lld < 0", fn, (long long)N);
  SQ_TRY(check_k(K, fn));
  if (!(alpha >= 0.0f && alpha <= 1.0f))
    return fail(SQ_ERR_INVALID_ARG, "%s: alpha=%g must lie in [0, 1]", fn, (double)alpha);
  SQ_REQ(amax_x, fn);
  SQ_REQ(s, fn);
  SQ_REQ(inv_s, fn);
  SQ_OPT(act_delta_static, fn);
  if (N > 0) SQ_REQ(w, fn);
  cudaStream_t st = (cudaStream_t)stream;
  // s first holds the weight column peaks (running max from 0)
  cudaError_t e = cudaMemsetAsync(s, 0, (size_t)K * sizeof(float), st);
  if (e == cudaSuccess && N > 0) e = launch_colmax(w, wt, N, K, s, st);
  if (e == cudaSuccess) e = launch_scales(amax_x, s, K, alpha, s, inv_s, act_delta_static, st);
  return e == cudaSuccess ? SQ_OK : cuda_fail(e, fn);
}

sq_status sq_weight_colmax(const void* w, sq_dtype wt, int64_t N, int64_t K, float* amax_w,
                           sq_stream stream) {
  const char* fn = "sq_weight_colmax";
  g_last_error[0] = 0;
  SQ_TRY(check_dtype(wt, fn));
  if (N < 0) return fail(SQ_ERR_SHAPE, "%s: N=%lld < 0", fn, (long long)N);
  SQ_TRY(check_k(K, fn));
  SQ_REQ(amax_w, fn);
  if (N > 0) SQ_REQ(w, fn);
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = cudaMemsetAsync(amax_w, 0, (size_t)K * sizeof(float), st);
  if (e == cudaSuccess && N > 0) e = launch_colmax(w, wt, N, K, amax_w, st);
  return e == cudaSuccess ? SQ_OK : cuda_fail(e, fn);
}

sq_status sq_smooth_scales_peaks(const float* amax_x, const float* amax_w, int64_t K, float alpha,
                                 float* s, float* inv_s, float* act_delta_static,
                                 sq_stream stream) {
  const char* fn = "sq_smooth_scales_peaks";
  g_last_error[0] = 0;
  SQ_TRY(check_k(K, fn));
  if (!(alpha >= 0.0f && alpha <= 1.0f))
    return fail(SQ_ERR_INVALID_ARG, "%s: alpha=%g must lie in [0, 1]", fn, (double)alpha);
  SQ_REQ(amax_x, fn);
  SQ_REQ(amax_w, fn);
  SQ_REQ(s, fn);
  SQ_REQ(inv_s, fn);
  SQ_OPT(act_delta_static, fn);
  cudaError_t e = launch_scales(amax_x, amax_w, K, alpha, s, inv_s, act_delta_static,
                                (cudaStream_t)stream);
  return e == cudaSuccess ? SQ_OK : cuda_fail(e, fn);
}

sq_status sq_fuse_weights_q8(const void* w, sq_dtype wt, int64_t N, int64_t K, const float* s,
                             int8_t* wq, float* w_scale, const float* gamma, const float* beta,
                             float* gamma_out, float* beta_out, sq_stream stream) {
  const char* fn = "sq_fuse_weights_q8";
  g_last_error[0] = 0;
  SQ_TRY(check_dtype(wt, fn));
  if (N < 0) return fail(SQ_ERR_SHAPE, "%s: N=%lld < 0", fn, (long long)N);
  SQ_TRY(check_k(K, fn));
  SQ_REQ(s, fn);
  SQ_OPT(gamma, fn);
  SQ_OPT(beta, fn);
  SQ_OPT(gamma_out, fn);
  SQ_OPT(beta_out, fn);
  if (N > 0) {
    SQ_REQ(w, fn);
    SQ_REQ(wq, fn);
    SQ_REQ(w_scale, fn);
  }
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = cudaSuccess;
  const bool fold_g = gamma && gamma_out, fold_b = beta && beta_out;
  if (N > 0) {
    // W_hat = W * s, then per-row (output channel) dynamic INT8: the same
    // row quantizer as the activations, with s as the column multiplier.
    // The same launch divides gamma and beta by s (no kernel of its own).
    RowArgs a{};
    a.x = w; a.T = N; a.K = K; a.mul = s; a.scale = w_scale; a.q = wq;
    a.fold_g = gamma; a.fold_g_out = fold_g ? gamma_out : nullptr;
    a.fold_b = beta; a.fold_b_out = fold_b ? beta_out : nullptr;
    e = launch_row(a, wt, ROW_DYNAMIC, st);
  } else if (fold_g || fold_b) {
    e = launch_fold_ln(gamma, beta, s, K, fold_g ? gamma_out : nullptr,
                       fold_b ? beta_out : nullptr, st);
  }
  return e == cudaSuccess ? SQ_OK : cuda_fail(e, fn);
}

namespace {
// The quantizer at granularity gran on validated arguments (a.scale is
// act_scale).  Per-tensor dynamic: two passes over x -- the peak of |y| over
// the call (into act_scale[0]), Delta of it in place, then the static
// quantizer with that step.
cudaError_t run_quant(const RowArgs& a, sq_dtype xt, sq_act_gran gran, cudaStream_t st) {
  if (gran != SQ_ACT_PER_TENSOR_DYNAMIC)
    return launch_row(a, xt, gran == SQ_ACT_PER_TOKEN_DYNAMIC ? ROW_DYNAMIC : ROW_STATIC, st);
  RowArgs p = a;
  p.q = nullptr;
  p.n_clipped = nullptr;
  p.peak = a.scale;
  // a kernel, not a memset node, so that the peak pass's launch overlaps
  // (measured: 30.4 -> 28.9 us for 2048 x 4096 tokens)
  cudaError_t e = launch_zero(a.scale, sizeof(float), st);
  if (e == cudaSuccess) e = launch_row(p, xt, ROW_PEAK, st);
  if (e == cudaSuccess) e = launch_peak_to_delta(a.scale, st);
  if (e == cudaSuccess) e = launch_row(a, xt, ROW_STATIC, st);
  return e;
}

sq_status quant_call(const char* fn, const void* x, sq_dtype xt, int64_t T, int64_t K,
                     const float* gamma_s, const float* beta_s, float ln_eps, int rms,
                     const float* inv_s, sq_act_gran gran, float* act_scale, int8_t* xq,
                     int64_t* n_clipped, sq_stream stream) {
  g_last_error[0] = 0;
  SQ_TRY(check_dtype(xt, fn));
  if (gran != SQ_ACT_PER_TENSOR_STATIC && gran != SQ_ACT_PER_TOKEN_DYNAMIC &&
      gran != SQ_ACT_PER_TENSOR_DYNAMIC)
    return fail(SQ_ERR_INVALID_ARG, "%s: unknown granularity %d", fn, (int)gran);
  if (T < 0) return fail(SQ_ERR_SHAPE, "%s: T=%lld < 0", fn, (long long)T);
  SQ_TRY(check_k(K, fn));
  SQ_REQ(x, fn);
  SQ_REQ(xq, fn);
  SQ_REQ(act_scale, fn);
  if (rms) SQ_REQ(gamma_s, fn);
  SQ_OPT(gamma_s, fn);
  SQ_OPT(beta_s, fn);
  SQ_OPT(inv_s, fn);
  if (n_clipped && (((uintptr_t)n_clipped) & 7u))
    return fail(SQ_ERR_ALIGN, "%s: n_clipped is not 8-byte aligned", fn);
  if (beta_s && !gamma_s) return fail(SQ_ERR_INVALID_ARG, "%s: beta_s given without gamma_s", fn);
  if (gamma_s && inv_s)
    return fail(SQ_ERR_INVALID_ARG, "%s: inv_s is folded into gamma_s/beta_s when a LayerNorm precedes; pass one of them", fn);
  if (gamma_s && !(ln_eps >= 0.0f && isfinite(ln_eps)))
    return fail(SQ_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", fn);
  if (T == 0) return SQ_OK;
  RowArgs a{};
  a.x = x; a.T = T; a.K = K; a.g = gamma_s; a.b = beta_s; a.eps = ln_eps; a.rms = rms;
  a.mul = inv_s;
  a.scale = act_scale; a.q = xq; a.n_clipped = (unsigned long long*)n_clipped;
  const cudaError_t e = run_quant(a, xt, gran, (cudaStream_t)stream);
  return e == cudaSuccess ? SQ_OK : cuda_fail(e, fn);
}
}  // namespace

sq_status sq_fold_into_producer(const float* s, int64_t K, float* w_scale, float* bias,
                                sq_stream stream) {
  const char* fn = "sq_fold_into_producer";
  g_last_error[0] = 0;
  if (K < 0) return fail(SQ_ERR_SHAPE, "%s: K=%lld < 0", fn, (long long)K);
  SQ_REQ(s, fn);
  SQ_REQ(w_scale, fn);
  SQ_OPT(bias, fn);
  if (K == 0) return SQ_OK;
  cudaError_t e = launch_fold_producer(s, K, w_scale, bias, (cudaStream_t)stream);
  return e == cudaSuccess ? SQ_OK : cuda_fail(e, fn);
}

sq_status sq_ln_smooth_quant_act(const void* x, sq_dtype xt, int64_t T, int64_t K,
                                 const float* gamma_s, const float* beta_s, float ln_eps,
                                 const float* inv_s, sq_act_gran gran, float* act_scale,
                                 int8_t* xq, int64_t* n_clipped, sq_stream stream) {
  return quant_call("sq_ln_smooth_quant_act", x, xt, T, K, gamma_s, beta_s, ln_eps, 0, inv_s,
                    gran, act_scale, xq, n_clipped, stream);
}

sq_status sq_rms_smooth_quant_act(const void* x, sq_dtype xt, int64_t T, int64_t K,
                                  const float* gamma_s, float eps, sq_act_gran gran,
                                  float* act_scale, int8_t* xq, int64_t* n_clipped,
                                  sq_stream stream) {
  return quant_call("sq_rms_smooth_quant_act", x, xt, T, K, gamma_s, nullptr, eps, 1, nullptr,
                    gran, act_scale, xq, n_clipped, stream);
}

sq_status sq_add_rms_smooth_quant_act(const void* x, const void* residual, sq_dtype xt, int64_t T,
                                      int64_t K, const float* gamma_s, float eps,
                                      sq_act_gran gran, void* h, float* act_scale, int8_t* xq,
                                      int64_t* n_clipped, sq_stream stream) {
  const char* fn = "sq_add_rms_smooth_quant_act";
  g_last_error[0] = 0;
  SQ_TRY(check_dtype(xt, fn));
  if (gran != SQ_ACT_PER_TENSOR_STATIC && gran != SQ_ACT_PER_TOKEN_DYNAMIC &&
      gran != SQ_ACT_PER_TENSOR_DYNAMIC)
    return fail(SQ_ERR_INVALID_ARG, "%s: unknown granularity %d", fn, (int)gran);
  if (T < 0) return fail(SQ_ERR_SHAPE, "%s: T=%lld < 0", fn, (long long)T);
  SQ_TRY(check_k(K, fn));
  if (!(eps >= 0.0f && isfinite(eps)))
    return fail(SQ_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", fn);
  if (T == 0) return SQ_OK;
  SQ_REQ(x, fn);
  SQ_REQ(residual, fn);
  SQ_REQ(gamma_s, fn);
  SQ_REQ(h, fn);
  SQ_REQ(act_scale, fn);
  SQ_REQ(xq, fn);
  if (n_clipped && (((uintptr_t)n_clipped) & 7u))
    return fail(SQ_ERR_ALIGN, "%s: n_clipped is not 8-byte aligned", fn);
  const cudaStream_t st = (cudaStream_t)stream;
  AddNormArgs a{};
  a.x = x; a.res = residual; a.h = h; a.T = T; a.K = K; a.g = gamma_s; a.eps = eps;
  a.scale = act_scale; a.q = xq; a.n_clipped = (unsigned long long*)n_clipped;
  cudaError_t e;
  if (gran != SQ_ACT_PER_TENSOR_DYNAMIC) {
    e = launch_addnorm(a, xt, gran == SQ_ACT_PER_TOKEN_DYNAMIC ? ROW_DYNAMIC : ROW_STATIC, st);
  } else {
    // h and the call's peak, the step, then the static quantizer on h
    a.peak = act_scale;
    e = launch_zero(act_scale, sizeof(float), st);
    if (e == cudaSuccess) e = launch_addnorm(a, xt, ROW_PEAK, st);
    if (e == cudaSuccess) e = launch_peak_to_delta(act_scale, st);
    RowArgs q{};
    q.x = h; q.T = T; q.K = K; q.g = gamma_s; q.eps = eps; q.rms = 1;
    q.scale = act_scale; q.q = xq; q.n_clipped = a.n_clipped;
    if (e == cudaSuccess) e = launch_row(q, xt, ROW_STATIC, st);
  }
  return e == cudaSuccess ? SQ_OK : cuda_fail(e, fn);
}

namespace {
constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxWidth = (int64_t)1 << 20;
constexpr int64_t kMaxCoord = (int64_t)1 << 30;

sq_status check_experts(int64_t E, const char* fn) {
  if (E < 1 || E > kMaxExperts)
    return fail(SQ_ERR_SHAPE, "%s: E=%lld must lie in [1, %d]", fn, (long long)E, kMaxExperts);
  return SQ_OK;
}
sq_status check_routing(int64_t T, int64_t top_k, const char* fn) {
  if (T < 0 || T > kMaxRows || top_k < 1 || top_k > kMaxRows || (T && top_k > kMaxRows / T))
    return fail(SQ_ERR_SHAPE, "%s: T=%lld >= 0, top_k=%lld >= 1 and T * top_k < 2^31 are needed",
                fn, (long long)T, (long long)top_k);
  return SQ_OK;
}
// The combine and its gradient step over a token's choices in 32-bit counters,
// up to eight past the last one.
sq_status check_choices(int64_t top_k, const char* fn) {
  if (top_k > kMaxCoord)
    return fail(SQ_ERR_SHAPE, "%s: top_k=%lld must not exceed 2^30", fn, (long long)top_k);
  return SQ_OK;
}
sq_status check_rows(int64_t R, int64_t width, const char* fn) {
  if (R < 0 || R > kMaxRows)
    return fail(SQ_ERR_SHAPE, "%s: R=%lld must lie in [0, 2^31)", fn, (long long)R);
  if (width < 1 || width > kMaxWidth)
    return fail(SQ_ERR_SHAPE, "%s: a row width of %lld is outside [1, 2^20]", fn, (long long)width);
  return SQ_OK;
}
}  // namespace

size_t sq_moe_sort_workspace_bytes(int64_t T, int64_t top_k, int64_t E) {
  if (T <= 0 || top_k < 1 || top_k > kMaxRows / T || E < 1 || E > kMaxExperts) return 0;
  return moe_sort_workspace_bytes(T * top_k, (int)E);
}

sq_status sq_moe_sort(const void* expert_ids, sq_dtype it, int64_t T, int64_t top_k, int64_t E,
                      int32_t* offsets, int32_t* pos, void* workspace, size_t workspace_bytes,
                      sq_stream stream) {
  const char* fn = "sq_moe_sort";
  g_last_error[0] = 0;
  if (it != SQ_I32 && it != SQ_I64)
    return fail(SQ_ERR_DTYPE, "%s: expert ids are int32 or int64, not type %d", fn, (int)it);
  SQ_TRY(check_routing(T, top_k, fn));
  SQ_TRY(check_experts(E, fn));
  SQ_REQ(offsets, fn);
  if (T > 0) {
    SQ_REQ(expert_ids, fn);
    SQ_REQ(pos, fn);
  }
  const size_t need = sq_moe_sort_workspace_bytes(T, top_k, E);
  if (need) {
    if (!workspace || workspace_bytes < need)
      return fail(SQ_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                  workspace ? workspace_bytes : (size_t)0);
    SQ_OPT(workspace, fn);
  }
  const cudaError_t e = launch_moe_sort(expert_ids, it == SQ_I64, T * top_k, (int)E, offsets, pos,
                                        workspace, (cudaStream_t)stream);
  return e == cudaSuccess ? SQ_OK : cuda_fail(e, fn);
}

sq_status sq_moe_gather(const void* x, sq_dtype xt, int64_t T, int64_t K, const float* scale,
                        const int32_t* pos, int64_t top_k, int64_t R, void* xs, float* scale_out,
                        sq_stream stream) {
  const char* fn = "sq_moe_gather";
  g_last_error[0] = 0;
  if (xt != SQ_I8 && xt != SQ_BF16 && xt != SQ_F32)
    return fail(SQ_ERR_DTYPE, "%s: rows are int8, bf16 or fp32, not type %d", fn, (int)xt);
  SQ_TRY(check_routing(T, top_k, fn));
  SQ_TRY(check_rows(R, K, fn));
  if (!scale != !scale_out)
    return fail(SQ_ERR_INVALID_ARG, "%s: pass scale and scale_out together", fn);
  if (T == 0 || R == 0) return SQ_OK;
  SQ_REQ(x, fn);
  SQ_REQ(pos, fn);
  SQ_REQ(xs, fn);
  SQ_OPT(scale, fn);
  SQ_OPT(scale_out, fn);
  MoeArgs a{};
  a.x = x; a.pos = pos; a.scale = scale; a.scale_out = scale_out; a.out = xs;
  a.T = T; a.R = R; a.N = K; a.top_k = (int)top_k;
  const cudaError_t e = launch_moe_gather(a, xt == SQ_I8 ? 1 : xt == SQ_BF16 ? 2 : 4,
                                          (cudaStream_t)stream);
  return e == cudaSuccess ? SQ_OK : cuda_fail(e, fn);
}

sq_status sq_moe_combine(const void* z, sq_dtype t, int64_t R, int64_t N, const int32_t* pos,
                         const float* w, int64_t T, int64_t top_k, const void* residual, void* y,
                         sq_stream stream) {
  const char* fn = "sq_moe_combine";
  g_last_error[0] = 0;
  SQ_TRY(check_dtype(t, fn));
  SQ_TRY(check_routing(T, top_k, fn));
  SQ_TRY(check_choices(top_k, fn));
  SQ_TRY(check_rows(R, N, fn));
  if (T == 0) return SQ_OK;
  if (R > 0) SQ_REQ(z, fn);
  SQ_REQ(pos, fn);
  SQ_OPT(w, fn);
  SQ_OPT(residual, fn);
  SQ_REQ(y, fn);
  MoeArgs a{};
  a.x = z; a.res = residual; a.pos = pos; a.w = w; a.out = y;
  a.T = T; a.R = R; a.N = N; a.top_k = (int)top_k;
  const cudaError_t e = launch_moe_combine(a, t, false, (cudaStream_t)stream);
  return e == cudaSuccess ? SQ_OK : cuda_fail(e, fn);
}

sq_status sq_moe_combine_grad(const void* dy, sq_dtype t, int64_t T, int64_t N, const int32_t* pos,
                              const float* w, int64_t top_k, const void* z, int64_t R, void* dz,
                              float* dw, sq_stream stream) {
  const char* fn = "sq_moe_combine_grad";
  g_last_error[0] = 0;
  SQ_TRY(check_dtype(t, fn));
  SQ_TRY(check_routing(T, top_k, fn));
  SQ_TRY(check_choices(top_k, fn));
  SQ_TRY(check_rows(R, N, fn));
  if (T == 0 || (!dz && !dw)) return SQ_OK;
  SQ_REQ(dy, fn);
  SQ_REQ(pos, fn);
  SQ_OPT(w, fn);
  if (dw && R > 0) SQ_REQ(z, fn);
  SQ_OPT(z, fn);
  SQ_OPT(dz, fn);
  SQ_OPT(dw, fn);
  MoeArgs a{};
  a.x = z; a.res = dy; a.pos = pos; a.w = w; a.out = dz; a.dw = dw;
  a.T = T; a.R = R; a.N = N; a.top_k = (int)top_k;
  const cudaError_t e = launch_moe_combine(a, t, true, (cudaStream_t)stream);
  return e == cudaSuccess ? SQ_OK : cuda_fail(e, fn);
}

sq_status sq_gemm_w8a8_grouped(const int8_t* xq, const int8_t* wq, const int32_t* offsets,
                               int64_t R, int64_t N, int64_t K, int64_t E, const float* act_scale,
                               int act_per_token, const float* w_scale, const float* bias, void* y,
                               sq_dtype yt, int32_t* acc_out, sq_stream stream) {
  const char* fn = "sq_gemm_w8a8_grouped";
  g_last_error[0] = 0;
  SQ_TRY(check_dtype(yt, fn));
  if (R < 0 || N < 0) return fail(SQ_ERR_SHAPE, "%s: R=%lld N=%lld must be >= 0", fn,
                                  (long long)R, (long long)N);
  SQ_TRY(check_k(K, fn));
  SQ_TRY(check_experts(E, fn));
  if (R == 0 || N == 0) return SQ_OK;
  // the kernel's row and channel coordinates run past R and N by a tile
  if (R > kMaxCoord || N > kMaxCoord || (R / 128 + E) > kMaxRows / ((N + 127) / 128))
    return fail(SQ_ERR_SHAPE,
                "%s: R and N must not exceed 2^30, and (R / 128 + E) x (N / 128) must stay below 2^31",
                fn);
  SQ_REQ(xq, fn);
  SQ_REQ(wq, fn);
  SQ_REQ(offsets, fn);
  SQ_REQ(act_scale, fn);
  SQ_REQ(w_scale, fn);
  SQ_OPT(bias, fn);
  SQ_REQ(y, fn);
  SQ_OPT(acc_out, fn);
  GroupArgs a{};
  a.xq = xq; a.wq = wq; a.offsets = offsets; a.R = R; a.N = N; a.K = K; a.E = E;
  a.act_scale = act_scale; a.act_per_token = act_per_token ? 1 : 0;
  a.w_scale = w_scale; a.bias = bias; a.y = y; a.yt = yt; a.acc_out = acc_out;
  return launch_gemm_grouped(a, (cudaStream_t)stream);
}

size_t sq_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0) return 0;
  return gemm_workspace_bytes(M, N, K);
}

namespace {
sq_status gemm_call(const char* fn, const int8_t* xq, const int8_t* wq, int64_t M, int64_t N,
                    int64_t K, const float* act_scale, int act_per_token, const float* w_scale,
                    const float* bias, void* y, sq_dtype yt, int32_t* acc_out, void* workspace,
                    size_t workspace_bytes, sq_stream stream) {
  g_last_error[0] = 0;
  SQ_TRY(check_dtype(yt, fn));
  if (M < 0 || N < 0) return fail(SQ_ERR_SHAPE, "%s: M=%lld N=%lld must be >= 0", fn,
                                  (long long)M, (long long)N);
  SQ_TRY(check_k(K, fn));
  if (M == 0 || N == 0) return SQ_OK;
  if (M > (int64_t)1 << 31 || N > (int64_t)1 << 31)
    return fail(SQ_ERR_SHAPE, "%s: M and N must be below 2^31", fn);
  SQ_REQ(xq, fn);
  SQ_REQ(wq, fn);
  SQ_REQ(act_scale, fn);
  SQ_REQ(w_scale, fn);
  SQ_REQ(y, fn);
  SQ_OPT(acc_out, fn);
  SQ_OPT(bias, fn);
  const size_t need = gemm_workspace_bytes(M, N, K);
  if (need) {
    if (!workspace || workspace_bytes < need)
      return fail(SQ_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                  workspace ? workspace_bytes : (size_t)0);
    SQ_OPT(workspace, fn);
  }
  GemmArgs a{};
  a.xq = xq; a.wq = wq; a.M = M; a.N = N; a.K = K; a.act_scale = act_scale;
  a.act_per_token = act_per_token ? 1 : 0; a.w_scale = w_scale; a.bias = bias; a.y = y;
  a.yt = yt; a.acc_out = acc_out; a.workspace = workspace; a.workspace_bytes = workspace_bytes;
  return launch_gemm(a, (cudaStream_t)stream);
}
}  // namespace

sq_status sq_gemm_w8a8(const int8_t* xq, const int8_t* wq, int64_t M, int64_t N, int64_t K,
                       const float* act_scale, int act_per_token, const float* w_scale, void* y,
                       sq_dtype yt, int32_t* acc_out, void* workspace, size_t workspace_bytes,
                       sq_stream stream) {
  return gemm_call("sq_gemm_w8a8", xq, wq, M, N, K, act_scale, act_per_token, w_scale, nullptr,
                   y, yt, acc_out, workspace, workspace_bytes, stream);
}

sq_status sq_gemm_w8a8_bias(const int8_t* xq, const int8_t* wq, int64_t M, int64_t N, int64_t K,
                            const float* act_scale, int act_per_token, const float* w_scale,
                            const float* bias, void* y, sq_dtype yt, int32_t* acc_out,
                            void* workspace, size_t workspace_bytes, sq_stream stream) {
  return gemm_call("sq_gemm_w8a8_bias", xq, wq, M, N, K, act_scale, act_per_token, w_scale, bias,
                   y, yt, acc_out, workspace, workspace_bytes, stream);
}

sq_status sq_bmm_w8a8(const int8_t* xq, const int8_t* wq, int64_t batch, int64_t M, int64_t N,
                      int64_t K, const float* act_scale, int act_per_token, const float* w_scale,
                      int w_per_channel, void* y, sq_dtype yt, int32_t* acc_out,
                      sq_stream stream) {
  const char* fn = "sq_bmm_w8a8";
  g_last_error[0] = 0;
  SQ_TRY(check_dtype(yt, fn));
  if (batch < 0 || M < 0 || N < 0)
    return fail(SQ_ERR_SHAPE, "%s: batch=%lld M=%lld N=%lld must be >= 0", fn, (long long)batch,
                (long long)M, (long long)N);
  SQ_TRY(check_k(K, fn));
  if (batch == 0 || M == 0 || N == 0) return SQ_OK;
  const int64_t tiles = batch * ((M + 127) / 128) * ((N + 127) / 128);
  if (M > (int64_t)1 << 31 || N > (int64_t)1 << 31 || tiles > ((int64_t)1 << 31) - 1 ||
      batch > ((int64_t)1 << 31) - 1)
    return fail(SQ_ERR_SHAPE, "%s: batch x tiles must stay below 2^31", fn);
  SQ_REQ(xq, fn);
  SQ_REQ(wq, fn);
  SQ_REQ(act_scale, fn);
  SQ_REQ(w_scale, fn);
  SQ_REQ(y, fn);
  SQ_OPT(acc_out, fn);
  BmmArgs a{};
  a.xq = xq; a.wq = wq; a.batch = batch; a.M = M; a.N = N; a.K = K;
  a.act_scale = act_scale; a.act_per_token = act_per_token ? 1 : 0;
  a.w_scale = w_scale; a.w_per_channel = w_per_channel ? 1 : 0;
  a.y = y; a.yt = yt; a.acc_out = acc_out;
  return launch_bmm(a, (cudaStream_t)stream);
}

sq_status sq_gemm_w8a8_noalloc(const int8_t* xq, const int8_t* wq, int64_t M, int64_t N,
                               int64_t K, const float* act_scale, int act_per_token,
                               const float* w_scale, void* y, sq_dtype yt, int32_t* acc_out,
                               sq_stream stream) {
  const char* fn = "sq_gemm_w8a8_noalloc";
  g_last_error[0] = 0;
  SQ_TRY(check_dtype(yt, fn));
  if (M < 0 || N < 0) return fail(SQ_ERR_SHAPE, "%s: M=%lld N=%lld must be >= 0", fn,
                                  (long long)M, (long long)N);
  SQ_TRY(check_k(K, fn));
  if (M == 0 || N == 0) return SQ_OK;
  if (M > (int64_t)1 << 31 || N > (int64_t)1 << 31)
    return fail(SQ_ERR_SHAPE, "%s: M and N must be below 2^31", fn);
  SQ_REQ(xq, fn);
  SQ_REQ(wq, fn);
  SQ_REQ(act_scale, fn);
  SQ_REQ(w_scale, fn);
  SQ_REQ(y, fn);
  SQ_OPT(acc_out, fn);
  GemmArgs a{};
  a.xq = xq; a.wq = wq; a.M = M; a.N = N; a.K = K; a.act_scale = act_scale;
  a.act_per_token = act_per_token ? 1 : 0; a.w_scale = w_scale; a.y = y; a.yt = yt;
  a.acc_out = acc_out;
  return launch_gemm_noalloc(a, (cudaStream_t)stream);
}

namespace {
// Workspace of sq_alpha_sweep, carved in this order (each piece 256-byte
// aligned): wmax, s, inv_s, Delta_A [K|K|K|4] fp32; gamma', beta' [K|K];
// w_scale [N]; act_scale [M]; wq [N,K]; xq [M,K]; y [M,N] fp32 (used only
// when the GEMM cannot fold the error into its epilogue); the error
// reduction's fp64 sums (per block, or per epilogue warp); then the GEMM's
// own workspace.
struct SweepLayout {
  size_t wmax, s, inv_s, dA, g2, b2, ws, act, wq, xq, y, sums, gemm, total;
};
SweepLayout sweep_layout(int64_t M, int64_t N, int64_t K) {
  auto al = [](size_t v) { return (v + 255) & ~(size_t)255; };
  SweepLayout L{};
  size_t o = 0;
  L.wmax = o; o += al(4 * (size_t)K);
  L.s = o; o += al(4 * (size_t)K);
  L.inv_s = o; o += al(4 * (size_t)K);
  L.dA = o; o += al(16);
  L.g2 = o; o += al(4 * (size_t)K);
  L.b2 = o; o += al(4 * (size_t)K);
  L.ws = o; o += al(4 * (size_t)N);
  L.act = o; o += al(4 * (size_t)M);
  L.wq = o; o += al((size_t)N * (size_t)K);
  L.xq = o; o += al((size_t)M * (size_t)K);
  L.y = o; o += al(4 * (size_t)M * (size_t)N);
  const size_t warp_sums = 2 * sizeof(double) * (size_t)gemm_err_max_slots();
  L.sums = o; o += al(std::max(output_error_scratch_bytes(), warp_sums));
  L.gemm = o; o += al(gemm_workspace_bytes(M, N, K));
  L.total = o;
  return L;
}
}  // namespace

size_t sq_alpha_sweep_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0) return 0;
  return sweep_layout(M, N, K).total;
}

sq_status sq_alpha_sweep(const float* amax_x, const void* w, sq_dtype wt, int64_t N, int64_t K,
                         const void* x, sq_dtype xt, int64_t M, const float* ln_gamma,
                         const float* ln_beta, float ln_eps, const float* y_ref,
                         const float* alphas, int n_alpha, sq_act_gran gran, double* err,
                         void* workspace, size_t workspace_bytes, sq_stream stream) {
  const char* fn = "sq_alpha_sweep";
  g_last_error[0] = 0;
  SQ_TRY(check_dtype(wt, fn));
  SQ_TRY(check_dtype(xt, fn));
  if (gran != SQ_ACT_PER_TENSOR_STATIC && gran != SQ_ACT_PER_TOKEN_DYNAMIC &&
      gran != SQ_ACT_PER_TENSOR_DYNAMIC)
    return fail(SQ_ERR_INVALID_ARG, "%s: unknown granularity %d", fn, (int)gran);
  if (M <= 0 || N <= 0) return fail(SQ_ERR_SHAPE, "%s: M=%lld N=%lld must be >= 1", fn,
                                    (long long)M, (long long)N);
  if (M > (int64_t)1 << 31 || N > (int64_t)1 << 31)
    return fail(SQ_ERR_SHAPE, "%s: M and N must be below 2^31", fn);
  SQ_TRY(check_k(K, fn));
  if (n_alpha < 0) return fail(SQ_ERR_INVALID_ARG, "%s: n_alpha=%d < 0", fn, n_alpha);
  if (n_alpha > 0 && !alphas) return fail(SQ_ERR_INVALID_ARG, "%s: alphas is NULL", fn);
  for (int i = 0; i < n_alpha; ++i)
    if (!(alphas[i] >= 0.0f && alphas[i] <= 1.0f))
      return fail(SQ_ERR_INVALID_ARG, "%s: alphas[%d] = %g is not in [0, 1]", fn, i,
                  (double)alphas[i]);
  SQ_REQ(amax_x, fn);
  SQ_REQ(w, fn);
  SQ_REQ(x, fn);
  SQ_REQ(y_ref, fn);
  SQ_REQ(err, fn);
  SQ_OPT(ln_gamma, fn);
  SQ_OPT(ln_beta, fn);
  if (ln_beta && !ln_gamma) return fail(SQ_ERR_INVALID_ARG, "%s: ln_beta given without ln_gamma", fn);
  if (ln_gamma && !(ln_eps >= 0.0f && isfinite(ln_eps)))
    return fail(SQ_ERR_INVALID_ARG, "%s: ln_eps must be finite and >= 0", fn);
  const SweepLayout L = sweep_layout(M, N, K);
  if (!workspace || workspace_bytes < L.total)
    return fail(SQ_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", fn, L.total,
                workspace ? workspace_bytes : (size_t)0);
  SQ_OPT(workspace, fn);
  if (n_alpha == 0) return SQ_OK;
  uint8_t* base = (uint8_t*)workspace;
  float* wmax = (float*)(base + L.wmax);
  float* s = (float*)(base + L.s);
  float* inv_s = (float*)(base + L.inv_s);
  float* dA = (float*)(base + L.dA);
  float* g2 = (float*)(base + L.g2);
  float* b2 = (float*)(base + L.b2);
  float* ws = (float*)(base + L.ws);
  float* act = (float*)(base + L.act);
  int8_t* wq = (int8_t*)(base + L.wq);
  int8_t* xq = (int8_t*)(base + L.xq);
  float* y = (float*)(base + L.y);
  double* sums = (double*)(base + L.sums);
  const cudaStream_t st = (cudaStream_t)stream;
  const bool stat = gran == SQ_ACT_PER_TENSOR_STATIC;
  // the weight column peaks do not depend on alpha
  cudaError_t e = cudaMemsetAsync(wmax, 0, 4 * (size_t)K, st);
  if (e == cudaSuccess) e = launch_colmax(w, wt, N, K, wmax, st);
  for (int i = 0; e == cudaSuccess && i < n_alpha; ++i) {
    // eq. (4) (and the static step) from the two sets of peaks
    e = launch_scales(amax_x, wmax, K, alphas[i], s, inv_s, stat ? dA : nullptr, st);
    // the fold: W * s -> wq, w_scale; gamma / s, beta / s in the same launch
    RowArgs f{};
    f.x = w; f.T = N; f.K = K; f.mul = s; f.scale = ws; f.q = wq;
    if (ln_gamma) {
      f.fold_g = ln_gamma; f.fold_g_out = g2;
      f.fold_b = ln_beta; f.fold_b_out = ln_beta ? b2 : nullptr;
    }
    if (e == cudaSuccess) e = launch_row(f, wt, ROW_DYNAMIC, st);
    // the quantizer
    RowArgs q{};
    q.x = x; q.T = M; q.K = K; q.eps = ln_eps; q.scale = act; q.q = xq;
    if (ln_gamma) {
      q.g = g2;
      q.b = ln_beta ? b2 : nullptr;
    } else {
      q.mul = inv_s;
    }
    if (e == cudaSuccess && stat)
      e = cudaMemcpyAsync(act, dA, sizeof(float), cudaMemcpyDeviceToDevice, st);
    if (e == cudaSuccess) e = run_quant(q, xt, gran, st);
    // the GEMM in fp32 and the error against y_ref: folded into the GEMM's
    // epilogue where the large-M kernel serves the shape (y never written),
    // else y, then a pass over y and y_ref
    GemmArgs g{};
    g.xq = xq; g.wq = wq; g.M = M; g.N = N; g.K = K; g.act_scale = act;
    g.act_per_token = gran == SQ_ACT_PER_TOKEN_DYNAMIC ? 1 : 0; g.w_scale = ws; g.y = y;
    g.yt = SQ_F32; g.workspace = base + L.gemm; g.workspace_bytes = L.total - L.gemm;
    if (e == cudaSuccess && gemm_err_ok(M, N)) {
      int nslots = 0;
      const sq_status gs = launch_gemm_err(g, y_ref, sums, &nslots, st);
      if (gs != SQ_OK) return gs;
      e = launch_output_error_final(sums, nslots, err + i, st);
    } else if (e == cudaSuccess) {
      const sq_status gs = launch_gemm(g, st);
      if (gs != SQ_OK) return gs;
      e = launch_output_error(y, y_ref, M * N, sums, err + i, st);
    }
  }
  return e == cudaSuccess ? SQ_OK : cuda_fail(e, fn);
}

sq_status sq_sync_status(sq_stream stream) {
  g_last_error[0] = 0;
  cudaError_t e = cudaStreamSynchronize((cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "sq_sync_status");
  unsigned int* sw = status_word();
  if (!sw) return fail(SQ_ERR_CUDA, "sq_sync_status: status word unavailable");
  unsigned int v = 0;
  e = cudaMemcpy(&v, sw, sizeof v, cudaMemcpyDeviceToHost);
  if (e == cudaSuccess && v) e = cudaMemset(sw, 0, sizeof v);
  if (e != cudaSuccess) return cuda_fail(e, "sq_sync_status");
  if (v) return fail((sq_status)v, "sq_sync_status: a kernel reported %s",
                     sq_status_string((sq_status)v));
  return SQ_OK;
}

const char* sq_status_string(sq_status s) {
  switch (s) {
    case SQ_OK: return "SQ_OK";
    case SQ_ERR_INVALID_ARG: return "SQ_ERR_INVALID_ARG";
    case SQ_ERR_SHAPE: return "SQ_ERR_SHAPE";
    case SQ_ERR_ALIGN: return "SQ_ERR_ALIGN";
    case SQ_ERR_DTYPE: return "SQ_ERR_DTYPE";
    case SQ_ERR_UNSUPPORTED: return "SQ_ERR_UNSUPPORTED";
    case SQ_ERR_CUDA: return "SQ_ERR_CUDA";
    case SQ_ERR_TIMEOUT: return "SQ_ERR_TIMEOUT";
    case SQ_ERR_WORKSPACE: return "SQ_ERR_WORKSPACE";
    case SQ_ERR_BOUNDS: return "SQ_ERR_BOUNDS";
  }
  return "SQ_ERR_UNKNOWN";
}

const char* sq_last_error(void) { return g_last_error; }

sq_status sq_selftest_bounded_wait(int64_t limit_ns, sq_stream stream) {
  g_last_error[0] = 0;
  if (limit_ns < 1 || limit_ns > 1000000000)
    return fail(SQ_ERR_INVALID_ARG, "sq_selftest_bounded_wait: limit_ns must be in [1, 1e9]");
  cudaError_t e = launch_wait_selftest(limit_ns, (cudaStream_t)stream);
  return e == cudaSuccess ? SQ_OK : cuda_fail(e, "sq_selftest_bounded_wait");
}

int sq_debug_bounds_enabled(void) {
#ifdef SQ_DEBUG_BOUNDS
  return 1;
#else
  return 0;
#endif
}

sq_status sq_selftest_bounds_check(sq_stream stream) {
  g_last_error[0] = 0;
  cudaError_t e = launch_bounds_selftest((cudaStream_t)stream);
  return e == cudaSuccess ? SQ_OK : cuda_fail(e, "sq_selftest_bounds_check");
}

sq_status sq_probe_mma_i8(int64_t kblocks, int grid, sq_stream stream) {
  g_last_error[0] = 0;
  if (kblocks < 1 || kblocks > ((int64_t)1 << 30))
    return fail(SQ_ERR_INVALID_ARG, "sq_probe_mma_i8: kblocks must be in [1, 2^30]");
  if (grid < 1 || grid > 65535)
    return fail(SQ_ERR_INVALID_ARG, "sq_probe_mma_i8: grid must be in [1, 65535]");
  cudaError_t e = launch_mma_probe(kblocks, grid, (cudaStream_t)stream);
  return e == cudaSuccess ? SQ_OK : cuda_fail(e, "sq_probe_mma_i8");
}

sq_status sq_probe_mma_i8_pair(int64_t kblocks, int pairs, sq_stream stream) {
  g_last_error[0] = 0;
  if (kblocks < 1 || kblocks > ((int64_t)1 << 30))
    return fail(SQ_ERR_INVALID_ARG, "sq_probe_mma_i8_pair: kblocks must be in [1, 2^30]");
  if (pairs < 1 || pairs > 32767)
    return fail(SQ_ERR_INVALID_ARG, "sq_probe_mma_i8_pair: pairs must be in [1, 32767]");
  cudaError_t e = launch_mma_pair_probe(kblocks, pairs, (cudaStream_t)stream);
  return e == cudaSuccess ? SQ_OK : cuda_fail(e, "sq_probe_mma_i8_pair");
}

}  // extern "C"
