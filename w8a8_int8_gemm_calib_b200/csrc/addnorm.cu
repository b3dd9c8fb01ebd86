// addnorm.cu -- the runtime quantizer of a residual network's pre-norm
// linear: h = x + residual, RMSNorm(h; gamma / s), symmetric INT8 codes.
//
//   h[t,k]  = rnd(x[t,k] + r[t,k])                    (rnd: to the type of x)
//   ms_t    = mean_k h[t,k]^2,  rstd_t = 1 / sqrt(ms_t + eps)
//   y[t,k]  = (h[t,k] * rstd_t) * g[k]
//   q[t,k]  = Q(y[t,k]; Delta),  Delta per token, or one step for the call
//
// Every operation after the addition is the RMSNorm quantizer's of
// rowops.cu / rowpipe.cu in the same order, so the codes, steps and clip
// counts equal those of that quantizer on the stored h bit for bit.
//
// The reduction order is the library's: slot j = 32*w + l (warp w of four,
// lane l) owns the 8-element chunks c = j, j + 128, ... and adds h^2 with one
// fused multiply-add per element in increasing k; a butterfly combines the
// 32 lanes, and the warps are combined as (r0 + r2) + (r1 + r3).
//
// Bound: HBM.  The call reads 2 and writes 1 value of x's type per element,
// and writes one code byte (7 bytes for bf16).  Done as an addition and the
// quantizer, h makes one more trip (9 bytes) and there is one more launch.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "launch.cuh"
#include "sq_device.cuh"
#include "sq_internal.h"

namespace sq {

namespace {

constexpr int kSlice = 128;  // threads per row: the 128 reduction slots
constexpr int kSlices = 4;   // rows a CTA works on at a time
constexpr int kThreads = kSlice * kSlices;

__device__ __forceinline__ void slice_bar(int slice) {
  asm volatile("bar.sync %0, %1;" ::"r"(slice + 1), "r"(kSlice) : "memory");
}

// h = x + r of one chunk, rounded to the storage type and packed in it.
__device__ __forceinline__ void add_chunk(const Raw8<float>& x, const Raw8<float>& r,
                                          Raw8<float>& h) {
  h.a = make_float4(__fadd_rn(x.a.x, r.a.x), __fadd_rn(x.a.y, r.a.y), __fadd_rn(x.a.z, r.a.z),
                    __fadd_rn(x.a.w, r.a.w));
  h.b = make_float4(__fadd_rn(x.b.x, r.b.x), __fadd_rn(x.b.y, r.b.y), __fadd_rn(x.b.z, r.b.z),
                    __fadd_rn(x.b.w, r.b.w));
}
__device__ __forceinline__ uint32_t add_pair(uint32_t x, uint32_t r) {
  __nv_bfloat162 t = __floats2bfloat162_rn(__fadd_rn(bf16lo(x), bf16lo(r)),
                                           __fadd_rn(bf16hi(x), bf16hi(r)));
  return *reinterpret_cast<uint32_t*>(&t);
}
__device__ __forceinline__ void add_chunk(const Raw8<uint16_t>& x, const Raw8<uint16_t>& r,
                                          Raw8<uint16_t>& h) {
  h.a = make_uint4(add_pair(x.a.x, r.a.x), add_pair(x.a.y, r.a.y), add_pair(x.a.z, r.a.z),
                   add_pair(x.a.w, r.a.w));
}
__device__ __forceinline__ void store_chunk(float* p, const Raw8<float>& h) {
  reinterpret_cast<float4*>(p)[0] = h.a;
  reinterpret_cast<float4*>(p)[1] = h.b;
}
__device__ __forceinline__ void store_chunk(uint16_t* p, const Raw8<uint16_t>& h) {
  *reinterpret_cast<uint4*>(p) = h.a;
}

// CM > 0: a thread's chunks of h (at most CM) stay in registers in their
// storage form.  CM == 0: h is read back from global memory, each chunk by
// the thread that wrote it.
template <typename T, int CM, int MODE>
__global__ void __launch_bounds__(kThreads) addnorm_kernel(const AddNormArgs a) {
  __shared__ float red[kSlices][2][4];
  pdl_launch_dependents();
  pdl_wait();
  const int slice = threadIdx.x / kSlice, j = threadIdx.x % kSlice;
  const int w = j >> 5, lane = j & 31;
  const int64_t K = a.K, nchunk = K >> 3, size = a.T * a.K;
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.res);
  T* hp = static_cast<T*>(a.h);
  const float kf = (float)K;
  const float static_inv = MODE == ROW_STATIC ? __fdiv_rn(1.0f, __ldcg(a.scale)) : 0.0f;
  unsigned clipped = 0;
  float peak = 0.0f;

  for (int64_t row = blockIdx.x + (int64_t)slice * gridDim.x; row < a.T;
       row += (int64_t)gridDim.x * kSlices) {
    const int64_t base = row * K;
    Raw8<T> h[CM > 0 ? CM : 1];
    float p = 0.0f;
    // h = x + r, stored, and its sum of squares
    auto first = [&](int64_t c, const Raw8<T>& xv, const Raw8<T>& rv, Raw8<T>& hv) {
      add_chunk(xv, rv, hv);
      if (in_bounds(base + c * 8, 8, size, a.status)) store_chunk(hp + base + c * 8, hv);
      float v[8];
      unpack(hv, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) p = __fmaf_rn(v[e], v[e], p);
    };
    if constexpr (CM > 0) {
      Raw8<T> xv[CM], rv[CM];
#pragma unroll
      for (int i = 0; i < CM; ++i) {
        const int64_t c = j + (int64_t)i * kSlice;
        if (c < nchunk && in_bounds(base + c * 8, 8, size, a.status)) {
          load_raw(x + base + c * 8, xv[i]);
          load_raw(res + base + c * 8, rv[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < CM; ++i) {
        const int64_t c = j + (int64_t)i * kSlice;
        if (c < nchunk) first(c, xv[i], rv[i], h[i]);
      }
    } else {
      for (int64_t c = j; c < nchunk; c += kSlice) {
        Raw8<T> xv{}, rv{}, hv;
        if (in_bounds(base + c * 8, 8, size, a.status)) {
          load_raw(x + base + c * 8, xv);
          load_raw(res + base + c * 8, rv);
        }
        first(c, xv, rv, hv);
      }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) p = __fadd_rn(p, __shfl_xor_sync(0xffffffffu, p, o));
    if (lane == 0) red[slice][0][w] = p;
    slice_bar(slice);
    const float ss = __fadd_rn(__fadd_rn(red[slice][0][0], red[slice][0][2]),
                               __fadd_rn(red[slice][0][1], red[slice][0][3]));
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, kf), a.eps)));

    // f(c, y[8]) over the thread's chunks
    auto each_y = [&](auto&& f) {
      auto lift = [&](int64_t c, const Raw8<T>& hv) {
        float v[8], g[8];
        unpack(hv, v);
        load8(a.g + c * 8, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __fmul_rn(__fmul_rn(v[e], rstd), g[e]);
        f(c, v);
      };
      if constexpr (CM > 0) {
#pragma unroll
        for (int i = 0; i < CM; ++i) {
          const int64_t c = j + (int64_t)i * kSlice;
          if (c < nchunk) lift(c, h[i]);
        }
      } else {
        for (int64_t c = j; c < nchunk; c += kSlice) {
          Raw8<T> hv{};
          if (in_bounds(base + c * 8, 8, size, a.status)) load_raw_cached(hp + base + c * 8, hv);
          lift(c, hv);
        }
      }
    };
    float inv = static_inv;
    if constexpr (MODE == ROW_PEAK) {
      each_y([&](int64_t, const float (&y)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) peak = fmaxf(peak, fabsf(y[e]));
      });
      slice_bar(slice);  // red is read by all before the next row writes it
      continue;
    }
    if constexpr (MODE == ROW_DYNAMIC) {
      float m = 0.0f;  // fmaxf: NaN elements are skipped
      each_y([&](int64_t, const float (&y)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(y[e]));
      });
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (lane == 0) red[slice][1][w] = m;
      slice_bar(slice);
      m = fmaxf(fmaxf(red[slice][1][0], red[slice][1][2]),
                fmaxf(red[slice][1][1], red[slice][1][3]));
      const float delta = __fdiv_rn(fmaxf(m, 1e-7f), 127.0f);
      inv = __fdiv_rn(1.0f, delta);
      if (j == 0 && in_bounds(row, 1, a.T, a.status)) a.scale[row] = delta;
    } else {
      slice_bar(slice);
    }
    const bool count = a.n_clipped != nullptr;
    each_y([&](int64_t c, const float (&y)[8]) {
      uint32_t b[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) b[e] = qbits(y[e], inv, count, clipped);
      if (in_bounds(base + c * 8, 8, size, a.status)) store_codes(a.q + base + c * 8, b);
    });
  }
  if constexpr (MODE == ROW_PEAK) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, o));
    if (lane == 0) atomicMax(reinterpret_cast<unsigned int*>(a.peak), __float_as_uint(peak));
  } else if (a.n_clipped) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) clipped += __shfl_xor_sync(0xffffffffu, clipped, o);
    if (lane == 0 && clipped) atomicAdd(a.n_clipped, (unsigned long long)clipped);
  }
}

template <typename T, int CM, int MODE>
cudaError_t launch_t(const AddNormArgs& a, cudaStream_t st) {
  int64_t grid = 4 * (int64_t)sm_count();
  if (grid > a.T) grid = a.T;
  return launch_pdl(addnorm_kernel<T, CM, MODE>, dim3((unsigned)grid), dim3(kThreads), 0, st, a);
}

template <typename T, int MODE>
cudaError_t launch_cm(const AddNormArgs& a, cudaStream_t st) {
  const int64_t per = (a.K / 8 + kSlice - 1) / kSlice;  // chunks per thread
  if (per <= 2) return launch_t<T, 2, MODE>(a, st);
  if (per <= 4) return launch_t<T, 4, MODE>(a, st);
  if constexpr (sizeof(T) == 2) {
    if (per <= 8) return launch_t<T, 8, MODE>(a, st);
  }
  return launch_t<T, 0, MODE>(a, st);
}

}  // namespace

cudaError_t launch_addnorm(AddNormArgs a, sq_dtype xt, RowMode mode, cudaStream_t st) {
  a.status = status_word();
  if (!a.status) return cudaErrorInvalidDevice;
  const bool bf16 = xt == SQ_BF16;
  switch (mode) {
    case ROW_DYNAMIC:
      return bf16 ? launch_cm<uint16_t, ROW_DYNAMIC>(a, st) : launch_cm<float, ROW_DYNAMIC>(a, st);
    case ROW_STATIC:
      return bf16 ? launch_cm<uint16_t, ROW_STATIC>(a, st) : launch_cm<float, ROW_STATIC>(a, st);
    case ROW_PEAK:
      return bf16 ? launch_cm<uint16_t, ROW_PEAK>(a, st) : launch_cm<float, ROW_PEAK>(a, st);
    default:
      return cudaErrorInvalidValue;
  }
}

}  // namespace sq
