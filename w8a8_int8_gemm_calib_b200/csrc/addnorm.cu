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
// Measured at 1965 MHz: 16384 x 8192 bf16 157 us per token (6.0 TB/s) and 171
// us with a static step, 2048 x 4096 per token 15 us, 1 x 4096 2.7 us; wider
// rows read h and gamma twice from L2: 4096 x 16384 per token 133 us (3.5 TB/s).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "launch.cuh"
#include "sq_device.cuh"
#include "sq_internal.h"

namespace sq {

namespace {

constexpr int kSlice = 128;  // threads per row: the 128 reduction slots

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
// storage form, its gamma in shared memory, and the next row's x and r are
// loaded while this row is reduced and quantized.  CM == 0, wider rows: h is
// read back from L2, each chunk by the thread that wrote it (h in shared
// memory instead measured no faster: fewer rows share an SM).
//
// A CTA is one 128-thread slice, so rows in different phases share an SM.
template <typename T, int CM, int MODE>
__global__ void __launch_bounds__(kSlice) addnorm_kernel(const AddNormArgs a) {
  __shared__ float red[2][2][4];  // [row parity][reduction][warp]
  extern __shared__ __align__(16) float gs[];  // CM > 0: gamma, [2 CM][128] float4
  pdl_launch_dependents();
  pdl_wait();
  const int j = threadIdx.x, w = j >> 5, lane = j & 31;
  const int64_t K = a.K, nchunk = K >> 3, size = a.T * a.K;
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.res);
  T* hp = static_cast<T*>(a.h);
  const float kf = (float)K;
  unsigned clipped = 0;
  float peak = 0.0f;

  constexpr int C = CM > 0 ? CM : 1;
  Raw8<T> xv[C], rv[C], h[C];
  auto load_rows = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < CM; ++i) {
      const int64_t c = j + i * kSlice, o = row * K + c * 8;
      if (c < nchunk && row < a.T && in_bounds(o, 8, size, a.status)) {
        load_raw(x + o, xv[i]);
        load_raw(res + o, rv[i]);
      }
    }
  };
  if constexpr (CM > 0) {
    load_rows(blockIdx.x);
    // the thread's own chunks of gamma: written and read by it alone
#pragma unroll
    for (int i = 0; i < CM; ++i) {
      const int64_t c = j + i * kSlice;
      if (c < nchunk) {
        float4* d = reinterpret_cast<float4*>(gs) + 2 * i * kSlice + j;
        d[0] = __ldcg(reinterpret_cast<const float4*>(a.g + c * 8));
        d[kSlice] = __ldcg(reinterpret_cast<const float4*>(a.g + c * 8) + 1);
      }
    }
  }
  const float static_inv = MODE == ROW_STATIC ? __fdiv_rn(1.0f, __ldcg(a.scale)) : 0.0f;

  int parity = 0;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, parity ^= 1) {
    const int64_t base = row * K;
    float p = 0.0f;
    // h = x + r, stored, and its sum of squares
    auto first = [&](int64_t c, const Raw8<T>& xc, const Raw8<T>& rc, Raw8<T>& hc) {
      add_chunk(xc, rc, hc);
      if (in_bounds(base + c * 8, 8, size, a.status)) store_chunk(hp + base + c * 8, hc);
      float v[8];
      unpack(hc, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) p = __fmaf_rn(v[e], v[e], p);
    };
    if constexpr (CM > 0) {
#pragma unroll
      for (int i = 0; i < CM; ++i) {
        const int64_t c = j + i * kSlice;
        if (c < nchunk) first(c, xv[i], rv[i], h[i]);
      }
      load_rows(row + gridDim.x);
    } else {
      constexpr int U = sizeof(T) == 2 ? 4 : 2;  // 128 bytes a thread in flight
      for (int64_t c0 = j; c0 < nchunk; c0 += U * kSlice) {
        Raw8<T> xc[U], rc[U], hc;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int64_t c = c0 + u * kSlice;
          if (c < nchunk && in_bounds(base + c * 8, 8, size, a.status)) {
            load_raw(x + base + c * 8, xc[u]);
            load_raw(res + base + c * 8, rc[u]);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int64_t c = c0 + u * kSlice;
          if (c < nchunk) first(c, xc[u], rc[u], hc);
        }
      }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) p = __fadd_rn(p, __shfl_xor_sync(0xffffffffu, p, o));
    float (&rd)[2][4] = red[parity];  // read before the next row's barriers
    if (lane == 0) rd[0][w] = p;
    __syncthreads();
    const float ss = __fadd_rn(__fadd_rn(rd[0][0], rd[0][2]), __fadd_rn(rd[0][1], rd[0][3]));
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, kf), a.eps)));

    // f(c, y[8]) over the thread's chunks
    auto each_y = [&](auto&& f) {
      auto lift = [&](int64_t c, const Raw8<T>& hc, const float (&g)[8]) {
        float v[8];
        unpack(hc, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __fmul_rn(__fmul_rn(v[e], rstd), g[e]);
        f(c, v);
      };
      float g[8];
      if constexpr (CM > 0) {
#pragma unroll
        for (int i = 0; i < CM; ++i) {
          const int64_t c = j + i * kSlice;
          if (c < nchunk) {
            const float4* s = reinterpret_cast<const float4*>(gs) + 2 * i * kSlice + j;
            const float4 u = s[0], v = s[kSlice];
            g[0] = u.x; g[1] = u.y; g[2] = u.z; g[3] = u.w;
            g[4] = v.x; g[5] = v.y; g[6] = v.z; g[7] = v.w;
            lift(c, h[i], g);
          }
        }
      } else {
#pragma unroll 4
        for (int64_t c = j; c < nchunk; c += kSlice) {
          Raw8<T> hc{};
          if (in_bounds(base + c * 8, 8, size, a.status)) load_raw_cached(hp + base + c * 8, hc);
          load8(a.g + c * 8, g);
          lift(c, hc, g);
        }
      }
    };
    float inv = static_inv;
    if constexpr (MODE == ROW_PEAK) {
      each_y([&](int64_t, const float (&y)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) peak = fmaxf(peak, fabsf(y[e]));
      });
    } else {
      if constexpr (MODE == ROW_DYNAMIC) {
        float m = 0.0f;  // fmaxf: NaN elements are skipped
        each_y([&](int64_t, const float (&y)[8]) {
#pragma unroll
          for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(y[e]));
        });
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane == 0) rd[1][w] = m;
        __syncthreads();
        m = fmaxf(fmaxf(rd[1][0], rd[1][2]), fmaxf(rd[1][1], rd[1][3]));
        const float delta = __fdiv_rn(fmaxf(m, 1e-7f), 127.0f);
        inv = __fdiv_rn(1.0f, delta);
        if (j == 0 && in_bounds(row, 1, a.T, a.status)) a.scale[row] = delta;
      }
      const bool count = a.n_clipped != nullptr;
      each_y([&](int64_t c, const float (&y)[8]) {
        uint32_t b[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) b[e] = qbits(y[e], inv, count, clipped);
        if (in_bounds(base + c * 8, 8, size, a.status)) store_codes(a.q + base + c * 8, b);
      });
    }
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

// As many CTAs as are resident at once walk the rows.
template <typename T, int CM, int MODE>
cudaError_t launch_t(const AddNormArgs& a, cudaStream_t st) {
  auto kern = addnorm_kernel<T, CM, MODE>;
  constexpr size_t smem = (size_t)CM * 8 * kSlice * sizeof(float);
  static std::once_flag once[64];
  static cudaError_t err[64];
  static int per_sm[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 64) return e != cudaSuccess ? e : cudaErrorInvalidDevice;
  std::call_once(once[dev], [&] {
    err[dev] = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm[dev], kern, kSlice, smem);
  });
  if (err[dev] != cudaSuccess) return err[dev];
  int64_t grid = (int64_t)per_sm[dev] * sm_count();
  if (grid < 1) return cudaErrorInvalidConfiguration;
  if (grid > a.T) grid = a.T;
  return launch_pdl(kern, dim3((unsigned)grid), dim3(kSlice), smem, st, a);
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
