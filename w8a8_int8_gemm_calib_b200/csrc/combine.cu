// combine.cu -- the experts' rows back to their tokens, and the gradient.
//
//   combine  y[t] = rnd(res[t] + sum_c w[t,c] z[pos[t,c]])
//   grad     dz[pos[t,c]] = rnd(w[t,c] dy[t]),
//            dw[t,c] = sum_n dy[t,n] z[pos[t,c],n]
//
// Both walk the tokens: a token's row is touched once, its top_k rows are
// read (and written), and every sum runs in one fixed order.
//
// Bound: HBM -- top_k + 2 rows a token, 2 top_k + 1 for the gradient.  Rows lie
// anywhere, so what counts is bytes in flight: a thread has eight 16-byte
// loads outstanding, of one token's rows or, with few rows a token, of
// several tokens', and the places of the next step are loaded before the
// rows of this one.  Measured (bf16 rows of 4096, 1965 MHz): 16384 tokens of 8
// rows, with a residual, 199 us (6.7 TB/s; rows in a random order 205), of 2
// rows 86 us; the gradients of 8192 tokens of 8 rows 200 us (5.7 TB/s, half of
// it writes).  So many loads in flight need the clock and the L1: at the 1.1 to
// 1.7 GHz that a power-capped GEMM leaves behind the first takes 220 to 290 us,
// and 236 us right behind a kernel that took all of the SMs' shared memory.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "launch.cuh"
#include "moe.cuh"
#include "sq_device.cuh"
#include "sq_internal.h"

namespace sq {

namespace {

constexpr int kBatch = 8;  // assignments whose rows are in flight together

// A thread's part of a row: U pieces of G bytes (V elements each).  G is 16,
// or what the rows' pitch keeps aligned (4, or a bf16's 2): then four pieces,
// a warp's 32 lanes side by side in each, so that they are at constant offsets
// from the first (c) and cost one address.
template <typename T, int G>
struct Part {
  static constexpr int V = G / (int)sizeof(T);
  static constexpr int U = G == 16 ? 1 : 4;
  static constexpr int E = U * V;
  uint32_t w[G == 16 ? 4 : U];

  // first column of thread `tid` of a block whose first column is c0
  static __device__ __forceinline__ int column(int c0, int tid) {
    return c0 + (tid & ~31) * E + (tid & 31) * V;
  }
  // column of element e of a thread whose first is c
  static __device__ __forceinline__ int column_of(int c, int e) { return c + e / V * 32 * V; }

  __device__ __forceinline__ void load(const T* row, int c, int n) {
    const T* p = row + c;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c + u * 32 * V >= n) continue;
      if constexpr (G == 16) {
        const uint4 q = ld_stream_u4(p);
        w[0] = q.x; w[1] = q.y; w[2] = q.z; w[3] = q.w;
      } else if constexpr (G == 4) {
        w[u] = __ldcg(reinterpret_cast<const unsigned int*>(p + u * 32 * V));
      } else {
        w[u] = __ldcg(reinterpret_cast<const unsigned short*>(p + u * 32 * V));
      }
    }
  }
  __device__ __forceinline__ void get(float (&v)[E]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = __uint_as_float(w[i]);
    } else if constexpr (G == 2) {
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = bf16lo(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        v[2 * i] = bf16lo(w[i]);
        v[2 * i + 1] = bf16hi(w[i]);
      }
    }
  }
  static __device__ __forceinline__ void put(T* row, int c, int n, const float (&v)[E]) {
    uint32_t o[G == 16 ? 4 : U];
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < E; ++i) o[i] = __float_as_uint(v[i]);
    } else if constexpr (G == 2) {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const __nv_bfloat16 h = __float2bfloat16_rn(v[i]);
        o[i] = *reinterpret_cast<const uint16_t*>(&h);
      }
    } else {
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        o[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    T* p = row + c;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c + u * 32 * V >= n) continue;
      if constexpr (G == 16)
        *reinterpret_cast<uint4*>(p) = make_uint4(o[0], o[1], o[2], o[3]);
      else if constexpr (G == 4)
        *reinterpret_cast<uint32_t*>(p + u * 32 * V) = o[u];
      else
        *reinterpret_cast<uint16_t*>(p + u * 32 * V) = (uint16_t)o[u];
    }
  }
};

// In a bounds-checked build: the row lies in a tensor of `rows` rows.
__device__ __forceinline__ bool row_ok(const MoeArgs& a, int64_t row, int64_t rows) {
  return in_bounds(row * a.N, a.N, rows * a.N, a.status);
}

// P tokens a step, their first kBatch / P assignments each: P may be 4 for
// top_k up to 2, 2 up to 4, else it is 1, with as many steps of 8 as top_k
// takes.  Lane b of every warp holds the place and weight of the step's
// assignment b.
template <int P>
struct Step {
  static constexpr int KK = kBatch / P;
  int row;
  float wt;
  __device__ __forceinline__ void fetch(const MoeArgs& a, int64_t t0, int k0, int lane) {
    const int b = lane & (kBatch - 1);
    const int64_t t = t0 + b / KK;
    const int k = t < a.T ? k0 + b % KK : a.top_k;
    wt = a.w && k < a.top_k ? __ldcg(a.w + t * a.top_k + k) : 1.0f;
    row = (int)place(a, t, k);
  }
};

// Resident blocks per SM (registers: 64 a thread, 80 with several tokens a
// step).  16384 x 8 rows of 4096 bf16 are combined in 230 / 204 / 277 us with
// 3 / 4 / 5 blocks; the gradients of 8192 x 8 rows take 194 / 201 / 217 us, of
// 1024 x 4 17.7 us with 3 and 15.4 with 4.
template <int P>
constexpr int kBlocks = P == 1 ? 4 : 3;

template <typename T, int G, int P>
__global__ void __launch_bounds__(kRowThreads, kBlocks<P>) combine_kernel(const MoeArgs a) {
  using L = Part<T, G>;
  constexpr int KK = Step<P>::KK;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, n = (int)a.N;
  const int c = L::column((int)(blockIdx.y * blockDim.x) * L::E, threadIdx.x);
  const T* z = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.res);
  T* y = static_cast<T*>(a.out);
  Step<P> next;
  next.fetch(a, (int64_t)blockIdx.x * P, 0, lane);
  for (int64_t t0 = (int64_t)blockIdx.x * P; t0 < a.T; t0 += (int64_t)gridDim.x * P) {
    L rs[P];
    float acc[L::E];
    for (int k0 = 0; k0 < a.top_k; k0 += KK) {
      const Step<P> now = next;
      if (k0 + KK < a.top_k) next.fetch(a, t0, k0 + KK, lane);
      else next.fetch(a, t0 + (int64_t)gridDim.x * P, 0, lane);
      L raw[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int r = __shfl_sync(0xffffffffu, now.row, b);
        if (r >= 0 && row_ok(a, r, a.R)) raw[b].load(z + r * a.N, c, n);
      }
      if (k0 == 0) {
#pragma unroll
        for (int p = 0; p < P; ++p)
          if (res && t0 + p < a.T && row_ok(a, t0 + p, a.T)) rs[p].load(res + (t0 + p) * a.N, c, n);
      }
#pragma unroll
      for (int p = 0; p < P; ++p) {
        if (k0 == 0) {
          if (res) {
            rs[p].get(acc);
          } else {
#pragma unroll
            for (int e = 0; e < L::E; ++e) acc[e] = 0.0f;
          }
        }
#pragma unroll
        for (int b = p * KK; b < (p + 1) * KK; ++b) {
          const int r = __shfl_sync(0xffffffffu, now.row, b);
          const float wt = __shfl_sync(0xffffffffu, now.wt, b);
          if (r < 0) continue;
          float v[L::E];
          raw[b].get(v);
          if (a.w) {
#pragma unroll
            for (int e = 0; e < L::E; ++e) acc[e] = __fmaf_rn(wt, v[e], acc[e]);
          } else {
#pragma unroll
            for (int e = 0; e < L::E; ++e) acc[e] = __fadd_rn(acc[e], v[e]);
          }
        }
        if (k0 + KK >= a.top_k && t0 + p < a.T && row_ok(a, t0 + p, a.T))
          L::put(y + (t0 + p) * a.N, c, n, acc);
      }
    }
  }
}

// Eight sums over 32 lanes: in the first three steps a lane passes on the half
// of its sums that the other lane keeps, so 9 shuffles do instead of 40; the
// sum of b ends in lanes 4 b .. 4 b + 3.
__device__ __forceinline__ float lanes_sum8(float (&v)[kBatch], int lane) {
#pragma unroll
  for (int s = 4; s >= 1; s >>= 1) {
    const int o = s * 4;  // 16, 8, 4
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < s; ++i) {
      const float give = up ? v[i] : v[i + s], keep = up ? v[i + s] : v[i];
      v[i] = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, give, o));
    }
  }
  const float r = __fadd_rn(v[0], __shfl_xor_sync(0xffffffffu, v[0], 2));
  return __fadd_rn(r, __shfl_xor_sync(0xffffffffu, r, 1));
}

// A block has whole rows.  Each thread adds its columns' products in
// increasing column, then lanes and warps are combined: one fixed order, fp32.
template <typename T, int G, int P>
__global__ void __launch_bounds__(kRowThreads, kBlocks<P>) combine_grad_kernel(const MoeArgs a) {
  using L = Part<T, G>;
  constexpr int KK = Step<P>::KK;
  __shared__ float part[2][kRowThreads / 32][kBatch];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nt = blockDim.x, n = (int)a.N;
  const T* dy = static_cast<const T*>(a.res);
  const T* z = static_cast<const T*>(a.x);
  T* dz = static_cast<T*>(a.out);
  const bool want_w = a.dw != nullptr;
  int parity = 0;
  Step<P> next;
  next.fetch(a, (int64_t)blockIdx.x * P, 0, lane);
  for (int64_t t0 = (int64_t)blockIdx.x * P; t0 < a.T; t0 += (int64_t)gridDim.x * P) {
    for (int k0 = 0; k0 < a.top_k; k0 += KK) {
      const Step<P> now = next;
      if (k0 + KK < a.top_k) next.fetch(a, t0, k0 + KK, lane);
      else next.fetch(a, t0 + (int64_t)gridDim.x * P, 0, lane);
      float dot[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) dot[b] = 0.0f;
      // whole warps run every step (the places are passed by shuffle)
      for (int c0 = 0; c0 < n; c0 += nt * L::E) {  // n <= 2^20
        const int c = L::column(c0, threadIdx.x);
        L dr[P], zr[kBatch];
#pragma unroll
        for (int p = 0; p < P; ++p)
          if (t0 + p < a.T && row_ok(a, t0 + p, a.T)) dr[p].load(dy + (t0 + p) * a.N, c, n);
        if (want_w) {
#pragma unroll
          for (int b = 0; b < kBatch; ++b) {
            const int r = __shfl_sync(0xffffffffu, now.row, b);
            if (r >= 0 && row_ok(a, r, a.R)) zr[b].load(z + r * a.N, c, n);
          }
        }
#pragma unroll
        for (int p = 0; p < P; ++p) {
          float d[L::E];
          dr[p].get(d);
#pragma unroll
          for (int b = p * KK; b < (p + 1) * KK; ++b) {
            const int r = __shfl_sync(0xffffffffu, now.row, b);
            const float wt = __shfl_sync(0xffffffffu, now.wt, b);
            if (r < 0) continue;
            float v[L::E];
            if (want_w) {
              zr[b].get(v);
#pragma unroll
              for (int e = 0; e < L::E; ++e)
                if (L::column_of(c, e) < n) dot[b] = __fmaf_rn(d[e], v[e], dot[b]);
            }
            if (dz && row_ok(a, r, a.R)) {
#pragma unroll
              for (int e = 0; e < L::E; ++e) v[e] = __fmul_rn(wt, d[e]);
              L::put(dz + r * a.N, c, n, v);
            }
          }
        }
      }
      if (!want_w) continue;
      const float s8 = lanes_sum8(dot, lane);
      if ((lane & 3) == 0) part[parity][warp][lane >> 2] = s8;
      __syncthreads();
      if (threadIdx.x < kBatch) {
        const int b = threadIdx.x, k = k0 + b % KK;
        const int64_t t = t0 + b / KK;
        if (t < a.T && k < a.top_k && in_bounds(t * a.top_k + k, 1, a.T * a.top_k, a.status)) {
          float s = 0.0f;
          for (int w = 0; w < (nt >> 5); ++w) s = __fadd_rn(s, part[parity][w][b]);
          a.dw[t * a.top_k + k] = s;
        }
      }
      parity ^= 1;  // the next step's sums do not wait for these reads
    }
  }
}

// Threads per block, blocks across a row, blocks that are resident at once,
// those of them that walk the tokens side by side and the steps over the
// tokens, for P tokens a step.
struct Plan {
  unsigned nt;
  int64_t segs, resident, walk, steps;
};
template <typename T, int G, int P>
Plan plan(const MoeArgs& a, bool grad) {
  Plan q;
  const int64_t pieces = (a.N + Part<T, G>::E - 1) / Part<T, G>::E;  // threads that cover a row
  q.nt = row_threads(pieces);
  q.segs = grad ? 1 : (pieces + q.nt - 1) / q.nt;
  q.resident = kBlocks<P> * (int64_t)sm_count() * (kRowThreads / q.nt);
  q.walk = (q.resident + q.segs - 1) / q.segs;
  q.steps = (a.T + P - 1) / P;
  return q;
}

template <typename T, int G, int P>
cudaError_t launch_gp(const MoeArgs& a, bool grad, cudaStream_t st) {
  const Plan q = plan<T, G, P>(a, grad);
  const dim3 grid((unsigned)(q.walk < q.steps ? q.walk : q.steps), (unsigned)q.segs);
  return grad ? launch_pdl(combine_grad_kernel<T, G, P>, grid, dim3(q.nt), 0, st, a)
              : launch_pdl(combine_kernel<T, G, P>, grid, dim3(q.nt), 0, st, a);
}

// Four tokens a step (top_k up to 2) where the steps still occupy half the
// blocks that fit.  us with 1 / 2 / 4 tokens a step, rows of 4096 bf16:
//   combine    512 x 2: 5.0 / 4.9 / 4.2    1024 x 1: 9.3 / 8.3 / 7.6
//              8192 x 2: 62.5 / 53.1 / 46.7
//   gradients  512 x 2: 5.1 / 5.8 / 7.7    1024 x 2: 11.1 / 12.5 / 10.7
//              8192 x 2: 65.8 / 60.2 / 59.0
// (512 x 2 is 128 steps for 444 blocks; the combine has two blocks on a row.)
//
// Else two (top_k up to 4) where the blocks then walk fewer rounds over the
// tokens, the gradients of 4 choices only where that is a single round.  us
// with 1 / 2 tokens a step, 4 choices:
//   combine    512: 6.6 / 7.4 (2 rounds both)   768: 10.0 / 9.6 (3 and 2)
//              8192: 73.9 / 66.9
//   gradients  512: 8.8 / 10.0 (1 both)   768: 13.8 / 12.2 (2 and 1)   1024:
//              15.4 / 18.4 (2 both)   8192: 96.5 / 104.7 (14 and 10); of 3
//              choices 8192: 80.3 / 77.1
template <typename T, int G, int P>
bool fills_half(const MoeArgs& a, bool grad) {
  const Plan q = plan<T, G, P>(a, grad);
  return 2 * q.steps * q.segs >= q.resident;
}
template <typename T, int G, int P>
int64_t rounds(const MoeArgs& a, bool grad) {
  const Plan q = plan<T, G, P>(a, grad);
  return (q.steps + q.walk - 1) / q.walk;
}
template <typename T, int G>
cudaError_t launch_g(const MoeArgs& a, bool grad, cudaStream_t st) {
  if (a.top_k <= Step<4>::KK && fills_half<T, G, 4>(a, grad))
    return launch_gp<T, G, 4>(a, grad, st);
  if (a.top_k <= Step<2>::KK) {
    const int64_t two = rounds<T, G, 2>(a, grad);
    if (two < rounds<T, G, 1>(a, grad) && (!grad || a.top_k < Step<2>::KK || two == 1))
      return launch_gp<T, G, 2>(a, grad, st);
  }
  return launch_gp<T, G, 1>(a, grad, st);
}

}  // namespace

cudaError_t launch_moe_combine(MoeArgs a, sq_dtype t, bool grad, cudaStream_t st) {
  a.status = status_word();
  if (!a.status) return cudaErrorInvalidDevice;
  if (t == SQ_BF16)
    return a.N % 8 == 0   ? launch_g<uint16_t, 16>(a, grad, st)
           : a.N % 2 == 0 ? launch_g<uint16_t, 4>(a, grad, st)
                          : launch_g<uint16_t, 2>(a, grad, st);
  return a.N % 4 == 0 ? launch_g<float, 16>(a, grad, st) : launch_g<float, 4>(a, grad, st);
}

}  // namespace sq
