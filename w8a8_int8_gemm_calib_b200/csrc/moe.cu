// moe.cu -- tokens sorted by expert, and their codes copied to the sorted
// rows: the way to a W8A8 linear whose weights are experts chosen per token.
//
//   sort     offsets[e] = #{i : id_i < e},  pos_i = offsets[id_i] +
//            #{j < i : id_j = id_i}   over the live assignments i = (t, c)
//   gather   xs[pos_i] = x[t]  (and its step)
//
// Places are indexed by token: a token's row is read once and its top_k
// copies are written, and neither this nor the way back (combine.cu) needs
// the inverse order.
//
// Bound: the gather by HBM; the sort moves 12 bytes per assignment and is
// bound by its launches.
#include <cuda_runtime.h>
#include <stdint.h>

#include "launch.cuh"
#include "moe.cuh"
#include "sq_device.cuh"
#include "sq_internal.h"

namespace sq {

namespace {

// ====================================================================== sort
// A stable counting sort.  The assignments are cut into one contiguous part
// per block and, within it, one contiguous run per warp.  A warp counts its
// run by expert; an assignment's place is then the expert's offset, plus the
// counts of the parts and runs before it, plus its rank in the run, which
// the warp finds 32 assignments at a time by matching equal experts.  Counts
// are integers, so the order the atomics run in changes nothing.
//
// W warps per block: 32 when there is work for them and their counts fit
// (E <= 256), else 8.  A warp takes 64 / W steps of 32 assignments at once,
// so one block holds 2048 either way.  32 assignments over 8 experts take
// 2.3 us with 8 warps and 3.2 with 32, 16384 over 64 experts 9.2 and 7.2;
// 131072 over 64 experts take 7.8 us.
constexpr int kSortItems = 2048;
constexpr int kSortWide = 256;   // experts
constexpr int kSortFew = 512;    // assignments that 8 warps place as fast

struct SortArgs {
  const void* ids;
  int ids64;
  int64_t n, part;  // assignments, and those of a block (a multiple of 32 W)
  int E, blocks;
  int32_t* offsets;
  int32_t* pos;
  int32_t* counts;  // [blocks][E], when there are several blocks
  unsigned int* status;
};

// expert of assignment i, or E when it goes to none
__device__ __forceinline__ int expert_of(const SortArgs& a, int64_t i) {
  if (!in_bounds(i, 1, a.n, a.status)) return a.E;
  const int64_t id = a.ids64 ? __ldcg(static_cast<const long long*>(a.ids) + i)
                             : (int64_t)__ldcg(static_cast<const int*>(a.ids) + i);
  return id >= 0 && id < a.E ? (int)id : a.E;
}

// A run is counted S = 64 / W steps at a time, their loads in flight
// together; a warp with no more than that keeps its experts for placing.
struct Run {
  int64_t begin, end;
};
template <int W>
__device__ __forceinline__ Run run_of(const SortArgs& a) {
  const int64_t run = a.part / W;
  Run r;
  r.begin = blockIdx.x * a.part + (threadIdx.x >> 5) * run;
  r.end = r.begin + run < a.n ? r.begin + run : a.n;
  return r;
}
template <int S>
__device__ __forceinline__ void load_steps(const SortArgs& a, int64_t i0, int64_t end,
                                           int (&e8)[S]) {
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int64_t i = i0 + s * 32 + (threadIdx.x & 31);
    e8[s] = i < end ? expert_of(a, i) : a.E;
  }
}
// cnt[warp][e] = the warp's assignments to e; rows of E + 1, so that a warp
// reading one expert's counts of 32 warps hits 32 banks
template <int W>
__device__ __forceinline__ void count_runs(const SortArgs& a, int* cnt, const Run& run,
                                           int (&e8)[64 / W]) {
  load_steps(a, run.begin, run.end, e8);
  for (int i = threadIdx.x; i < W * (a.E + 1); i += 32 * W) cnt[i] = 0;
  __syncthreads();
  int* mine = cnt + (threadIdx.x >> 5) * (a.E + 1);
  for (int64_t i0 = run.begin;;) {
#pragma unroll
    for (int s = 0; s < 64 / W; ++s)
      if (e8[s] < a.E) atomicAdd(mine + e8[s], 1);
    i0 += 32 * (64 / W);
    if (i0 >= run.end) break;
    load_steps(a, i0, run.end, e8);
  }
  __syncthreads();
}

template <int W>
__global__ void __launch_bounds__(32 * W) sort_count_kernel(const SortArgs a) {
  extern __shared__ int cnt[];
  pdl_launch_dependents();
  pdl_wait();
  int e8[64 / W];
  count_runs<W>(a, cnt, run_of<W>(a), e8);
  for (int e = threadIdx.x; e < a.E; e += 32 * W) {
    int s = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) s += cnt[w * (a.E + 1) + e];
    const int64_t o = (int64_t)blockIdx.x * a.E + e;
    if (in_bounds(o, 1, (int64_t)a.blocks * a.E, a.status)) a.counts[o] = s;
  }
}

template <int W>
__global__ void __launch_bounds__(32 * W) sort_place_kernel(const SortArgs a) {
  constexpr int kSortThreads = 32 * W, S = 64 / W;
  // [warps][E + 1], the experts' totals [E] and their assignments in the
  // blocks before this one [E]
  extern __shared__ int cnt[];
  int* total = cnt + W * (a.E + 1);
  int* before = total + a.E;
  __shared__ int warp_sum[W];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < 2 * a.E; e += kSortThreads) total[e] = 0;
  const Run run = run_of<W>(a);
  int e8[S];
  count_runs<W>(a, cnt, run, e8);
  const bool kept = run.end - run.begin <= 32 * S;
  if (a.blocks > 1) {
    // every block's counts, summed by all threads, eight loads in flight
    const unsigned all = (unsigned)a.blocks * a.E, mine = blockIdx.x * a.E;
    for (unsigned o0 = threadIdx.x; o0 < all; o0 += 8 * kSortThreads) {
      int v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const unsigned o = o0 + u * kSortThreads;
        v[u] = o < all && in_bounds(o, 1, all, a.status) ? __ldcg(a.counts + o) : 0;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const unsigned o = o0 + u * kSortThreads, e = o % (unsigned)a.E;
        if (v[u]) {
          atomicAdd(total + e, v[u]);
          if (o < mine) atomicAdd(before + e, v[u]);
        }
      }
    }
    __syncthreads();
  }
  // the runs' starts within the block: of 8 runs a thread per expert adds
  // them up, of 32 a warp
  if constexpr (W == 8) {
    for (int e = threadIdx.x; e < a.E; e += kSortThreads) {
      int s = 0;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const int v = cnt[w * (a.E + 1) + e];
        cnt[w * (a.E + 1) + e] = s;
        s += v;
      }
      if (a.blocks == 1) total[e] = s;
    }
  } else {
    static_assert(W == 32, "a lane per run");
    for (int e = warp; e < a.E; e += W) {
      const int v = cnt[lane * (a.E + 1) + e];
      int s = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
      }
      cnt[lane * (a.E + 1) + e] = s - v;
      if (a.blocks == 1 && lane == 31) total[e] = s;
    }
  }
  __syncthreads();
  // exclusive sums of the totals are the offsets; with the blocks before
  // this one they replace `before`
  int carry = 0;
  for (int e0 = 0; e0 < a.E; e0 += kSortThreads) {
    const int e = e0 + threadIdx.x;
    const int v = e < a.E ? total[e] : 0;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += u;
    }
    if (lane == 31) warp_sum[warp] = s;
    __syncthreads();
    // the warps' sums, one per lane
    int ws = lane < W ? warp_sum[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, ws, o);
      if (lane >= o) ws += u;
    }
    const int upto = __shfl_sync(0xffffffffu, ws, warp > 0 ? warp - 1 : 0);
    const int at = carry + (warp > 0 ? upto : 0) + s - v;
    carry += __shfl_sync(0xffffffffu, ws, 31);
    if (e < a.E) {
      if (blockIdx.x == 0) a.offsets[e] = at;
      before[e] += at;
    }
    __syncthreads();
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[a.E] = carry;
  // places, 32 assignments at a time in order
  int* next = cnt + warp * (a.E + 1);
  for (int64_t i0 = run.begin; i0 < run.end; i0 += 32 * S) {
    if (!kept) load_steps(a, i0, run.end, e8);
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int64_t i = i0 + s * 32 + lane;
      const int e = e8[s];
      const unsigned same = __match_any_sync(0xffffffffu, e);
      const int rank = __popc(same & ((1u << lane) - 1u));
      int at = -1;
      if (e < a.E) at = before[e] + next[e] + rank;
      __syncwarp();
      if (e < a.E && rank == 0) next[e] += __popc(same);
      __syncwarp();
      if (i < run.end && in_bounds(i, 1, a.n, a.status)) a.pos[i] = at;
    }
  }
}

// Blocks: one up to 2048 assignments, then as many as that leaves work for,
// one per SM at most (every block sums the counts of all).
int sort_blocks(int64_t n) {
  const int64_t b = (n + kSortItems - 1) / kSortItems;
  const int64_t most = sm_count();
  return (int)(b < 1 ? 1 : b > most ? most : b);
}

template <int W>
cudaError_t launch_sort_t(SortArgs a, cudaStream_t st) {
  const int64_t part = (a.n + a.blocks - 1) / a.blocks;
  a.part = (part + 32 * W - 1) / (32 * W) * (32 * W);
  const size_t smem = (size_t)W * (a.E + 1) * sizeof(int);
  if (a.blocks > 1) {
    const cudaError_t e =
        launch_pdl(sort_count_kernel<W>, dim3(a.blocks), dim3(32 * W), smem, st, a);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(sort_place_kernel<W>, dim3(a.blocks), dim3(32 * W),
                    smem + 2 * (size_t)a.E * sizeof(int), st, a);
}

// ====================================================================== rows
// ---------------------------------------------------------------- gather
// U: the unit a row is copied in.  A block is blockDim.x units of blockDim.y
// tokens' rows: short rows share a block (16384 x 2 rows of 1024 bytes take
// 9.6 us, with a block each 18).  16384 x 8 rows of 4096 codes take 99 us, 6.1
// TB/s of the 604 MB.
template <typename U>
__global__ void __launch_bounds__(kRowThreads) gather_kernel(const MoeArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= a.T) return;
  const int64_t n = a.N;  // units per row
  const int64_t c = (int64_t)blockIdx.y * blockDim.x + threadIdx.x;
  if (a.scale) {
    for (int64_t k = c; k < a.top_k; k += (int64_t)gridDim.y * blockDim.x) {
      const int64_t r = place(a, t, (int)k);
      if (r >= 0 && in_bounds(t, 1, a.T, a.status)) a.scale_out[r] = __ldcg(a.scale + t);
    }
  }
  if (c >= n || !in_bounds(t * n + c, 1, a.T * n, a.status)) return;
  const U v = __ldcg(static_cast<const U*>(a.x) + t * n + c);
  for (int k = 0; k < a.top_k; ++k) {
    const int64_t r = place(a, t, k);
    if (r >= 0 && in_bounds(r * n + c, 1, a.R * n, a.status)) static_cast<U*>(a.out)[r * n + c] = v;
  }
}

template <typename U>
cudaError_t launch_gather_t(MoeArgs a, size_t row_bytes, cudaStream_t st) {
  a.N = (int64_t)(row_bytes / sizeof(U));
  const unsigned nt = row_threads(a.N), tokens = kRowThreads / nt;
  const dim3 grid((unsigned)((a.T + tokens - 1) / tokens), (unsigned)((a.N + nt - 1) / nt));
  return launch_pdl(gather_kernel<U>, grid, dim3(nt, tokens), 0, st, a);
}

}  // namespace

size_t moe_sort_workspace_bytes(int64_t n, int E) {
  const int b = sort_blocks(n);
  return b > 1 ? (size_t)b * (size_t)E * sizeof(int32_t) : 0;
}

cudaError_t launch_moe_sort(const void* ids, bool ids64, int64_t n, int E, int32_t* offsets,
                            int32_t* pos, void* workspace, cudaStream_t st) {
  SortArgs a{};
  a.ids = ids; a.ids64 = ids64; a.n = n; a.E = E;
  a.blocks = sort_blocks(n);
  a.offsets = offsets; a.pos = pos;
  a.counts = static_cast<int32_t*>(workspace);
  a.status = status_word();
  if (!a.status) return cudaErrorInvalidDevice;
  return E <= kSortWide && n > kSortFew ? launch_sort_t<32>(a, st) : launch_sort_t<8>(a, st);
}

cudaError_t launch_moe_gather(MoeArgs a, size_t elem, cudaStream_t st) {
  a.status = status_word();
  if (!a.status) return cudaErrorInvalidDevice;
  const size_t row = (size_t)a.N * elem;
  if (row % 16 == 0) return launch_gather_t<uint4>(a, row, st);
  if (row % 4 == 0) return launch_gather_t<uint32_t>(a, row, st);
  if (row % 2 == 0) return launch_gather_t<uint16_t>(a, row, st);
  return launch_gather_t<uint8_t>(a, row, st);
}

}  // namespace sq
