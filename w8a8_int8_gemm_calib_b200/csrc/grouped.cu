// grouped.cu -- the routed experts' INT8 GEMM: one weight matrix per group of
// rows, the groups (offsets) known to the device alone.
//
//   acc[r,n] = sum_k xq[r,k] * wq[e,n,k],  offsets[e] <= r < offsets[e+1]
//   y[r,n]   = (float)acc[r,n] * (as_r * w_scale[e,n]) (+ bias[e,n])
//
// Bound: an expert with few rows by the stream of its weights (HBM), one with
// many by the tensor cores; they meet near 280 rows per expert.
//
// The operands are swapped: 256 of an expert's output channels fill the M
// dimension of the MMA and up to 256 of its rows the N dimension, which takes
// any multiple of 32.  So an expert with 300 rows computes 320 (two tiles of
// 160), where 256-row tiles would compute 512: rows per expert are ragged,
// channels are not.  The weights then stream through the A operand once per
// 256 rows (32, where the experts have few) whatever the number of rows is.
//
// Persistent CTA pairs (tcgen05 cta_group::2, one pair per two SMs): each CTA
// loads 128 channels of weights and half the tile's rows per 128-byte k-block
// (16 KB + up to 16 KB; 2 KB with 32-row tiles), the even CTA issues the MMAs for both, each CTA
// drains its 128 channels.  Two accumulators of 256 TMEM columns, so one
// tile's epilogue runs under the next tile's main loop.  Warp 0 issues the
// loads, warp 1 the MMAs, the others drain.  Every wait is bounded.
//
// The accumulator has channels along the TMEM lanes and rows along its
// columns; the epilogue turns it round through shared memory.
//
// Measured (bf16 out): 8 experts of 14336x4096 with 1024 rows each 320 us, 3000
// TOPS, the tensor pipe active 96 % of the time (power-capped: 1.5 GHz); 64
// experts of 4096x4096 with 8 rows each 165 us, 6.5 TB/s.  In between neither
// bound is reached: 64 such experts with 256 rows each take 234 us, 2350 TOPS
// and 5.4 TB/s, with uneven ones 263 to 280 us; what holds them is not known.
// With K = 512 the epilogue does: 64 experts of 2048x512 with 512 rows each
// take 63 us, 33 without it and 48 without its proxy fences alone.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <mutex>

#include "launch.cuh"
#include "sq_device.cuh"
#include "sq_internal.h"
#include "tc_ptx.cuh"
#include "tmaps.h"

namespace sq {

namespace {

constexpr int BK = 128;              // bytes of K per stage: one 128-byte swizzle row
constexpr int UK = 32;               // K per tcgen05.mma kind::i8
constexpr int CH = 128;              // channels per CTA
constexpr int TILE_N = 2 * CH;       // channels per pair
constexpr int STEP_R = 32;           // granularity of a tile's rows (MMA N of a CTA pair)
constexpr int W_BYTES = CH * BK;     // a stage's weights
constexpr int BOXES = 4;             // row boxes of 16, 32, 64 and 128
constexpr uint64_t kWaitNs = 4000000000ull;   // 4 s: far above any pipeline step
constexpr uint64_t kDrainNs = 1000000000ull;  // waits for copies already in flight
constexpr uint64_t kPairGraceNs = 2000000ull; // after a time-out: the peer's copies land

// TILE_R: rows per tile, at most (256, or 32 for a few rows per expert).
template <bool BF16, int TILE_R>
struct Cfg {
  static constexpr int EPI_W = TILE_R > 32 ? 8 : 4;  // epilogue warps
  static constexpr uint32_t TMEM_COLS = 2 * TILE_R;
  static constexpr int X_BYTES = TILE_R / 2 * BK;    // a stage's rows, at most
  static constexpr int STAGE = W_BYTES + X_BYTES;
  static constexpr int THREADS = 64 + 32 * EPI_W;
  static constexpr int EPI_BUF = BF16 ? 32 * 64 : 32 * 128;  // 32 rows x 32 channels
  static constexpr int NB = EPI_W > 4 ? 1 : 2;               // buffers per warp
  static constexpr int EPI_BYTES = EPI_W * NB * EPI_BUF;
  static constexpr int MY_CHUNKS = TILE_R / 32 / (EPI_W / 4);  // 32-row chunks a warp drains
  static constexpr int AS_BYTES = EPI_W * MY_CHUNKS * 32 * 4;  // their rows' steps
  static constexpr int TABLE = 2 * (kMaxExperts + 1) * 4;
  static_assert(MY_CHUNKS >= 1 && STAGE % 1024 == 0, "chunks, swizzle atoms");
  static constexpr int FIXED = 1024 + EPI_BYTES + AS_BYTES + 256 + TABLE;
  static constexpr int STAGES = (227 * 1024 - FIXED) / STAGE;
  static constexpr size_t SMEM = FIXED + (size_t)STAGES * STAGE;
  static_assert(STAGES >= 4, "main-loop stages");
};

struct Params {
  int R, N, E;
  int n_tiles, nk;
  int band;  // row tiles of a raster band
  const int32_t* offsets;
  const float* act_scale;
  int per_token;
  const float* w_scale;
  const float* bias;
  void* y;
  int tma_store;
  int piece;  // bytes that the rows' pitch keeps aligned: 16, 8, 4, or a bf16's 2
  int32_t* acc;
  unsigned int* status;
};

struct RowMaps {
  CUtensorMap m[BOXES];
};

// One warp fills the CTA's table: off[e], the experts' first rows, and
// tiles[e], the row tiles before expert e.  Offsets outside [0, R] or falling
// ones are clamped to a rising sequence, so a bad table gives rows to the
// wrong expert but touches nothing outside the arrays.
__device__ __forceinline__ void group_table(const Params& p, int tile_r, int* off, int* tiles) {
  const int lane = threadIdx.x & 31;
  int top = 0, before = 0;
  for (int e0 = 0; e0 <= p.E; e0 += 32) {
    const int e = e0 + lane;
    int v = e <= p.E ? min(max(__ldcg(p.offsets + e), 0), p.R) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v = max(v, u);
    }
    v = max(v, top);
    const int prev = __shfl_up_sync(0xffffffffu, v, 1);
    // the rows between offsets e - 1 and e are expert e - 1's
    const int n = e > 0 && e <= p.E ? (v - (lane ? prev : top) + tile_r - 1) / tile_r : 0;
    int s = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += u;
    }
    if (e <= p.E) {
      off[e] = v;
      tiles[e] = before + s;
    }
    top = __shfl_sync(0xffffffffu, v, 31);
    before += __shfl_sync(0xffffffffu, s, 31);
  }
}

// A tile: expert e, channels n0 .. n0 + 255, rows row0 .. row0 + rows - 1,
// computed as mma_n rows.
struct Tile {
  int e, n0, row0, rows, mma_n;
};

// An expert's tiles in bands of p.band row tiles, each band sweeping every
// channel with its row tiles innermost: the band's rows stay in L2 and a
// channel tile's weights are read from HBM once per band.  Tiles ascend, so
// the search for e goes on from the last tile's.  An expert's row tiles are
// all of the same size but the last: its rows split evenly, up to a multiple
// of 32.
__device__ __forceinline__ void locate(const Params& p, const int* off, const int* tiles, int tile,
                                       Tile& t) {
  while (tile >= tiles[t.e + 1] * p.n_tiles) ++t.e;
  const int m_tiles = tiles[t.e + 1] - tiles[t.e];
  const int local = tile - tiles[t.e] * p.n_tiles;
  const int per_band = p.band * p.n_tiles;
  const int b = local / per_band, first = b * p.band;
  const int bm = min(m_tiles - first, p.band), r = local - b * per_band;
  const int mb = first + r % bm;
  t.n0 = r / bm * TILE_N;
  const int all = off[t.e + 1] - off[t.e];
  const int per = ((all + m_tiles - 1) / m_tiles + STEP_R - 1) / STEP_R * STEP_R;
  t.row0 = off[t.e] + mb * per;
  t.rows = min(per, all - mb * per);
  t.mma_n = (t.rows + STEP_R - 1) / STEP_R * STEP_R;
}

// Rows row0 .. row0 + valid - 1, channels col0 .. col0 + 31, from a swizzled
// buffer in pieces of G bytes (G divides the rows' pitch), several rows a step.
template <int G> struct Piece;
template <> struct Piece<16> { using T = uint4; };
template <> struct Piece<8> { using T = uint2; };
template <> struct Piece<4> { using T = uint32_t; };
template <> struct Piece<2> { using T = uint16_t; };
template <bool BF16, int G>
__device__ __forceinline__ void store_rows(const Params& p, const uint8_t* buf, int row0, int valid,
                                           int col0, int lane) {
  if constexpr (BF16 || G > 2) {
    using T = typename Piece<G>::T;
    constexpr int ES = BF16 ? 2 : 4, ROW = 32 * ES;  // a row's bytes in the buffer
    constexpr int LANES = ROW / G;                   // lanes on a row
    constexpr int ROWS = 32 / LANES;                 // rows a step
    constexpr int STEPS = 32 / ROWS, U = 4;  // STEPS is 4, 8, 16 or 32
    const int off = lane % LANES * G, n = col0 + off / ES;
    if (n >= p.N) return;
    const int64_t first = (int64_t)(row0 + lane / LANES) * p.N + n, step = (int64_t)ROWS * p.N;
    uint8_t* y = static_cast<uint8_t*>(p.y) + first * ES;
#pragma unroll 1
    for (int s0 = 0; s0 < STEPS && s0 * ROWS < valid; s0 += U) {
      T v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = (s0 + u) * ROWS + lane / LANES;
        const int k = (off >> 4) ^ (BF16 ? (i >> 1) & 3 : i & 7);
        v[u] = *reinterpret_cast<const T*>(buf + i * ROW + k * 16 + (off & 15));
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if ((s0 + u) * ROWS + lane / LANES < valid &&
            in_bounds(first + (s0 + u) * step, G / ES, (int64_t)p.R * p.N, p.status))
          *reinterpret_cast<T*>(y) = v[u];
        y += step * ES;
      }
    }
  }
}

template <bool BF16, int TILE_R>
__global__ void __launch_bounds__(Cfg<BF16, TILE_R>::THREADS, 1)
grouped_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ RowMaps tmX,
               const __grid_constant__ CUtensorMap tmY, const Params p) {
  using C = Cfg<BF16, TILE_R>;
  constexpr int STAGES = C::STAGES, X_BYTES = C::X_BYTES, EPI_W = C::EPI_W;
  constexpr uint32_t TMEM_COLS = C::TMEM_COLS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sW = smem;
  uint8_t* sX = smem + STAGES * W_BYTES;
  uint8_t* sEpi = smem + STAGES * C::STAGE;  // 1024-aligned
  float* sAs = reinterpret_cast<float*>(sEpi + C::EPI_BYTES);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sEpi + C::EPI_BYTES + C::AS_BYTES);
  // bars: full[STAGES], empty[STAGES], tfull[2], tempty[2], drain
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* off = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + 256);
  int* tiles = off + kMaxExperts + 1;

  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto full_bar = [&](int s) { return tc::smem_u32(bars + s); };
  auto empty_bar = [&](int s) { return tc::smem_u32(bars + STAGES + s); };
  auto tfull_bar = [&](int b) { return tc::smem_u32(bars + 2 * STAGES + b); };
  auto tempty_bar = [&](int b) { return tc::smem_u32(bars + 2 * STAGES + 2 + b); };
  const uint32_t drain_bar = tc::smem_u32(bars + 2 * STAGES + 4);
  const int rank = (int)tc::cluster_ctarank();
  const bool leader = rank == 0;
  const int unit0 = (int)(blockIdx.x >> 1), units = (int)(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      tc::mbar_init(full_bar(s), 1);
      tc::mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(tfull_bar(b), 1);
      tc::mbar_init(tempty_bar(b), 2 * EPI_W);  // the epilogue warps of both CTAs
    }
    tc::mbar_init(drain_bar, 1);
    *abort_flag = 0;
    tc::mbar_fence_init();
    tc::tma_prefetch_desc(&tmW);
    for (int i = 0; i < BOXES; ++i) tc::tma_prefetch_desc(&tmX.m[i]);
  }
  if (warp == 1) {
    tc::tmem_alloc_pair(tc::smem_u32(tmem_slot), TMEM_COLS);
    tc::tmem_relinquish_pair();
  }
  pdl_wait();  // nothing before this touches global memory
  if (warp == 0) group_table(p, TILE_R, off, tiles);
  tc::tc_fence_before();
  tc::cluster_sync();  // the peer's barriers are initialised, this CTA's table is filled
  tc::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int num_tiles = tiles[p.E] * p.n_tiles;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (tc::elect_one()) {
      uint32_t stage = 0, phase = 0, issued = 0, issued_par = 0;
      bool ok = true;
      Tile t{};
      for (int tile = unit0; ok && tile < num_tiles; tile += units) {
        locate(p, off, tiles, tile, t);
        const int half = t.mma_n / 2;  // this CTA's rows of the MMA
        const int box = half <= 16 ? 0 : half <= 32 ? 1 : half <= 64 ? 2 : 3;
        const CUtensorMap* mx = &tmX.m[box];
        const uint32_t bytes = W_BYTES + (16u << box) * BK;
        for (int kb = 0; kb < p.nk; ++kb) {
          if (!tc::mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, kWaitNs, p.status)) {
            ok = false;
            break;
          }
          // both CTAs' bytes complete on the even CTA's barrier, which alone
          // expects them; rows past the tile are loaded and not stored
          const uint32_t fb = tc::mapa_shared(full_bar(stage), 0);
          if (leader) tc::mbar_arrive_expect_tx(full_bar(stage), 2 * bytes);
          tc::tma_load_3d_pair(tc::smem_u32(sW + stage * W_BYTES), &tmW, kb * BK, t.n0 + rank * CH,
                               t.e, fb);
          tc::tma_load_2d_pair(tc::smem_u32(sX + stage * X_BYTES), mx, kb * BK,
                               t.row0 + rank * half, fb);
          issued |= 1u << stage;
          issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok) {
        // let every load already issued land before the CTA exits; the odd
        // CTA's complete on the even CTA's barriers, which it cannot wait on:
        // a fixed grace period
        int never = 0;
        if (leader)
          for (int s = 0; s < STAGES; ++s)
            if (issued & (1u << s))
              tc::mbar_wait(full_bar(s), (issued_par >> s) & 1u, &never, kDrainNs, p.status);
        const uint64_t t0 = global_ns();
        while (global_ns() - t0 < kPairGraceNs) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (leader && tc::elect_one()) {
      uint32_t stage = 0, phase = 0, abuf = 0, aphase = 0;
      bool ok = true;
      Tile t{};
      for (int tile = unit0; ok && tile < num_tiles; tile += units) {
        locate(p, off, tiles, tile, t);
        const uint32_t idesc = tc::idesc_i8(TILE_N, t.mma_n);
        if (!tc::mbar_wait(tempty_bar(abuf), aphase ^ 1u, abort_flag, kWaitNs, p.status)) {
          ok = false;
          break;
        }
        tc::tc_fence_after();
        const uint32_t d = tmem_base + abuf * TILE_R;
        for (int kb = 0; kb < p.nk; ++kb) {
          if (!tc::mbar_wait(full_bar(stage), phase, abort_flag, kWaitNs, p.status)) {
            ok = false;
            break;
          }
          tc::tc_fence_after();
          const uint32_t w0 = tc::smem_u32(sW + stage * W_BYTES);
          const uint32_t x0 = tc::smem_u32(sX + stage * X_BYTES);
#pragma unroll
          for (int k = 0; k < BK / UK; ++k)
            tc::mma_i8_pair(d, tc::desc_k_sw128(w0 + k * UK), tc::desc_k_sw128(x0 + k * UK), idesc,
                            (kb | k) != 0);
          tc::mma_commit_pair(empty_bar(stage), 0x3);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        tc::mma_commit_pair(tfull_bar(abuf), 0x3);
        abuf ^= 1u;
        if (abuf == 0) aphase ^= 1u;
      }
      // every MMA issued so far must finish before TMEM is released
      tc::mma_commit_pair(drain_bar, 0x1);
      int never = 0;
      tc::mbar_wait(drain_bar, 0, &never, kDrainNs, p.status);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    // A warp drains 32 channels x 32 rows at a time with two 16x256b loads: in
    // fragment m (channels 16 m ..), lane l holds channels cl and cl + 8, cl =
    // l / 4, of rows 2 (l % 4) and the next, for each of four groups of 8
    // rows.  Transposing 8x8 stores of bf16 pairs (stmatrix.trans) then write
    // whole 16-byte pieces of output rows.
    const int quarter = warp & 3;        // TMEM lanes 32*quarter .. +31: this warp's channels
    const int chunk0 = (warp - 2) >> 2;  // first of its 32-row chunks
    const int cl = lane >> 2, rl = 2 * (lane & 3);
    const uint64_t y_policy = tc::l2_policy_evict_first();  // y is not read back here
    uint8_t* ebuf = sEpi + (warp - 2) * C::NB * C::EPI_BUF;
    float* as_w = sAs + (warp - 2) * C::MY_CHUNKS * 32;
    uint32_t nstore = 0, abuf = 0, aphase = 0;
    // A tile's place, its channels' steps and biases (col0 + cl + 8 i) and its
    // rows' steps (one per lane and chunk) are fetched a tile ahead.
    Tile next{};
    float ws_n[4], bs_n[4], as_n[C::MY_CHUNKS];
    auto fetch = [&](int tile) {
      if (tile >= num_tiles) return;
      locate(p, off, tiles, tile, next);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = next.n0 + rank * CH + quarter * 32 + cl + 8 * i;
        const int64_t sn = (int64_t)next.e * p.N + n;
        const bool ok = n < p.N && in_bounds(sn, 1, (int64_t)p.E * p.N, p.status);
        ws_n[i] = ok ? __ldcg(p.w_scale + sn) : 0.0f;
        bs_n[i] = ok && p.bias ? __ldcg(p.bias + sn) : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < C::MY_CHUNKS; ++i) {
        const int c = (chunk0 + i * (EPI_W / 4)) * 32 + lane;
        as_n[i] = __ldcg(p.act_scale + (p.per_token ? next.row0 + min(c, next.rows - 1) : 0));
      }
    };
    fetch(unit0);
    for (int tile = unit0; tile < num_tiles; tile += units) {
      const Tile t = next;
      const int col0 = t.n0 + rank * CH + quarter * 32;
      float ws[4], bs[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ws[i] = ws_n[i];
        bs[i] = bs_n[i];
      }
      __syncwarp();  // the last tile's steps are read
#pragma unroll
      for (int i = 0; i < C::MY_CHUNKS; ++i) as_w[i * 32 + lane] = as_n[i];
      __syncwarp();
      fetch(tile + units);
      const bool got = tc::mbar_wait(tfull_bar(abuf), aphase, abort_flag, kWaitNs, p.status);
      if (!__all_sync(0xffffffffu, got)) break;  // the warp gives up as one
      tc::tc_fence_after();
      const float* as_c = as_w;
      const uint32_t taddr = tmem_base + abuf * TILE_R + ((uint32_t)(quarter * 32) << 16);
#pragma unroll 1
      for (int c = chunk0 * 32; c < t.mma_n; c += 8 * EPI_W, as_c += 32) {
        const int row0 = t.row0 + c, valid = min(32, t.rows - c);
        // r[m][4 g + ...]: channels 16 m + {cl, cl, cl + 8, cl + 8}, rows 8 g +
        // {rl, rl + 1, rl, rl + 1}
        uint32_t r[2][16];
        tc::tmem_ld_16x256b_x4(taddr + c, r[0]);
        tc::tmem_ld_16x256b_x4(taddr + c + (16u << 16), r[1]);
        tc::tmem_ld_wait();
        if (p.acc) {
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int row = 8 * (i >> 2) + rl + (i & 1);
              const int n = col0 + 16 * m + cl + 8 * ((i >> 1) & 1);
              const int64_t o = (int64_t)(row0 + row) * p.N + n;
              if (row < valid && n < p.N && in_bounds(o, 1, (int64_t)p.R * p.N, p.status))
                p.acc[o] = (int)r[m][i];
            }
        }
        uint8_t* buf = ebuf + nstore % C::NB * C::EPI_BUF;
        if (lane == 0) tc::bulk_wait_read<C::NB - 1>();  // the store that last read `buf` is done
        __syncwarp();
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float2 as = *reinterpret_cast<const float2*>(as_c + 8 * g + rl);
          float v[2][4];
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              // (float)acc * (as * ws), then the bias: separate fp32 roundings
              const int w = 2 * m + (i >> 1);
              const float y = __fmul_rn(__int2float_rn((int)r[m][4 * g + i]),
                                        __fmul_rn(i & 1 ? as.y : as.x, ws[w]));
              v[m][i] = p.bias ? __fadd_rn(y, bs[w]) : y;
            }
          if constexpr (BF16) {
            // Output rows 8 g .. 8 g + 7 of 64 bytes: piece k (8 channels) of
            // row i at k ^ ((i >> 1) & 3), the 64-byte swizzle.  Lane l gives
            // the address of row l % 8 of piece l / 8.
            uint32_t q[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float* vk = v[k >> 1] + 2 * (k & 1);
              const __nv_bfloat162 h = __floats2bfloat162_rn(vk[0], vk[1]);
              q[k] = *reinterpret_cast<const uint32_t*>(&h);
            }
            const int i = 8 * g + (lane & 7), k = (lane >> 3) ^ ((i >> 1) & 3);
            tc::stmatrix_x4_trans(tc::smem_u32(buf + i * 64 + k * 16), q);
          } else {
            // Output rows of 128 bytes: 16-byte piece k of row i at k ^ (i & 7),
            // the 128-byte swizzle; 8 lanes write 32 bytes of one row, the four
            // rows of a warp's write differ in their banks.
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int i = 8 * g + rl + (e & 1), ch = 16 * m + cl + 8 * (e >> 1);
                const int k = (ch >> 2) ^ (i & 7);
                *reinterpret_cast<float*>(buf + i * 128 + k * 16 + (ch & 3) * 4) = v[m][e];
              }
          }
        }
        if (p.tma_store && valid == 32) {
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (col0 < p.N) tc::tma_store_2d_hint(&tmY, tc::smem_u32(buf), col0, row0, y_policy);
            tc::bulk_commit();
          }
          ++nstore;
          continue;
        }
        // A TMA store clips at the tensor's edge, not at the expert's, and
        // needs 16-byte row pitches: otherwise the rows go from the buffer in
        // the pieces their pitch keeps aligned.
        __syncwarp();
        switch (p.piece) {
          case 16: store_rows<BF16, 16>(p, buf, row0, valid, col0, lane); break;
          case 8: store_rows<BF16, 8>(p, buf, row0, valid, col0, lane); break;
          case 4: store_rows<BF16, 4>(p, buf, row0, valid, col0, lane); break;
          default: store_rows<BF16, 2>(p, buf, row0, valid, col0, lane); break;
        }
        __syncwarp();  // read before the next chunk overwrites it
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive_cluster(tc::mapa_shared(tempty_bar(abuf), 0));
      abuf ^= 1u;
      if (abuf == 0) aphase ^= 1u;
    }
    if (lane == 0) tc::bulk_wait_all();  // staged outputs written before the CTA exits
    __syncwarp();
  }

  tc::tc_fence_before();
  __syncthreads();
  // neither CTA leaves while the other may still reach its barriers or
  // shared memory
  tc::cluster_sync();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

// Row tiles per raster band: about 32 MB of rows, 4 to 16 tiles, as the plain
// GEMM's CTA pairs take it.
int band_tiles(int64_t K) {
  const int64_t t = ((int64_t)32 << 20) / (256 * K);
  return t > 16 ? 16 : t < 4 ? 4 : (int)t;
}

// Tiles of 32 rows leave room for 11 stages of weights where 256 rows leave
// 6, and with few rows the stream of the weights is all there is.  us with
// tiles of 256 / 32 rows: 8 experts of 4096x4096 with a row each 26.0 / 24.8,
// of 14336x4096 with 32 rows each 81.5 / 75.5; 64 of 4096x4096 with 8 rows each
// 166.6 / 165.3, with 32 rows each 170.0 / 170.4.  The host knows only the
// average: an expert with more rows reads its weights from L2 once per 32 of
// them (those 64 with half of the 2048 rows in one 176.7 / 201.2, with all
// 28.1 / 82.4), and with short K there are more epilogues (64 of 2048x512 with
// 32 rows each 23.2 / 25.6).
int tile_rows(int64_t R, int64_t E) { return R <= 32 * E ? 32 : 256; }

// The number of pairs that can be resident at once is queried once per
// device; a persistent launch never asks for more.
template <bool BF16, int TILE_R>
cudaError_t launch_t(const CUtensorMap& tw, const RowMaps& tx, const CUtensorMap& ty,
                     const Params& p, int64_t most, cudaStream_t st) {
  using C = Cfg<BF16, TILE_R>;
  auto kern = grouped_kernel<BF16, TILE_R>;
  static std::once_flag once[64];
  static cudaError_t err[64];
  static int max_pairs[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 64) return e != cudaSuccess ? e : cudaErrorInvalidDevice;
  std::call_once(once[dev], [&] {
    err[dev] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
    if (err[dev] != cudaSuccess) return;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2 * (unsigned)(sm_count() / 2));
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    err[dev] = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
    max_pairs[dev] = n;
  });
  if (err[dev] != cudaSuccess) return err[dev];
  if (max_pairs[dev] < 1) return cudaErrorInvalidConfiguration;
  int64_t pairs = sm_count() / 2;
  if (pairs > max_pairs[dev]) pairs = max_pairs[dev];
  if (pairs > most) pairs = most;
  return launch_pdl_cluster(kern, dim3(2 * (unsigned)pairs), dim3(C::THREADS), C::SMEM, st, 2u, tw,
                            tx, ty, p);
}

}  // namespace

sq_status launch_gemm_grouped(const GroupArgs& a, cudaStream_t st) {
  const char* fn = "sq_gemm_w8a8_grouped";
  unsigned int* sw = status_word();
  if (!sw) return fail(SQ_ERR_CUDA, "%s: device status word unavailable", fn);
  const bool bf16 = a.yt == SQ_BF16;
  CUtensorMap tw, ty;
  RowMaps tx;
  memset(&ty, 0, sizeof ty);
  bool ok = make_tmap3(&tw, a.wq, (uint64_t)a.K, (uint64_t)a.N, (uint64_t)a.E, CH);
  for (int i = 0; ok && i < BOXES; ++i)
    ok = make_tmap(&tx.m[i], a.xq, (uint64_t)a.K, (uint64_t)a.R, 16u << i);
  if (!ok) return fail(SQ_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed", fn);
  Params p{};
  p.R = (int)a.R; p.N = (int)a.N; p.E = (int)a.E;
  p.n_tiles = (int)((a.N + TILE_N - 1) / TILE_N);
  p.nk = (int)((a.K + BK - 1) / BK);
  p.band = band_tiles(a.K);
  p.offsets = a.offsets;
  p.act_scale = a.act_scale;
  p.per_token = a.act_per_token;
  p.w_scale = a.w_scale;
  p.bias = a.bias;
  p.y = a.y;
  p.acc = a.acc_out;
  p.status = sw;
  // TMA stores need 16-byte row pitches; other widths store directly
  p.tma_store = (a.N % (bf16 ? 8 : 4)) == 0 &&
                make_tmap_out(&ty, a.y, (uint64_t)a.N, (uint64_t)a.R, bf16, bf16 ? 64 : 128);
  const int64_t pitch = a.N * (bf16 ? 2 : 4);
  p.piece = pitch % 16 == 0 ? 16 : pitch % 8 == 0 ? 8 : pitch % 4 == 0 ? 4 : 2;
  const int tile_r = tile_rows(a.R, a.E);
  // tiles, whatever the offsets
  const int64_t most = ((a.R + tile_r - 1) / tile_r + a.E) * p.n_tiles;
  cudaError_t e;
  if (tile_r == 32)
    e = bf16 ? launch_t<true, 32>(tw, tx, ty, p, most, st)
             : launch_t<false, 32>(tw, tx, ty, p, most, st);
  else
    e = bf16 ? launch_t<true, 256>(tw, tx, ty, p, most, st)
             : launch_t<false, 256>(tw, tx, ty, p, most, st);
  if (e != cudaSuccess) return fail(SQ_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
  return SQ_OK;
}

}  // namespace sq
