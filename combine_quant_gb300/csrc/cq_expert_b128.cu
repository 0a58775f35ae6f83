// cq_expert_b128.cu -- expert products from fp8 rows with one scale per 128 columns
// and fp8 weights with one per 128 x 128 block, on the tensor cores (tcgen05):
// forward (SwiGLU, results in 16 bits or in fp8 with scales) and the gradient of
// the input.
//
// A persistent kernel on pairs of CTAs, as cq_expert_gemm.cu's, with copies by warp 0
// and products by warp 1 of the first CTA. What differs is that a scale holds for 128
// of the contraction only:
//
//   acc[j, i] += (xs[j, B] ws[B]) * sum over k in B of x[j, k] w[i, k]
//
// So every stage (128 of the contraction, four products) goes into a TMEM accumulator
// of its own, two in turn, and eight warps take it from there into registers, scaled:
// 128 sums a thread, all of a tile. That work, not the products, is the bound where there
// are many tokens: it takes 1000 clocks a stage where the products take 590. Tokens lie on
// the accumulator's lanes (up to 128 in each CTA) and weight rows on its columns: a lane's
// factor is one number per 128 columns. With tokens on the columns the factors are a
// vector that every warp reads anew for every stage (512 rows an expert, hidden 7168,
// SwiGLU: 813 us, now 442); so that is done where a tile has 128 tokens or fewer, which
// are few columns then (16 rows an expert: 123 us by lanes, now 87). What a warp does for a
// stage is kept short and in registers: 24 spilled bytes in that loop cost a quarter, and
// scales read into registers by the warps themselves a tenth (486 us; 442 with two warps
// that copy them into shared memory). Twelve or sixteen warps with fewer sums each were
// slower (505, 676), as were halves of an accumulator handed over apart (520).
//
// SwiGLU: the columns are 16 gates, 16 ups, 16 gates, ... (one 5-D copy). fp8 results:
// a group of 128 outputs is a thread's own columns, with SwiGLU those of two threads.
// dx: w with its columns along the tile (MN-major), the contraction runs over n.
//
// Measured on one GB300 (copy 6.78 TB/s, cuBLAS bf16 1.9 PFLOP/s): 8192^3 499 us, 2.2
// PFLOP/s; 32 experts of 512 rows, hidden 7168, SwiGLU with n 2048: 442 us, 2.2 PFLOP/s
// (uneven experts of 512 on average: 540, whose lanes are four fifths full); 16 rows each,
// n 7168, k 2048: 87 us, 5.5 TB/s.
#include <cuda_runtime.h>

#include <algorithm>

#include "cq_expert.cuh"
#include "cq_permute_impl.cuh"
#include "cq_tensor.cuh"

namespace cq {
namespace expert {
namespace {

using namespace tensor;
using async::mbar_arrive;
using async::mbar_arrive_expect_tx;
using async::mbar_init;
using async::mbar_wait;
using async::mbar_wait_warp;

__device__ uint32_t g_status;  // CQ_ST_* bits of these kernels on this device

struct B128Args : Args {
  const float* xs;
  const float* ws;
  float* ys;
  int32_t n, nb, kb;    // n, its blocks of 128, k's blocks
  int32_t blocks;       // of the contraction
  int32_t half_blocks;  // dx: of one half of it; forward: all
  int32_t half_len;     // the contraction's length, dx: of one half
  int32_t out_cols;     // columns of the result: n, or (dx) k
  int32_t tiles_i;
  int32_t wide;         // rows of the results (and of saved products) are whole 32-byte pieces
};

constexpr int kStages = 6;
constexpr int kABytes = 128 * 128;         // A (tokens) of one stage, one CTA
constexpr int kStageBytes = 2 * kABytes;   // B: half of up to 256 weight rows
constexpr int kNT = 256;                   // TMEM columns of an accumulator
constexpr int kDrainWarps = 8;             // two for each quarter of the lanes
constexpr int kThreads = 128 + 32 * kDrainWarps;
// Registers: 384 threads are launched with 168 each (64512); the drain warps keep 128
// sums and need 224, the others 56, which is the same total.
constexpr int kOtherRegs = 56, kDrainRegs = 224;
constexpr int kAllRegs = 128 * kOtherRegs + 32 * kDrainWarps * kDrainRegs;
static_assert(kAllRegs <= 168 * kThreads, "setmaxnreg would wait forever");
constexpr int kFew = 128;                  // most rows of a tile with tokens on the columns
constexpr int kEntry = 4;                  // blocks in an entry of the scales' ring
constexpr int kScaleRing = 3;
constexpr int kScaleFloats = kEntry * 128 + kEntry * 2;  // the rows', and two of the weights
constexpr uint32_t kTmemCols = 512;
constexpr int kBand = 8;                   // tiles along i taken together, for reuse in L2

struct RowMaps {
  CUtensorMap b128, b64, b32;
};

struct Bars {
  uint64_t full[kStages], empty[kStages];
  uint64_t tfull[2], tempty[2];
  uint64_t sfull[kScaleRing], sempty[kScaleRing];
  uint64_t few_top[2];  // the same of tokens on the columns, by the warps' half
  uint64_t top[4];  // fp8 results: the largest values of a quarter's two warps
  uint64_t done;    // the products in flight when their warp gave up
  uint32_t tmem;
};

struct Tile {
  int e, row0, rows;  // first token row and rows of the tile
  int i0, cols;       // first output and weight rows (both CTAs)
  bool few;           // tokens on the accumulator's columns
  int jh;             // tokens of the first CTA
};

// Tiles of at most 256 that an expert's rows make: equal parts (unsigned: rows + 255 may pass 2^31).
__device__ __forceinline__ int parts_of(int rows) { return (int)(((uint32_t)rows + 255) / 256); }

// GATES: a tile is 128 outputs, else 256. Columns in steps of 64 (16 outputs a CTA) or 32.
template <bool GATES, bool OUT8>
__device__ __forceinline__ Tile tile_at(const B128Args& a, const int* s_begin, const int* s_tile, int t) {
  Tile x;
  x.e = expert_of(s_tile, a.G, t);
  const int l = t - s_tile[x.e];
  const int begin = s_begin[x.e], rows = s_begin[x.e + 1] - begin;
  const int parts = parts_of(rows);
  const int band = l / (kBand * parts), first_i = band * kBand;
  const int wide = min(kBand, a.tiles_i - first_i), m = l - first_i * parts;
  const int ti = first_i + m % wide, tj = m / wide;
  const int step = (int)(((uint32_t)rows + parts - 1) / parts);
  x.row0 = begin + tj * step;
  x.rows = min(step, rows - tj * step);
  constexpr int kOuts = GATES ? 128 : 256;
  x.i0 = ti * kOuts;
  const int outs = (min(kOuts, a.out_cols - x.i0) + 31) / 32 * 32;
  x.cols = GATES ? 2 * outs : outs;
  // (fp8 results: unless a group of 128 outputs would end within a CTA's rows)
  x.few = x.rows <= kFew && (!OUT8 || GATES || x.cols <= 128 || x.cols == 256);
  x.jh = (x.rows + 1) / 2;
  if (x.few) x.jh = (x.jh + 7) / 8 * 8;
  return x;
}

using Pair = unsigned long long;  // two floats
__device__ __forceinline__ Pair pair_of(uint32_t lo, uint32_t hi) {
  Pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "r"(lo), "r"(hi));
  return p;
}
__device__ __forceinline__ Pair pair_of(float lo, float hi) {
  return pair_of(__float_as_uint(lo), __float_as_uint(hi));
}
__device__ __forceinline__ float lo_of(Pair p) { return __uint_as_float((uint32_t)p); }
__device__ __forceinline__ float hi_of(Pair p) { return __uint_as_float((uint32_t)(p >> 32)); }
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// acc += 32 columns, the first 16 times sg, the others times su.
__device__ __forceinline__ void add_scaled(const uint32_t (&v)[32], Pair sg, Pair su, Pair (&acc)[16]) {
#pragma unroll
  for (int k = 0; k < 16; ++k) acc[k] = fma2(pair_of(v[2 * k], v[2 * k + 1]), k < 8 ? sg : su, acc[k]);
}

__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ void ld_pairs(uint32_t addr, Pair& a, Pair& b) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr) : "memory");
}
__device__ __forceinline__ void copy4_async(uint32_t dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// An arrival on `bar` when this thread's copies so far have landed.
__device__ __forceinline__ void arrive_on_copies(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// 32 bytes to or from global memory: one access, or two where a row need not begin
// on 32 bytes.
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
__device__ __forceinline__ void load32(const void* p, uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  } else {
    const uint4 a = __ldg(static_cast<const uint4*>(p)), b = __ldg(static_cast<const uint4*>(p) + 1);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
}

// 16 values (8 pairs) rounded to 16 bits.
template <typename T>
__device__ __forceinline__ void store16(uint16_t* p, const Pair* v, bool wide) {
  uint32_t w[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) w[k] = T::pack2(lo_of(v[k]), hi_of(v[k]));
  store32(p, w, wide);
}

__device__ __forceinline__ float top_of(const Pair* v, float top) {  // 8 pairs
#pragma unroll
  for (int k = 0; k < 8; ++k) top = fmaxf(top, fmaxf(fabsf(lo_of(v[k])), fabsf(hi_of(v[k]))));
  return top;
}

// What a group's values are multiplied by for their codes, of s = 448 / their largest: 0 where s
// is infinite (a largest value of 0, or below 1.3e-36), as the scale 1 / s is; 0 * infinity
// would be a NaN code.
__device__ __forceinline__ float code_factor(float s) { return s <= 3.402823466e38f ? s : 0.f; }

// 16 values times mult in e4m3.
__device__ __forceinline__ uint4 codes16(const Pair* v, float mult) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    auto two = [&](Pair p) { return permute_detail::e4m3x2(__fmul_rn(lo_of(p), mult), __fmul_rn(hi_of(p), mult)); };
    w[k] = two(v[2 * k]) | (two(v[2 * k + 1]) << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// DX: the input's gradient. ACT: forward with SwiGLU, or the gradient through it.
// OUT8: results in fp8 with scales.
template <bool DX, typename T, bool ACT, bool OUT8>
__global__ void __launch_bounds__(kThreads, 1)
b128_kernel(const __grid_constant__ B128Args a, const __grid_constant__ CUtensorMap map_w,
            const __grid_constant__ RowMaps rows_map) {
  constexpr bool kGates = ACT && !DX;
  extern __shared__ __align__(1024) uint8_t dyn[];
  __shared__ Bars bars;
  __shared__ float s_top[OUT8 && kGates ? 2 * 2 * 128 : 1];
  __shared__ float s_few[OUT8 ? 2 * 8 * kFew : 1];  // [turn][warp][token]
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
  float* s_scales = reinterpret_cast<float*>(ring + kStages * kStageBytes);
  int* s_begin = reinterpret_cast<int*>(s_scales + kScaleRing * kScaleFloats);
  int* s_tile = s_begin + a.G + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  if (threadIdx.x == 0) {
    prefetch_map(&map_w);
    prefetch_map(&rows_map.b128);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars.full[s], 1);
      mbar_init(&bars.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars.tfull[b], 1);
      mbar_init(&bars.tempty[b], kDrainWarps * 2);
    }
    for (int q = 0; q < 4; ++q) mbar_init(&bars.top[q], 2);
    for (int h = 0; h < 2; ++h) mbar_init(&bars.few_top[h], 8);
    for (int s = 0; s < kScaleRing; ++s) {
      mbar_init(&bars.sfull[s], 64);
      mbar_init(&bars.sempty[s], kDrainWarps);
    }
    mbar_init(&bars.done, 1);
    async::mbar_fence_init();
  }
  if (warp == 1) tmem_alloc(&bars.tmem, kTmemCols);
  // No early release of the next kernel: the permute kernel reads token rows before its
  // own wait, and they may be these results.
  griddep_wait();
  const bool bad = group_scan<kThreads>(a, s_begin, s_tile, [&](int rows) { return a.tiles_i * parts_of(rows); });
  if (bad && blockIdx.x == 0) atomicOr(&g_status, (uint32_t)CQ_ST_BAD_ROWS);
  fence_before();
  cluster_sync();
  fence_after();
  const uint32_t tmem = bars.tmem;
  const int n_tiles = s_tile[a.G];
  const int first = blockIdx.x / 2, step = gridDim.x / 2;
  // One verdict for the warp: the lanes go on to elect.sync and to .aligned instructions.
  auto wait = [&](uint64_t* bar, uint32_t parity, bool pair = false) {
    for (int r = 0; r < 2; ++r)
      if (pair ? wait_pair(bar, parity) : mbar_wait_warp(bar, parity)) return true;
    atomicOr(&g_status, (uint32_t)CQ_ST_TIMEOUT);
    return false;
  };
  auto lead = [&](uint64_t* bar) { return leader_addr(smem_u32(bar)); };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 0) {
      // ---- copies ----
      uint32_t s = 0, lap = 0;  // stage, times the ring has gone round
      bool ok = true;
      for (int t = first; t < n_tiles && ok; t += step) {
        const Tile x = tile_at<kGates, OUT8>(a, s_begin, s_tile, t);
        // tokens: each CTA its half, in copies of 128 rows, 64, 32, or 64 + 32
        const int jh = x.jh, row = x.row0 + (int)rank * jh;
        const bool b128 = jh > 96, b64 = !b128 && jh > 32, b32 = !b128 && (jh <= 32 || jh > 64);
        const uint32_t bytes = kABytes + (b128 ? 16384 : (b64 ? 8192 : 0) + (b32 ? 4096 : 0));
        const int i = x.i0 + (int)rank * x.cols / (kGates ? 4 : 2);  // this CTA's half of the columns
        int half = 0, k0 = 0;
        for (int kb = 0; kb < a.blocks; ++kb) {
          if (lap > 0 && !(ok = wait(&bars.empty[s], (lap & 1) ^ 1))) break;
          if (elect_one()) {
            const uint32_t sa = smem_u32(ring + s * kStageBytes), sb = sa + kABytes;
            const uint32_t bar = lead(&bars.full[s]);
            if (rank == 0) mbar_arrive_expect_tx(&bars.full[s], bytes * 2);
            if constexpr (kGates) tma_load5(sb, &map_w, k0, 0, 0, i / 16, x.e, bar);
            else if constexpr (DX) tma_load4<2>(sb, &map_w, i, k0, half, x.e, bar);
            else tma_load3<2>(sb, &map_w, k0, i, x.e, bar);
            if (b128) tma_load3<2>(sa, &rows_map.b128, k0, half, row, bar);
            if (b64) tma_load3<2>(sa, &rows_map.b64, k0, half, row, bar);
            if (b32) tma_load3<2>(sa + (b64 ? 8192 : 0), &rows_map.b32, k0, half, row + (b64 ? 64 : 0), bar);
          }
          __syncwarp();
          k0 += 128;
          if (k0 >= a.half_blocks * 128) k0 = 0, ++half;
          if (++s == kStages) s = 0, ++lap;
        }
      }
      // The last use of every stage, oldest first: nothing may arrive here after the CTA
      // has gone. Gave up: let the copies in flight land (with a limit) before it goes; those
      // of both CTAs complete on the leader's barrier, for which the other CTA stays.
      for (int v = 0; v < kStages; ++v) {
        const uint32_t u = (s + v) % kStages, laps = lap + (u < s ? 1 : 0);  // uses of stage u
        if (laps == 0) continue;
        if (ok) ok = wait(&bars.empty[u], (laps - 1) & 1);
        if (!ok && rank == 0) mbar_wait(&bars.full[u], (laps - 1) & 1);
      }
    } else if (warp == 1 && rank == 0) {
      // ---- products ----
      constexpr uint32_t ka = 32 >> 4, kbs = (DX ? 4096 : 32) >> 4;
      const uint64_t da = desc_at(desc_base(16), smem_u32(ring));
      const uint64_t db = desc_at(desc_base(16), smem_u32(ring) + kABytes);
      uint32_t s = 0, lap = 0, buf = 0;
      bool ok = true;
      for (int t = first; t < n_tiles && ok; t += step) {
        const Tile x = tile_at<kGates, OUT8>(a, s_begin, s_tile, t);
        const int xf = a.x_dtype == kMxE5M2, wf = a.w_dtype;
        const uint32_t idesc = x.few ? idesc_fp8(wf, xf, DX, false, 256, 2 * x.jh) : idesc_fp8(xf, wf, false, DX, 256, x.cols);
        const uint64_t first_op = x.few ? db : da, second_op = x.few ? da : db;
        const uint32_t k1 = x.few ? kbs : ka, k2 = x.few ? ka : kbs;
        int left = a.half_len;
        for (int kb = 0; kb < a.blocks; ++kb) {
          const uint32_t b = buf & 1, use = buf >> 1;
          ++buf;
          if (use > 0 && !(ok = wait(&bars.tempty[b], (use - 1) & 1, true))) break;
          if (!(ok = wait(&bars.full[s], lap & 1))) break;
          fence_after();
          if (elect_one()) {
            const uint64_t ad = first_op + s * (kStageBytes >> 4), bd = second_op + s * (kStageBytes >> 4);
            const uint32_t d = tmem + b * kNT;
            if (left > 96) {
              mma_fp8(d, ad, bd, idesc, false);
              mma_fp8(d, ad + k1, bd + k2, idesc, true);
              mma_fp8(d, ad + 2 * k1, bd + 2 * k2, idesc, true);
              mma_fp8(d, ad + 3 * k1, bd + 3 * k2, idesc, true);
            } else {
              for (int q = 0; 32 * q < left; ++q) mma_fp8(d, ad + q * k1, bd + q * k2, idesc, q > 0);
            }
            commit(smem_u32(&bars.empty[s]));
            commit(smem_u32(&bars.tfull[b]));
          }
          __syncwarp();
          left -= 128;
          if (left <= 0) left = a.half_len;
          if (++s == kStages) s = 0, ++lap;
        }
      }
      if (!ok) {  // gave up: let the products in flight end (with a limit), which read both CTAs' memory
        if (elect_one()) commit(smem_u32(&bars.done));
        __syncwarp();
        wait_pair(&bars.done, 0);
      }
    } else if (warp >= 2) {
      // ---- scales, four blocks an entry: of this CTA's tokens (tokens on the columns: of all),
      // and of the weights the two blocks of columns, or gates' and ups'. What is not there
      // keeps what the memory held: no stored result meets it ----
      const int l64 = (warp - 2) * 32 + lane;
      const uint32_t base = smem_u32(s_scales);
      uint32_t s = 0, lap = 0;
      bool ok = true;
      for (int t = first; t < n_tiles && ok; t += step) {
        const Tile x = tile_at<kGates, OUT8>(a, s_begin, s_tile, t);
        const int j0 = x.few ? 0 : (int)rank * x.jh, rows = x.few ? x.rows : rank ? x.rows - x.jh : x.jh;
        const float* xs = a.xs + (size_t)(x.row0 + j0 + l64) * a.blocks;
        const int k = lane >> 1, which = lane & 1, ib = x.i0 / 128 + (kGates ? 0 : which);
        const bool weights = warp == 2 && lane < 2 * kEntry && ib * 128 < a.out_cols;
        const float* ws = DX ? a.ws + ((size_t)x.e * a.blocks + k) * a.kb + ib
                             : a.ws + ((size_t)x.e * (kGates ? 2 * a.nb : a.nb) + (kGates ? which * a.nb : 0) + ib) * a.kb + k;
        for (int b0 = 0; b0 < a.blocks; b0 += kEntry) {
          if (lap > 0 && !(ok = wait(&bars.sempty[s], (lap & 1) ^ 1))) break;
          const uint32_t to = base + s * kScaleFloats * 4;
          const int nb = min(kEntry, a.blocks - b0);
#pragma unroll
          for (int m = 0; m < 2; ++m)
            if (l64 + 64 * m < rows)
              for (int c = 0; c < nb; ++c)
                copy4_async(to + (c * 128 + l64 + 64 * m) * 4, xs + (size_t)(64 * m) * a.blocks + b0 + c);
          if (weights && k < nb) copy4_async(to + (kEntry * 128 + lane) * 4, ws + (size_t)b0 * (DX ? a.kb : 1));
          arrive_on_copies(&bars.sfull[s]);
          if (++s == kScaleRing) s = 0, ++lap;
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    // ---- scaled sums, and results ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kDrainRegs));
    const int q = warp & 3, half = (warp - 4) >> 2;
    const bool wide = a.wide;
    uint32_t buf = 0, se = 0, se_lap = 0, nth = 0, nth_few = 0;  // tiles so far, of either kind
    // what a warp does for every block is kept short: longer code is fetched too slowly
    const uint32_t release[2] = {lead(&bars.tempty[0]), lead(&bars.tempty[1])};
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
    bool ok = true;
    for (int t = first; t < n_tiles && ok; t += step) {
      const Tile x = tile_at<kGates, OUT8>(a, s_begin, s_tile, t);
      if (x.few) {
        // ---- tokens on the columns, weight rows on the lanes ----
        const int c0 = half * x.jh, chunks = (x.jh + 15) / 16;  // this warp's columns, 16 a chunk
        Pair sum[4][8];
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
          for (int k = 0; k < 8; ++k) sum[m][k] = 0;
        const int l = 32 * q + lane;
        // this lane's of an entry's two weights
        const int which = kGates ? lane >> 4 : (x.i0 + (int)rank * x.cols / 2 + l) / 128 - x.i0 / 128;
        for (int b0 = 0; b0 < a.blocks && ok; b0 += kEntry) {
          if (!(ok = wait(&bars.sfull[se], se_lap & 1))) break;
          const float* sc = s_scales + se * kScaleFloats;
          const int nb = min(kEntry, a.blocks - b0);
#pragma unroll 1
          for (int k = 0; k < nb; ++k) {
            const uint32_t b = buf & 1;
            const float w = sc[kEntry * 128 + 2 * k + which];
            const Pair pw = pair_of(w, w);
            const uint32_t xs = smem_u32(sc + k * 128 + c0), src = lanes + b * kNT + c0;
            if (!(ok = wait(&bars.tfull[b], (buf >> 1) & 1))) break;
            ++buf;
            fence_after();
#pragma unroll
            for (int m = 0; m < 2; ++m) {  // 32 columns
              if (2 * m >= chunks) break;
              uint32_t v[32];
              tmem_ld32(src + 32 * m, v);
              tmem_wait();
              if (2 * m + 2 >= chunks) {  // the accumulator is read
                fence_before();
                __syncwarp();
                if (lane == 0) arrive_cluster_relaxed(release[b]);
              }
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                if (2 * m + h >= chunks) break;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  Pair s0, s1;
                  ld_pairs(xs + (32 * m + 16 * h + 4 * i) * 4, s0, s1);
                  Pair(&to)[8] = sum[2 * m + h];
                  to[2 * i] = fma2(pair_of(v[16 * h + 4 * i], v[16 * h + 4 * i + 1]), mul2(s0, pw), to[2 * i]);
                  to[2 * i + 1] = fma2(pair_of(v[16 * h + 4 * i + 2], v[16 * h + 4 * i + 3]), mul2(s1, pw), to[2 * i + 1]);
                }
              }
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.sempty[se]);
          if (++se == kScaleRing) se = 0, ++se_lap;
        }
        if (!ok) break;
        // Lanes lie along the results' rows: 2 bytes each, 64 (SwiGLU: 32) together.
        const int i = kGates ? x.i0 + (int)rank * x.cols / 4 + 16 * q + (lane & 15) : x.i0 + (int)rank * x.cols / 2 + l;
        const bool in = l < x.cols / 2 && i < a.out_cols;
        if constexpr (OUT8) {
          // The largest value of each token's group: over the lanes, then over the quarters and
          // (one group on both CTAs' lanes) the CTAs. Every warp tells both CTAs. Two buffers by
          // the tiles' turn: who writes the next but one has seen all arrive for the next, and
          // they had read this one.
          const bool joint = kGates || x.cols <= 128, mine = in && (!kGates || lane < 16);
          float* tb = s_few + (nth_few & 1) * 8 * kFew + c0;
          const int from = joint ? (int)rank * 4 + q : q;
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            if (m >= chunks) break;
            float tops = 0.f;  // of token 16 m + lane
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              Pair& p = sum[m][k / 2];
              float v = k & 1 ? hi_of(p) : lo_of(p);
              if constexpr (kGates) {
                const float u = __shfl_xor_sync(~0u, v, 16);
                if (a.pre_out && in && 16 * m + k < x.jh && c0 + 16 * m + k < x.rows)
                  static_cast<uint16_t*>(a.pre_out)[((size_t)x.row0 + c0 + 16 * m + k) * 2 * a.n + (lane >= 16 ? a.n : 0) + i] =
                      (uint16_t)T::pack2(v, 0.f);
                v = swiglu(v, u);  // of use in lanes 0-15
                p = k & 1 ? pair_of(lo_of(p), v) : pair_of(v, hi_of(p));
              }
              const float t = permute_detail::warp_max(mine ? fabsf(v) : 0.f);
              if (lane == k) tops = t;
            }
            if (lane < 16 && 16 * m + lane < x.jh) {
              tb[from * kFew + 16 * m + lane] = tops;
              if (joint)
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr_in(smem_u32(tb + from * kFew + 16 * m + lane), rank ^ 1)),
                             "f"(tops)
                             : "memory");
            }
          }
          __syncwarp();
          if (lane == 0) {
            arrive_cluster(addr_in(smem_u32(&bars.few_top[half]), rank ^ 1));
            arrive_cluster(addr_in(smem_u32(&bars.few_top[half]), rank));
          }
          if (!(ok = wait(&bars.few_top[half], nth_few & 1, true))) break;
          ++nth_few;
          uint8_t* out = static_cast<uint8_t*>(a.out) + ((size_t)x.row0 + c0) * a.out_cols + i;
          const int group = joint ? x.i0 / 128 : x.i0 / 128 + (int)rank;
          const bool writes = q == 0 && (!joint || rank == 0) && group < a.nb;
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            if (m >= chunks) break;
            const int j = 16 * m + (lane & 15);
            float top = 0.f;
            if (j < x.jh)
              for (int w = 0; w < (joint ? 8 : 4); ++w) top = fmaxf(top, tb[w * kFew + j]);
            const float s = __fdiv_rn(448.f, top), mult = code_factor(s);
            if (writes && lane < 16 && j < x.jh && c0 + j < x.rows) a.ys[((size_t)x.row0 + c0 + j) * a.nb + group] = __fdiv_rn(1.f, s);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float v = k & 1 ? hi_of(sum[m][k / 2]) : lo_of(sum[m][k / 2]);
              const float f = __shfl_sync(~0u, mult, k);
              if (mine && 16 * m + k < x.jh && c0 + 16 * m + k < x.rows)
                out[(size_t)(16 * m + k) * a.out_cols] = (uint8_t)permute_detail::e4m3x2(__fmul_rn(v, f), 0.f);
            }
          }
          continue;
        }
        const int count = in ? min(x.jh, x.rows - c0) : 0;  // of this warp's tokens
        const size_t ld = kGates || (DX && ACT) ? 2 * (size_t)a.out_cols : a.out_cols;
        const size_t at = ((size_t)x.row0 + c0) * ld + i;
        uint16_t* out = static_cast<uint16_t*>(a.out) + (kGates ? ((size_t)x.row0 + c0) * a.n + i : at);
        uint16_t* pre = static_cast<uint16_t*>(kGates ? a.pre_out : const_cast<void*>(a.pre_in)) + at + (kGates && lane >= 16 ? a.n : 0);
        const bool saves = kGates && a.pre_out;
        // saved products of 16 tokens, gates' in the lower half, read together (one after the
        // other, each waited for HBM: 48 experts of 35 rows, n 800, k 4832: 211 us, now 101)
        uint32_t saved[16];
        auto load = [&](int m) {
          if constexpr (DX && ACT) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const uint16_t* p = pre + (size_t)(16 * m + k) * ld;
              saved[k] = 16 * m + k < count ? __ldg(p) | (uint32_t)__ldg(p + a.out_cols) << 16 : 0;
            }
          }
        };
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          if (m >= chunks) break;
          load(m);
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float v = k & 1 ? hi_of(sum[m][k / 2]) : lo_of(sum[m][k / 2]);
            const bool here = 16 * m + k < count;
            if constexpr (kGates) {
              const float u = __shfl_xor_sync(~0u, v, 16);
              if (here && saves) *pre = (uint16_t)T::pack2(v, 0.f);
              if (here && lane < 16) *out = (uint16_t)T::pack2(swiglu(v, u), 0.f);
              pre += ld;
              out += a.n;
            } else if constexpr (DX && ACT) {
              if (here) {
                float dg, du;
                swiglu_gradient(v, T::lo(saved[k]), T::hi(saved[k]), dg, du);
                out[0] = (uint16_t)T::pack2(dg, 0.f);
                out[a.out_cols] = (uint16_t)T::pack2(du, 0.f);
              }
              out += ld;
            } else {
              if (here) *out = (uint16_t)T::pack2(v, 0.f);
              out += ld;
            }
          }
        }
        continue;
      }
      const int jh = x.jh, rows = rank ? x.rows - jh : jh;  // of this CTA
      // chunks of 32 columns of this warp's 128; none where its lanes hold no tokens
      const int chunks = 32 * q < rows ? min(4, max(0, (x.cols - 128 * half + 31) / 32)) : 0;
      Pair acc[4][16];
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int k = 0; k < 16; ++k) acc[m][k] = 0;
      for (int b0 = 0; b0 < a.blocks && ok; b0 += kEntry) {
        if (!(ok = wait(&bars.sfull[se], se_lap & 1))) break;
        const float* sc = s_scales + se * kScaleFloats;
        const int nb = min(kEntry, a.blocks - b0);
#pragma unroll 1
        for (int k = 0; k < nb; ++k) {
          const uint32_t b = buf & 1;
          const float xv = sc[k * 128 + 32 * q + lane];
          const float* wc = sc + kEntry * 128 + 2 * k;
          const float sg = xv * wc[kGates ? 0 : half], su = kGates ? xv * wc[1] : sg;
          const Pair pg = pair_of(sg, sg), pu = pair_of(su, su);
          const uint32_t src = lanes + b * kNT + 128 * half;
          if (!(ok = wait(&bars.tfull[b], (buf >> 1) & 1))) break;
          ++buf;
          fence_after();
          if (chunks > 0) {
            uint32_t v[32];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              tmem_ld32(src + 32 * m, v);
              tmem_wait();
              if (m == 3) {
                fence_before();
                __syncwarp();
                if (lane == 0) arrive_cluster_relaxed(release[b]);
              }
              add_scaled(v, pg, pu, acc[m]);
            }
          } else {
            __syncwarp();
            if (lane == 0) arrive_cluster_relaxed(release[b]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.sempty[se]);
        if (++se == kScaleRing) se = 0, ++se_lap;
      }
      if (!ok) break;
      const int j = 32 * q + lane;
      const bool real = j < rows;
      const size_t row = (size_t)(x.row0 + (int)rank * jh + j);
      if constexpr (kGates) {
        const int o0 = x.i0 + 64 * half;  // a chunk is 16 outputs
        float top = 0.f;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          if (m >= chunks) break;
          const int o = o0 + 16 * m;
          const bool in = real && o < a.n;
          if (a.pre_out && in) {
            uint16_t* pre = static_cast<uint16_t*>(a.pre_out) + row * 2 * a.n + o;
            store16<T>(pre, acc[m], wide);
            store16<T>(pre + a.n, acc[m] + 8, wide);
          }
#pragma unroll
          for (int k = 0; k < 8; ++k)
            acc[m][k] = pair_of(swiglu(lo_of(acc[m][k]), lo_of(acc[m][8 + k])),
                                swiglu(hi_of(acc[m][k]), hi_of(acc[m][8 + k])));
          if constexpr (OUT8) {
            if (o < a.n) top = top_of(acc[m], top);
          } else if (in) {
            store16<T>(static_cast<uint16_t*>(a.out) + row * a.n + o, acc[m], wide);
          }
        }
        if constexpr (OUT8) {
          // The other half of the group's outputs is with the other warp of this quarter.
          // Two buffers by the tiles' turn: who writes the next but one has seen the other
          // arrive for the next, and that one had read this one.
          float* tb = s_top + (nth & 1) * 256 + 32 * q + lane;
          tb[128 * half] = top;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.top[q]);
          if (!(ok = wait(&bars.top[q], nth & 1))) break;
          top = fmaxf(top, tb[128 * (half ^ 1)]);
          const float s = __fdiv_rn(448.f, top), mult = code_factor(s);
          if (half == 0 && real) a.ys[row * a.nb + x.i0 / 128] = __fdiv_rn(1.f, s);
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const int o = o0 + 16 * m;
            if (m >= chunks || !real || o >= a.n) break;
            *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + row * a.n + o) = codes16(acc[m], mult);
          }
        }
      } else {
        const int i0 = x.i0 + 128 * half, left = real ? a.out_cols - i0 : 0;
        if constexpr (DX && ACT) {
          const uint16_t* pre = static_cast<const uint16_t*>(a.pre_in) + row * 2 * a.out_cols + i0;
          uint16_t* out = static_cast<uint16_t*>(a.out) + row * 2 * a.out_cols + i0;
          uint32_t g[2][8], u[2][8];  // the next 16 columns' are read ahead
          auto load = [&](int k) {
            if (32 * chunks <= 16 * k || 16 * k >= left) return;
            load32(pre + 16 * k, g[k & 1], wide);
            load32(pre + a.out_cols + 16 * k, u[k & 1], wide);
          };
          load(0);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (k + 1 < 8) load(k + 1);
            if (32 * chunks <= 16 * k || 16 * k >= left) continue;
            uint32_t(&gk)[8] = g[k & 1];
            uint32_t(&uk)[8] = u[k & 1];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const Pair d = acc[k / 2][8 * (k & 1) + c];
              float dg0, du0, dg1, du1;
              swiglu_gradient(lo_of(d), T::lo(gk[c]), T::lo(uk[c]), dg0, du0);
              swiglu_gradient(hi_of(d), T::hi(gk[c]), T::hi(uk[c]), dg1, du1);
              gk[c] = T::pack2(dg0, dg1);
              uk[c] = T::pack2(du0, du1);
            }
            store32(out + 16 * k, gk, wide);
            store32(out + a.out_cols + 16 * k, uk, wide);
          }
        } else if constexpr (OUT8) {
          float top = 0.f;
#pragma unroll
          for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (m < chunks && 32 * m + 16 * h < left) top = top_of(acc[m] + 8 * h, top);
          const float s = __fdiv_rn(448.f, top), mult = code_factor(s);
          if (left > 0) a.ys[row * a.nb + i0 / 128] = __fdiv_rn(1.f, s);
          uint8_t* out = static_cast<uint8_t*>(a.out) + row * a.out_cols + i0;
#pragma unroll
          for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (m < chunks && 32 * m + 16 * h < left)
                *reinterpret_cast<uint4*>(out + 32 * m + 16 * h) = codes16(acc[m] + 8 * h, mult);
        } else {
          uint16_t* out = static_cast<uint16_t*>(a.out) + row * a.out_cols + i0;
#pragma unroll
          for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (m < chunks && 32 * m + 16 * h < left) store16<T>(out + 32 * m + 16 * h, acc[m] + 8 * h, wide);
        }
      }
      ++nth;
    }
  }
  __syncwarp();
  fence_before();
  cluster_sync();
  fence_after();
  if (warp == 1) tmem_free(tmem, kTmemCols);
}

// ---- host ----
template <bool DX, typename T, bool ACT, bool OUT8>
cudaError_t launch_t(const B128Args& a, const CUtensorMap& mw, const RowMaps& mr, cudaStream_t s) {
  constexpr auto kernel = b128_kernel<DX, T, ACT, OUT8>;
  const size_t smem = 1024 + kStages * kStageBytes + kScaleRing * kScaleFloats * 4 + 8 * ((size_t)a.G + 1);
  cudaError_t e = prepare_kernel<kernel>(smem);
  if (e == cudaSuccess) e = check_registers<kernel>(kThreads, kAllRegs);
  if (e != cudaSuccess) return e;
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorUnknown;
  const int64_t most = (int64_t)a.tiles_i * (a.R / 256 + std::min(a.G, a.R));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(sms / 2, most) * 2);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {2, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a, mw, mr);
}

template <typename T>
cudaError_t launch_type(bool dx, B128Args& a, cudaStream_t s) {
  const uint64_t G = a.G, R = a.R, N = a.N, K = a.K, n = a.n, halves = N / n;
  const bool act = a.act && !dx;
  CUtensorMap mw;
  RowMaps mr;
  a.blocks = dx ? (int)halves * a.nb : a.kb;
  a.half_blocks = dx ? a.nb : a.kb;
  a.half_len = dx ? a.n : a.K;
  a.out_cols = dx ? a.K : a.n;
  a.tiles_i = act ? a.nb : (a.out_cols + 255) / 256;
  auto whole = [](const void* p, int64_t row, int unit) { return (reinterpret_cast<uintptr_t>(p) | row) % unit == 0; };
  // every 16 values of a result's row begin on 32 bytes if the first do
  a.wide = whole(a.out, 0, 32) && whole(a.pre_in, 0, 32) && whole(a.pre_out, 0, 32);
  {  // rows: of both halves side by side for dx
    const uint64_t len = a.half_len, h = dx ? halves : 1, d[] = {len, h, R}, st[] = {len, len * h};
    const uint32_t b[] = {128, 1, 128}, b64[] = {128, 1, 64}, b32[] = {128, 1, 32};
    if (!make_map(&mr.b128, a.x, kMapU8, 3, d, st, b) || !make_map(&mr.b64, a.x, kMapU8, 3, d, st, b64) ||
        !make_map(&mr.b32, a.x, kMapU8, 3, d, st, b32))
      return cudaErrorUnknown;
  }
  if (dx) {
    const uint64_t d[] = {K, n, halves, G}, st[] = {K, n * K, N * K};
    const uint32_t b[] = {128, 128, 1, 1};
    if (!make_map(&mw, a.w, kMapU8, 4, d, st, b)) return cudaErrorUnknown;
    return a.pre_in ? launch_t<true, T, true, false>(a, mw, mr, s) : launch_t<true, T, false, false>(a, mw, mr, s);
  }
  if (act) {  // columns: 16 gates, 16 ups, 16 gates, ...
    const uint64_t d[] = {K, 16, 2, n / 16, G}, st[] = {K, n * K, 16 * K, N * K};
    const uint32_t b[] = {128, 16, 2, 4, 1};
    if (!make_map(&mw, a.w, kMapU8, 5, d, st, b)) return cudaErrorUnknown;
    return a.ys ? launch_t<false, T, true, true>(a, mw, mr, s) : launch_t<false, T, true, false>(a, mw, mr, s);
  }
  const uint64_t d[] = {K, N, G}, st[] = {K, N * K};
  const uint32_t b[] = {128, 128, 1};
  if (!make_map(&mw, a.w, kMapU8, 3, d, st, b)) return cudaErrorUnknown;
  return a.ys ? launch_t<false, T, false, true>(a, mw, mr, s) : launch_t<false, T, false, false>(a, mw, mr, s);
}

int validate(const cq_expert_config* c) {
  if (!c) return CQ_ERR_ARG;
  cq_expert_config m = *c;  // the mx types' rules, but for k
  if (c->x_dtype < kMxE4M3 || c->out_dtype == 2) return CQ_ERR_ARG;
  if (c->k % 16 == 0 && c->k >= 16) m.k = 32;
  if (c->k > 65536) return CQ_ERR_ARG;
  return cq_check_expert_config(&m);
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

B128Args base_args(const cq_expert_config* c, const int64_t* group_rows) {
  B128Args a = {};
  a.G = c->experts;
  a.R = c->rows;
  a.N = c->act ? 2 * c->n : c->n;
  a.K = c->k;
  a.x_dtype = c->x_dtype;
  a.w_dtype = c->w_dtype;
  a.out_dtype = c->out_dtype == 1 ? 1 : 0;
  a.act = c->act;
  a.rows_type = c->rows_type;
  a.L = c->experts_per_rank;
  a.group_rows = group_rows;
  a.n = c->n;
  a.nb = (c->n + 127) / 128;
  a.kb = (c->k + 127) / 128;
  return a;
}

int launch(bool dx, B128Args& a, cudaStream_t s) {
  if (a.R == 0) return CQ_OK;
  const cudaError_t e = a.out_dtype ? launch_type<F16>(dx, a, s) : launch_type<BF16>(dx, a, s);
  return e == cudaSuccess ? CQ_OK : CQ_ERR_CUDA;
}

}  // namespace

int b128_status(uint32_t* read, cudaStream_t s) { return status_word(g_status, read, s); }

}  // namespace expert
}  // namespace cq

using namespace cq::expert;

extern "C" {

int cq_check_expert_b128_config(const cq_expert_config* cfg) { return validate(cfg); }

int cq_expert_matmul_b128(const cq_expert_config* cfg, const void* x, const float* x_scales,
                          const void* w, const float* w_scales, const int64_t* group_rows, void* y,
                          float* y_scales, void* pre, void* stream) {
  const int rc = validate(cfg);
  if (rc != CQ_OK) return rc;
  const bool rows = cfg->rows > 0;
  if ((rows && (!x || !x_scales || !y)) || !w || !w_scales || !group_rows) return CQ_ERR_ARG;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(y, 16) || !aligned(pre, 16) ||
      !aligned(x_scales, 4) || !aligned(w_scales, 4) || !aligned(y_scales, 4) || !aligned(group_rows, 8))
    return CQ_ERR_ARG;
  if (pre && cfg->act != 1) return CQ_ERR_ARG;
  B128Args a = base_args(cfg, group_rows);
  a.x = x;
  a.w = w;
  a.xs = x_scales;
  a.ws = w_scales;
  a.out = y;
  a.ys = y_scales;
  a.pre_out = pre;
  return launch(false, a, static_cast<cudaStream_t>(stream));
}

int cq_expert_matmul_b128_dx(const cq_expert_config* cfg, const void* dy, const float* dy_scales,
                             const void* w, const float* w_scales, const int64_t* group_rows,
                             const void* pre, void* dx, void* stream) {
  const int rc = validate(cfg);
  if (rc != CQ_OK) return rc;
  const bool rows = cfg->rows > 0;
  if ((rows && (!dy || !dy_scales || !dx)) || !w || !w_scales || !group_rows) return CQ_ERR_ARG;
  if (!aligned(dy, 16) || !aligned(w, 16) || !aligned(dx, 16) || !aligned(pre, 16) ||
      !aligned(dy_scales, 4) || !aligned(w_scales, 4) || !aligned(group_rows, 8))
    return CQ_ERR_ARG;
  B128Args a = base_args(cfg, group_rows);
  a.x = dy;
  a.w = w;
  a.xs = dy_scales;
  a.ws = w_scales;
  a.pre_in = pre;
  a.out = dx;
  return launch(true, a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
