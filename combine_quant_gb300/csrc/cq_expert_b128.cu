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
// 128 sums a thread, all of a tile. That is what bounds it, and why tokens lie on the
// accumulator's lanes here (up to 128 in each CTA) and weight rows on its columns: a
// lane's factor is one number per 128 columns. With tokens on the columns the factors
// are a vector to be read for every block (measured: 813 us where this takes XX, at 512
// rows an expert), though a ragged expert then wastes no lanes.
//
// SwiGLU: the columns are 16 gates, 16 ups, 16 gates, ... (one 5-D copy). fp8 results:
// a group of 128 outputs is a thread's own columns, with SwiGLU those of two threads.
// dx: B = w with its columns along N (MN-major), the contraction runs over n.
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
  int32_t vec;          // rows of xs are whole 16-byte pieces
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
static_assert(128 * kOtherRegs + 32 * kDrainWarps * kDrainRegs <= 168 * kThreads, "setmaxnreg would wait forever");
constexpr uint32_t kTmemCols = 512;
constexpr int kBand = 8;                   // tiles along i taken together, for reuse in L2

struct RowMaps {
  CUtensorMap b128, b64, b32;
};

struct Bars {
  uint64_t full[kStages], empty[kStages];
  uint64_t tfull[2], tempty[2];
  uint64_t top[4];  // fp8 results: the largest values of a quarter's two warps
  uint64_t done;    // the products in flight when their warp gave up
  uint32_t tmem;
};

struct Tile {
  int e, row0, rows;  // first token row and rows of the tile
  int i0, cols;       // first output and accumulator columns (of B, both CTAs)
};

// GATES: a tile is 128 outputs, else 256. Columns in steps of 64 (16 outputs a CTA) or 32.
template <bool GATES>
__device__ __forceinline__ Tile tile_at(const B128Args& a, const int* s_begin, const int* s_tile, int t) {
  Tile x;
  x.e = expert_of(s_tile, a.G, t);
  const int l = t - s_tile[x.e];
  const int begin = s_begin[x.e], rows = s_begin[x.e + 1] - begin;
  const int parts = (rows + 255) / 256;
  const int band = l / (kBand * parts), first_i = band * kBand;
  const int wide = min(kBand, a.tiles_i - first_i), m = l - first_i * parts;
  const int ti = first_i + m % wide, tj = m / wide;
  const int step = (rows + parts - 1) / parts;  // equal parts
  x.row0 = begin + tj * step;
  x.rows = min(step, rows - tj * step);
  constexpr int kOuts = GATES ? 128 : 256;
  x.i0 = ti * kOuts;
  const int outs = (min(kOuts, a.out_cols - x.i0) + 31) / 32 * 32;
  x.cols = GATES ? 2 * outs : outs;
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
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
  int* s_begin = reinterpret_cast<int*>(ring + kStages * kStageBytes);
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
    mbar_init(&bars.done, 1);
    async::mbar_fence_init();
  }
  if (warp == 1) tmem_alloc(&bars.tmem, kTmemCols);
  // No early release of the next kernel: the permute kernel reads token rows before its
  // own wait, and they may be these results.
  griddep_wait();
  const bool bad = group_scan<kThreads>(
      a, s_begin, s_tile, [&](int rows) { return a.tiles_i * ((rows + 255) / 256); });
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
        const Tile x = tile_at<kGates>(a, s_begin, s_tile, t);
        // tokens: each CTA its half, in copies of 128 rows, 64, 32, or 64 + 32
        const int jh = (x.rows + 1) / 2, row = x.row0 + (int)rank * jh;
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
        const Tile x = tile_at<kGates>(a, s_begin, s_tile, t);
        const uint32_t idesc = idesc_fp8(a.x_dtype == kMxE5M2, a.w_dtype, DX, 256, x.cols);
        int left = a.half_len;
        for (int kb = 0; kb < a.blocks; ++kb) {
          const uint32_t b = buf & 1, use = buf >> 1;
          ++buf;
          if (use > 0 && !(ok = wait(&bars.tempty[b], (use - 1) & 1, true))) break;
          if (!(ok = wait(&bars.full[s], lap & 1))) break;
          fence_after();
          if (elect_one()) {
            const uint64_t ad = da + s * (kStageBytes >> 4), bd = db + s * (kStageBytes >> 4);
            const uint32_t d = tmem + b * kNT;
            if (left > 96) {
              mma_fp8(d, ad, bd, idesc, false);
              mma_fp8(d, ad + ka, bd + kbs, idesc, true);
              mma_fp8(d, ad + 2 * ka, bd + 2 * kbs, idesc, true);
              mma_fp8(d, ad + 3 * ka, bd + 3 * kbs, idesc, true);
            } else {
              for (int q = 0; 32 * q < left; ++q) mma_fp8(d, ad + q * ka, bd + q * kbs, idesc, q > 0);
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
    }
  } else {
    // ---- scaled sums, and results ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kDrainRegs));
    const int q = warp & 3, half = (warp - 4) >> 2;
    const bool wide = a.wide;
    uint32_t buf = 0, nth = 0;  // nth: tiles so far
    // Factors of four blocks, read four blocks ahead: the row's, and the weights' in
    // lanes 0-3 (with SwiGLU the ups' in lanes 4-7).
    float4 xn = {};
    float wn = 0.f;
    auto fetch = [&](const Tile& x, int b0) {
      const int jh = (x.rows + 1) / 2, j = min((int)rank * jh + 32 * q + lane, x.rows - 1);
      const float* p = a.xs + (size_t)(x.row0 + j) * a.blocks + b0;
      const int left = a.blocks - b0;
      if (a.vec) {
        xn = __ldg(reinterpret_cast<const float4*>(p));
      } else {
        xn.x = __ldg(p);
        if (left > 1) xn.y = __ldg(p + 1);
        if (left > 2) xn.z = __ldg(p + 2);
        if (left > 3) xn.w = __ldg(p + 3);
      }
      const int k = lane & 3, which = lane >> 2;
      wn = 0.f;
      if (k >= left) return;
      if constexpr (kGates) {
        if (which < 2) wn = __ldg(a.ws + ((size_t)x.e * 2 * a.nb + which * a.nb + x.i0 / 128) * a.kb + b0 + k);
      } else {
        const int ib = x.i0 / 128 + half;  // the block of this warp's columns
        if (which == 0 && ib * 128 < a.out_cols)
          wn = __ldg(DX ? a.ws + ((size_t)x.e * a.blocks + b0 + k) * a.kb + ib
                        : a.ws + ((size_t)x.e * a.nb + ib) * a.kb + b0 + k);
      }
    };
    bool ok = true;
    Tile x = {}, next = {};
    if (first < n_tiles) {
      next = tile_at<kGates>(a, s_begin, s_tile, first);
      fetch(next, 0);
    }
    for (int t = first; t < n_tiles && ok; t += step) {
      x = next;
      const int jh = (x.rows + 1) / 2, rows = rank ? x.rows - jh : jh;  // of this CTA
      // chunks of 32 columns of this warp's 128; none where its lanes hold no tokens
      const int chunks = 32 * q < rows ? min(4, max(0, (x.cols - 128 * half + 31) / 32)) : 0;
      Pair acc[4][16];
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int k = 0; k < 16; ++k) acc[m][k] = 0;
      float4 xc = {};
      float wc = 0.f;
      for (int kb = 0; kb < a.blocks; ++kb) {
        const uint32_t b = buf & 1, use = buf >> 1;
        ++buf;
        if ((kb & 3) == 0) {
          xc = xn;
          wc = wn;
          if (kb + 4 < a.blocks) {
            fetch(x, kb + 4);
          } else if (t + step < n_tiles) {
            next = tile_at<kGates>(a, s_begin, s_tile, t + step);
            fetch(next, 0);
          }
        }
        const float sg = xc.x * __shfl_sync(~0u, wc, kb & 3);
        const float su = kGates ? xc.x * __shfl_sync(~0u, wc, 4 + (kb & 3)) : sg;
        const Pair pg = pair_of(sg, sg), pu = pair_of(su, su);
        xc.x = xc.y, xc.y = xc.z, xc.z = xc.w;
        if (!(ok = wait(&bars.tfull[b], use & 1))) break;
        fence_after();
        const uint32_t src = tmem + b * kNT + ((uint32_t)(q * 32) << 16) + 128 * half;
        uint32_t v[2][32];
        if (chunks > 0) tmem_ld32(src, v[0]);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          if (m >= chunks) break;
          tmem_wait();
          if (m + 1 < 4 && m + 1 < chunks) {
            tmem_ld32(src + 32 * (m + 1), v[(m + 1) & 1]);
          } else {  // the accumulator is read
            fence_before();
            __syncwarp();
            if (lane == 0) arrive_cluster_relaxed(lead(&bars.tempty[b]));
          }
          add_scaled(v[m & 1], pg, pu, acc[m]);
        }
        if (chunks == 0) {
          __syncwarp();
          if (lane == 0) arrive_cluster_relaxed(lead(&bars.tempty[b]));
        }
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
          const float s = __fdiv_rn(448.f, top), mult = top == 0.f ? 0.f : s;
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
#pragma unroll
          for (int m = 0; m < 4; ++m) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int c = 32 * m + 16 * h;
              if (m >= chunks || c >= left) break;
              uint32_t g[8], u[8];
              load32(pre + c, g, wide);
              load32(pre + a.out_cols + c, u, wide);
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const Pair d = acc[m][8 * h + k];
                float dg0, du0, dg1, du1;
                swiglu_gradient(lo_of(d), T::lo(g[k]), T::lo(u[k]), dg0, du0);
                swiglu_gradient(hi_of(d), T::hi(g[k]), T::hi(u[k]), dg1, du1);
                g[k] = T::pack2(dg0, dg1);
                u[k] = T::pack2(du0, du1);
              }
              store32(out + c, g, wide);
              store32(out + a.out_cols + c, u, wide);
            }
          }
        } else if constexpr (OUT8) {
          float top = 0.f;
#pragma unroll
          for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (m < chunks && 32 * m + 16 * h < left) top = top_of(acc[m] + 8 * h, top);
          const float s = __fdiv_rn(448.f, top), mult = top == 0.f ? 0.f : s;
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
  const size_t smem = 1024 + kStages * kStageBytes + 8 * ((size_t)a.G + 1);
  cudaError_t e = prepare_kernel<kernel>(smem);
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
  a.vec = whole(a.xs, 4 * (int64_t)a.blocks, 16);
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

int b128_status(uint32_t* status, cudaStream_t s) { return read_status_word(g_status, status, s); }

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
