// cq_expert_b128.cu -- expert products from fp8 rows with one scale per 128 columns
// and fp8 weights with one per 128 x 128 block, on the tensor cores (tcgen05):
// forward (SwiGLU, results in 16 bits or in fp8 with scales) and the gradient of
// the input.
//
// A persistent kernel on pairs of CTAs, as cq_expert_gemm.cu's: a tile is 256
// weight rows (the accumulator's lanes, 128 in each CTA) by up to 256 tokens (its
// columns, in steps of 16), copies by warp 0, products by warp 1 of the first CTA.
// What differs is that a scale holds for 128 of the contraction only:
//
//   acc[i, j] += (xs[j, B] ws[B]) * sum over k in B of w[i, k] x[j, k]
//
// So every stage (128 of the contraction, four products) goes into a TMEM
// accumulator of its own, two in turn, and eight warps take it from there into
// registers, scaled: 128 sums a thread, all of a tile. The scales of the columns are
// the vector: with lane r / 4 + 8 h of the accumulator and columns 8 n + 2 c + b a
// thread (16x256b loads) needs 32 scales for 128 sums, not 128 as it would with a
// lane each; pairs of columns multiply in packed f32x2 instructions. Warps 2 and 3
// fetch the scales, four blocks at a time; where a CTA's weight rows have one block
// scale it is multiplied in there, with SwiGLU (gate and up rows) by the reader.
//
// dx: A = w with its columns on the lanes (MN-major), the contraction runs over n.
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
  int32_t vec;          // rows of xs are whole 16-byte pieces
  int32_t I, tiles_i;   // rows of A: weight rows, or (dx) columns of w
};

constexpr int kNT = 256;                   // most columns of a tile
constexpr int kStages = 5;
constexpr int kABytes = 128 * 128;         // A of one stage, one CTA
constexpr int kStageBytes = 2 * kABytes;   // B: half of up to 256 columns
constexpr int kDrainWarps = 8;             // two for each quarter of the lanes
constexpr int kThreads = 128 + 32 * kDrainWarps;
// Registers: 384 threads are launched with 168 each (64512); the drain warps keep 128
// sums and need 224, the others 56, which is the same total.
constexpr int kOtherRegs = 56, kDrainRegs = 224;
static_assert(128 * kOtherRegs + 32 * kDrainWarps * kDrainRegs <= 168 * kThreads, "setmaxnreg would wait forever");
constexpr int kEntry = 4;                  // blocks in an entry of the scales' ring
constexpr int kScaleRing = 3;
constexpr int kScaleFloats = kEntry * kNT + 2 * kEntry;  // columns', then gates' and ups'
constexpr int kStaging = 16 * 33 * 4;      // bytes of a drain warp's staging buffer
constexpr uint32_t kTmemCols = 512;
constexpr int kBand = 8;                   // tiles along i taken together, for reuse in L2

struct FewMaps {
  CUtensorMap b64, b32;
};

struct Bars {
  uint64_t full[kStages], empty[kStages];
  uint64_t sfull[kScaleRing], sempty[kScaleRing];
  uint64_t tfull[2], tempty[2];
  uint64_t top[2];  // fp8 results: the columns' largest values of a half of the warps
  uint64_t done;    // the products in flight when their warp gave up
  uint32_t tmem;
};

struct Tile {
  int e, begin, i0, j0, jn;
};

__device__ __forceinline__ Tile tile_at(const B128Args& a, const int* s_begin, const int* s_tile, int t) {
  Tile x;
  x.e = expert_of(s_tile, a.G, t);
  const int l = t - s_tile[x.e];
  x.begin = s_begin[x.e];
  const int rows = s_begin[x.e + 1] - x.begin;
  const int parts = (rows + kNT - 1) / kNT;
  const int band = l / (kBand * parts), first_i = band * kBand;
  const int wide = min(kBand, a.tiles_i - first_i), m = l - first_i * parts;
  const int ti = first_i + m % wide, tj = m / wide;
  x.i0 = ti * 256;
  const int step = ((rows + parts - 1) / parts + 15) / 16 * 16;  // equal parts, in whole steps
  x.j0 = tj * step;
  x.jn = min(step, rows - x.j0);
  return x;
}

// Columns of B that a CTA loads for a tile: its half.
__device__ __forceinline__ int half_cols(const Tile& x) { return (x.jn + 15) / 16 * 8; }

using Pair = unsigned long long;  // two floats
__device__ __forceinline__ Pair pair_of(uint32_t lo, uint32_t hi) {
  Pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "r"(lo), "r"(hi));
  return p;
}
__device__ __forceinline__ float lo_of(Pair p) { return __uint_as_float((uint32_t)p); }
__device__ __forceinline__ float hi_of(Pair p) { return __uint_as_float((uint32_t)(p >> 32)); }
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ void ld_pairs(uint32_t addr, Pair& a, Pair& b) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr) : "memory");
}

// Where column j's scale lies among its 32: a thread's 8 (c = j / 2 % 4) side by side.
__device__ __forceinline__ int scale_place(int j) {
  return (j & ~31) | ((j >> 1 & 3) << 3) | ((j >> 3 & 3) << 1) | (j & 1);
}

// 32 columns of a warp's 32 lanes, as pairs of columns: v[2 n + h] lanes 0-15, v[8 + 2 n + h]
// lanes 16-31; row lane / 4 + 8 h, columns 8 n + 2 (lane % 4), + 1.
struct Block {
  uint32_t lo[16], hi[16];
};
__device__ __forceinline__ void load_block(uint32_t src, Block& v) {
  tmem_ld16(src, v.lo);
  tmem_ld16(src + (16u << 16), v.hi);
}

template <bool ACT>
__device__ __forceinline__ void add_block(const Block& v, uint32_t scales, Pair wg, Pair wu, Pair (&acc)[16]) {
  Pair s[4];
  ld_pairs(scales, s[0], s[1]);
  ld_pairs(scales + 16, s[2], s[3]);
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const Pair sg = ACT ? mul2(s[n], wg) : s[n], su = ACT ? mul2(s[n], wu) : s[n];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = 4 * n + 2 * h;
      acc[2 * n + h] = fma2(pair_of(v.lo[k], v.lo[k + 1]), sg, acc[2 * n + h]);
      acc[8 + 2 * n + h] = fma2(pair_of(v.hi[k], v.hi[k + 1]), su, acc[8 + 2 * n + h]);
    }
  }
}

// ---- results of 32 columns from c0, out of registers ----

// 16-bit results: turned in shared memory (16-byte pieces, XORed with bits of the
// row number), out in 16-byte stores. act: gates and ups of 16 outputs.
template <typename T>
__device__ __forceinline__ void store_rows(const Pair (&v)[16], uint16_t* out, size_t ld, int i, bool in,
                                           int jn, uint8_t* stage) {
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const uint32_t st = smem_u32(stage);
  auto pack = [&](int k) { return T::pack2(lo_of(v[k]), hi_of(v[k])); };
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const int j = 8 * n + (lane & 7);
    st_matrix_t(st + j * 64 + (((lane >> 3) ^ ((j >> 1) & 3)) << 4), pack(2 * n), pack(2 * n + 1),
                pack(8 + 2 * n), pack(8 + 2 * n + 1));
  }
  __syncwarp();
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int j = 8 * p + r;
    const uint4 w = async::ld_shared_v4(stage + j * 64 + ((c ^ ((j >> 1) & 3)) << 4));
    if (in && j < jn) *reinterpret_cast<uint4*>(out + (size_t)j * ld + i) = w;
  }
  __syncwarp();
}

// The same for 16 outputs (SwiGLU): rows of 32 bytes.
template <typename T>
__device__ __forceinline__ void store_half_rows(const Pair (&y)[8], uint16_t* out, size_t ld, int i, bool in,
                                                int jn, uint8_t* stage) {
  const int lane = threadIdx.x & 31;
  const uint32_t st = smem_u32(stage);
  auto pack = [&](int k) { return T::pack2(lo_of(y[k]), hi_of(y[k])); };
#pragma unroll
  for (int n = 0; n < 4; n += 2) {
    const int j = 8 * (n + (lane >> 4)) + (lane & 7);
    st_matrix_t(st + j * 32 + ((((lane >> 3) & 1) ^ ((j >> 2) & 1)) << 4), pack(2 * n), pack(2 * n + 1),
                pack(2 * n + 2), pack(2 * n + 3));
  }
  __syncwarp();
  const int r2 = lane >> 1, c2 = lane & 1;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int j = 16 * p + r2;
    const uint4 w = async::ld_shared_v4(stage + j * 32 + ((c2 ^ ((j >> 2) & 1)) << 4));
    if (in && j < jn) *reinterpret_cast<uint4*>(out + (size_t)j * ld + i + 8 * c2) = w;
  }
  __syncwarp();
}

// The largest |v| of each of 32 columns over a warp's lanes: lane 4 (2 n + b) + c gets
// column 8 n + 2 c + b. Each step halves the columns that a lane looks after.
template <int N>
__device__ __forceinline__ float column_tops(const Pair (&v)[N]) {
  const int lane = threadIdx.x & 31;
  float t[8];  // 2 n + b
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    float a = fmaxf(fabsf(lo_of(v[2 * n])), fabsf(lo_of(v[2 * n + 1])));
    float b = fmaxf(fabsf(hi_of(v[2 * n])), fabsf(hi_of(v[2 * n + 1])));
    if constexpr (N == 16) {
      a = fmaxf(a, fmaxf(fabsf(lo_of(v[8 + 2 * n])), fabsf(lo_of(v[8 + 2 * n + 1]))));
      b = fmaxf(b, fmaxf(fabsf(hi_of(v[8 + 2 * n])), fabsf(hi_of(v[8 + 2 * n + 1]))));
    }
    t[2 * n] = a;
    t[2 * n + 1] = b;
  }
#pragma unroll
  for (int o = 4; o; o >>= 1) {  // lane bits 4, 3, 2
    const bool up = lane & (4 * o);
#pragma unroll
    for (int k = 0; k < o; ++k) {
      const float keep = up ? t[k + o] : t[k], give = up ? t[k] : t[k + o];
      t[k] = fmaxf(keep, __shfl_xor_sync(~0u, give, 4 * o));
    }
  }
  return t[0];
}

// fp8 results: codes of v times the column's `mult` (the lane of column_tops has it),
// 16 or 32 outputs; bytes into rows of 48, out in 16-byte stores.
template <int N>
__device__ __forceinline__ void store_codes(const Pair (&v)[N], float mult, uint8_t* out, size_t ld, int i,
                                            int left, int jn, uint8_t* stage) {
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const float m0 = __shfl_sync(~0u, mult, 8 * n + c), m1 = __shfl_sync(~0u, mult, 8 * n + 4 + c);
    uint8_t* to = stage + (8 * n + 2 * c) * 48 + r;
#pragma unroll
    for (int p = 0; p < N / 8; ++p)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const Pair w = v[8 * p + 2 * n + h];
        const uint32_t q = permute_detail::e4m3x2(__fmul_rn(lo_of(w), m0), __fmul_rn(hi_of(w), m1));
        to[16 * p + 8 * h] = (uint8_t)q;
        to[16 * p + 8 * h + 48] = (uint8_t)(q >> 8);
      }
  }
  __syncwarp();
  if (lane < jn) {
#pragma unroll
    for (int p = 0; p < N / 8; ++p)
      if (16 * p < left)
        *reinterpret_cast<uint4*>(out + (size_t)lane * ld + i + 16 * p) =
            async::ld_shared_v4(stage + lane * 48 + 16 * p);
  }
  __syncwarp();
}

// dx through SwiGLU: a lane's 8 gates and ups of 4 of 32 columns, read ahead.
struct Saved {
  uint4 g[4], u[4];
};
__device__ __forceinline__ void load_saved(const B128Args& a, const Tile& x, int i_warp, int c0, Saved& v) {
  const int lane = threadIdx.x & 31, r = lane >> 2, i = i_warp + 8 * (lane & 3);
  const size_t ld = 2 * (size_t)a.I;
  const uint16_t* pre =
      static_cast<const uint16_t*>(a.pre_in) + ((size_t)(x.begin + x.j0) + c0 + r) * ld + i;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const bool ok = i < a.I && c0 + 8 * p + r < x.jn;
    v.g[p] = ok ? __ldg(reinterpret_cast<const uint4*>(pre + 8 * p * ld)) : make_uint4(0, 0, 0, 0);
    v.u[p] = ok ? __ldg(reinterpret_cast<const uint4*>(pre + 8 * p * ld + a.I)) : make_uint4(0, 0, 0, 0);
  }
}

template <typename T>
__device__ __forceinline__ void store_gradients(const B128Args& a, const Pair (&v)[16], const Saved& s,
                                                uint16_t* out, int i_warp, int jn, uint8_t* stage) {
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3, i = i_warp + 8 * c;
  const size_t ld = 2 * (size_t)a.I;
  float* buf = reinterpret_cast<float*>(stage);  // 16 columns, rows of 33 floats
#pragma unroll
  for (int half = 0; half < 2; ++half) {
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k) {  // rows r + 8 k
        const Pair w = v[8 * (k >> 1) + 2 * (2 * half + n) + (k & 1)];
        float* to = buf + (8 * n + 2 * c) * 33 + 8 * k + r;
        to[0] = lo_of(w);
        to[33] = hi_of(w);
      }
    __syncwarp();
#pragma unroll
    for (int p = 2 * half; p < 2 * half + 2; ++p) {
      const float* d = buf + (8 * (p - 2 * half) + r) * 33 + 8 * c;
      const uint32_t gw[4] = {s.g[p].x, s.g[p].y, s.g[p].z, s.g[p].w};
      const uint32_t uw[4] = {s.u[p].x, s.u[p].y, s.u[p].z, s.u[p].w};
      uint32_t dg[4], du[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float dg0, du0, dg1, du1;
        swiglu_gradient(d[2 * k], T::lo(gw[k]), T::lo(uw[k]), dg0, du0);
        swiglu_gradient(d[2 * k + 1], T::hi(gw[k]), T::hi(uw[k]), dg1, du1);
        dg[k] = T::pack2(dg0, dg1);
        du[k] = T::pack2(du0, du1);
      }
      if (i < a.I && 8 * p + r < jn) {
        uint16_t* to = out + (size_t)(8 * p + r) * ld + i;
        *reinterpret_cast<uint4*>(to) = make_uint4(dg[0], dg[1], dg[2], dg[3]);
        *reinterpret_cast<uint4*>(to + a.I) = make_uint4(du[0], du[1], du[2], du[3]);
      }
    }
    __syncwarp();
  }
}

// DX: the input's gradient. ACT: forward with SwiGLU, or the gradient through it.
// OUT8: results in fp8 with scales.
template <bool DX, typename T, bool ACT, bool OUT8>
__global__ void __launch_bounds__(kThreads, 1)
b128_kernel(const __grid_constant__ B128Args a, const __grid_constant__ CUtensorMap map_a,
            const __grid_constant__ CUtensorMap map_b, const __grid_constant__ FewMaps few) {
  constexpr bool kGates = ACT && !DX;  // two block scales a CTA
  extern __shared__ __align__(1024) uint8_t dyn[];
  __shared__ Bars bars;
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = ring + kStages * kStageBytes;
  float* s_scales = reinterpret_cast<float*>(staging + kDrainWarps * kStaging);
  float* s_top = s_scales + kScaleRing * kScaleFloats;  // OUT8: [2][8][256]
  int* s_begin = reinterpret_cast<int*>(s_top + (OUT8 ? 2 * 8 * kNT : 0));
  int* s_tile = s_begin + a.G + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  if (threadIdx.x == 0) {
    prefetch_map(&map_a);
    prefetch_map(&map_b);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars.full[s], 1);
      mbar_init(&bars.empty[s], 1);
    }
    for (int s = 0; s < kScaleRing; ++s) {
      mbar_init(&bars.sfull[s], 2);
      mbar_init(&bars.sempty[s], kDrainWarps);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars.tfull[b], 1);
      mbar_init(&bars.tempty[b], kDrainWarps * 2);
      mbar_init(&bars.top[b], kGates ? 8 : 4);
    }
    mbar_init(&bars.done, 1);
    async::mbar_fence_init();
  }
  if (warp == 1) tmem_alloc(&bars.tmem, kTmemCols);
  // No early release of the next kernel: the permute kernel reads token rows before its
  // own wait, and they may be these results.
  griddep_wait();
  const bool bad = group_scan<kThreads>(
      a, s_begin, s_tile, [&](int rows) { return a.tiles_i * ((rows + kNT - 1) / kNT); });
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
        const Tile x = tile_at(a, s_begin, s_tile, t);
        const int i_cta = x.i0 + (int)rank * 128;
        const int jh = half_cols(x), jb = x.j0 + (int)rank * jh;
        const bool b128 = jh > 96, b64 = !b128 && jh > 32, b32 = !b128 && (jh <= 32 || jh > 64);
        const uint32_t bytes = kABytes + (b128 ? 16384 : (b64 ? 8192 : 0) + (b32 ? 4096 : 0));
        int half = 0, k0 = 0;
        for (int kb = 0; kb < a.blocks; ++kb) {
          if (lap > 0 && !(ok = wait(&bars.empty[s], (lap & 1) ^ 1))) break;
          if (elect_one()) {
            const uint32_t sa = smem_u32(ring + s * kStageBytes), sb = sa + kABytes;
            const uint32_t bar = lead(&bars.full[s]);
            if (rank == 0) mbar_arrive_expect_tx(&bars.full[s], bytes * 2);
            if constexpr (kGates) tma_load5(sa, &map_a, k0, 0, 0, i_cta / 32, x.e, bar);
            else if constexpr (DX) tma_load4<2>(sa, &map_a, i_cta, k0, half, x.e, bar);
            else tma_load3<2>(sa, &map_a, k0, i_cta, x.e, bar);
            if (b128) tma_load3<2>(sb, &map_b, k0, half, x.begin + jb, bar);
            if (b64) tma_load3<2>(sb, &few.b64, k0, half, x.begin + jb, bar);
            if (b32) tma_load3<2>(sb + (b64 ? 8192 : 0), &few.b32, k0, half, x.begin + jb + (b64 ? 64 : 0), bar);
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
      constexpr uint32_t ka = (DX ? 4096 : 32) >> 4, kbs = 32 >> 4;
      const uint64_t da = desc_at(desc_base(16), smem_u32(ring));
      const uint64_t db = desc_at(desc_base(16), smem_u32(ring) + kABytes);
      uint32_t s = 0, lap = 0, buf = 0;
      bool ok = true;
      for (int t = first; t < n_tiles && ok; t += step) {
        const Tile x = tile_at(a, s_begin, s_tile, t);
        const uint32_t idesc = idesc_fp8(a.w_dtype, a.x_dtype == kMxE5M2, DX, 256, half_cols(x) * 2);
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
    } else if (warp >= 2) {
      // ---- scales: a lane has every 64th column, four blocks at a time ----
      const int l64 = (warp - 2) * 32 + lane;
      const int entries = (a.blocks + kEntry - 1) / kEntry;
      int t_load = first, q_load = 0;
      Tile x = {};
      auto load = [&](float (&v)[4][4], float (&w)[4], float& w2) {
        if (t_load >= n_tiles) return;
        if (q_load == 0) x = tile_at(a, s_begin, s_tile, t_load);
        const int b0 = q_load * kEntry, nb = min(kEntry, a.blocks - b0);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const int j = l64 + 64 * m;
#pragma unroll
          for (int k = 0; k < 4; ++k) v[m][k] = 0.f;
          if (j >= x.jn) continue;
          const float* p = a.xs + (size_t)(x.begin + x.j0 + j) * a.blocks + b0;
          if (a.vec) {
            const float4 f = __ldg(reinterpret_cast<const float4*>(p));
            v[m][0] = f.x, v[m][1] = f.y, v[m][2] = f.z, v[m][3] = f.w;
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k < nb) v[m][k] = __ldg(p + k);
          }
        }
        const int i_cta = x.i0 + (int)rank * 128;
        w2 = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = 0.f;
        if constexpr (kGates) {
          // lanes 0-3 the gates' four, 4-7 the ups'
          const int half = lane >> 2, k = lane & 3, ob = i_cta / 256;
          if (half < 2 && k < nb && ob < a.nb)
            w2 = __ldg(a.ws + ((size_t)x.e * 2 * a.nb + half * a.nb + ob) * a.kb + b0 + k);
        } else if (i_cta < a.I) {
          const size_t at = DX ? ((size_t)x.e * a.blocks + b0) * a.kb + i_cta / 128
                               : ((size_t)x.e * a.nb + i_cta / 128) * a.kb + b0;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k < nb) w[k] = __ldg(a.ws + at + (size_t)k * (DX ? a.kb : 1));
        }
        if (++q_load == entries) q_load = 0, t_load += step;
      };
      float v[4][4], w[4], w2;  // the entry in flight
      load(v, w, w2);
      const int64_t total = n_tiles > first ? (int64_t)((n_tiles - 1 - first) / step + 1) * entries : 0;
      uint32_t s = 0, lap = 0;
      for (int64_t i = 0; i < total; ++i) {
        if (lap > 0 && !wait(&bars.sempty[s], (lap & 1) ^ 1)) break;
        float* to = s_scales + s * kScaleFloats;
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            to[k * kNT + scale_place(l64 + 64 * m)] = kGates ? v[m][k] : v[m][k] * w[k];
        if (kGates && warp == 2 && lane < 8) to[kEntry * kNT + lane] = w2;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.sfull[s]);
        if (++s == kScaleRing) s = 0, ++lap;
        load(v, w, w2);
      }
    }
  } else {
    // ---- scaled sums, and results ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kDrainRegs));
    const int q = warp & 3, half = (warp - 4) >> 2, c = lane & 3;
    uint8_t* stage = staging + (warp - 4) * kStaging;
    uint32_t buf = 0, se = 0, se_lap = 0, nth = 0;  // nth: tiles so far
    bool ok = true;
    for (int t = first; t < n_tiles && ok; t += step) {
      const Tile x = tile_at(a, s_begin, s_tile, t);
      const int i_cta = x.i0 + (int)rank * 128, i_warp = i_cta + 32 * q;
      Pair acc[4][16];
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int k = 0; k < 16; ++k) acc[m][k] = 0;
      const int mine = min(4, max(0, (x.jn - 32 * half + 63) / 64));  // chunks of 32 columns
      for (int kb = 0; kb < a.blocks; ++kb) {
        const uint32_t b = buf & 1, use = buf >> 1;
        ++buf;
        if ((kb & 3) == 0 && !(ok = wait(&bars.sfull[se], se_lap & 1))) break;
        const float* sc = s_scales + se * kScaleFloats;
        Pair wg = 0, wu = 0;
        if (kGates) {
          const uint32_t g = __float_as_uint(sc[kEntry * kNT + (kb & 3)]), u = __float_as_uint(sc[kEntry * kNT + 4 + (kb & 3)]);
          wg = pair_of(g, g);
          wu = pair_of(u, u);
        }
        const uint32_t scales = smem_u32(sc + (kb & 3) * kNT + 32 * half + 8 * c);
        if (!(ok = wait(&bars.tfull[b], use & 1))) break;
        fence_after();
        const uint32_t src = tmem + b * kNT + ((uint32_t)(q * 32) << 16) + 32 * half;
        Block v[2];
        if (mine > 0) load_block(src, v[0]);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          if (m >= mine) break;
          tmem_wait();
          if (m + 1 < 4 && m + 1 < mine) load_block(src + 64 * (m + 1), v[(m + 1) & 1]);
          if (m + 1 == mine) {  // the accumulator is read
            fence_before();
            __syncwarp();
            if (lane == 0) arrive_cluster_relaxed(lead(&bars.tempty[b]));
          }
          add_block<kGates>(v[m & 1], scales + 256 * m, wg, wu, acc[m]);
        }
        if (mine == 0) {
          __syncwarp();
          if (lane == 0) arrive_cluster_relaxed(lead(&bars.tempty[b]));
        }
        if ((kb & 3) == 3 || kb == a.blocks - 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.sempty[se]);
          if (++se == kScaleRing) se = 0, ++se_lap;
        }
      }
      if (!ok) break;
      const size_t row0 = (size_t)(x.begin + x.j0) + 32 * half;
      if constexpr (DX && ACT) {
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          if (m >= mine) break;
          Saved saved;
          load_saved(a, x, i_warp, 32 * half + 64 * m, saved);
          store_gradients<T>(a, acc[m], saved, static_cast<uint16_t*>(a.out) + (row0 + 64 * m) * 2 * a.I, i_warp,
                             x.jn - 32 * half - 64 * m, stage);
        }
      } else {
        const int o = kGates ? i_warp / 2 : i_warp, n_out = kGates ? a.n : a.I;  // outputs
        const bool in = o < n_out;
        float tops[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          if (m >= mine) break;
          const int jn = x.jn - 32 * half - 64 * m;
          const size_t row = row0 + 64 * m;
          if constexpr (kGates) {
            if (a.pre_out) {  // the first two pieces are gates, the others ups
              const int i = o + 8 * (c & 1) + (c & 2 ? a.n : 0);
              store_rows<T>(acc[m], static_cast<uint16_t*>(a.pre_out) + row * 2 * a.n, 2 * (size_t)a.n, i, in, jn, stage);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float y0 = swiglu(lo_of(acc[m][k]), lo_of(acc[m][8 + k]));
              const float y1 = swiglu(hi_of(acc[m][k]), hi_of(acc[m][8 + k]));
              acc[m][k] = pair_of(__float_as_uint(y0), __float_as_uint(y1));
            }
            const Pair(&y)[8] = reinterpret_cast<const Pair(&)[8]>(acc[m]);
            if constexpr (OUT8) tops[m] = column_tops(y);
            else store_half_rows<T>(y, static_cast<uint16_t*>(a.out) + row * a.n, a.n, o, in, jn, stage);
          } else {
            if constexpr (OUT8) tops[m] = column_tops(acc[m]);
            else store_rows<T>(acc[m], static_cast<uint16_t*>(a.out) + row * n_out, n_out, i_warp + 8 * c, i_warp + 8 * c < n_out, jn, stage);
          }
        }
        if constexpr (OUT8) {
          // A group of 128 outputs is on the lanes of one CTA, with SwiGLU on those of both:
          // the warps leave their columns' largest values with all who need them. Two buffers
          // by the tiles' turn: who writes the next but one has seen all arrive for the next,
          // and they had read this one.
          const int from = kGates ? (int)rank * 4 + q : q;
          const int col = 8 * (lane >> 3) + 2 * c + ((lane >> 2) & 1);  // of column_tops
          float* tb = s_top + (nth & 1) * 8 * kNT + 32 * half + col;
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            if (m >= mine) break;
            tb[from * kNT + 64 * m] = tops[m];
            if (kGates) {
              const uint32_t to = addr_in(smem_u32(tb + from * kNT + 64 * m), rank ^ 1);
              asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(tops[m]) : "memory");
            }
          }
          __syncwarp();
          if (lane == 0) {
            if (kGates) arrive_cluster(addr_in(smem_u32(&bars.top[half]), rank ^ 1));
            arrive_cluster(addr_in(smem_u32(&bars.top[half]), rank));
          }
          if (!(ok = wait(&bars.top[half], nth & 1, true))) break;
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            if (m >= mine) break;
            float top = 0.f;
#pragma unroll
            for (int k = 0; k < (kGates ? 8 : 4); ++k) top = fmaxf(top, tb[k * kNT + 64 * m]);
            const float s = __fdiv_rn(448.f, top), mult = top == 0.f ? 0.f : s;
            const int jn = x.jn - 32 * half - 64 * m;
            const size_t row = row0 + 64 * m;
            if (q == 0 && (!kGates || rank == 0) && o < n_out && col < jn)
              a.ys[(row + col) * a.nb + o / 128] = __fdiv_rn(1.f, s);
            uint8_t* out = static_cast<uint8_t*>(a.out) + row * n_out;
            if constexpr (kGates)
              store_codes(reinterpret_cast<const Pair(&)[8]>(acc[m]), mult, out, n_out, o, n_out - o, jn, stage);
            else
              store_codes(acc[m], mult, out, n_out, o, n_out - o, jn, stage);
          }
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
cudaError_t launch_t(const B128Args& a, const CUtensorMap& ma, const CUtensorMap& mb, const FewMaps& few, cudaStream_t s) {
  constexpr auto kernel = b128_kernel<DX, T, ACT, OUT8>;
  const size_t smem = 1024 + kStages * kStageBytes + kDrainWarps * kStaging + kScaleRing * kScaleFloats * 4 +
                      (OUT8 ? 2 * 8 * kNT * 4 : 0) + 8 * ((size_t)a.G + 1);
  cudaError_t e = prepare_kernel<kernel>(smem);
  if (e != cudaSuccess) return e;
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorUnknown;
  const int64_t most = (int64_t)a.tiles_i * (a.R / kNT + std::min(a.G, a.R));
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
  return cudaLaunchKernelEx(&cfg, kernel, a, ma, mb, few);
}

template <typename T>
cudaError_t launch_type(bool dx, B128Args& a, cudaStream_t s) {
  const uint64_t G = a.G, R = a.R, N = a.N, K = a.K, n = a.n, halves = N / n;
  CUtensorMap ma, mb;
  FewMaps few = {};
  a.blocks = dx ? (int)halves * a.nb : a.kb;
  a.half_blocks = dx ? a.nb : a.kb;
  a.half_len = dx ? a.n : a.K;
  a.vec = a.blocks % 4 == 0 && reinterpret_cast<uintptr_t>(a.xs) % 16 == 0;
  a.I = dx ? a.K : a.N;
  a.tiles_i = (a.I + 255) / 256;
  {  // rows: of both halves side by side for dx
    const uint64_t len = a.half_len, h = dx ? halves : 1, d[] = {len, h, R}, st[] = {len, len * h};
    const uint32_t b[] = {128, 1, 128}, b64[] = {128, 1, 64}, b32[] = {128, 1, 32};
    if (!make_map(&mb, a.x, kMapU8, 3, d, st, b) || !make_map(&few.b64, a.x, kMapU8, 3, d, st, b64) ||
        !make_map(&few.b32, a.x, kMapU8, 3, d, st, b32))
      return cudaErrorUnknown;
  }
  if (dx) {
    const uint64_t d[] = {K, n, halves, G}, st[] = {K, n * K, N * K};
    const uint32_t b[] = {128, 128, 1, 1};
    if (!make_map(&ma, a.w, kMapU8, 4, d, st, b)) return cudaErrorUnknown;
    return a.pre_in ? launch_t<true, T, true, false>(a, ma, mb, few, s) : launch_t<true, T, false, false>(a, ma, mb, few, s);
  }
  if (a.act) {  // a tile's rows: 16 gates, 16 ups, 16 gates, ...
    const uint64_t d[] = {K, 16, 2, n / 16, G}, st[] = {K, n * K, 16 * K, N * K};
    const uint32_t b[] = {128, 16, 2, 4, 1};
    if (!make_map(&ma, a.w, kMapU8, 5, d, st, b)) return cudaErrorUnknown;
    return a.ys ? launch_t<false, T, true, true>(a, ma, mb, few, s) : launch_t<false, T, true, false>(a, ma, mb, few, s);
  }
  const uint64_t d[] = {K, N, G}, st[] = {K, N * K};
  const uint32_t b[] = {128, 128, 1};
  if (!make_map(&ma, a.w, kMapU8, 3, d, st, b)) return cudaErrorUnknown;
  return a.ys ? launch_t<false, T, false, true>(a, ma, mb, few, s) : launch_t<false, T, false, false>(a, ma, mb, few, s);
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
