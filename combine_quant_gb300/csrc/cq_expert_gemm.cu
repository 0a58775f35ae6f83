// cq_expert_gemm.cu -- grouped matrix products of the experts on the tensor
// cores (tcgen05): forward (16-bit operands, or mx fp8 with block scales),
// gradient of the input, gradient of the weights.
//
// One persistent kernel on pairs of CTAs (cta_group::2). An output tile is 256 x
// up to 256 elements of out[j, i]. The axis i lies on the accumulator's lanes
// (128 in each CTA) and j on its columns, whose number is free in steps of 16:
// the ragged axis of the forward product and of the input's gradient, the
// tokens, is j, so an expert with 3 rows costs 16 columns, not a padded tile.
//
//   forward  out = y,  i = weight rows, j = tokens, sum over k:  A = w (K-major),  B = x (K-major)
//   dx       out = dx, i = weight cols, j = tokens, sum over n:  A = w (MN-major), B = dy (K-major)
//   dw       out = dw, i = columns of dy, j = columns of x, sum over the expert's
//            rows:  A = dy (MN-major), B = x (MN-major); here j is the contiguous axis
//
// Every CTA reads the counts itself and walks the same list of tiles (group_scan
// in cq_expert.cuh): no host read, no extra launch, any counts.
//
// Warp 0 fills a ring of shared-memory stages with tiled copies (64 of the
// contraction, or 128 bytes of fp8; 128-byte swizzle; each CTA its half of A and
// of B), warp 1 of the first CTA issues the products into one of two TMEM
// accumulators, warps 4-11 drain the other one. A whole warp runs each of these
// loops and one elected lane issues: with a single thread in the loop the issue
// itself was the bound (1560 instead of 1870 TFLOP/s at 8192^3).
//
// SwiGLU: a tile's weight rows are 16 gate rows, 16 up rows, 16 gate rows, ...
// (one 5-D copy picks them up in that order), so that the 16-lane TMEM loads
// give a thread a gate and its up product; both are f32 until the result is
// rounded. Its gradient (dx with the saved products) multiplies in the drain.
// dw's last rows: those of the next expert that a copy brings in are overwritten
// with zeros by warp 2 before the products read them.
// mx: three warps fetch the scales, tcgen05.cp puts them into TMEM a stage ahead
// of their products.
//
// What bounds it: below about 280 rows an expert reading the weights, above the
// tensor cores. Measured on one GB300 (copy 6.79 TB/s): 8192^3 1.89 PFLOP/s where
// cuBLAS ran at 2.01 in the same process; 32 experts of 512 rows, hidden 7168,
// SwiGLU with n 2048: 553 us, 1.74 PFLOP/s; 64 experts, 777 rows in fp16, n 1536,
// k 4096: 116 us, 6.2 TB/s; mx fp8, 32 experts of 480 rows: 344 us, 2.62 PFLOP/s,
// of 16 rows (n 7168, k 2048): 87 us, 5.4 TB/s; dw, 32 experts of 512 rows, 4096 x
// 7168: 663 us, 1.45 PFLOP/s (its 1.9 GB of results and eight stages per tile).
#include <cuda_runtime.h>

#include <algorithm>

#include "cq_expert.cuh"
#include "cq_tensor.cuh"

namespace cq {
namespace expert {
namespace {

using namespace tensor;
using async::mbar_arrive_expect_tx;
using async::mbar_init;
using async::mbar_wait;
using async::mbar_wait_warp;

__device__ uint32_t g_status;  // CQ_ST_* bits of these kernels on this device

constexpr int kDrainWarps = 8;             // two for each quarter of the lanes
constexpr int kScaleWarps = 3;             // mx: fetch the scales, 128 rows each
template <bool MX>
constexpr int kThreads = 128 + 32 * kDrainWarps + (MX ? 32 * kScaleWarps : 0);
// Most columns (j) of a tile. Two accumulators of 256 fill TMEM; mx needs 24
// columns of it for two stages' scales.
template <bool MX>
constexpr int kNT = MX ? 240 : 256;
constexpr int kStepJ = 16;                 // columns come in steps of
constexpr int kScaleBytes = 3 * 512;       // mx: scales of a stage: 128 rows of A, 256 of B
constexpr int kScaleRing = 3;              // entries of four stages' scales
constexpr int kABytes = 128 * 128;         // A of one stage, one CTA
constexpr uint32_t kTmemCols = 512;
constexpr int kBand = 8;                   // tiles along i taken together, for reuse in L2

constexpr int kStageBytes = kABytes + 128 * 128;  // B: half of up to 256 columns
// Stages of the ring: what is left beside the results' staging, the scales and
// the lists of 2048 experts.
template <Op OP, bool ACT, bool MX>
constexpr int kStages = MX ? 5 : 6;

struct Shape {
  int I, J, KK;        // extents: out columns (physical A rows), dw: out rows, contraction
  int n_out;           // forward: n
  int tiles_i;         // tiles along i
  int tiles_j;         // dw: tiles along j
  int whole;           // MN-major operands are whole blocks of 64: one copy takes two of them
};

// B by rows (K-major) in copies of 64 and of 32: an expert's last part of the
// tokens rarely fills one of 128, and the rest would be another expert's rows.
struct FewMaps {
  CUtensorMap b64, b32;
};

struct Bars {
  uint64_t full[8], empty[8], tail[8], tail_full[8];
  uint64_t swritten[4], sfull[4], sempty[4];  // mx: scales written, visible to the copies, used
  uint64_t tfull[2], tempty[2];
  uint64_t done;  // the products in flight when their warp gave up
  uint32_t tmem;
};

// A tile of the work list.
struct Tile {
  int e, begin, i0, j0, jn, nkb, kk;  // jn: real columns; kk: contraction length
};

template <Op OP, bool MX>
__device__ __forceinline__ Tile tile_at(const Shape& sh, const int* s_begin, const int* s_tile,
                                        int G, int t) {
  constexpr int NT = kNT<MX>, SJ = kStepJ;
  Tile x;
  x.e = expert_of(s_tile, G, t);
  const int l = t - s_tile[x.e];
  x.begin = s_begin[x.e];
  const int rows = s_begin[x.e + 1] - x.begin;
  const int nj = OP == kDw ? sh.tiles_j : (rows + NT - 1) / NT;
  const int band = l / (kBand * nj), first_i = band * kBand;
  const int wide = min(kBand, sh.tiles_i - first_i), m = l - first_i * nj;
  const int ti = first_i + m % wide, tj = m / wide;
  x.i0 = ti * 256;
  if (OP == kDw) {
    x.kk = rows;
    x.j0 = tj * NT;
    x.jn = min(NT, sh.J - x.j0);
  } else {
    // equal parts, in whole steps
    const int parts = (rows + NT - 1) / NT;
    const int step = ((rows + parts - 1) / parts + SJ - 1) / SJ * SJ;
    x.kk = sh.KK;
    x.j0 = tj * step;
    x.jn = min(step, rows - x.j0);
  }
  x.nkb = (x.kk + (MX ? 127 : 63)) / (MX ? 128 : 64);
  return x;
}

// Bytes of one results warp's staging buffer: 32 columns (j) of its 32 lanes
// (i) in 16 bits, or 16 in 32 bits where another factor still comes (rows of 33
// floats, so that neither the columns' stores nor the rows' loads meet in a bank).
// dw: 32 rows (i) of 64 bytes.
template <Op OP, bool ACT>
constexpr int kStagingBytes = OP == kDx && ACT ? 16 * 33 * 4 : 32 * 64;

// dw: drains 64 bytes of each of this warp's 32 rows (32 columns in 16 bits, 16
// in f32) from column c0: through shared memory, swizzled as the map of the
// result has it, and out by a tiled copy, which also cuts off what lies outside.
template <typename T, bool F32>
__device__ __forceinline__ void drain_dw(const Shape& sh, const CUtensorMap* map, const Tile& x,
                                         int i_warp, int c0, uint32_t src, uint8_t* stage) {
  const int lane = threadIdx.x & 31;
  uint32_t v[16];
  if constexpr (F32) {
    tmem_ld16c(src + c0, v);
    tmem_wait();
  } else {
    uint32_t acc[32];
    tmem_ld32(src + c0, acc);
    tmem_wait();
#pragma unroll
    for (int c = 0; c < 16; ++c)
      v[c] = T::pack2(__uint_as_float(acc[2 * c]), __uint_as_float(acc[2 * c + 1]));
  }
  tma_store_wait_read();  // of the lane that issued the last copy; nothing for the others
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<uint4*>(stage + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) =
        make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if (lane == 0 && i_warp < sh.I) tma_store3(map, smem_u32(stage), x.j0 + c0, i_warp, x.e);
}

// dx through SwiGLU: a lane's 8 gates and ups of 4 of 32 columns (j), read ahead of
// the columns' turn.
struct Saved {
  uint4 g[4], u[4];
};
__device__ __forceinline__ void load_saved(const Args& a, const Shape& sh, const Tile& x, int i_warp,
                                           int c0, Saved& v) {
  const int lane = threadIdx.x & 31, r = lane >> 2, i = i_warp + 8 * (lane & 3);
  const size_t ld = 2 * (size_t)sh.I;
  const uint16_t* pre =
      static_cast<const uint16_t*>(a.pre_in) + ((size_t)(x.begin + x.j0) + c0 + r) * ld + i;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const bool ok = i < sh.I && c0 + 8 * p + r < x.jn;
    v.g[p] = ok ? __ldg(reinterpret_cast<const uint4*>(pre + 8 * p * ld)) : make_uint4(0, 0, 0, 0);
    v.u[p] = ok ? __ldg(reinterpret_cast<const uint4*>(pre + 8 * p * ld + sh.I)) : make_uint4(0, 0, 0, 0);
  }
}

// Drains columns [c0, c0 + 32) of a tile: out[j][i .. i + 31] of 32 j. The
// accumulator holds i on lanes and j on columns, memory wants i contiguous, so
// the block is turned in shared memory (16-byte pieces of a 64-byte row, XORed
// with bits of the row number: no bank conflicts either way) and written in
// 16-byte stores, 64 bytes a row.
template <Op OP, typename T, bool ACT>
__device__ __forceinline__ void drain(const Args& a, const Shape& sh, const Tile& x, int i_warp,
                                      int c0, uint32_t src, uint8_t* stage, Saved& saved) {
  const int lane = threadIdx.x & 31;
  const int jn = x.jn - c0;  // columns that exist
  const size_t row0 = (size_t)(x.begin + x.j0) + c0;
  const uint32_t st = smem_u32(stage);
  if constexpr (OP == kDx && ACT) {
    const int r = lane >> 2, i = i_warp + 8 * (lane & 3);
    const size_t ld = 2 * (size_t)sh.I;
    uint16_t* out = static_cast<uint16_t*>(a.out) + (row0 + r) * ld + i;
    const Saved now = saved;
    if (c0 + 64 < x.jn) load_saved(a, sh, x, i_warp, c0 + 64, saved);  // of this warp's next columns
    const uint4(&g)[4] = now.g;
    const uint4(&u)[4] = now.u;
    float* buf = reinterpret_cast<float*>(stage);
    uint32_t acc[32];
    tmem_ld32(src + c0, acc);
    tmem_wait();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int c = 0; c < 16; ++c) buf[c * 33 + lane] = __uint_as_float(acc[16 * h + c]);
      __syncwarp();
#pragma unroll
      for (int p = 2 * h; p < 2 * h + 2; ++p) {
        const float* d = buf + (8 * (p - 2 * h) + r) * 33 + 8 * (lane & 3);
        const uint32_t gw[4] = {g[p].x, g[p].y, g[p].z, g[p].w}, uw[4] = {u[p].x, u[p].y, u[p].z, u[p].w};
        uint32_t dg[4], du[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float g0 = T::lo(gw[k]), g1 = T::hi(gw[k]), u0 = T::lo(uw[k]), u1 = T::hi(uw[k]);
          float dg0, du0, dg1, du1;
          swiglu_gradient(d[2 * k], g0, u0, dg0, du0);
          swiglu_gradient(d[2 * k + 1], g1, u1, dg1, du1);
          dg[k] = T::pack2(dg0, dg1);
          du[k] = T::pack2(du0, du1);
        }
        if (i < sh.I && 8 * p + r < jn) {
          *reinterpret_cast<uint4*>(out + 8 * p * ld) = make_uint4(dg[0], dg[1], dg[2], dg[3]);
          *reinterpret_cast<uint4*>(out + 8 * p * ld + sh.I) = make_uint4(du[0], du[1], du[2], du[3]);
        }
      }
      __syncwarp();
    }
  } else {
    uint32_t v0[16], v1[16];  // lanes 0-15 and 16-31 (SwiGLU: gates and ups of 16 outputs)
    tmem_ld16(src + c0, v0);
    tmem_ld16(src + c0 + (16u << 16), v1);
    tmem_wait();
    auto f = [](uint32_t w) { return __uint_as_float(w); };
    constexpr bool kAct = OP == kForward && ACT;
    const int r = lane >> 2, c = lane & 3;
    if (!kAct || a.pre_out) {
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int j = 8 * n + (lane & 7);
        st_matrix_t(st + j * 64 + (((lane >> 3) ^ ((j >> 1) & 3)) << 4),
                    T::pack2(f(v0[4 * n]), f(v0[4 * n + 1])), T::pack2(f(v0[4 * n + 2]), f(v0[4 * n + 3])),
                    T::pack2(f(v1[4 * n]), f(v1[4 * n + 1])), T::pack2(f(v1[4 * n + 2]), f(v1[4 * n + 3])));
      }
      __syncwarp();
      const size_t ld = kAct ? 2 * (size_t)sh.n_out : (size_t)sh.I;
      // SwiGLU: the first two pieces are gates, the others ups
      const int i = kAct ? i_warp / 2 + 8 * (c & 1) + (c & 2 ? sh.n_out : 0) : i_warp + 8 * c;
      const bool in = kAct ? i_warp / 2 < sh.n_out : i < sh.I;
      uint16_t* out = static_cast<uint16_t*>(kAct ? a.pre_out : a.out) + (row0 + r) * ld + i;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int j = 8 * p + r;
        const uint4 w = async::ld_shared_v4(stage + j * 64 + ((c ^ ((j >> 1) & 3)) << 4));
        if (in && j < jn) *reinterpret_cast<uint4*>(out + 8 * p * ld) = w;
      }
      __syncwarp();
    }
    if constexpr (kAct) {
#pragma unroll
      for (int n = 0; n < 16; ++n) v0[n] = __float_as_uint(swiglu(f(v0[n]), f(v1[n])));
#pragma unroll
      for (int n = 0; n < 4; n += 2) {
        // rows of 32 bytes: block 0, 1 = outputs 0-7, 8-15 of columns 8 n.., 2, 3 of 8 (n + 1)..
        const int j = 8 * (n + (lane >> 4)) + (lane & 7);
        st_matrix_t(st + j * 32 + ((((lane >> 3) & 1) ^ ((j >> 2) & 1)) << 4),
                    T::pack2(f(v0[4 * n]), f(v0[4 * n + 1])), T::pack2(f(v0[4 * n + 2]), f(v0[4 * n + 3])),
                    T::pack2(f(v0[4 * n + 4]), f(v0[4 * n + 5])), T::pack2(f(v0[4 * n + 6]), f(v0[4 * n + 7])));
      }
      __syncwarp();
      const int r2 = lane >> 1, c2 = lane & 1, o = i_warp / 2;
      uint16_t* out = static_cast<uint16_t*>(a.out) + (row0 + r2) * (size_t)sh.n_out + o + 8 * c2;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int j = 16 * p + r2;
        const uint4 w = async::ld_shared_v4(stage + j * 32 + ((c2 ^ ((j >> 2) & 1)) << 4));
        if (o < sh.n_out && j < jn) *reinterpret_cast<uint4*>(out + 16 * p * (size_t)sh.n_out) = w;
      }
      __syncwarp();
    }
  }
}

// Zeros for a tile of an expert without rows (dw): 128 rows from i0.
template <bool F32>
__device__ __forceinline__ void store_zeros(const Args& a, const Shape& sh, const Tile& x, int i0) {
  constexpr int kPer = F32 ? 4 : 8, kSize = F32 ? 4 : 2;  // elements of 16 bytes, bytes of one
  const int cols = x.jn / kPer, rows = min(128, sh.I - i0);
  char* out = static_cast<char*>(a.out) + (((size_t)x.e * sh.I + i0) * sh.J + x.j0) * kSize;
  for (int v = threadIdx.x - 128; v < rows * cols; v += kDrainWarps * 32)
    *reinterpret_cast<uint4*>(out + ((size_t)(v / cols) * sh.J + v % cols * kPer) * kSize) = make_uint4(0, 0, 0, 0);
}

template <Op OP, typename T, bool F32, bool ACT, bool MX>
__global__ void __launch_bounds__(kThreads<MX>, 1)
gemm_kernel(const __grid_constant__ Args a, const __grid_constant__ Shape sh,
            const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
            const __grid_constant__ CUtensorMap map_out, const __grid_constant__ FewMaps few) {
  constexpr int S = kStages<OP, ACT, MX>;
  constexpr int SB = kStageBytes;
  constexpr int NT = kNT<MX>, KB = MX ? 128 : 64;  // columns; contraction of a stage
  constexpr bool A_MN = OP != kForward, B_MN = OP == kDw;
  extern __shared__ __align__(1024) uint8_t dyn[];
  __shared__ Bars bars;
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = ring + S * SB;
  uint8_t* s_sf = staging + kDrainWarps * kStagingBytes<OP, ACT>;
  int* s_begin = reinterpret_cast<int*>(s_sf + (MX ? kScaleRing * 4 * kScaleBytes : 0));
  int* s_tile = s_begin + a.G + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  if (threadIdx.x == 0) {
    prefetch_map(&map_a);
    prefetch_map(&map_b);
    for (int s = 0; s < S; ++s) {
      mbar_init(&bars.full[s], 1);
      mbar_init(&bars.empty[s], 1);
      mbar_init(&bars.tail[s], 1);
      mbar_init(&bars.tail_full[s], 2);
    }
    for (int s = 0; s < kScaleRing; ++s) {
      mbar_init(&bars.swritten[s], kScaleWarps);
      mbar_init(&bars.sfull[s], 2);
      mbar_init(&bars.sempty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars.tfull[b], 1);
      mbar_init(&bars.tempty[b], kDrainWarps * 2);
    }
    mbar_init(&bars.done, 1);
    async::mbar_fence_init();
  }
  if (warp == 1) tmem_alloc(&bars.tmem, kTmemCols);
  // No early release of the next kernel here: the permute kernel reads token rows
  // before its own wait, and they may be these results.
  griddep_wait();
  const bool bad = group_scan<kThreads<MX>>(a, s_begin, s_tile, [&](int rows) {
    return OP == kDw ? sh.tiles_i * sh.tiles_j : sh.tiles_i * ((rows + NT - 1) / NT);
  });
  if (bad && blockIdx.x == 0) atomicOr(&g_status, (uint32_t)CQ_ST_BAD_ROWS);
  fence_before();
  cluster_sync();
  fence_after();
  const uint32_t tmem = bars.tmem;
  const int n_tiles = s_tile[a.G];
  const int first = blockIdx.x / 2, step = gridDim.x / 2;
  // One verdict for the warp: the lanes go on to elect.sync and to .aligned instructions.
  auto wait = [&](uint64_t* bar, uint32_t parity, int rounds, bool pair = false) {
    for (int r = 0; r < rounds; ++r)
      if (pair ? wait_pair(bar, parity) : mbar_wait_warp(bar, parity)) return true;
    atomicOr(&g_status, (uint32_t)CQ_ST_TIMEOUT);
    return false;
  };
  auto lead = [&](uint64_t* bar) { return leader_addr(smem_u32(bar)); };

  // Columns of B that this CTA loads for a tile: its half of jn, in copies of
  // 32 rows (K-major) or 64 columns (MN-major).
  auto half_cols = [&](const Tile& x) {
    const int unit = OP != kDw ? kStepJ : sh.whole ? 128 : 32;
    return (x.jn + unit - 1) / unit * unit / 2;
  };

  if (warp == 0) {
    // ---- copies ----
    uint32_t s = 0, lap = 0;  // stage, times the ring has gone round
    // dw, bit s: the last copies into stage s complete on tail[s]; the parity of their number
    uint32_t on_tail = 0, tail_odd = 0;
    bool ok = true;
    for (int t = first; t < n_tiles && ok; t += step) {
      const Tile x = tile_at<OP, MX>(sh, s_begin, s_tile, a.G, t);
      const int i_cta = x.i0 + (int)rank * 128;
      const int jh = half_cols(x), jb = x.j0 + (int)rank * jh;
      const bool ragged = OP == kDw && (x.kk & 15) != 0;
      // B_MN: whole blocks of 64 (two per copy, or one); else 128 rows, 64, 32, or 64 + 32
      const int n64 = (jh + 63) / 64;
      const bool b128 = jh > 96, b64 = !b128 && jh > 32, b32 = !b128 && (jh <= 32 || jh > 64);
      const uint32_t bytes =
          kABytes + (B_MN ? (sh.whole ? 2 : n64) * 8192 : b128 ? 16384 : (b64 ? 8192 : 0) + (b32 ? 4096 : 0));
      for (int kb = 0; kb < x.nkb; ++kb) {
        if (lap > 0 && !(ok = wait(&bars.empty[s], (lap & 1) ^ 1, 1))) break;
        const bool tail = ragged && kb == 0;
        on_tail = (on_tail & ~(1u << s)) | ((uint32_t)tail << s);
        tail_odd ^= (uint32_t)tail << s;
        if (elect_one()) {
          const uint32_t sa = smem_u32(ring + s * SB), sb = sa + kABytes;
          uint32_t bar;
          if (tail) {
            // zeros go in before the product may read: each CTA's copies complete
            // on its own barrier, warp 2 takes it from there
            bar = smem_u32(&bars.tail[s]);
            mbar_arrive_expect_tx(&bars.tail[s], bytes);
            if (rank == 0) async::mbar_arrive(&bars.full[s]);
          } else {
            bar = lead(&bars.full[s]);
            if (rank == 0) mbar_arrive_expect_tx(&bars.full[s], bytes * 2);
          }
          const int k0 = (!ragged ? kb : kb == 0 ? x.nkb - 1 : kb - 1) * KB;
          if constexpr (OP == kForward && ACT) {
            tma_load5(sa, &map_a, k0, 0, 0, i_cta / 32, x.e, bar);
          } else if constexpr (OP == kForward) {
            tma_load3<2>(sa, &map_a, k0, i_cta, x.e, bar);
          } else if constexpr (OP == kDx) {
            if (sh.whole) {
              tma_load4<2>(sa, &map_a, 0, k0, i_cta / 64, x.e, bar);
            } else {
              tma_load3<2>(sa, &map_a, i_cta, k0, x.e, bar);
              tma_load3<2>(sa + 8192, &map_a, i_cta + 64, k0, x.e, bar);
            }
          } else {
            if (sh.whole) {
              tma_load3<2>(sa, &map_a, 0, x.begin + k0, i_cta / 64, bar);
            } else {
              tma_load2(sa, &map_a, i_cta, x.begin + k0, bar);
              tma_load2(sa + 8192, &map_a, i_cta + 64, x.begin + k0, bar);
            }
          }
          if constexpr (!B_MN) {
            if (b128) tma_load2(sb, &map_b, k0, x.begin + jb, bar);
            if (b64) tma_load2(sb, &few.b64, k0, x.begin + jb, bar);
            if (b32) tma_load2(sb + (b64 ? 8192 : 0), &few.b32, k0, x.begin + jb + (b64 ? 64 : 0), bar);
          } else if (sh.whole) {
            tma_load3<2>(sb, &map_b, 0, x.begin + k0, jb / 64, bar);
          } else {
            for (int b = 0; b < n64; ++b)
              tma_load2(sb + b * 8192, &map_b, jb + b * 64, x.begin + k0, bar);
          }
        }
        __syncwarp();
        if (++s == S) s = 0, ++lap;
      }
    }
    // The last use of every stage, oldest first. Done: nothing may arrive here
    // after the CTA has gone. Gave up: let the copies in flight land (with a
    // limit) before it goes; those of both CTAs complete on the leader's barrier,
    // for which the other CTA stays.
    for (int v = 0; v < S; ++v) {
      const uint32_t u = (s + v) % S, laps = lap + (u < s ? 1 : 0);  // uses of stage u
      if (laps == 0) continue;
      if (ok) ok = wait(&bars.empty[u], (laps - 1) & 1, 1);
      if (ok) continue;
      if (OP == kDw && (on_tail >> u & 1)) mbar_wait(&bars.tail[u], (tail_odd >> u & 1) ^ 1);
      else if (rank == 0) mbar_wait(&bars.full[u], (laps - 1) & 1);
    }
  } else if (warp == 1 && rank == 0) {
    // ---- products ----
    constexpr uint32_t ka = (A_MN ? 2048 : 32) >> 4, kbs = (B_MN ? 2048 : 32) >> 4;
    const uint64_t da = desc_at(desc_base(A_MN ? 8192 : 16), smem_u32(ring));
    const uint64_t db = desc_at(desc_base(B_MN ? 8192 : 16), smem_u32(ring) + kABytes);
    uint32_t s = 0, lap = 0, buf = 0, tail_uses[S] = {};
    // dw: where an expert's rows do not end with a step of 16, a tile begins with
    // the stage of the last rows. It waits for warp 2's zeros in both CTAs; up to
    // kLate other stages go before it (the ring has S - 1).
    constexpr int kLate = 2;
    static_assert(kLate < S, "the ring must be able to run on while a stage waits");
    auto finish_late = [&](uint32_t late, uint32_t d, uint32_t idesc, int rows, bool add) {
      uint32_t use_t = 0;
#pragma unroll
      for (int q = 0; q < S; ++q)
        if (q == late) use_t = tail_uses[q]++;
      if (!wait(&bars.tail_full[late], use_t & 1, 1, true)) return false;
      fence_after();
      if (elect_one()) {
        const uint64_t ad = da + late * (SB >> 4), bd = db + late * (SB >> 4);
        for (int q = 0; 16 * q < rows; ++q)
          mma_f16(d, ad + q * ka, bd + q * kbs, idesc, add || q > 0);
        commit(smem_u32(&bars.empty[late]));
      }
      __syncwarp();
      return true;
    };
    // mx: entry of scales; set of 12 TMEM columns (A then B) to fill, to use. Stage
    // kb's scales are copied by one lane (copy), once they are there (waits).
    uint32_t se = 0, se_lap = 0, sf_fill = 0, sf_use = 0;
    const uint64_t sf_desc = desc_scales(smem_u32(s_sf));
    auto scales_wait = [&](int kb) { return (kb & 3) != 0 || wait(&bars.sfull[se], se_lap & 1, 1, true); };
    auto scales_copy = [&](int kb, int nkb, bool wide) {
      const uint32_t sf = tmem + 2 * NT + 12 * sf_fill;
      const uint64_t ds = sf_desc + (se * 4 + (kb & 3)) * (kScaleBytes >> 4);
      copy_scales(sf, ds);
      copy_scales(sf + 4, ds + (512 >> 4));
      if (wide) copy_scales(sf + 8, ds + (1024 >> 4));
      if ((kb & 3) == 3 || kb == nkb - 1) commit(smem_u32(&bars.sempty[se]));
    };
    auto scales_next = [&](int kb, int nkb) {
      sf_fill ^= 1;
      if (((kb & 3) == 3 || kb == nkb - 1) && ++se == kScaleRing) se = 0, ++se_lap;
    };
    bool ok = true;
    for (int t = first; t < n_tiles && ok; t += step) {
      const Tile x = tile_at<OP, MX>(sh, s_begin, s_tile, a.G, t);
      if (x.nkb == 0) continue;
      const uint32_t b = buf & 1, use = buf >> 1;
      ++buf;
      if (use > 0 && !(ok = wait(&bars.tempty[b], (use - 1) & 1, 1, true))) break;
      const uint32_t d = tmem + b * NT;
      const uint32_t idesc =
          MX ? idesc_mx(a.w_dtype, a.x_dtype == kMxE5M2, 256, half_cols(x) * 2)
             : idesc_f16(T::kBf16, A_MN, B_MN, 256, half_cols(x) * 2);
      const bool wide = MX && half_cols(x) * 2 > 128;
      const bool ragged = OP == kDw && (x.kk & 15) != 0;
      const int lead_kb = ragged ? 1 : 0;  // the first stage whose products go in at once
      uint32_t late = 0;
      for (int kb = 0; kb < x.nkb; ++kb) {
        if (ragged && kb == 0) {
          late = s;
          if (++s == S) s = 0, ++lap;
          if (x.nkb == 1) ok = finish_late(late, d, idesc, x.kk, false);
          continue;
        }
        if (!(ok = wait(&bars.full[s], lap & 1, 1))) break;
        // mx: the next stage's scales go into the other set of TMEM columns ahead of
        // this stage's products, which then need not wait for a copy
        const bool more = kb + 1 < x.nkb;
        if (MX && kb == 0) {
          if (!(ok = scales_wait(0))) break;
          fence_after();
          if (elect_one()) scales_copy(0, x.nkb, wide);
          __syncwarp();
          scales_next(0, x.nkb);
        }
        if (MX && more && !(ok = scales_wait(kb + 1))) break;
        fence_after();
        if (elect_one()) {
          const uint64_t ad = da + s * (SB >> 4), bd = db + s * (SB >> 4);
          const int left = x.kk - (kb - lead_kb) * KB;
          const bool add = kb > lead_kb;
          if constexpr (MX) {
            if (more) scales_copy(kb + 1, x.nkb, wide);
            const uint32_t sf = tmem + 2 * NT + 12 * sf_use;
            if (left > 96) {
              mma_mx(d, ad, bd, idesc, sf, sf + 4, add);
              mma_mx(d, ad + ka, bd + kbs, idesc_sf(idesc, 1), sf, sf + 4, true);
              mma_mx(d, ad + 2 * ka, bd + 2 * kbs, idesc_sf(idesc, 2), sf, sf + 4, true);
              mma_mx(d, ad + 3 * ka, bd + 3 * kbs, idesc_sf(idesc, 3), sf, sf + 4, true);
            } else {
              for (int q = 0; 32 * q < left; ++q)
                mma_mx(d, ad + q * ka, bd + q * kbs, idesc_sf(idesc, q), sf, sf + 4, add || q > 0);
            }
          } else if (left > 48) {
            mma_f16(d, ad, bd, idesc, add);
            mma_f16(d, ad + ka, bd + kbs, idesc, true);
            mma_f16(d, ad + 2 * ka, bd + 2 * kbs, idesc, true);
            mma_f16(d, ad + 3 * ka, bd + 3 * kbs, idesc, true);
          } else {
            for (int q = 0; 16 * q < left; ++q)
              mma_f16(d, ad + q * ka, bd + q * kbs, idesc, add || q > 0);
          }
          commit(smem_u32(&bars.empty[s]));
        }
        __syncwarp();
        if constexpr (MX) {
          sf_use ^= 1;
          if (more) scales_next(kb + 1, x.nkb);
        }
        if (++s == S) s = 0, ++lap;
        if (ragged && kb == min(kLate, x.nkb - 1))
          if (!(ok = finish_late(late, d, idesc, x.kk - (x.nkb - 1) * KB, true))) break;
      }
      if (ok && elect_one()) commit(smem_u32(&bars.tfull[b]));
      __syncwarp();
    }
    if (!ok) {  // gave up: let the products in flight end (with a limit), which read both CTAs' memory
      if (elect_one()) commit(smem_u32(&bars.done));
      __syncwarp();
      wait_pair(&bars.done, 0);
    }
  } else if (OP == kDw && warp == 2) {
    // ---- zeros over the rows past an expert's last (up to the next 16) ----
    uint32_t it = 0, tail_uses[S] = {};
    bool ok = true;
    for (int t = first; t < n_tiles && ok; t += step) {
      const Tile x = tile_at<OP, MX>(sh, s_begin, s_tile, a.G, t);
      const int s = it % S;  // a ragged tile begins with the stage of its last rows
      it += x.nkb;
      if (x.nkb == 0 || (x.kk & 15) == 0) continue;
      uint32_t use_t = 0;
#pragma unroll
      for (int q = 0; q < S; ++q)
        if (q == s) use_t = tail_uses[q]++;
      if (!(ok = wait(&bars.tail[s], use_t & 1, 8))) break;
      const int r0 = (x.kk - 1) % 64 + 1, r1 = (r0 + 15) / 16 * 16;
      const int blocks = 2 + (half_cols(x) + 63) / 64;
      uint8_t* base = ring + s * SB;
      for (int r = r0 + (lane >> 3); r < r1; r += 4)
        for (int b = 0; b < blocks; ++b)
          *reinterpret_cast<uint4*>(base + b * 8192 + r * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) arrive_cluster(leader_addr(smem_u32(&bars.tail_full[s])));
    }
  } else if (MX && warp >= 4 + kDrainWarps) {
    // ---- scales: one word (4 blocks of 32) a row and stage ----
    // Line r % 32 of a 512-byte atom holds the words of rows r % 32 + 0, 32, 64,
    // 96. A warp takes one atom (A, or 128 rows of B), four stages at a time: a
    // lane loads 16 bytes of each of its line's four rows and stores whole lines,
    // which meet in no bank; kAhead such steps are in flight, across tiles. The
    // fence that the tensor copies need would wait for those loads, so warp 3
    // executes it, after these warps' arrivals.
    constexpr int kAhead = 3;
    const int w = warp - 4 - kDrainWarps;
    const int blocks = sh.KK / 32, quads = (sh.KK + 511) / 512;
    // Rows of whole 16-byte pieces are read as such. Others are read as aligned words,
    // which start 2 bytes early where a row does (SC is even): the words are shifted
    // into place when they are stored, so that no load is waited for here. Scales past
    // K (a pad column, a next row's) meet no product.
    const bool whole = a.SC % 16 == 0;
    const uint8_t* rows[4];  // scale rows, NULL where there is none
    int t_load = first, q_load = 0;
    auto load = [&](uint4 (&v)[4], uint32_t (&past)[4], uint32_t& shift) {
      if (t_load >= n_tiles) return;
      if (q_load == 0) {
        const Tile x = tile_at<OP, MX>(sh, s_begin, s_tile, a.G, t_load);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          rows[b] = nullptr;
          if (w == 0) {
            int row = x.i0 + (int)rank * 128 + 32 * b + lane;  // of the tile's weight rows
            bool in = row < sh.I;
            if (ACT) {
              const int o = row / 32 * 16 + (lane & 15);
              in = o < sh.n_out;
              row = o + (lane >= 16 ? sh.n_out : 0);
            }
            if (in) rows[b] = a.w_scales + ((size_t)x.e * a.N + row) * a.SC;
          } else {
            const int j = 128 * (w - 1) + 32 * b + lane;
            if (j < x.jn) rows[b] = a.x_scales + (size_t)(x.begin + x.j0 + j) * a.SC;
          }
        }
      }
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        v[b] = make_uint4(0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu);
        if (!rows[b]) continue;
        if (whole) {
          v[b] = __ldg(reinterpret_cast<const uint4*>(rows[b] + q_load * 16));
        } else {
          const uint32_t early = reinterpret_cast<uintptr_t>(rows[b]) & 2;
          const uint8_t* from = rows[b] + q_load * 16 - early;
          const int left = blocks - q_load * 16 + (int)early, in = a.SC - q_load * 16 + (int)early;
          auto word = [&](int h, uint32_t& to) {
            if (4 * h >= left) return;
            to = 4 * h + 4 <= in ? __ldg(reinterpret_cast<const uint32_t*>(from + 4 * h))
                                 : __ldg(reinterpret_cast<const uint16_t*>(from + 4 * h));
          };
          word(0, v[b].x);
          word(1, v[b].y);
          word(2, v[b].z);
          word(3, v[b].w);
          if (early) word(4, past[b]);
          shift = early * 8;
        }
      }
      if (++q_load == quads) q_load = 0, t_load += step;
    };
    uint4 v[kAhead][4];
    uint32_t past[kAhead][4] = {}, shift[kAhead] = {};
#pragma unroll
    for (int u = 0; u < kAhead; ++u) load(v[u], past[u], shift[u]);
    const int total = n_tiles > first ? ((n_tiles - 1 - first) / step + 1) * quads : 0;
    uint32_t s = 0, lap = 0;
    bool ok = true;
    for (int i = 0; i < total && ok; i += kAhead) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (i + u >= total || !ok) break;
        if (lap > 0 && !(ok = wait(&bars.sempty[s], (lap & 1) ^ 1, 1))) break;
        uint4* to = reinterpret_cast<uint4*>(s_sf + s * 4 * kScaleBytes + w * 512 + lane * 16);
        uint4 r[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint4 f = v[u][b];
          r[b].x = __funnelshift_r(f.x, f.y, shift[u]);
          r[b].y = __funnelshift_r(f.y, f.z, shift[u]);
          r[b].z = __funnelshift_r(f.z, f.w, shift[u]);
          r[b].w = __funnelshift_r(f.w, past[u][b], shift[u]);
        }
        to[0] = make_uint4(r[0].x, r[1].x, r[2].x, r[3].x);
        to[kScaleBytes / 16] = make_uint4(r[0].y, r[1].y, r[2].y, r[3].y);
        to[2 * kScaleBytes / 16] = make_uint4(r[0].z, r[1].z, r[2].z, r[3].z);
        to[3 * kScaleBytes / 16] = make_uint4(r[0].w, r[1].w, r[2].w, r[3].w);
        __syncwarp();
        if (lane == 0) async::mbar_arrive(&bars.swritten[s]);
        if (++s == kScaleRing) s = 0, ++lap;
        load(v[u], past[u], shift[u]);
      }
    }
  } else if (MX && warp == 3) {
    // ---- the scales' way from ordinary stores to the tensor copies ----
    const int quads = (sh.KK + 511) / 512;
    const int total = n_tiles > first ? ((n_tiles - 1 - first) / step + 1) * quads : 0;
    uint32_t s = 0, lap = 0;
    for (int i = 0; i < total; ++i) {
      if (!wait(&bars.swritten[s], lap & 1, 1)) break;
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) arrive_cluster(leader_addr(smem_u32(&bars.sfull[s])));
      if (++s == kScaleRing) s = 0, ++lap;
    }
  } else if (warp >= 4) {
    // ---- results ----
    const int q = warp & 3, half = (warp - 4) >> 2;
    uint8_t* stage = staging + (warp - 4) * kStagingBytes<OP, ACT>;
    uint32_t buf = 0;
    bool ok = true;
    for (int t = first; t < n_tiles && ok; t += step) {
      const Tile x = tile_at<OP, MX>(sh, s_begin, s_tile, a.G, t);
      const int i_cta = x.i0 + (int)rank * 128;
      if (x.nkb == 0) {
        if (i_cta < sh.I) store_zeros<F32>(a, sh, x, i_cta);
        continue;
      }
      const uint32_t b = buf & 1, use = buf >> 1;
      ++buf;
      Saved saved;
      if (OP == kDx && ACT) load_saved(a, sh, x, i_cta + 32 * q, 32 * half, saved);
      if (!(ok = wait(&bars.tfull[b], use & 1, 2 + x.nkb / 65536))) break;
      fence_after();
      const uint32_t src = tmem + b * NT + ((uint32_t)(q * 32) << 16);
      if constexpr (OP == kDw) {
        constexpr int kCols = F32 ? 16 : 32;
        for (int c0 = kCols * half; c0 < x.jn; c0 += 2 * kCols)
          drain_dw<T, F32>(sh, &map_out, x, i_cta + 32 * q, c0, src, stage);
      } else {
        for (int c0 = 32 * half; c0 < x.jn; c0 += 64)
          drain<OP, T, ACT>(a, sh, x, i_cta + 32 * q, c0, src, stage, saved);
      }
      fence_before();
      __syncwarp();
      if (lane == 0) arrive_cluster_relaxed(leader_addr(smem_u32(&bars.tempty[b])));
    }
    if (OP == kDw) tma_store_wait();
  }
  __syncwarp();
  fence_before();
  cluster_sync();
  fence_after();
  if (warp == 1) tmem_free(tmem, kTmemCols);
}

// ---- host ----
template <Op OP, typename T, bool F32, bool ACT, bool MX>
cudaError_t launch_t(const Args& a, const Shape& sh, const CUtensorMap& ma, const CUtensorMap& mb,
                     const CUtensorMap& out, const FewMaps& few, cudaStream_t s) {
  constexpr auto kernel = gemm_kernel<OP, T, F32, ACT, MX>;
  const size_t smem = 1024 + (size_t)kStages<OP, ACT, MX> * kStageBytes +
                      kDrainWarps * kStagingBytes<OP, ACT> +
                      (MX ? kScaleRing * 4 * kScaleBytes : 0) + 8 * ((size_t)a.G + 1);
  cudaError_t e = prepare_kernel<kernel>(smem);
  if (e != cudaSuccess) return e;
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorUnknown;
  const int64_t most = OP == kDw ? (int64_t)a.G * sh.tiles_i * sh.tiles_j
                                 : (int64_t)sh.tiles_i * (a.R / kNT<MX> + std::min(a.G, a.R));
  const int clusters = (int)std::min<int64_t>(sms / 2, most);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(clusters * 2);
  cfg.blockDim = dim3(kThreads<MX>);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {2, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a, sh, ma, mb, out, few);
}

// B's maps, rows of K elements 64 (16-bit) or 128 (bytes) at a time.
bool make_b(CUtensorMap* mb, FewMaps* few, const void* p, MapType type, uint64_t cols, uint64_t rows) {
  const uint64_t size = type == kMapU8 ? 1 : 2, d[] = {cols, rows}, st[] = {size * cols};
  const uint32_t inner = type == kMapU8 ? 128 : 64, b[] = {inner, 128}, b64[] = {inner, 64}, b32[] = {inner, 32};
  return make_map(mb, p, type, 2, d, st, b) && make_map(&few->b64, p, type, 2, d, st, b64) &&
         make_map(&few->b32, p, type, 2, d, st, b32);
}

template <typename T>
cudaError_t launch_op(Op op, const Args& a, cudaStream_t s) {
  const MapType type = T::kBf16 ? kMapBF16 : kMapF16;
  const uint64_t G = a.G, R = a.R, N = a.N, K = a.K;
  CUtensorMap ma, mb;
  FewMaps few = {};
  Shape sh = {};
  if (op == kForward) {
    sh.n_out = a.act ? a.N / 2 : a.N;
    sh.I = a.N;
    sh.KK = a.K;
    sh.tiles_i = (a.N + 255) / 256;
    if (!make_b(&mb, &few, a.x, type, K, R)) return cudaErrorUnknown;
    if (a.act) {
      const uint64_t n = N / 2, d[] = {K, 16, 2, n / 16, G}, st[] = {2 * K, 2 * n * K, 32 * K, 2 * N * K};
      const uint32_t b[] = {64, 16, 2, 4, 1};
      if (!make_map(&ma, a.w, type, 5, d, st, b)) return cudaErrorUnknown;
      return launch_t<kForward, T, false, true, false>(a, sh, ma, mb, ma, few, s);
    }
    const uint64_t d[] = {K, N, G}, st[] = {2 * K, 2 * N * K};
    const uint32_t b[] = {64, 128, 1};
    if (!make_map(&ma, a.w, type, 3, d, st, b)) return cudaErrorUnknown;
    return launch_t<kForward, T, false, false, false>(a, sh, ma, mb, ma, few, s);
  }
  if (op == kDx) {
    sh.I = a.K;
    sh.tiles_i = (a.K + 255) / 256;
    sh.KK = a.N;
    sh.whole = K % 64 == 0;
    if (!make_b(&mb, &few, a.x, type, N, R)) return cudaErrorUnknown;
    if (sh.whole) {
      const uint64_t d[] = {64, N, K / 64, G}, st[] = {2 * K, 128, 2 * N * K};
      const uint32_t b[] = {64, 64, 2, 1};
      if (!make_map(&ma, a.w, type, 4, d, st, b)) return cudaErrorUnknown;
    } else {
      const uint64_t d[] = {K, N, G}, st[] = {2 * K, 2 * N * K};
      const uint32_t b[] = {64, 64, 1};
      if (!make_map(&ma, a.w, type, 3, d, st, b)) return cudaErrorUnknown;
    }
    return a.pre_in ? launch_t<kDx, T, false, true, false>(a, sh, ma, mb, ma, few, s)
                    : launch_t<kDx, T, false, false, false>(a, sh, ma, mb, ma, few, s);
  }
  sh.I = a.N;
  sh.J = a.K;
  sh.tiles_i = (a.N + 255) / 256;
  sh.tiles_j = (a.K + kNT<false> - 1) / kNT<false>;
  sh.whole = K % 64 == 0 && N % 64 == 0;
  if (sh.whole) {
    const uint64_t d[] = {64, R, N / 64}, st[] = {2 * N, 128}, db[] = {64, R, K / 64}, sb[] = {2 * K, 128};
    const uint32_t b[] = {64, 64, 2};
    if (!make_map(&ma, a.w, type, 3, d, st, b) || !make_map(&mb, a.x, type, 3, db, sb, b))
      return cudaErrorUnknown;
  } else {
    const uint64_t d[] = {N, R}, st[] = {2 * N}, db[] = {K, R}, sb[] = {2 * K};
    const uint32_t b[] = {64, 64};
    if (!make_map(&ma, a.w, type, 2, d, st, b) || !make_map(&mb, a.x, type, 2, db, sb, b))
      return cudaErrorUnknown;
  }
  // The result: 64 bytes of 32 rows at a time.
  const bool f32 = a.out_dtype == 2;
  const uint64_t size = f32 ? 4 : 2, dd[] = {K, N, G}, sd[] = {size * K, size * N * K};
  const uint32_t bd[] = {f32 ? 16u : 32u, 32, 1};
  CUtensorMap md;
  if (!make_map(&md, a.out, f32 ? kMapF32 : type, 3, dd, sd, bd, kSwizzle64)) return cudaErrorUnknown;
  return f32 ? launch_t<kDw, T, true, false, false>(a, sh, ma, mb, md, few, s)
             : launch_t<kDw, T, false, false, false>(a, sh, ma, mb, md, few, s);
}

// Forward from mx fp8 operands; T is the output's type.
template <typename T>
cudaError_t launch_mx(const Args& a, cudaStream_t s) {
  const uint64_t G = a.G, R = a.R, N = a.N, K = a.K;
  CUtensorMap ma, mb;
  FewMaps few = {};
  Shape sh = {};
  sh.n_out = a.act ? a.N / 2 : a.N;
  sh.I = a.N;
  sh.KK = a.K;
  sh.tiles_i = (a.N + 255) / 256;
  if (!make_b(&mb, &few, a.x, kMapU8, K, R)) return cudaErrorUnknown;
  if (a.act) {
    const uint64_t n = N / 2, d[] = {K, 16, 2, n / 16, G}, st[] = {K, n * K, 16 * K, N * K};
    const uint32_t b[] = {128, 16, 2, 4, 1};
    if (!make_map(&ma, a.w, kMapU8, 5, d, st, b)) return cudaErrorUnknown;
    return launch_t<kForward, T, false, true, true>(a, sh, ma, mb, ma, few, s);
  }
  const uint64_t d[] = {K, N, G}, st[] = {K, N * K};
  const uint32_t b[] = {128, 128, 1};
  if (!make_map(&ma, a.w, kMapU8, 3, d, st, b)) return cudaErrorUnknown;
  return launch_t<kForward, T, false, false, true>(a, sh, ma, mb, ma, few, s);
}

}  // namespace

int launch_gemm(Op op, const Args& a, cudaStream_t s) {
  cudaError_t e;
  if (a.R == 0) {
    if (op != kDw) return CQ_OK;
    e = cudaMemsetAsync(a.out, 0, (size_t)a.G * a.N * a.K * (a.out_dtype == 2 ? 4 : 2), s);
  } else if (a.x_dtype >= kMxE4M3) {
    e = a.out_dtype == 1 ? launch_mx<F16>(a, s) : launch_mx<BF16>(a, s);
  } else {
    e = a.x_dtype == kF16 ? launch_op<F16>(op, a, s) : launch_op<BF16>(op, a, s);
  }
  return e == cudaSuccess ? CQ_OK : CQ_ERR_CUDA;
}

int gemm_status(uint32_t* read, cudaStream_t s) { return status_word(g_status, read, s); }

}  // namespace expert
}  // namespace cq
