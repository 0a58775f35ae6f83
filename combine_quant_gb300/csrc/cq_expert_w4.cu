// cq_expert_w4.cu -- the experts' product with 4-bit weights, for few rows per
// expert (decoding): bound by reading the codes, k / 2 bytes a weight row.
//
// W[i, k] = (q - z) s, one s (and z) per `group` of k. The codes go into the
// 16-bit product of mma.m16n8k16 as exact small integers: OR-ing a nibble into
// the fraction of a power of two gives 128 + q (bf16) or 64 + q (fp16) in one
// instruction. Over one group sum_k (q - z) x = sum_k (OFF + q) x - (OFF + z)
// sum_k x; the second term is what the accumulator starts from (sum_k x comes
// from the same instruction with ones for weights), so it costs nothing per
// weight row, and s multiplies the group's f32 sum: no rounding but f32's.
//
// One tile: 32 MTW weight rows (SwiGLU: half gates, half ups) x up to 8 NT
// tokens. Warp 10 streams 256 of k per stage with tiled copies (codes in 128-byte
// rows, x in 64-byte rows, both swizzled: no bank conflicts). Warps 0-7 multiply:
// 4 take 64 of k each, times 2 halves of the rows, so each code is read from
// shared memory once and each x twice; their sums are added in a fixed order at
// the end. Warps 8 and 9 bring the scales as floats in the order the multiplying
// threads want them. The k order inside 32 is permuted alike in codes and x: a
// thread's nibbles i and i + 4 of one word are neighbours in the product.
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
using async::release_slot;

__device__ uint32_t g_status;  // CQ_ST_* bits of these kernels on this device

constexpr int kThreads = 352;
constexpr int kMul = 256;      // multiplying threads
constexpr int kLoad = 64;      // threads that bring scales
constexpr int kStages = 4, kEntries = 4;

struct Shape {
  int n_out;     // outputs (with SwiGLU half the weight rows)
  int tiles_n;   // tiles along the weight rows
  int KG;        // groups of k
  int group;
  int vec;       // scales may be read in 16-byte (zeros: 8-byte) pieces
};

struct Bars {
  uint64_t full[kStages], empty[kStages], sfull[kEntries], sempty[kEntries];
};

struct Tile {
  int e, begin, j0, jn, o0, nt;  // o0: first row of each half
};

template <int MTW, int NTMAX, bool ACT>
__device__ __forceinline__ Tile tile_at(const Shape& sh, const int* s_begin, const int* s_tile,
                                        int G, int t) {
  Tile x;
  x.e = expert_of(s_tile, G, t);
  x.begin = s_begin[x.e];
  const int rows = s_begin[x.e + 1] - x.begin;
  const int parts = (rows + 8 * NTMAX - 1) / (8 * NTMAX);
  const int step = ((rows + parts - 1) / parts + 7) / 8 * 8;
  const int l = t - s_tile[x.e];
  x.j0 = l % parts * step;
  x.jn = min(step, rows - x.j0);
  x.o0 = l / parts * (ACT ? 16 * MTW : 32 * MTW);
  const int nt = (x.jn + 7) / 8;
  x.nt = nt > 2 ? 4 : nt;
  return x;
}

template <bool kBf16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kBf16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Nibbles i and i + 4 of a word of eight codes as OFF + q in two 16-bit halves.
template <bool kBf16, int I>
__device__ __forceinline__ uint32_t codes2(uint32_t w) {
  if constexpr (kBf16) {
    return ((w >> (4 * I)) & 0x000f000fu) | 0x43004300u;  // 128 + q
  } else {
    const uint32_t v = I == 0 ? w << 4 : w >> (I == 0 ? 0 : 4 * I - 4);
    return (v & 0x00f000f0u) | 0x54005400u;  // 64 + q
  }
}

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

template <int MTW>
constexpr int kScaleStride = MTW == 4 ? 12 : 2 * MTW;  // floats of one row group, padded

// One stage of one multiplying warp: 64 of k (two blocks of 32) of its half.
template <typename T, int MTW, int NT, int NTMAX, bool ZEROS, bool G32>
__device__ __forceinline__ void multiply(float (&acc)[MTW][NTMAX][4], uint32_t sw, uint32_t sx,
                                         const float* scale, const float* zero, int kw) {
  constexpr bool kBf16 = T::kBf16;
  constexpr float kOff = kBf16 ? 128.f : 64.f;
  constexpr uint32_t kOne = kBf16 ? 0x3f803f80u : 0x3c003c00u;
  constexpr int kSpans = G32 ? 2 : 1;  // spans of k with one scale
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  uint32_t b[2][NT][4];
  float sum[kSpans][NT][4];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = 8 * n + g;
      uint32_t v0, v1, v2, v3;
      asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(v0), "=r"(v1), "=r"(v2), "=r"(v3)
                   : "r"(sx + (2 * kw + h) * (512 * NT) + row * 64 + ((q ^ ((row >> 1) & 3)) << 4))
                   : "memory");
      b[h][n][0] = __byte_perm(v0, v2, 0x5410);
      b[h][n][1] = __byte_perm(v0, v2, 0x7632);
      b[h][n][2] = __byte_perm(v1, v3, 0x5410);
      b[h][n][3] = __byte_perm(v1, v3, 0x7632);
    }
  const uint32_t ones[4] = {kOne, kOne, kOne, kOne};
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int p = 0; p < kSpans; ++p) {
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[p][n][i] = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (!G32 || h == p) {
          mma<kBf16>(sum[p][n], ones, b[h][n][0], b[h][n][1]);
          mma<kBf16>(sum[p][n], ones, b[h][n][2], b[h][n][3]);
        }
    }
#pragma unroll
  for (int m = 0; m < MTW; ++m) {
    const uint32_t at = sw + (16 * m + g) * 128 + 4 * q;
    float d[NT][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int p = G32 ? h : 0;
      const uint32_t c = ((uint32_t)(2 * kw + h) ^ (uint32_t)g) << 4;
      const uint32_t w0 = ld_shared_u32(at + c), w1 = ld_shared_u32(at + c + 1024);
      if (G32 || h == 0) {
        float o0 = -(kOff + 8.f), o1 = o0;
        if constexpr (ZEROS) {
          const float2 o = *reinterpret_cast<const float2*>(zero + p * 16 * kScaleStride<MTW> + 2 * m);
          o0 = o.x;
          o1 = o.y;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          d[n][0] = o0 * sum[p][n][0];
          d[n][1] = o0 * sum[p][n][1];
          d[n][2] = o1 * sum[p][n][0];
          d[n][3] = o1 * sum[p][n][1];
        }
      }
      const uint32_t a0[4] = {codes2<kBf16, 0>(w0), codes2<kBf16, 0>(w1), codes2<kBf16, 1>(w0), codes2<kBf16, 1>(w1)};
      const uint32_t a1[4] = {codes2<kBf16, 2>(w0), codes2<kBf16, 2>(w1), codes2<kBf16, 3>(w0), codes2<kBf16, 3>(w1)};
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma<kBf16>(d[n], a0, b[h][n][0], b[h][n][1]);
        mma<kBf16>(d[n], a1, b[h][n][2], b[h][n][3]);
      }
      if (G32 || h == 1) {
        const float2 sc = *reinterpret_cast<const float2*>(scale + p * 16 * kScaleStride<MTW> + 2 * m);
        const float s0 = sc.x, s1 = sc.y;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          acc[m][n][0] = fmaf(s0, d[n][0], acc[m][n][0]);
          acc[m][n][1] = fmaf(s0, d[n][1], acc[m][n][1]);
          acc[m][n][2] = fmaf(s1, d[n][2], acc[m][n][2]);
          acc[m][n][3] = fmaf(s1, d[n][3], acc[m][n][3]);
        }
      }
    }
  }
}

__device__ __forceinline__ void bar_mul() { asm volatile("bar.sync 1, %0;" ::"n"(kMul) : "memory"); }

template <typename T>
__device__ __forceinline__ void store1(void* p, size_t i, float v) {
  if constexpr (T::kBf16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p)[i] = __float2half_rn(v);
}

template <typename T, int MTW, int NTMAX, bool ACT, bool ZEROS, bool G32>
__global__ void __launch_bounds__(kThreads, NTMAX == 1 ? 2 : 1)
w4_kernel(const __grid_constant__ Args a, const __grid_constant__ Shape sh,
          const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x1,
          const __grid_constant__ CUtensorMap map_x2, const __grid_constant__ CUtensorMap map_x4) {
  constexpr int kHalf = 16 * MTW * 128;                 // code bytes of one half of a stage
  constexpr int kStage = 2 * kHalf + 8 * 512 * NTMAX;
  constexpr int SG = kScaleStride<MTW>;
  constexpr int kEntry = 8 * 2 * 8 * SG;                // floats of one entry of scales
  constexpr int kRed = 4 * 2 * 8 * NTMAX * 20;          // floats of the sums' exchange
  extern __shared__ __align__(1024) uint8_t dyn[];
  __shared__ Bars bars;
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
  float* s_scale = reinterpret_cast<float*>(ring + kStages * kStage);
  float* s_zero = s_scale + kEntries * kEntry;
  float* red = s_zero + (ZEROS ? kEntries * kEntry : 0);
  int* s_begin = reinterpret_cast<int*>(red + kRed);
  int* s_tile = s_begin + a.G + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    prefetch_map(&map_w);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars.full[s], 1);
      mbar_init(&bars.empty[s], kMul / 32);
    }
    for (int s = 0; s < kEntries; ++s) {
      mbar_init(&bars.sfull[s], kLoad);
      mbar_init(&bars.sempty[s], kMul / 32);
    }
    async::mbar_fence_init();
  }
  griddep_wait();
  const bool bad = group_scan<kThreads>(a, s_begin, s_tile, [&](int rows) {
    return sh.tiles_n * ((rows + 8 * NTMAX - 1) / (8 * NTMAX));
  });
  if (bad && blockIdx.x == 0) atomicOr(&g_status, (uint32_t)CQ_ST_BAD_ROWS);
  const int n_tiles = s_tile[a.G];
  const int n_stages = (a.K + 255) / 256, n_entries = (sh.KG + 7) / 8;
  const int spe = sh.group / 32;  // stages that one entry of 8 groups serves: 1, 2, 4
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_wait(bar, parity)) return true;
    atomicOr(&g_status, (uint32_t)CQ_ST_TIMEOUT);
    return false;
  };

  if (warp == 10) {
    // ---- copies of codes and x ----
    uint32_t s = 0, lap = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < n_tiles && ok; t += gridDim.x) {
      const Tile x = tile_at<MTW, NTMAX, ACT>(sh, s_begin, s_tile, a.G, t);
      const CUtensorMap* mx = NTMAX == 1 || x.nt == 1 ? &map_x1 : x.nt == 2 ? &map_x2 : &map_x4;
      const int r1 = ACT ? sh.n_out + x.o0 : x.o0 + 16 * MTW;
      for (int st = 0; st < n_stages; ++st) {
        if (lap > 0 && !(ok = wait(&bars.empty[s], (lap & 1) ^ 1))) break;
        if (elect_one()) {
          const uint32_t base = smem_u32(ring + s * kStage), bar = smem_u32(&bars.full[s]);
          mbar_arrive_expect_tx(&bars.full[s], 2 * kHalf + 8 * 512 * x.nt);
          tma_load3<1>(base, &map_w, st * 128, x.o0, x.e, bar);
          tma_load3<1>(base + kHalf, &map_w, st * 128, r1, x.e, bar);
#pragma unroll
          for (int c = 0; c < 8; ++c)
            tma_load2<1>(base + 2 * kHalf + c * 512 * x.nt, mx, st * 256 + c * 32, x.begin + x.j0, bar);
        }
        __syncwarp();
        if (++s == kStages) s = 0, ++lap;
      }
    }
    if (!ok) {  // gave up: let the copies in flight land (with a limit)
      for (int v = 0; v < kStages; ++v) {
        const uint32_t laps = lap + ((uint32_t)v < s ? 1 : 0);
        if (laps > 0) mbar_wait(&bars.full[v], (laps - 1) & 1);
      }
    }
  } else if (warp >= 8) {
    // ---- scales: a thread takes rows r and r + 64, 8 groups at a time, two entries ahead ----
    constexpr int kRows = (32 * MTW + kLoad - 1) / kLoad;
    const uint16_t* scales = static_cast<const uint16_t*>(a.scales4);
    const int per_cta = n_tiles > (int)blockIdx.x ? (n_tiles - 1 - blockIdx.x) / gridDim.x + 1 : 0;
    const int total = per_cta * n_entries;
    struct Piece {
      uint4 s[kRows];
      uint2 z[kRows];
    } p0, p1;
    int cur = -1;
    size_t row_at[kRows] = {};
    bool in[kRows] = {};
    auto load = [&](int i, Piece& p) {
#pragma unroll
      for (int b = 0; b < kRows; ++b) p.s[b] = make_uint4(0, 0, 0, 0), p.z[b] = make_uint2(0, 0);
      if (i >= total) return;
      const int tile = i / n_entries, first = (i - tile * n_entries) * 8;
      if (tile != cur) {
        cur = tile;
        const Tile x = tile_at<MTW, NTMAX, ACT>(sh, s_begin, s_tile, a.G, blockIdx.x + tile * gridDim.x);
#pragma unroll
        for (int b = 0; b < kRows; ++b) {
          const int r = threadIdx.x - kMul + b * kLoad, half = r / (16 * MTW), r16 = r % (16 * MTW);
          const int row = ACT ? half * sh.n_out + x.o0 + r16 : x.o0 + half * 16 * MTW + r16;
          in[b] = r < 32 * MTW && (ACT ? x.o0 + r16 < sh.n_out : row < a.N);
          row_at[b] = ((size_t)x.e * a.N + row) * sh.KG;
        }
      }
#pragma unroll
      for (int b = 0; b < kRows; ++b) {
        if (!in[b]) continue;
        const size_t at = row_at[b] + first;
        if (sh.vec) {
          p.s[b] = __ldg(reinterpret_cast<const uint4*>(scales + at));
          if (ZEROS) p.z[b] = __ldg(reinterpret_cast<const uint2*>(a.zeros4 + at));
        } else {
          uint32_t w[4] = {}, z[2] = {};
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (first + k < sh.KG) {
              w[k / 2] |= (uint32_t)__ldg(scales + at + k) << (16 * (k & 1));
              if (ZEROS) z[k / 4] |= (uint32_t)__ldg(a.zeros4 + at + k) << (8 * (k & 3));
            }
          p.s[b] = make_uint4(w[0], w[1], w[2], w[3]);
          p.z[b] = make_uint2(z[0], z[1]);
        }
      }
    };
    load(0, p0);
    load(1, p1);
    for (int i = 0; i < total; ++i) {
      const int s = i % kEntries;
      if (i >= kEntries && !wait(&bars.sempty[s], ((i / kEntries) & 1) ^ 1)) break;
#pragma unroll
      for (int b = 0; b < kRows; ++b) {
        const int r = threadIdx.x - kMul + b * kLoad;
        if (r >= 32 * MTW) continue;
        const int slot = (r / (16 * MTW) * 8 + r % 8) * SG + 2 * (r / 16 % MTW) + r / 8 % 2;
        const uint32_t w[4] = {p0.s[b].x, p0.s[b].y, p0.s[b].z, p0.s[b].w};
        float* to = s_scale + s * kEntry + slot;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          to[(2 * k) * 16 * SG] = T::lo(w[k]);
          to[(2 * k + 1) * 16 * SG] = T::hi(w[k]);
        }
        if (ZEROS) {
          constexpr float kOff = T::kBf16 ? 128.f : 64.f;
          float* tz = s_zero + s * kEntry + slot;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            tz[k * 16 * SG] = -(kOff + (float)(((k < 4 ? p0.z[b].x : p0.z[b].y) >> (8 * (k & 3))) & 255));
        }
      }
      async::mbar_arrive(&bars.sfull[s]);
      p0 = p1;
      load(i + 2, p1);
    }
  } else {
    // ---- products ----
    const int kw = warp & 3, half = warp >> 2, g = lane >> 2, q = lane & 3;
    uint32_t s = 0, lap = 0, ent = 0, elap = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < n_tiles && ok; t += gridDim.x) {
      const Tile x = tile_at<MTW, NTMAX, ACT>(sh, s_begin, s_tile, a.G, t);
      float acc[MTW][NTMAX][4] = {};
      for (int st = 0; st < n_stages; ++st) {
        const int sub = st % spe;
        if (sub == 0 && !(ok = wait(&bars.sfull[ent], elap & 1))) break;
        if (!(ok = wait(&bars.full[s], lap & 1))) break;
        if (st * 256 + kw * 64 < a.K) {
          const uint32_t base = smem_u32(ring + s * kStage);
          const int grp = (sub * 256 + kw * 64) / sh.group;  // within the entry
          const int at = ent * kEntry + ((grp * 2 + half) * 8 + g) * SG;
          const uint32_t sw = base + half * kHalf, sx = base + 2 * kHalf;
          if constexpr (NTMAX == 1) {
            multiply<T, MTW, 1, NTMAX, ZEROS, G32>(acc, sw, sx, s_scale + at, s_zero + at, kw);
          } else {
            if (x.nt == 1) multiply<T, MTW, 1, NTMAX, ZEROS, G32>(acc, sw, sx, s_scale + at, s_zero + at, kw);
            else if (x.nt == 2) multiply<T, MTW, 2, NTMAX, ZEROS, G32>(acc, sw, sx, s_scale + at, s_zero + at, kw);
            else multiply<T, MTW, 4, NTMAX, ZEROS, G32>(acc, sw, sx, s_scale + at, s_zero + at, kw);
          }
        }
        release_slot(&bars.empty[s]);
        if (++s == kStages) s = 0, ++lap;
        if (sub == spe - 1 || st == n_stages - 1) {
          __syncwarp();
          if (lane == 0) async::mbar_arrive(&bars.sempty[ent]);
          if (++ent == kEntries) ent = 0, ++elap;
        }
      }
      if (!ok) break;
      // Sums of the four k warps, added in order: 16 rows of both halves at a time.
#pragma unroll
      for (int m = 0; m < MTW; ++m) {
        bar_mul();
        float* to = red + (kw * 2 + half) * (8 * NTMAX * 20);
#pragma unroll
        for (int n = 0; n < NTMAX; ++n)
          if (n < x.nt) {
            to[(8 * n + 2 * q) * 20 + g] = acc[m][n][0];
            to[(8 * n + 2 * q + 1) * 20 + g] = acc[m][n][1];
            to[(8 * n + 2 * q) * 20 + g + 8] = acc[m][n][2];
            to[(8 * n + 2 * q + 1) * 20 + g + 8] = acc[m][n][3];
          }
        bar_mul();
        auto total = [&](int h, int j, int i) {
          float v = 0.f;
#pragma unroll
          for (int w = 0; w < 4; ++w) v += red[((w * 2 + h) * 8 * NTMAX + j) * 20 + i];
          return v;
        };
        if constexpr (ACT) {
          for (int v = threadIdx.x; v < x.jn * 16; v += kMul) {
            const int i = v & 15, j = v >> 4, o = x.o0 + 16 * m + i;
            const float gv = total(0, j, i), uv = total(1, j, i);
            if (o < sh.n_out)
              store1<T>(a.out, (size_t)(x.begin + x.j0 + j) * sh.n_out + o,
                        __fdividef(uv * gv, 1.f + __expf(-gv)));
          }
        } else {
          for (int v = threadIdx.x; v < x.jn * 32; v += kMul) {
            const int i = v & 15, h = (v >> 4) & 1, j = v >> 5, o = x.o0 + 16 * MTW * h + 16 * m + i;
            const float y = total(h, j, i);
            if (o < sh.n_out) store1<T>(a.out, (size_t)(x.begin + x.j0 + j) * sh.n_out + o, y);
          }
        }
      }
    }
  }
}

// ---- host ----
template <typename T, int MTW, int NTMAX, bool ACT, bool ZEROS, bool G32>
cudaError_t launch_t(const Args& a, cudaStream_t s) {
  constexpr auto kernel = w4_kernel<T, MTW, NTMAX, ACT, ZEROS, G32>;
  Shape sh = {};
  sh.n_out = ACT ? a.N / 2 : a.N;
  sh.tiles_n = ACT ? (sh.n_out + 16 * MTW - 1) / (16 * MTW) : (a.N + 32 * MTW - 1) / (32 * MTW);
  sh.group = a.group;
  sh.KG = a.K / a.group;
  sh.vec = sh.KG % 8 == 0;
  const uint64_t G = a.G, R = a.R, N = a.N, K = a.K;
  CUtensorMap mw, mx[3];
  const uint64_t dw[] = {K / 2, N, G}, sw[] = {K / 2, N * (K / 2)}, dx[] = {K, R}, sx[] = {K * 2};
  const uint32_t bw[] = {128, 16 * MTW, 1};
  if (!make_map(&mw, a.w, kMapU8, 3, dw, sw, bw, kSwizzle128)) return cudaErrorUnknown;
  for (int i = 0; i < (NTMAX == 1 ? 1 : 3); ++i) {
    const uint32_t bx[] = {32, 8u << i};
    if (!make_map(&mx[i], a.x, T::kBf16 ? kMapBF16 : kMapF16, 2, dx, sx, bx, kSwizzle64))
      return cudaErrorUnknown;
  }
  if (NTMAX == 1) mx[1] = mx[2] = mx[0];
  const size_t smem = 1024 + kStages * (size_t)(2 * 16 * MTW * 128 + 8 * 512 * NTMAX) +
                      (ZEROS ? 2 : 1) * kEntries * 8 * 2 * 8 * kScaleStride<MTW> * 4 +
                      4 * 2 * 8 * NTMAX * 20 * 4 + 8 * ((size_t)a.G + 1);
  cudaError_t e = prepare_kernel<kernel>(smem);
  if (e != cudaSuccess) return e;
  int per_sm = 0;
  e = occupancy_blocks<kernel>(kThreads, smem, &per_sm);
  if (e != cudaSuccess) return e;
  const int sms = sm_count();
  if (sms <= 0 || per_sm <= 0) return cudaErrorUnknown;
  const int64_t most = (int64_t)sh.tiles_n * (a.R / (8 * NTMAX) + std::min(a.G, a.R));
  const int grid = (int)std::min<int64_t>((int64_t)sms * per_sm, most);
  return launch_pdl(kernel, dim3(grid), dim3(kThreads), smem, s, a, sh, mw, mx[0], mx[1], mx[2]);
}

template <typename T, int MTW, int NTMAX, bool ACT>
cudaError_t launch_g(const Args& a, cudaStream_t s) {
  if (a.zeros4)
    return a.group == 32 ? launch_t<T, MTW, NTMAX, ACT, true, true>(a, s)
                         : launch_t<T, MTW, NTMAX, ACT, true, false>(a, s);
  return a.group == 32 ? launch_t<T, MTW, NTMAX, ACT, false, true>(a, s)
                       : launch_t<T, MTW, NTMAX, ACT, false, false>(a, s);
}

// Up to 8 rows in all take the narrow kernel with tiles small enough to reach
// every SM; more rows the one of 128 weight rows and up to 32 tokens.
template <typename T, bool ACT>
cudaError_t launch_a(const Args& a, cudaStream_t s) {
  if (a.R > 8) return launch_g<T, 4, 4, ACT>(a, s);
  const int64_t rows = (int64_t)std::min(a.G, a.R) * a.N;  // most weight rows read
  if (rows >= 128 * 152 * 2) return launch_g<T, 4, 1, ACT>(a, s);
  return launch_g<T, 1, 1, ACT>(a, s);
}

}  // namespace

int launch_w4(const Args& a, cudaStream_t s) {
  if (a.R == 0) return CQ_OK;
  cudaError_t e;
  if (a.x_dtype == kF16) e = a.act ? launch_a<F16, true>(a, s) : launch_a<F16, false>(a, s);
  else e = a.act ? launch_a<BF16, true>(a, s) : launch_a<BF16, false>(a, s);
  return e == cudaSuccess ? CQ_OK : CQ_ERR_CUDA;
}

int w4_status(uint32_t* status, cudaStream_t s) { return read_status_word(g_status, status, s); }

}  // namespace expert
}  // namespace cq
