// cq_expert_w4.cu -- the experts' product with 4-bit weights, for few rows per
// expert (decoding): bound by reading the codes, k / 2 bytes a weight row.
//
// W[i, k] = (q - z) s, one s (and z) per `group` of k. The codes go into the
// 16-bit product of mma.m16n8k16 exactly: OR-ing a nibble into the fraction of 1
// gives 1 + q / OFF in one instruction, OFF = 128 (bf16) or 64 (fp16). Over one
// group sum_k (q - z) x = OFF (sum_k (1 + q / OFF) x - (1 + z / OFF) sum_k x); the
// second term is what the accumulator starts from (sum_k x comes from the same
// instruction with ones for weights), so it costs nothing per weight row, s
// multiplies the group's f32 sum, and OFF the result: no rounding but f32's. (With
// OFF + q, the same in every bit, rows beyond 2^120 left f32's range on the way.)
//
// One tile: 64 MTW weight rows (SwiGLU: half gates, half ups) x up to 16
// tokens, 512 of k per stage of the ring. Warp 22 streams codes (128-byte rows)
// and x (64-byte rows) with tiled copies, both swizzled so that no access below
// meets a bank twice. Warps 16-19 put each 8 of x into the order in which the
// nibbles come out of a word (i, i + 4 are neighbours in the product) and form
// the sums of x. Warps 20-21 bring the scales as floats in the order the
// multiplying threads read them. Warps 0-15 multiply: 4 shares of k times 4 of
// the rows; the four k shares' sums are added in a fixed order at the end.
//
// mma.sync rather than tcgen05: the codes have to pass through registers anyway,
// and a group's sum has to come back to them to meet its scale. What bounds it:
// the codes' bytes as far as the memory goes (5.9 TB/s with the multiplying taken
// out), in practice the multiplying warps' instructions. Measured on one GB300, 32
// experts, hidden 7168, SwiGLU with n 2048, groups of 128 (485 MB): up to 8 rows an
// expert 112 us (4.3 TB/s), 16 rows 143 us, every further 16 rows about 130 us; one
// row through 8192 x 8192 15.2 us, with groups of 32 and zero points 19.5 us. 23 warps
// leave 80 registers a thread, and 34 of the 60 forms spill (172 bytes of reloads at
// most).
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

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
using async::release_slot;

__device__ uint32_t g_status;  // CQ_ST_* bits of these kernels on this device

constexpr int kMulWarps = 16, kSumWarps = 4, kScaleWarps = 2;
constexpr int kThreads = 32 * (kMulWarps + kSumWarps + kScaleWarps + 1);
constexpr int kMaxStages = 8;
constexpr int kMaxNT = 2;  // blocks of 8 tokens of a tile, at most

// Dynamic shared memory that a CTA may use, beside a little static.
constexpr size_t kSmemBytes = 227 * 1024 - 1024;

struct Shape {
  int n_out;     // outputs (with SwiGLU half the weight rows)
  int tiles_n;   // tiles along the weight rows
  int KG;        // groups of k
  int shift;     // log2 of a group's length
  int vec;       // rows of scales are whole pieces of 8 groups (2), of 4 (1; or not: ANY)
  int stages;    // stages of the ring
};

struct Bars {
  uint64_t full[kMaxStages];   // codes and x have landed
  uint64_t ready[kMaxStages];  // x in order, sums and scales there
  uint64_t empty[kMaxStages];
};

struct Tile {
  int e, begin, j0, jn, o0, nt;  // o0: first row of the tile (of each half)
};

template <int MTW, bool ACT>
__device__ __forceinline__ Tile tile_at(const Shape& sh, const int* s_begin, const int* s_tile,
                                        int G, int t) {
  Tile x;
  x.e = expert_of(s_tile, G, t);
  x.begin = s_begin[x.e];
  const int rows = s_begin[x.e + 1] - x.begin;
  // Whole parts and a rest (a rest of up to 8 tokens costs less than equal parts would).
  // The parts of one set of weight rows lie tiles_n apart: in flight together, so
  // the second finds the codes in L2, and spread over the CTAs.
  const int l = t - s_tile[x.e], part = l / sh.tiles_n;
  x.j0 = part * (8 * kMaxNT);
  x.jn = min(8 * kMaxNT, rows - x.j0);
  x.o0 = (l - part * sh.tiles_n) * (ACT ? 32 * MTW : 64 * MTW);
  x.nt = (x.jn + 7) / 8;
  return x;
}

// d = a b + c.
template <bool kBf16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                    float c0, float c1, float c2, float c3) {
  if constexpr (kBf16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// (v & mask) | magic in one instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t magic) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(v), "r"(mask), "r"(magic));
  return r;
}

// Nibbles i and i + 4 of a word of eight codes as 1 + q / OFF in two 16-bit halves.
template <bool kBf16, int I>
__device__ __forceinline__ uint32_t codes2(uint32_t w) {
  if constexpr (kBf16) return and_or(I == 0 ? w : w >> (4 * I), 0x000f000fu, 0x3f803f80u);  // 1 + q / 128
  else return and_or(I == 0 ? w << 4 : w >> (I == 0 ? 0 : 4 * I - 4), 0x00f000f0u, 0x3c003c00u);  // 1 + q / 64
}

// Sizes of a stage: codes, x, scales (and zero points) and sums of x.
template <int MTW, bool ZEROS, bool G32>
struct Stage {
  static constexpr int kRows = 64 * MTW;
  static constexpr int kChunk = kRows * 128;                // codes of 256 of k
  static constexpr int kX = 2 * kChunk;
  static constexpr int kScale = kX + 16 * 512 * kMaxNT;
  static constexpr int kGroups = G32 ? 16 : 8;              // most groups of 512 of k
  static constexpr int kGroupFloats = ZEROS ? 2 * kRows : kRows;  // of one group: s, or s and -(1 + z / OFF)
  static constexpr int kSum = kScale + kGroups * kGroupFloats * 4;
  static constexpr int kSpans = G32 ? 2 : 1;                // spans with one scale in 64 of k
  static constexpr int kBytes = (kSum + 8 * kSpans * 8 * kMaxNT * 4 + 1023) / 1024 * 1024;
};

// 64 of k (two blocks of 32) of one multiplying warp. sw0, sw1: this thread's
// code words of the two blocks (+ 2048 m, + 1024 for rows g + 8); sx: its x
// (+ (h NT + n) 512); sum, scale: of its tokens and rows.
template <typename T, int MTW, int NT, bool ZEROS, bool G32>
__device__ __forceinline__ void multiply(float (&acc)[MTW][kMaxNT][4], const uint8_t* sw0,
                                         const uint8_t* sw1, const uint8_t* sx, const float* sum,
                                         const float* scale) {
  constexpr bool kBf16 = T::kBf16;
  constexpr int kSpan = Stage<MTW, ZEROS, G32>::kGroupFloats;  // from one group's scales to the next
  // H blocks of 32 of k under one scale, from block h0.
  auto span = [&](auto first, auto blocks) {
    constexpr int h0 = decltype(first)::value, H = decltype(blocks)::value, p = G32 ? h0 : 0;
    // All of a block's products side by side: MTW x NT chains in flight.
    float d[MTW][NT][4];
#pragma unroll
    for (int h = 0; h < H; ++h) {
      uint4 b[NT];
      uint32_t a0[MTW][4], a1[MTW][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) b[n] = *reinterpret_cast<const uint4*>(sx + ((h0 + h) * NT + n) * 512);
#pragma unroll
      for (int m = 0; m < MTW; ++m) {
        const uint8_t* at = (h0 + h ? sw1 : sw0) + 2048 * m;
        const uint32_t w0 = *reinterpret_cast<const uint32_t*>(at);
        const uint32_t w1 = *reinterpret_cast<const uint32_t*>(at + 1024);
        a0[m][0] = codes2<kBf16, 0>(w0), a0[m][1] = codes2<kBf16, 0>(w1);
        a0[m][2] = codes2<kBf16, 1>(w0), a0[m][3] = codes2<kBf16, 1>(w1);
        a1[m][0] = codes2<kBf16, 2>(w0), a1[m][1] = codes2<kBf16, 2>(w1);
        a1[m][2] = codes2<kBf16, 3>(w0), a1[m][3] = codes2<kBf16, 3>(w1);
      }
      if (h == 0) {
        float2 c[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) c[n] = *reinterpret_cast<const float2*>(sum + p * 8 * kMaxNT + 8 * n);
#pragma unroll
        for (int m = 0; m < MTW; ++m) {
          float2 o = make_float2(1.f, 1.f);
          if constexpr (ZEROS) o = make_float2(scale[p * kSpan + 4 * m + 1], scale[p * kSpan + 4 * m + 3]);
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma<kBf16>(d[m][n], a0[m], b[n].x, b[n].y, o.x * c[n].x, o.x * c[n].y, o.y * c[n].x, o.y * c[n].y);
        }
      } else {
#pragma unroll
        for (int m = 0; m < MTW; ++m)
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma<kBf16>(d[m][n], a0[m], b[n].x, b[n].y, d[m][n][0], d[m][n][1], d[m][n][2], d[m][n][3]);
      }
#pragma unroll
      for (int m = 0; m < MTW; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
          mma<kBf16>(d[m][n], a1[m], b[n].z, b[n].w, d[m][n][0], d[m][n][1], d[m][n][2], d[m][n][3]);
    }
#pragma unroll
    for (int m = 0; m < MTW; ++m) {
      float2 f;
      if constexpr (ZEROS) f = make_float2(scale[p * kSpan + 4 * m], scale[p * kSpan + 4 * m + 2]);
      else f = *reinterpret_cast<const float2*>(scale + p * kSpan + 2 * m);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        acc[m][n][0] = fmaf(f.x, d[m][n][0], acc[m][n][0]);
        acc[m][n][1] = fmaf(f.x, d[m][n][1], acc[m][n][1]);
        acc[m][n][2] = fmaf(f.y, d[m][n][2], acc[m][n][2]);
        acc[m][n][3] = fmaf(f.y, d[m][n][3], acc[m][n][3]);
      }
    }
  };
  using std::integral_constant;
  if constexpr (G32) {
    span(integral_constant<int, 0>{}, integral_constant<int, 1>{});
    asm volatile("" ::: "memory");  // the second block's loads stay behind: 80 registers
    span(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  } else {
    span(integral_constant<int, 0>{}, integral_constant<int, 2>{});
  }
}

// This thread's byte offsets in a stage.
struct Places {
  uint32_t w, x, sum, scale, scale_next;
};

// All of k for one tile: false when a wait gave up.
template <typename T, int MTW, int NT, bool ZEROS, bool G32>
__device__ __forceinline__ bool multiply_tile(float (&acc)[MTW][kMaxNT][4], Bars& bars,
                                              const uint8_t* ring, int S, uint32_t& s, uint32_t& lap,
                                              const Places& at, int kw, int K) {
  using St = Stage<MTW, ZEROS, G32>;
  const uint32_t at_x = at.x + kw * 2 * 512 * NT;
  for (int left = K - kw * 64; left + kw * 64 > 0; left -= 512) {
    if (!mbar_wait_warp(&bars.ready[s], lap & 1)) return false;
    const uint8_t* base = ring + s * St::kBytes;
    auto chunk = [&](int c) {
      const uint8_t* scale = base + at.scale + c * at.scale_next;
      multiply<T, MTW, NT, ZEROS, G32>(
          acc, base + c * St::kChunk + at.w, base + c * St::kChunk + (at.w ^ 16),
          base + at_x + c * (8 * 512 * NT),
          reinterpret_cast<const float*>(base + at.sum + c * (4 * St::kSpans * 8 * kMaxNT * 4)),
          reinterpret_cast<const float*>(scale));
    };
#pragma unroll
    for (int c = 0; c < 2; ++c)
      if (left > 256 * c) chunk(c);
    release_slot(&bars.empty[s]);
    if (++s == (uint32_t)S) s = 0, ++lap;
  }
  return true;
}

__device__ __forceinline__ void bar_mul() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kMulWarps) : "memory");
}

template <typename T>
__device__ __forceinline__ void store1(void* p, size_t i, float v) {
  if constexpr (T::kBf16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p)[i] = __float2half_rn(v);
}

// ANY: rows of scales of any number of groups, else of whole fours.
template <typename T, int MTW, bool ACT, bool ZEROS, bool G32, bool ANY>
__global__ void __launch_bounds__(kThreads, 1)
w4_kernel(const __grid_constant__ Args a, const __grid_constant__ Shape sh,
          const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x1,
          const __grid_constant__ CUtensorMap map_x2) {
  using St = Stage<MTW, ZEROS, G32>;
  constexpr float kOff = T::kBf16 ? 128.f : 64.f;
  constexpr int kRed = 4 * 4 * 8 * kMaxNT * 20;  // floats of the sums' exchange
  extern __shared__ __align__(1024) uint8_t dyn[];
  __shared__ Bars bars;
  const int S = sh.stages;
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
  float* red = reinterpret_cast<float*>(ring + S * St::kBytes);
  int* s_begin = reinterpret_cast<int*>(red + kRed);
  int* s_tile = s_begin + a.G + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  if (threadIdx.x == 0) {
    prefetch_map(&map_w);
    for (int s = 0; s < S; ++s) {
      mbar_init(&bars.full[s], 1);
      mbar_init(&bars.ready[s], kSumWarps + kScaleWarps);
      mbar_init(&bars.empty[s], kMulWarps);
    }
    async::mbar_fence_init();
  }
  griddep_wait();
  const bool bad = group_scan<kThreads>(a, s_begin, s_tile, [&](int rows) {
    return sh.tiles_n * ((rows + 8 * kMaxNT - 1) / (8 * kMaxNT));
  });
  if (bad && blockIdx.x == 0) atomicOr(&g_status, (uint32_t)CQ_ST_BAD_ROWS);
  const int n_tiles = s_tile[a.G];
  const int n_stages = (a.K + 511) / 512;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_wait_warp(bar, parity)) return true;
    atomicOr(&g_status, (uint32_t)CQ_ST_TIMEOUT);
    return false;
  };
  uint32_t s = 0, lap = 0;
  auto next = [&]() {
    if (++s == (uint32_t)S) s = 0, ++lap;
  };
  bool ok = true;

  if (warp < kMulWarps) {
    // ---- products ----
    const int kw = warp & 3, rq = warp >> 2;
    Places at;
    at.w = rq * (16 * MTW * 128) + g * 128 + (((2 * kw) ^ g) << 4) + 4 * q;
    at.x = St::kX + g * 64 + ((q ^ ((g >> 1) & 3)) << 4);
    at.sum = St::kSum + (kw * (St::kSpans * 8 * kMaxNT) + 2 * q) * 4;
    at.scale = St::kScale + ((kw * 64 >> sh.shift) * St::kGroupFloats + (rq * 8 + g) * (St::kGroupFloats / 32)) * 4;
    at.scale_next = (256 >> sh.shift) * St::kGroupFloats * 4;
    for (int t = blockIdx.x; t < n_tiles && ok; t += gridDim.x) {
      const Tile x = tile_at<MTW, ACT>(sh, s_begin, s_tile, a.G, t);
      float acc[MTW][kMaxNT][4] = {};
      if (x.nt == 1)
        ok = multiply_tile<T, MTW, 1, ZEROS, G32>(acc, bars, ring, S, s, lap, at, kw, a.K);
      else
        ok = multiply_tile<T, MTW, kMaxNT, ZEROS, G32>(acc, bars, ring, S, s, lap, at, kw, a.K);
      if (!ok) atomicOr(&g_status, (uint32_t)CQ_ST_TIMEOUT);
      // A warp that gave up attends all the same: the others would wait for it without
      // a limit. They leave together.
      if (!(ok = async::meet<32 * kMulWarps>(ok))) break;
      // Sums of the four k shares, added in order: 16 rows of every quarter at a time.
#pragma unroll
      for (int m = 0; m < MTW; ++m) {
        if (m > 0) bar_mul();
        float* to = red + (kw * 4 + rq) * (8 * kMaxNT * 20);
#pragma unroll
        for (int n = 0; n < kMaxNT; ++n)
          if (n < x.nt) {
            to[(8 * n + 2 * q) * 20 + g] = acc[m][n][0];
            to[(8 * n + 2 * q + 1) * 20 + g] = acc[m][n][1];
            to[(8 * n + 2 * q) * 20 + g + 8] = acc[m][n][2];
            to[(8 * n + 2 * q + 1) * 20 + g + 8] = acc[m][n][3];
          }
        bar_mul();
        auto total = [&](int r, int j, int i) {
          float v = 0.f;
#pragma unroll
          for (int w = 0; w < 4; ++w) v += red[((w * 4 + r) * 8 * kMaxNT + j) * 20 + i];
          return v * kOff;
        };
        const int i = threadIdx.x & 15;
        if constexpr (ACT) {
          for (int v = threadIdx.x; v < x.jn * 32; v += 32 * kMulWarps) {
            const int r = (v >> 4) & 1, j = v >> 5, o = x.o0 + 16 * MTW * r + 16 * m + i;
            const float gv = total(r, j, i), uv = total(r + 2, j, i);
            if (o < sh.n_out)
              store1<T>(a.out, (size_t)(x.begin + x.j0 + j) * sh.n_out + o,
                        swiglu(gv, uv));
          }
        } else {
          for (int v = threadIdx.x; v < x.jn * 64; v += 32 * kMulWarps) {
            const int r = (v >> 4) & 3, j = v >> 6, o = x.o0 + 16 * MTW * r + 16 * m + i;
            const float y = total(r, j, i);
            if (o < sh.n_out) store1<T>(a.out, (size_t)(x.begin + x.j0 + j) * sh.n_out + o, y);
          }
        }
      }
    }
  } else if (warp < kMulWarps + kSumWarps) {
    // ---- x in the nibbles' order, and its sums ----
    const int kw = warp - kMulWarps;
    constexpr uint32_t kOne = T::kBf16 ? 0x3f803f80u : 0x3c003c00u;
    const uint32_t ones[4] = {kOne, kOne, kOne, kOne};
    for (int t = blockIdx.x; t < n_tiles && ok; t += gridDim.x) {
      const Tile x = tile_at<MTW, ACT>(sh, s_begin, s_tile, a.G, t);
      for (int st = 0; st < n_stages; ++st) {
        if (!(ok = wait(&bars.full[s], lap & 1))) break;
        uint8_t* base = ring + s * St::kBytes;
        for (int n = 0; n < x.nt; ++n) {
          // blocks of 32 past k are zeros, codes and x: no harm in summing them
          uint4 w[2][2];
          uint8_t* at = base + St::kX + (kw * 2 * x.nt + n) * 512 + g * 64 + ((q ^ ((g >> 1) & 3)) << 4);
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              w[c][h] = *reinterpret_cast<const uint4*>(at + (8 * c + h) * x.nt * 512);
          float v[2][2][4];
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint4 u = w[c][h];
              *reinterpret_cast<uint4*>(at + (8 * c + h) * x.nt * 512) =
                  make_uint4(__byte_perm(u.x, u.z, 0x5410), __byte_perm(u.x, u.z, 0x7632),
                             __byte_perm(u.y, u.w, 0x5410), __byte_perm(u.y, u.w, 0x7632));
              mma<T::kBf16>(v[c][h], ones, u.x, u.y, 0.f, 0.f, 0.f, 0.f);
              mma<T::kBf16>(v[c][h], ones, u.z, u.w, v[c][h][0], v[c][h][1], v[c][h][2], v[c][h][3]);
            }
          if (g == 0) {
            const float f = ZEROS ? 1.f : -(1.f + 8.f / kOff);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float* sum = reinterpret_cast<float*>(base + St::kSum) +
                           (c * 4 + kw) * (St::kSpans * 8 * kMaxNT) + 2 * q + 8 * n;
              if constexpr (G32) {
                *reinterpret_cast<float2*>(sum) = make_float2(f * v[c][0][0], f * v[c][0][1]);
                *reinterpret_cast<float2*>(sum + 8 * kMaxNT) = make_float2(f * v[c][1][0], f * v[c][1][1]);
              } else {
                *reinterpret_cast<float2*>(sum) =
                    make_float2(f * (v[c][0][0] + v[c][1][0]), f * (v[c][0][1] + v[c][1][1]));
              }
            }
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) async::mbar_arrive(&bars.ready[s]);
        next();
      }
    }
  } else if (warp < kMulWarps + kSumWarps + kScaleWarps) {
    // ---- scales: a thread takes rows r and r + 64, kAhead stages ahead ----
    constexpr int kPer = (St::kRows + 63) / 64, kW = St::kGroups / 2;  // rows; words of a row
    constexpr int kZW = kW / 2 + ANY;                             // zero points: a word more
    constexpr int kFit = 48 / (kPer * (kW + (ZEROS ? kZW : 0)));  // in 48 registers
    constexpr int kMost = MTW == 2 && ZEROS ? 3 : 4;              // (groups of 64: 74 us against 94 with 4)
    constexpr int kAhead = kFit > kMost ? kMost : kFit;
    static_assert(!ANY || kAhead >= 2, "a row's last word comes from the next stage's buffer");
    const uint16_t* scales = static_cast<const uint16_t*>(a.scales4);
    const int per_cta = n_tiles > (int)blockIdx.x ? (n_tiles - 1 - blockIdx.x) / gridDim.x + 1 : 0;
    const int total = per_cta * n_stages, ng = 512 >> sh.shift;
    const int r0 = threadIdx.x - 32 * (kMulWarps + kSumWarps);
    int tile = -1, st = n_stages - 1, st_store = 0;
    size_t row_at[kPer] = {};
    bool in[kPer] = {};
    uint32_t sbuf[kAhead][kPer][kW] = {}, zbuf[kAhead][kPer][kZW] = {};
    // ANY: aligned words are read, from where a row's part begins or up to 3 bytes before,
    // and shifted into place when they are stored, so that nothing here waits for a load
    // (single groups put together at once: 163 us against 94, groups of 64, zero points,
    // 32 experts of 4 rows, 2048 x 7232). The word past a full stage's scales is the next
    // stage's first; a tile's last stage is not full then. The rows' offsets modulo 4 are
    // those of r0 (tiles and experts begin at multiples of 16 rows), and the tensors end
    // at whole words.
    const uint32_t s_shift = 16 * (r0 * sh.KG & 1), z_shift = 8 * (r0 * sh.KG & 3);
    auto load = [&](int i, uint32_t (&sv)[kPer][kW], uint32_t (&zv)[kPer][kZW]) {
      if (i >= total) return;
      if (++st == n_stages) st = 0, ++tile;
      const int first = st * ng;
      if (st == 0) {
        const Tile x = tile_at<MTW, ACT>(sh, s_begin, s_tile, a.G, blockIdx.x + tile * gridDim.x);
#pragma unroll
        for (int b = 0; b < kPer; ++b) {
          const int r = r0 + 64 * b, half = ACT ? r / (32 * MTW) : 0, rh = r - half * 32 * MTW;
          in[b] = x.o0 + rh < sh.n_out;
          row_at[b] = ((size_t)x.e * a.N + half * sh.n_out + x.o0 + rh) * sh.KG;
        }
      }
#pragma unroll
      for (int b = 0; b < kPer; ++b) {
#pragma unroll
        for (int w = 0; w < kW; ++w) sv[b][w] = 0;
#pragma unroll
        for (int w = 0; w < kW / 2; ++w) zv[b][w] = 0;
        if (!in[b]) continue;
        const size_t at = row_at[b] + first;
        if constexpr (ANY) {
          const int n = min(ng, sh.KG - first);
          const uint32_t* from = reinterpret_cast<const uint32_t*>(scales + at - s_shift / 16);
#pragma unroll
          for (int w = 0; w < kW; ++w)
            if (4 * w < 2 * n + (int)(s_shift / 8)) sv[b][w] = __ldg(from + w);
          if constexpr (ZEROS) {
            const uint32_t* zfrom = reinterpret_cast<const uint32_t*>(a.zeros4 + at - z_shift / 8);
#pragma unroll
            for (int w = 0; w < kZW; ++w)
              if (4 * w < n + (int)(z_shift / 8)) zv[b][w] = __ldg(zfrom + w);
          }
        } else if (sh.vec == 2) {
          // 4 groups (of 128), 8, or twice 8, the second of which may not exist
          const uint16_t* from = scales + at;
          const uint8_t* zfrom = a.zeros4 + at;
          if (!G32 && ng == 4) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(from));
            sv[b][0] = v.x, sv[b][1] = v.y;
            if (ZEROS) zv[b][0] = __ldg(reinterpret_cast<const uint32_t*>(zfrom));
          } else {
#pragma unroll
            for (int w = 0; w < kW; w += 4)
              if (first + 2 * w < sh.KG) {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(from + 2 * w));
                sv[b][w] = v.x, sv[b][w + 1] = v.y, sv[b][w + 2] = v.z, sv[b][w + 3] = v.w;
                if (ZEROS) {
                  const uint2 z = __ldg(reinterpret_cast<const uint2*>(zfrom + 2 * w));
                  zv[b][w / 2] = z.x, zv[b][w / 2 + 1] = z.y;
                }
              }
          }
        } else {
#pragma unroll
          for (int w = 0; w < kW; w += 2)
            if (2 * w < ng && first + 2 * w < sh.KG) {
              const uint2 v = __ldg(reinterpret_cast<const uint2*>(scales + at + 2 * w));
              sv[b][w] = v.x, sv[b][w + 1] = v.y;
              if (ZEROS) zv[b][w / 2] = __ldg(reinterpret_cast<const uint32_t*>(a.zeros4 + at + 2 * w));
            }
        }
      }
    };
#pragma unroll
    for (int u = 0; u < kAhead; ++u) load(u, sbuf[u], zbuf[u]);
    for (int i0 = 0; i0 < total && ok; i0 += kAhead) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (i0 + u >= total || !ok) break;
        if (lap > 0 && !(ok = wait(&bars.empty[s], (lap & 1) ^ 1))) break;
        uint8_t* base = ring + s * St::kBytes;
        const int have = sh.KG - st_store * ng;  // groups from this stage on
        if (++st_store == n_stages) st_store = 0;
#pragma unroll
        for (int b = 0; b < kPer; ++b) {
          const int r = r0 + 64 * b;
          const int slot = (r / (16 * MTW) * 8 + r % 8) * (2 * MTW) + 2 * (r / 16 % MTW) + r / 8 % 2;
          float* to = reinterpret_cast<float*>(base + St::kScale) + slot * (ZEROS ? 2 : 1);
          auto put = [&](int k, uint32_t v, uint32_t zw) {
            const float f = k & 1 ? T::hi(v) : T::lo(v);
            if constexpr (ZEROS) {
              // 2^23 / OFF + z / OFF has z in its last bits; all of this is exact
              constexpr float kBase = 8388608.f / kOff;
              constexpr uint32_t kBits = T::kBf16 ? 0x47800000u : 0x48000000u;  // of kBase
              const float z = __uint_as_float(__byte_perm(zw, kBits, 0x7640 + (k & 3)));
              *reinterpret_cast<float2*>(to + k * St::kGroupFloats) = make_float2(f, (kBase - 1.f) - z);
            } else {
              to[k * St::kGroupFloats] = f;
            }
          };
          if constexpr (!ANY) {
#pragma unroll
            for (int k = 0; k < St::kGroups; ++k)
              if (k < ng) put(k, sbuf[u][b][k / 2], zbuf[u][b][k / 4]);
          } else {
#pragma unroll
            for (int k = 0; k < St::kGroups; ++k)
              if (k < ng) {
                const uint32_t past = k / 2 + 1 < kW ? sbuf[u][b][(k / 2 + 1) % kW] : sbuf[(u + 1) % kAhead][b][0];
                const uint32_t v = __funnelshift_r(sbuf[u][b][k / 2], past, s_shift);
                // past KG lies the next row's
                put(k, k < have ? v : 0u, __funnelshift_r(zbuf[u][b][k / 4], zbuf[u][b][k / 4 + 1], z_shift));
              }
          }
        }
        __syncwarp();
        if (lane == 0) async::mbar_arrive(&bars.ready[s]);
        next();
        load(i0 + u + kAhead, sbuf[u], zbuf[u]);
      }
    }
  } else {
    // ---- copies of codes and x ----
    for (int t = blockIdx.x; t < n_tiles && ok; t += gridDim.x) {
      const Tile x = tile_at<MTW, ACT>(sh, s_begin, s_tile, a.G, t);
      const CUtensorMap* mx = x.nt == 1 ? &map_x1 : &map_x2;
      for (int st = 0; st < n_stages; ++st) {
        if (lap > 0 && !(ok = wait(&bars.empty[s], (lap & 1) ^ 1))) break;
        if (elect_one()) {
          const uint32_t base = smem_u32(ring + s * St::kBytes), bar = smem_u32(&bars.full[s]);
          mbar_arrive_expect_tx(&bars.full[s], St::kX + 16 * 512 * x.nt);
          tma_load4<1>(base, &map_w, st * 256, x.o0, 0, x.e, bar);
          tma_load4<1>(base + St::kChunk, &map_w, st * 256 + 128, x.o0, 0, x.e, bar);
          tma_load3<1>(base + St::kX, mx, 0, x.begin + x.j0, st * 16, bar);
        }
        __syncwarp();
        next();
      }
    }
    // Let the copies in flight land (with a limit): the warps that read them may have
    // given up before this one noticed.
    for (int v = 0; v < S; ++v) {
      const uint32_t laps = lap + ((uint32_t)v < s ? 1 : 0);
      if (laps > 0) mbar_wait(&bars.full[v], (laps - 1) & 1);
    }
  }
}

// ---- host ----
template <typename T, int MTW, bool ACT, bool ZEROS, bool G32, bool ANY>
cudaError_t launch_t(const Args& a, cudaStream_t s) {
  constexpr auto kernel = w4_kernel<T, MTW, ACT, ZEROS, G32, ANY>;
  using St = Stage<MTW, ZEROS, G32>;
  Shape sh = {};
  sh.n_out = ACT ? a.N / 2 : a.N;
  sh.tiles_n = (a.N + St::kRows - 1) / St::kRows;
  sh.shift = a.group == 32 ? 5 : a.group == 64 ? 6 : 7;
  sh.KG = a.K / a.group;
  sh.vec = sh.KG % 8 == 0 ? 2 : 1;
  const uint64_t G = a.G, R = a.R, N = a.N, K = a.K;
  CUtensorMap mw, mx[2];
  // codes: the two halves of a tile in one copy; x: 16 blocks of 32 of k in one
  const uint64_t halves = ACT ? 2 : 1;
  const uint64_t dw[] = {K / 2, N / halves, halves, G}, sw[] = {K / 2, N / 2 * (K / 2), N * (K / 2)};
  const uint32_t bw[] = {128, (uint32_t)(St::kRows / halves), (uint32_t)halves, 1};
  if (!make_map(&mw, a.w, kMapU8, 4, dw, sw, bw, kSwizzle128)) return cudaErrorUnknown;
  const uint64_t dx[] = {32, R, K / 32}, sx[] = {K * 2, 64};
  for (int i = 0; i < kMaxNT; ++i) {
    const uint32_t bx[] = {32, 8u << i, 16};
    if (!make_map(&mx[i], a.x, T::kBf16 ? kMapBF16 : kMapF16, 3, dx, sx, bx, kSwizzle64))
      return cudaErrorUnknown;
  }
  // As many stages as fit beside the exchange of the sums and the lists.
  const size_t fixed = 1024 + 4 * 4 * 8 * kMaxNT * 20 * 4 + 8 * ((size_t)a.G + 1);
  sh.stages = (int)std::min<size_t>(kMaxStages, (kSmemBytes - fixed) / St::kBytes);
  const size_t smem = fixed + sh.stages * (size_t)St::kBytes;
  cudaError_t e = prepare_kernel<kernel>(smem);
  if (e != cudaSuccess) return e;
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorUnknown;
  const int64_t most = (int64_t)sh.tiles_n * (a.R / (8 * kMaxNT) + std::min(a.G, a.R));
  const int grid = (int)std::min<int64_t>(sms, most);
  return launch_pdl(kernel, dim3(grid), dim3(kThreads), smem, s, a, sh, mw, mx[0], mx[1]);
}

template <typename T, int MTW, bool ACT, bool ZEROS, bool G32>
cudaError_t launch_r(const Args& a, cudaStream_t s) {
  if (a.K / a.group % 4 == 0) return launch_t<T, MTW, ACT, ZEROS, G32, false>(a, s);
  // Tiles of 128 rows, zero points, groups of 32: the scales of two rows would not fit
  // the registers (215 us against 119 in tiles of 64: 32 experts of 4 rows, 2048 x 7200).
  return launch_t<T, ZEROS && G32 ? 1 : MTW, ACT, ZEROS, G32, true>(a, s);
}

template <typename T, int MTW, bool ACT>
cudaError_t launch_g(const Args& a, cudaStream_t s) {
  if (a.zeros4)
    return a.group == 32 ? launch_r<T, MTW, ACT, true, true>(a, s)
                         : launch_r<T, MTW, ACT, true, false>(a, s);
  return a.group == 32 ? launch_r<T, MTW, ACT, false, true>(a, s)
                       : launch_r<T, MTW, ACT, false, false>(a, s);
}

// Tiles of 128 weight rows where they give every SM two, else of 64 (a tile of 64
// takes about 0.6 of the time of one of 128, so it pays where SMs would idle:
// 8192 x 8192 has 64 tiles of 128 and 128 of 64).
template <typename T, bool ACT>
cudaError_t launch_a(const Args& a, cudaStream_t s) {
  const int64_t rows = (int64_t)std::min(a.G, a.R) * a.N;  // most weight rows read
  if (rows >= 128 * 2 * (int64_t)sm_count()) return launch_g<T, 2, ACT>(a, s);
  return launch_g<T, 1, ACT>(a, s);
}

}  // namespace

int launch_w4(const Args& a, cudaStream_t s) {
  if (a.R == 0) return CQ_OK;
  cudaError_t e;
  if (a.x_dtype == kF16) e = a.act ? launch_a<F16, true>(a, s) : launch_a<F16, false>(a, s);
  else e = a.act ? launch_a<BF16, true>(a, s) : launch_a<BF16, false>(a, s);
  return e == cudaSuccess ? CQ_OK : CQ_ERR_CUDA;
}

int w4_status(uint32_t* read, cudaStream_t s) { return status_word(g_status, read, s); }

}  // namespace expert
}  // namespace cq
