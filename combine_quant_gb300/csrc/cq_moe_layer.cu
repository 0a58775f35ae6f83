// cq_moe_layer.cu -- the whole layer for a few tokens: gate and up products with
// SwiGLU (up_kernel), down product with the weighted sum (down_kernel).
//
// The weights of the experts that the tokens name are read once, and that is the bound:
// both kernels stream them through a ring of shared memory (tiled copies by one warp)
// and multiply on the way with mma.sync, whose 8 columns suit a few tokens; its rate,
// 1024 products a clock and SM, is no bound there. Warps take 64 bytes of a row each;
// with k in an order of the thread's choice (its 16 bytes of a row against the same 16
// bytes of a token) one 16-byte load feeds two to four products.
//
// Every CTA sorts the (token, expert) pairs itself into items: an expert and up to 8 NB
// of its tokens, ascending. A token that names an expert twice is one pair with both
// weights. up_kernel: an item's tile of 16 (64) gates and their ups is one CTA's work;
// its warps' shares of k are added through shared memory, in order (few
// units: a cluster's work, whose CTAs take shares of k too). down_kernel: a tile of 32
// (96, 128) output rows is one cluster's work: the CTAs share the stages of all items
// evenly, each keeps the weighted sums of all tokens, and the CTAs' sums are added
// through distributed shared memory, in order. Results do not depend on timing. The
// second kernel's copies of weights start before the first one has ended.
//
// Tokens' rows come a stage at a time by one tiled copy: all tokens' (up; fp8 weights:
// only an item's, by three warps), an item's, which lie together (down). Row by row, 256
// bytes each, the copies were the bound (64 tokens, bf16: 852 -> 563 us).
//
// Between the two SwiGLU's results are held as two numbers of the token type, whose sum
// keeps 16 bits or more: rounding them to one would add an error as large as y's own
// rounding.
//
// fp8 weights and large tiles: the products are bound by instructions, and a code
// becomes an fp16 number in half of one, a bf16 number in two and a half. So the products
// run in fp16 there, whose range powers of two provide: each token's row is scaled by one
// (scale_kernel, where tokens are bf16: exact down to 2^-31 of the row's largest value, below
// that off by 2^-39 of it at most, or by 2^-135 in rows below 2^-96), SwiGLU's results by one for
// 64 of a pair, which the down product's warps multiply back.
// Where y is bf16 these are rounded to fp16 once, to 11 bits: an eighth of y's own rounding
// (64 tokens: 461 -> 367 us). Where y is fp16 or f32 that would be as much as y's rounding or
// thousands of times it, so there two numbers stay, 22 bits of a value and 2^-39 of the 64's
// largest (64 tokens, f32 y: 339 us, with one number 307; 16 tokens: 238, 229; 43 tokens,
// hidden 2064, inter 752, fp16: 39.5, 37.8).
//
// Measured on one GB300 (copy 6.78 TB/s), hidden 7168, inter 2048, 8 of 32 experts, in a
// graph: 1 token, bf16: 111 us, 6.4 TB/s; 16 tokens: 411 us, 6.9 TB/s; 64 tokens: 460 us,
// 6.1 TB/s; fp8 weights: 71 us (5.0), 226 us (6.2), 303 us (4.7). Hidden 1024, inter 512, 4
// tokens: 13 us, most of it the start and end of two kernels.
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

__device__ uint32_t g_status;  // CQ_ST_* bits of these kernels on this device

struct LayerArgs {
  int32_t T, G, K, H, I, mask_ndim, out_f32;
  int32_t stages, cluster;   // of the ring; CTAs that share a tile (down_kernel) or a unit (up_kernel)
  int32_t whole;             // rows of x (h) are whole blocks of 64: one copy takes a stage's
  int32_t two;               // scaled: h as two numbers
  const uint16_t* x;
  const int32_t* ids;
  const float* scales;
  const uint8_t* mask;
  const float* w13_scales;
  const float* w2_scales;
  uint16_t* h;  // [2][T * K][I]: both numbers, or [T * K][I]
  float* h_scales;           // scaled: [T * K][units of 64]
  float* x_scales;           // scaled, bf16 tokens: [T], else NULL
  uint16_t* x16;             // and their rows [T][H]
  void* y;
};

// Row groups of 32 rows in a tile: 1, or 4 (down_kernel: 3 or 4). A stage is boxes of 32 RG rows of 128 bytes;
// a warp takes a row group and half of a box. One more warp copies.
template <int RG>
constexpr int kBoxes = RG == 1 ? 4 : 2;
template <int RG>
constexpr int kSegs = 2 * kBoxes<RG>;
template <int RG>
constexpr int kWarps = kSegs<RG> * RG;
// With twelve or sixteen warps that multiply, three more that do nothing fill the copying
// warp's warpgroup, so that registers can be moved: of 640 x 96 (512 x 128) the multiplying
// warps get 112 (160) a thread, the others 32, the same in all.
template <int RG>
constexpr int kThreads = 32 * (kWarps<RG> + (RG == 1 ? 1 : 4));
constexpr int kOtherRegs = 32;
template <int RG>
constexpr int kProductRegs = RG == 3 ? 160 : 112;
template <int RG>
constexpr int kAllRegs = 128 * kOtherRegs + 32 * kWarps<RG> * kProductRegs<RG>;
static_assert(kAllRegs<4> <= 96 * kThreads<4> && kAllRegs<3> <= 128 * kThreads<3>, "setmaxnreg would wait forever");
template <int RG>
constexpr int kStageW = kBoxes<RG> * 32 * RG * 128;  // weights of a stage
// Products in fp16 with powers of two taken out.
template <bool FP8, int RG>
constexpr bool kScaled = FP8 && RG > 1;
// The down kernel's sums: of every share of k, or (more than 16 tokens, large tiles) one that
// two shares add to in turn. Lines of 4 floats more than rows: neighbouring tokens' lines
// then begin four banks apart.
template <int RG, int NB>
constexpr bool kTurns = RG > 1 && NB > 2;
template <int RG, int NB>
constexpr int kDownSums = kTurns<RG, NB> ? kSegs<RG> / 2 : kSegs<RG>;
template <int RG>
constexpr int kDownLine = 32 * RG + 4;
// The up kernel's shares of k meet in shared memory: small tiles, [share][row][token]; large
// ones, boxes of 16 bytes a lane that the warps of a row group hand over, and what a
// tile's largest values are found with.
template <int RG, int NB>
constexpr int kBoxLines = NB / 2;  // 16-byte pieces a lane and box
template <int RG, int NB>
constexpr int kUpFloats = RG == 1 ? kSegs<RG> * 32 * (8 * NB + 1)
                                  : kWarps<RG> * (NB == 2 ? 3 : 1) * kBoxLines<RG, NB> * 128 + 2 * RG * 32;
constexpr int kMaxWarps = kThreads<4> / 32;
constexpr int kMaxPairs = 64 * 16, kMaxItems = kMaxPairs + 32;

// k of a stage.
template <bool FP8, int RG>
constexpr int kChunk = kBoxes<RG> * (FP8 ? 128 : 64);
// Rows of 16-bit numbers lie in a stage as blocks of 64 of their k: 128-byte lines, the
// block's rows one after the other, swizzled as the copies have it.
template <bool FP8, int RG>
constexpr int kBlocks = kChunk<FP8, RG> / 64;

// Tokens' lines of a stage in the up kernel: an item's, which the threads gather (fp8 weights,
// large tiles), or all tokens', by one tiled copy.
template <bool FP8, int NB, int RG>
__host__ __device__ constexpr int up_lines(int T) {
  return kScaled<FP8, RG> ? 8 * NB : (T + 7) / 8 * 8;
}

struct Items {
  int n;                        // items
  uint16_t e[kMaxItems], off[kMaxItems];  // expert, first pair
  uint8_t m[kMaxItems];         // pairs
  uint8_t tok[kMaxPairs + 32];  // of each pair the token and its weight (zeros behind the last)
  float weight[kMaxPairs];
  uint32_t scan[kMaxWarps];
  int plan[2];                  // units, and a CTA's distance between its own
  int twice;                    // a token names an expert twice
};

// Sorts the pairs (all threads; a barrier has to follow). `scratch`: 10 bytes an expert and 8 a
// pair. Its latency is paid twice a call, so the ids are on their way before anything else, and
// a thread keeps its pairs in registers; only where a token names an expert twice are the
// token's others looked at.
template <int PER, int kThreads>
__device__ __forceinline__ void sort_pairs(const LayerArgs& a, Items& it, uint8_t* scratch, bool report) {
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, P = a.T * a.K;
  unsigned long long* masks = reinterpret_cast<unsigned long long*>(scratch);  // tokens of each expert
  uint32_t* words = reinterpret_cast<uint32_t*>(scratch);
  int* ids = reinterpret_cast<int*>(masks + a.G);
  float* scales = reinterpret_cast<float*>(ids + P);
  uint16_t* first = reinterpret_cast<uint16_t*>(scales + P);  // pair of each expert
  constexpr int kMine = (kMaxPairs + kThreads - 1) / kThreads;
  int mine[kMine];
  float weight[kMine] = {};
#pragma unroll
  for (int v = 0; v < kMine; ++v) {
    const int p = t + v * kThreads;
    mine[v] = -1;
    if (p >= P) continue;
    const bool on = !a.mask_ndim || a.mask[a.mask_ndim == 1 ? p / a.K : p];
    weight[v] = a.scales[p];
    const int e = a.ids[p];
    if (on) mine[v] = e;
    if (on && (unsigned)e >= (unsigned)a.G) {
      if (report) atomicOr(&g_status, (uint32_t)CQ_ST_BAD_ID);
      mine[v] = -1;
    }
  }
  for (int e = t; e < a.G; e += kThreads) masks[e] = 0;
  for (int p = t; p < P + 32; p += kThreads) it.tok[p] = 0;
  if (t == 0) it.twice = 0;
  __syncthreads();
#pragma unroll
  for (int v = 0; v < kMine; ++v) {
    const int p = t + v * kThreads, tok = p / a.K;
    if (p >= P) break;
    ids[p] = mine[v];
    scales[p] = weight[v];
    if (mine[v] >= 0 && atomicOr(words + 2 * mine[v] + tok / 32, 1u << (tok % 32)) >> (tok % 32) & 1) it.twice = 1;
  }
  __syncthreads();
  const int per = (a.G + kThreads - 1) / kThreads, e0 = min(a.G, t * per), e1 = min(a.G, e0 + per);
  // pairs below, items above: both stay below 2^16
  static_assert(kMaxItems < 1 << 15);
  uint32_t counts = 0;
  for (int e = e0; e < e1; ++e) {
    const int c = __popcll(masks[e]);
    counts += c + ((c + PER - 1) / PER << 16);
  }
  uint32_t sum = counts;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(~0u, sum, o);
    if (lane >= o) sum += v;
  }
  if (lane == 31) it.scan[warp] = sum;
  __syncthreads();
  static_assert(kMaxWarps <= 32);
  sum += __reduce_add_sync(~0u, lane < warp ? it.scan[lane] : 0u);
  int p0 = (sum - counts) & 0xffff, i0 = (sum - counts) >> 16;
  for (int e = e0; e < e1; ++e) {
    first[e] = (uint16_t)p0;
    for (int left = __popcll(masks[e]); left > 0; left -= PER, ++i0) {
      it.e[i0] = (uint16_t)e;
      it.off[i0] = (uint16_t)p0;
      it.m[i0] = (uint8_t)min(left, PER);
      p0 += min(left, PER);
    }
  }
  if (t == kThreads - 1) it.n = i0;
  __syncthreads();
#pragma unroll
  for (int v = 0; v < kMine; ++v) {
    const int p = t + v * kThreads, e = mine[v], tok = p / a.K;
    if (e < 0) continue;
    float w = 0.f + weight[v];
    if (it.twice) {
      w = 0.f;
      bool before = false;
      for (int j = tok * a.K; j < tok * a.K + a.K; ++j) {
        if (ids[j] != e) continue;
        before |= j < p;
        w += scales[j];
      }
      if (before) continue;
    }
    const int at = first[e] + __popcll(masks[e] & ((1ull << tok) - 1));
    it.tok[at] = (uint8_t)tok;
    it.weight[at] = w;
  }
}

__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// d += a b, or (FIRST) d = a b.
template <typename T, bool FIRST>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
#define CQ_MMA(type)                                                                                              \
  if constexpr (FIRST)                                                                                            \
    asm("mma.sync.aligned.m16n8k16.row.col.f32." type "." type                                                     \
        ".f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"                                  \
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])                                                             \
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));                                            \
  else                                                                                                            \
    asm("mma.sync.aligned.m16n8k16.row.col.f32." type "." type                                                     \
        ".f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"                                      \
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])                                                             \
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1))
  if constexpr (T::kBf16) {
    CQ_MMA("bf16");
  } else {
    CQ_MMA("f16");
  }
#undef CQ_MMA
}

// Four e4m3 codes as two words of 16-bit numbers, exactly. bf16: a code with its sign
// spread over the byte above it, shifted by four and cut to sign, exponent and fraction
// where bf16 has them, is the value times 2^-120 (also below the normal range).
template <typename T>
__device__ __forceinline__ void decode4(uint32_t q, uint32_t& lo, uint32_t& hi) {
  if constexpr (T::kBf16) {
    constexpr uint32_t k2to120 = 0x7b807b80u;
    asm("prmt.b32 %0, %2, 0, 0x9180;\n prmt.b32 %1, %2, 0, 0xb3a2;" : "=&r"(lo), "=r"(hi) : "r"(q));
    lo = (lo << 4) & 0x87f087f0u;
    hi = (hi << 4) & 0x87f087f0u;
    asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(lo) : "r"(k2to120));
    asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(hi) : "r"(k2to120));
  } else {
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}"
        : "=r"(lo), "=r"(hi)
        : "r"(q));
  }
}

// Row of a box that row g of a fragment stands for: rows whose 16-byte pieces a quarter of
// a warp reads together differ in bit 2, which the swizzle turns into the other 64 bytes.
__device__ __forceinline__ int fragment_row(int g) { return ((g & 1) << 2) | (g >> 1); }

// The token of a block of 8 that column j of a fragment stands for, for the same reason
// (fp8 weights take 32 bytes of a token's line, where neighbouring rows do not meet).
template <bool FP8>
__device__ __forceinline__ int fragment_column(int j) {
  return FP8 ? j : fragment_row(j);
}

// Two fragments of 16 rows (at r0, r1 of a box) times up to 8 NB tokens over this warp's
// 64 bytes of the rows. `lines`: shared address of the tokens' lines of this k, row[n] the
// line of this thread's token of block n. PARTS: the tokens' numbers are sums of so many,
// part_bytes apart. FP8: s0, s1 are the fragments' factors here; nan collects codes that
// are NaN (bf16, whose decoding does not know them): bit 7 of a byte, by fragment and
// upper rows.
// COLUMNS: a token's factor meets them, `column` in the token's lane.
template <typename T, bool FP8, int NB, int PARTS, bool COLUMNS = false>
__device__ __forceinline__ void multiply(uint32_t box, int r0, int r1, int half, uint32_t lines, const int (&token)[NB],
                                         int part_bytes, int n8, float s0, float s1, float (&acc)[2][NB][4],
                                         uint32_t (&nan)[4], float column = 1.f) {
  const int lane = threadIdx.x & 31, row = fragment_row(lane >> 2), c = lane & 3;
  const uint32_t piece = ((half * 4 + c) ^ row) << 4;
  uint4 w[2][2];
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int u = 0; u < 2; ++u) w[f][u] = lds16(box + ((f ? r1 : r0) + 8 * u + row) * 128 + piece);
  constexpr int kSteps = FP8 ? 4 : 2;  // products of 16 k
  uint32_t v[2][2][2 * kSteps];
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t q[4] = {w[f][u].x, w[f][u].y, w[f][u].z, w[f][u].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (FP8) decode4<T>(q[k], v[f][u][2 * k], v[f][u][2 * k + 1]);
        else v[f][u][k] = q[k];
      }
      if constexpr (FP8 && T::kBf16) {
        uint32_t t[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) t[k] = (q[k] & 0x7f7f7f7fu) + 0x01010101u;
        nan[2 * f + u] |= (t[0] | t[1] | t[2]) | t[3];
      }
    }
  // Two blocks of tokens side by side, where there are two: a product waits for the one
  // before it in its sum. (A second block that is not there cost 332 us against 322: 64
  // tokens, fp8, 16 tokens an expert.)
  auto blocks = [&](auto n_of, auto side_of) {
    constexpr int n = n_of.value, kSide = side_of.value;
    float sum[kSide][2][4];
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
      uint32_t x[kSide][2 * kSteps];
#pragma unroll
      for (int b = 0; b < kSide; ++b) {
        const uint32_t line = lines + token[n + b] * 128 + p * part_bytes;
#pragma unroll
        for (int k = 0; k < kSteps / 2; ++k) {
          const int at = FP8 ? 2 * c + k : half * 4 + c;
          const uint4 t = lds16(line + ((at ^ (token[n + b] & 7)) << 4));
          x[b][4 * k] = t.x, x[b][4 * k + 1] = t.y, x[b][4 * k + 2] = t.z, x[b][4 * k + 3] = t.w;
        }
      }
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
#pragma unroll
        for (int b = 0; b < kSide; ++b)
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const uint32_t(&q)[2][2 * kSteps] = v[f];
            if (FP8 && p == 0 && k == 0)
              mma16<T, true>(sum[b][f], q[0][0], q[1][0], q[0][1], q[1][1], x[b][0], x[b][1]);
            else
              mma16<T, false>(FP8 ? sum[b][f] : acc[f][n + b], q[0][2 * k], q[1][2 * k], q[0][2 * k + 1], q[1][2 * k + 1],
                              x[b][2 * k], x[b][2 * k + 1]);
          }
    }
    if constexpr (FP8) {
#pragma unroll
      for (int b = 0; b < kSide; ++b) {
        float f0[2] = {s0, s0}, f1[2] = {s1, s1};
        if constexpr (COLUMNS) {
#pragma unroll
          for (int i = 0; i < 2; ++i) f0[i] = f1[i] = s0 * __shfl_sync(~0u, column, 8 * (n + b) + 2 * c + i);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[0][n + b][i] = fmaf(sum[b][0][i], f0[i & 1], acc[0][n + b][i]);
          acc[1][n + b][i] = fmaf(sum[b][1][i], f1[i & 1], acc[1][n + b][i]);
        }
      }
    }
  };
  using std::integral_constant;
  if constexpr (NB > 2) {
    static_assert(NB == 4);
    if (n8 > 1) blocks(integral_constant<int, 0>{}, integral_constant<int, 2>{});
    else blocks(integral_constant<int, 0>{}, integral_constant<int, 1>{});
    if (n8 > 3) blocks(integral_constant<int, 2>{}, integral_constant<int, 2>{});
    else if (n8 > 2) blocks(integral_constant<int, 2>{}, integral_constant<int, 1>{});
  } else {
    blocks(integral_constant<int, 0>{}, integral_constant<int, 1>{});
    if constexpr (NB == 2)
      if (n8 > 1) blocks(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  }
}

// Rows with a NaN code have NaN sums.
template <int NB>
__device__ __forceinline__ void spread_nan(uint32_t (&nan)[4], float (&acc)[2][NB][4]) {
  uint32_t all = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) all |= (nan[k] & 0x80808080u) ? 1u << k : 0u;
  all |= __shfl_xor_sync(~0u, all, 1);
  all |= __shfl_xor_sync(~0u, all, 2);
  if (all) {
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (all >> (2 * f + (i >> 1)) & 1) acc[f][n][i] = __uint_as_float(0x7fffffffu);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) nan[k] = 0;
}

struct Ring {
  uint64_t full[8], empty[8];
};

struct TokenMaps {
  CUtensorMap rows8, rows16, rows32;
};
// Lines that an item of m pairs is copied as.
__device__ __forceinline__ int lines_of(int m) { return m <= 8 ? 8 : m <= 16 ? 16 : 32; }

// 16 bytes, or zeros where `bytes` is 0.
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// An arrival on `bar` when this thread's copies so far have landed.
__device__ __forceinline__ void arrive_on_copies(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// The rings' start: barriers, and shared memory that sort_pairs used handed to the copies.
__device__ __forceinline__ void init_ring(Ring& r, int stages, int warps, int fills = 1) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&r.full[s], fills);
      mbar_init(&r.empty[s], warps);
    }
    async::mbar_fence_init();
  }
}

template <int RG, bool PRODUCTS>
__device__ __forceinline__ void set_registers() {
  if constexpr (RG == 1) return;
  if constexpr (PRODUCTS) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kProductRegs<RG>));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
}

__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity) {
  if (mbar_wait_warp(bar, parity)) return true;
  atomicOr(&g_status, (uint32_t)CQ_ST_TIMEOUT);
  return false;
}

// Copies in flight when a wait gave up land (with a limit) before the CTA goes.
__device__ __forceinline__ void end_copies(Ring& r, int stages, uint32_t s, uint32_t lap) {
  for (int v = 0; v < stages; ++v) {
    const uint32_t u = (s + v) % stages, laps = lap + (u < s ? 1 : 0);
    if (laps > 0) mbar_wait(&r.full[u], (laps - 1) & 1);
  }
}

template <typename T>
__device__ __forceinline__ uint16_t rounded(float v) {
  return (uint16_t)T::pack2(v, 0.f);
}

// The exponent of the power of two that brings the finite value m > 0 into [2^14, 2^15); at
// most 110 (m below 2^-96 stays below 2^14), so that the reciprocal times a block's scale stays
// a normal number.
__device__ __forceinline__ int f16_exponent(float m) { return m > 0.f ? min(110, 14 - ilogbf(m)) : 0; }

// bf16 rows times a power of two each, in fp16, and its reciprocal: a block a row.
// Infinities and NaN stay what they are.
__global__ void __launch_bounds__(256) scale_kernel(const uint16_t* x, uint16_t* to, float* scales, int H) {
  __shared__ float tops[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint4* row = reinterpret_cast<const uint4*>(x + (size_t)blockIdx.x * H);
  uint4* out = reinterpret_cast<uint4*>(to + (size_t)blockIdx.x * H);
  griddep_wait();
  float top = 0.f;
  for (int v = threadIdx.x; v < H / 8; v += 256) {
    const uint4 q = row[v];
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float a = fabsf(BF16::lo(w[k])), b = fabsf(BF16::hi(w[k]));
      if (a <= 3.402823466e38f) top = fmaxf(top, a);
      if (b <= 3.402823466e38f) top = fmaxf(top, b);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  if (lane == 0) tops[warp] = top;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 8; ++k) top = fmaxf(top, tops[k]);
  const int e = f16_exponent(top);
  for (int v = threadIdx.x; v < H / 8; v += 256) {
    const uint4 q = row[v];
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    uint32_t r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = F16::pack2(ldexpf(BF16::lo(w[k]), e), ldexpf(BF16::hi(w[k]), e));
    out[v] = make_uint4(r[0], r[1], r[2], r[3]);
  }
  if (threadIdx.x == 0) scales[blockIdx.x] = ldexpf(1.f, -e);
}

// A result of SwiGLU as two numbers of type T, or as the first alone.
template <typename T>
__device__ __forceinline__ void store_h(const LayerArgs& a, int pair, int i, float r, bool two) {
  const uint16_t hi = rounded<T>(r);
  uint16_t* to = a.h + (size_t)pair * a.I + i;
  to[0] = hi;
  // an infinite first number would make the second NaN
  if (two) to[(size_t)a.T * a.K * a.I] = rounded<T>(fabsf(T::lo(hi)) <= 3.402823466e38f ? r - T::lo(hi) : 0.f);
}

// Large tiles: the four shares of k of a row group are added, SwiGLU, and the results
// stored. Of a row group's sums (2 fragments, NB blocks of tokens) each of its warps ends
// with a quarter: a block of tokens, or (NB 2) the upper or lower rows of one. The others
// hand it theirs through boxes of shared memory, 16 bytes a lane, warp seg + r in step r.
// (Adding to one array in turn, where the lanes met in the banks, took 3 us a tile: 43
// tokens, 17 experts, hidden 2064, inter 752, fp8: 62 us, now 54; 64 tokens, hidden 7168,
// inter 2048: 350, now 332.) All warps come through the same barriers whatever `ok` is; the result is
// false where a warp that waits at them gave up.
template <typename T, bool FP8, int NB, int RG>
__device__ __forceinline__ bool finish(const LayerArgs& a, const Items& items, int item, int i0, bool ok, int turn,
                                       float* red, float4* far, float (&acc)[2][NB][4]) {
  constexpr int WARPS = kWarps<RG>, PIECES = kBoxLines<RG, NB>;
  constexpr bool kAll = NB == 2;  // all three boxes of a warp at once
  static_assert(kSegs<RG> == 4 && (NB == 2 || NB == 4));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane & 3, seg = warp / RG, group = warp % RG;
  const int m = items.m[item], n8 = (m + 7) / 8, off = items.off[item];
  const int block = NB == 4 ? seg : seg >> 1;  // this warp's tokens
  float4* boxes = reinterpret_cast<float4*>(red) + lane;
  float* tops = red + WARPS * (kAll ? 3 : 1) * PIECES * 128 + turn * RG * 32;  // [group (and rows' half)][token]
  auto box = [&](int to, int r) { return boxes + (((kAll ? r - 1 : 0) * RG + group) * 4 + to) * PIECES * 32; };
  // piece p of quarter q: NB 4, fragment p's four; NB 2, both fragments' of the upper or lower rows
  auto piece = [&](int q, int p) {
    if constexpr (NB == 4) return make_float4(acc[p][q][0], acc[p][q][1], acc[p][q][2], acc[p][q][3]);
    const int n = q >> 1, i = 2 * (q & 1);
    return make_float4(acc[0][n][i], acc[0][n][i + 1], acc[1][n][i], acc[1][n][i + 1]);
  };
  float4 mine[PIECES];
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int p = 0; p < PIECES; ++p)
      if (q == seg) mine[p] = piece(q, p);
#pragma unroll
  for (int r = 1; r < 4; ++r) {
    const int to = (seg + r) & 3;
    float4* there = box(to, r);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (q == to && (NB == 4 ? q : q >> 1) < n8)
#pragma unroll
        for (int p = 0; p < PIECES; ++p) there[32 * p] = piece(q, p);
    if (kAll && r < 3) continue;
    ok = async::meet<32 * 4>(ok, 2 + group);
    if (block < n8) {
#pragma unroll
      for (int b = kAll ? 1 : r; b <= r; ++b)
#pragma unroll
        for (int p = 0; p < PIECES; ++p) {
          const float4 v = box(seg, b)[32 * p];
          mine[p].x += v.x, mine[p].y += v.y, mine[p].z += v.z, mine[p].w += v.w;
        }
    }
    ok = async::meet<32 * 4>(ok, 2 + group);  // the boxes are read
  }
  if (a.cluster > 1) {
    // The CTAs' shares, in order; the first one's ring, which nothing uses any more, takes them.
    const uint32_t rank = cluster_rank();
    cluster_wait();
    if (rank > 0 && block < n8) {
#pragma unroll
      for (int p = 0; p < PIECES; ++p)
        asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                         addr_in(smem_u32(far + (((rank - 1) * WARPS + warp) * PIECES + p) * 32 + lane), 0)),
                     "f"(mine[p].x), "f"(mine[p].y), "f"(mine[p].z), "f"(mine[p].w)
                     : "memory");
    }
    cluster_sync();
    if (rank > 0) return ok;
    if (block < n8) {
      for (int r = 1; r < a.cluster; ++r)
#pragma unroll
        for (int p = 0; p < PIECES; ++p) {
          const float4 v = far[(((r - 1) * WARPS + warp) * PIECES + p) * 32 + lane];
          mine[p].x += v.x, mine[p].y += v.y, mine[p].z += v.z, mine[p].w += v.w;
        }
    }
  }
  // value [h][i]: row fragment_row(lane / 4) + 8 * (NB 4: h, else seg & 1), token 8 block + column(2 c + i)
  constexpr int HALVES = NB / 2;
  float v[HALVES][2];
  const int first = 16 * group + fragment_row(lane >> 2) + (NB == 4 ? 0 : 8 * (seg & 1));
  const bool in = i0 + 16 * group < a.I && block < n8;  // whole groups: I is a multiple of 16
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = 8 * block + fragment_column<FP8>(2 * c + i);
    const float f = kScaled<FP8, RG> && a.x_scales && in && j < m ? a.x_scales[items.tok[off + j]] : 1.f;
#pragma unroll
    for (int h = 0; h < HALVES; ++h) {
      float g, w;
      if constexpr (NB == 4) {
        const float gs[4] = {mine[0].x, mine[0].y, mine[0].z, mine[0].w};
        const float us[4] = {mine[1].x, mine[1].y, mine[1].z, mine[1].w};
        g = gs[2 * h + i], w = us[2 * h + i];
      } else {
        g = i ? mine[0].y : mine[0].x, w = i ? mine[0].w : mine[0].z;
      }
      v[h][i] = swiglu(g * f, w * f);
      if (!kScaled<FP8, RG> && in && j < m) store_h<T>(a, off + j, i0 + first + 8 * h, v[h][i], true);
    }
  }
  if constexpr (kScaled<FP8, RG>) {
    // a pair's 64 results have one power of two
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float top = 0.f;
#pragma unroll
      for (int h = 0; h < HALVES; ++h)
        if (in && fabsf(v[h][i]) <= 3.402823466e38f) top = fmaxf(top, fabsf(v[h][i]));
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
      // NB 2: the two warps of a block of tokens have a line each
      if (lane < 4) tops[(group * (4 / NB) + (NB == 4 ? 0 : seg & 1)) * 8 * NB + 8 * block + fragment_column<FP8>(2 * c + i)] = top;
    }
    ok = async::meet<32 * WARPS>(ok);
    const int units = (a.I + 63) / 64;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = 8 * block + fragment_column<FP8>(2 * c + i);
      float top = 0.f;
#pragma unroll
      for (int q = 0; q < RG * (4 / NB); ++q) top = fmaxf(top, tops[q * 8 * NB + j]);
      if (!in || j >= m) continue;
      const int e = f16_exponent(top);
#pragma unroll
      for (int h = 0; h < HALVES; ++h) store_h<F16>(a, off + j, i0 + first + 8 * h, ldexpf(v[h][i], e), a.two);
      if (group == 0 && lane < 4 && (NB == 4 || !(seg & 1))) a.h_scales[(size_t)(off + j) * units + i0 / 64] = ldexpf(1.f, -e);
    }
  }
  return ok;
}

// Gate and up products and SwiGLU. NB: token blocks of 8; RG: row groups.
template <typename T, bool FP8, int NB, int RG>
__global__ void __launch_bounds__(kThreads<RG>, RG == 1 ? 2 : 1)
up_kernel(const __grid_constant__ LayerArgs a, const __grid_constant__ CUtensorMap map,
          const __grid_constant__ CUtensorMap map_x) {
  constexpr int KC = kChunk<FP8, RG>, BLOCKS = kBlocks<FP8, RG>, SEGS = kSegs<RG>, M = 8 * NB, WARPS = kWarps<RG>;
  constexpr int kOuts = 16 * RG, kRows = 32 * RG, BOXES = kBoxes<RG>, kBoxK = KC / BOXES, SW = kStageW<RG>;
  extern __shared__ __align__(1024) uint8_t dyn[];
  __shared__ Ring ring;
  __shared__ Items items;
  uint8_t* stage0 = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
  // weights of all stages (1024-byte aligned), then the tokens' parts, then the warps' sums
  constexpr bool kGather = kScaled<FP8, RG>;
  const int lines = up_lines<FP8, NB, RG>(a.T), kTokens = BLOCKS * lines * 128;
  uint8_t* tokens0 = stage0 + a.stages * SW;
  float* red = reinterpret_cast<float*>(tokens0 + a.stages * kTokens);  // [segs][rows][M + 1]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  init_ring(ring, a.stages, WARPS, kGather ? 1 + 96 : 1);
  if (threadIdx.x == 0) prefetch_map(&map);
  griddep_wait();
  griddep_launch_dependents();  // the down kernel reads results only after its own wait
  sort_pairs<M, kThreads<RG>>(a, items, stage0, blockIdx.x == 0);
  using M16 = std::conditional_t<kScaled<FP8, RG>, F16, T>;  // of the products
  const int tiles = (a.I + kOuts - 1) / kOuts, units = items.n * tiles;
  const int all_stages = (a.H + KC - 1) / KC, cta = blockIdx.x / a.cluster, ctas = gridDim.x / a.cluster;
  const int rank = a.cluster > 1 ? (int)cluster_rank() : 0;
  const int first_stage = all_stages * rank / a.cluster, n_stages = all_stages * (rank + 1) / a.cluster;
  // the same number of units for every CTA that has any, so that all end together
  const int rounds = max(1, (units + ctas - 1) / ctas), step = (units + rounds - 1) / rounds;
  if (threadIdx.x == 0) items.plan[0] = units, items.plan[1] = step;
  // read there: the products need their registers (116 spilled bytes: 330 us, 8: 305)
  const volatile int* plan = items.plan;
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
  uint32_t s = 0, lap = 0;
  if (warp >= WARPS) {
    set_registers<RG, false>();
    bool ok = true;
    if (warp > WARPS) {
      if constexpr (kGather) {
        // ---- an item's tokens, a warp a row: the others' lines would be as many bytes as the
        // weights (9 tokens, 26 experts, hidden 2528, inter 1008: 56 us, now 54; four rows by a
        // gathering tiled copy: 64 tokens 361 us where all tokens' took 321). bf16 weights gain
        // nothing (64 tokens: 460 us, so 465) ----
        static_assert(KC == 8 * 32);
        const int piece = lane;
        const uint32_t to0 = smem_u32(tokens0) + (piece >> 3) * lines * 128;
        for (int u = cta < step ? cta : units; u < units && ok; u += step) {
          const int item = u / tiles, m = items.m[item];
          const uint8_t* tok = items.tok + items.off[item];
          for (int k = first_stage; k < n_stages; ++k) {
            if (lap > 0 && !(ok = wait_warp(&ring.empty[s], (lap & 1) ^ 1))) break;
            const int col = k * KC + piece * 8;
            const uint32_t bytes = col < a.H ? 16 : 0, to = to0 + s * kTokens;
            const uint16_t* from = a.x + (bytes ? col : 0);
            for (int j = warp - WARPS - 1; j < m; j += 3)
              copy16_async(to + j * 128 + (((piece ^ j) & 7) << 4), from + (size_t)tok[j] * a.H, bytes);
            arrive_on_copies(&ring.full[s]);
            if (++s == a.stages) s = 0, ++lap;
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
      }
      return;
    }
    // ---- copies ----
    for (int u = cta < step ? cta : units; u < units && ok; u += step) {
      const int item = u / tiles, i0 = u % tiles * kOuts;
      for (int k = first_stage; k < n_stages; ++k) {
        if (lap > 0 && !(ok = wait_warp(&ring.empty[s], (lap & 1) ^ 1))) break;
        if (lane == 0) {
          const uint32_t bar = smem_u32(&ring.full[s]), to = smem_u32(tokens0 + s * kTokens);
          mbar_arrive_expect_tx(&ring.full[s], SW + (kGather ? 0 : kTokens));
          for (int b = 0; b < BOXES; ++b)
            tma_load4<1>(smem_u32(stage0 + s * SW + b * kRows * 128), &map, k * KC + b * kBoxK, i0, 0, items.e[item], bar);
          if constexpr (!kGather) {
            if (a.whole) tma_load3<1>(to, &map_x, 0, 0, k * BLOCKS, bar);
            else for (int b = 0; b < BLOCKS; ++b) tma_load3<1>(to + b * lines * 128, &map_x, k * KC + b * 64, 0, 0, bar);
          }
        }
        __syncwarp();
        if (++s == a.stages) s = 0, ++lap;
      }
    }
    if (!ok) end_copies(ring, a.stages, s, lap);
    return;
  }
  // ---- products ----
  set_registers<RG, true>();
  const int seg = warp / RG, group = warp % RG, c = lane & 3;
  const int box = seg >> 1, half = seg & 1;
  const int kb = (a.H + 127) / 128, ib = (a.I + 127) / 128;
  // FP8: factors of 32 stages, a lane each; those of the next unit are read ahead
  float gn = 0.f, un = 0.f;
  auto factors = [&](int u, int first, float& g, float& w) {
    const int block = ((first + lane) * KC + seg * 64) / 128;
    if (!FP8 || u >= plan[0] || first + lane >= n_stages || block >= kb) return;
    const float* p = a.w13_scales + ((size_t)items.e[u / tiles] * 2 * ib + u % tiles * kOuts / 128) * kb + block;
    g = __ldg(p);
    w = __ldg(p + (size_t)ib * kb);
  };
  factors(cta, first_stage & ~31, gn, un);
  bool ok = true;
  for (int u = cta < step ? cta : units, turn = 0; u < plan[0]; u += plan[1], turn ^= 1) {
    const int item = u / tiles, m = items.m[item], n8 = (m + 7) / 8, off = items.off[item];
    float acc[2][NB][4] = {};
    uint32_t nan[4] = {};
    int token[NB];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const int j = 8 * n + fragment_column<FP8>(lane >> 2);
      token[n] = kGather ? j : items.tok[off + j];
    }
    float g = gn, w = un;
    factors(u + plan[1], 0, gn, un);  // (more than one unit: a cluster of 1)
    for (int k = first_stage; k < n_stages; ++k) {
      if (FP8 && k > first_stage && (k & 31) == 0) factors(u, k, g, w);
      const float sg = FP8 ? __shfl_sync(~0u, g, k & 31) : 1.f, su = FP8 ? __shfl_sync(~0u, w, k & 31) : 1.f;
      if (!(ok = wait_warp(&ring.full[s], lap & 1))) break;
      multiply<M16, FP8, NB, 1>(smem_u32(stage0 + s * SW + box * kRows * 128), 16 * group, kOuts + 16 * group, half,
                              smem_u32(tokens0 + s * kTokens + (FP8 ? seg : box) * lines * 128), token, 0, n8, sg, su, acc, nan);
      async::release_slot(&ring.empty[s]);
      if (++s == a.stages) s = 0, ++lap;
    }
    if (FP8 && M16::kBf16) spread_nan(nan, acc);
    const int i0 = u % tiles * kOuts;
    if constexpr (RG > 1) {
      if (a.cluster > 1) cluster_arrive();  // done with the ring
      if (!(ok = finish<T, FP8, NB, RG>(a, items, item, i0, ok, turn, red, reinterpret_cast<float4*>(stage0), acc))) break;
      continue;
    }
    // the warps' shares: red[seg][row][token]
    const int row = 32 * group + fragment_row(lane >> 2);
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          red[(seg * kRows + row + 16 * f + 8 * (i >> 1)) * (M + 1) + 8 * n + fragment_column<FP8>(2 * c + (i & 1))] = acc[f][n][i];
    if (!(ok = async::meet<32 * WARPS>(ok))) break;
    for (int v = threadIdx.x; v < kOuts * m; v += 32 * WARPS) {
      const int o = v % kOuts, j = v / kOuts;
      if (i0 + o >= a.I) continue;
      const float* p = red + (32 * (o / 16) + o % 16) * (M + 1) + j;
      float pg = 0.f, pu = 0.f;
#pragma unroll
      for (int q = 0; q < SEGS; ++q) {
        pg += p[q * kRows * (M + 1)];
        pu += p[(q * kRows + 16) * (M + 1)];
      }
      store_h<T>(a, off + j, i0 + o, swiglu(pg, pu), true);
    }
    if (!async::meet<32 * WARPS>(true)) break;
  }
}

// Down product and weighted sum. TWO: h as two numbers.
template <typename T, bool FP8, int NB, int RG, bool TWO>
__global__ void __launch_bounds__(kThreads<RG>, RG == 1 ? 2 : 1)
down_kernel(const __grid_constant__ LayerArgs a, const __grid_constant__ CUtensorMap map,
            const __grid_constant__ TokenMaps map_h) {
  constexpr int KC = kChunk<FP8, RG>, BLOCKS = kBlocks<FP8, RG>, M = 8 * NB, WARPS = kWarps<RG>;
  constexpr int kRows = 32 * RG, BOXES = kBoxes<RG>, kBoxK = KC / BOXES, kLine = kDownLine<RG>, SW = kStageW<RG>;
  constexpr bool SCALED = kScaled<FP8, RG>;
  constexpr int PARTS = TWO ? 2 : 1, kTokens = BLOCKS * PARTS * M * 128;  // the numbers' lines
  using M16 = std::conditional_t<SCALED, F16, T>;  // of the products
  constexpr int kSums = kDownSums<RG, NB>;
  extern __shared__ __align__(1024) uint8_t dyn[];
  __shared__ Ring ring;
  __shared__ Items items;
  uint8_t* stage0 = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
  uint8_t* tokens0 = stage0 + a.stages * SW;
  float* sums = reinterpret_cast<float*>(tokens0 + a.stages * kTokens);  // [kSums][T][kLine]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = a.cluster > 1 ? (int)cluster_rank() : 0;
  const int o0 = blockIdx.x / a.cluster * kRows;
  init_ring(ring, a.stages, WARPS);
  if (threadIdx.x == 0) prefetch_map(&map);
  // ids, mask and weights were complete before the up kernel let this one start
  sort_pairs<M, kThreads<RG>>(a, items, stage0, false);
  for (int v = threadIdx.x; v < kSums * a.T * kLine; v += kThreads<RG>) sums[v] = 0.f;
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
  const int per = (a.I + KC - 1) / KC, total = items.n * per;
  const int begin = (int)((int64_t)total * rank / a.cluster), end = (int)((int64_t)total * (rank + 1) / a.cluster);
  uint32_t s = 0, lap = 0;
  if (warp >= WARPS) {
    set_registers<RG, false>();
    if (warp == WARPS) {
    // ---- copies: weights of as many stages as the ring has before the wait for h ----
    auto load_weights = [&](int v, int st) {
      const int item = v / per, k = v % per;
      if (lane == 0) {
        mbar_arrive_expect_tx(&ring.full[st], SW + BLOCKS * PARTS * 128 * lines_of(items.m[item]));
        for (int b = 0; b < BOXES; ++b)
          tma_load3<1>(smem_u32(stage0 + st * SW + b * kRows * 128), &map, k * KC + b * kBoxK, o0, items.e[item],
                       smem_u32(&ring.full[st]));
      }
      __syncwarp();
    };
    auto load_tokens = [&](int v, int st) {  // an item's rows of h lie together
      const int item = v / per, k = v % per, rows = lines_of(items.m[item]);
      const CUtensorMap* from = rows == 8 ? &map_h.rows8 : rows == 16 ? &map_h.rows16 : &map_h.rows32;
      const uint32_t to = smem_u32(tokens0 + st * kTokens), bar = smem_u32(&ring.full[st]);
      if (lane == 0) {
        if (a.whole) {
          tma_load4<1>(to, from, 0, items.off[item], 0, k * BLOCKS, bar);
        } else {
          for (int b = 0; b < BLOCKS; ++b)
            tma_load4<1>(to + b * PARTS * rows * 128, from, k * KC + b * 64, items.off[item], 0, 0, bar);
        }
      }
      __syncwarp();
    };
    const int ahead = min(a.stages, end - begin);
    for (int v = 0; v < ahead; ++v) load_weights(begin + v, v);
    griddep_wait();
    for (int v = 0; v < ahead; ++v) load_tokens(begin + v, v);
    s = ahead == a.stages ? 0 : ahead;
    lap = ahead == a.stages ? 1 : 0;
    bool ok = true;
    for (int v = begin + ahead; v < end; ++v) {
      if (!(ok = wait_warp(&ring.empty[s], (lap & 1) ^ 1))) break;
      load_weights(v, s);
      load_tokens(v, s);
      if (++s == a.stages) s = 0, ++lap;
    }
    if (!ok) end_copies(ring, a.stages, s, lap);
    }
  } else {
    // ---- products ----
    set_registers<RG, true>();
    const int seg = warp / RG, group = warp % RG, c = lane & 3;
    const int box = seg >> 1, half = seg & 1;
    int token[NB];
#pragma unroll
    for (int n = 0; n < NB; ++n) token[n] = 8 * n + fragment_column<FP8>(lane >> 2);
    const int hb = (a.H + 127) / 128, ib = (a.I + 127) / 128;
    const int ob = min((o0 + 32 * group) / 128, hb - 1);  // the block of this warp's rows
    float fn = 0.f;
    auto factors = [&](int item, int first, float& f) {
      const int block = ((first + lane) * KC + seg * 64) / 128;
      if (!FP8 || item >= items.n || first + lane >= per || block >= ib) return;
      f = __ldg(a.w2_scales + ((size_t)items.e[item] * hb + ob) * ib + block);
    };
    if (begin < end) factors(begin / per, 0, fn);
    // scaled: h's powers of two, a pair a lane, of this warp's 64 k of a stage. Ordinary loads: the
    // up kernel may still write them while this kernel starts, and a read-only load need not stay
    // behind the wait.
    const int units = (a.I + 63) / 64;
    float column = 1.f;
    auto columns = [&](int v) {
      if (!SCALED || v >= end) return;
      const int item = v / per, unit = v % per * BLOCKS + seg;
      if (lane < items.m[item] && unit < units) column = a.h_scales[(size_t)(items.off[item] + lane) * units + unit];
    };
    if (SCALED) griddep_wait();
    columns(begin);
    bool ok = true;
    int turn = 0;
    for (int v = begin; v < end && ok;) {
      const int item = v / per, m = items.m[item], n8 = (m + 7) / 8, off = items.off[item];
      const int k0 = v % per, k1 = min(per, k0 + end - v), part = lines_of(m) * 128;
      float acc[2][NB][4] = {};
      uint32_t nan[4] = {};
      float f = fn;
      factors(item + 1, 0, fn);
      if (FP8 && k0 >= 32) factors(item, k0 & ~31, f);
      for (int k = k0; k < k1; ++k) {
        if (FP8 && k > k0 && (k & 31) == 0) factors(item, k, f);
        const float sf = FP8 ? __shfl_sync(~0u, f, k & 31) : 1.f, now = column;
        columns(v + k - k0 + 1);
        if (!(ok = wait_warp(&ring.full[s], lap & 1))) break;
        multiply<M16, FP8, NB, PARTS, SCALED>(smem_u32(stage0 + s * SW + box * kRows * 128), 32 * group, 32 * group + 16, half,
                                              smem_u32(tokens0 + s * kTokens + (FP8 ? seg : box) * PARTS * part), token, part,
                                              n8, sf, sf, acc, nan, now);
        async::release_slot(&ring.empty[s]);
        if (++s == a.stages) s = 0, ++lap;
      }
      v += k1 - k0;
      if (FP8 && M16::kBf16) spread_nan(nan, acc);
      // an item's tokens all differ, and a warp's rows are its own
      const int row = 32 * group + fragment_row(lane >> 2);
      auto add = [&] {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int j = 8 * n + fragment_column<FP8>(2 * c + i);
            if (j >= m) continue;
            const float wt = items.weight[off + j];
            float* to = sums + ((kTurns<RG, NB> ? seg >> 1 : seg) * a.T + items.tok[off + j]) * kLine + row;
#pragma unroll
            for (int r = 0; r < 4; ++r) to[8 * r] = fmaf(wt, acc[r >> 1][n][2 * (r & 1) + i], to[8 * r]);
          }
      };
      if constexpr (kTurns<RG, NB>) {
        // two warps share rows and sums: the first to add is the other one for the next item,
        // so that they meet once an item
        const bool leads = ((seg ^ turn) & 1) == 0;
        turn ^= 1;
        if (leads) add();
        ok = async::meet<64>(ok, 2 + 2 * group + (seg >> 1));
        if (!leads && ok) add();
      } else {
        add();
      }
    }
  }
  __syncthreads();
  for (int v = threadIdx.x; v < a.T * kLine; v += kThreads<RG>) {
    float t = sums[v];
#pragma unroll
    for (int q = 1; q < kSums; ++q) t += sums[q * a.T * kLine + v];
    sums[v] = t;
  }
  if (a.cluster > 1) cluster_sync();
  else __syncthreads();
  // The tile's results, shared out among the CTAs.
  constexpr int kMany = 32 * WARPS;
  if (warp < WARPS) {
    for (int v = rank * kMany + threadIdx.x; v < a.T * kRows; v += a.cluster * kMany) {
      const int t = v / kRows, o = v % kRows;
      float r = 0.f;
      if (a.cluster > 1) {
        for (int q = 0; q < a.cluster; ++q) {
          float w;
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(w) : "r"(addr_in(smem_u32(sums + t * kLine + o), q)) : "memory");
          r += w;
        }
      } else {
        r = sums[t * kLine + o];
      }
      if (o0 + o >= a.H) continue;
      const size_t at = (size_t)t * a.H + o0 + o;
      if (a.out_f32) static_cast<float*>(a.y)[at] = r;
      else static_cast<uint16_t*>(a.y)[at] = rounded<T>(r);
    }
  }
  if (a.cluster > 1) cluster_sync();
}

// ---- host ----
struct Maps {
  CUtensorMap w13, w2, x;
  TokenMaps h;
};

// Stages of a ring: what fits beside `rest` with `ctas` a SM.
int fit_stages(size_t rest, size_t stage, int ctas) {
  const size_t room = (227 * 1024) / ctas - sizeof(Items) - 2048;
  return (int)std::min<size_t>(8, (room - 1024 - rest) / stage);
}

template <typename T, bool FP8, int NB, int RG>
cudaError_t launch_up(LayerArgs a, const Maps& maps, int sms, cudaStream_t s) {
  constexpr auto kernel = up_kernel<T, FP8, NB, RG>;
  constexpr int M = 8 * NB, kPerSm = RG == 1 ? 2 : 1;
  constexpr size_t rest = 4 * kUpFloats<RG, NB>;
  const size_t stage = kStageW<RG> + kBlocks<FP8, RG> * up_lines<FP8, NB, RG>(a.T) * 128;
  a.stages = fit_stages(rest, stage, kPerSm);
  a.whole = a.H % 64 == 0;
  const size_t smem = 1024 + a.stages * stage + rest;
  // sort_pairs' scratch lies in the ring: 29 KB at most
  if (a.stages < 2 || smem < 1024 + 10 * (size_t)a.G + 8 * (size_t)(a.T * a.K)) return cudaErrorInvalidValue;
  cudaError_t e = prepare_kernel<kernel>(smem);
  if (e == cudaSuccess && RG > 1) e = check_registers<kernel>(kThreads<RG>, kAllRegs<RG>);
  if (e != cudaSuccess) return e;
  // An expert's tokens make one item, and one more for every M of them.
  const int experts = std::min(a.G, a.T * a.K), items = experts + (a.T > M ? a.T * a.K / M : 0);
  const int64_t most = (int64_t)items * ((a.I + 16 * RG - 1) / (16 * RG));
  // Few units: clusters share the stages of one, as many CTAs as find a place at once, two
  // stages each at least (46 tokens, 6 experts, hidden 5840, inter 288, 16-bit
  // weights: 48 us, so 35; 40 tokens, 3 experts, hidden 4096, inter 384, fp8: 31, so 20).
  a.cluster = 1;
  if (RG > 1 && 2 * most <= sms)
    for (int c = (int)std::min<int64_t>({8, sms / most, (a.H + kChunk<FP8, RG> - 1) / kChunk<FP8, RG> / 2}); c > 1; --c)
      if ((size_t)(c - 1) * kWarps<RG> * kBoxLines<RG, NB> * 512 <= a.stages * stage &&
          most + (c > 2) <= active_clusters<kernel>(c, kThreads<RG>, smem)) {
        a.cluster = c;
        break;
      }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(std::min<int64_t>(most, sms * kPerSm) * a.cluster));
  cfg.blockDim = dim3(kThreads<RG>);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)a.cluster, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = a.cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, maps.w13, maps.x);
}

// The down kernel's launch: tiles, and as many CTAs a tile as are all on the GPU at once: a
// second wave pays its start again (1 token, hidden 7168: 134 us with 4, 117 with 1; 64
// tokens, fp8: 529 with 8, 491 with 2). Clusters that the SMs would hold need not all find a
// place (hidden 2064, 17 tiles: 15 clusters of 8; 54 us, with 22 tiles and clusters of 6:
// 40), and while the up kernel ends, one fewer may (hidden 5840, 46 tiles, as many clusters of
// 3: 49 us; 61 of 2: 38).
template <typename T, bool FP8, int NB, int RG, bool TWO>
struct Down {
  static constexpr auto kernel = down_kernel<T, FP8, NB, RG, TWO>;
  static constexpr int kRows = 32 * RG, kPerSm = RG == 1 ? 2 : 1;
  int tiles, cluster = 1, stages;
  size_t smem;
  Down(const LayerArgs& a, int sms) : tiles((a.H + kRows - 1) / kRows) {
    constexpr size_t stage = kStageW<RG> + kBlocks<FP8, RG> * (TWO ? 2 : 1) * 8 * NB * 128;
    const size_t rest = 4 * (size_t)kDownSums<RG, NB> * a.T * kDownLine<RG>;
    stages = fit_stages(rest, stage, kPerSm);
    smem = 1024 + stages * stage + rest;
    for (int c = std::min(8, kPerSm * sms / tiles); c > 1; --c)
      if (tiles + (c > 2) <= active_clusters<kernel>(c, kThreads<RG>, smem)) {
        cluster = c;
        break;
      }
  }
};

template <typename T, bool FP8, int NB, int RG, bool TWO>
cudaError_t launch_down(LayerArgs a, const Maps& maps, int sms, cudaStream_t s) {
  const Down<T, FP8, NB, RG, TWO> d(a, sms);
  constexpr auto kernel = d.kernel;
  const size_t smem = d.smem;
  a.stages = d.stages;
  a.cluster = d.cluster;
  a.whole = a.I % 64 == 0;
  if (a.stages < 2 || smem < 1024 + 10 * (size_t)a.G + 8 * (size_t)(a.T * a.K)) return cudaErrorInvalidValue;
  cudaError_t e = prepare_kernel<kernel>(smem);
  if (e == cudaSuccess && RG > 1) e = check_registers<kernel>(kThreads<RG>, kAllRegs<RG>);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(d.tiles * d.cluster);
  cfg.blockDim = dim3(kThreads<RG>);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)d.cluster, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a, maps.w2, maps.h);
}

// RU, RD: row groups of the two kernels.
template <typename T, bool FP8, int NB, int RU, int RD, bool TWO>
cudaError_t launch_t(LayerArgs a, const void* w13, const void* w2, int sms, cudaStream_t s) {
  constexpr int M = 8 * NB;
  constexpr bool kScale = kScaled<FP8, RD>;
  static_assert(kScaled<FP8, RU> == kScale && (TWO || kScale), "both kernels hold h alike");
  a.two = TWO;
  const MapType type = FP8 ? kMapU8 : T::kBf16 ? kMapBF16 : kMapF16, token = T::kBf16 && !kScale ? kMapBF16 : kMapF16;
  if (kScale && T::kBf16) {
    const cudaError_t e = launch_pdl(scale_kernel, dim3(a.T), dim3(256), 0, s, a.x, a.x16, a.x_scales, a.H);
    if (e != cudaSuccess) return e;
    a.x = a.x16;
  } else {
    a.x_scales = nullptr;
  }
  const uint64_t es = FP8 ? 1 : 2, H = a.H, I = a.I, G = a.G, P = (uint64_t)a.T * a.K;
  Maps m = {};
  {
    const uint64_t d[] = {H, I, 2, G}, st[] = {es * H, es * I * H, es * 2 * I * H};
    const uint32_t b[] = {(uint32_t)(128 / es), 16 * RU, 2, 1};
    if (!make_map(&m.w13, w13, type, 4, d, st, b)) return cudaErrorUnknown;
  }
  {
    const uint64_t d[] = {I, H, G}, st[] = {es * I, es * I * H};
    const uint32_t b[] = {(uint32_t)(128 / es), 32 * RD, 1};
    if (!make_map(&m.w2, w2, type, 3, d, st, b)) return cudaErrorUnknown;
  }
  if (!kScale) {
    const bool whole = H % 64 == 0;
    const uint64_t d[] = {whole ? 64 : H, (uint64_t)a.T, whole ? H / 64 : 1}, st[] = {2 * H, whole ? 128 : 2 * H * a.T};
    const uint32_t b[] = {64, (uint32_t)(a.T + 7) / 8 * 8, whole ? (uint32_t)kBlocks<FP8, RU> : 1};
    if (!make_map(&m.x, a.x, token, 3, d, st, b)) return cudaErrorUnknown;
  }
  const bool whole = I % 64 == 0;
  const uint64_t d[] = {whole ? 64 : I, P, TWO ? 2 : 1, whole ? I / 64 : 1};
  const uint64_t st[] = {2 * I, 2 * I * P, whole ? 128 : 4 * I * P};
  CUtensorMap* const to[] = {&m.h.rows8, &m.h.rows16, &m.h.rows32};
  for (int k = 0; k < 3 && 8 << k <= M; ++k) {
    const uint32_t b[] = {64, 8u << k, TWO ? 2 : 1, whole ? (uint32_t)kBlocks<FP8, RD> : 1};
    if (!make_map(to[k], a.h, token, 4, d, st, b)) return cudaErrorUnknown;
  }
  const cudaError_t e = launch_up<T, FP8, NB, RU>(a, m, sms, s);
  return e == cudaSuccess ? launch_down<T, FP8, NB, RD, TWO>(a, m, sms, s) : e;
}

template <typename T, bool FP8, int NB, bool TWO>
cudaError_t launch_tiles(const LayerArgs& a, const void* w13, const void* w2, int sms, cudaStream_t s) {
  const Down<T, FP8, NB, 3, TWO> d3(a, sms);
  const Down<T, FP8, NB, 4, TWO> d4(a, sms);
  return d3.tiles * d3.cluster > d4.tiles * d4.cluster ? launch_t<T, FP8, NB, 4, 3, TWO>(a, w13, w2, sms, s)
                                                       : launch_t<T, FP8, NB, 4, 4, TWO>(a, w13, w2, sms, s);
}

template <typename T, bool FP8, int NB>
cudaError_t launch_large(const LayerArgs& a, const void* w13, const void* w2, int sms, cudaStream_t s) {
  if constexpr (FP8 && T::kBf16)
    if (!a.out_f32) return launch_tiles<T, FP8, NB, false>(a, w13, w2, sms, s);
  return launch_tiles<T, FP8, NB, true>(a, w13, w2, sms, s);
}

// Tiles of 128 rows and sixteen warps, one CTA a SM, where that gives each SM a unit of the
// up kernel (hidden 7168, inter 2048, bf16, 8 tokens: 366 us against 383 with tiles of 32
// rows and two CTAs a SM; fp8, 2 tokens: 131 against 132, 8 tokens: 244 against 269; fp16
// tokens with fp8 weights need no cheaper decoding: small tiles up to 4 tokens (2 tokens,
// hidden 512, inter 1536: 20 against 23; hidden 4096, inter 1408: 57 against 60; hidden 7168,
// inter 2048: 107 against 104)). With fewer units and up to 8 tokens, the small ones where rows
// are short (hidden 1024, inter 512, 8 tokens: 14.2 against 15.0) or bf16 tokens would be scaled
// first (fp8, hidden 4096, inter 512, 8 tokens: 18 against 23), else clusters of large ones
// (hidden 7168, inter 1024, 1 token: 17 against 21; hidden 1552, inter 384, 2 tokens: 16 against
// 17).
// The down kernel takes tiles of 96 rows where those and their clusters cover more SMs
// (hidden 7168: 150 of 152 instead of 112; 64 tokens, bf16: 524 -> 494 us).
template <typename T, bool FP8>
cudaError_t launch(const LayerArgs& a, const void* w13, const void* w2, cudaStream_t s) {
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorUnknown;
  const bool units = (int64_t)std::min(a.G, a.T * a.K) * ((a.I + 63) / 64) >= sms;
  const bool small = units ? FP8 && !T::kBf16 && a.T <= 4 : (FP8 && T::kBf16) || a.H < 1536;
  if (a.T <= 8 && small) return launch_t<T, FP8, 1, 1, 1, true>(a, w13, w2, sms, s);
  return a.T <= 16 ? launch_large<T, FP8, 2>(a, w13, w2, sms, s) : launch_large<T, FP8, 4>(a, w13, w2, sms, s);
}

int validate(const cq_moe_config* c) {
  if (!c || c->tokens < 0 || c->tokens > 64 || c->experts < 1 || c->experts > 2048) return CQ_ERR_ARG;
  if (c->topk < 1 || c->topk > 16) return CQ_ERR_ARG;
  if (c->hidden < 16 || c->hidden > 65536 || c->inter < 16 || c->inter > 65536) return CQ_ERR_ARG;
  if (c->x_dtype < 0 || c->x_dtype > 1 || c->w_dtype < 0 || c->w_dtype > 1) return CQ_ERR_ARG;
  if (c->mask_ndim < 0 || c->mask_ndim > 2 || c->out_dtype < 0 || c->out_dtype > 1) return CQ_ERR_ARG;
  if (c->hidden % 16 != 0 || c->inter % 16 != 0) return CQ_ERR_UNSUPPORTED;
  return CQ_OK;
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// The workspace: h, and for fp8 weights its scales, the tokens' and the scaled tokens.
struct Layout {
  size_t h_scales, x_scales, x16, bytes;
  explicit Layout(const cq_moe_config& c) {
    const size_t P = (size_t)c.tokens * c.topk;
    h_scales = align256(4 * P * c.inter);
    x_scales = h_scales + (c.w_dtype ? align256(4 * P * ((c.inter + 63) / 64)) : 0);
    x16 = x_scales + (c.w_dtype ? 256 : 0);  // 64 floats
    bytes = x16 + (c.w_dtype ? align256(2 * (size_t)c.tokens * c.hidden) : 0) + 256;
  }
};

}  // namespace

int layer_status(uint32_t* read, cudaStream_t s) { return status_word(g_status, read, s); }

}  // namespace expert
}  // namespace cq

using namespace cq::expert;

extern "C" {

int cq_check_moe_config(const cq_moe_config* cfg) { return validate(cfg); }

size_t cq_moe_workspace_size(const cq_moe_config* cfg) {
  if (validate(cfg) != CQ_OK) return 0;
  return Layout(*cfg).bytes;
}

int cq_moe_layer(const cq_moe_config* cfg, const void* x, const int32_t* expert_ids,
                 const float* expert_scales, const uint8_t* x_active_mask, const void* w13,
                 const float* w13_scales, const void* w2, const float* w2_scales, void* y,
                 void* workspace, size_t workspace_bytes, void* stream) {
  const int rc = validate(cfg);
  if (rc != CQ_OK) return rc;
  const bool rows = cfg->tokens > 0;
  if ((rows && (!x || !expert_ids || !expert_scales || !y)) || !w13 || !w2) return CQ_ERR_ARG;
  if (cfg->mask_ndim ? rows && !x_active_mask : x_active_mask != nullptr) return CQ_ERR_ARG;
  if (cfg->w_dtype ? !w13_scales || !w2_scales : w13_scales || w2_scales) return CQ_ERR_ARG;
  for (const void* p : {x, w13, w2, (const void*)y})
    if (!aligned(p, 16)) return CQ_ERR_ARG;
  for (const void* p : {(const void*)expert_ids, (const void*)expert_scales, (const void*)w13_scales,
                        (const void*)w2_scales})
    if (!aligned(p, 4)) return CQ_ERR_ARG;
  if (!rows) return CQ_OK;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < cq_moe_workspace_size(cfg))
    return CQ_ERR_WORKSPACE;
  LayerArgs a = {};
  a.T = cfg->tokens;
  a.G = cfg->experts;
  a.K = cfg->topk;
  a.H = cfg->hidden;
  a.I = cfg->inter;
  a.mask_ndim = cfg->mask_ndim;
  a.out_f32 = cfg->out_dtype;
  a.x = static_cast<const uint16_t*>(x);
  a.ids = expert_ids;
  a.scales = expert_scales;
  a.mask = x_active_mask;
  a.w13_scales = w13_scales;
  a.w2_scales = w2_scales;
  const Layout at(*cfg);
  char* ws = static_cast<char*>(workspace);
  a.h = reinterpret_cast<uint16_t*>(ws);
  a.h_scales = reinterpret_cast<float*>(ws + at.h_scales);
  a.x_scales = reinterpret_cast<float*>(ws + at.x_scales);
  a.x16 = reinterpret_cast<uint16_t*>(ws + at.x16);
  a.y = y;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = cfg->x_dtype == 1
                            ? (cfg->w_dtype ? launch<cq::F16, true>(a, w13, w2, s) : launch<cq::F16, false>(a, w13, w2, s))
                            : (cfg->w_dtype ? launch<cq::BF16, true>(a, w13, w2, s) : launch<cq::BF16, false>(a, w13, w2, s));
  return e == cudaSuccess ? CQ_OK : CQ_ERR_CUDA;
}

}  // extern "C"
