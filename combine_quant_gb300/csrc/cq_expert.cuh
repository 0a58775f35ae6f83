// cq_expert.cuh -- argument blocks and device helpers shared by the expert
// products (grouped matrix products between dispatch and combine).
#pragma once

#include "cq_internal.cuh"

namespace cq {
namespace expert {

// The token type of a product's operands.
enum { kBF16 = 0, kF16 = 1, kMxE4M3 = 2, kMxE5M2 = 3 };

enum Op { kForward, kDx, kDw };

struct Args {
  int32_t G, R, N, K;   // experts, rows, weight rows (2n with SwiGLU), inner length
  int32_t x_dtype, w_dtype, out_dtype, act, group;
  int32_t rows_type, L;
  int32_t SC;           // mx scale columns
  const void* x;        // forward: x; dx: dy; dw: x
  const void* w;        // forward, dx: weights; dw: dy
  const uint8_t* x_scales;
  const uint8_t* w_scales;
  const void* scales4;   // 4-bit weights: scales and zero points
  const uint8_t* zeros4;
  const int64_t* group_rows;
  const void* pre_in;   // dx through SwiGLU: the saved products
  void* pre_out;        // forward with SwiGLU: receives them, or NULL
  void* out;
};

// Rows of expert e before clipping. Running sums restart every L entries; an
// entry below its predecessor (the unused entries of a shared-expert rank,
// which hold 0) has no rows.
__device__ __forceinline__ int64_t group_count(const int64_t* v, int e, int rows_type, int L) {
  const int64_t c = v[e];
  if (rows_type == 1 || e % L == 0) return c;
  const int64_t p = v[e - 1];
  return c < p ? 0 : c - p;
}

// First rows of the experts, clipped to R, in begin[0..G], and the running
// sums of their tile counts tiles_of(rows) in tile[0..G]. Called by every
// thread of a CTA of THREADS threads; every CTA repeats it (G <= 2048 values
// from L2), which spares a launch and a round trip through memory.
template <int THREADS, typename F>
__device__ __forceinline__ bool group_scan(const Args& a, int* begin, int* tile, F tiles_of) {
  constexpr int kWarps = THREADS / 32;
  __shared__ int64_t s_rows[kWarps];
  __shared__ int s_tiles[kWarps];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int per = (a.G + THREADS - 1) / THREADS;
  const int e0 = min(a.G, t * per), e1 = min(a.G, e0 + per);
  bool bad = false;
  auto count = [&](int e) {
    int64_t c = group_count(a.group_rows, e, a.rows_type, a.L);
    if (c < 0) bad = true, c = 0;
    if (c > a.R) bad = true, c = a.R;
    return c;
  };
  int64_t sum = 0;
  for (int e = e0; e < e1; ++e) sum += count(e);
  int64_t run = sum;
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(~0u, run, o);
    if (lane >= o) run += v;
  }
  if (lane == 31) s_rows[warp] = run;
  __syncthreads();
  int64_t first = run - sum;
  for (int w = 0; w < warp; ++w) first += s_rows[w];
  int mine = 0;
  for (int e = e0; e < e1; ++e) {
    const int64_t c = count(e);
    const int b = (int)min(first, (int64_t)a.R);
    first += c;
    const int n = (int)min(first, (int64_t)a.R) - b;
    bad |= first > a.R;
    begin[e] = b;
    mine += tiles_of(n);
    tile[e] = tiles_of(n);
  }
  if (e0 < a.G && e1 == a.G) begin[a.G] = (int)min(first, (int64_t)a.R);
  int tr = mine;
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(~0u, tr, o);
    if (lane >= o) tr += v;
  }
  if (lane == 31) s_tiles[warp] = tr;
  __syncthreads();
  int at = tr - mine;
  for (int w = 0; w < warp; ++w) at += s_tiles[w];
  for (int e = e0; e < e1; ++e) {
    const int n = tile[e];
    tile[e] = at;
    at += n;
  }
  if (e0 < a.G && e1 == a.G) tile[a.G] = at;
  __syncthreads();
  return bad;
}

// The expert of tile t: the last e with tile[e] <= t (t < tile[G]).
__device__ __forceinline__ int expert_of(const int* tile, int G, int t) {
  int lo = 0, hi = G;  // tile[lo] <= t < tile[hi]
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (tile[m] <= t) lo = m;
    else hi = m;
  }
  return lo;
}

// y = u * g / (1 + exp(-g)) in 32 bits. exp(-g) leaves 32 bits for gates below -88 (and
// __fdividef's range from -87.4), and u * g may where y does not. So with h =
// exp(-|g| / 2): y = u * g / (1 + h^2) for g >= 0, else (u * h) * (g * h) / (1 + h^2).
__device__ __forceinline__ float swiglu(float g, float u) {
  const float h = __expf(-0.5f * fabsf(g)), r = __fdividef(1.f, fmaf(h, h, 1.f));
  const float a = g >= 0.f ? 1.f : h;
  return u * a * (g * a * r);
}

// Reads and clears a translation unit's status word, waiting for the stream.
template <typename Word>
int read_status_word(Word& word, uint32_t* status, cudaStream_t s) {
  uint32_t v = 0;
  const uint32_t zero = 0;
  if (cudaMemcpyFromSymbolAsync(&v, word, sizeof v, 0, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return CQ_ERR_CUDA;
  *status = v;
  if (v &&
      (cudaMemcpyToSymbolAsync(word, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, s) != cudaSuccess ||
       cudaStreamSynchronize(s) != cudaSuccess))
    return CQ_ERR_CUDA;
  return CQ_OK;
}

// Launchers, and the status words of their kernels (read and cleared).
int launch_gemm(Op op, const Args& a, cudaStream_t s);
int launch_w4(const Args& a, cudaStream_t s);
int gemm_status(uint32_t* status, cudaStream_t s);
int w4_status(uint32_t* status, cudaStream_t s);

}  // namespace expert
}  // namespace cq
