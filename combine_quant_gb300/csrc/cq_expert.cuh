// cq_expert.cuh -- argument blocks and device helpers shared by the expert
// products (grouped matrix products between dispatch and combine).
#pragma once

#include "cq_internal.cuh"

namespace cq {
namespace expert {

// The token type of a product's operands.
enum { kBF16 = 0, kF16 = 1, kMxE4M3 = 2, kMxE5M2 = 3 };

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

}  // namespace expert
}  // namespace cq
