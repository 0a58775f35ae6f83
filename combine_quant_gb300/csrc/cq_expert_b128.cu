// cq_expert_b128.cu -- expert products from fp8 rows with one scale per 128 columns
// and fp8 weights with one per 128 x 128 block: forward (SwiGLU, results in 16 bits
// or in fp8 with scales) and the gradient of the input.
//
// The simplest form: a warp computes 128 results of a row, one after the other.
#include <cuda_fp8.h>

#include "cq_expert.cuh"

namespace cq {
namespace expert {
namespace {

__device__ uint32_t g_status;  // CQ_ST_* bits of these kernels on this device

struct B128Args : Args {
  const float* xs;
  const float* ws;
  float* ys;
  int32_t n, nb, kb;  // n, its blocks, k's blocks
};

template <bool E5>
__device__ __forceinline__ float fp8_value(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, E5 ? __NV_E5M2 : __NV_E4M3)));
}
__device__ __forceinline__ float value(uint8_t c, bool e5) {
  return e5 ? fp8_value<true>(c) : fp8_value<false>(c);
}

__device__ __forceinline__ float warp_sum(float v) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

template <typename T>
__device__ __forceinline__ void put(void* p, size_t at, float v) {
  static_cast<uint16_t*>(p)[at] = (uint16_t)T::pack2(v, 0.f);
}
template <typename T>
__device__ __forceinline__ float get(const void* p, size_t at) {
  return T::lo(static_cast<const uint16_t*>(p)[at]);
}

template <typename T>
__global__ void __launch_bounds__(256) forward_kernel(const __grid_constant__ B128Args a) {
  extern __shared__ int lists[];
  int *begin = lists, *tile = lists + a.G + 1;
  griddep_wait();
  const bool bad = group_scan<256>(a, begin, tile, [](int rows) { return rows; });
  if (bad && blockIdx.x == 0) atomicOr(&g_status, (uint32_t)CQ_ST_BAD_ROWS);
  const int lane = threadIdx.x & 31;
  const int64_t total = (int64_t)tile[a.G] * a.nb;
  for (int64_t task = blockIdx.x * 8 + (threadIdx.x >> 5); task < total; task += gridDim.x * 8) {
    const int r = (int)(task / a.nb), b = (int)(task % a.nb);
    const int e = expert_of(tile, a.G, r);
    const uint8_t* x = static_cast<const uint8_t*>(a.x) + (size_t)r * a.K;
    auto dot = [&](int half, int o) {
      const uint8_t* w = static_cast<const uint8_t*>(a.w) + ((size_t)e * a.N + half * a.n + o) * a.K;
      const float* ws = a.ws + ((size_t)e * (a.N / a.n) * a.nb + half * a.nb + o / 128) * a.kb;
      float sum = 0.f;
      for (int j = lane; j < a.K; j += 32)
        sum = fmaf(value(x[j], a.x_dtype == kMxE5M2) * value(w[j], a.w_dtype == 1),
                   a.xs[(size_t)r * a.kb + j / 128] * ws[j / 128], sum);
      return warp_sum(sum);
    };
    float v[4] = {}, g[4] = {}, u[4] = {};
    for (int o = 0; o < 128 && b * 128 + o < a.n; ++o) {
      const float p = dot(0, b * 128 + o), q = a.act ? dot(1, b * 128 + o) : 0.f;
#pragma unroll
      for (int m = 0; m < 4; ++m)
        if (o == 32 * m + lane) g[m] = p, u[m] = q, v[m] = a.act ? swiglu(p, q) : p;
    }
    float top = 0.f;
    for (int m = 0; m < 4; ++m) top = fmaxf(top, fabsf(v[m]));
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    const float s = __fdiv_rn(448.f, top), mult = top == 0.f ? 0.f : s;
    for (int m = 0; m < 4; ++m) {
      const int o = b * 128 + 32 * m + lane;
      if (o >= a.n) continue;
      if (a.ys)
        static_cast<uint8_t*>(a.out)[(size_t)r * a.n + o] =
            __nv_cvt_float_to_fp8(v[m] * mult, __NV_SATFINITE, __NV_E4M3);
      else
        put<T>(a.out, (size_t)r * a.n + o, v[m]);
      if (a.pre_out) {
        put<T>(a.pre_out, (size_t)r * a.N + o, g[m]);
        put<T>(a.pre_out, (size_t)r * a.N + a.n + o, u[m]);
      }
    }
    if (a.ys && lane == 0) a.ys[(size_t)r * a.nb + b] = __fdiv_rn(1.f, s);
  }
}

template <typename T>
__global__ void __launch_bounds__(256) dx_kernel(const __grid_constant__ B128Args a) {
  extern __shared__ int lists[];
  int *begin = lists, *tile = lists + a.G + 1;
  griddep_wait();
  const bool bad = group_scan<256>(a, begin, tile, [](int rows) { return rows; });
  if (bad && blockIdx.x == 0) atomicOr(&g_status, (uint32_t)CQ_ST_BAD_ROWS);
  const int lane = threadIdx.x & 31, blocks = a.N / a.n * a.nb;
  const int64_t total = (int64_t)tile[a.G] * a.kb;
  for (int64_t task = blockIdx.x * 8 + (threadIdx.x >> 5); task < total; task += gridDim.x * 8) {
    const int r = (int)(task / a.kb), b = (int)(task % a.kb);
    const int e = expert_of(tile, a.G, r), c0 = b * 128 + lane * 4;
    if (c0 >= a.K) continue;
    float d[4] = {};
    for (int nb = 0; nb < blocks; ++nb) {
      const int half = nb / a.nb, i0 = nb % a.nb * 128;
      const float s = a.xs[(size_t)r * blocks + nb] * a.ws[((size_t)e * blocks + nb) * a.kb + b];
      float p[4] = {};
      for (int i = i0; i < min(a.n, i0 + 128); ++i) {
        const size_t row = (size_t)half * a.n + i;
        const float y = value(static_cast<const uint8_t*>(a.x)[(size_t)r * a.N + row], a.x_dtype == kMxE5M2);
        const uint8_t* w = static_cast<const uint8_t*>(a.w) + ((size_t)e * a.N + row) * a.K + c0;
        for (int m = 0; m < 4; ++m) p[m] = fmaf(y, value(w[m], a.w_dtype == 1), p[m]);
      }
      for (int m = 0; m < 4; ++m) d[m] = fmaf(p[m], s, d[m]);
    }
    for (int m = 0; m < 4; ++m) {
      if (!a.pre_in) {
        put<T>(a.out, (size_t)r * a.K + c0 + m, d[m]);
        continue;
      }
      const size_t at = (size_t)r * 2 * a.K + c0 + m;
      float dg, du;
      swiglu_gradient(d[m], get<T>(a.pre_in, at), get<T>(a.pre_in, at + a.K), dg, du);
      put<T>(a.out, at, dg);
      put<T>(a.out, at + a.K, du);
    }
  }
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

int launch(bool dx, const B128Args& a, cudaStream_t s) {
  if (a.R == 0) return CQ_OK;
  const size_t smem = 8 * ((size_t)a.G + 1);
  const dim3 g(152 * 8), b(256);
  cudaError_t e;
  if (dx)
    e = a.out_dtype ? launch_pdl(dx_kernel<F16>, g, b, smem, s, a) : launch_pdl(dx_kernel<BF16>, g, b, smem, s, a);
  else
    e = a.out_dtype ? launch_pdl(forward_kernel<F16>, g, b, smem, s, a)
                    : launch_pdl(forward_kernel<BF16>, g, b, smem, s, a);
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
