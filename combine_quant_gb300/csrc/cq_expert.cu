// cq_expert.cu -- entry points of the expert products (see include/cq.h) and
// their kernels: matrix products grouped by expert, forward and backward, and
// the form for 4-bit weights.
#include <cuda_fp8.h>

#include "cq_expert.cuh"

namespace cq {
namespace expert {
namespace {

__device__ uint32_t g_status;  // CQ_ST_* bits of the expert products on this device

template <int T>
__device__ __forceinline__ float load16(const void* p, size_t i) {
  const uint16_t v = static_cast<const uint16_t*>(p)[i];
  return T == kF16 ? F16::lo(v) : BF16::lo(v);
}

__device__ __forceinline__ float load_fp8(const void* p, size_t i, bool e5m2) {
  const __nv_fp8_storage_t b = static_cast<const uint8_t*>(p)[i];
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(b, e5m2 ? __NV_E5M2 : __NV_E4M3)));
}

// 2^(s - 127), s = 255 is NaN.
__device__ __forceinline__ float e8m0(uint8_t s) {
  return s == 255 ? __int_as_float(0x7fffffff)
         : s == 0 ? __int_as_float(0x00400000)
                  : __int_as_float((int)s << 23);
}

// A 64 x 64 tile of out[j, i] (i contiguous) = sum_k A(k, i) B(k, j), the
// operands gathered element by element into shared memory.
template <Op OP, int T>
__global__ void __launch_bounds__(256) simple_kernel(const Args a) {
  __shared__ float sa[2][16][65], sb[16][65];
  __shared__ int64_t s_sum[256];
  __shared__ int s_begin, s_count;
  const int e = blockIdx.y;
  int64_t sum = 0;
  bool bad = false;
  for (int t = threadIdx.x; t < e; t += 256) {
    const int64_t c = group_count(a.group_rows, t, a.rows_type, a.L);
    sum += c < 0 ? 0 : c < a.R ? c : a.R;
  }
  s_sum[threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = 0;
    for (int t = 0; t < 256; ++t) sum += s_sum[t];
    int64_t c = group_count(a.group_rows, e, a.rows_type, a.L);
    if (c < 0) bad = true, c = 0;
    if (sum > a.R) sum = a.R;
    if (c > a.R - sum) bad = true, c = a.R - sum;
    s_begin = (int)sum;
    s_count = (int)c;
    if (bad && blockIdx.x == 0) atomicOr(&g_status, (uint32_t)CQ_ST_BAD_ROWS);
  }
  __syncthreads();
  const int begin = s_begin, count = s_count;
  const int n_out = a.act ? a.N / 2 : a.N;
  const int I = OP == kForward || OP == kW4 ? n_out : a.K;       // out columns
  const int J = OP == kDw ? a.N : count;                         // out rows
  const int KK = OP == kDw ? count : OP == kDx ? a.N : a.K;      // contraction
  const bool two = a.act && (OP == kForward || OP == kW4);
  const int i0 = blockIdx.x * 64;
  const int ti = threadIdx.x % 16, tj = threadIdx.x / 16;
  auto wval = [&](int kk, int i) -> float {  // A operand
    if (OP == kDx) return load16<T>(a.w, ((size_t)e * a.N + kk) * a.K + i);
    if (OP == kDw) return load16<T>(a.x, (size_t)(begin + kk) * a.K + i);
    const size_t row = (size_t)e * a.N + i;
    if (OP == kW4) {
      const uint8_t b = static_cast<const uint8_t*>(a.w)[row * (a.K / 2) + kk / 2];
      const size_t g = row * (a.K / a.group) + kk / a.group;
      const float z = a.zeros4 ? (float)a.zeros4[g] : 8.f;
      return ((float)(kk & 1 ? b >> 4 : b & 15) - z) * load16<T>(a.scales4, g);
    }
    if (T >= kMxE4M3)
      return load_fp8(a.w, row * a.K + kk, a.w_dtype == 1) * e8m0(a.w_scales[row * a.SC + kk / 32]);
    return load16<T>(a.w, row * a.K + kk);
  };
  auto xval = [&](int kk, int j) -> float {  // B operand
    if (OP == kDw) return load16<T>(a.w, (size_t)(begin + kk) * a.N + j);
    const size_t row = (size_t)(begin + j);
    if (OP == kDx) return load16<T>(a.x, row * a.N + kk);
    if (T >= kMxE4M3)
      return load_fp8(a.x, row * a.K + kk, T == kMxE5M2) * e8m0(a.x_scales[row * a.SC + kk / 32]);
    return load16<T>(a.x, row * a.K + kk);
  };
  auto store = [&](void* p, size_t at, float v) {
    if (a.out_dtype == 2) static_cast<float*>(p)[at] = v;
    else if (a.out_dtype == 1) static_cast<__half*>(p)[at] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(p)[at] = __float2bfloat16_rn(v);
  };
  for (int j0 = blockIdx.z * 64; j0 < J; j0 += 64 * gridDim.z) {
    float acc[2][4][4] = {};
    for (int k0 = 0; k0 < KK; k0 += 16) {
      for (int t = threadIdx.x; t < 1024; t += 256) {
        const int kk = OP == kDx || OP == kDw ? t / 64 : t % 16, i = OP == kDx || OP == kDw ? t % 64 : t / 16;
        const bool in = k0 + kk < KK;
        sa[0][kk][i] = in && i0 + i < I ? wval(k0 + kk, i0 + i) : 0.f;
        if (two) sa[1][kk][i] = in && i0 + i < I ? wval(k0 + kk, I + i0 + i) : 0.f;
        const int kb = OP == kDw ? t / 64 : t % 16, j = OP == kDw ? t % 64 : t / 16;
        sb[kb][j] = k0 + kb < KK && j0 + j < J ? xval(k0 + kb, j0 + j) : 0.f;
      }
      __syncthreads();
      for (int kk = 0; kk < 16; ++kk)
        for (int p = 0; p < 4; ++p)
          for (int q = 0; q < 4; ++q) {
            acc[0][p][q] = fmaf(sa[0][kk][ti + 16 * p], sb[kk][tj + 16 * q], acc[0][p][q]);
            if (two) acc[1][p][q] = fmaf(sa[1][kk][ti + 16 * p], sb[kk][tj + 16 * q], acc[1][p][q]);
          }
      __syncthreads();
    }
    for (int p = 0; p < 4; ++p)
      for (int q = 0; q < 4; ++q) {
        const int i = i0 + ti + 16 * p, j = j0 + tj + 16 * q;
        if (i >= I || j >= J) continue;
        float v = acc[0][p][q];
        const size_t row = OP == kDw ? (size_t)e * a.N + j : (size_t)(begin + j);
        if (two) {
          const float u = acc[1][p][q];
          if (a.pre_out) {
            store(a.pre_out, row * a.N + i, v);
            store(a.pre_out, row * a.N + I + i, u);
          }
          v = u * v / (1.f + expf(-v));
        }
        if (OP == kDx && a.pre_in) {
          const float g = load16<T>(a.pre_in, row * 2 * I + i), u = load16<T>(a.pre_in, row * 2 * I + I + i);
          const float s = 1.f / (1.f + expf(-g));
          store(a.out, row * 2 * I + i, v * u * (s + g * s * (1.f - s)));
          store(a.out, row * 2 * I + I + i, v * g * s);
        } else {
          store(a.out, row * I + i, v);
        }
      }
  }
}

template <Op OP>
int launch(const Args& a, cudaStream_t s) {
  if (a.R == 0 && OP != kDw) return CQ_OK;
  const int I = OP == kForward || OP == kW4 ? (a.act ? a.N / 2 : a.N) : a.K;
  const int J = OP == kDw ? a.N : (a.R + a.G - 1) / a.G;
  const dim3 grid((I + 63) / 64, a.G, (J + 63) / 64 < 64 ? (J + 63) / 64 : 64);
  switch (a.x_dtype) {
    case kBF16: simple_kernel<OP, kBF16><<<grid, 256, 0, s>>>(a); break;
    case kF16: simple_kernel<OP, kF16><<<grid, 256, 0, s>>>(a); break;
    case kMxE4M3:
      if constexpr (OP == kForward) simple_kernel<OP, kMxE4M3><<<grid, 256, 0, s>>>(a);
      break;
    default:
      if constexpr (OP == kForward) simple_kernel<OP, kMxE5M2><<<grid, 256, 0, s>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? CQ_OK : CQ_ERR_CUDA;
}

int validate(const cq_expert_config* c) {
  if (!c) return CQ_ERR_ARG;
  if (c->experts < 1 || c->experts > 2048 || c->rows < 0) return CQ_ERR_ARG;
  if (c->n < 16 || c->n > 65536 || c->k < 16 || c->k > 65536) return CQ_ERR_ARG;
  if (c->x_dtype < 0 || c->x_dtype > 3 || c->act < 0 || c->act > 1) return CQ_ERR_ARG;
  const bool mx = c->x_dtype >= kMxE4M3;
  if (c->w_dtype < 0 || c->w_dtype > (mx ? 1 : 0)) return CQ_ERR_ARG;
  if (c->out_dtype < -1 || c->out_dtype > 2) return CQ_ERR_ARG;
  if (!mx && (c->out_dtype == 0 || c->out_dtype == 1) && c->out_dtype != c->x_dtype)
    return CQ_ERR_ARG;
  if (c->rows_type != 0 && c->rows_type != 1) return CQ_ERR_ARG;
  if (c->rows_type == 0 && c->experts_per_rank < 1) return CQ_ERR_ARG;
  if (c->n % 16 != 0 || c->k % (mx ? 32 : 16) != 0) return CQ_ERR_UNSUPPORTED;
  return CQ_OK;
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// A required pointer of the row tensors: aligned, and not NULL unless there are no rows.
bool row_ptr(const cq_expert_config* c, const void* p) {
  return (p || c->rows == 0) && aligned(p, 16);
}
bool ptr(const void* p) { return p && aligned(p, 16); }

Args base_args(const cq_expert_config* c, const int64_t* group_rows) {
  Args a = {};
  a.G = c->experts;
  a.R = c->rows;
  a.N = c->act ? 2 * c->n : c->n;
  a.K = c->k;
  a.x_dtype = c->x_dtype;
  a.w_dtype = c->w_dtype;
  a.out_dtype = c->out_dtype >= 0 ? c->out_dtype : c->x_dtype == kF16 ? 1 : 0;
  a.act = c->act;
  a.group = c->group;
  a.rows_type = c->rows_type;
  a.L = c->experts_per_rank;
  a.SC = (c->k / 32 + 1) / 2 * 2;
  a.group_rows = group_rows;
  return a;
}

}  // namespace
}  // namespace expert
}  // namespace cq

using namespace cq::expert;

extern "C" {

int cq_check_expert_config(const cq_expert_config* cfg) { return validate(cfg); }

int cq_expert_matmul(const cq_expert_config* cfg, const void* x, const uint8_t* x_scales,
                     const void* w, const uint8_t* w_scales, const int64_t* group_rows, void* y,
                     void* pre, void* stream) {
  const int rc = validate(cfg);
  if (rc != CQ_OK) return rc;
  if (cfg->out_dtype == 2) return CQ_ERR_ARG;
  if (!row_ptr(cfg, x) || !ptr(w) || !row_ptr(cfg, y) || !group_rows || !aligned(group_rows, 8))
    return CQ_ERR_ARG;
  if (!aligned(pre, 16) || (pre && cfg->act != 1)) return CQ_ERR_ARG;
  if (cfg->x_dtype >= kMxE4M3) {
    if (!row_ptr(cfg, x_scales) || !ptr(w_scales)) return CQ_ERR_ARG;
  } else if (x_scales || w_scales) {
    return CQ_ERR_ARG;
  }
  Args a = base_args(cfg, group_rows);
  a.x = x;
  a.w = w;
  a.x_scales = x_scales;
  a.w_scales = w_scales;
  a.out = y;
  a.pre_out = pre;
  if (cfg->x_dtype <= kF16) return launch_gemm(kForward, a, static_cast<cudaStream_t>(stream));
  return launch<kForward>(a, static_cast<cudaStream_t>(stream));
}

int cq_expert_matmul_dx(const cq_expert_config* cfg, const void* dy, const void* w,
                        const int64_t* group_rows, const void* pre, void* dx, void* stream) {
  const int rc = validate(cfg);
  if (rc != CQ_OK) return rc;
  if (cfg->x_dtype > kF16 || cfg->out_dtype == 2) return CQ_ERR_ARG;
  if (!row_ptr(cfg, dy) || !ptr(w) || !row_ptr(cfg, dx) || !aligned(pre, 16) || !group_rows ||
      !aligned(group_rows, 8))
    return CQ_ERR_ARG;
  Args a = base_args(cfg, group_rows);
  a.act = 0;
  a.x = dy;
  a.w = w;
  a.pre_in = pre;
  a.out = dx;
  return launch_gemm(kDx, a, static_cast<cudaStream_t>(stream));
}

int cq_expert_matmul_dw(const cq_expert_config* cfg, const void* dy, const void* x,
                        const int64_t* group_rows, void* dw, void* stream) {
  const int rc = validate(cfg);
  if (rc != CQ_OK) return rc;
  if (cfg->x_dtype > kF16) return CQ_ERR_ARG;
  if (!row_ptr(cfg, dy) || !row_ptr(cfg, x) || !ptr(dw) || !group_rows || !aligned(group_rows, 8))
    return CQ_ERR_ARG;
  Args a = base_args(cfg, group_rows);
  a.act = 0;
  a.x = x;
  a.w = dy;
  a.out = dw;
  return launch_gemm(kDw, a, static_cast<cudaStream_t>(stream));
}

int cq_expert_matmul_w4(const cq_expert_config* cfg, const void* x, const uint8_t* codes,
                        const void* scales, const uint8_t* zeros, const int64_t* group_rows,
                        void* y, void* stream) {
  const int rc = validate(cfg);
  if (rc != CQ_OK) return rc;
  if (cfg->x_dtype > kF16 || cfg->out_dtype == 2) return CQ_ERR_ARG;
  if (cfg->group != 32 && cfg->group != 64 && cfg->group != 128) return CQ_ERR_ARG;
  if (cfg->k % 32 != 0) return CQ_ERR_UNSUPPORTED;
  if (cfg->k % cfg->group != 0) return CQ_ERR_ARG;
  if (!row_ptr(cfg, x) || !ptr(codes) || !ptr(scales) || !aligned(zeros, 16) || !row_ptr(cfg, y) ||
      !group_rows || !aligned(group_rows, 8))
    return CQ_ERR_ARG;
  Args a = base_args(cfg, group_rows);
  a.x = x;
  a.w = codes;
  a.scales4 = scales;
  a.zeros4 = zeros;
  a.out = y;
  return launch_w4(a, static_cast<cudaStream_t>(stream));
}

int cq_read_expert_status(uint32_t* status, void* stream) {
  if (!status) return CQ_ERR_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t v[3] = {};
  int rc = read_status_word(g_status, &v[0], s);
  if (rc == CQ_OK) rc = gemm_status(&v[1], s);
  if (rc == CQ_OK) rc = w4_status(&v[2], s);
  if (rc == CQ_OK) *status = v[0] | v[1] | v[2];
  return rc;
}

}  // extern "C"
