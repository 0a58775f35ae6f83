// cq_moe_layer.cu -- the whole layer for a few tokens: gate and up products with
// SwiGLU (up_kernel), down product with the weighted sum (down_kernel).
//
// The simplest form: a warp a result.
#include <cuda_fp8.h>

#include "cq_expert.cuh"

namespace cq {
namespace expert {
namespace {

__device__ uint32_t g_status;  // CQ_ST_* bits of these kernels on this device

struct LayerArgs {
  int32_t T, G, K, H, I, mask_ndim, out_f32;
  const uint16_t* x;
  const int32_t* ids;
  const float* scales;
  const uint8_t* mask;
  const void* w13;
  const float* w13_scales;
  const void* w2;
  const float* w2_scales;
  float* h;  // [T * K, I]
  void* y;
};

__device__ __forceinline__ int expert_of_pair(const LayerArgs& a, int p) {
  if (a.mask_ndim && !a.mask[a.mask_ndim == 1 ? p / a.K : p]) return -1;
  const int e = a.ids[p];
  if ((unsigned)e < (unsigned)a.G) return e;
  atomicOr(&g_status, (uint32_t)CQ_ST_BAD_ID);
  return -1;
}

template <typename T, bool FP8>
__device__ __forceinline__ float weight_at(const void* w, size_t at) {
  if (FP8) return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(w)[at], __NV_E4M3)));
  return T::lo(static_cast<const uint16_t*>(w)[at]);
}

__device__ __forceinline__ float warp_sum(float v) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

template <typename T, bool FP8>
__global__ void __launch_bounds__(256) up_kernel(const __grid_constant__ LayerArgs a) {
  griddep_wait();
  const int lane = threadIdx.x & 31, hb = (a.H + 127) / 128, ib = (a.I + 127) / 128;
  const int total = a.T * a.K * a.I;
  for (int task = blockIdx.x * 8 + (threadIdx.x >> 5); task < total; task += gridDim.x * 8) {
    const int p = task / a.I, i = task % a.I, e = expert_of_pair(a, p);
    if (e < 0) continue;
    float v[2];
    for (int half = 0; half < 2; ++half) {
      float sum = 0.f;
      for (int j = lane; j < a.H; j += 32) {
        float w = weight_at<T, FP8>(a.w13, ((size_t)e * 2 * a.I + half * a.I + i) * a.H + j);
        if (FP8) w *= a.w13_scales[((size_t)e * 2 * ib + half * ib + i / 128) * hb + j / 128];
        sum = fmaf(w, T::lo(a.x[(size_t)(p / a.K) * a.H + j]), sum);
      }
      v[half] = warp_sum(sum);
    }
    if (lane == 0) a.h[(size_t)p * a.I + i] = swiglu(v[0], v[1]);
  }
}

template <typename T, bool FP8>
__global__ void __launch_bounds__(256) down_kernel(const __grid_constant__ LayerArgs a) {
  griddep_wait();
  const int lane = threadIdx.x & 31, hb = (a.H + 127) / 128, ib = (a.I + 127) / 128;
  const int total = a.T * a.H;
  for (int task = blockIdx.x * 8 + (threadIdx.x >> 5); task < total; task += gridDim.x * 8) {
    const int t = task / a.H, o = task % a.H;
    float y = 0.f;
    for (int k = 0; k < a.K; ++k) {
      const int p = t * a.K + k, e = expert_of_pair(a, p);
      if (e < 0) continue;
      float sum = 0.f;
      for (int j = lane; j < a.I; j += 32) {
        float w = weight_at<T, FP8>(a.w2, ((size_t)e * a.H + o) * a.I + j);
        if (FP8) w *= a.w2_scales[((size_t)e * hb + o / 128) * ib + j / 128];
        sum = fmaf(w, a.h[(size_t)p * a.I + j], sum);
      }
      y = fmaf(a.scales[p], warp_sum(sum), y);
    }
    if (lane != 0) continue;
    if (a.out_f32) static_cast<float*>(a.y)[task] = y;
    else static_cast<uint16_t*>(a.y)[task] = (uint16_t)T::pack2(y, 0.f);
  }
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

template <typename T, bool FP8>
cudaError_t launch(const LayerArgs& a, cudaStream_t s) {
  const dim3 g(152 * 8), b(256);
  const cudaError_t e = launch_pdl(up_kernel<T, FP8>, g, b, 0, s, a);
  return e == cudaSuccess ? launch_pdl(down_kernel<T, FP8>, g, b, 0, s, a) : e;
}

}  // namespace

int layer_status(uint32_t* status, cudaStream_t s) { return read_status_word(g_status, status, s); }

}  // namespace expert
}  // namespace cq

using namespace cq::expert;

extern "C" {

int cq_check_moe_config(const cq_moe_config* cfg) { return validate(cfg); }

size_t cq_moe_workspace_size(const cq_moe_config* cfg) {
  if (validate(cfg) != CQ_OK) return 0;
  return cq::align256(4 * (size_t)cfg->tokens * cfg->topk * cfg->inter) + 256;
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
  a.w13 = w13;
  a.w13_scales = w13_scales;
  a.w2 = w2;
  a.w2_scales = w2_scales;
  a.h = static_cast<float*>(workspace);
  a.y = y;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = cfg->x_dtype == 1
                            ? (cfg->w_dtype ? launch<cq::F16, true>(a, s) : launch<cq::F16, false>(a, s))
                            : (cfg->w_dtype ? launch<cq::BF16, true>(a, s) : launch<cq::BF16, false>(a, s));
  return e == cudaSuccess ? CQ_OK : CQ_ERR_CUDA;
}

}  // extern "C"
