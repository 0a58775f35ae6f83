// cq_norm.cu -- the norm before the layer with the residual's addition and the
// rows in fp8 or int8 (norm_kernel), and its gradient (grad_kernel, sum_kernel).
//
// Both read and write each value once, and that bounds them. norm_kernel: a block takes
// a row; a thread holds two units of 16 columns, as the permute kernels do, and
// quantises them with their code (cq_permute_impl.cuh), so that codes and scales follow
// dispatch's rules exactly. grad_kernel: persistent blocks, rows by bulk copies into a
// ring of shared memory, so that the next rows are on their way while two sums over a
// row wait at a barrier; a thread keeps one unit and its columns' share of dw.
//
// Measured on one GB300 (copy 6.78 TB/s), 16384 x 7168 bf16: residual, sum, y and fp8 rows
// 167 us, 6.4 TB/s; gradient with the residual's 162 us, 5.8 TB/s (408 us with a row read
// after the other).
#include "cq_expert.cuh"
#include "cq_permute_impl.cuh"

namespace cq {
namespace norm {
namespace {

using namespace permute_detail;

// grad_kernel's blocks: 8192 columns a SM, which holds up to 8 of them; each leaves a row
// of partial sums of dw.
constexpr int kSms = 152, kMaxStages = 8;
constexpr int kRing = 200 * 1024;  // bytes of a SM's rings

__device__ uint32_t g_status;  // CQ_ST_TIMEOUT of grad_kernel on this device

struct NormArgs {
  int32_t H, norm;
  float eps;
  const uint16_t* x;
  const uint16_t* residual;
  const uint16_t* weight;
  uint16_t* sum;
  uint16_t* y;
  uint8_t* codes;
  uint8_t* scales;
  int32_t scale_bytes;  // of a row of scales
};

struct GradArgs {
  int32_t R, H, stages;
  float eps;
  const uint16_t* dy;
  const uint16_t* x;
  const uint16_t* weight;
  const uint16_t* dsum;
  uint16_t* dx;
  float* part;  // [blocks][H], or NULL
};

// Sum of a float per thread over the block, the same bits in every thread: lanes by
// a butterfly, warps in order. `buf` holds 8 floats; not reused before a barrier.
__device__ __forceinline__ float block_sum(float v, float* buf, int nt) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < (nt >> 5); ++w) s += buf[w];
  return s;
}

// The power of two by which values are multiplied before they are squared, from the
// sum of their squares: 1, unless that sum left 32 bits or (where eps would not cover
// it) lost its digits below.
__device__ __forceinline__ float square_scale(float ss, float eps) {
  if (ss > 1e36f) return 0x1p-80f;
  if (ss < 1e-24f && eps < 1e-24f) return 0x1p80f;
  return 1.f;
}

template <class T>
__device__ __forceinline__ void unpack16(const uint4 (&u)[2], float (&f)[16]) {
  unit_values<T, kNoSmooth>(u, nullptr, 0.f, 0, f);
}

__device__ __forceinline__ void load_unit(const uint16_t* p, int unit, uint4 (&u)[2]) {
  const uint4* q = reinterpret_cast<const uint4*>(p) + 2 * unit;
  u[0] = q[0];
  u[1] = q[1];
}

template <class T>
__device__ __forceinline__ void store_unit(uint16_t* p, int unit, const float (&f)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int t = 0; t < 8; ++t) w[t] = T::pack2(f[2 * t], f[2 * t + 1]);
  uint4* q = reinterpret_cast<uint4*>(p) + 2 * unit;
  q[0] = make_uint4(w[0], w[1], w[2], w[3]);
  q[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

template <class T, int Q>
__global__ void __launch_bounds__(256) norm_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float red[64], sums[16];
  const int nt = blockDim.x;
  const size_t row = blockIdx.x, at = row * a.H;
  griddep_wait();
  Units U;
  float f[2][16];
  float ss = 0.f;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int u = threadIdx.x + q * nt;
    U.ok[q] = 16 * u < a.H;
#pragma unroll
    for (int t = 0; t < 16; ++t) f[q][t] = 0.f;
    if (!U.ok[q]) continue;
    load_unit(a.x + at, u, U.v[q]);
    unpack16<T>(U.v[q], f[q]);
    if (a.residual) {
      uint4 v[2];
      float r[16];
      load_unit(a.residual + at, u, v);
      unpack16<T>(v, r);
#pragma unroll
      for (int t = 0; t < 16; ++t) f[q][t] += r[t];
    }
    if (a.sum) store_unit<T>(a.sum + at, u, f[q]);
#pragma unroll
    for (int t = 0; t < 16; ++t) ss = fmaf(f[q][t], f[q][t], ss);
  }
  if (a.norm) {
    ss = block_sum(ss, sums, nt);
    const float m = square_scale(ss, a.eps);
    if (m != 1.f) {  // the same in every thread
      ss = 0.f;
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int t = 0; t < 16; ++t) f[q][t] *= m, ss = fmaf(f[q][t], f[q][t], ss);
      ss = block_sum(ss, sums + 8, nt);
    }
    const float r = 1.f / sqrtf(ss / a.H + a.eps * m * m);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int u = threadIdx.x + q * nt;
      if (!U.ok[q]) continue;
#pragma unroll
      for (int t = 0; t < 16; ++t) f[q][t] *= r;
      if (a.weight) {
        uint4 v[2];
        float w[16];
        load_unit(a.weight, u, v);
        unpack16<T>(v, w);
#pragma unroll
        for (int t = 0; t < 16; ++t) f[q][t] *= w[t];
      }
    }
  }
  if (a.y) {
#pragma unroll
    for (int q = 0; q < 2; ++q)
      if (U.ok[q]) store_unit<T>(a.y + at, threadIdx.x + q * nt, f[q]);
  }
  if (Q != 0) {
    uint8_t* scales = a.scales + row * a.scale_bytes;
    const float carried = quantise<Q, true>(f, U, a.codes + at, scales, red, nt);
    if (q_mode(Q) == 2 && threadIdx.x == 0) *reinterpret_cast<float*>(scales) = carried;
    if (q_mode(Q) >= 4 && threadIdx.x == 0 && a.H / 32 < a.scale_bytes) scales[a.H / 32] = 0;
  }
}

// dx, and each block's share of dw: rows blockIdx.x, + gridDim.x, ...
template <class T>
__global__ void __launch_bounds__(512) grad_kernel(const __grid_constant__ GradArgs a) {
  extern __shared__ __align__(128) uint8_t ring[];  // [stages][x, dy, dsum][H]
  __shared__ uint64_t full[kMaxStages];
  __shared__ float sums[3][2][16];
  const int nt = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool mine = 16 * threadIdx.x < a.H;
  const uint32_t line = 2 * a.H, entry = (a.dsum ? 3 : 2) * line;
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) mbar_init(&full[s], 1);
    mbar_fence_init();
  }
  __syncthreads();
  griddep_wait();
  auto load = [&](int64_t row, int s) {
    uint8_t* to = ring + s * entry;
    const size_t at = row * a.H;
    mbar_arrive_expect_tx(&full[s], entry);
    bulk_load(to, a.x + at, line, &full[s]);
    bulk_load(to + line, a.dy + at, line, &full[s]);
    if (a.dsum) bulk_load(to + 2 * line, a.dsum + at, line, &full[s]);
  };
  if (threadIdx.x == 0)
    for (int s = 0; s < a.stages && blockIdx.x + s * gridDim.x < a.R; ++s) load(blockIdx.x + s * gridDim.x, s);
  uint4 wv[2] = {};
  if (a.weight && mine) load_unit(a.weight, threadIdx.x, wv);
  float dw[16] = {};
  int s = 0, lap = 0, turn = 0;
  bool ok = true;
  for (int64_t row = blockIdx.x; row < a.R; row += gridDim.x) {  // (the last step may pass 2^31)
    ok = mbar_wait_warp(&full[s], lap & 1);
    uint4 xv[2] = {}, dv[2] = {}, sv[2] = {};
    if (ok && mine) {
      const uint8_t* from = ring + s * entry + 32 * threadIdx.x;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        xv[k] = ld_shared_v4(from + 16 * k);
        dv[k] = ld_shared_v4(from + line + 16 * k);
        if (a.dsum) sv[k] = ld_shared_v4(from + 2 * line + 16 * k);
      }
    }
    float x[16], d[16], w[16];
    unpack16<T>(xv, x);
    unpack16<T>(dv, d);
    if (a.weight) {
      unpack16<T>(wv, w);
    } else {
#pragma unroll
      for (int t = 0; t < 16; ++t) w[t] = 1.f;
    }
    // sums of (x m)^2 and dy w (x m) over the row, the same in every thread
    auto reduce = [&](float m, float& ss, float& sd, float (&buf)[2][16], bool& go) {
      ss = sd = 0.f;
#pragma unroll
      for (int t = 0; t < 16; ++t) {
        const float v = x[t] * m;
        ss = fmaf(v, v, ss);
        sd = fmaf(d[t] * w[t], v, sd);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        ss += __shfl_xor_sync(kFull, ss, o);
        sd += __shfl_xor_sync(kFull, sd, o);
      }
      if (lane == 0) buf[0][warp] = ss, buf[1][warp] = sd;
      go = __syncthreads_and(go);
      ss = sd = 0.f;
      for (int k = 0; k < (nt >> 5); ++k) ss += buf[0][k], sd += buf[1][k];
    };
    // this thread's reads of the row come before the copy that follows into its place
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    float ss, sd;
    reduce(1.f, ss, sd, sums[turn], ok);
    if (!ok) break;  // in every thread
    turn ^= 1;
    if (threadIdx.x == 0) {
      const int64_t next = row + (int64_t)a.stages * gridDim.x;
      if (next < a.R) load(next, s);
    }
    if (++s == a.stages) s = 0, ++lap;
    const float m = square_scale(ss, a.eps);
    if (m != 1.f) {
      bool all = true;
      __syncthreads();  // sums[2] of an earlier row is read
      reduce(m, ss, sd, sums[2], all);
    }
    // with xs = x m: x r = xs rs, and r^2 x mean(dy w x) = xs rs * (rs mean(dy w xs))
    const float rs = 1.f / sqrtf(ss / a.H + a.eps * m * m), r = m * rs, c = rs * (sd / a.H);
    float o[16], e[16];
    unpack16<T>(sv, e);
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      const float hat = x[t] * m * rs;
      dw[t] = fmaf(d[t], hat, dw[t]);
      o[t] = r * (d[t] * w[t] - hat * c) + e[t];
    }
    if (mine) store_unit<T>(a.dx + row * a.H, threadIdx.x, o);
  }
  if (!ok) {
    if (threadIdx.x == 0) {  // copies in flight land (with a limit) before the block goes
      atomicOr(&g_status, (uint32_t)CQ_ST_TIMEOUT);
      for (int k = 0; k < a.stages; ++k) mbar_wait(&full[(s + k) % a.stages], (lap + (s + k) / a.stages) & 1);
    }
    return;
  }
  if (a.part && mine) {
    float4* to = reinterpret_cast<float4*>(a.part + (size_t)blockIdx.x * a.H + 16 * threadIdx.x);
#pragma unroll
    for (int t = 0; t < 4; ++t) to[t] = make_float4(dw[4 * t], dw[4 * t + 1], dw[4 * t + 2], dw[4 * t + 3]);
  }
}

// dw[h] = the blocks' shares: 32 runs of them each in order, then the runs in order.
__global__ void __launch_bounds__(1024) sum_kernel(const float* part, float* dw, int parts, int H) {
  __shared__ float s[32][33];
  const int c = threadIdx.x & 31, g = threadIdx.x >> 5, h = blockIdx.x * 32 + c;
  griddep_wait();
  float v = 0.f;
  const int per = (parts + 31) / 32;
  if (h < H) {
#pragma unroll 8
    for (int p = g * per; p < min(parts, (g + 1) * per); ++p) v += part[(size_t)p * H + h];
  }
  s[g][c] = v;
  __syncthreads();
  if (g == 0 && h < H) {
    for (int k = 1; k < 32; ++k) v += s[k][c];
    dw[h] = v;
  }
}

int validate(const cq_norm_config* c) {
  if (!c || c->rows < 0 || c->hidden < 16 || c->hidden > 8192) return CQ_ERR_ARG;
  if (c->x_dtype != 0 && c->x_dtype != 1) return CQ_ERR_ARG;
  if (c->norm != 0 && c->norm != 1) return CQ_ERR_ARG;
  if (c->quant_mode != 0 && (c->quant_mode < 2 || c->quant_mode > 5)) return CQ_ERR_ARG;
  if (c->y_dtype < 0 || c->y_dtype > (c->quant_mode >= 3 ? 1 : 0)) return CQ_ERR_ARG;
  if (!(c->eps >= 0.f && c->eps <= 3.402823466e38f)) return CQ_ERR_ARG;
  if (c->hidden % (c->quant_mode >= 4 ? 32 : 16) != 0) return CQ_ERR_UNSUPPORTED;
  return CQ_OK;
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int threads_for(int H) { return (H / 16 + 63) / 64 * 32; }  // two units of 16 each

template <class T>
cudaError_t launch_norm(int q, const NormArgs& a, int rows, cudaStream_t s) {
  const dim3 g(rows), b(threads_for(a.H));
  switch (q) {
    case 0: return launch_pdl(norm_kernel<T, 0>, g, b, 0, s, a);
    case 2: return launch_pdl(norm_kernel<T, 2>, g, b, 0, s, a);
    case 3: return launch_pdl(norm_kernel<T, 3>, g, b, 0, s, a);
    case 4: return launch_pdl(norm_kernel<T, 4>, g, b, 0, s, a);
    case 5: return launch_pdl(norm_kernel<T, 5>, g, b, 0, s, a);
    case 13: return launch_pdl(norm_kernel<T, 13>, g, b, 0, s, a);
    case 14: return launch_pdl(norm_kernel<T, 14>, g, b, 0, s, a);
    default: return launch_pdl(norm_kernel<T, 15>, g, b, 0, s, a);
  }
}

// grad_kernel's blocks a SM, and in all.
int per_sm(const cq_norm_config* c) {
  const int n = 8192 / c->hidden;
  return n < 1 ? 1 : n > 8 ? 8 : n;
}
int parts_of(const cq_norm_config* c) {
  const int n = kSms * per_sm(c);
  return c->rows < n ? c->rows : n;
}

template <class T>
cudaError_t launch_grad(GradArgs a, int parts, int per, cudaStream_t s) {
  constexpr auto kernel = grad_kernel<T>;
  const int entry = (a.dsum ? 3 : 2) * 2 * a.H;
  a.stages = kRing / per / entry;
  if (a.stages > kMaxStages) a.stages = kMaxStages;
  const size_t smem = (size_t)a.stages * entry;
  const cudaError_t e = cq::prepare_kernel<kernel>(smem);
  if (e != cudaSuccess) return e;
  return cq::launch_pdl(kernel, dim3(parts), dim3((a.H / 16 + 31) / 32 * 32), smem, s, a);
}

}  // namespace
}  // namespace norm

namespace expert {
int norm_status(uint32_t* read, cudaStream_t s) { return status_word(norm::g_status, read, s); }
}  // namespace expert
}  // namespace cq

using namespace cq::norm;

extern "C" {

int cq_check_norm_config(const cq_norm_config* cfg) { return validate(cfg); }

size_t cq_norm_workspace_size(const cq_norm_config* cfg) {
  if (validate(cfg) != CQ_OK) return 0;
  return cq::align256(sizeof(float) * (size_t)parts_of(cfg) * cfg->hidden) + 256;
}

int cq_norm_quant(const cq_norm_config* cfg, const void* x, const void* residual,
                  const void* weight, void* sum, void* y, void* codes, void* scales, void* stream) {
  const int rc = validate(cfg);
  if (rc != CQ_OK) return rc;
  const bool rows = cfg->rows > 0;
  if ((!x && rows) || (weight && !cfg->norm)) return CQ_ERR_ARG;
  if (cfg->quant_mode == 0 ? (codes || scales || (!y && rows)) : (rows && (!codes || !scales)))
    return CQ_ERR_ARG;
  for (const void* p : {x, residual, weight, (const void*)sum, (const void*)y, (const void*)codes})
    if (!aligned(p, 16)) return CQ_ERR_ARG;
  if (cfg->quant_mode <= 3 && !aligned(scales, 4)) return CQ_ERR_ARG;
  if (!rows) return CQ_OK;
  NormArgs a = {};
  a.H = cfg->hidden;
  a.norm = cfg->norm;
  a.eps = cfg->eps;
  a.x = static_cast<const uint16_t*>(x);
  a.residual = static_cast<const uint16_t*>(residual);
  a.weight = static_cast<const uint16_t*>(weight);
  a.sum = static_cast<uint16_t*>(sum);
  a.y = static_cast<uint16_t*>(y);
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = static_cast<uint8_t*>(scales);
  a.scale_bytes = cfg->quant_mode == 2   ? 4
                  : cfg->quant_mode == 3 ? 4 * ((cfg->hidden + 127) / 128)
                                         : (cfg->hidden / 32 + 1) / 2 * 2;
  const int q = cfg->quant_mode + 10 * cfg->y_dtype;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = cfg->x_dtype == 1 ? launch_norm<cq::F16>(q, a, cfg->rows, s)
                                          : launch_norm<cq::BF16>(q, a, cfg->rows, s);
  return e == cudaSuccess ? CQ_OK : CQ_ERR_CUDA;
}

int cq_norm_grad(const cq_norm_config* cfg, const void* dy, const void* x, const void* weight,
                 const void* dsum, void* dx, float* dw, void* workspace, size_t workspace_bytes,
                 void* stream) {
  const int rc = validate(cfg);
  if (rc != CQ_OK) return rc;
  const bool rows = cfg->rows > 0;
  if (!cfg->norm || (rows && (!dy || !x || !dx))) return CQ_ERR_ARG;
  for (const void* p : {dy, x, weight, dsum, (const void*)dx})
    if (!aligned(p, 16)) return CQ_ERR_ARG;
  if (!aligned(dw, 4)) return CQ_ERR_ARG;
  if (dw && rows &&
      (!workspace || !aligned(workspace, 256) || workspace_bytes < cq_norm_workspace_size(cfg)))
    return CQ_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!rows) {
    if (!dw) return CQ_OK;
    return cudaMemsetAsync(dw, 0, sizeof(float) * cfg->hidden, s) == cudaSuccess ? CQ_OK : CQ_ERR_CUDA;
  }
  GradArgs a = {};
  a.R = cfg->rows;
  a.H = cfg->hidden;
  a.eps = cfg->eps;
  a.dy = static_cast<const uint16_t*>(dy);
  a.x = static_cast<const uint16_t*>(x);
  a.weight = static_cast<const uint16_t*>(weight);
  a.dsum = static_cast<const uint16_t*>(dsum);
  a.dx = static_cast<uint16_t*>(dx);
  a.part = dw ? static_cast<float*>(workspace) : nullptr;
  const int parts = parts_of(cfg), per = per_sm(cfg);
  cudaError_t e = cfg->x_dtype == 1 ? launch_grad<cq::F16>(a, parts, per, s) : launch_grad<cq::BF16>(a, parts, per, s);
  if (e == cudaSuccess && dw)
    e = cq::launch_pdl(sum_kernel, dim3((a.H + 31) / 32), dim3(1024), 0, s, a.part, dw, parts, a.H);
  return e == cudaSuccess ? CQ_OK : CQ_ERR_CUDA;
}

}  // extern "C"
