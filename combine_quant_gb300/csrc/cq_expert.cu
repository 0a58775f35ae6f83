// cq_expert.cu -- entry points of the expert products (see include/cq.h for the
// contract). Every argument rule is checked before anything is enqueued; the
// kernels are in cq_expert_gemm.cu (tensor cores) and cq_expert_w4.cu (4-bit
// weights).
#include "cq_expert.cuh"
#include "cq_status.h"

namespace cq {
namespace expert {
namespace {

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

// Page-locked words of this thread for the status copies: copies to other memory wait each
// by itself (five words: 54 us a call of cq_read_expert_status from Python, 21 with one wait).
constexpr int kStatusWords = 5;
uint32_t* host_words() {
  struct Words {
    uint32_t* p = nullptr;
    ~Words() {  // a thread may end while another one captures a graph, which this must not end
      cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
      if (p && cudaThreadExchangeStreamCaptureMode(&mode) == cudaSuccess) cudaFreeHost(p);
    }
  };
  static thread_local Words words;
  if (!words.p && cudaHostAlloc(reinterpret_cast<void**>(&words.p), 4 * kStatusWords, cudaHostAllocPortable) != cudaSuccess) {
    cudaGetLastError();
    words.p = nullptr;
  }
  return words.p;
}

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
  return launch_gemm(kForward, a, static_cast<cudaStream_t>(stream));
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
  constexpr int (*kWords[])(uint32_t*, cudaStream_t) = {gemm_status, w4_status, b128_status, layer_status, norm_status};
  static_assert(sizeof kWords / sizeof *kWords == kStatusWords);
  uint32_t* host = host_words();
  if (!host) return CQ_ERR_CUDA;
  return cq::collect_status(
      kStatusWords, host, [&](int i, uint32_t* read) { return kWords[i](read, s); },
      [&] { return cudaStreamSynchronize(s) == cudaSuccess ? CQ_OK : CQ_ERR_CUDA; },
      [&](int i) { return kWords[i](nullptr, s); }, status);
}

}  // extern "C"
