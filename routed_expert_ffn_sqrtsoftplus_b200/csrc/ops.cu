// Entry points of the operators that need no handle: routing from logits and its gradient, and
// the microscaled FP4 quantisers and product. Arguments are checked before anything is enqueued.
#include <atomic>
#include <cmath>
#include <initializer_list>

#include "../../include/moe.h"
#include "common.cuh"
#include "kernels.h"

using namespace moe;

namespace {

std::atomic<uint64_t> wait_ns{2000000000ull};  // limit of every device-side wait

cudaStream_t as_stream(moe_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Values that the quantisers take in one call (they count runs in 32 bits).
constexpr int64_t kMaxQuantized = int64_t(1) << 33;

int value_bytes(int32_t dtype) {
  return dtype == MOE_VAL_FP32 ? 4 : dtype == MOE_VAL_BF16 || dtype == MOE_VAL_FP16 ? 2 : 0;
}

// MOE_OK when every given pointer is memory of the current device.
moe_status on_device(std::initializer_list<const void*> ptrs) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  for (const void* p : ptrs)
    if (p != nullptr && !device_pointer_on(p, dev)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status launched(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  cudaGetLastError();
  return MOE_ERR_CUDA;
}

moe_status check_route(const moe_route_config* c) {
  if (c == nullptr) return MOE_ERR_INVALID_ARG;
  if (c->score < MOE_SCORE_SOFTMAX || c->score > MOE_SCORE_SQRTSOFTPLUS) return MOE_ERR_INVALID_ARG;
  if (!(c->route_scale > 0.f) || !std::isfinite(c->route_scale)) return MOE_ERR_INVALID_ARG;
  if (c->n_experts < 1 || c->top_k < 1 || c->n_groups < 1 || c->topk_groups < 1) return MOE_ERR_INVALID_ARG;
  if (c->topk_groups > c->n_groups || c->n_experts % c->n_groups != 0) return MOE_ERR_INVALID_ARG;
  if (c->top_k > c->topk_groups * (c->n_experts / c->n_groups)) return MOE_ERR_INVALID_ARG;
  if (c->n_experts > 512 || c->top_k > 32 || c->n_groups > 32) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

bool fp4_format_ok(int32_t f) { return f == MOE_FP4_MX || f == MOE_FP4_NV; }
bool product_shape_ok(int32_t T, int32_t N, int32_t K, int32_t E) {
  return T >= 0 && N >= 1 && K >= 1 && E >= 1 && T <= 1 << 22 && N <= 1 << 18 && K <= 1 << 18 && E <= 512;
}
// Alignment of scale rows that are read as they are (by a product without a workspace).
int scale_unit(int32_t format) { return format == MOE_FP4_NV ? 16 : 8; }
// Bytes of a row of quantised scales in moe_fp4_linear's workspace.
int64_t padded_scales(int32_t format, int32_t K) { return (K / (format == MOE_FP4_NV ? 16 : 32) + 15) / 16 * 16; }

// What moe_fp4_matmul and moe_fp4_linear check alike.
moe_status check_product(const moe_fp4_product& p) {
  if (!fp4_format_ok(p.format) || p.T < 0 || p.N < 1 || p.K < 1 || p.E < 1 || p.K % 32 != 0 ||
      value_bytes(p.out_dtype) == 0)
    return MOE_ERR_INVALID_ARG;
  if (p.offsets == nullptr && p.E != 1) return MOE_ERR_INVALID_ARG;
  if (p.w_scale_stride < p.K / (p.format == MOE_FP4_NV ? 16 : 32)) return MOE_ERR_INVALID_ARG;
  if (p.format == MOE_FP4_MX && (p.x_tensor_scale != nullptr || p.w_tensor_scale != nullptr))
    return MOE_ERR_INVALID_ARG;
  if (!product_shape_ok(p.T, p.N, p.K, p.E)) return MOE_ERR_UNSUPPORTED;
  if (p.T == 0) return MOE_OK;
  if (p.w == nullptr || p.w_scales == nullptr || p.y == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned(p.w, 16) || !aligned(p.y, value_bytes(p.out_dtype)) || !aligned(p.offsets, 4) ||
      !aligned(p.x_tensor_scale, 4) || !aligned(p.w_tensor_scale, 4) || !aligned(p.status, 4) ||
      !aligned(p.workspace, 16))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// The shape of its tiles, and its workspace.
struct Planned {
  Fp4Plan plan;
  int64_t bytes;
};
Planned plan_product(int32_t format, int32_t T, int32_t N, int32_t K, int32_t E) {
  const int num_kb = (K + 255) / 256;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    cudaGetLastError();
  if (sms < 1) sms = 148;  // no device: what a B200 would need
  const Fp4Plan plan = fp4_plan(T, N, E, num_kb, sms);
  return Planned{plan, fp4_workspace(format, T, N, E, num_kb, plan)};
}
// Where the scales are read as they are, their rows are aligned.
bool scales_ok(const moe_fp4_product& p, const Planned& planned) {
  const int unit = scale_unit(p.format);
  return planned.bytes > 0 || (p.w_scale_stride % unit == 0 && aligned(p.w_scales, unit) &&
                               p.x_scale_stride % unit == 0 && aligned(p.x_scales, unit));
}

// Bytes of w's scales in rows that a product without a workspace can read.
int64_t padded_w(int32_t format, int32_t N, int32_t K, int32_t E) {
  return padded_scales(format, K) * N * E;
}

// The launches of a checked product.
moe_status run_product(const moe_fp4_product& p, const Fp4Plan& plan, cudaStream_t stream) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return launched(cudaErrorInvalidDevice);
  Fp4GemmArgs a{};
  a.xs = p.x_scales;
  a.ws = p.w_scales;
  a.xs_stride = p.x_scale_stride;
  a.ws_stride = p.w_scale_stride;
  a.sf_cols = p.K / (p.format == MOE_FP4_NV ? 16 : 32);
  a.x_ts = p.x_tensor_scale;
  a.w_ts = p.w_tensor_scale;
  a.offsets = p.offsets;
  a.T = p.T;
  a.N = p.N;
  a.E = p.E;
  a.num_kb = (p.K + 255) / 256;
  a.out = p.y;
  a.out_dtype = p.out_dtype;
  a.status = p.status;
  a.timeout_ns = wait_ns.load(std::memory_order_relaxed);
  a.splits = plan.splits;
  a.m_tiles = (p.N + plan.cols - 1) / plan.cols;
  CUtensorMap tw, tx;
  if (!encode_tmap_bytes(&tw, p.w, static_cast<uint64_t>(p.E) * p.N, p.K / 2, plan.cols) ||
      !encode_tmap_bytes(&tx, p.x, p.T, p.K / 2, 32))
    return MOE_ERR_CUDA;
  return launched(launch_gemm_fp4(p.format, tw, tx, a, p.workspace, plan, sms, stream));
}

}  // namespace

extern "C" {

moe_status moe_route(const moe_route_config* cfg, const void* logits, int32_t dtype, int64_t row_stride,
                     const float* bias, int32_t T, int32_t* topk_idx, float* topk_w, moe_stream_t stream) {
  moe_status st = check_route(cfg);
  if (st != MOE_OK) return st;
  const int vb = value_bytes(dtype);
  if (vb == 0 || T < 0 || row_stride < cfg->n_experts) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (logits == nullptr || topk_idx == nullptr || topk_w == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned(logits, vb) || !aligned(bias, 4) || !aligned(topk_idx, 4) || !aligned(topk_w, 4))
    return MOE_ERR_INVALID_ARG;
  if ((st = on_device({logits, bias, topk_idx, topk_w})) != MOE_OK) return st;
  RouteArgs r{};
  r.logits = logits;
  r.dtype = dtype;
  r.row_stride = row_stride;
  r.bias = bias;
  r.T = T;
  r.E = cfg->n_experts;
  r.k = cfg->top_k;
  r.n_groups = cfg->n_groups;
  r.topk_groups = cfg->topk_groups;
  r.score = cfg->score;
  r.group_sum2 = cfg->group_top2 != 0;
  r.renorm = cfg->renormalize != 0;
  r.scale = cfg->route_scale;
  r.idx = topk_idx;
  r.w = topk_w;
  return launched(launch_route(r, as_stream(stream)));
}

moe_status moe_route_backward(const moe_route_config* cfg, const float* grad_w, const void* logits, int32_t dtype,
                              int64_t row_stride, const int32_t* topk_idx, int32_t T, void* grad_logits,
                              moe_stream_t stream) {
  moe_status st = check_route(cfg);
  if (st != MOE_OK) return st;
  const int vb = value_bytes(dtype);
  if (vb == 0 || T < 0 || row_stride < cfg->n_experts) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (grad_w == nullptr || logits == nullptr || topk_idx == nullptr || grad_logits == nullptr || grad_logits == logits)
    return MOE_ERR_INVALID_ARG;
  if (!aligned(logits, vb) || !aligned(grad_logits, vb) || !aligned(topk_idx, 4) || !aligned(grad_w, 4))
    return MOE_ERR_INVALID_ARG;
  if ((st = on_device({grad_w, logits, topk_idx, grad_logits})) != MOE_OK) return st;
  RouteGradArgs r{};
  r.grad_w = grad_w;
  r.logits = logits;
  r.dtype = dtype;
  r.row_stride = row_stride;
  r.idx = topk_idx;
  r.T = T;
  r.E = cfg->n_experts;
  r.k = cfg->top_k;
  r.score = cfg->score;
  r.renorm = cfg->renormalize != 0;
  r.scale = cfg->route_scale;
  r.out = grad_logits;
  return launched(launch_route_grad(r, as_stream(stream)));
}

moe_status moe_quantize_fp4(int32_t format, const void* src, int32_t dtype, int64_t rows, int32_t cols,
                            int64_t row_stride, const float* tensor_scale, uint8_t* codes, uint8_t* scales,
                            int64_t scale_stride, moe_stream_t stream) {
  const int vb = value_bytes(dtype);
  if (!fp4_format_ok(format) || vb == 0 || rows < 0 || cols <= 0 || cols % 32 != 0 || row_stride < cols)
    return MOE_ERR_INVALID_ARG;
  if (scale_stride < cols / (format == MOE_FP4_NV ? 16 : 32)) return MOE_ERR_INVALID_ARG;
  if (format == MOE_FP4_MX && tensor_scale != nullptr) return MOE_ERR_INVALID_ARG;
  if (rows > kMaxQuantized / cols) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (src == nullptr || codes == nullptr || scales == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned(src, vb) || !aligned(codes, 16) || !aligned(tensor_scale, 4)) return MOE_ERR_INVALID_ARG;
  const moe_status st = on_device({src, tensor_scale, codes, scales});
  if (st != MOE_OK) return st;
  return launched(launch_quantize_fp4(format, src, dtype, rows, cols, row_stride, tensor_scale, codes, scales,
                                      scale_stride, as_stream(stream)));
}

moe_status moe_dequantize_fp4(int32_t format, const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t cols,
                              int64_t scale_stride, const float* tensor_scale, void* dst, int32_t dtype,
                              moe_stream_t stream) {
  const int vb = value_bytes(dtype);
  if (!fp4_format_ok(format) || vb == 0 || rows < 0 || cols <= 0 || cols % 32 != 0) return MOE_ERR_INVALID_ARG;
  if (scale_stride < cols / (format == MOE_FP4_NV ? 16 : 32)) return MOE_ERR_INVALID_ARG;
  if (format == MOE_FP4_MX && tensor_scale != nullptr) return MOE_ERR_INVALID_ARG;
  if (rows > kMaxQuantized / cols) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (codes == nullptr || scales == nullptr || dst == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned(codes, 16) || !aligned(dst, vb) || !aligned(tensor_scale, 4)) return MOE_ERR_INVALID_ARG;
  const moe_status st = on_device({codes, scales, tensor_scale, dst});
  if (st != MOE_OK) return st;
  return launched(launch_dequantize_fp4(format, codes, scales, rows, cols, scale_stride, tensor_scale, dst, dtype,
                                        as_stream(stream)));
}

moe_status moe_fp4_pad_scales(const uint8_t* src, int64_t rows, int32_t cols, uint8_t* dst, int64_t dst_stride,
                              moe_stream_t stream) {
  if (rows < 0 || cols < 1 || dst_stride < cols || dst_stride % 16 != 0) return MOE_ERR_INVALID_ARG;
  if (dst_stride > 1 << 20 || rows > (int64_t(1) << 38) / dst_stride) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (src == nullptr || dst == nullptr || !aligned(dst, 16)) return MOE_ERR_INVALID_ARG;
  const moe_status st = on_device({src, dst});
  if (st != MOE_OK) return st;
  return launched(launch_pad_scales(src, cols, rows, cols, dst, dst_stride, as_stream(stream)));
}

int64_t moe_fp4_workspace_bytes(int32_t format, int32_t T, int32_t N, int32_t K, int32_t E) {
  if (!fp4_format_ok(format) || !product_shape_ok(T, N, K, E) || T == 0) return 0;
  return plan_product(format, T, N, K, E).bytes;
}

moe_status moe_fp4_matmul(const moe_fp4_product* p, moe_stream_t stream) {
  if (p == nullptr) return MOE_ERR_INVALID_ARG;
  moe_status st = check_product(*p);
  if (st != MOE_OK || p->T == 0) return st;
  if (p->x == nullptr || p->x_scales == nullptr || !aligned(p->x, 16) || p->x == p->y) return MOE_ERR_INVALID_ARG;
  const int cols = p->K / (p->format == MOE_FP4_NV ? 16 : 32);
  if (p->x_scale_stride < cols) return MOE_ERR_INVALID_ARG;
  const Planned planned = plan_product(p->format, p->T, p->N, p->K, p->E);
  if (!scales_ok(*p, planned) || p->workspace_bytes < planned.bytes || (planned.bytes > 0 && p->workspace == nullptr))
    return MOE_ERR_INVALID_ARG;
  st = on_device({p->x, p->x_scales, p->w, p->w_scales, p->y, p->offsets, p->x_tensor_scale, p->w_tensor_scale,
                  p->status, p->workspace});
  if (st != MOE_OK) return st;
  return run_product(*p, planned.plan, as_stream(stream));
}

moe_status moe_fp4_set_wait_timeout(uint64_t timeout_ns) {
  if (timeout_ns == 0) return MOE_ERR_INVALID_ARG;
  wait_ns.store(timeout_ns, std::memory_order_relaxed);
  return MOE_OK;
}

moe_status moe_fp4_get_status(void) {
  int v = 0;
  if (take_fp4_status(&v) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return v & kStatusTimeout ? MOE_ERR_TIMEOUT : MOE_OK;
}

int64_t moe_fp4_linear_workspace_bytes(int32_t format, int32_t T, int32_t N, int32_t K, int32_t E) {
  if (!fp4_format_ok(format) || !product_shape_ok(T, N, K, E) || K % 32 != 0 || T == 0 || T > kMaxQuantized / K)
    return 0;
  int64_t bytes = plan_product(format, T, N, K, E).bytes;
  if (bytes == 0 && K / (format == MOE_FP4_NV ? 16 : 32) % scale_unit(format) != 0) bytes = padded_w(format, N, K, E);
  return T * (K / 2 + padded_scales(format, K)) + bytes;
}

moe_status moe_fp4_linear(const moe_fp4_product* p, int32_t x_dtype, int64_t x_row_stride, moe_stream_t stream) {
  if (p == nullptr) return MOE_ERR_INVALID_ARG;
  moe_status st = check_product(*p);
  if (st != MOE_OK || p->T == 0) return st;
  if (p->T > kMaxQuantized / p->K) return MOE_ERR_UNSUPPORTED;
  const int vb = value_bytes(x_dtype);
  if (vb == 0 || x_row_stride < p->K || p->x == nullptr || !aligned(p->x, vb) || p->x == p->y ||
      p->workspace == nullptr)
    return MOE_ERR_INVALID_ARG;
  const Planned planned = plan_product(p->format, p->T, p->N, p->K, p->E);
  const int64_t xs_stride = padded_scales(p->format, p->K), own = p->T * (p->K / 2 + xs_stride);
  if (p->workspace_bytes < own + planned.bytes) return MOE_ERR_INVALID_ARG;
  // the workspace: codes, scales in rows padded to 16 bytes (read in whole vectors), the product's own
  moe_fp4_product q = *p;
  uint8_t* codes = static_cast<uint8_t*>(p->workspace);
  q.x = codes;
  q.x_scale_stride = xs_stride;
  uint8_t* scales = codes + static_cast<int64_t>(p->T) * (p->K / 2);
  q.x_scales = scales;
  q.workspace = codes + own;
  q.workspace_bytes = p->workspace_bytes - own;
  const bool pad_w = !scales_ok(q, planned);
  if (pad_w && q.workspace_bytes < padded_w(p->format, p->N, p->K, p->E)) return MOE_ERR_INVALID_ARG;
  st = on_device({p->x, p->w, p->w_scales, p->y, p->offsets, p->x_tensor_scale, p->w_tensor_scale, p->status,
                  p->workspace});
  if (st != MOE_OK) return st;
  if (pad_w) {  // in front of the quantiser, whose end the product's start then overlaps
    st = launched(launch_pad_scales(p->w_scales, p->w_scale_stride, static_cast<int64_t>(p->E) * p->N,
                                    p->K / (p->format == MOE_FP4_NV ? 16 : 32), codes + own, xs_stride,
                                    as_stream(stream)));
    if (st != MOE_OK) return st;
    q.w_scales = codes + own;
    q.w_scale_stride = xs_stride;
  }
  st = launched(launch_quantize_fp4(p->format, p->x, x_dtype, p->T, p->K, x_row_stride, p->x_tensor_scale, codes, scales,
                                    q.x_scale_stride, as_stream(stream)));
  if (st != MOE_OK) return st;
  return run_product(q, planned.plan, as_stream(stream));
}

}  // extern "C"
