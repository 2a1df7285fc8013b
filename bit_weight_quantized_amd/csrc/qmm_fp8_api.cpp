// C-ABI entry points of the block-scaled e4m3 path, the top-k router, the
// gather and the norms: argument validation (host only, before any HIP call)
// and error mapping.  See include/qmm.h.
#include <hip/hip_runtime.h>

#include <math.h>

#include "qmm_fp8.h"
#include "qmm_internal.h"

namespace {

using qmm::api_fail;
using qmm::api_hip_fail;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t k2G = int64_t(1) << 31;

qmm_status check_fp8_shape(int64_t n, int64_t d) {
  if (n < 1 || d < 1) return api_fail(QMM_E_ARG, "n and d must be >= 1");
  if (n > qmm::kMaxN || d > qmm::kMaxD || d % 16)
    return api_fail(QMM_E_SHAPE, "d must be a multiple of 16 and <= 65536, n <= 2^28");
  return QMM_OK;
}

qmm_status grouped(const char* name, bool glu, const uint8_t* w_stack, const float* w_scales, int32_t n_experts,
                   int64_t n, int64_t d, const uint8_t* x, const float* x_scales, int64_t t_x,
                   const int32_t* row_index, const int32_t* seg_expert, const int32_t* seg_offsets, int32_t n_seg,
                   int32_t m_total, int32_t max_seg_rows, qmm_bf16* y, void* stream) {
  api_fail(QMM_OK, "");
  qmm_status st = check_fp8_shape(n, d);
  if (st) return st;
  if (glu && n % 2) return api_fail(QMM_E_SHAPE, "a gate_up stack needs an even n (gate rows, then up rows)");
  if (n_experts < 1) return api_fail(QMM_E_ARG, "n_experts must be >= 1");
  if (n_seg < 0 || m_total < 0 || t_x < 1) return api_fail(QMM_E_ARG, "n_seg, m_total >= 0 and t_x >= 1 required");
  if (n_seg > 65535) return api_fail(QMM_E_SHAPE, "n_seg must be <= 65535");
  if (t_x > qmm::kMaxT || t_x * d >= k2G) return api_fail(QMM_E_SHAPE, "x must be under 2 GiB, t_x <= 2^24");
  if (n_seg == 0 || m_total == 0) return QMM_OK;
  if (!w_stack || !w_scales || !x || !x_scales || !y) return api_fail(QMM_E_ARG, "NULL pointer");
  if (!seg_expert || !seg_offsets) return api_fail(QMM_E_ARG, "NULL routing table");
  if (max_seg_rows < 1) return api_fail(QMM_E_ARG, "max_seg_rows must be >= 1");
  if (!aligned(w_stack, 16) || !aligned(x, 16)) return api_fail(QMM_E_ALIGN, "w_stack and x must be 16-byte aligned");
  if (!aligned(w_scales, 4) || !aligned(x_scales, 4)) return api_fail(QMM_E_ALIGN, "scales must be 4-byte aligned");
  if (!aligned(y, 2)) return api_fail(QMM_E_ALIGN, "y must be 2-byte aligned");
  if (!aligned(row_index, 4) || !aligned(seg_expert, 4) || !aligned(seg_offsets, 4))
    return api_fail(QMM_E_ALIGN, "routing tables must be 4-byte aligned");
  qmm::Fp8GemmArgs a{};
  a.w = w_stack;
  a.ws = w_scales;
  a.x = x;
  a.xs = x_scales;
  a.y = y;
  a.t = m_total;
  a.ldy = glu ? n / 2 : n;
  a.n = int(n);
  a.d = int(d);
  a.t_x = t_x;
  a.row_index = row_index;
  a.seg_expert = seg_expert;
  a.seg_offsets = seg_offsets;
  a.n_experts = n_experts;
  a.n_seg = n_seg;
  a.m_total = m_total;
  a.max_seg_rows = max_seg_rows < m_total ? max_seg_rows : m_total;
  a.glu = glu;
  const int err = qmm::launch_fp8_product(a, stream);
  return err ? api_hip_fail(err, name) : QMM_OK;
}

}  // namespace

extern "C" {

qmm_status qmm_fp8_quant(const qmm_bf16* x, int64_t t, int64_t d, int64_t ldx, uint8_t* q, float* scales,
                         void* stream) {
  api_fail(QMM_OK, "");
  if (t < 0 || d < 1) return api_fail(QMM_E_ARG, "t must be >= 0 and d >= 1");
  if (d > qmm::kMaxD || d % 16) return api_fail(QMM_E_SHAPE, "d must be a multiple of 16 and <= 65536");
  if (t > qmm::kMaxT || t * qmm::fp8_blocks(d) > (int64_t(1) << 28))
    return api_fail(QMM_E_SHAPE, "t must be <= 2^24, t times the blocks of a row <= 2^28");
  if (ldx < d) return api_fail(QMM_E_ARG, "ldx must be >= d");
  if (t == 0) return QMM_OK;
  if (!x || !q || !scales) return api_fail(QMM_E_ARG, "NULL pointer");
  if (!aligned(x, 16) || ldx % 8) return api_fail(QMM_E_ALIGN, "rows of x must be 16-byte aligned (ldx a multiple of 8)");
  if (!aligned(q, 16) || !aligned(scales, 4)) return api_fail(QMM_E_ALIGN, "q must be 16-byte, scales 4-byte aligned");
  const int err = qmm::launch_fp8_quant({x, t, ldx, int(d), q, scales}, stream);
  return err ? api_hip_fail(err, "qmm_fp8_quant") : QMM_OK;
}

qmm_status qmm_fp8_gemm(const uint8_t* w, const float* w_scales, int64_t t, int64_t n, int64_t d, const uint8_t* x,
                        const float* x_scales, qmm_bf16* y, int64_t ldy, void* stream) {
  api_fail(QMM_OK, "");
  qmm_status st = check_fp8_shape(n, d);
  if (st) return st;
  if (t < 0) return api_fail(QMM_E_ARG, "t must be >= 0");
  if (t > qmm::kMaxT) return api_fail(QMM_E_SHAPE, "t must be <= 2^24");
  if (ldy < n) return api_fail(QMM_E_ARG, "ldy must be >= n");
  if (t == 0) return QMM_OK;
  if (!w || !w_scales || !x || !x_scales || !y) return api_fail(QMM_E_ARG, "NULL pointer");
  if (!aligned(w, 16) || !aligned(x, 16)) return api_fail(QMM_E_ALIGN, "w and x must be 16-byte aligned");
  if (!aligned(w_scales, 4) || !aligned(x_scales, 4)) return api_fail(QMM_E_ALIGN, "scales must be 4-byte aligned");
  if (!aligned(y, 2)) return api_fail(QMM_E_ALIGN, "y must be 2-byte aligned");
  qmm::Fp8GemmArgs a{};
  a.w = w;
  a.ws = w_scales;
  a.x = x;
  a.xs = x_scales;
  a.y = y;
  a.t = t;
  a.ldy = ldy;
  a.n = int(n);
  a.d = int(d);
  const int err = qmm::launch_fp8_product(a, stream);
  return err ? api_hip_fail(err, "qmm_fp8_gemm") : QMM_OK;
}

qmm_status qmm_fp8_grouped_gemm(const uint8_t* w_stack, const float* w_scales, int32_t n_experts, int64_t n, int64_t d,
                                const uint8_t* x, const float* x_scales, int64_t t_x, const int32_t* row_index,
                                const int32_t* seg_expert, const int32_t* seg_offsets, int32_t n_seg, int32_t m_total,
                                int32_t max_seg_rows, qmm_bf16* y, void* stream) {
  return grouped("qmm_fp8_grouped_gemm", false, w_stack, w_scales, n_experts, n, d, x, x_scales, t_x, row_index,
                 seg_expert, seg_offsets, n_seg, m_total, max_seg_rows, y, stream);
}

qmm_status qmm_fp8_grouped_gemm_swiglu(const uint8_t* w_stack, const float* w_scales, int32_t n_experts, int64_t n,
                                       int64_t d, const uint8_t* x, const float* x_scales, int64_t t_x,
                                       const int32_t* row_index, const int32_t* seg_expert, const int32_t* seg_offsets,
                                       int32_t n_seg, int32_t m_total, int32_t max_seg_rows, qmm_bf16* h,
                                       void* stream) {
  return grouped("qmm_fp8_grouped_gemm_swiglu", true, w_stack, w_scales, n_experts, n, d, x, x_scales, t_x, row_index,
                 seg_expert, seg_offsets, n_seg, m_total, max_seg_rows, h, stream);
}

size_t qmm_route_topk_workspace_bytes(int64_t t, int32_t n_experts) {
  if (t < 1 || t > qmm::kMaxT || n_experts < 1 || n_experts > qmm::kRouteMaxExperts) return 0;
  return qmm::topk_ws_bytes(t, n_experts);
}

qmm_status qmm_route_topk(const void* logits, qmm_dtype dtype, int64_t t, int32_t n_experts, int64_t ld,
                          qmm_score score, const float* bias, int32_t n_groups, int32_t keep_groups,
                          qmm_group_score group_score, int32_t k, int32_t renorm, float scale, int32_t* topk,
                          float* weights, int32_t* seg_expert, int32_t* seg_offsets, int32_t* row_index,
                          int32_t* slot_row, void* ws, size_t ws_bytes, void* stream) {
  api_fail(QMM_OK, "");
  if (dtype != QMM_BF16 && dtype != QMM_F32) return api_fail(QMM_E_ARG, "unknown type of the logits");
  if (score != QMM_SCORE_SOFTMAX && score != QMM_SCORE_SIGMOID) return api_fail(QMM_E_ARG, "unknown score");
  if (group_score != QMM_GROUP_MAX && group_score != QMM_GROUP_TOP2) return api_fail(QMM_E_ARG, "unknown group score");
  if (t < 0 || n_experts < 1 || k < 1) return api_fail(QMM_E_ARG, "t >= 0, n_experts >= 1 and k >= 1 required");
  if (n_experts > qmm::kRouteMaxExperts) return api_fail(QMM_E_SHAPE, "n_experts must be <= 1024");
  if (k > qmm::kRouteMaxK || k > n_experts) return api_fail(QMM_E_SHAPE, "k must be <= min(64, n_experts)");
  if (n_groups < 1 || n_groups > 64 || n_experts % n_groups)
    return api_fail(QMM_E_SHAPE, "n_groups must divide n_experts and be <= 64");
  if (keep_groups < 1 || keep_groups > n_groups) return api_fail(QMM_E_ARG, "keep_groups must be in 1..n_groups");
  if (ld < n_experts) return api_fail(QMM_E_ARG, "ld must be >= n_experts");
  if (t > qmm::kMaxT || t * k >= (int64_t(1) << 30)) return api_fail(QMM_E_SHAPE, "t must be <= 2^24 and t*k below 2^30");
  if (!isfinite(scale)) return api_fail(QMM_E_ARG, "scale must be finite");
  if (!seg_expert || !seg_offsets || (t && (!logits || !topk || !weights || !row_index || !slot_row)))
    return api_fail(QMM_E_ARG, "NULL pointer");
  if (!aligned(logits, dtype == QMM_BF16 ? 2 : 4)) return api_fail(QMM_E_ALIGN, "logits must be aligned to their type");
  if (!aligned(bias, 4) || !aligned(topk, 4) || !aligned(weights, 4) || !aligned(seg_expert, 4) ||
      !aligned(seg_offsets, 4) || !aligned(row_index, 4) || !aligned(slot_row, 4))
    return api_fail(QMM_E_ALIGN, "bias, weights and the tables must be 4-byte aligned");
  const size_t need = t ? qmm::topk_ws_bytes(t, n_experts) : 0;
  if (need && (!ws || ws_bytes < need))
    return api_fail(QMM_E_WORKSPACE, "workspace NULL or smaller than qmm_route_topk_workspace_bytes()");
  if (need && !aligned(ws, 4)) return api_fail(QMM_E_ALIGN, "ws must be 4-byte aligned");
  const qmm::TopkArgs a{logits, dtype == QMM_BF16, t, ld, n_experts, score == QMM_SCORE_SIGMOID, bias,
                        n_groups, keep_groups, group_score == QMM_GROUP_TOP2, k, renorm != 0, scale, topk, weights,
                        seg_expert, seg_offsets, row_index, slot_row, static_cast<int32_t*>(ws)};
  const int err = qmm::launch_topk(a, stream);
  return err ? api_hip_fail(err, "qmm_route_topk") : QMM_OK;
}

qmm_status qmm_moe_gather(const qmm_bf16* o, int32_t m_total, int64_t d, int64_t t, int32_t k, const int32_t* slot_row,
                          const float* weights, const qmm_bf16* shared, qmm_bf16* out, void* stream) {
  api_fail(QMM_OK, "");
  if (t < 0 || k < 1 || m_total < 0) return api_fail(QMM_E_ARG, "t >= 0, k >= 1 and m_total >= 0 required");
  if (k > qmm::kRouteMaxK) return api_fail(QMM_E_SHAPE, "k must be <= 64");
  if (d < 8 || d % 8 || d > qmm::kMaxD) return api_fail(QMM_E_SHAPE, "d must be a multiple of 8 in [8, 65536]");
  if (t > qmm::kMaxT || t * k >= (int64_t(1) << 30)) return api_fail(QMM_E_SHAPE, "t must be <= 2^24 and t*k below 2^30");
  if (t == 0) return QMM_OK;
  if (!o || !slot_row || !weights || !out) return api_fail(QMM_E_ARG, "NULL pointer");
  if (!aligned(o, 16) || !aligned(shared, 16) || !aligned(out, 16))
    return api_fail(QMM_E_ALIGN, "o, shared and out must be 16-byte aligned");
  if (!aligned(slot_row, 4) || !aligned(weights, 4)) return api_fail(QMM_E_ALIGN, "slot_row and weights must be 4-byte aligned");
  const int err = qmm::launch_gather({o, m_total, int(d), k, t, slot_row, weights, shared, out}, stream);
  return err ? api_hip_fail(err, "qmm_moe_gather") : QMM_OK;
}

qmm_status qmm_norm_residual(int64_t t, int64_t d, const qmm_bf16* o, int64_t ldo, const qmm_bf16* post_w,
                             const qmm_bf16* gate, int64_t ldg, int64_t gate_rows, const void* r, qmm_dtype r_type,
                             int64_t ldr, float res_scale, void* r_out, int64_t ldr_out, const qmm_bf16* pre_w,
                             float w_offset, float eps, qmm_bf16* h, int64_t ldh, uint8_t* q, float* q_scales,
                             void* stream) {
  api_fail(QMM_OK, "");
  if (r_type != QMM_BF16 && r_type != QMM_F32) return api_fail(QMM_E_ARG, "unknown type of the residual");
  if (t < 0 || d < 1) return api_fail(QMM_E_ARG, "t must be >= 0 and d >= 1");
  if (d % 8 || d > qmm::kMaxD) return api_fail(QMM_E_SHAPE, "d must be a multiple of 8 and <= 65536");
  if (t > qmm::kMaxT) return api_fail(QMM_E_SHAPE, "t must be <= 2^24");
  if (t == 0) return QMM_OK;
  if (!r) return api_fail(QMM_E_ARG, "NULL residual");
  if (!o && (post_w || gate)) return api_fail(QMM_E_ARG, "post_w and gate apply to the block output o");
  if (!r_out && !h && !q) return api_fail(QMM_E_ARG, "no output asked for");
  if ((h || q) && !pre_w) return api_fail(QMM_E_ARG, "h and q need pre_w");
  if (!q != !q_scales) return api_fail(QMM_E_ARG, "q and q_scales come together");
  if ((o && ldo < d) || ldr < d || (r_out && ldr_out < d) || (h && ldh < d))
    return api_fail(QMM_E_ARG, "row strides must be >= d");
  if (gate && ((ldg && ldg < d) || gate_rows < 1)) return api_fail(QMM_E_ARG, "ldg must be 0 or >= d, gate_rows >= 1");
  if (!(eps >= 0.f) || !isfinite(eps) || !isfinite(res_scale) || !isfinite(w_offset))
    return api_fail(QMM_E_ARG, "eps must be finite and >= 0, res_scale and w_offset finite");
  const int64_t rm = r_type == QMM_F32 ? 4 : 8;   // elements of 16 bytes
  if (!aligned(o, 16) || !aligned(post_w, 16) || !aligned(gate, 16) || !aligned(r, 16) || !aligned(r_out, 16) ||
      !aligned(pre_w, 16) || !aligned(h, 16) || (o && ldo % 8) || (gate && ldg % 8) || ldr % rm ||
      (r_out && ldr_out % rm) || (h && ldh % 8))
    return api_fail(QMM_E_ALIGN, "rows must be 16-byte aligned");
  if (!aligned(q, 8) || !aligned(q_scales, 4)) return api_fail(QMM_E_ALIGN, "q must be 8-byte, q_scales 4-byte aligned");
  const qmm::NormArgs a{t, int(d), o, ldo, post_w, gate, ldg, gate_rows, r, r_type == QMM_F32, ldr, res_scale,
                        r_out, ldr_out, pre_w, w_offset, eps, h, ldh, q, q_scales};
  const int err = qmm::launch_norm_residual(a, stream);
  return err ? api_hip_fail(err, "qmm_norm_residual") : QMM_OK;
}

}  // extern "C"
