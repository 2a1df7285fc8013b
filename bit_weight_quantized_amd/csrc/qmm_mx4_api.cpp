// C-ABI entry points of the microscaled 4-bit path and of the expert layer: argument validation (host only,
// before any HIP call) and error mapping.  See include/qmm.h.
#include <hip/hip_runtime.h>

#include "qmm_internal.h"
#include "qmm_moe_layer.h"
#include "qmm_mx4.h"

#include <math.h>

namespace {

using qmm::api_fail;
using qmm::api_hip_fail;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t k2G = int64_t(1) << 31;

bool known(qmm_mx_rule rule) { return rule == QMM_MX_FLOOR || rule == QMM_MX_FIT; }

// [n, d] as packed weights of the kernels, which address one matrix with 32-bit offsets
qmm_status check_matrix(int64_t n, int64_t d) {
  if (n < 1 || d < 1) return api_fail(QMM_E_ARG, "n and d must be >= 1");
  qmm::Layout l;
  if (!qmm::layout_of(QMM_MXFP4_G32, n, d, &l))
    return api_fail(QMM_E_SHAPE, "d must be a multiple of 32 and <= 65536, n <= 2^28");
  if (n * (d / 2) >= k2G || l.meta_bytes >= k2G)
    return api_fail(QMM_E_SHAPE, "32-bit offsets: n*d/2 of a matrix must be below 2^31");
  return QMM_OK;
}

qmm_status check_grouped(const qmm::Mx4GemmArgs& g, int64_t n, int64_t d, bool any) {
  qmm_status st = check_matrix(n, d);
  if (st) return st;
  if (g.glu && n % 2) return api_fail(QMM_E_SHAPE, "a gate_up stack needs an even n (gate rows, then up rows)");
  if (g.n_experts < 1) return api_fail(QMM_E_ARG, "n_experts must be >= 1");
  if (g.n_seg < 0 || g.m_total < 0 || g.t_x < 1)
    return api_fail(QMM_E_ARG, "n_seg, m_total >= 0 and t_x >= 1 required");
  if (g.n_seg > 65535) return api_fail(QMM_E_SHAPE, "n_seg must be <= 65535");
  if (g.t_x > qmm::kMaxT || g.t_x * (d / 2) >= k2G)
    return api_fail(QMM_E_SHAPE, "the codes of x must be under 2 GiB, t_x <= 2^24");
  if (g.hq && (n / 2) % 32) return api_fail(QMM_E_SHAPE, "quantised outputs need n/2 to be a multiple of 32");
  const int64_t size = int64_t(qmm_packed_bytes(QMM_MXFP4_G32, n, d));
  if (g.expert_stride < size || g.expert_stride % 256)
    return api_fail(QMM_E_ARG, "the stride of the stack must be a multiple of 256 and >= qmm_packed_bytes()");
  if (!any) return QMM_OK;
  if (!g.packed || !g.x || !g.xs) return api_fail(QMM_E_ARG, "NULL pointer");
  if (!g.seg_expert || !g.seg_offsets) return api_fail(QMM_E_ARG, "NULL routing table");
  if (g.max_seg_rows < 1) return api_fail(QMM_E_ARG, "max_seg_rows must be >= 1");
  if (!aligned(g.packed, 256)) return api_fail(QMM_E_ALIGN, "packed_stack must be 256-byte aligned");
  if (!aligned(g.x, 16) || !aligned(g.xs, 16)) return api_fail(QMM_E_ALIGN, "x and x_scales must be 16-byte aligned");
  if (!aligned(g.y, 2)) return api_fail(QMM_E_ALIGN, "bf16 outputs must be 2-byte aligned");
  if (!aligned(g.hq, 16) || !aligned(g.hs, 16)) return api_fail(QMM_E_ALIGN, "hq and h_scales must be 16-byte aligned");
  if (!aligned(g.row_index, 4) || !aligned(g.seg_expert, 4) || !aligned(g.seg_offsets, 4))
    return api_fail(QMM_E_ALIGN, "routing tables must be 4-byte aligned");
  return QMM_OK;
}

}  // namespace

extern "C" {

size_t qmm_mxfp4_scale_bytes(int64_t d) {
  if (d < 32 || d > qmm::kMaxD || d % 32) return 0;
  return size_t(qmm::mx_scale_bytes(int(d)));
}

qmm_status qmm_mxfp4_quant(const qmm_bf16* x, int64_t t, int64_t d, int64_t ldx, qmm_mx_rule rule, uint8_t* q,
                           uint8_t* scales, void* stream) {
  api_fail(QMM_OK, "");
  if (t < 0 || d < 1) return api_fail(QMM_E_ARG, "t must be >= 0 and d >= 1");
  if (d > qmm::kMaxD || d % 32) return api_fail(QMM_E_SHAPE, "d must be a multiple of 32 and <= 65536");
  if (t > qmm::kMaxT) return api_fail(QMM_E_SHAPE, "t must be <= 2^24");
  if (!known(rule)) return api_fail(QMM_E_ARG, "unknown rule of the exponents");
  if (ldx < d) return api_fail(QMM_E_ARG, "ldx must be >= d");
  if (t == 0) return QMM_OK;
  if (!x || !q || !scales) return api_fail(QMM_E_ARG, "NULL pointer");
  if (!aligned(x, 16) || ldx % 8) return api_fail(QMM_E_ALIGN, "rows of x must be 16-byte aligned (ldx a multiple of 8)");
  if (!aligned(q, 16) || !aligned(scales, 16)) return api_fail(QMM_E_ALIGN, "q and scales must be 16-byte aligned");
  const int err = qmm::launch_mx4_quant({x, t, ldx, int(d), rule == QMM_MX_FIT, q, scales}, stream);
  return err ? api_hip_fail(err, "qmm_mxfp4_quant") : QMM_OK;
}

qmm_status qmm_mxfp4_gemm(const void* packed, int64_t t, int64_t n, int64_t d, const uint8_t* x, const uint8_t* x_scales,
                          qmm_bf16* y, int64_t ldy, void* stream) {
  api_fail(QMM_OK, "");
  qmm_status st = check_matrix(n, d);
  if (st) return st;
  if (t < 0) return api_fail(QMM_E_ARG, "t must be >= 0");
  if (t > qmm::kMaxT) return api_fail(QMM_E_SHAPE, "t must be <= 2^24");
  if (ldy < n) return api_fail(QMM_E_ARG, "ldy must be >= n");
  if (t == 0) return QMM_OK;
  if (!packed || !x || !x_scales || !y) return api_fail(QMM_E_ARG, "NULL pointer");
  if (!aligned(packed, 256)) return api_fail(QMM_E_ALIGN, "packed must be 256-byte aligned");
  if (!aligned(x, 16) || !aligned(x_scales, 16)) return api_fail(QMM_E_ALIGN, "x and x_scales must be 16-byte aligned");
  if (!aligned(y, 2)) return api_fail(QMM_E_ALIGN, "y must be 2-byte aligned");
  qmm::Mx4GemmArgs a{};
  a.packed = static_cast<const uint8_t*>(packed);
  a.x = x;
  a.xs = x_scales;
  a.y = y;
  a.t = t;
  a.ldy = ldy;
  a.n = int(n);
  a.d = int(d);
  const int err = qmm::launch_mx4_product(a, stream);
  return err ? api_hip_fail(err, "qmm_mxfp4_gemm") : QMM_OK;
}

qmm_status qmm_mxfp4_grouped_gemm(const void* packed_stack, int64_t expert_stride_bytes, int32_t n_experts, int64_t n,
                                  int64_t d, const uint8_t* x, const uint8_t* x_scales, int64_t t_x,
                                  const int32_t* row_index, const int32_t* seg_expert, const int32_t* seg_offsets,
                                  int32_t n_seg, int32_t m_total, int32_t max_seg_rows, qmm_bf16* y, void* stream) {
  api_fail(QMM_OK, "");
  qmm::Mx4GemmArgs a{static_cast<const uint8_t*>(packed_stack), expert_stride_bytes, x, x_scales, m_total, n, y, int(n),
                     int(d), t_x, row_index, seg_expert, seg_offsets, n_experts, n_seg, m_total,
                     max_seg_rows < m_total ? max_seg_rows : m_total, false, false, nullptr, nullptr};
  const bool any = n_seg != 0 && m_total != 0;
  const qmm_status st = check_grouped(a, n, d, any);
  if (st || !any) return st;
  if (!y) return api_fail(QMM_E_ARG, "NULL pointer");
  const int err = qmm::launch_mx4_product(a, stream);
  return err ? api_hip_fail(err, "qmm_mxfp4_grouped_gemm") : QMM_OK;
}

qmm_status qmm_mxfp4_grouped_gemm_swiglu(const void* packed_stack, int64_t expert_stride_bytes, int32_t n_experts,
                                         int64_t n, int64_t d, const uint8_t* x, const uint8_t* x_scales, int64_t t_x,
                                         const int32_t* row_index, const int32_t* seg_expert,
                                         const int32_t* seg_offsets, int32_t n_seg, int32_t m_total,
                                         int32_t max_seg_rows, qmm_mx_rule rule, qmm_bf16* h, uint8_t* hq,
                                         uint8_t* h_scales, void* stream) {
  api_fail(QMM_OK, "");
  if (!hq != !h_scales) return api_fail(QMM_E_ARG, "hq and h_scales come together");
  if (h && hq) return api_fail(QMM_E_ARG, "one output: h, or hq with h_scales");
  if (hq && !known(rule)) return api_fail(QMM_E_ARG, "unknown rule of the exponents");
  qmm::Mx4GemmArgs a{static_cast<const uint8_t*>(packed_stack), expert_stride_bytes, x, x_scales, m_total, n / 2, h,
                     int(n), int(d), t_x, row_index, seg_expert, seg_offsets, n_experts, n_seg, m_total,
                     max_seg_rows < m_total ? max_seg_rows : m_total, true, rule == QMM_MX_FIT, hq, h_scales};
  const bool any = n_seg != 0 && m_total != 0;
  const qmm_status st = check_grouped(a, n, d, any);
  if (st || !any) return st;
  if (!h && !hq) return api_fail(QMM_E_ARG, "no output asked for");
  const int err = qmm::launch_mx4_product(a, stream);
  return err ? api_hip_fail(err, "qmm_mxfp4_grouped_gemm_swiglu") : QMM_OK;
}

size_t qmm_moe_layer_workspace_bytes(int64_t t, int32_t k, int64_t inter) {
  if (t < 1 || t > qmm::kLayerMaxTokens || k < 1 || k > qmm::kRouteMaxK || t * k > qmm::kLayerMaxPairs) return 0;
  if (inter < 32 || inter > qmm::kMaxD || inter % 32) return 0;
  return size_t(4 * t * k * inter);
}

qmm_status qmm_moe_layer(qmm_format f, const void* gate_up, int64_t gate_up_stride_bytes, const void* down,
                         int64_t down_stride_bytes, int32_t n_experts, int64_t d, int64_t inter, const qmm_bf16* x,
                         int64_t t, const void* logits, qmm_dtype dtype, int64_t ld, qmm_score score,
                         const float* bias, int32_t n_groups, int32_t keep_groups, qmm_group_score group_score,
                         int32_t k, int32_t renorm, float scale, const qmm_bf16* shared, int32_t* topk,
                         float* weights, qmm_bf16* out, void* ws, size_t ws_bytes, void* stream) {
  api_fail(QMM_OK, "");
  if (f != QMM_MXFP4_G32)
    return api_fail(f == QMM_AFFINE4_G64 ? QMM_E_UNSUPPORTED : QMM_E_ARG, "the expert layer takes QMM_MXFP4_G32 weights");
  if (dtype != QMM_BF16 && dtype != QMM_F32) return api_fail(QMM_E_ARG, "unknown type of the logits");
  if (score != QMM_SCORE_SOFTMAX && score != QMM_SCORE_SIGMOID) return api_fail(QMM_E_ARG, "unknown score");
  if (group_score != QMM_GROUP_MAX && group_score != QMM_GROUP_TOP2) return api_fail(QMM_E_ARG, "unknown group score");
  if (t < 0 || n_experts < 1 || k < 1) return api_fail(QMM_E_ARG, "t >= 0, n_experts >= 1 and k >= 1 required");
  if (d < 1 || inter < 1) return api_fail(QMM_E_ARG, "d and inter must be >= 1");
  if (d > qmm::kMaxD || d % 32 || inter > qmm::kMaxD || inter % 32)
    return api_fail(QMM_E_SHAPE, "d and inter must be multiples of 32 and <= 65536");
  qmm_status st = check_matrix(2 * inter, d);
  if (st || (st = check_matrix(d, inter))) return st;
  if (n_experts > qmm::kRouteMaxExperts) return api_fail(QMM_E_SHAPE, "n_experts must be <= 1024");
  if (k > qmm::kRouteMaxK || k > n_experts) return api_fail(QMM_E_SHAPE, "k must be <= min(64, n_experts)");
  if (n_groups < 1 || n_groups > 64 || n_experts % n_groups)
    return api_fail(QMM_E_SHAPE, "n_groups must divide n_experts and be <= 64");
  if (keep_groups < 1 || keep_groups > n_groups) return api_fail(QMM_E_ARG, "keep_groups must be in 1..n_groups");
  if (ld < n_experts) return api_fail(QMM_E_ARG, "ld must be >= n_experts");
  if (t > qmm::kLayerMaxTokens || t * k > qmm::kLayerMaxPairs) return api_fail(QMM_E_SHAPE, "t must be <= 16 and t*k <= 256");
  if (!isfinite(scale)) return api_fail(QMM_E_ARG, "scale must be finite");
  if (gate_up_stride_bytes < int64_t(qmm_packed_bytes(f, 2 * inter, d)) || gate_up_stride_bytes % 256 ||
      down_stride_bytes < int64_t(qmm_packed_bytes(f, d, inter)) || down_stride_bytes % 256)
    return api_fail(QMM_E_ARG, "the stride of a stack must be a multiple of 256 and >= qmm_packed_bytes()");
  if (t == 0) return QMM_OK;
  if (!gate_up || !down || !x || !logits || !topk || !weights || !out) return api_fail(QMM_E_ARG, "NULL pointer");
  if (!aligned(gate_up, 256) || !aligned(down, 256)) return api_fail(QMM_E_ALIGN, "stacks must be 256-byte aligned");
  if (!aligned(x, 16)) return api_fail(QMM_E_ALIGN, "x must be 16-byte aligned");
  if (!aligned(shared, 8) || !aligned(out, 8)) return api_fail(QMM_E_ALIGN, "shared and out must be 8-byte aligned");
  if (!aligned(logits, dtype == QMM_BF16 ? 2 : 4)) return api_fail(QMM_E_ALIGN, "logits must be aligned to their type");
  if (!aligned(bias, 4) || !aligned(topk, 4) || !aligned(weights, 4))
    return api_fail(QMM_E_ALIGN, "bias, topk and weights must be 4-byte aligned");
  // half the size, as the call took it first, in whole 16 bytes: h in pairs
  const size_t full = qmm_moe_layer_workspace_bytes(t, k, inter);
  const bool pairs = ws_bytes < full;
  if (!ws || ws_bytes < full / 2 || (pairs && ws_bytes % 16))
    return api_fail(QMM_E_WORKSPACE, "workspace NULL, or not of qmm_moe_layer_workspace_bytes() or half of it");
  if (!aligned(ws, 16)) return api_fail(QMM_E_ALIGN, "ws must be 16-byte aligned");
  const qmm::MoeLayerArgs a{static_cast<const uint8_t*>(gate_up), gate_up_stride_bytes,
                            static_cast<const uint8_t*>(down), down_stride_bytes, n_experts, int(d), int(inter), x,
                            int(t), logits, dtype == QMM_BF16, ld, score == QMM_SCORE_SIGMOID, bias, n_groups,
                            keep_groups, group_score == QMM_GROUP_TOP2, k, renorm != 0, scale, shared, topk, weights,
                            out, static_cast<uint16_t*>(ws), pairs};
  const int err = qmm::launch_moe_layer(a, stream);
  return err ? api_hip_fail(err, "qmm_moe_layer") : QMM_OK;
}

}  // extern "C"
