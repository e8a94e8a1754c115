// C ABI of the operators around the MoE block and of the dense MLP: argument checks
// and launches.
// See include/beam_moe.h for the contract.
#include "operators.h"

#include <math.h>

#include "../../include/beam_moe.h"

using namespace beam;

namespace {

constexpr int kMaxT = 1 << 22;

bool misaligned(const void* p) { return p && (((uintptr_t)p) & 15u) != 0; }
template <typename... P>
bool any_misaligned(P... p) {
  return (misaligned(p) || ...);
}
bool float_dtype(int32_t d) { return d == BEAM_F32 || d == BEAM_BF16; }
beam_status launched(hipError_t e) { return e == hipSuccess ? BEAM_OK : BEAM_ERR_HIP; }

beam_status check_norm(const beam_moe_norm* c, int32_t T) {
  if (!c) return BEAM_ERR_NULL;
  if (!isfinite(c->keep) || !isfinite(c->add) || !isfinite(c->eps) || c->eps < 0.f)
    return BEAM_ERR_CONFIG;
  if (!float_dtype(c->x_dtype)) return BEAM_ERR_DTYPE;
  if (c->hidden < 1 || c->hidden > kNormMaxH || T < 0 || T > kMaxT) return BEAM_ERR_SHAPE;
  return BEAM_OK;
}

beam_status check_gate(const beam_moe_gate_config* c, int32_t T) {
  if (!c) return BEAM_ERR_NULL;
  const int E = c->n_experts, G = c->n_group;
  if (E < 1 || E > kGateMaxE || G < 1 || G > 64 || E % G != 0) return BEAM_ERR_CONFIG;
  if (c->topk_group < 1 || c->topk_group > G) return BEAM_ERR_CONFIG;
  if (c->top_k < 1 || c->top_k > kGateMaxK || c->top_k > c->topk_group * (E / G))
    return BEAM_ERR_CONFIG;
  if ((c->score != BEAM_SCORE_SIGMOID && c->score != BEAM_SCORE_SOFTMAX) ||
      (c->group_score != BEAM_GROUP_TOP2 && c->group_score != BEAM_GROUP_MAX) ||
      (c->renormalise != 0 && c->renormalise != 1) || !isfinite(c->routed_scaling_factor))
    return BEAM_ERR_CONFIG;
  if (!float_dtype(c->z_dtype)) return BEAM_ERR_DTYPE;
  if (T < 0 || T > kMaxT) return BEAM_ERR_SHAPE;
  return BEAM_OK;
}

beam_status check_mx4_rows(int64_t rows, int32_t cols) {
  if (rows < 0 || cols < 32 || cols % 32 != 0 || rows > (1LL << 40) / cols) return BEAM_ERR_SHAPE;
  return BEAM_OK;
}

beam_status check_linear(const beam_moe_linear* c, int32_t T) {
  if (!c) return BEAM_ERR_NULL;
  if (c->x_format < BEAM_X_E4M3_ROW || c->x_format > BEAM_X_MXFP4) return BEAM_ERR_CONFIG;
  if (!float_dtype(c->out_dtype)) return BEAM_ERR_DTYPE;
  if (c->n < 1 || c->n > (1 << 20) || c->k < 32 || c->k > 65536 || c->k % 32 != 0 || T < 0 ||
      T > kMaxT)
    return BEAM_ERR_SHAPE;
  return BEAM_OK;
}

beam_status check_gated(const beam_moe_gated* c, int32_t T) {
  if (!c) return BEAM_ERR_NULL;
  if (c->activation != BEAM_ACT_SILU && c->activation != BEAM_ACT_GELU) return BEAM_ERR_CONFIG;
  if (c->pre_f32 != 0 && c->pre_f32 != 1) return BEAM_ERR_CONFIG;
  if (c->dtype != BEAM_BF16) return BEAM_ERR_DTYPE;
  if (c->hidden < 8 || c->hidden > kMlpMaxH || c->hidden % 8 != 0 || c->intermediate < 8 ||
      c->intermediate > kMlpMaxF || c->intermediate % 8 != 0 || T < 0 || T > kMaxT)
    return BEAM_ERR_SHAPE;
  return BEAM_OK;
}

beam_status check_lora_plan(int32_t T, int32_t n_adapters) {
  if (n_adapters < 1 || n_adapters > kLoraMaxE) return BEAM_ERR_CONFIG;
  return T < 0 || T > kMaxT ? BEAM_ERR_SHAPE : BEAM_OK;
}

beam_status check_lora(const beam_moe_lora_config* c, int32_t T) {
  if (!c) return BEAM_ERR_NULL;
  if (c->rank < 8 || c->rank > kLoraMaxR || c->rank % 8 != 0) return BEAM_ERR_CONFIG;
  if (c->dtype != BEAM_BF16) return BEAM_ERR_DTYPE;
  if (c->k < 8 || c->k > 65536 || c->k % 8 != 0 || c->n < 8 || c->n > kMlpMaxF || c->n % 8 != 0)
    return BEAM_ERR_SHAPE;
  return check_lora_plan(T, c->n_adapters);
}

// Elements dropped of 65536, or a status
beam_status check_dropout(const beam_moe_dropout_config* c, int64_t n) {
  if (!c) return BEAM_ERR_NULL;
  if (!(c->p >= 0.f && c->p <= 1.f) || !isfinite(c->keep) || !isfinite(c->add)) return BEAM_ERR_CONFIG;
  if (!float_dtype(c->dtype)) return BEAM_ERR_DTYPE;
  return n < 0 || n > (1LL << 40) ? BEAM_ERR_SHAPE : BEAM_OK;
}

DropoutArgs dropout_args(const beam_moe_dropout_config* c, int64_t n, const void* x, uint64_t seed,
                         uint64_t offset, const int64_t* offset_dev) {
  DropoutArgs a{};
  a.x = x;
  a.n = n;
  a.seed = seed;
  a.offset = offset;
  a.offset_dev = offset_dev;
  a.border = (uint32_t)floor((double)c->p * 65536.0 + 0.5);
  // border 65536 keeps nothing
  a.scale = a.border < 65536 ? (float)(65536.0 / (65536.0 - a.border)) : 0.f;
  a.keep = c->keep;
  a.add = c->add;
  return a;
}

}  // namespace

extern "C" {

beam_status beam_moe_add_rms_norm(const beam_moe_norm* cfg, int32_t T, const void* x,
                                  const void* stream_in, const float* norm_weight,
                                  void* stream_out, void* y, void* q, void* q_scale,
                                  void* stream) {
  const beam_status cs = check_norm(cfg, T);
  if (cs != BEAM_OK) return cs;
  const int quant = cfg->quant;
  if (quant < BEAM_QUANT_NONE || quant > BEAM_QUANT_BLOCK) return BEAM_ERR_CONFIG;
  if (quant == BEAM_QUANT_BLOCK && cfg->hidden % 32 != 0) return BEAM_ERR_SHAPE;
  if (T == 0) return BEAM_OK;
  if (!x || !norm_weight || (!stream_out && !y && quant == BEAM_QUANT_NONE)) return BEAM_ERR_NULL;
  if (quant != BEAM_QUANT_NONE && (!q || !q_scale)) return BEAM_ERR_NULL;
  if (quant == BEAM_QUANT_NONE && (q || q_scale)) return BEAM_ERR_CONFIG;
  if (any_misaligned(x, stream_in, norm_weight, stream_out, y, q, q_scale)) return BEAM_ERR_ALIGN;
  const NormArgs a{x,       stream_in, norm_weight, stream_out, y,        (uint8_t*)q,
                   q_scale, T,         cfg->hidden, cfg->keep,  cfg->add, cfg->eps};
  return launched(launch_add_rms_norm(a, cfg->x_dtype == BEAM_F32, quant, (hipStream_t)stream));
}

size_t beam_moe_add_rms_norm_backward_workspace_bytes(const beam_moe_norm* cfg, int32_t T) {
  if (check_norm(cfg, T) != BEAM_OK || T == 0) return 0;
  return (size_t)norm_bwd_groups(T, cfg->hidden) * cfg->hidden * sizeof(float);
}

beam_status beam_moe_add_rms_norm_backward(const beam_moe_norm* cfg, int32_t T, const void* dy,
                                           const void* s, const float* norm_weight,
                                           const void* d_stream_out, void* dx, void* d_stream_in,
                                           float* d_norm_weight, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  const beam_status cs = check_norm(cfg, T);
  if (cs != BEAM_OK) return cs;
  if (T == 0) return BEAM_OK;
  if (!dy || !s || !norm_weight || !dx) return BEAM_ERR_NULL;
  if (d_norm_weight &&
      (!workspace || workspace_bytes < beam_moe_add_rms_norm_backward_workspace_bytes(cfg, T)))
    return BEAM_ERR_WORKSPACE;
  if (any_misaligned(dy, s, norm_weight, d_stream_out, dx, d_stream_in, d_norm_weight, workspace))
    return BEAM_ERR_ALIGN;
  const NormBwdArgs a{dy,  s, norm_weight, d_stream_out, dx,       d_stream_in,
                      d_norm_weight ? (float*)workspace : nullptr, d_norm_weight,
                      T,   cfg->hidden,    cfg->keep,    cfg->add, cfg->eps};
  return launched(launch_add_rms_norm_backward(a, cfg->x_dtype == BEAM_F32, (hipStream_t)stream));
}

beam_status beam_moe_gate(const beam_moe_gate_config* cfg, int32_t T, const void* logits,
                          const float* expert_bias, const uint8_t* valid, int32_t* topk_idx,
                          float* topk_w, int32_t* expert_counts, void* stream) {
  const beam_status cs = check_gate(cfg, T);
  if (cs != BEAM_OK) return cs;
  if (T == 0) return BEAM_OK;
  if (!logits || !topk_idx || !topk_w) return BEAM_ERR_NULL;
  if (any_misaligned(logits, expert_bias, valid, topk_idx, topk_w, expert_counts))
    return BEAM_ERR_ALIGN;
  GateArgs a{};
  a.z = logits;
  a.bias = expert_bias;
  a.valid = valid;
  a.idx = topk_idx;
  a.w = topk_w;
  a.counts = expert_counts;
  a.T = T;
  a.E = cfg->n_experts;
  a.n_group = cfg->n_group;
  a.topk_group = cfg->topk_group;
  a.k = cfg->top_k;
  a.softmax = cfg->score == BEAM_SCORE_SOFTMAX;
  a.top2 = cfg->group_score == BEAM_GROUP_TOP2;
  a.renorm = cfg->renormalise;
  a.rsf = cfg->routed_scaling_factor;
  return launched(launch_gate(a, cfg->z_dtype == BEAM_F32, (hipStream_t)stream));
}

beam_status beam_moe_gate_backward(const beam_moe_gate_config* cfg, int32_t T,
                                   const float* d_topk_w, const void* logits,
                                   const int32_t* topk_idx, void* d_logits, void* stream) {
  const beam_status cs = check_gate(cfg, T);
  if (cs != BEAM_OK) return cs;
  if (T == 0) return BEAM_OK;
  if (!d_topk_w || !logits || !topk_idx || !d_logits) return BEAM_ERR_NULL;
  if (any_misaligned(d_topk_w, logits, topk_idx, d_logits)) return BEAM_ERR_ALIGN;
  GateBwdArgs a{};
  a.dw = d_topk_w;
  a.z = logits;
  a.idx = topk_idx;
  a.dz = d_logits;
  a.T = T;
  a.E = cfg->n_experts;
  a.k = cfg->top_k;
  a.softmax = cfg->score == BEAM_SCORE_SOFTMAX;
  a.renorm = cfg->renormalise;
  a.rsf = cfg->routed_scaling_factor;
  return launched(launch_gate_backward(a, cfg->z_dtype == BEAM_F32, (hipStream_t)stream));
}

beam_status beam_moe_mx4_quantize(const void* src, int64_t rows, int32_t cols, int32_t x_dtype,
                                  int32_t layout, void* codes, void* scales, void* stream) {
  const beam_status cs = check_mx4_rows(rows, cols);
  if (cs != BEAM_OK) return cs;
  if (!float_dtype(x_dtype)) return BEAM_ERR_DTYPE;
  if (layout != BEAM_LAYOUT_ROW_MAJOR && layout != BEAM_LAYOUT_PACKED) return BEAM_ERR_CONFIG;
  const bool packed = layout == BEAM_LAYOUT_PACKED;
  if (packed && (rows % 16 != 0 || cols % 512 != 0)) return BEAM_ERR_SHAPE;
  if (rows == 0) return BEAM_OK;
  if (!src || !codes || !scales) return BEAM_ERR_NULL;
  if (any_misaligned(src, codes, scales)) return BEAM_ERR_ALIGN;
  return launched(launch_mx4_quantize(src, x_dtype == BEAM_F32, rows, cols, packed,
                                      (uint8_t*)codes, (uint8_t*)scales, (hipStream_t)stream));
}

beam_status beam_moe_mx4_dequantize(const void* codes, const void* scales, int64_t rows,
                                    int32_t cols, int32_t out_dtype, void* out, void* stream) {
  const beam_status cs = check_mx4_rows(rows, cols);
  if (cs != BEAM_OK) return cs;
  if (!float_dtype(out_dtype)) return BEAM_ERR_DTYPE;
  if (rows == 0) return BEAM_OK;
  if (!codes || !scales || !out) return BEAM_ERR_NULL;
  if (any_misaligned(codes, scales, out)) return BEAM_ERR_ALIGN;
  return launched(launch_mx4_dequantize((const uint8_t*)codes, (const uint8_t*)scales, rows, cols,
                                        out_dtype == BEAM_F32, out, (hipStream_t)stream));
}

beam_status beam_moe_mx4_linear(const beam_moe_linear* cfg, int32_t T, const void* x,
                                const void* x_scale, const void* w, const void* w_scale,
                                void* out, void* stream) {
  const beam_status cs = check_linear(cfg, T);
  if (cs != BEAM_OK) return cs;
  if (T == 0) return BEAM_OK;
  if (!x || !x_scale || !w || !w_scale || !out) return BEAM_ERR_NULL;
  if (any_misaligned(x, x_scale, w, w_scale, out)) return BEAM_ERR_ALIGN;
  const Mx4LinearArgs a{(const uint8_t*)x, x_scale, (const uint8_t*)w, (const uint8_t*)w_scale,
                        out, T, cfg->n, cfg->k, cfg->out_dtype == BEAM_F32};
  return launched(launch_mx4_linear(a, cfg->x_format, (hipStream_t)stream));
}

size_t beam_moe_gated_linear_workspace_bytes(const beam_moe_gated* cfg, int32_t T) {
  if (check_gated(cfg, T) != BEAM_OK || T == 0) return 0;
  return gated_workspace_bytes(T, cfg->hidden, cfg->intermediate);
}

beam_status beam_moe_gated_linear(const beam_moe_gated* cfg, int32_t T, const void* x,
                                  const void* w_gate, const void* w_up, const void* add_gate,
                                  const void* add_up, void* h, void* gate, void* up, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  const beam_status cs = check_gated(cfg, T);
  if (cs != BEAM_OK) return cs;
  if (T == 0) return BEAM_OK;
  if (!x || !w_gate || !w_up || !h) return BEAM_ERR_NULL;
  const size_t need = beam_moe_gated_linear_workspace_bytes(cfg, T);
  if (need && (!workspace || workspace_bytes < need)) return BEAM_ERR_WORKSPACE;
  if (any_misaligned(x, w_gate, w_up, add_gate, add_up, h, gate, up, workspace)) return BEAM_ERR_ALIGN;
  // rows of twice the bytes: a workgroup would write over another's shares
  if (cfg->pre_f32 && ((gate && (gate == add_gate || gate == add_up)) || (up && (up == add_gate || up == add_up))))
    return BEAM_ERR_CONFIG;
  const GatedArgs a{(const uint16_t*)x,        (const uint16_t*)w_gate, (const uint16_t*)w_up,
                    (const uint16_t*)add_gate, (const uint16_t*)add_up, (uint16_t*)h,
                    gate,                      up,                      (float*)workspace,
                    T,                         cfg->hidden,             cfg->intermediate,
                    cfg->pre_f32 != 0};
  return launched(launch_gated_linear(a, cfg->activation == BEAM_ACT_GELU, (hipStream_t)stream));
}

size_t beam_moe_gated_linear_backward_workspace_bytes(const beam_moe_gated* cfg, int32_t T) {
  if (check_gated(cfg, T) != BEAM_OK || T == 0) return 0;
  return gated_bwd_workspace_bytes(T, cfg->hidden, cfg->intermediate);
}

beam_status beam_moe_gated_linear_backward(const beam_moe_gated* cfg, int32_t T, const void* dh,
                                           const void* x, const void* w_gate, const void* w_up,
                                           const void* gate, const void* up, void* d_gate, void* d_up,
                                           void* dx, void* d_w_gate, void* d_w_up, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  const beam_status cs = check_gated(cfg, T);
  if (cs != BEAM_OK) return cs;
  if (T == 0) return BEAM_OK;
  if (!dh || !gate || !up || !d_gate || !d_up) return BEAM_ERR_NULL;
  if (dx && (!w_gate || !w_up)) return BEAM_ERR_NULL;
  if (!d_w_gate != !d_w_up || (d_w_gate && !x)) return BEAM_ERR_NULL;
  const size_t need = dx || d_w_gate ? beam_moe_gated_linear_backward_workspace_bytes(cfg, T) : 0;
  if (need && (!workspace || workspace_bytes < need)) return BEAM_ERR_WORKSPACE;
  if (any_misaligned(dh, x, w_gate, w_up, gate, up, d_gate, d_up, dx, d_w_gate, d_w_up, workspace))
    return BEAM_ERR_ALIGN;
  if (cfg->pre_f32 && (d_gate == gate || d_gate == up || d_up == gate || d_up == up)) return BEAM_ERR_CONFIG;
  const GatedBwdArgs a{(const uint16_t*)dh,   (const uint16_t*)x,  (const uint16_t*)w_gate,
                       (const uint16_t*)w_up, gate,                up,
                       (uint16_t*)d_gate,     (uint16_t*)d_up,     (uint16_t*)dx,
                       (uint16_t*)d_w_gate,   (uint16_t*)d_w_up,   (float*)workspace,
                       T,                     cfg->hidden,         cfg->intermediate,
                       cfg->pre_f32 != 0};
  return launched(launch_gated_linear_backward(a, cfg->activation == BEAM_ACT_GELU, (hipStream_t)stream));
}

size_t beam_moe_lora_plan_bytes(int32_t T, int32_t n_adapters) {
  if (check_lora_plan(T, n_adapters) != BEAM_OK || T == 0) return 0;
  return LoraPlanLayout(T, n_adapters).words * sizeof(int32_t);
}

beam_status beam_moe_lora_plan(const int32_t* index, int32_t T, int32_t n_adapters, void* plan,
                               size_t plan_bytes, void* stream) {
  const beam_status cs = check_lora_plan(T, n_adapters);
  if (cs != BEAM_OK) return cs;
  if (T == 0) return BEAM_OK;
  if (!index || !plan) return BEAM_ERR_NULL;
  if (plan_bytes < beam_moe_lora_plan_bytes(T, n_adapters)) return BEAM_ERR_WORKSPACE;
  if (any_misaligned(index, plan)) return BEAM_ERR_ALIGN;
  return launched(launch_lora_plan(index, T, n_adapters, (int32_t*)plan, (hipStream_t)stream));
}

size_t beam_moe_lora_workspace_bytes(const beam_moe_lora_config* cfg, int32_t T) {
  if (check_lora(cfg, T) != BEAM_OK || T == 0) return 0;
  return lora_workspace_bytes(T, cfg->k, cfg->n, cfg->rank, cfg->n_adapters);
}

beam_status beam_moe_lora(const beam_moe_lora_config* cfg, int32_t T, const void* x, const void* a,
                          const void* b, const float* scale, const void* plan, const void* base,
                          void* out, float* v, void* workspace, size_t workspace_bytes, void* stream) {
  const beam_status cs = check_lora(cfg, T);
  if (cs != BEAM_OK) return cs;
  if (T == 0) return BEAM_OK;
  if (!x || !a || !b || !plan || !out) return BEAM_ERR_NULL;
  if (!workspace || workspace_bytes < beam_moe_lora_workspace_bytes(cfg, T)) return BEAM_ERR_WORKSPACE;
  if (any_misaligned(x, a, b, scale, plan, base, out, v, workspace)) return BEAM_ERR_ALIGN;
  const LoraArgs p{(const uint16_t*)x,    (const uint16_t*)a, (const uint16_t*)b, scale,
                   (const int32_t*)plan,  (const uint16_t*)base, (uint16_t*)out,  v,
                   (float*)workspace,     T, cfg->k, cfg->n, cfg->rank, cfg->n_adapters};
  return launched(launch_lora(p, (hipStream_t)stream));
}

size_t beam_moe_lora_backward_workspace_bytes(const beam_moe_lora_config* cfg, int32_t T) {
  if (check_lora(cfg, T) != BEAM_OK || T == 0) return 0;
  return lora_bwd_workspace_bytes(T, cfg->k, cfg->n, cfg->rank, cfg->n_adapters);
}

beam_status beam_moe_lora_backward(const beam_moe_lora_config* cfg, int32_t T, const void* dy,
                                   const void* x, const float* v, const void* a, const void* b,
                                   const float* scale, const void* plan, const void* base, void* dx,
                                   void* d_a, void* d_b, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  const beam_status cs = check_lora(cfg, T);
  if (cs != BEAM_OK) return cs;
  if (T == 0) return BEAM_OK;
  if (!dy || !a || !b || !plan || (!dx && !d_a)) return BEAM_ERR_NULL;
  if (!d_a != !d_b || (d_a && (!x || !v))) return BEAM_ERR_NULL;
  if (!workspace || workspace_bytes < beam_moe_lora_backward_workspace_bytes(cfg, T))
    return BEAM_ERR_WORKSPACE;
  if (any_misaligned(dy, x, v, a, b, scale, plan, base, dx, d_a, d_b, workspace)) return BEAM_ERR_ALIGN;
  const LoraBwdArgs p{(const uint16_t*)dy, (const uint16_t*)x, v, (const uint16_t*)a,
                      (const uint16_t*)b,  scale, (const int32_t*)plan, (const uint16_t*)base,
                      (uint16_t*)dx,       (uint16_t*)d_a, (uint16_t*)d_b, workspace,
                      T, cfg->k, cfg->n, cfg->rank, cfg->n_adapters};
  return launched(launch_lora_backward(p, (hipStream_t)stream));
}

beam_status beam_moe_dropout(const beam_moe_dropout_config* cfg, int64_t n, const void* x,
                             const void* stream_in, uint64_t seed, uint64_t offset,
                             const int64_t* offset_dev, void* out, void* stream) {
  const beam_status cs = check_dropout(cfg, n);
  if (cs != BEAM_OK) return cs;
  if (n == 0) return BEAM_OK;
  if (!x || !out) return BEAM_ERR_NULL;
  if (any_misaligned(x, stream_in, out) || (((uintptr_t)offset_dev) & 7u)) return BEAM_ERR_ALIGN;
  DropoutArgs a = dropout_args(cfg, n, x, seed, offset, offset_dev);
  a.stream_in = stream_in;
  a.out = out;
  return launched(launch_dropout(a, cfg->dtype == BEAM_F32, (hipStream_t)stream));
}

beam_status beam_moe_dropout_backward(const beam_moe_dropout_config* cfg, int64_t n, const void* dy,
                                      uint64_t seed, uint64_t offset, const int64_t* offset_dev,
                                      void* dx, void* d_stream_in, void* stream) {
  const beam_status cs = check_dropout(cfg, n);
  if (cs != BEAM_OK) return cs;
  if (n == 0) return BEAM_OK;
  if (!dy || !dx) return BEAM_ERR_NULL;
  if (any_misaligned(dy, dx, d_stream_in) || (((uintptr_t)offset_dev) & 7u)) return BEAM_ERR_ALIGN;
  DropoutArgs a = dropout_args(cfg, n, dy, seed, offset, offset_dev);
  a.out = dx;
  a.kept_grad = d_stream_in;
  return launched(launch_dropout(a, cfg->dtype == BEAM_F32, (hipStream_t)stream));
}

}  // extern "C"
