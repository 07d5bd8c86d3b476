// The C entry points of the gate on given logits and its gradient (include/moe.h): argument checks and launches; the
// ones that score x first are in api.hip. Host code only.
#include <math.h>

#include "api_util.h"
#include "gate.h"

using namespace moe;

moe_status moe::check_rule(const moe_shape& s, const moe_gate_rule* r) {
  if (!r) return fail(MOE_ERR_INVALID_ARG, "rule is NULL");
  if (r->score != MOE_SCORE_SOFTMAX && r->score != MOE_SCORE_SIGMOID) return fail(MOE_ERR_INVALID_ARG, "bad score %d", (int)r->score);
  if (r->groups < 1 || r->groups > GATE_GROUPS_MAX || s.E % r->groups)
    return fail(MOE_ERR_INVALID_ARG, "groups=%d must divide E=%d and be in 1..%d", r->groups, s.E, GATE_GROUPS_MAX);
  if (r->top_groups < 1 || r->top_groups > r->groups || r->top_groups * (s.E / r->groups) < s.k)
    return fail(MOE_ERR_INVALID_ARG, "top_groups=%d must be in 1..groups=%d and hold k=%d experts", r->top_groups, r->groups, s.k);
  if (r->group_top != 1 && r->group_top != 2) return fail(MOE_ERR_INVALID_ARG, "group_top=%d is neither 1 nor 2", r->group_top);
  if (r->renormalize != 0 && r->renormalize != 1) return fail(MOE_ERR_INVALID_ARG, "renormalize=%d is neither 0 nor 1", r->renormalize);
  if (!isfinite(r->scale)) return fail(MOE_ERR_INVALID_ARG, "scale=%g is not finite", r->scale);
  return MOE_OK;
}

GateArgs moe::gate_args(const moe_shape& s, const moe_gate_rule& r) {
  GateArgs a{};
  a.scale = r.scale;
  a.ldl = s.E;
  a.nparts = 1;
  a.T = s.T;
  a.E = s.E;
  a.k = s.k;
  a.sigmoid = r.score == MOE_SCORE_SIGMOID;
  a.renormalize = r.renormalize;
  a.groups = r.groups;
  a.top_groups = r.top_groups;
  a.group_top = r.group_top;
  return a;
}

extern "C" {

moe_status moe_gate(const moe_shape* shape, const moe_gate_rule* rule, const float* logits, const float* bias,
                    int32_t* topk_idx, float* topk_w, moe_stream_t stream) {
  moe_status s = check_shape(shape);
  if (s != MOE_OK) return s;
  if ((s = check_rule(*shape, rule)) != MOE_OK) return s;
  if (!aligned(logits, 4) || !aligned(bias, 4) || !aligned(topk_idx, 4) || !aligned(topk_w, 4))
    return fail(MOE_ERR_INVALID_ARG, "logits, bias, topk_idx and topk_w must be 4-byte aligned");
  if (shape->T == 0) return MOE_OK;
  if (!logits || !topk_idx || !topk_w) return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
  const size_t rows = (size_t)shape->T * 4;
  s = check_outputs({{topk_idx, rows * shape->k}, {topk_w, rows * shape->k}}, {{logits, rows * shape->E}, {bias, (size_t)shape->E * 4}});
  if (s != MOE_OK) return s;
  GateArgs a = gate_args(*shape, *rule);
  a.logits = logits;
  a.bias = bias;
  a.idx = topk_idx;
  a.w = topk_w;
  return hip_status(launch_gate(a, (hipStream_t)stream), "gate");
}

moe_status moe_gate_backward(const moe_shape* shape, const moe_gate_rule* rule, const float* logits,
                             const int32_t* topk_idx, const float* dtopk_w, float* dlogits, moe_stream_t stream) {
  moe_status s = check_shape(shape);
  if (s != MOE_OK) return s;
  if ((s = check_rule(*shape, rule)) != MOE_OK) return s;
  if (!aligned(logits, 4) || !aligned(topk_idx, 4) || !aligned(dtopk_w, 4) || !aligned(dlogits, 4))
    return fail(MOE_ERR_INVALID_ARG, "logits, topk_idx, dtopk_w and dlogits must be 4-byte aligned");
  if (shape->T == 0) return MOE_OK;
  if (!logits || !topk_idx || !dtopk_w || !dlogits) return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
  const size_t rows = (size_t)shape->T * 4;
  s = check_outputs({{dlogits, rows * shape->E}},
                    {{topk_idx, rows * shape->k}, {dtopk_w, rows * shape->k}, {logits == dlogits ? nullptr : logits, rows * shape->E}});
  if (s != MOE_OK) return s;
  GateArgs a = gate_args(*shape, *rule);
  a.logits = logits;
  a.chosen = topk_idx;
  a.dw = dtopk_w;
  a.dlogits = dlogits;
  return hip_status(launch_gate_backward(a, (hipStream_t)stream), "gate gradient");
}

}  // extern "C"
