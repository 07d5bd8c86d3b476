// The C entry points of training (include/moe.h): argument checks, workspace and launches. Host
// code only.
#include <math.h>

#include <algorithm>
#include <initializer_list>
#include <new>

#include "api_util.h"
#include "train.h"

using namespace moe;

namespace {

bool al16(const void* p) { return (uintptr_t)p % 16 == 0; }
bool al4(const void* p) { return (uintptr_t)p % 4 == 0; }
size_t up(size_t x) { return (x + WS_ALIGN - 1) / WS_ALIGN * WS_ALIGN; }

moe_status check_train_shape(const moe_shape* s) {
  moe_shape any = s ? *s : moe_shape{};
  any.path = MOE_PATH_AUTO;  // the path is the inference forward's
  const moe_status r = check_shape(s ? &any : nullptr);
  if (r != MOE_OK) return r;
  if (s->w_routed != s->act)
    return fail(MOE_ERR_UNSUPPORTED, "training takes weights of the activations' type, F32 or BF16");
  if (s->I_shared)
    return fail(MOE_ERR_UNSUPPORTED, "I_shared=%d: a shared expert is a call of its own with E = k = 1", s->I_shared);
  return MOE_OK;
}

struct TrainWs {
  size_t h, dgu, xg, total;
};
TrainWs train_ws(const moe_shape& s) {
  const size_t P = (size_t)s.T * s.k, b = s.act == MOE_F32 ? 4 : 2;
  TrainWs w;
  w.h = 0;
  w.dgu = up(P * s.I * b);
  w.xg = w.dgu + up(P * s.I * 2 * b);
  w.total = w.xg + (s.act == MOE_BF16 ? up(P * s.H * b) : 0) + WS_ALIGN;
  return w;
}

// Bytes of the block's arguments: x, rows of H and of I, a weight matrix of every expert, the indices, the workspace
struct Sizes {
  size_t x, h, i, w, off, slot, ws;
  Sizes(const moe_shape& s, int xrows) {
    const size_t b = s.act == MOE_F32 ? 4 : 2, P = (size_t)s.T * s.k;
    x = (size_t)xrows * s.H * b;
    h = P * s.H * b;
    i = P * s.I * b;
    w = (size_t)s.E * s.H * s.I * b;
    off = ((size_t)s.E + 1) * 4;
    slot = P * 4;
    ws = train_ws(s).total;
  }
};

// Checks common to the block and its gradient, and the arguments they share.
moe_status train_args(const moe_shape* s, const void* x, const int32_t* off, const int32_t* slot_token,
                      const moe_weights* w, void* ws, size_t ws_bytes, TrainArgs* a) {
  moe_status r = check_train_shape(s);
  if (r != MOE_OK) return r;
  if (!w || !w->gate || !w->up || !w->down) return fail(MOE_ERR_INVALID_ARG, "weight pointer is NULL");
  if (!off && s->E != 1) return fail(MOE_ERR_INVALID_ARG, "expert_offsets may be NULL for one expert only (E=%d)", s->E);
  const int P = s->T * s->k;
  if (P && !x) return fail(MOE_ERR_INVALID_ARG, "x is NULL");
  if (!al16(x) || !al16(w->gate) || !al16(w->up) || !al16(w->down))
    return fail(MOE_ERR_INVALID_ARG, "x and the weights must be 16-byte aligned");
  if (!al4(off) || !al4(slot_token)) return fail(MOE_ERR_INVALID_ARG, "index arrays must be 4-byte aligned");
  const TrainWs l = train_ws(*s);
  if (!ws) return fail(MOE_ERR_INVALID_ARG, "workspace is NULL");
  if (ws_bytes < l.total) return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < %zu needed", ws_bytes, l.total);
  if ((uintptr_t)ws % WS_ALIGN) return fail(MOE_ERR_INVALID_ARG, "workspace must be %zu-byte aligned", WS_ALIGN);
  *a = TrainArgs{};
  a->off = off;
  a->slot_token = slot_token;
  a->E = s->E;
  a->P = P;
  a->T = s->T;
  a->H = s->H;
  a->I = s->I;
  a->xrows = slot_token ? s->T : P;
  a->x = x;
  a->gate = w->gate;
  a->up = w->up;
  a->down = w->down;
  a->h = (char*)ws + l.h;
  a->dgu = (char*)ws + l.dgu;
  a->xg = (char*)ws + l.xg;
  return MOE_OK;
}

hipError_t product(TrainForm form, int act, const TrainArgs& a, hipStream_t st) {
  return act == MOE_F32 ? launch_train_f32(form, a, st) : launch_train_bf16(form, a, st);
}

// No two of the updated arrays share memory, and none holds an input: two workgroups would reach it in no order.
moe_status check_apart(const moe_adamw_config* c, const moe_adamw_tensor* t, int count) {
  const bool q8 = c->state == MOE_ADAM_E4M3;
  const size_t p_bytes = c->p_type == MOE_F32 ? 4 : 2, g_bytes = c->g_type == MOE_F32 ? 4 : 2, state_bytes = q8 ? 1 : 4;
  struct Range {
    uintptr_t at, end;
  };
  Range* r = new (std::nothrow) Range[6 * (size_t)count];
  if (!r) return fail(MOE_ERR_INVALID_ARG, "no host memory to check %d tensors", count);
  size_t n = 0;
  auto add = [&](const void* p, size_t bytes) {
    if (p) r[n++] = Range{(uintptr_t)p, (uintptr_t)p + bytes};
  };
  for (int i = 0; i < count; ++i) {
    if (!t[i].n) continue;
    const size_t each = (size_t)t[i].n;
    add(t[i].p, each * p_bytes);
    add(t[i].m, each * state_bytes);
    add(t[i].v, each * state_bytes);
    add(t[i].master, each * 4);
    if (q8) {
      add(t[i].m_scale, (each + 255) / 256 * 4);
      add(t[i].v_scale, (each + 255) / 256 * 4);
    }
  }
  std::sort(r, r + n, [](const Range& x, const Range& y) { return x.at < y.at; });
  bool apart = true;
  for (size_t i = 1; i < n; ++i) apart = apart && r[i - 1].end <= r[i].at;
  // whether an input is apart from all of them: the first that ends behind its start starts behind its end
  auto outside = [&](const void* p, size_t bytes) {
    if (!p) return true;
    const Range* const q = std::upper_bound(r, r + n, (uintptr_t)p, [](uintptr_t at, const Range& x) { return at < x.end; });
    return q == r + n || (uintptr_t)p + bytes <= q->at;
  };
  bool inputs = true;
  for (int i = 0; apart && i < count; ++i) inputs = inputs && (!t[i].n || outside(t[i].g, (size_t)t[i].n * g_bytes));
  if (apart) inputs = inputs && outside(c->lr_dev, 4) && outside(c->step_dev, 8) && outside(c->grad_scale, 4);
  delete[] r;
  if (!apart) return fail(MOE_ERR_INVALID_ARG, "parameters, states, scales or master copies overlap");
  return inputs ? MOE_OK : fail(MOE_ERR_INVALID_ARG, "a gradient or device value overlaps an updated array");
}

}  // namespace

extern "C" {

moe_status moe_train_workspace_size(const moe_shape* shape, size_t* bytes) {
  const moe_status s = check_train_shape(shape);
  if (s != MOE_OK) return s;
  if (!bytes) return fail(MOE_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = train_ws(*shape).total;
  return MOE_OK;
}

moe_status moe_gated_ffn(const moe_shape* shape, const void* x, const int32_t* expert_offsets, const int32_t* slot_token,
                         const moe_weights* weights, void* gate_pre, void* up_pre, void* y_perm, void* ws,
                         size_t ws_bytes, moe_stream_t stream) {
  TrainArgs a;
  moe_status s = train_args(shape, x, expert_offsets, slot_token, weights, ws, ws_bytes, &a);
  if (s != MOE_OK) return s;
  if (!gate_pre != !up_pre) return fail(MOE_ERR_INVALID_ARG, "gate_pre and up_pre are kept both or not at all");
  if (!al16(gate_pre) || !al16(up_pre) || !al16(y_perm))
    return fail(MOE_ERR_INVALID_ARG, "gate_pre, up_pre and y_perm must be 16-byte aligned");
  if (a.P == 0) return MOE_OK;
  if (!y_perm) return fail(MOE_ERR_INVALID_ARG, "y_perm is NULL");
  const Sizes z(*shape, a.xrows);
  s = check_outputs({{gate_pre, z.i}, {up_pre, z.i}, {y_perm, z.h}, {ws, z.ws}},
                    {{x, z.x}, {expert_offsets, z.off}, {slot_token, z.slot}, {weights->gate, z.w}, {weights->up, z.w}, {weights->down, z.w}});
  if (s != MOE_OK) return s;
  a.g = gate_pre;
  a.u = up_pre;
  a.y = y_perm;
  const hipStream_t st = (hipStream_t)stream;
  hipError_t e = product(TF_GATE_UP, shape->act, a, st);
  if (e == hipSuccess) e = product(TF_DOWN, shape->act, a, st);
  return hip_status(e, "gated FFN");
}

moe_status moe_gated_ffn_backward(const moe_shape* shape, const void* x, const int32_t* expert_offsets,
                                  const int32_t* slot_token, const moe_weights* weights, const void* gate_pre,
                                  const void* up_pre, const void* dy_perm, void* dx_perm, const moe_weight_grads* grads,
                                  void* ws, size_t ws_bytes, moe_stream_t stream) {
  TrainArgs a;
  moe_status s = train_args(shape, x, expert_offsets, slot_token, weights, ws, ws_bytes, &a);
  if (s != MOE_OK) return s;
  if (!dx_perm && !grads) return fail(MOE_ERR_INVALID_ARG, "neither dx_perm nor grads is asked for");
  if (grads && (!grads->gate || !grads->up || !grads->down)) return fail(MOE_ERR_INVALID_ARG, "gradient pointer is NULL");
  if (a.P && (!gate_pre || !up_pre || !dy_perm)) return fail(MOE_ERR_INVALID_ARG, "gate_pre, up_pre or dy_perm is NULL");
  if (!al16(gate_pre) || !al16(up_pre) || !al16(dy_perm) || !al16(dx_perm) ||
      (grads && (!al16(grads->gate) || !al16(grads->up) || !al16(grads->down))))
    return fail(MOE_ERR_INVALID_ARG, "pre-activations and gradients must be 16-byte aligned");
  const Sizes z(*shape, a.xrows);
  s = check_outputs({{dx_perm, z.h}, {grads ? grads->gate : nullptr, z.w}, {grads ? grads->up : nullptr, z.w},
                     {grads ? grads->down : nullptr, z.w}, {ws, z.ws}},
                    {{x, z.x}, {expert_offsets, z.off}, {slot_token, z.slot}, {weights->gate, z.w}, {weights->up, z.w},
                     {weights->down, z.w}, {gate_pre, z.i}, {up_pre, z.i}, {dy_perm, z.h}});
  if (s != MOE_OK) return s;
  a.g = const_cast<void*>(gate_pre);
  a.u = const_cast<void*>(up_pre);
  a.dy = dy_perm;
  a.dx = dx_perm;
  const hipStream_t st = (hipStream_t)stream;
  if (grads) {
    a.dgate = grads->gate;
    a.dup = grads->up;
    a.ddown = grads->down;
  }
  hipError_t e = hipSuccess;
  if (a.P) e = product(TF_DH, shape->act, a, st);
  const bool dx = a.P && dx_perm;
  if (e == hipSuccess && dx && grads && shape->act == MOE_F32) {
    e = launch_gradients_f32(a, st);
  } else {
    if (e == hipSuccess && dx) e = product(TF_DX, shape->act, a, st);
    if (e == hipSuccess && grads && a.slot_token && shape->act == MOE_BF16) {
      e = launch_gather_rows(a, st);
      a.x = a.xg;
      a.slot_token = nullptr;
    }
    if (e == hipSuccess && grads) e = product(TF_DW, shape->act, a, st);  // also without rows: the gradients are zero then
  }
  return hip_status(e, "gated FFN gradient");
}

moe_status moe_combine_backward(const moe_shape* shape, const void* dy, const void* y_perm, const int32_t* pair_slot,
                                const float* topk_w, void* dy_perm, float* dtopk_w, moe_stream_t stream) {
  moe_status s = check_shape(shape);
  if (s != MOE_OK) return s;
  if (!al16(dy) || !al16(y_perm) || !al16(dy_perm))
    return fail(MOE_ERR_INVALID_ARG, "dy, y_perm and dy_perm must be 16-byte aligned");
  if (!al4(pair_slot) || !al4(topk_w) || !al4(dtopk_w))
    return fail(MOE_ERR_INVALID_ARG, "index and routing-weight arrays must be 4-byte aligned");
  if (shape->T == 0) return MOE_OK;
  if (!dy || !y_perm || !pair_slot || !topk_w || !dy_perm || !dtopk_w) return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
  const size_t P = (size_t)shape->T * shape->k, row = (size_t)shape->H * (shape->act == MOE_F32 ? 4 : 2);
  // a pair's weight is read before its gradient is written, so the gradient may take its place
  s = check_outputs({{dy_perm, P * row}, {dtopk_w, P * 4}},
                    {{dy, shape->T * row}, {y_perm, P * row}, {pair_slot, P * 4}, {topk_w == dtopk_w ? nullptr : topk_w, P * 4}});
  if (s != MOE_OK) return s;
  return hip_status(launch_combine_backward(shape->act, dy, y_perm, pair_slot, topk_w, dy_perm, dtopk_w, shape->T,
                                            shape->H, shape->k, (hipStream_t)stream),
                    "combine gradient");
}

moe_status moe_adamw(const moe_adamw_config* c, const moe_adamw_tensor* tensors, int32_t count, moe_stream_t stream) {
  if (!c) return fail(MOE_ERR_INVALID_ARG, "config is NULL");
  if (count < 0) return fail(MOE_ERR_INVALID_ARG, "count=%d < 0", count);
  if (c->p_type != MOE_F32 && c->p_type != MOE_BF16) return fail(MOE_ERR_INVALID_ARG, "p_type must be F32 or BF16");
  if (c->g_type != MOE_F32 && c->g_type != MOE_BF16) return fail(MOE_ERR_INVALID_ARG, "g_type must be F32 or BF16");
  if (c->state != MOE_ADAM_F32 && c->state != MOE_ADAM_E4M3) return fail(MOE_ERR_INVALID_ARG, "bad state %d", (int)c->state);
  if (!(c->beta1 >= 0.0 && c->beta1 < 1.0) || !(c->beta2 >= 0.0 && c->beta2 < 1.0))
    return fail(MOE_ERR_INVALID_ARG, "beta1=%g, beta2=%g must be in [0, 1)", c->beta1, c->beta2);
  if (!(c->eps >= 0.0) || !(c->weight_decay >= 0.0) || (!c->lr_dev && !(c->lr >= 0.0)))
    return fail(MOE_ERR_INVALID_ARG, "lr=%g, eps=%g and weight_decay=%g must not be negative", c->lr, c->eps, c->weight_decay);
  // the kernel's reciprocal takes smaller divisors for 0, and an element whose m and v are 0 would become NaN
  if (c->eps > 0.0 && c->eps < 0x1p-126) return fail(MOE_ERR_INVALID_ARG, "eps=%g is neither 0 nor a normal fp32 number", c->eps);
  if (!c->step_dev && c->step < 1) return fail(MOE_ERR_INVALID_ARG, "step=%lld < 1", (long long)c->step);
  if (!al4(c->lr_dev) || !al4(c->grad_scale) || (uintptr_t)c->step_dev % 8)
    return fail(MOE_ERR_INVALID_ARG, "lr_dev and grad_scale must be 4-byte and step_dev 8-byte aligned");
  if (count == 0) return MOE_OK;
  if (!tensors) return fail(MOE_ERR_INVALID_ARG, "tensors is NULL");
  const bool q8 = c->state == MOE_ADAM_E4M3;
  int master = -1;
  for (int i = 0; i < count; ++i) {
    const moe_adamw_tensor& t = tensors[i];
    if (t.n < 0 || t.n > (1LL << 40)) return fail(MOE_ERR_INVALID_ARG, "tensor %d: n=%lld outside [0, 2^40]", i, (long long)t.n);
    if (t.n == 0) continue;
    if (!t.p || !t.g || !t.m || !t.v || (q8 && (!t.m_scale || !t.v_scale)))
      return fail(MOE_ERR_INVALID_ARG, "tensor %d: NULL pointer", i);
    if (!al16(t.p) || !al16(t.g) || !al16(t.m) || !al16(t.v) || !al16(t.master) || !al4(t.m_scale) || !al4(t.v_scale))
      return fail(MOE_ERR_INVALID_ARG, "tensor %d: p, g, m, v and master must be 16-byte, scales 4-byte aligned", i);
    if (master >= 0 && master != (t.master != nullptr))
      return fail(MOE_ERR_INVALID_ARG, "tensor %d: either every tensor has a master copy or none", i);
    master = t.master != nullptr;
  }
  if (master < 0) return MOE_OK;  // only empty tensors
  if (master && c->p_type == MOE_F32) return fail(MOE_ERR_INVALID_ARG, "F32 parameters take no master copy");
  const moe_status s = check_apart(c, tensors, count);
  if (s != MOE_OK) return s;

  AdamArgs a{};
  a.lr = (float)c->lr;
  a.beta1 = (float)c->beta1;
  a.beta2 = (float)c->beta2;
  a.one_minus_beta1 = (float)(1.0 - c->beta1);
  a.one_minus_beta2 = (float)(1.0 - c->beta2);
  a.eps = (float)c->eps;
  a.wd = (float)c->weight_decay;
  a.log_beta1 = (float)log(c->beta1);
  a.log_beta2 = (float)log(c->beta2);
  a.seed = c->seed;
  a.step = c->step;
  if (!c->step_dev) {
    a.bc1 = (float)(1.0 - pow(c->beta1, (double)c->step));
    a.inv_root_bc2 = (float)(1.0 / sqrt(1.0 - pow(c->beta2, (double)c->step)));
  }
  a.lr_dev = c->lr_dev;
  a.step_dev = c->step_dev;
  a.grad_scale = c->grad_scale;
  int64_t elements = 0;
  for (int i = 0; i < count; ++i) elements += tensors[i].n;
  const int chunk = adamw_chunk(elements);
  a.passes = adamw_passes(chunk);
  hipError_t e = hipSuccess;
  long long groups = 0;
  auto flush = [&] {
    if (a.count && e == hipSuccess) e = launch_adamw(c->p_type, c->g_type, master == 1, q8, a, (hipStream_t)stream);
    a.count = 0;
    groups = 0;
  };
  for (int i = 0; i < count; ++i) {
    const moe_adamw_tensor& t = tensors[i];
    if (t.n == 0) continue;
    const long long need = (t.n + chunk - 1) / chunk;
    if (a.count == ADAM_MAX || groups + need > 0x7fffffff) flush();
    a.t[a.count] = AdamTensor{t.p, t.g, t.m, t.v, t.m_scale, t.v_scale, t.master, t.n};
    a.first[a.count++] = (int)groups;
    groups += need;
    a.first[a.count] = (int)groups;
  }
  flush();
  return hip_status(e, "AdamW");
}

}  // extern "C"
