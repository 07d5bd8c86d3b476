// The C entry points of the orthogonalisation and the Muon step (include/moe.h): argument checks, workspace and
// launches. Host code only.
#include <math.h>

#include <algorithm>
#include <new>

#include "api_util.h"
#include "muon.h"

using namespace moe;

namespace {

size_t up(size_t x) { return (x + WS_ALIGN - 1) / WS_ALIGN * WS_ALIGN; }

// Matrices of one size class, and what the workspace holds of a chunk of them
struct Class {
  int M, N, Mp, Np, chunk, parts;
  int kept;  // thin matrices: those that there is room for in xs
  bool split;
  size_t sums, q, xs, x, x_lo, xo, xo_lo, A, A_lo, C, C_lo, da, dc, partial, total;
};

Class class_of(int rows, int cols, long long count, bool split) {
  Class c{};
  c.M = std::min(rows, cols);
  c.N = std::max(rows, cols);
  c.Mp = (c.M + MUON_PAD - 1) / MUON_PAD * MUON_PAD;
  c.Np = (c.N + MUON_PAD - 1) / MUON_PAD * MUON_PAD;
  c.split = split;
  if (!muon_thin(c.M, c.N) && muon_small(c.M, c.N)) {
    c.chunk = (int)std::min<long long>(count, 65535);  // a launch's grid
    return c;
  }
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += up(bytes);
    return at;
  };
  if (muon_thin(c.M, c.N)) {
    // within 256 MiB, and a launch's grid
    const int side = thin_side(c.M), part = thin_part(c.N);
    c.parts = (c.N + part - 1) / part;
    const size_t square = (size_t)side * side * 8, each = (c.parts + 1) * square;
    c.chunk = (int)std::min<long long>(std::min<long long>(std::max<long long>((long long)((256ull << 20) / each), 1), 65535), count);
    c.sums = take(c.chunk * c.parts * square);
    c.q = take(c.chunk * (square + 8));
    // X between runs of steps, which few calls have: within 256 MiB of its own, whatever the chunk
    const size_t x = (size_t)c.M * c.N * 8;
    c.kept = (int)std::min<long long>(std::max<long long>((long long)((256ull << 20) / x), 1), c.chunk);
    c.xs = take(c.kept * x);
    c.total = o;
    return c;
  }
  const size_t xb = (size_t)c.Np * c.Mp * 2, ab = (size_t)c.Mp * c.Mp * 2;
  // As many matrices at a time as give the symmetric products, which have the fewest tiles, about 4 rounds of the
  // card, within 4 GiB
  const long long t = (c.Mp + 255) / 256, tiles = t * (t + 1) / 2;
  const size_t each = (split ? 4 : 3) * xb + (split ? 4 : 2) * ab;
  long long n = std::max<long long>((1152 + tiles - 1) / tiles, 1);
  n = std::min<long long>(n, std::max<long long>((long long)((4ull << 30) / each), 1));
  c.chunk = (int)std::min(n, count);
  const size_t k = c.chunk;
  c.parts = muon_parts((long long)c.M * c.N);
  c.sums = take(k * c.parts * 8);
  c.da = take(k * c.Mp * 4);
  c.dc = take(k * c.Mp * 4);
  c.x = take(k * xb);
  c.x_lo = take(k * xb);
  c.xo = take(k * xb);
  c.xo_lo = split ? take(k * xb) : c.x_lo;
  c.A = take(k * ab);
  c.C = take(k * ab);
  c.A_lo = split ? take(k * ab) : c.A;
  c.C_lo = split ? take(k * ab) : c.C;
  // of a whole chunk and of the last
  const int last = (int)(count % c.chunk);
  c.partial = take(2 * (size_t)std::max(muon_runs(c.Mp, c.Np, c.chunk, split), last ? muon_runs(c.Mp, c.Np, last, split) : 0) * 128 * 128 * 4);
  c.total = o;
  return c;
}

moe_status check_sizes(int32_t count, int32_t rows, int32_t cols) {
  if (count < 0 || rows < 0 || cols < 0) return fail(MOE_ERR_INVALID_ARG, "count=%d, rows=%d, cols=%d must not be negative", count, rows, cols);
  if (std::min(rows, cols) > 32768 || std::max(rows, cols) > (1 << 20))
    return fail(MOE_ERR_UNSUPPORTED, "%d x %d: the shorter side is at most 32768, the longer 2^20", rows, cols);
  return MOE_OK;
}

// What a step makes of singular values up to `top`: the largest, and the polynomial's largest value
struct StepRange {
  double most, poly;
};
StepRange step_range(const moe_newton_schulz& ns, double top) {
  const double a = ns.a, b = ns.b, c = ns.c, t1 = top * top;
  auto f = [&](double t) { return t >= 0.0 && t <= t1 ? fabs(sqrt(t) * (a + t * (b + t * c))) : 0.0; };
  auto g = [&](double t) { return t >= 0.0 && t <= t1 ? fabs(a + t * (b + t * c)) : 0.0; };
  StepRange r{f(t1), std::max(std::max(g(0.0), g(t1)), c != 0.0 ? g(-b / (2.0 * c)) : 0.0)};
  // where d/ds (a s + b s^3 + c s^5) = a + 3 b t + 5 c t^2 is 0
  const double d = 9.0 * b * b - 20.0 * a * c;
  if (c != 0.0 && d >= 0.0) {
    r.most = std::max(r.most, std::max(f((-3.0 * b + sqrt(d)) / (10.0 * c)), f((-3.0 * b - sqrt(d)) / (10.0 * c))));
  } else if (c == 0.0 && b != 0.0) {
    r.most = std::max(r.most, f(-a / (3.0 * b)));
  }
  return r;
}
// The bound on the next step's singular values: a step's rounding is far below the 2% that each is given.
double next_top(const StepRange& r) { return std::max(r.most * 1.02, 1e-3); }

// The steps keep X, A and C within fp16 at MUON_SCALE: 15.99. From singular values up to 1.
moe_status check_ns(const moe_newton_schulz* ns) {
  if (!ns) return fail(MOE_ERR_INVALID_ARG, "Newton-Schulz parameters are NULL");
  if (ns->steps < 1 || ns->steps > 32) return fail(MOE_ERR_INVALID_ARG, "steps=%d outside 1..32", ns->steps);
  if (!isfinite(ns->a) || !isfinite(ns->b) || !isfinite(ns->c)) return fail(MOE_ERR_INVALID_ARG, "coefficients must be finite");
  if (!(ns->eps >= 0.0) || !isfinite(ns->eps)) return fail(MOE_ERR_INVALID_ARG, "eps=%g must be finite and not negative", ns->eps);
  double top = 1.0;
  for (int i = 0; i < ns->steps; ++i) {
    const StepRange r = step_range(*ns, top);
    if (!(r.poly <= 14.0) || !(r.most * 1.02 <= 3.7))
      return fail(MOE_ERR_UNSUPPORTED, "coefficients %g, %g, %g take a singular value to %g and the polynomial to %g in step %d: "
                  "3.7 and 14 are the most", ns->a, ns->b, ns->c, r.most, r.poly, i + 1);
    top = next_top(r);
  }
  return MOE_OK;
}

// Equal runs of steps that thin matrices take, each short enough that an eigenvalue's rounding, 2^-53, grows by 2^29 at most:
// in a step by the derivative of t (a + b t + c t^2)^2 = (a + b t + c t^2) (a + 3 b t + 5 c t^2), here at 65 points of the range.
int thin_runs(const moe_newton_schulz& ns) {
  double top = 1.0, widest = 1.0, growth = 1.0;
  for (int i = 1; i < ns.steps; ++i) widest = std::max(widest, top = next_top(step_range(ns, top)));
  for (int i = 0; i <= 64; ++i) {
    const double t = widest * widest * i / 64;
    growth = std::max(growth, fabs((ns.a + t * (ns.b + t * ns.c)) * (ns.a + t * (3.0 * ns.b + t * 5.0 * ns.c))));
  }
  int most = 1;
  for (double all = growth * growth; most < ns.steps && all <= 0x1p29; all *= growth) ++most;
  return (ns.steps + most - 1) / most;
}

// All steps of the matrices of one class, `total` of them in the stacks of a, the first `wide` with their short side first.
hipError_t run_class(MuonArgs a, const Class& c, const moe_newton_schulz& ns, int total, int wide, void* ws, hipStream_t st) {
  char* const w = (char*)ws;
  a.M = c.M;
  a.N = c.N;
  a.Mp = c.Mp;
  a.Np = c.Np;
  a.split = c.split;
  a.parts = c.parts;
  a.eps = ns.eps;
  a.a = ns.a;
  a.b = ns.b;
  a.c = ns.c;
  a.sums = (double*)(w + c.sums);
  a.da = (float*)(w + c.da);
  a.dc = (float*)(w + c.dc);
  a.A = (uint16_t*)(w + c.A);
  a.A_lo = (uint16_t*)(w + c.A_lo);
  a.C = (uint16_t*)(w + c.C);
  a.C_lo = (uint16_t*)(w + c.C_lo);
  a.partial = (float*)(w + c.partial);
  hipError_t e = hipSuccess;
  if (muon_thin(c.M, c.N)) {
    a.q = (double*)(w + c.q);
    a.part = thin_part(c.N);
    const int runs = thin_runs(ns), chunk = runs > 1 ? c.kept : c.chunk;
    a.xs = (double*)(w + c.xs);
    for (long long first = 0; first < total && e == hipSuccess; first += chunk) {
      a.first = (int)first;
      a.count = (int)std::min<long long>(chunk, total - first);
      e = launch_muon_thin(a, ns.steps, runs, st);
    }
    return e;
  }
  if (muon_small(c.M, c.N)) {
    for (long long first = 0; first < total && e == hipSuccess; first += c.chunk) {
      a.first = (int)first;
      a.count = (int)std::min<long long>(c.chunk, total - first);
      e = launch_muon_small(a, ns.steps, st);
    }
    return e;
  }
  for (long long first = 0; first < total && e == hipSuccess; first += c.chunk) {
    a.first = (int)first;
    a.count = (int)std::min<long long>(c.chunk, total - first);
    a.x = (uint16_t*)(w + c.x);
    a.x_lo = (uint16_t*)(w + c.x_lo);
    a.xo = (uint16_t*)(w + c.xo);
    a.xo_lo = (uint16_t*)(w + c.xo_lo);
    a.runs = muon_runs(c.Mp, c.Np, a.count, c.split);
    e = launch_muon_momentum(a, st);
    if (e == hipSuccess) e = launch_muon_normalize(a, st);
    for (int i = 0; i < ns.steps && e == hipSuccess; ++i) {
      const bool last = i + 1 == ns.steps;
      a.whole_c = last;
      e = launch_muon_product(MF_GRAM, a, st);
      if (e == hipSuccess) e = launch_muon_product(MF_POLY, a, st);
      if (e != hipSuccess || last) break;
      MuonArgs s = a;
      if (!c.split && i + 2 == ns.steps) s.xo_lo = nullptr;  // the last step reads x alone
      e = launch_muon_product(MF_STEP, s, st);
      std::swap(a.x, a.xo);
      std::swap(a.x_lo, a.xo_lo);
    }
    // the matrices that are wide, then the others
    const int n = (int)std::min<long long>(std::max<long long>(wide - first, 0), a.count), all = a.count;
    for (int turned = 0; turned < 2 && e == hipSuccess; ++turned) {
      a.turned = turned;
      a.skip = turned ? n : 0;
      a.count = turned ? all - n : n;
      if (a.count) e = launch_muon_product(MF_LAST, a, st);
    }
    a.skip = 0;
  }
  return e;
}

moe_status check_muon_ws(void* ws, size_t ws_bytes, size_t need) {
  if (!need) return MOE_OK;
  if (!ws) return fail(MOE_ERR_INVALID_ARG, "workspace is NULL");
  if (ws_bytes < need) return fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < %zu needed", ws_bytes, need);
  if (!aligned(ws, WS_ALIGN)) return fail(MOE_ERR_INVALID_ARG, "workspace must be %zu-byte aligned", WS_ALIGN);
  return MOE_OK;
}

moe_status check_type(moe_dtype t, const char* what) {
  return t == MOE_F32 || t == MOE_BF16 ? MOE_OK : fail(MOE_ERR_INVALID_ARG, "%s must be F32 or BF16", what);
}
size_t bytes_of(moe_dtype t) { return t == MOE_F32 ? 4 : 2; }

bool empty(const moe_muon_tensor& t) { return !t.count || !t.rows || !t.cols; }
bool same_class(const moe_muon_tensor& a, const moe_muon_tensor& b) {
  return std::min(a.rows, a.cols) == std::min(b.rows, b.cols) && std::max(a.rows, a.cols) == std::max(b.rows, b.cols);
}
// f(the stacks of a class that go together, how many, their matrices), class by class
template <typename F>
moe_status each_class(const moe_muon_tensor* t, int32_t count, F f) {
  bool* const done = new (std::nothrow) bool[(size_t)count]();
  if (!done) return fail(MOE_ERR_INVALID_ARG, "no host memory to sort %d stacks", count);
  moe_status r = MOE_OK;
  for (int i = 0; i < count && r == MOE_OK; ++i) {
    if (done[i] || empty(t[i])) continue;
    int of[MUON_STACKS], n = 0;
    long long matrices = 0;
    for (int j = i; j < count && n < MUON_STACKS; ++j) {
      if (done[j] || empty(t[j]) || !same_class(t[i], t[j]) || matrices + t[j].count > 0x7fffffff) continue;
      of[n++] = j;
      done[j] = true;
      matrices += t[j].count;
    }
    r = f(of, n, (int)matrices);
  }
  delete[] done;
  return r;
}

moe_status muon_need(moe_dtype p_type, const moe_muon_tensor* t, int32_t count, size_t* bytes) {
  for (int i = 0; i < count; ++i) {
    const moe_status r = check_sizes(t[i].count, t[i].rows, t[i].cols);
    if (r != MOE_OK) return r;
  }
  size_t need = 0;
  const moe_status r = each_class(t, count, [&](const int* of, int, int matrices) {
    need = std::max(need, class_of(t[of[0]].rows, t[of[0]].cols, matrices, p_type == MOE_F32).total);
    return MOE_OK;
  });
  *bytes = need;
  return r;
}

// No two of the updated arrays, the workspace being one, share memory, and none holds an input.
moe_status check_muon_apart(const moe_muon_config* c, const moe_muon_tensor* t, int count, Span ws) {
  struct Range {
    uintptr_t at, end;
  };
  Range* const r = new (std::nothrow) Range[3 * (size_t)count + 1];
  if (!r) return fail(MOE_ERR_INVALID_ARG, "no host memory to check %d stacks", count);
  size_t n = 0;
  auto add = [&](const void* p, size_t bytes) {
    if (p && bytes) r[n++] = Range{(uintptr_t)p, (uintptr_t)p + bytes};
  };
  auto elements = [](const moe_muon_tensor& x) { return (size_t)x.count * x.rows * x.cols; };
  add(ws.p, ws.bytes);
  for (int i = 0; i < count; ++i) {
    add(t[i].p, elements(t[i]) * bytes_of(c->p_type));
    add(t[i].m, elements(t[i]) * 4);
    add(t[i].master, elements(t[i]) * 4);
  }
  std::sort(r, r + n, [](const Range& x, const Range& y) { return x.at < y.at; });
  bool apart = true;
  for (size_t i = 1; i < n; ++i) apart = apart && r[i - 1].end <= r[i].at;
  // the first range that ends behind an input's start starts behind its end
  auto outside = [&](const void* p, size_t bytes) {
    if (!p || !bytes) return true;
    const Range* const q = std::upper_bound(r, r + n, (uintptr_t)p, [](uintptr_t at, const Range& x) { return at < x.end; });
    return q == r + n || (uintptr_t)p + bytes <= q->at;
  };
  bool inputs = true;
  for (int i = 0; apart && i < count; ++i) inputs = inputs && outside(t[i].g, elements(t[i]) * bytes_of(c->g_type));
  if (apart) inputs = inputs && outside(c->lr_dev, 4) && outside(c->grad_scale, 4);
  delete[] r;
  if (!apart) return fail(MOE_ERR_INVALID_ARG, "parameters, momenta, master copies or the workspace overlap");
  return inputs ? MOE_OK : fail(MOE_ERR_INVALID_ARG, "a gradient or device value overlaps an updated array or the workspace");
}

}  // namespace

extern "C" {

moe_status moe_orthogonalize_workspace_size(moe_dtype type, int32_t count, int32_t rows, int32_t cols, size_t* bytes) {
  moe_status s = check_type(type, "type");
  if (s != MOE_OK) return s;
  if ((s = check_sizes(count, rows, cols)) != MOE_OK) return s;
  if (!bytes) return fail(MOE_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = count && rows && cols ? class_of(rows, cols, count, type == MOE_F32).total : 0;
  return MOE_OK;
}

moe_status moe_orthogonalize(const moe_newton_schulz* ns, moe_dtype type, int32_t count, int32_t rows, int32_t cols,
                             const void* g, void* o, void* ws, size_t ws_bytes, moe_stream_t stream) {
  moe_status s = check_ns(ns);
  if (s != MOE_OK) return s;
  if ((s = check_type(type, "type")) != MOE_OK) return s;
  if ((s = check_sizes(count, rows, cols)) != MOE_OK) return s;
  if (!aligned(g, 16) || !aligned(o, 16)) return fail(MOE_ERR_INVALID_ARG, "g and o must be 16-byte aligned");
  if (!count || !rows || !cols) return MOE_OK;
  if (!g || !o) return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
  const Class c = class_of(rows, cols, count, type == MOE_F32);
  if ((s = check_muon_ws(ws, ws_bytes, c.total)) != MOE_OK) return s;
  const size_t bytes = (size_t)count * rows * cols * bytes_of(type);
  if ((s = check_outputs({{o, bytes}, {ws, c.total}}, {{g, bytes}})) != MOE_OK) return s;
  MuonArgs a{};
  a.s[0] = MuonStack{g, nullptr, o, nullptr, 1.f, 0, rows < cols};
  a.stacks = 1;
  a.g_f32 = a.out_f32 = type == MOE_F32;
  return hip_status(run_class(a, c, *ns, count, rows < cols ? count : 0, ws, (hipStream_t)stream), "orthogonalisation");
}

moe_status moe_muon_workspace_size(moe_dtype p_type, const moe_muon_tensor* tensors, int32_t count, size_t* bytes) {
  const moe_status s = check_type(p_type, "p_type");
  if (s != MOE_OK) return s;
  if (count < 0) return fail(MOE_ERR_INVALID_ARG, "count=%d < 0", count);
  if (!bytes || (count && !tensors)) return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
  return muon_need(p_type, tensors, count, bytes);
}

moe_status moe_muon(const moe_muon_config* c, const moe_muon_tensor* tensors, int32_t count, void* ws, size_t ws_bytes,
                    moe_stream_t stream) {
  if (!c) return fail(MOE_ERR_INVALID_ARG, "config is NULL");
  moe_status s = check_ns(&c->ns);
  if (s != MOE_OK) return s;
  if ((s = check_type(c->p_type, "p_type")) != MOE_OK || (s = check_type(c->g_type, "g_type")) != MOE_OK) return s;
  if (!(c->momentum >= 0.0 && c->momentum < 1.0)) return fail(MOE_ERR_INVALID_ARG, "momentum=%g must be in [0, 1)", c->momentum);
  if (!(c->weight_decay >= 0.0) || (!c->lr_dev && !(c->lr >= 0.0)))
    return fail(MOE_ERR_INVALID_ARG, "lr=%g and weight_decay=%g must not be negative", c->lr, c->weight_decay);
  if (c->nesterov != 0 && c->nesterov != 1) return fail(MOE_ERR_INVALID_ARG, "nesterov=%d is neither 0 nor 1", c->nesterov);
  if (!aligned(c->lr_dev, 4) || !aligned(c->grad_scale, 4)) return fail(MOE_ERR_INVALID_ARG, "lr_dev and grad_scale must be 4-byte aligned");
  if (count < 0) return fail(MOE_ERR_INVALID_ARG, "count=%d < 0", count);
  if (count == 0) return MOE_OK;
  if (!tensors) return fail(MOE_ERR_INVALID_ARG, "tensors is NULL");
  size_t need;
  if ((s = muon_need(c->p_type, tensors, count, &need)) != MOE_OK) return s;
  int master = -1;
  for (int i = 0; i < count; ++i) {
    const moe_muon_tensor& t = tensors[i];
    if (empty(t)) continue;
    if (!t.p || !t.g || !t.m) return fail(MOE_ERR_INVALID_ARG, "stack %d: NULL pointer", i);
    if (!aligned(t.p, 16) || !aligned(t.g, 16) || !aligned(t.m, 16) || !aligned(t.master, 16))
      return fail(MOE_ERR_INVALID_ARG, "stack %d: p, g, m and master must be 16-byte aligned", i);
    if (!isfinite(t.scale)) return fail(MOE_ERR_INVALID_ARG, "stack %d: scale=%g is not finite", i, t.scale);
    if (master >= 0 && master != (t.master != nullptr))
      return fail(MOE_ERR_INVALID_ARG, "stack %d: either every stack has a master copy or none", i);
    master = t.master != nullptr;
  }
  if (master < 0) return MOE_OK;  // only empty stacks
  if (master && c->p_type == MOE_F32) return fail(MOE_ERR_INVALID_ARG, "F32 parameters take no master copy");
  if ((s = check_muon_ws(ws, ws_bytes, need)) != MOE_OK) return s;
  if ((s = check_muon_apart(c, tensors, count, Span{ws, need})) != MOE_OK) return s;
  return each_class(tensors, count, [&](const int* of, int n, int matrices) {
    MuonArgs a{};
    a.stacks = n;
    a.g_f32 = c->g_type == MOE_F32;
    a.out_f32 = c->p_type == MOE_F32;
    a.nesterov = c->nesterov;
    a.momentum = (float)c->momentum;
    a.lr = (float)c->lr;
    a.wd = (float)c->weight_decay;
    a.lr_dev = c->lr_dev;
    a.grad_scale = c->grad_scale;
    int first = 0, wide = 0, at = 0;
    for (int turned = 0; turned < 2; ++turned)
      for (int i = 0; i < n; ++i) {
        const moe_muon_tensor& t = tensors[of[i]];
        if ((t.rows < t.cols) == (turned != 0)) continue;
        a.s[at++] = MuonStack{t.g, t.m, t.p, t.master, (float)t.scale, first, !turned};
        first += t.count;
        if (!turned) wide = first;
      }
    const moe_muon_tensor& t = tensors[of[0]];
    return hip_status(run_class(a, class_of(t.rows, t.cols, matrices, c->p_type == MOE_F32), c->ns, matrices, wide, ws, (hipStream_t)stream),
                      "Muon");
  });
}

}  // extern "C"
