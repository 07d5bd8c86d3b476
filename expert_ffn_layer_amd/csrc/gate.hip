// The gate of one layer and its gradient. Per token, with logits l, s = 1 / (1 + e^-l) or the softmax of l, choice
// c = s + b (l itself without a bias: the same order):
//   a group's value is its largest c or the sum of its two largest; the best groups stay; the k largest c in them are chosen
//   w_j = scale s_j, divided by the sum of the chosen s where the rule says so.
// Scores and choices are formed in 64 bits, so that the order is that of the real numbers wherever two choices differ by
// more than about 2^-50. Order keys are those doubles as unsigned integers: 0 for an expert that is off (logit or bias
// -inf), the largest for NaN.
// A wave takes a token; lane l holds experts l, l + 64, ...
#include "gate.h"

namespace moe {

namespace {

constexpr int WAVES = 4;
constexpr uint64_t KEY_NAN = ~0ull;

__device__ __forceinline__ uint64_t order_key(double v) {
  if (v != v) return KEY_NAN;
  const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);  // -0 and 0 are equal
  return (u >> 63) ? ~u : u | (1ull << 63);
}
__device__ __forceinline__ double key_value(uint64_t k) {
  if (k == KEY_NAN) return __longlong_as_double(0x7FF8000000000000ll);
  return __longlong_as_double((long long)((k >> 63) ? k & ~(1ull << 63) : ~k));
}

__device__ __forceinline__ double sigmoid64(double l) { return 1.0 / (1.0 + exp(-l)); }

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  return v;
}
// NaN if any is
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const float o = __shfl_xor(v, d);
    v = v != v ? v : (o != o || o > v) ? o : v;
  }
  return v;
}

template <int PL>
__global__ void __launch_bounds__(64 * WAVES) gate_kernel(const GateArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const long long t = (long long)blockIdx.x * WAVES + wave;
  extern __shared__ uint64_t shared_keys[];
  uint64_t* const keys = shared_keys + (size_t)wave * a.E;
  if (t >= a.T) return;  // no barrier below: a wave works alone
  const int E = a.E;
  float l[PL];
  uint64_t key[PL];
#pragma unroll
  for (int j = 0; j < PL; ++j) {
    const int e = lane + 64 * j;
    l[j] = -INFINITY;
    if (e < E) {
      float v = 0.f;
      for (int p = 0; p < a.nparts; ++p) v += a.logits[((size_t)p * a.T + t) * a.ldl + e];
      l[j] = v;
      if (a.sums) a.sums[t * E + e] = v;
    }
  }
  double m = 0.0, inv = 1.0;  // softmax: s = e^(l - m) inv
  if (!a.sigmoid) {
    float top = l[0];
#pragma unroll
    for (int j = 1; j < PL; ++j) top = top != top ? top : (l[j] != l[j] || l[j] > top) ? l[j] : top;
    top = wave_max(top);
    m = top == -INFINITY ? 0.0 : (double)top;
    double z = 0.0;
#pragma unroll
    for (int j = 0; j < PL; ++j) z += l[j] == -INFINITY ? 0.0 : exp((double)l[j] - m);
    inv = 1.0 / wave_sum(z);
  }
  const bool by_score = a.bias || (a.groups > 1 && a.group_top == 2);
#pragma unroll
  for (int j = 0; j < PL; ++j) {
    const int e = lane + 64 * j;
    key[j] = 0;
    if (e >= E || l[j] == -INFINITY) continue;
    const float b = a.bias ? a.bias[e] : 0.f;
    if (b == -INFINITY) continue;
    const double s = !by_score ? (double)l[j] : a.sigmoid ? sigmoid64(l[j]) : exp((double)l[j] - m) * inv;
    key[j] = order_key(s + (double)b);
  }
  if (a.groups > 1) {
    const int n = E / a.groups;
#pragma unroll
    for (int j = 0; j < PL; ++j)
      if (lane + 64 * j < E) keys[lane + 64 * j] = key[j];
    __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    uint64_t mine = 0;
    if (lane < a.groups) {
      uint64_t first = 0, second = 0;
      for (int i = 0; i < n; ++i) {
        const uint64_t v = keys[lane * n + i];
        if (v > first) {
          second = first;
          first = v;
        } else if (v > second) {
          second = v;
        }
      }
      mine = a.group_top == 2 && second ? order_key(key_value(first) + key_value(second)) : first;
    }
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
      const uint64_t v = __shfl(mine, g);
      rank += v > mine || (v == mine && g < lane);
    }
    const uint64_t stays = __ballot(lane < a.groups && rank < a.top_groups);
#pragma unroll
    for (int j = 0; j < PL; ++j)
      if (lane + 64 * j < E && !((stays >> ((lane + 64 * j) / n)) & 1)) key[j] = 0;
    // the scores were needed for the groups only: without a bias the logits order the experts
  }
  // k rounds: the largest key, the lowest index among equals
  uint32_t taken = 0;  // of this lane's experts
  int left = a.k;
  for (int r = 0; r < a.k; ++r) {
    uint64_t best = 0;
    int at = 1 << 30;
#pragma unroll
    for (int j = 0; j < PL; ++j)
      if (!((taken >> j) & 1) && key[j] > best) {
        best = key[j];
        at = lane + 64 * j;
      }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint64_t v = __shfl_xor(best, d);
      const int o = __shfl_xor(at, d);
      if (v > best || (v == best && o < at)) {
        best = v;
        at = o;
      }
    }
    if (best == 0) break;
    --left;
    if ((at & 63) == lane) taken |= 1u << (at >> 6);
  }
  // weights: e^(x - most) / (1 + e^-|l|) for a sigmoid with x = min(l, 0), e^(l - m) for a softmax; only the ratio
  // to the sum is taken where weights are renormalised, with the largest exponent as 0
  double most = m;
  if (a.renormalize) {
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < PL; ++j)
      if ((taken >> j) & 1) {
        const float x = a.sigmoid && l[j] > 0.f ? 0.f : l[j];
        top = top != top ? top : (x != x || x > top) ? x : top;
      }
    top = wave_max(top);
    most = top == -INFINITY ? 0.0 : (double)top;
  }
  double s[PL], sum = 0.0;
#pragma unroll
  for (int j = 0; j < PL; ++j) {
    s[j] = 0.0;
    if ((taken >> j) & 1) {
      const double v = l[j];
      if (!a.sigmoid) s[j] = exp(v - most);
      else if (!a.renormalize) s[j] = sigmoid64(v);
      else s[j] = exp((v > 0.0 ? 0.0 : v) - most) / (1.0 + exp(-__builtin_fabs(v)));
    }
    sum += s[j];
  }
  // inv is NaN for a softmax of NaN or infinity
  const double factor = a.scale * (a.renormalize ? (inv != inv ? inv : 1.0 / wave_sum(sum)) : inv);
  int base = 0;
#pragma unroll
  for (int j = 0; j < PL; ++j) {
    const uint64_t pick = __ballot((taken >> j) & 1);
    if ((taken >> j) & 1) {
      const int rank = base + __popcll(pick & ((1ull << lane) - 1));
      a.idx[t * a.k + rank] = lane + 64 * j;
      a.w[t * a.k + rank] = (float)(s[j] * factor);
    }
    base += __popcll(pick);
  }
  if (lane >= a.k - left && lane < a.k) {
    a.idx[t * a.k + lane] = -1;
    a.w[t * a.k + lane] = 0.f;
  }
}

// dl_e = ds/dl by the chosen weights' gradient; r_j = s_j / (sum of the chosen s):
//   sigmoid, renormalised  scale r_j (1 - s_j) (dw_j - sum_i r_i dw_i)      else  scale s_j (1 - s_j) dw_j
//   softmax, renormalised  scale r_j (dw_j - sum_i r_i dw_i)                else  scale p_e ([e chosen] dw_e - sum_i p_i dw_i)
// Lane j < k holds the j-th chosen expert; every lane then writes the experts lane, lane + 64, ...
__global__ void __launch_bounds__(64 * WAVES) gate_backward_kernel(const GateArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, E = a.E, k = a.k;
  const long long t = (long long)blockIdx.x * WAVES + wave;
  if (t >= a.T) return;
  const float* const row = a.logits + t * a.ldl;
  const bool dense = !a.sigmoid && !a.renormalize;
  int e = -1;
  float l = -INFINITY;
  double dw = 0.0;
  if (lane < k) {
    e = a.chosen[t * k + lane];
    if (e < 0 || e >= E) e = -1;
    else l = row[e];
    if (l == -INFINITY) e = -1;
    if (e >= 0) dw = a.dw[t * k + lane];
  }
  double m = 0.0, inv = 1.0;
  if (dense) {
    float top = -INFINITY;
    for (int i = lane; i < E; i += 64) {
      const float v = row[i];
      top = top != top ? top : (v != v || v > top) ? v : top;
    }
    top = wave_max(top);
    m = top == -INFINITY ? 0.0 : (double)top;
    double z = 0.0;
    for (int i = lane; i < E; i += 64) z += row[i] == -INFINITY ? 0.0 : exp((double)row[i] - m);
    inv = 1.0 / wave_sum(z);
  } else if (a.renormalize) {
    const float x = a.sigmoid && l > 0.f ? 0.f : l;
    const float top = wave_max(e >= 0 ? x : -INFINITY);
    m = top == -INFINITY ? 0.0 : (double)top;
  }
  double r = 0.0, rest = 1.0;  // score (over the sum), 1 - score
  if (e >= 0) {
    const double v = l;
    if (!a.sigmoid) {
      r = exp(v - m) * inv;
    } else {
      const double q = exp(-__builtin_fabs(v));
      rest = (v > 0.0 ? q : 1.0) / (1.0 + q);
      r = a.renormalize ? exp((v > 0.0 ? 0.0 : v) - m) / (1.0 + q) : (v > 0.0 ? 1.0 : q) / (1.0 + q);
    }
  }
  if (a.renormalize) {
    const double z = wave_sum(r);
    r = e >= 0 ? r / z : 0.0;
  }
  const double mean = a.renormalize || dense ? wave_sum(r * dw) : 0.0;
  double d;
  if (dense) d = dw;
  else d = a.scale * r * (a.sigmoid ? rest : 1.0) * (dw - mean);
  if (e < 0) d = 0.0;
  for (int i0 = 0; i0 < E; i0 += 64) {
    const int i = i0 + lane;
    double out = 0.0;
    for (int j = 0; j < k; ++j) {
      const int ej = __shfl(e, j);
      const double dj = __shfl(d, j);
      if (ej == i) out += dj;
    }
    if (i >= E) break;
    if (dense) out = row[i] == -INFINITY ? 0.0 : a.scale * exp((double)row[i] - m) * inv * (out - mean);
    a.dlogits[t * E + i] = (float)out;
  }
}

}  // namespace

hipError_t launch_gate(const GateArgs& a, hipStream_t st) {
  if (a.T == 0) return hipSuccess;
  const dim3 grid((unsigned)((a.T + WAVES - 1) / WAVES)), block(64 * WAVES);
  const size_t lds = a.groups > 1 ? (size_t)WAVES * a.E * 8 : 0;
  const int pl = (a.E + 63) / 64;
#define MOE_GATE(PL) gate_kernel<PL><<<grid, block, lds, st>>>(a)
  if (pl <= 1) MOE_GATE(1);
  else if (pl <= 2) MOE_GATE(2);
  else if (pl <= 4) MOE_GATE(4);
  else if (pl <= 8) MOE_GATE(8);
  else MOE_GATE(16);
#undef MOE_GATE
  return hipGetLastError();
}

hipError_t launch_gate_backward(const GateArgs& a, hipStream_t st) {
  if (a.T == 0) return hipSuccess;
  gate_backward_kernel<<<dim3((unsigned)((a.T + WAVES - 1) / WAVES)), dim3(64 * WAVES), 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace moe
