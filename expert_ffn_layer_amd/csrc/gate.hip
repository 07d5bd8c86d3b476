// The gate of one layer and its gradient. Per token, with logits l, s = 1 / (1 + e^-l) or the softmax of l, choice
// c = s + b (l itself without a bias: the same order):
//   a group's value is its largest c or the sum of its two largest; the best groups stay; the k largest c in them are chosen
//   w_j = scale s_j, divided by the sum of the chosen s where the rule says so.
// The order is to be that of the real numbers. Choices are formed in fp32 first. Where those that border on each other (the
// last chosen and the first that is not, of experts and of groups) are further apart than fp32 can be off, the order is
// settled. The few tokens where they are not (one in 1000 of sigmoids over 256 experts) are done again, each by a whole wave,
// with choices in 64 bits; those with NaN or infinity, by order keys of 64 bits. Weights are formed of the chosen only, in 64
// bits.
#include "gate.h"

namespace moe {

namespace {

constexpr int WAVES = 4, LIST = 16;
constexpr uint64_t KEY_NAN = ~0ull;

// LDS that a wave's lanes exchange data through: its accesses run in the order in which they are issued, and this keeps
// the compiler from changing that order.
__device__ __forceinline__ void in_order() { __asm__ volatile("" ::: "memory"); }

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
// f over each run of LN lanes, in all of them
template <int LN, typename F>
__device__ __forceinline__ float reduce(float v, F f) {
  auto step = [&](uint32_t o) { v = f(v, __uint_as_float(o)); };
  if (LN > 1) step(dpp<0xB1>(__float_as_uint(v)));   // lane ^ 1
  if (LN > 2) step(dpp<0x4E>(__float_as_uint(v)));   // lane ^ 2
  if (LN > 4) step(dpp<0x141>(__float_as_uint(v)));  // the other half of 8
  if (LN > 8) step(dpp<0x140>(__float_as_uint(v)));  // the other half of 16
  if (LN > 16) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = f(__uint_as_float(p[0]), __uint_as_float(p[1]));
  }
  if (LN > 32) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = f(__uint_as_float(p[0]), __uint_as_float(p[1]));
  }
  return v;
}
__device__ __forceinline__ float larger(float a, float b) { return a > b ? a : b; }
// The largest of an array, where none is NaN; the compiler's own form would quiet every operand first
template <int N>
__device__ __forceinline__ float largest(const float (&v)[N]) {
  float m[N];
#pragma unroll
  for (int j = 0; j < N; ++j) m[j] = v[j];
#pragma unroll
  for (int n = N; n > 1; n = (n + 2) / 3) {
#pragma unroll
    for (int i = 0; i < (n + 2) / 3; ++i) {
      const float a = m[3 * i], b = m[3 * i + 1 < n ? 3 * i + 1 : 3 * i], c = m[3 * i + 2 < n ? 3 * i + 2 : 3 * i];
      if (3 * i + 1 < n) __asm__("v_max3_f32 %0, %1, %2, %3" : "=v"(m[i]) : "v"(a), "v"(b), "v"(c));
      else m[i] = a;
    }
  }
  return m[0];
}
// The same for the maximum of numbers, with the moves in the instruction; two wait states behind the one that wrote v
template <int LN>
__device__ __forceinline__ float run_max(float v) {
#define MOE_MAX(HOW) __asm__("s_nop 1\n\tv_max_f32_dpp %0, %1, %1 " HOW " row_mask:0xf bank_mask:0xf" : "=v"(v) : "v"(v))
  if (LN > 1) MOE_MAX("quad_perm:[1,0,3,2]");
  if (LN > 2) MOE_MAX("quad_perm:[2,3,0,1]");
  if (LN > 4) MOE_MAX("row_half_mirror");
  if (LN > 8) MOE_MAX("row_mirror");
#undef MOE_MAX
  if (LN > 16) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = larger(__uint_as_float(p[0]), __uint_as_float(p[1]));
  }
  if (LN > 32) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = larger(__uint_as_float(p[0]), __uint_as_float(p[1]));
  }
  return v;
}
template <int LN>
__device__ __forceinline__ float run_min(float v) { return reduce<LN>(v, [](float a, float b) { return a < b ? a : b; }); }
template <int LN>
__device__ __forceinline__ float run_sum(float v) { return reduce<LN>(v, [](float a, float b) { return a + b; }); }
// The same for 64 bits, over runs of `lanes`
template <typename F>
__device__ __forceinline__ double reduce64(double v, int lanes, F f) {
  auto both = [&](auto move) {
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = move((uint32_t)u), hi = move((uint32_t)(u >> 32));
    v = f(v, __longlong_as_double((long long)((uint64_t)hi << 32 | lo)));
  };
  if (lanes > 1) both([](uint32_t x) { return dpp<0xB1>(x); });
  if (lanes > 2) both([](uint32_t x) { return dpp<0x4E>(x); });
  if (lanes > 4) both([](uint32_t x) { return dpp<0x141>(x); });
  if (lanes > 8) both([](uint32_t x) { return dpp<0x140>(x); });
  auto halves = [&](auto swap) {
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    const auto lo = swap((uint32_t)u), hi = swap((uint32_t)(u >> 32));
    v = f(__longlong_as_double((long long)((uint64_t)hi[0] << 32 | lo[0])), __longlong_as_double((long long)((uint64_t)hi[1] << 32 | lo[1])));
  };
  if (lanes > 16) halves([](uint32_t x) { return __builtin_amdgcn_permlane16_swap(x, x, false, false); });
  if (lanes > 32) halves([](uint32_t x) { return __builtin_amdgcn_permlane32_swap(x, x, false, false); });
  return v;
}
// v of a lane that is the same for all
__device__ __forceinline__ double of_lane(double v, int lane) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane), hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
  return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}
__device__ __forceinline__ double larger64(double a, double b) { return a > b ? a : b; }
__device__ __forceinline__ double sum64(double a, double b) { return a + b; }

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
__device__ __forceinline__ float nan_max(float a, float b) { return a != a ? a : (b != b || b > a) ? b : a; }

// Place of element i of a wave's rows in LDS: 16 bytes apart every 128, so that lanes that read runs of 32 do so without
// bank conflicts
__host__ __device__ __forceinline__ int place(int i) { return i + 4 * (i >> 5); }

struct Chosen {
  int e;
  float l;
};

// A chosen expert's score of logit v, or its ratio to e^most: e^x / (1 + e^-|v|) for a sigmoid with x = min(v, 0), e^v for a
// softmax; rest: 1 - s for a sigmoid, else 1. In 64 bits a sigmoid needs no most but where all are below e^-600.
struct Score {
  double s, rest;
};
__device__ __forceinline__ float most_of(bool sigmoid, float top) { return top == -INFINITY || (sigmoid && top > -600.f) ? 0.f : top; }
__device__ __forceinline__ Score score_of(bool sigmoid, float v, float most) {
  const double e = exp(sigmoid ? -(double)__builtin_fabsf(v) : (double)v - (double)most);
  if (!sigmoid) return Score{e, 1.0};
  const double f = 1.0 / (1.0 + e);
  double s = v > 0.f ? 1.0 : e;
  if (__any(most != 0.f)) s = exp((double)(v > 0.f ? 0.f : v) - (double)most);
  return Score{s * f, (v > 0.f ? e : 1.0) * f};
}

// Weights of one token by the LN lanes q = 0.. that belong to it: list holds its n chosen in ascending order. m, inv: a
// softmax's largest logit and 1 / sum (NaN for one of NaN or infinity). Where weights are renormalised only the ratio to the
// sum is taken, so that scores that vanish keep their ratios.
// In 64 bits, rounded once: of 16384 tokens with 8 of 256 experts 15.7 us as called, in fp32 with about ten roundings 15.3.
template <int LN>
__device__ __forceinline__ void write_weights(const GateArgs& a, const Chosen* list, int n, long long t, int q, bool on, float m, double inv) {
  constexpr int PER = LIST > LN ? LIST / LN : 1;
  Chosen mine[PER];
  float top = -INFINITY;
  double s[PER], sum = 0.0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    mine[i] = Chosen{-1, -INFINITY};
    if (q + i * LN < n) mine[i] = list[q + i * LN];
    top = nan_max(top, a.sigmoid && mine[i].l > 0.f ? 0.f : mine[i].l);
  }
  float most = a.sigmoid ? 0.f : m;
  if (a.renormalize) {
    top = reduce<LN>(top, nan_max);
    most = most_of(a.sigmoid, top);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const float v = mine[i].l;
    const double score = score_of(a.sigmoid, v, most).s;
    s[i] = v == -INFINITY ? 0.0 : score;
    sum += s[i];
  }
  const double factor = a.scale * (a.renormalize ? (inv != inv ? inv : 1.0 / reduce64(sum, LN, sum64)) : inv);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = q + i * LN;
    if (on && j < a.k) {
      a.idx[t * a.k + j] = mine[i].e;
      a.w[t * a.k + j] = j < n ? (float)(s[i] * factor) : 0.f;
    }
  }
}

// One token by a whole wave, with choices in 64 bits: row(e) is its logit, keys an array of E in LDS. Order keys are the
// choices as unsigned integers: 0 for an expert that is off (logit or bias -inf), the largest for NaN.
template <typename Row>
__device__ void ordered_token(const GateArgs& a, long long t, Row row, uint64_t* keys, Chosen* list) {
  const int lane = threadIdx.x & 63, E = a.E;
  float m = 0.f;
  double inv = 1.0;
  if (!a.sigmoid) {
    float top = -INFINITY;
    for (int e = lane; e < E; e += 64) top = nan_max(top, row(e));
    top = reduce<64>(top, nan_max);
    m = top == -INFINITY ? 0.f : top;
    double z = 0.0;
    for (int e = lane; e < E; e += 64) z += row(e) == -INFINITY ? 0.0 : exp((double)row(e) - (double)m);
    inv = 1.0 / reduce64(z, 64, sum64);
  }
  auto key_of = [&](int e, bool score) {
    const float l = row(e), b = a.bias ? a.bias[e] : 0.f;
    if (l == -INFINITY || b == -INFINITY) return (uint64_t)0;
    const double s = !score ? (double)l : a.sigmoid ? sigmoid64(l) : exp((double)l - (double)m) * inv;
    return order_key(s + (double)b);
  };
  in_order();
  const bool pairs = a.groups > 1 && a.group_top == 2;
  for (int e = lane; e < E; e += 64) keys[e] = key_of(e, a.bias || pairs);
  in_order();
  if (a.groups > 1) {
    const int n = E / a.groups;
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
      mine = pairs && second ? order_key(key_value(first) + key_value(second)) : first;
    }
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
      const uint64_t v = __shfl(mine, g);
      rank += v > mine || (v == mine && g < lane);
    }
    const uint64_t stays = __ballot(lane < a.groups && rank < a.top_groups);
    in_order();
    for (int e = lane; e < E; e += 64) {
      if (!((stays >> (e / n)) & 1)) keys[e] = 0;
      else if (pairs && !a.bias) keys[e] = key_of(e, false);  // the logits order the experts
    }
    in_order();
  }
  // k rounds: the largest key, the lowest index among equals; lane r keeps the r-th
  int n = 0, mine = 1 << 30;
  for (; n < a.k; ++n) {
    uint64_t best = 0;
    int at = 1 << 30;
    for (int e = lane; e < E; e += 64) {
      const uint64_t v = keys[e];
      if (v > best) {
        best = v;
        at = e;
      }
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
    in_order();
    if ((at & 63) == lane) keys[at] = 0;
    in_order();
    if (lane == n) mine = at;
  }
  int rank = 0;
  for (int i = 0; i < n; ++i) rank += __shfl(mine, i) < mine;
  in_order();
  if (lane < n) list[rank] = Chosen{mine, row(mine)};
  in_order();
  write_weights<64>(a, list, n, t, lane, true, m, inv);
  in_order();
}

// Bytes of LDS of a wave that takes `tokens`: their rows, a list each, the keys of one
__host__ __device__ __forceinline__ int tile_floats(const GateArgs& a, int tokens) { return (place(tokens * a.ldl) + 7) / 4 * 4; }
__host__ __device__ __forceinline__ int wave_bytes(const GateArgs& a, int tokens) {
  return tile_floats(a, tokens) * 4 + tokens * LIST * (int)sizeof(Chosen) + (a.E + 1) / 2 * 16;
}

// The rows of a wave's tokens, with their parts added, to LDS and to sums
__device__ __forceinline__ void stage(const GateArgs& a, long long t0, int tokens, float* tile) {
  const int lane = threadIdx.x & 63, n = tokens * a.ldl;
  const float* const from = a.logits + t0 * a.ldl;
  const size_t part = (size_t)a.T * a.ldl;
  if (a.whole) {
    for (int i = 4 * lane; i < n; i += 256) {
      f32x4 v = *(const f32x4*)(from + i);
      for (int p = 1; p < a.nparts; ++p) v += *(const f32x4*)(from + p * part + i);
      *(f32x4*)(tile + place(i)) = v;
    }
  } else {
    for (int i = lane; i < n; i += 64) {
      float v = from[i];
      for (int p = 1; p < a.nparts; ++p) v += from[p * part + i];
      tile[place(i)] = v;
    }
  }
  in_order();
  if (a.sums)
    for (int i = lane; i < tokens * a.E; i += 64) a.sums[t0 * a.E + i] = tile[place(i / a.E * a.ldl + i % a.E)];
}

__host__ __device__ __forceinline__ int backward_wave_bytes(const GateArgs& a) {
  return (64 / LIST * a.E + 3) / 4 * 16 + 64 * 16;  // rows, and an Entry a lane
}

__global__ void __launch_bounds__(64 * WAVES) gate_exact_kernel(const GateArgs a) {
  extern __shared__ __align__(16) uint8_t lds[];
  const int wave = threadIdx.x >> 6;
  const long long t = (long long)blockIdx.x * WAVES + wave;
  if (t >= a.T) return;  // no barrier below: a wave works alone
  float* const tile = (float*)(lds + (size_t)wave * wave_bytes(a, 1));
  Chosen* const list = (Chosen*)(tile + tile_floats(a, 1));
  stage(a, t, 1, tile);
  ordered_token(a, t, [&](int e) { return tile[place(e)]; }, (uint64_t*)(list + LIST), list);
}

// Where a lane's experts are: those of one group follow each other in its LN / groups lanes, so that lanes and places
// within a lane are in the experts' order.
struct Place {
  int size, lanes, per, g, e0, n;  // experts and lanes of a group, experts of a lane; this lane's group, first expert and experts
};
template <int LN>
__device__ __forceinline__ Place place_of(const GateArgs& a, int q, bool on) {
  Place p;
  p.size = a.E / a.groups;
  p.lanes = LN / a.groups;
  p.per = (p.size + p.lanes - 1) / p.lanes;
  p.g = q / p.lanes;
  const int before = q % p.lanes * p.per;
  p.e0 = p.g * p.size + before;
  p.n = !on || before >= p.size ? 0 : p.size - before < p.per ? p.size - before : p.per;
  return p;
}

// Whether the lane's group is one of the best: worth is the same in all lanes of a group
template <int LN>
__device__ __forceinline__ bool group_stays(const GateArgs& a, const Place& p, float worth, int first_lane) {
  int rank = 0;
#pragma unroll 4
  for (int o = 0; o < a.groups; ++o) {
    const float w = __shfl(worth, first_lane + o * p.lanes);
    rank += w > worth || (w == worth && o < p.g);
  }
  return rank < a.top_groups;
}

// The two largest of v over the lanes of a group
template <int PL>
__device__ __forceinline__ void two_largest(const float (&v)[PL], int lanes, float& first, float& second) {
  first = second = -INFINITY;
#pragma unroll
  for (int j = 0; j < PL; ++j) {
    second = __builtin_amdgcn_fmed3f(first, second, v[j]);
    first = larger(first, v[j]);
  }
  for (int d = 1; d < lanes; d <<= 1) {
    const float f = __shfl_xor(first, d), s = __shfl_xor(second, d);
    second = larger(__builtin_amdgcn_fmed3f(first, second, f), s);
    first = larger(first, f);
  }
}

// Bit j: v[j] is -inf
template <int PL>
__device__ __forceinline__ uint32_t lowest_bits(const float (&v)[PL]) {
  uint32_t bits = 0;
#pragma unroll
  for (int j = PL - 1; j >= 0; --j)
    __asm__("v_cmp_eq_f32 vcc, %1, %2\n\tv_addc_co_u32 %0, vcc, %0, %0, vcc" : "+v"(bits) : "v"(v[j]), "v"(-INFINITY) : "vcc");
  return bits;
}

// k rounds, each of which takes the largest v of a token's LN lanes away. taken: bits of this lane's; got: rounds that found
// one; top and last: the first and the last that was taken; left: the largest that stays. Equal ones go in one round: then
// more are taken than rounds, which the caller has to look for.
struct Rounds {
  uint32_t taken;
  int got;
  float top, last, left;
};
template <int LN, int PL>
__device__ __forceinline__ Rounds take_largest(float (&v)[PL], int k) {
  Rounds r{0u, 0, -INFINITY, -INFINITY, -INFINITY};
  const uint32_t off = lowest_bits(v);
  for (int i = 0;; ++i) {
    const float best = run_max<LN>(largest(v));
    r.left = best;
    if (i == k) break;
    const bool has = best > -INFINITY;
    r.got += has;
    r.last = has ? best : r.last;
    r.top = i == 0 ? best : r.top;
#pragma unroll
    for (int j = 0; j < PL; ++j) v[j] = v[j] == best ? -INFINITY : v[j];
  }
  r.taken = lowest_bits(v) & ~off;
  return r;
}

// Of a token of sigmoids and a bias, of which at least k were taken, the experts that fp32 cannot tell apart from the k-th
// largest, by choices in 64 bits: those more than tol above it stay taken, of those within tol the largest fill the k. A choice
// is off by less than tol / 3 and fewer than k are above the k-th, so that no k experts can be above one that stays for sure.
// False where that does not settle it: more than 16 are near. Lanes of other tokens have doubt = false.
template <int LN, int PL, typename Row, typename Tol>
__device__ __forceinline__ bool settle_border(const GateArgs& a, const Place& p, const float (&v)[PL], float last, Tol tol_of, bool more, bool doubt, int q,
                                              int first_lane, Row row, uint32_t& taken) {
  auto choice = [&](int e) { return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-row(e) * 1.4426950408889634f)) + a.bias[e]; };
  // Equal ones went in one round: where they leave more than k the k-th largest may be above the last round's. The lowest of
  // the taken go until fewer than k would stay; they have k values at most.
  if (__any(doubt && more)) {
    float c[PL];
#pragma unroll
    for (int j = 0; j < PL; ++j) {
      const float x = choice(j < p.n ? p.e0 + j : 0);
      c[j] = (taken >> j) & 1 ? x : INFINITY;
    }
    bool open = doubt && more;
    int have = (int)run_sum<LN>((float)__popc(taken));
    for (int i = 0; i < a.k && __any(open); ++i) {
      float low = INFINITY;
#pragma unroll
      for (int j = 0; j < PL; ++j) low = c[j] < low ? c[j] : low;
      low = run_min<LN>(low);
      int equal = 0;
#pragma unroll
      for (int j = 0; j < PL; ++j) {
        equal += c[j] == low;
        c[j] = c[j] == low ? INFINITY : c[j];
      }
      have -= (int)run_sum<LN>((float)equal);
      last = open ? low : last;
      open = open && have >= a.k;
    }
  }
  const float tol = tol_of(last);
  uint32_t near = 0, sure = taken;
#pragma unroll
  for (int j = 0; j < PL; ++j) near |= v[j] > -INFINITY && v[j] >= last - tol ? 1u << j : 0u;  // v is -inf where taken
  for (uint32_t left = taken; doubt && left; left &= left - 1) {
    const uint32_t bit = left & -left;
    const float c = choice(p.e0 + __ffs((int)left) - 1);
    if (c <= last + tol) {
      sure &= ~bit;
      near |= c >= last - tol ? bit : 0u;
    }
  }
  const int counts = (int)run_sum<LN>((float)(__popc(sure) + 1024 * __popc(near)));  // at most 1024 experts of either
  int need = a.k - counts % 1024;
  const bool settled = doubt && need >= 0 && counts / 1024 <= 16;
  if (!settled) need = 0;
  near = settled ? near : 0;
  const uint64_t token = (~0ull >> (64 - LN)) << first_lane;
  while (__any(need > 0)) {
    double best = -INFINITY;
    uint32_t which = 0;
    for (uint32_t left = need > 0 ? near : 0; left; left &= left - 1) {
      const int e = p.e0 + __ffs((int)left) - 1;
      const double c = sigmoid64(row(e)) + (double)a.bias[e];
      which = c > best ? left & -left : which;
      best = larger64(best, c);
    }
    const double most = reduce64(best, LN, larger64);
    const uint64_t has = __ballot(need > 0 && best == most && which) & token;
    if (has && __ffsll((long long)has) - 1 == first_lane + q) {
      sure |= which;
      near &= ~which;
    }
    --need;
  }
  if (settled) taken = sure;
  return settled;
}

// The taken experts of a token to its list, in ascending order
// (at most LIST of them); returns how many there are
template <int LN, typename Row>
__device__ __forceinline__ int write_list(uint32_t taken, int q, int e0, Row row, Chosen* list) {
  const int count = __popc(taken);
  int upto = count;
#pragma unroll
  for (int d = 1; d < LN; d <<= 1) {
    const int o = __shfl_up(upto, d, LN);
    if (q >= d) upto += o;
  }
  int at = upto - count;
  in_order();
  while (taken && at < LIST) {
    const int j = __ffs((int)taken) - 1;
    taken &= taken - 1;
    list[at++] = Chosen{e0 + j, row(e0 + j)};
  }
  in_order();
  return __shfl(upto, LN - 1, LN);
}

// One token by a whole wave, without NaN or infinity, where fp32 leaves the order open: choices in 64 bits
template <int PL, typename Row>
__device__ __forceinline__ void exact_token(const GateArgs& a, long long t, Row row, Chosen* list, float m) {
  const int lane = threadIdx.x & 63;
  const Place p = place_of<64>(a, lane, true);
  double c[PL], inv = 1.0, z = 0.0;
  float l[PL], b[PL];
#pragma unroll
  for (int j = 0; j < PL; ++j) {
    l[j] = j < p.n ? row(p.e0 + j) : -INFINITY;
    b[j] = a.bias ? a.bias[j < p.n ? p.e0 + j : 0] : 0.f;
  }
  // Without a bias and sums of two the logits are the order, also where scores are 1 or 0 in 64 bits. m is there where the
  // exponentials are.
  const bool scored = a.bias || (a.groups > 1 && a.group_top == 2);
  if (scored || (!a.sigmoid && !a.renormalize)) {
#pragma unroll
    for (int j = 0; j < PL; ++j) {
      c[j] = exp(a.sigmoid ? -(double)l[j] : (double)l[j] - (double)m);
      z += c[j];
    }
    if (!a.sigmoid) inv = 1.0 / reduce64(z, 64, sum64);
#pragma unroll
    for (int j = 0; j < PL; ++j) c[j] = l[j] > -INFINITY ? (a.sigmoid ? 1.0 / (1.0 + c[j]) : c[j] * inv) + (double)b[j] : -INFINITY;
  }
  if (!scored) {
#pragma unroll
    for (int j = 0; j < PL; ++j) c[j] = l[j];
  }
  if (a.groups > 1) {
    // the largest of the group, and the largest of the others: all but the first place that has it
    double here = c[0];
#pragma unroll
    for (int j = 1; j < PL; ++j) here = larger64(here, c[j]);
    const double first = reduce64(here, p.lanes, larger64);
    double worth = first;
    if (a.group_top == 2) {
      const uint64_t has = __ballot(here == first) >> (p.g * p.lanes) & (~0ull >> (64 - p.lanes));
      bool skip = lane - p.g * p.lanes == __ffsll((long long)has) - 1;
      double second = -INFINITY;
#pragma unroll
      for (int j = 0; j < PL; ++j) {
        const bool it = skip && c[j] == first;
        skip = skip && !it;
        second = it ? second : larger64(second, c[j]);
      }
      second = reduce64(second, p.lanes, larger64);
      worth = second > -INFINITY ? first + second : first;
    }
    int rank = 0;
    for (int o = 0; o < a.groups; ++o) {
      const double w = of_lane(worth, o * p.lanes);
      rank += w > worth || (w == worth && o < p.g);
    }
#pragma unroll
    for (int j = 0; j < PL; ++j) {
      if (rank >= a.top_groups) c[j] = -INFINITY;
      else if (!a.bias && c[j] > -INFINITY) c[j] = l[j];  // the logits order the experts
    }
  }
  uint32_t taken = 0;
  int got = 0;
  for (; got < a.k; ++got) {
    double here = c[0];
#pragma unroll
    for (int j = 1; j < PL; ++j) here = larger64(here, c[j]);
    const double best = reduce64(here, 64, larger64);
    if (!(best > -INFINITY)) break;
    bool take = __ffsll((long long)__ballot(here == best)) - 1 == lane;
#pragma unroll
    for (int j = 0; j < PL; ++j) {
      const bool it = take && c[j] == best;
      c[j] = it ? -INFINITY : c[j];
      taken |= it ? 1u << j : 0u;
      take = take && !it;
    }
  }
  write_list<64>(taken, lane, p.e0, row, list);
  write_weights<64>(a, list, got, t, lane, true, m, inv);
  in_order();
}

// LN lanes a token, up to PL experts a lane; 64 / LN tokens take their rounds together. Few lanes a token share the
// reductions over lanes among more tokens, many make a token's rounds shorter. XPL: experts of a lane where 64 take a token.
template <int LN, int PL, int XPL>
__global__ void __launch_bounds__(64 * WAVES) gate_kernel(const GateArgs a) {
  constexpr int TOKENS = 64 / LN;
  extern __shared__ __align__(16) uint8_t lds[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane % LN, mine = lane / LN, first_lane = mine * LN;
  const long long t0 = ((long long)blockIdx.x * WAVES + wave) * TOKENS;
  if (t0 >= a.T) return;  // no barrier below: a wave works alone
  const int tokens = a.T - t0 < TOKENS ? (int)(a.T - t0) : TOKENS;
  const bool on = mine < tokens;
  float* const tile = (float*)(lds + (size_t)wave * wave_bytes(a, TOKENS));
  Chosen* const lists = (Chosen*)(tile + tile_floats(a, TOKENS));
  const Place p = place_of<LN>(a, q, on);
  const int row = mine * a.ldl + p.e0;
  const bool fours = a.whole && p.size % 4 == 0 && p.per % 4 == 0;  // and so are all numbers and places
  float l[PL], v[PL];
#pragma unroll
  for (int j = 0; j < PL; ++j) v[j] = 0.f;
  if (a.bias && fours) {
#pragma unroll
    for (int j = 0; j < PL; j += 4)
      if (j < p.n) {
        const f32x4 x = *(const f32x4*)(a.bias + p.e0 + j);
#pragma unroll
        for (int z = 0; z < 4; ++z) v[j + z] = x[z];
      }
  } else if (a.bias) {
#pragma unroll
    for (int j = 0; j < PL; ++j)
      if (j < p.n) v[j] = a.bias[p.e0 + j];
  }
  stage(a, t0, tokens, tile);
  if (fours) {
#pragma unroll
    for (int j = 0; j < PL; j += 4) {
      const f32x4 x = *(const f32x4*)(tile + place(j < p.n ? row + j : 0));
#pragma unroll
      for (int z = 0; z < 4; ++z) l[j + z] = j < p.n ? x[z] : -INFINITY;
    }
  } else {
#pragma unroll
    for (int j = 0; j < PL; ++j) {
      const float x = tile[place(j < p.n ? row + j : 0)];
      l[j] = j < p.n ? x : -INFINITY;
    }
  }

  bool unsure = false, strange = false;
  float m = 0.f, top = 1.f;  // top: the largest score that there may be
  double inv = 1.0;
  const bool pairs = a.groups > 1 && a.group_top == 2, scored = a.bias || pairs;
  const float inv_log2 = 1.4426950408889634f;
  if (!a.sigmoid && (scored || !a.renormalize)) {
    m = run_max<LN>(largest(l));
    strange = m == INFINITY;
    m = m == -INFINITY ? 0.f : m;
    double z[4] = {0.0, 0.0, 0.0, 0.0};
    if (a.renormalize) {  // for choices only
#pragma unroll
      for (int j = 0; j < PL; ++j) z[j % 4] += (double)__builtin_amdgcn_exp2f((l[j] - m) * inv_log2);
    } else {
#pragma unroll
      for (int j = 0; j < PL; ++j) z[j % 4] += exp((double)l[j] - (double)m);
    }
    inv = 1.0 / reduce64((z[0] + z[1]) + (z[2] + z[3]), LN, sum64);
    top = (float)inv;
  }
  // fp32 choices of size c are off by less than tol(c) / 3: the sum with b by 2^-24 of c; the score by 2^-22 of top, of which
  // a sigmoid's 1 + e and its reciprocal make 2^-24 and 2^-23, and e, 2^-23 by itself and |x| 2^-23.4 by its argument, makes
  // s (1 - s) times that, 0.42 2^-23 at most; a softmax's e^x likewise, with e^x |x| < 0.37, and 1 / sum 2^-23.
  auto tol = [&](float c) { return 0x1.8p-21f * top + 0x1.8p-23f * __builtin_fabsf(c); };
  bool nan = false;
  auto scores = [&](auto score) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < PL; ++j) {
      const float c = score(l[j]) + v[j];
      v[j] = l[j] == -INFINITY ? -INFINITY : c;
    }
  };
  if (!scored) {
#pragma unroll
    for (int j = 0; j < PL; ++j) v[j] = l[j];
  } else if (a.sigmoid) {
    scores([&](float x) { return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-x * inv_log2)); });
  } else {
    scores([&](float x) { return __builtin_amdgcn_exp2f((x - m) * inv_log2) * top; });
  }
#pragma unroll
  for (int j = 0; j < PL; ++j) nan |= v[j] != v[j];
  strange |= run_max<LN>(nan ? 1.f : 0.f) > 0.f;
  if (a.groups > 1) {
    float first, second;
    two_largest<PL>(v, p.lanes, first, second);
    const float worth = pairs && second > -INFINITY ? first + second : first;
    const bool stays = group_stays<LN>(a, p, worth, first_lane);
    if (scored) {
      // A sum of two is off by what both are, however much of them cancels, and by its own rounding: less than 2/3 of this.
      // Where no difference can be formed the order is open, too.
      const float off = pairs && second > -INFINITY ? 0x1.8p-21f * top + 0x1.8p-23f * (__builtin_fabsf(first) + __builtin_fabsf(second)) : tol(first);
      const float low = run_min<LN>(stays && worth > -INFINITY ? worth - off : INFINITY), high = run_max<LN>(stays || worth == -INFINITY ? -INFINITY : worth + off);
      unsure |= high > -INFINITY && !(low > high);
    }
#pragma unroll
    for (int j = 0; j < PL; ++j) v[j] = !stays || v[j] == -INFINITY ? -INFINITY : pairs && !a.bias ? l[j] : v[j];
  }
  Rounds r = take_largest<LN, PL>(v, a.k);
  // infinite choices have no differences, and an infinite logit makes its softmax's weights NaN
  strange |= r.top == INFINITY && (!a.sigmoid || a.bias);
  if (a.bias) {
    // equal choices that went in one round leave more than k
    const bool more = run_sum<LN>((float)__popc(r.taken)) > (float)r.got;
    const bool border = r.got == a.k && (more || (r.left > -INFINITY && r.last - r.left <= tol(r.last)));
    const bool doubt = border && !unsure && !strange;
    bool settled = false;
    if (a.sigmoid && __any(doubt))
      settled = settle_border<LN>(a, p, v, r.last, tol, more, doubt, q, first_lane, [&](int e) { return tile[place(mine * a.ldl + e)]; }, r.taken);
    unsure |= border && !settled;
  }
  Chosen* const list = lists + mine * LIST;
  unsure |= write_list<LN>(r.taken, q, p.e0, [&](int e) { return tile[place(mine * a.ldl + e)]; }, list) > r.got;
  write_weights<LN>(a, list, r.got, t0 + mine, q, on && !unsure && !strange, m, inv);
  in_order();
  const uint64_t open = __ballot(unsure && !strange && on && q == 0), odd = __ballot(strange && on && q == 0);
  for (uint64_t again = open | odd; again; again &= again - 1) {
    const int at = __ffsll((long long)again) - 1, i = at / LN;
    auto from = [&](int e) { return tile[place(i * a.ldl + e)]; };
    if ((open >> at) & 1) {
      exact_token<XPL>(a, t0 + i, from, lists + i * LIST, __shfl(m, at));
    } else {
      ordered_token(a, t0 + i, from, (uint64_t*)(lists + TOKENS * LIST), lists + i * LIST);
    }
  }
}

// The gradient, for r_j = s_j / (sum of the chosen s):
//   sigmoid, renormalised  dl_j = scale r_j (1 - s_j) (dw_j - sum_i r_i dw_i)    else  scale s_j (1 - s_j) dw_j
//   softmax, renormalised  dl_j = scale r_j (dw_j - sum_i r_i dw_i)              else  scale p_e ([e chosen] dw_e - sum_i p_i dw_i)
// 0 elsewhere in the first three, which read the chosen logits only and are bound by writing zeros. Formed in 64 bits and
// rounded once.

// An entry of a token: its expert (negative: it takes no part) and gradient
struct Entry {
  double d;
  int e;
};

// The forms with zeros: 16 lanes a token. Rows are put together in LDS and written 16 bytes a lane.
__global__ void __launch_bounds__(64 * WAVES) gate_backward_kernel(const GateArgs a) {
  constexpr int LN = LIST, TOKENS = 64 / LN;
  extern __shared__ __align__(16) uint8_t lds[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane % LN, mine = lane / LN, E = a.E, k = a.k;
  const long long t0 = ((long long)blockIdx.x * (blockDim.x >> 6) + wave) * TOKENS, t = t0 + mine;
  if (t0 >= a.T) return;  // no barrier below: a wave works alone
  const int n = (int)(a.T - t0 < TOKENS ? a.T - t0 : TOKENS) * E;  // elements of the wave's rows
  float* const tile = (float*)(lds + (size_t)wave * backward_wave_bytes(a));
  Entry* const list = (Entry*)(tile + (TOKENS * E + 3) / 4 * 4) + mine * LIST;
  int e = -1;
  float g = 0.f, l = -INFINITY;
  if (t < a.T && q < k) {
    e = a.chosen[t * k + q];
    g = a.dw[t * k + q];
  }
  for (int i = 4 * lane; i < TOKENS * E; i += 256) *(f32x4*)(tile + i) = f32x4{0.f, 0.f, 0.f, 0.f};
  if (e >= 0 && e < E) l = a.logits[t * E + e];
  const bool here = l != -INFINITY;  // takes part
  const double dw = here ? (double)g : 0.0;
  // r, and 1 - s for a sigmoid, however far the logit is
  const float x = a.sigmoid && l > 0.f ? 0.f : l;
  float most = 0.f;
  if (a.renormalize) {
    const float top = reduce<LN>(here ? x : -INFINITY, nan_max);
    most = most_of(a.sigmoid, top);
  }
  const Score score = score_of(a.sigmoid, l, most);
  double r = here ? score.s : 0.0;
  const double rest = score.rest;
  double d = dw;
  if (a.renormalize) {
    r /= reduce64(r, LN, sum64);  // 1 of one alone, whose gradient is 0
    r = here ? r : 0.0;
    d = dw - reduce64(r * dw, LN, sum64);
  }
  d = here ? a.scale * r * rest * d : 0.0;
  list[q] = Entry{d, here ? e : -1 - q};
  in_order();
  if (here) {
    double sum = 0.0;
    bool first = true;
    for (int i = 0; i < k; ++i) {
      const Entry o = list[i];
      sum += o.e == e ? o.d : 0.0;
      first = first && (o.e != e || i >= q);
    }
    if (first) tile[mine * E + e] = (float)sum;
  }
  in_order();
  float* const to = a.dlogits + t0 * E;
  if (a.whole) {
    for (int i = 4 * lane; i < n; i += 256) *(f32x4*)(to + i) = *(const f32x4*)(tile + i);
  } else {
    for (int i = lane; i < n; i += 64) to[i] = tile[i];
  }
}

// A softmax that is not renormalised: a wave a token, experts lane, lane + 64, ...
template <int PL>
__global__ void __launch_bounds__(64 * WAVES) gate_backward_dense_kernel(const GateArgs a) {
  __shared__ Entry lists[WAVES][LIST];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, E = a.E, k = a.k;
  const long long t = (long long)blockIdx.x * WAVES + wave;
  if (t >= a.T) return;  // no barrier below: a wave works alone
  const float* const row = a.logits + t * E;
  int e = -1;
  float dw = 0.f, l[PL], top = -INFINITY;
  double p[PL];
  if (lane < k) {
    e = a.chosen[t * k + lane];
    dw = a.dw[t * k + lane];
  }
#pragma unroll
  for (int j = 0; j < PL; ++j) {
    l[j] = lane + 64 * j < E ? row[lane + 64 * j] : -INFINITY;
    top = nan_max(top, l[j]);
  }
  const float at = e >= 0 && e < E ? row[e] : -INFINITY;
  const bool here = at != -INFINITY;
  top = reduce<64>(top, nan_max);
  const float m = top == -INFINITY ? 0.f : top;
  double z = 0.0;
#pragma unroll
  for (int j = 0; j < PL; ++j) {
    p[j] = l[j] == -INFINITY ? 0.0 : exp((double)l[j] - (double)m);
    z += p[j];
  }
  const double inv = 1.0 / reduce64(z, 64, sum64);
  const double mean = reduce64(here ? (double)dw * exp((double)at - (double)m) * inv : 0.0, 64, sum64);
  Entry* const list = lists[wave];
  if (lane < LIST) list[lane] = Entry{(double)dw, here ? e : -1};
  in_order();
#pragma unroll
  for (int j = 0; j < PL; ++j) {
    const int i = lane + 64 * j;
    double sum = 0.0;
    for (int o = 0; o < k; ++o) sum += list[o].e == i ? list[o].d : 0.0;
    if (i < E) a.dlogits[t * E + i] = l[j] == -INFINITY ? 0.f : (float)(a.scale * (p[j] * inv) * (sum - mean));
  }
}

template <int LN, int PL, int XPL>
void launch(const GateArgs& a, hipStream_t st) {
  constexpr int TOKENS = 64 / LN * WAVES;
  gate_kernel<LN, PL, XPL><<<dim3((unsigned)((a.T + TOKENS - 1) / TOKENS)), dim3(64 * WAVES), WAVES * wave_bytes(a, 64 / LN), st>>>(a);
}

}  // namespace

hipError_t launch_gate(const GateArgs& args, hipStream_t st) {
  GateArgs a = args;
  if (a.T == 0) return hipSuccess;
  a.whole = a.ldl % 4 == 0 && (uintptr_t)a.logits % 16 == 0 && (uintptr_t)a.bias % 16 == 0;
  if (a.groups & (a.groups - 1)) {  // groups that share no run of lanes evenly
    gate_exact_kernel<<<dim3((unsigned)((a.T + WAVES - 1) / WAVES)), dim3(64 * WAVES), WAVES * wave_bytes(a, 1), st>>>(a);
    return hipGetLastError();
  }
  // Lanes of a token. A wave a token is the shortest way for few tokens; for many, 8 to 16 experts a lane. 256 experts in 8
  // groups: 2048 tokens 12.3 us by 64 lanes each, 13.2 by 16 (7.0 by 64 without a doubtful token among them); 16384 tokens 33.5
  // by 64, 31.4 by 32, 18.0 by 16, 19.1 by 8. 64 experts, 16384 tokens: 5.8 us by 8 lanes, 9.2 by 16; 512 experts: 22 by 32, 31 by 64.
  int ln = a.T <= 2048 ? 64 : a.E <= 128 ? 8 : a.E <= 256 ? 16 : a.E <= 512 ? 32 : 64;
  if (ln < a.groups) ln = a.groups;
  const int lanes = ln / a.groups, per = (a.E / a.groups + lanes - 1) / lanes;  // lanes of a group, experts of a lane
  if (ln == 8 && per <= 8) launch<8, 8, 4>(a, st);
  else if (ln == 8) launch<8, 16, 4>(a, st);
  else if (ln == 16) launch<16, 16, 4>(a, st);
  else if (ln == 32) launch<32, 16, 8>(a, st);
  else if (per <= 4) launch<64, 4, 4>(a, st);
  else if (per <= 8) launch<64, 8, 8>(a, st);
  else launch<64, 16, 16>(a, st);
  return hipGetLastError();
}

hipError_t launch_gate_backward(const GateArgs& args, hipStream_t st) {
  GateArgs a = args;
  if (a.T == 0) return hipSuccess;
  a.whole = a.E % 4 == 0 && (uintptr_t)a.dlogits % 16 == 0;
  if (a.sigmoid || a.renormalize) {
    const int waves = a.E <= 512 ? WAVES : WAVES / 2, tokens = 64 / LIST * waves;  // at most 36 KiB of LDS
    gate_backward_kernel<<<dim3((unsigned)((a.T + tokens - 1) / tokens)), dim3(64 * waves), waves * backward_wave_bytes(a), st>>>(a);
    return hipGetLastError();
  }
  const dim3 grid((unsigned)((a.T + WAVES - 1) / WAVES)), block(64 * WAVES);
  const int pl = (a.E + 63) / 64;
  if (pl <= 2) gate_backward_dense_kernel<2><<<grid, block, 0, st>>>(a);
  else if (pl <= 4) gate_backward_dense_kernel<4><<<grid, block, 0, st>>>(a);
  else if (pl <= 8) gate_backward_dense_kernel<8><<<grid, block, 0, st>>>(a);
  else gate_backward_dense_kernel<16><<<grid, block, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace moe
