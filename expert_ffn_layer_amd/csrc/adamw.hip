// AdamW over many tensors in one launch:
//   g' = s g                       m = b1 m + (1 - b1) g'        v = b2 v + (1 - b2) g'^2
//   p = p - lr wd p - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// in fp32 throughout; a bf16 p is rounded once (from the fp32 master copy when there is one).
//
// The 8-bit form keeps m and r = sqrt(v) as e4m3 codes over one fp32 scale per 256 consecutive
// elements (the largest magnitude / 448). The root halves the exponent range that v needs. A value
// between two codes is rounded up with the probability of its place between them: a step changes r
// by 2.5% at most downwards (beta2 = 0.95), less than half a code step of 6 to 12%, so that rounding
// to the nearest code would never let an element fall and r would only grow. The random bits are a
// hash of element, step and seed, so a run repeats bit for bit. p moves by the new m and v before
// they are rounded.
//
// Bound by memory: every array is read or written once. A workgroup takes 8192 consecutive elements
// of one tensor, 8 a lane and pass, so 32 lanes hold one block of the 8-bit form and its maximum takes
// 5 lane exchanges; 2048 where that would leave CUs without work (five tensors of 0.8 M elements: 10.1
// us by 8192, 6.8 by 2048; twelve of 14.7 M 5.3 TB/s with fp32 states and master copies, ten 4.9 TB/s with
// 8-bit ones, where a large copy reaches 4.9). The tensor table travels in the kernel arguments: no copy,
// no table kept.
#include <type_traits>

#include "train.h"

namespace moe {

namespace {

constexpr int ATHR = 256;
constexpr int AV = 8;                    // elements per lane and pass
constexpr int ASTEP = ATHR * AV;         // elements of a workgroup and pass
constexpr int APASS = 4;                 // most passes per workgroup
constexpr int64_t SMALL = 8 << 20;       // elements in all below which a workgroup makes one pass only
constexpr float E4M3_MAX = 448.0f;
constexpr float MIN_TOP = 0x1p-100f;     // keeps 448 / top finite: smaller values become code 0

__device__ __forceinline__ void load8(const float* p, float (&v)[AV]) {
  const f32x4 a = *(const f32x4*)p, b = *(const f32x4*)(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[AV]) {
  const u32x4 a = *(const u32x4*)p;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[2 * i] = bf16lo(a[i]), v[2 * i + 1] = bf16hi(a[i]);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[AV]) {
  *(f32x4*)p = f32x4{v[0], v[1], v[2], v[3]};
  *(f32x4*)(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[AV]) {
  *(u32x4*)p = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = (uint16_t)pack_bf16x2(v, 0.f); }

// the lane's elements at, at + 1, ... below n; the others read as zero. FULL: all 8 are below n
template <bool FULL, typename T>
__device__ __forceinline__ void load_some(const T* p, int64_t at, int64_t n, float (&v)[AV]) {
  if (FULL || at + AV <= n) {
    load8(p + at, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < AV; ++i) v[i] = at + i < n ? load1(p + at + i) : 0.f;
}
template <bool FULL, typename T>
__device__ __forceinline__ void store_some(T* p, int64_t at, int64_t n, const float (&v)[AV]) {
  if (FULL || at + AV <= n) {
    store8(p + at, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < AV; ++i)
    if (at + i < n) store1(p + at + i, v[i]);
}

template <bool FULL>
__device__ __forceinline__ u32x2 load_codes(const uint8_t* p, int64_t at, int64_t n) {
  if (FULL || at + AV <= n) return *(const u32x2*)(p + at);
  u32x2 c = {0u, 0u};
#pragma unroll
  for (int i = 0; i < AV; ++i)
    if (at + i < n) c[i >> 2] |= (uint32_t)p[at + i] << (8 * (i & 3));
  return c;
}
template <bool FULL>
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t at, int64_t n, u32x2 c) {
  if (FULL || at + AV <= n) {
    *(u32x2*)(p + at) = c;
    return;
  }
#pragma unroll
  for (int i = 0; i < AV; ++i)
    if (at + i < n) p[at + i] = (uint8_t)(c[i >> 2] >> (8 * (i & 3)));
}
__device__ __forceinline__ void decode(u32x2 c, float s, float (&v)[AV]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(c[h], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(c[h], true);
    v[4 * h] = lo[0] * s;
    v[4 * h + 1] = lo[1] * s;
    v[4 * h + 2] = hi[0] * s;
    v[4 * h + 3] = hi[1] * s;
  }
}
// Random words of the 8-bit form: a multiply-xorshift hash of element index and key, the key one of
// seed and step. m uses a word's upper 20 bits, the root its lower 20. The multipliers 0x9E3779B1 and 0x85EBCA77 are
// the first two primes of XXH32, and the shifts of 15 and 13 with the second between them are the first half of its
// final mix (Y. Collet's published xxHash specification).
__device__ __forceinline__ uint32_t dither_key(uint32_t seed, uint32_t step) {
  uint32_t k = seed + step * 0x9E3779B9u;
  k = (k ^ (k >> 16)) * 0x85EBCA77u;
  return k ^ (k >> 13);
}
__device__ __forceinline__ uint32_t dither(uint32_t index, uint32_t key) {
  uint32_t x = index * 0x9E3779B1u + key;
  x = (x ^ (x >> 15)) * 0x85EBCA77u;
  return x ^ (x >> 13);
}
// y (at most about 448 in magnitude) to an e4m3 value: adding 20 random bits below the 3 kept
// mantissa bits and cutting carries with the probability wanted. Under 2^-6 the codes are 2^-9
// apart, which adding 2^-6 turns into the same cut. A NaN's word could carry into the sign, so the
// minimum makes a number of it first and 0 y brings it back: no more operations than a compare and select.
__device__ __forceinline__ float to_e4m3(float y, uint32_t bits) {
  const float a = __builtin_fminf(__builtin_fabsf(y), E4M3_MAX);
  const float low = a < 0x1p-6f ? 0x1p-6f : 0.0f;
  const float z = __uint_as_float((__float_as_uint(a + low) + bits) & 0xFFF00000u) - low;
  return __builtin_copysignf(__builtin_fmaf(0.0f, y, z), y);
}
// codes of the lane's 8 values over their block's scale, which the block's 32 lanes agree on
__device__ __forceinline__ u32x2 encode(const float (&v)[AV], const uint32_t (&bits)[AV], float& scale) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < AV; ++i) top = __builtin_fmaxf(top, __builtin_fabsf(v[i]));  // a NaN does not count
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) top = __builtin_fmaxf(top, __shfl_xor(top, s));
  top = __builtin_fmaxf(top, MIN_TOP);
  const float inv = E4M3_MAX * (1.0f / top);
  scale = top * (1.0f / E4M3_MAX);
  float z[AV];
#pragma unroll
  for (int i = 0; i < AV; ++i) z[i] = to_e4m3(v[i] * inv, bits[i]);
  u32x2 c;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(z[4 * h], z[4 * h + 1], 0, false);
    c[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(z[4 * h + 2], z[4 * h + 3], w, true);
  }
  return c;
}

// Square root by one Newton step on v * rsq(v) with an exact residual: correctly rounded but for rare halfway cases.
// Values below 2^-96 go through 2^24 times them, for the hardware's rsq takes no denormals. 11 operations where the
// compiler's takes 17, of 76 an element of the 8-bit form. 0 and NaN stay, and an infinity becomes NaN: that has a code
// and does not reach the scale of its block.
__device__ __forceinline__ float root(float v) {
  const bool low = v < 0x1p-96f;
  const float x = v * (low ? 0x1p24f : 1.0f);
  const float y = __builtin_amdgcn_rsqf(__builtin_fmaxf(x, 0x1p-126f)), s = x * y;
  return __builtin_fmaf(__builtin_fmaf(-s, s, x), 0.5f * y, s) * (low ? 0x1p-12f : 1.0f);
}

template <typename PT, typename GT, bool MASTER, bool Q8>
__global__ void __launch_bounds__(ATHR) adamw_kernel(const AdamArgs a) {
  // every product and sum rounds by itself, so the 8-bit codes are the same whatever the compiler would fuse
#pragma clang fp contract(off)
  const int lane = threadIdx.x & 63, block = blockIdx.x;
  // the tensor whose workgroups hold this one: those before it have all ended
  const bool after = lane < a.count && block >= a.first[lane < a.count ? lane + 1 : 1];
  const int ti = __builtin_popcountll(__ballot(after));
  const AdamTensor& t = a.t[ti];
  const int64_t n = t.n, base = (int64_t)(block - a.first[ti]) * (a.passes * ASTEP) + threadIdx.x * AV;
  const int64_t wave_end = (int64_t)(block - a.first[ti]) * (a.passes * ASTEP) + (__builtin_amdgcn_readfirstlane(threadIdx.x >> 6) + 1) * 64 * AV;
  PT* const p = (PT*)t.p;
  const GT* const g = (const GT*)t.g;

  // rate and step come from device memory where given, so that a captured launch follows them
  const float lr = a.lr_dev ? *a.lr_dev : a.lr;
  float bc1 = a.bc1, inv_root_bc2 = a.inv_root_bc2;
  int64_t step = a.step;
  if (a.step_dev) {
    step = *a.step_dev;
    if (step < 1) step = 1;
    const float s = (float)step;
    bc1 = -expm1f(s * a.log_beta1);
    inv_root_bc2 = 1.0f / __builtin_sqrtf(-expm1f(s * a.log_beta2));
  }
  const float step_size = lr / bc1, lrwd = lr * a.wd;
  const uint32_t key = Q8 ? dither_key(a.seed, (uint32_t)step) : 0u;
  const float gs = a.grad_scale ? *a.grad_scale : 1.0f;

  auto pass_at = [&](int64_t at, auto full) __attribute__((always_inline)) {
    constexpr bool FULL = decltype(full)::value;
    float w[AV], gv[AV], m[AV], v[AV], r[AV];
    if constexpr (MASTER) load_some<FULL>(t.master, at, n, w);
    else load_some<FULL>((const PT*)p, at, n, w);
    load_some<FULL>(g, at, n, gv);
    if constexpr (Q8) {
      const int64_t b = at >> 8;
      const u32x2 cm = load_codes<FULL>((const uint8_t*)t.m, at, n), cr = load_codes<FULL>((const uint8_t*)t.v, at, n);
      decode(cm, t.ms[b], m);
      decode(cr, t.vs[b], r);
#pragma unroll
      for (int i = 0; i < AV; ++i) v[i] = r[i] * r[i];
    } else {
      load_some<FULL>((const float*)t.m, at, n, m);
      load_some<FULL>((const float*)t.v, at, n, v);
    }
#pragma unroll
    for (int i = 0; i < AV; ++i) {
      const float gi = gv[i] * gs;
      m[i] = a.beta1 * m[i] + a.one_minus_beta1 * gi;
      v[i] = a.beta2 * v[i] + a.one_minus_beta2 * (gi * gi);
      r[i] = Q8 ? root(v[i]) : __builtin_sqrtf(v[i]);
      // hardware reciprocal, about 1 ulp of an update that is itself about lr
      const float low = __builtin_fmaf(r[i], inv_root_bc2, a.eps);
      w[i] -= __builtin_fmaf(lrwd, w[i], step_size * (m[i] * __builtin_amdgcn_rcpf(low)));
    }
    if constexpr (MASTER) store_some<FULL>(t.master, at, n, w);
    store_some<FULL>(p, at, n, w);
    if constexpr (Q8) {
      float sm, sr;
      uint32_t bm[AV], br[AV];
#pragma unroll
      for (int i = 0; i < AV; ++i) {
        const uint32_t x = dither((uint32_t)at + i, key);
        bm[i] = x >> 12;
        br[i] = x & 0xFFFFFu;
        m[i] = __builtin_fmaf(0.f, r[i], m[i]);  // NaN where the root is
      }
      const u32x2 cm = encode(m, bm, sm), cr = encode(r, br, sr);
      store_codes<FULL>((uint8_t*)t.m, at, n, cm);
      store_codes<FULL>((uint8_t*)t.v, at, n, cr);
      if ((lane & 31) == 0) {
        t.ms[at >> 8] = sm;
        t.vs[at >> 8] = sr;
      }
    } else {
      store_some<FULL>((float*)t.m, at, n, m);
      store_some<FULL>((float*)t.v, at, n, v);
    }
  };
  for (int pass = 0; pass < a.passes; ++pass) {
    const int64_t at = base + (int64_t)pass * ASTEP;
    // A wave whose elements are all there takes a path without conditions, whose loads leave together (fp32 states
    // with master copies 945 us, 957 by the other path); the 8-bit form, with more to compute between its loads, is
    // 7% slower by it. In the other path a half wave without elements leaves together, so every
    // block's lanes stay for its maximum.
    if (!Q8 && wave_end + (int64_t)pass * ASTEP <= n) {
      pass_at(at, std::true_type{});
    } else {
      if ((at & ~(int64_t)255) >= n) return;
      pass_at(at, std::false_type{});
    }
  }
}

}  // namespace

int adamw_chunk(int64_t elements) { return elements < SMALL ? ASTEP : ASTEP * APASS; }
int adamw_passes(int chunk) { return chunk / ASTEP; }

hipError_t launch_adamw(int p_type, int g_type, bool master, bool q8, const AdamArgs& a, hipStream_t st) {
  const int grid = a.first[a.count];
  if (grid == 0) return hipSuccess;
  auto go = [&](auto kernel) -> hipError_t {
    kernel<<<grid, ATHR, 0, st>>>(a);
    return hipGetLastError();
  };
  if (p_type == MOE_F32) {
    if (master) return hipErrorInvalidValue;
    if (g_type == MOE_F32) return q8 ? go(adamw_kernel<float, float, false, true>) : go(adamw_kernel<float, float, false, false>);
    return q8 ? go(adamw_kernel<float, uint16_t, false, true>) : go(adamw_kernel<float, uint16_t, false, false>);
  }
  if (master) {
    if (g_type == MOE_F32)
      return q8 ? go(adamw_kernel<uint16_t, float, true, true>) : go(adamw_kernel<uint16_t, float, true, false>);
    return q8 ? go(adamw_kernel<uint16_t, uint16_t, true, true>) : go(adamw_kernel<uint16_t, uint16_t, true, false>);
  }
  if (g_type == MOE_F32)
    return q8 ? go(adamw_kernel<uint16_t, float, false, true>) : go(adamw_kernel<uint16_t, float, false, false>);
  return q8 ? go(adamw_kernel<uint16_t, uint16_t, false, true>) : go(adamw_kernel<uint16_t, uint16_t, false, false>);
}

}  // namespace moe
