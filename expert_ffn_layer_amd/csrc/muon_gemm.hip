// The products of the Newton-Schulz steps (v_mfma_f32_32x32x16_f16); forms as listed in muon.h.
//
// out[m][n] = sum_k P(m, k) Q(n, k), a tile of 128 x 128 per workgroup of 4 waves. A and C are symmetric: their tiles
// on and under the diagonal are computed and written to both places.
//
// Numerics: sums are fp32. X is a pair of fp16, x + x_lo, 22 bits; the products read x alone (11 bits) unless
// `split` asks for fp32 results: then x y_lo and x_lo y are added to x y. The diagonals of A and C are kept apart in fp32:
// where singular values are near each other the diagonal holds most of A and C, and its rounding would be most of the error.
#include "muon.h"

namespace moe {

namespace {

typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;
typedef __attribute__((ext_vector_type(4))) uint16_t u16x4;
typedef __attribute__((ext_vector_type(16))) float f32x16;

constexpr int THR = 256, TILE = 128, BK = 32, LD = BK + 8;

__device__ __forceinline__ uint16_t half_bits(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
__device__ __forceinline__ float half_value(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }

template <int FORM>
__global__ void __launch_bounds__(THR) product_kernel(const MuonArgs a) {
  constexpr bool SYM = FORM == MF_GRAM || FORM == MF_POLY;
  __shared__ __align__(16) uint16_t ps[TILE * LD], qs[TILE * LD];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wr = wave >> 1, wc = wave & 1;
  const int b = blockIdx.y;
  const int rows = SYM ? a.Mp : a.Np, K = FORM == MF_GRAM ? a.Np : a.Mp;
  int tm, tn;
  if (SYM) {
    tm = 0;
    int id = blockIdx.x;
    while (id > tm) id -= ++tm;
    tn = id;
  } else {
    const int cols = (a.Mp + TILE - 1) / TILE;
    tm = blockIdx.x / cols;
    tn = blockIdx.x % cols;
  }
  const int m0 = tm * TILE, n0 = tn * TILE;
  const size_t xat = (size_t)b * a.Np * a.Mp, aat = (size_t)b * a.Mp * a.Mp;

  f32x16 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

  for (int pass = 0; pass < (a.split ? 3 : 1); ++pass) {
    const uint16_t *p, *q;
    if (FORM == MF_GRAM) {
      p = (pass == 2 ? a.x_lo : a.x) + xat;
      q = (pass == 1 ? a.x_lo : a.x) + xat;
    } else if (FORM == MF_POLY) {
      p = (pass == 2 ? a.A_lo : a.A) + aat;
      q = (pass == 1 ? a.A_lo : a.A) + aat;
    } else {
      p = (pass == 2 ? a.x_lo : a.x) + xat;
      q = (pass == 1 ? a.C_lo : a.C) + aat;
    }
    for (int k0 = 0; k0 < K; k0 += BK) {
      __syncthreads();
      for (int i = tid; i < TILE * BK / 4; i += THR) {
        if (FORM == MF_GRAM) {  // [k][m] in memory
          const int k = i / (TILE / 4), m = i % (TILE / 4) * 4;
          u16x4 v{}, w{};
          if (m0 + m < a.Mp) v = *(const u16x4*)(p + (size_t)(k0 + k) * a.Mp + m0 + m);
          if (n0 + m < a.Mp) w = *(const u16x4*)(q + (size_t)(k0 + k) * a.Mp + n0 + m);
          for (int z = 0; z < 4; ++z) {
            ps[(m + z) * LD + k] = v[z];
            qs[(m + z) * LD + k] = w[z];
          }
        } else {
          const int m = i / (BK / 4), k = i % (BK / 4) * 4;
          u16x4 v{}, w{};
          if (m0 + m < rows) v = *(const u16x4*)(p + (size_t)(m0 + m) * a.Mp + k0 + k);
          if (n0 + m < a.Mp) w = *(const u16x4*)(q + (size_t)(n0 + m) * a.Mp + k0 + k);
          *(u16x4*)(ps + m * LD + k) = v;
          *(u16x4*)(qs + m * LD + k) = w;
        }
      }
      __syncthreads();
#pragma unroll
      for (int h = 0; h < BK; h += 16) {
        f16x8 pf[2], qf[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          pf[i] = *(const f16x8*)(ps + (wr * 64 + i * 32 + (lane & 31)) * LD + h + 8 * (lane >> 5));
          qf[i] = *(const f16x8*)(qs + (wc * 64 + i * 32 + (lane & 31)) * LD + h + 8 * (lane >> 5));
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            acc[t][i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(qf[t], pf[i], acc[t][i], 0, 0, 0);
      }
    }
  }

  // element 4 q + j of a tile is column 8 q + 4 (lane / 32) + j of row lane % 32
  const float inv = 1.f / MUON_SCALE;
  const float lr = a.lr_dev ? *a.lr_dev : a.lr;
  for (int t = 0; t < 2; ++t)
    for (int i = 0; i < 2; ++i)
      for (int e = 0; e < 16; ++e) {
        const int m = m0 + wr * 64 + i * 32 + (lane & 31), n = n0 + wc * 64 + t * 32 + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
        if (m >= rows || n >= a.Mp) continue;
        const float v = acc[t][i][e] * inv;  // times SCALE
        if (SYM) {
          float* const d = (FORM == MF_GRAM ? a.da : a.dc) + (size_t)b * a.Mp;
          uint16_t* const out = (FORM == MF_GRAM ? a.A : a.C) + aat;
          uint16_t* const out_lo = (FORM == MF_GRAM ? a.A_lo : a.C_lo) + aat;
          float r = v;
          if (FORM == MF_POLY) {
            const float* const da = a.da + (size_t)b * a.Mp;
            if (m == n) {
              r = MUON_SCALE * (a.b * da[m] + a.c * (da[m] * da[m] + v * inv));
            } else {
              float x = half_value(a.A[aat + (size_t)m * a.Mp + n]);
              if (a.split) x += half_value(a.A_lo[aat + (size_t)m * a.Mp + n]);
              r = a.b * x + a.c * ((da[m] + da[n]) * x + v);
            }
          }
          if (m == n) {
            d[m] = r * inv;
            r = 0.f;
          }
          const uint16_t hi = half_bits(r), lo = half_bits(r - half_value(hi));
          out[(size_t)m * a.Mp + n] = hi;
          if (a.split) out_lo[(size_t)m * a.Mp + n] = lo;
          if (tm != tn) {
            out[(size_t)n * a.Mp + m] = hi;
            if (a.split) out_lo[(size_t)n * a.Mp + m] = lo;
          }
        } else {
          const size_t at = xat + (size_t)m * a.Mp + n;
          const float x = half_value(a.x[at]) + half_value(a.x_lo[at]);
          const float r = (a.a + a.dc[(size_t)b * a.Mp + n]) * x + v;
          if (FORM == MF_STEP) {
            const uint16_t hi = half_bits(r);
            a.xo[at] = hi;
            a.xo_lo[at] = half_bits(r - half_value(hi));
          } else {
            if (m >= a.N || n >= a.M) continue;
            const MuonStack& s = muon_stack(a, a.first + b);
            const size_t o = (size_t)(a.first + b - s.first) * a.M * a.N + (s.wide ? (size_t)n * a.N + m : (size_t)m * a.M + n);
            float w = r * inv;
            if (s.m) {
              const float old = s.master ? s.master[o] : a.out_f32 ? ((const float*)s.out)[o] : bf16_to_f32(((const uint16_t*)s.out)[o]);
              w = old * (1.f - lr * a.wd) - lr * s.scale * w;
              if (s.master) s.master[o] = w;
            }
            if (a.out_f32) ((float*)s.out)[o] = w;
            else ((uint16_t*)s.out)[o] = __builtin_bit_cast(uint16_t, (__bf16)w);
          }
        }
      }
}

}  // namespace

hipError_t launch_muon_product(MuonForm form, const MuonArgs& a, hipStream_t st) {
  const unsigned m = (a.Mp + TILE - 1) / TILE, n = (a.Np + TILE - 1) / TILE, sym = m * (m + 1) / 2;
  switch (form) {
    case MF_GRAM: product_kernel<MF_GRAM><<<dim3(sym, a.count), THR, 0, st>>>(a); break;
    case MF_POLY: product_kernel<MF_POLY><<<dim3(sym, a.count), THR, 0, st>>>(a); break;
    case MF_STEP: product_kernel<MF_STEP><<<dim3(m * n, a.count), THR, 0, st>>>(a); break;
    case MF_LAST: product_kernel<MF_LAST><<<dim3(m * n, a.count), THR, 0, st>>>(a); break;
  }
  return hipGetLastError();
}

}  // namespace moe
