// The whole orthogonalisation, or Muon step, of a small matrix by one workgroup: X stays in registers in fp32 from the first
// read of the gradient to the last write of the parameters, A, C and the fp16 operands of the products in LDS.
//
// X is [MB][NB], the short side first, zeros beyond the matrix's size, in tiles of 32 x 32. Wave (wm, wn) of MB / 32 x WN holds CT
// tiles of A and C, (wm, wn CT + c), and the tiles (wm, wn + i WN) of X, as the matrix instruction leaves them: lane l has row
// l % 32 and, as its elements 4 q + j, columns 8 q + 4 (l / 32) + j. Operands in LDS are rows of fp16, X's of CH columns at a time:
// read along the rows for X X^T, A^2 and C, across them by the transposing read for X in C X. The same formulas and
// roundings as muon_gemm.hip's, but that X is not rounded between steps, only as an operand.
//
// What bounds it is the one CU that a matrix has: of 128 x 256 in fp32 the matrix cores need 32 us for the five steps, and the
// operands' reads from LDS as long.
#include <type_traits>

#include "muon.h"
#include "tile_ring.h"

namespace moe {

namespace {

typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;
typedef __attribute__((ext_vector_type(4))) _Float16 f16x4;
typedef __attribute__((address_space(3))) u32x2 lds_u32x2;

// A matrix of fp16 in LDS, rows of W elements: 16-byte chunk c of row r sits at c ^ (r % 16), which spreads 32 rows' reads of one
// chunk, and the transposing read's 4 rows, over the banks
template <int W>
struct Rows {
  static constexpr int MASK = W / 8 < 16 ? W / 8 - 1 : 15;
  __device__ static int chunk(int r, int c) { return r * (W * 2) + ((c ^ (r & MASK)) << 4); }
  // rows 32 t.. + 32 as indices, 16 elements of each from column 16 h as reduction
  __device__ static f16x8 along(const lds_byte* p, int t, int h, int l) {
    return __builtin_bit_cast(f16x8, *(const lds_bf16x8*)(p + chunk(t * 32 + (l & 31), 2 * h + (l >> 5))));
  }
  // columns 32 t.. + 32 as indices, 16 rows from 16 h as reduction
  __device__ static f16x8 across(const lds_byte* p, int t, int h, int l) {
    const int r = 16 * h + 8 * (l >> 5) + ((l & 15) >> 2), c = 2 * (2 * t + ((l >> 4) & 1)) + ((l & 3) >> 1);
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + chunk(r, c) + (l & 1) * 8));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + chunk(r + 4, c) + (l & 1) * 8));
    typedef __attribute__((ext_vector_type(8))) short s16x8;
    return __builtin_bit_cast(f16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
  // 4 columns of row r from c, a multiple of 4
  __device__ static void put(lds_byte* p, int r, int c, f16x4 v) {
    *(lds_u32x2*)(p + chunk(r, c >> 3) + (c & 4) * 2) = __builtin_bit_cast(u32x2, v);
  }
};

__device__ __forceinline__ f32x16 product(f16x8 a, f16x8 b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }

// Waves of an MB x MB product: at 128 those have two tiles each, which reads fewer operands and leaves a lane 256 registers
constexpr int tiles_of_a(int MB) { return MB == 128 ? 2 : 1; }
constexpr int waves_of(int MB) { return MB / 32 * (MB / 32) / tiles_of_a(MB); }

// f(std::integral_constant) of 0 .. N - 1
template <int N, typename F>
__device__ __forceinline__ void each_of(F f) {
  if constexpr (N > 0) {
    each_of<N - 1>(f);
    f(std::integral_constant<int, N - 1>{});
  }
}

template <int MB, int TILES, bool SPLIT>
__global__ void __launch_bounds__(64 * waves_of(MB)) small_kernel(const MuonArgs a, int steps) {
  constexpr int MT = MB / 32, CT = tiles_of_a(MB), WN = MT / CT, NB = 32 * WN * TILES;
  constexpr int MOST = 256 / (SPLIT ? 2 : 1), CH = MB == 128 && NB > MOST ? MOST : NB;
  constexpr int CHUNKS = NB / CH, EACH = TILES / CHUNKS, WAVES = MT * WN, PARTS = SPLIT ? 2 : 1, PAIR = EACH % 2 ? 1 : 2;
  using RX = Rows<CH>;
  using RA = Rows<MB>;
  __shared__ __align__(16) uint8_t xs[PARTS][MB * CH * 2], as[PARTS][MB * MB * 2];
  __shared__ float da[MB], dc[MB];
  __shared__ double sums[WAVES];
  lds_byte* const xp[2] = {(lds_byte*)xs[0], (lds_byte*)xs[PARTS - 1]};
  lds_byte* const ap[2] = {(lds_byte*)as[0], (lds_byte*)as[PARTS - 1]};
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave / WN, wn = wave % WN;
  const int row = wm * 32 + (lane & 31), hi4 = 4 * (lane >> 5);
  const MuonStack s = muon_stack(a, a.first + blockIdx.x);
  const int M = a.M, N = a.N;
  const bool g_f32 = a.g_f32, out_f32 = a.out_f32, nesterov = a.nesterov, rescale = a.grad_scale != nullptr;
  const float mu = a.momentum, pa = (float)a.a, pb = (float)a.b, pc = (float)a.c;
  const size_t base = (size_t)(a.first + blockIdx.x - s.first) * M * N;
  f32x16 x[TILES];
#pragma unroll
  for (int i = 0; i < TILES; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) x[i][e] = 0.f;
  // the user's elements: f(X's tile, element of it, place), 4 at a time where they lie together
  const bool fours = s.wide && N % 4 == 0;
  auto each = [&](auto f4, auto f1) __attribute__((always_inline)) {
    each_of<TILES>([&](auto tile) __attribute__((always_inline)) {
      constexpr int i = decltype(tile)::value;
      __asm__ volatile("" ::: "memory");  // a tile at a time: all at once need more registers than there are
      const int n0 = (wn + i * WN) * 32 + hi4;
      if (fours) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (row < M && n0 + 8 * q < N) f4(x[i], 4 * q, base + (size_t)row * N + n0 + 8 * q);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int n = n0 + 8 * (e >> 2) + (e & 3);
          if (row < M && n < N) f1(x[i], e, base + (s.wide ? (size_t)row * N + n : (size_t)n * M + row));
        }
      }
    });
  };

  // --- u, the new momentum and the norm
  const float gs = a.grad_scale ? *a.grad_scale : 1.f;
  auto scaled = [&](float g) { return rescale ? g * gs : g; };
  auto momentum = [&](float g, float& m) {
    m = mu * m + g;
    return nesterov ? g + mu * m : m;
  };
  each(
      [&](f32x16& t, int e, size_t at) __attribute__((always_inline)) {
        f32x4 u, m;
        if (g_f32) {
          u = *(const f32x4*)((const float*)s.g + at);
        } else {
          const u32x2 w = *(const u32x2*)((const uint16_t*)s.g + at);
          u = f32x4{bf16lo(w[0]), bf16hi(w[0]), bf16lo(w[1]), bf16hi(w[1])};
        }
        if (s.m) m = *(const f32x4*)(s.m + at);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          u[j] = scaled(u[j]);
          if (s.m) {
            float mj = m[j];
            u[j] = momentum(u[j], mj);
            m[j] = mj;
          }
          t[e + j] = u[j];
        }
        if (s.m) *(f32x4*)(s.m + at) = m;
      },
      [&](f32x16& t, int e, size_t at) __attribute__((always_inline)) {
        float u = scaled(g_f32 ? ((const float*)s.g)[at] : bf16_to_f32(((const uint16_t*)s.g)[at]));
        if (s.m) {
          float m = s.m[at];
          u = momentum(u, m);
          s.m[at] = m;
        }
        t[e] = u;
      });
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < TILES; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) sum += (double)x[i][e] * x[i][e];
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
  if (lane == 0) sums[wave] = sum;
  __syncthreads();
  sum = 0.0;
  for (int w = 0; w < WAVES; ++w) sum += sums[w];
  const double norm = sqrt(sum) + a.eps, f = norm == 0.0 ? 0.0 : (double)MUON_SCALE / norm;
#pragma unroll
  for (int i = 0; i < TILES; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) x[i][e] = (float)(x[i][e] * f);

  // --- the steps
  const float inv = 1.f / MUON_SCALE;
  // a tile's 4 columns as fp16, and what that leaves
  auto put = [&](lds_byte* const (&to)[2], auto rows, int r, int c, const float* v) __attribute__((always_inline)) {
    f16x4 hi, lo;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      hi[j] = (_Float16)v[j];
      lo[j] = (_Float16)(v[j] - (float)hi[j]);
    }
    decltype(rows)::put(to[0], r, c, hi);
    if (SPLIT) decltype(rows)::put(to[1], r, c, lo);
  };
  auto stage = [&](auto chunk) __attribute__((always_inline)) {
    constexpr int ch = decltype(chunk)::value;
#pragma unroll
    for (int i = ch * EACH; i < (ch + 1) * EACH; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float v[4] = {x[i][4 * q], x[i][4 * q + 1], x[i][4 * q + 2], x[i][4 * q + 3]};
        put(xp, RX{}, row, (wn + (i - ch * EACH) * WN) * 32 + 8 * q + hi4, v);
      }
  };
  f32x16 zero;
#pragma unroll
  for (int e = 0; e < 16; ++e) zero[e] = 0.f;
  // acc[c] += rows of p (tile t) times rows of q (tiles u.. of it), K columns
  auto gram = [&](lds_byte* const (&from)[2], auto rows, int K, f32x16 (&acc)[CT]) __attribute__((always_inline)) {
    using R = decltype(rows);
#pragma unroll 2
    for (int h = 0; h < K / 16; ++h) {
      const f16x8 p = R::along(from[0], wm, h, lane), p_lo = SPLIT ? R::along(from[1], wm, h, lane) : p;
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        const f16x8 q = R::along(from[0], wn * CT + c, h, lane);
        acc[c] = product(q, p, acc[c]);
        if constexpr (SPLIT) {
          acc[c] = product(R::along(from[1], wn * CT + c, h, lane), p, acc[c]);
          acc[c] = product(q, p_lo, acc[c]);
        }
      }
    }
  };
  for (int step = 0; step < steps; ++step) {
    f32x16 acc[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) acc[c] = zero;
    each_of<CHUNKS>([&](auto chunk) __attribute__((always_inline)) {
      __syncthreads();
      stage(chunk);
      __syncthreads();
      gram(xp, RX{}, CH, acc);
    });
    // A, its diagonal apart
    f32x16 own[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n0 = (wn * CT + c) * 32 + 8 * q + hi4;
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[j] = acc[c][4 * q + j] * inv;
          if (n0 + j == row) {
            da[row] = v[j] * inv;
            v[j] = 0.f;
          }
          const float hi = (float)(_Float16)v[j];
          own[c][4 * q + j] = SPLIT ? hi + (float)(_Float16)(v[j] - hi) : hi;
        }
        put(ap, RA{}, row, n0, v);
      }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < CT; ++c) acc[c] = zero;
    gram(ap, RA{}, MB, acc);
    const float dm = da[row];
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int n = (wn * CT + c) * 32 + 8 * (e >> 2) + hi4 + (e & 3);
        const float v = acc[c][e] * inv, x2 = own[c][e];
        own[c][e] = pb * x2 + pc * ((dm + da[n]) * x2 + v);
        if (n == row) {
          dc[row] = pa + pb * dm + pc * (dm * dm + v * inv);
          own[c][e] = 0.f;
        }
      }
    __syncthreads();  // all have read A: C takes its place
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float v[4] = {own[c][4 * q], own[c][4 * q + 1], own[c][4 * q + 2], own[c][4 * q + 3]};
        put(ap, RA{}, row, (wn * CT + c) * 32 + 8 * q + hi4, v);
      }
    __syncthreads();
    const float d = dc[row];
    // C X, the chunk that is still there first
    each_of<CHUNKS>([&](auto back) __attribute__((always_inline)) {
      constexpr std::integral_constant<int, CHUNKS - 1 - decltype(back)::value> chunk{};
      if constexpr (decltype(back)::value > 0) {
        __syncthreads();
        stage(chunk);
        __syncthreads();
      }
      each_of<EACH / PAIR>([&](auto pair) __attribute__((always_inline)) {
        constexpr int first = decltype(pair)::value * PAIR;  // of the chunk's tiles
        f32x16 sum[PAIR];
#pragma unroll
        for (int z = 0; z < PAIR; ++z) sum[z] = zero;
#pragma unroll 2
        for (int h = 0; h < MB / 16; ++h) {
          const f16x8 p = RA::along(ap[0], wm, h, lane), p_lo = SPLIT ? RA::along(ap[1], wm, h, lane) : p;
#pragma unroll
          for (int z = 0; z < PAIR; ++z) {
            const int t = wn + (first + z) * WN;
            const f16x8 q = RX::across(xp[0], t, h, lane);
            sum[z] = product(q, p, sum[z]);
            if constexpr (SPLIT) {
              sum[z] = product(RX::across(xp[1], t, h, lane), p, sum[z]);
              sum[z] = product(q, p_lo, sum[z]);
            }
          }
        }
#pragma unroll
        for (int z = 0; z < PAIR; ++z) {
          f32x16& to = x[decltype(chunk)::value * EACH + first + z];
#pragma unroll
          for (int e = 0; e < 16; ++e) to[e] = d * to[e] + sum[z][e] * inv;
        }
      });
    });
  }

  // --- O, or the parameters' step
  const float lr = a.lr_dev ? *a.lr_dev : a.lr, keep = 1.f - lr * a.wd, by = lr * s.scale;
  each(
      [&](f32x16& t, int e, size_t at) __attribute__((always_inline)) {
        f32x4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = t[e + j] * inv;
        if (s.m) {
          f32x4 old;
          if (s.master || out_f32) {
            old = *(const f32x4*)((s.master ? s.master : (const float*)s.out) + at);
          } else {
            const u32x2 w = *(const u32x2*)((const uint16_t*)s.out + at);
            old = f32x4{bf16lo(w[0]), bf16hi(w[0]), bf16lo(w[1]), bf16hi(w[1])};
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = old[j] * keep - by * v[j];
          if (s.master) *(f32x4*)(s.master + at) = v;
        }
        if (out_f32) *(f32x4*)((float*)s.out + at) = v;
        else *(u32x2*)((uint16_t*)s.out + at) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      },
      [&](f32x16& t, int e, size_t at) __attribute__((always_inline)) {
        float v = t[e] * inv;
        if (s.m) {
          const float old = s.master ? s.master[at] : out_f32 ? ((const float*)s.out)[at] : bf16_to_f32(((const uint16_t*)s.out)[at]);
          v = old * keep - by * v;
          if (s.master) s.master[at] = v;
        }
        if (out_f32) ((float*)s.out)[at] = v;
        else ((uint16_t*)s.out)[at] = __builtin_bit_cast(uint16_t, (__bf16)v);
      });
}

template <int MB, int TILES>
void launch(const MuonArgs& a, int steps, hipStream_t st) {
  if (a.split) small_kernel<MB, TILES, true><<<a.count, 64 * waves_of(MB), 0, st>>>(a, steps);
  else small_kernel<MB, TILES, false><<<a.count, 64 * waves_of(MB), 0, st>>>(a, steps);
}

}  // namespace

bool muon_small(int M, int N) { return M <= 128 && N <= 256; }

hipError_t launch_muon_small(const MuonArgs& a, int steps, hipStream_t st) {
  if (!muon_small(a.M, a.N)) return hipErrorInvalidValue;
  if (a.N <= 128) launch<128, 2>(a, steps, st);
  else launch<128, 4>(a, steps, st);
  return hipGetLastError();
}

}  // namespace moe
