// The whole orthogonalisation, or Muon step, of a small matrix by one workgroup: X stays in registers in fp32 from the first
// read of the gradient to the last write of the parameters, A, C and the fp16 operands of the products in LDS.
//
// X is [MB][NB], the short side first, zeros beyond the matrix's size, in tiles of 32 x 32. Wave (wm, wn) of MT x WN holds CT
// tiles of A and C, (wm, wn CT + c), and the tiles (wm, wn + i WN) of X, as the matrix instruction leaves them: lane l has row
// l % 32 and, as its elements 4 q + j, columns 8 q + 4 (l / 32) + j. Operands in LDS are rows of fp16, X's of CH columns at a time:
// read along the rows for X X^T, A^2 and C, across them by the transposing read for X in C X. The same formulas and
// roundings as muon_gemm.hip's, but that X is not rounded between steps, only as an operand.
//
// What bounds it is the one CU that a matrix has. Eight of 256 x 128 take 75 us in fp32, of which the matrix cores need 32
// for the five steps, and 41 us in bf16; a CU also moves 2.6 MB of operands out of LDS and forms the pairs of 5 x 3 arrays
// with its vector units. With addresses computed for every read these took 90 and 54. By launches of products, each of
// which fills few CUs, they take 160.
#include <type_traits>

#include "muon.h"
#include "tile_ring.h"

namespace moe {

namespace {

typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;
typedef __attribute__((ext_vector_type(4))) _Float16 f16x4;
typedef __attribute__((address_space(3))) u32x2 lds_u32x2;

__device__ __forceinline__ f32x16 product(f16x8 a, f16x8 b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }

constexpr int MB = 128, MT = MB / 32;                 // the short side, padded, and its tiles
constexpr int CT = 2, WN = MT / CT, WAVES = MT * WN;  // two tiles of A a wave read fewer operands than one, and leave a lane 256 registers

// A matrix of fp16 in LDS, rows of W >= 128 elements: 16-byte chunk c of row r sits at c ^ (r % 16), which spreads 32 rows' reads
// of one chunk, and the transposing read's 4 rows, over the banks. A fragment is 32 indices x 16 reduction elements. What a
// lane has to add for it is one register, with the place in an exclusive or and a sum with constants.
template <int W>
struct Rows {
  // rows as indices: 16 columns from 16 h of row 0 and on are at along_at ^ (h << 5), of row 32 t and on t * ROWS32 behind
  static constexpr int ROWS32 = 32 * W * 2;
  __device__ static int along_at(int l) { return (l & 31) * (W * 2) + (((l >> 5) ^ (l & 15)) << 4); }
  // columns as indices: rows 0 to 15 of columns 32 t and on are at across_at ^ (t << 6), and those from 4 on likewise with
  // `four`; rows from 16 h are h * ROWS16 behind
  static constexpr int ROWS16 = 16 * W * 2;
  __device__ static int across_at(int l, int four) {
    const int r = 8 * (l >> 5) + ((l & 15) >> 2) + four, c = 2 * ((l >> 4) & 1) + ((l & 3) >> 1);
    return r * (W * 2) + ((c ^ r) << 4) + (l & 1) * 8;
  }
  // 4 columns of row r from c, a multiple of 4
  __device__ static int put_at(int r, int c) { return r * (W * 2) + (((c >> 3) ^ (r & 15)) << 4) + (c & 4) * 2; }
};
__device__ __forceinline__ f16x8 read_along(const lds_byte* p) { return __builtin_bit_cast(f16x8, *(const lds_bf16x8*)p); }
__device__ __forceinline__ f16x8 read_across(const lds_byte* p, const lds_byte* p4) {
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p), hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p4);
  typedef __attribute__((ext_vector_type(8))) short s16x8;
  return __builtin_bit_cast(f16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// f(std::integral_constant) of 0 .. N - 1
template <int N, typename F>
__device__ __forceinline__ void each_of(F f) {
  if constexpr (N > 0) {
    each_of<N - 1>(f);
    f(std::integral_constant<int, N - 1>{});
  }
}

template <int TILES, bool SPLIT>
__global__ void __launch_bounds__(64 * WAVES) small_kernel(const MuonArgs a, int steps) {
  constexpr int NB = 32 * WN * TILES, PARTS = SPLIT ? 2 : 1, MOST = 256 / PARTS, CH = NB > MOST ? MOST : NB;
  constexpr int CHUNKS = NB / CH, EACH = TILES / CHUNKS, PAIR = 2;
  static_assert(EACH % PAIR == 0, "tiles of a chunk go in pairs");
  using RX = Rows<CH>;
  using RA = Rows<MB>;
  constexpr int XS = MB * CH * 2, AS = MB * MB * 2;  // bytes of a part; the lower halves of pairs follow the upper
  __shared__ __align__(1024) uint8_t xs[PARTS * XS], as[PARTS * AS];
  __shared__ float da[MB], dc[MB];
  __shared__ double sums[WAVES];
  lds_byte *const xp = (lds_byte*)xs, *const ap = (lds_byte*)as;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave / WN, wn = wave % WN;
  const int row = wm * 32 + (lane & 31), hi4 = 4 * (lane >> 5);
  const MuonStack s = muon_stack(a, a.first + blockIdx.x);
  const int M = a.M, N = a.N;
  const bool g_f32 = a.g_f32, out_f32 = a.out_f32, nesterov = a.nesterov;
  const float mu = a.momentum, pa = (float)a.a, pb = (float)a.b, pc = (float)a.c;
  const size_t base = (size_t)(a.first + blockIdx.x - s.first) * M * N;
  // A tile of the user's elements, 4 at a time where they lie together. No load waits for another: what lies outside reads the
  // matrix's first element, and counts as 0.
  const bool fours = s.wide && N % 4 == 0;
  const int row_step = s.wide ? N : 1, col_step = s.wide ? 1 : M;
  auto column = [&](int i, int e) { return (wn + i * WN) * 32 + hi4 + 8 * (e >> 2) + (e & 3); };
  auto load = [&](const void* from, bool f32, int i) __attribute__((always_inline)) {
    f32x16 t;
    if (fours) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = column(i, 4 * q);
        const size_t at = base + (row < M && n < N ? row * N + n : 0);
        f32x4 v;
        if (f32) {
          v = *(const f32x4*)((const float*)from + at);
        } else {
          const u32x2 w = *(const u32x2*)((const uint16_t*)from + at);
          v = f32x4{bf16lo(w[0]), bf16hi(w[0]), bf16lo(w[1]), bf16hi(w[1])};
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) t[4 * q + j] = row < M && n < N ? v[j] : 0.f;
      }
    } else {
      auto all = [&](auto one) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int n = column(i, e);
          t[e] = one(base + (row < M && n < N ? row * row_step + n * col_step : 0));
        }
      };
      if (f32) all([&](size_t at) __attribute__((always_inline)) { return ((const float*)from)[at]; });
      else all([&](size_t at) __attribute__((always_inline)) { return bf16_to_f32(((const uint16_t*)from)[at]); });
#pragma unroll
      for (int e = 0; e < 16; ++e) t[e] = row < M && column(i, e) < N ? t[e] : 0.f;
    }
    return t;
  };
  auto store = [&](void* to, bool f32, int i, const f32x16& t) __attribute__((always_inline)) {
    if (fours) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = column(i, 4 * q);
        if (row >= M || n >= N) continue;
        const size_t at = base + row * N + n;
        if (f32) *(f32x4*)((float*)to + at) = f32x4{t[4 * q], t[4 * q + 1], t[4 * q + 2], t[4 * q + 3]};
        else *(u32x2*)((uint16_t*)to + at) = u32x2{pack_bf16x2(t[4 * q], t[4 * q + 1]), pack_bf16x2(t[4 * q + 2], t[4 * q + 3])};
      }
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int n = column(i, e);
        if (row >= M || n >= N) continue;
        const size_t at = base + row * row_step + n * col_step;
        if (f32) ((float*)to)[at] = t[e];
        else ((uint16_t*)to)[at] = __builtin_bit_cast(uint16_t, (__bf16)t[e]);
      }
    }
  };

  // --- u, the new momentum and the norm
  f32x16 x[TILES];
  each_of<TILES>([&](auto tile) __attribute__((always_inline)) { x[decltype(tile)::value] = load(s.g, g_f32, decltype(tile)::value); });
  if (a.grad_scale) {
    const float gs = *a.grad_scale;
#pragma unroll
    for (int i = 0; i < TILES; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) x[i][e] *= gs;
  }
  if (s.m) {
    each_of<TILES>([&](auto tile) __attribute__((always_inline)) {
      constexpr int i = decltype(tile)::value;
      f32x16 m = load(s.m, true, i);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        m[e] = mu * m[e] + x[i][e];
        x[i][e] = nesterov ? x[i][e] + mu * m[e] : m[e];
      }
      store(s.m, true, i, m);
    });
  }
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
  // 4 columns as fp16, and what that leaves
  auto put = [&](lds_byte* to, int part, const float (&v)[4]) __attribute__((always_inline)) {
    f16x4 hi, lo;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      hi[j] = (_Float16)v[j];
      lo[j] = (_Float16)(v[j] - (float)hi[j]);
    }
    *(lds_u32x2*)to = __builtin_bit_cast(u32x2, hi);
    if (SPLIT) *(lds_u32x2*)(to + part) = __builtin_bit_cast(u32x2, lo);
  };
  auto stage = [&](auto chunk) __attribute__((always_inline)) {
    constexpr int ch = decltype(chunk)::value;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const f32x16& t = x[ch * EACH + i];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        put(xp + RX::put_at(row, (wn + i * WN) * 32 + 8 * q + hi4), XS, {t[4 * q], t[4 * q + 1], t[4 * q + 2], t[4 * q + 3]});
    }
  };
  f32x16 zero;
#pragma unroll
  for (int e = 0; e < 16; ++e) zero[e] = 0.f;
  // acc[c] += rows of tile wm times rows of tile wn CT + c, over K columns
  auto gram = [&](const lds_byte* from, int at, auto rows, auto columns, auto part, f32x16 (&acc)[CT]) __attribute__((always_inline)) {
    constexpr int ROWS32 = decltype(rows)::ROWS32, K = decltype(columns)::value, LO = decltype(part)::value;
    const lds_byte *const p0 = from + wm * ROWS32, *const q0 = from + wn * CT * ROWS32;
    each_of<K / 16>([&](auto hc) __attribute__((always_inline)) {
      const int here = at ^ (decltype(hc)::value << 5);
      const f16x8 p = read_along(p0 + here);
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        const f16x8 q = read_along(q0 + here + c * ROWS32);
        acc[c] = product(q, p, acc[c]);
        if constexpr (SPLIT) {
          acc[c] = product(read_along(q0 + here + c * ROWS32 + LO), p, acc[c]);
          acc[c] = product(q, read_along(p0 + here + LO), acc[c]);
        }
      }
    });
  };
  const int along_x = RX::along_at(lane), along_a = RA::along_at(lane);
  const int across_x = RX::across_at(lane, 0), across_x4 = RX::across_at(lane, 4);
  const bool on_diagonal[CT] = {wn * CT == wm, wn * CT + 1 == wm};
  const int diagonal = lane & 31;  // the lane's row of a tile on the diagonal
  for (int step = 0; step < steps; ++step) {
    f32x16 acc[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) acc[c] = zero;
    each_of<CHUNKS>([&](auto chunk) __attribute__((always_inline)) {
      __syncthreads();
      stage(chunk);
      __syncthreads();
      gram(xp, along_x, RX{}, std::integral_constant<int, CH>{}, std::integral_constant<int, XS>{}, acc);
    });
    // A, its diagonal apart
    f32x16 own[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
#pragma unroll
      for (int e = 0; e < 16; ++e) own[c][e] = acc[c][e] * inv;
      if (on_diagonal[c])
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (8 * (e >> 2) + hi4 + (e & 3) == diagonal) {
            da[row] = own[c][e] * inv;
            own[c][e] = 0.f;
          }
#pragma unroll
      for (int q = 0; q < 4; ++q)
        put(ap + RA::put_at(row, (wn * CT + c) * 32 + 8 * q + hi4), AS, {own[c][4 * q], own[c][4 * q + 1], own[c][4 * q + 2], own[c][4 * q + 3]});
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float hi = (float)(_Float16)own[c][e];
        own[c][e] = SPLIT ? hi + (float)(_Float16)(own[c][e] - hi) : hi;
      }
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < CT; ++c) acc[c] = zero;
    gram(ap, along_a, RA{}, std::integral_constant<int, MB>{}, std::integral_constant<int, AS>{}, acc);
    const float dm = da[row];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4 dn = *(const f32x4*)(da + (wn * CT + c) * 32 + 8 * q + hi4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = 4 * q + j;
          acc[c][e] *= inv;
          own[c][e] = pb * own[c][e] + pc * ((dm + dn[j]) * own[c][e] + acc[c][e]);
        }
      }
      if (on_diagonal[c])
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (8 * (e >> 2) + hi4 + (e & 3) == diagonal) {
            dc[row] = pa + pb * dm + pc * (dm * dm + acc[c][e] * inv);
            own[c][e] = 0.f;
          }
    }
    __syncthreads();  // all have read A: C takes its place
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        put(ap + RA::put_at(row, (wn * CT + c) * 32 + 8 * q + hi4), AS, {own[c][4 * q], own[c][4 * q + 1], own[c][4 * q + 2], own[c][4 * q + 3]});
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
        const lds_byte *q0[PAIR], *q4[PAIR], *const p0 = ap + wm * RA::ROWS32;
#pragma unroll
        for (int z = 0; z < PAIR; ++z) {
          sum[z] = zero;
          const int t = (wn + (first + z) * WN) << 6;
          q0[z] = xp + (across_x ^ t);
          q4[z] = xp + (across_x4 ^ t);
        }
        each_of<MB / 16>([&](auto hc) __attribute__((always_inline)) {
          constexpr int h = decltype(hc)::value;
          const lds_byte* const at = p0 + (along_a ^ (h << 5));
          const f16x8 p = read_along(at);
#pragma unroll
          for (int z = 0; z < PAIR; ++z) {
            const f16x8 q = read_across(q0[z] + h * RX::ROWS16, q4[z] + h * RX::ROWS16);
            sum[z] = product(q, p, sum[z]);
            if constexpr (SPLIT) {
              sum[z] = product(read_across(q0[z] + h * RX::ROWS16 + XS, q4[z] + h * RX::ROWS16 + XS), p, sum[z]);
              sum[z] = product(q, read_along(at + AS), sum[z]);
            }
          }
        });
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
  each_of<TILES>([&](auto tile) __attribute__((always_inline)) {
    constexpr int i = decltype(tile)::value;
    f32x16 v;
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = x[i][e] * inv;
    if (s.m) {
      const f32x16 old = load(s.master ? s.master : s.out, s.master || out_f32, i);
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = old[e] * keep - by * v[e];
      if (s.master) store(s.master, true, i, v);
    }
    store(s.out, out_f32, i, v);
  });
}

template <int TILES>
void launch(const MuonArgs& a, int steps, hipStream_t st) {
  if (a.split) small_kernel<TILES, true><<<a.count, 64 * WAVES, 0, st>>>(a, steps);
  else small_kernel<TILES, false><<<a.count, 64 * WAVES, 0, st>>>(a, steps);
}

}  // namespace

// Of 2048 matrices, too: of 128 x 256 375 us in bf16 and 715 in fp32, by launches of products 1172 and 1956.
bool muon_small(int M, int N) { return M <= MB && N <= 256; }

hipError_t launch_muon_small(const MuonArgs& a, int steps, hipStream_t st) {
  if (!muon_small(a.M, a.N)) return hipErrorInvalidValue;
  if (a.N <= 128) launch<2>(a, steps, st);
  else launch<4>(a, steps, st);
  return hipGetLastError();
}

}  // namespace moe
