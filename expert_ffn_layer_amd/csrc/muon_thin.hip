// Orthogonalisation and Muon step of matrices whose short side is at most 32, or 64 beside a long one, in 64 bits (v_mfma_f64_16x16x4_f64).
//
// With A_0 = X_0 X_0^T every step's polynomial is one in A_0, so the steps need X only before and after them:
//   B_i = a I + b A_i + c A_i^2,  A_{i+1} = B_i A_i B_i,  Q = B_last ... B_0,  O = Q X_0
// and the long side is read twice for several steps: once for A_0 (gram), once for Q X_0 (apply). The steps themselves (steps)
// are a few products of at most 64 x 64 by one workgroup. But a step multiplies what rounding adds to A's small eigenvalues by
// the derivative of lambda (a + b lambda + c lambda^2)^2, a^2 = 12 at 0, and one that rounding makes negative leaves the
// polynomial's range in the end; and Q's large entries cancel on large singular values. So A is formed anew from X after as many
// steps as multiply rounding by 2^29 at most (8 of the usual coefficients), from 2^-53 to below fp32's, with X kept in 64 bits
// between: by A alone 16 steps were off by their norm and 20 infinite where the rank was below the short side. One of 256 x 8
// takes 34 us for 8 steps, 67 for 16; 4096 of 32 x 2048 1.24 and 3.35 ms.
//
// What bounds them is latency: three launches, and in `steps` 17 products one after the other. One of 256 x 8: 9 + 12 + 6 us, by
// one workgroup in one launch 33; in `steps` a short side of up to 32 takes 12 to 13 us, of 64 61, of which the matrix
// instructions of one CU need 31. By the products of 16-bit operands, for which the short side is
// padded to 128, two of 24 x 1577 took 333 us, here 30.
#include <type_traits>

#include "muon.h"

namespace moe {

namespace {

typedef __attribute__((ext_vector_type(4))) double f64x4;

constexpr int THR = 256, COLS = 64, LD = COLS + 4;  // columns of the long side at a time, and floats of a row of them in LDS

// v_mfma_f64_16x16x4_f64: lane l gives row l % 16 of the first operand and column l % 16 of the second at reduction element
// l / 16, and gets rows l / 16 + 4 r of column l % 16.
__device__ __forceinline__ f64x4 product(double a, double b, f64x4 c) { return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, 0, 0, 0); }

// The user's elements of columns n0.. + 64 of the long side, 4 of a row of theirs at a time: f(place, row and column of X,
// how many there are, step of X's column per element or 0 where its row runs)
template <int MB, typename F>
__device__ __forceinline__ void user_elements(const MuonArgs& a, const MuonStack& s, size_t base, int n0, F f) {
  const int w = s.wide ? COLS : MB, per_row = w / 4, rows = s.wide ? MB : COLS;
  const int c = 4 * (threadIdx.x % per_row);
  for (int r = threadIdx.x / per_row; r < rows; r += THR / per_row) {
    const int j = s.wide ? r : c, n = n0 + (s.wide ? c : r);
    if (j >= a.M || n >= a.N) continue;
    const int left = s.wide ? a.N - n : a.M - j;
    f(base + (s.wide ? (size_t)j * a.N + n : (size_t)n * a.M + j), j, n - n0, left < 4 ? left : 4);
  }
}

// u at `n` consecutive places; with `update` m is stepped first, else it has been
__device__ __forceinline__ f32x4 read_u(const MuonArgs& a, const MuonStack& s, size_t at, int n, bool whole, float gs, bool update) {
  f32x4 u = {0.f, 0.f, 0.f, 0.f}, m = u;
  if (whole) {
    if (a.g_f32) {
      u = *(const f32x4*)((const float*)s.g + at);
    } else {
      const u32x2 w = *(const u32x2*)((const uint16_t*)s.g + at);
      u = f32x4{bf16lo(w[0]), bf16hi(w[0]), bf16lo(w[1]), bf16hi(w[1])};
    }
    if (s.m) m = *(const f32x4*)(s.m + at);
  } else {
#pragma unroll
    for (int z = 0; z < 4; ++z)
      if (z < n) {
        u[z] = a.g_f32 ? ((const float*)s.g)[at + z] : bf16_to_f32(((const uint16_t*)s.g)[at + z]);
        if (s.m) m[z] = s.m[at + z];
      }
  }
  if (a.grad_scale) u = u * gs;
  if (!s.m) return u;
  if (update) {
    m = a.momentum * m + u;
    if (whole) {
      *(f32x4*)(s.m + at) = m;
    } else {
#pragma unroll
      for (int z = 0; z < 4; ++z)
        if (z < n) s.m[at + z] = m[z];
    }
  }
  return a.nesterov ? u + a.momentum * m : m;
}

// X between two runs of steps
__device__ __forceinline__ double* kept_x(const MuonArgs& a, int b) { return a.xs + (size_t)b * a.M * a.N; }

// 64 columns of it, zeros beyond its size
template <int MB>
__device__ __forceinline__ void read_x(const MuonArgs& a, int b, int n0, double* to) {
  const double* const x = kept_x(a, b);
  for (int i = threadIdx.x; i < MB * COLS; i += THR) {
    const int j = i / COLS, n = i % COLS;
    to[j * LD + n] = j < a.M && n0 + n < a.N ? x[(size_t)j * a.N + n0 + n] : 0.0;
  }
}

// Partial sums of u u^T over a part's columns, and the new momentum, or of X X^T. Parts are always the same columns: the same
// bits on every run.
template <int MB, bool FROM_X>
__global__ void __launch_bounds__(THR) gram_kernel(const MuonArgs a) {
  constexpr int T = MB / 16, EACH = T * T / 4;  // tiles of 16 a side, and of each of 4 waves
  using Element = std::conditional_t<FROM_X, double, float>;
  __shared__ __align__(16) Element u[MB * LD];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, k4 = lane >> 4, b = blockIdx.y;
  const int ti = wave * EACH / T, tj = wave * EACH % T;
  const MuonStack& s = muon_stack(a, a.first + b);
  const size_t base = (size_t)(a.first + b - s.first) * a.M * a.N;
  const bool whole = (s.wide ? a.N : a.M) % 4 == 0;
  const float gs = a.grad_scale ? *a.grad_scale : 1.f;
  f64x4 acc[EACH];
#pragma unroll
  for (int i = 0; i < EACH; ++i) acc[i] = f64x4{0.0, 0.0, 0.0, 0.0};
  const int from = blockIdx.x * a.part, to = from + a.part < a.N ? from + a.part : a.N;
  for (int n0 = from; n0 < to; n0 += COLS) {
    __syncthreads();
    if constexpr (FROM_X) {
      read_x<MB>(a, b, n0, u);
    } else {
      for (int i = threadIdx.x; i < MB * LD / 4; i += THR) *(f32x4*)(u + 4 * i) = f32x4{0.f, 0.f, 0.f, 0.f};
      __syncthreads();
      user_elements<MB>(a, s, base, n0, [&](size_t at, int j, int n, int left) {
        const f32x4 v = read_u(a, s, at, left, whole, gs, true);
#pragma unroll
        for (int z = 0; z < 4; ++z)
          if (z < left) u[s.wide ? j * LD + n + z : (j + z) * LD + n] = v[z];
      });
    }
    __syncthreads();
    for (int k = 0; k < COLS; k += 4) {
      const double p = u[(ti * 16 + l16) * LD + k + k4];
#pragma unroll
      for (int i = 0; i < EACH; ++i) acc[i] = product(p, (double)u[((tj + i) * 16 + l16) * LD + k + k4], acc[i]);
    }
  }
  double* const out = a.sums + ((size_t)b * a.parts + blockIdx.x) * MB * MB;
#pragma unroll
  for (int i = 0; i < EACH; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) out[((ti * T + tj + i) * 4 + r) * 64 + lane] = acc[i][r];
}

// Q and 1 / (|u| + eps) of a matrix, 1 for sums over X itself; wave w of (MB / 16)^2 holds tile w of every matrix here
template <int MB>
__global__ void __launch_bounds__(MB* MB / 4) steps_kernel(const MuonArgs a, int steps, bool from_x) {
  constexpr int T = MB / 16, LQ = MB + 4;
  __shared__ double A[MB * LQ], B[MB * LQ], Q[MB * LQ], W[MB * LQ], traces[T * T];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, k4 = lane >> 4, ti = wave / T, tj = wave % T, b = blockIdx.x;
  const double* const in = a.sums + (size_t)b * a.parts * MB * MB;
  double mine[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 4
  for (int p = 0; p < a.parts; ++p)
#pragma unroll
    for (int r = 0; r < 4; ++r) mine[r] += in[(size_t)p * MB * MB + (wave * 4 + r) * 64 + lane];
  // the place of element r
  auto at = [&](int r) { return (ti * 16 + k4 + 4 * r) * LQ + tj * 16 + l16; };
  auto diagonal = [&](int r) { return ti == tj && k4 + 4 * r == l16; };
  double trace = 0.0;
#pragma unroll
  for (int r = 0; r < 4; ++r) trace += diagonal(r) ? mine[r] : 0.0;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) trace += __shfl_xor(trace, d);
  if (lane == 0) traces[wave] = trace;
  __syncthreads();
  trace = 0.0;
  for (int i = 0; i < T * T; ++i) trace += traces[i];
  const double norm = sqrt(trace) + a.eps, f = from_x ? 1.0 : norm == 0.0 ? 0.0 : 1.0 / norm;
#pragma unroll
  for (int r = 0; r < 4; ++r) A[at(r)] = mine[r] * f * f;
  // rows of p times rows of q: all matrices here are symmetric
  auto multiply = [&](const double* p, const double* q) {
    // two sums: a product takes twice as long to end as to start
    f64x4 even = {0.0, 0.0, 0.0, 0.0}, odd = even;
#pragma unroll 4
    for (int k = 0; k < MB; k += 8) {
      even = product(p[(ti * 16 + l16) * LQ + k + k4], q[(tj * 16 + l16) * LQ + k + k4], even);
      odd = product(p[(ti * 16 + l16) * LQ + k + 4 + k4], q[(tj * 16 + l16) * LQ + k + 4 + k4], odd);
    }
    return even + odd;
  };
  const double ca = a.a, cb = a.b, cc = a.c;
  for (int step = 0; step < steps; ++step) {
    __syncthreads();
    const f64x4 square = multiply(A, A);
#pragma unroll
    for (int r = 0; r < 4; ++r) B[at(r)] = cb * A[at(r)] + cc * square[r] + (diagonal(r) ? ca : 0.0);
    __syncthreads();
    f64x4 q, w;
    if (step == 0) {
#pragma unroll
      for (int r = 0; r < 4; ++r) q[r] = B[at(r)];
    } else {
      q = multiply(B, Q);
    }
    if (step + 1 < steps) {
      w = multiply(B, A);
#pragma unroll
      for (int r = 0; r < 4; ++r) W[at(r)] = w[r];
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; ++r) Q[at(r)] = q[r];
    if (step + 1 < steps) {
      w = multiply(W, B);
#pragma unroll
      for (int r = 0; r < 4; ++r) A[at(r)] = w[r];
    }
  }
  __syncthreads();
  double* const out = a.q + (size_t)b * (MB * MB + 1);
  for (int i = threadIdx.x; i < MB * MB; i += MB * MB / 4) out[i] = Q[i / MB * LQ + i % MB];
  if (threadIdx.x == 0) out[MB * MB] = f;
}

// O = Q u / (|u| + eps) or Q X of 64 columns: X, the user's result, or the parameters' step by it
template <int MB, bool FROM_X, bool TO_X>
__global__ void __launch_bounds__(THR) apply_kernel(const MuonArgs a) {
  constexpr int T = MB / 16, LQ = MB + 4;
  using Element = std::conditional_t<FROM_X, double, float>;
  __shared__ __align__(16) Element u[MB * LD];
  __shared__ double Q[MB * LQ];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, k4 = lane >> 4, b = blockIdx.y, n0 = blockIdx.x * COLS;
  const MuonStack& s = muon_stack(a, a.first + b);
  const size_t base = (size_t)(a.first + b - s.first) * a.M * a.N;
  const bool whole = (s.wide ? a.N : a.M) % 4 == 0;
  const float gs = a.grad_scale ? *a.grad_scale : 1.f;
  const double* const in = a.q + (size_t)b * (MB * MB + 1);
  for (int i = threadIdx.x; i < MB * MB; i += THR) Q[i / MB * LQ + i % MB] = in[i];
  const double f = in[MB * MB];
  if constexpr (FROM_X) {
    read_x<MB>(a, b, n0, u);
  } else {
    for (int i = threadIdx.x; i < MB * LD / 4; i += THR) *(f32x4*)(u + 4 * i) = f32x4{0.f, 0.f, 0.f, 0.f};
    __syncthreads();
    user_elements<MB>(a, s, base, n0, [&](size_t at, int j, int n, int left) {
      const f32x4 v = read_u(a, s, at, left, whole, gs, false);
#pragma unroll
      for (int z = 0; z < 4; ++z)
        if (z < left) u[s.wide ? j * LD + n + z : (j + z) * LD + n] = v[z];
    });
  }
  __syncthreads();
  f64x4 acc[T];  // all rows of 16 columns
#pragma unroll
  for (int i = 0; i < T; ++i) acc[i] = f64x4{0.0, 0.0, 0.0, 0.0};
  for (int k = 0; k < MB; k += 4) {
    const double x = u[(k + k4) * LD + wave * 16 + l16] * f;
#pragma unroll
    for (int i = 0; i < T; ++i) acc[i] = product(Q[(i * 16 + l16) * LQ + k + k4], x, acc[i]);
  }
  if constexpr (TO_X) {  // in place: these columns are this workgroup's, and have been read
    double* const x = kept_x(a, b);
    const int n = n0 + wave * 16 + l16;
#pragma unroll
    for (int i = 0; i < T; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = i * 16 + k4 + 4 * r;
        if (j < a.M && n < a.N) x[(size_t)j * a.N + n] = acc[i][r];
      }
    return;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < T; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) u[(i * 16 + k4 + 4 * r) * LD + wave * 16 + l16] = (float)acc[i][r];
  __syncthreads();
  const float lr = a.lr_dev ? *a.lr_dev : a.lr, keep = 1.f - lr * a.wd, by = lr * s.scale;
  user_elements<MB>(a, s, base, n0, [&](size_t at, int j, int n, int left) {
    f32x4 v;
#pragma unroll
    for (int z = 0; z < 4; ++z) v[z] = z < left ? (float)u[s.wide ? j * LD + n + z : (j + z) * LD + n] : 0.f;
    if (whole) {
      if (s.m) {
        f32x4 old;
        if (s.master || a.out_f32) {
          old = *(const f32x4*)((s.master ? s.master : (const float*)s.out) + at);
        } else {
          const u32x2 w = *(const u32x2*)((const uint16_t*)s.out + at);
          old = f32x4{bf16lo(w[0]), bf16hi(w[0]), bf16lo(w[1]), bf16hi(w[1])};
        }
        v = old * keep - by * v;
        if (s.master) *(f32x4*)(s.master + at) = v;
      }
      if (a.out_f32) *(f32x4*)((float*)s.out + at) = v;
      else *(u32x2*)((uint16_t*)s.out + at) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      return;
    }
#pragma unroll
    for (int z = 0; z < 4; ++z)
      if (z < left) {
        float w = v[z];
        if (s.m) {
          const float old = s.master ? s.master[at + z] : a.out_f32 ? ((const float*)s.out)[at + z] : bf16_to_f32(((const uint16_t*)s.out)[at + z]);
          w = old * keep - by * w;
          if (s.master) s.master[at + z] = w;
        }
        if (a.out_f32) ((float*)s.out)[at + z] = w;
        else ((uint16_t*)s.out)[at + z] = __builtin_bit_cast(uint16_t, (__bf16)w);
      }
  });
}

template <int MB, bool FROM_X, bool TO_X>
void launch(const MuonArgs& a, int steps, hipStream_t st) {
  gram_kernel<MB, FROM_X><<<dim3(a.parts, a.count), THR, 0, st>>>(a);
  steps_kernel<MB><<<a.count, MB * MB / 4, 0, st>>>(a, steps, FROM_X);
  apply_kernel<MB, FROM_X, TO_X><<<dim3((a.N + COLS - 1) / COLS, a.count), THR, 0, st>>>(a);
}

// `runs` equal runs of steps
template <int MB>
void launch_runs(const MuonArgs& a, int steps, int runs, hipStream_t st) {
  if (runs == 1) return launch<MB, false, false>(a, steps, st);
  for (int i = 0; i < runs; ++i) {
    const int n = steps * (i + 1) / runs - steps * i / runs;
    if (i == 0) launch<MB, false, true>(a, n, st);
    else if (i + 1 < runs) launch<MB, true, true>(a, n, st);
    else launch<MB, true, false>(a, n, st);
  }
}

}  // namespace

// Columns of a part: enough parts to spread a long matrix over the card, no more than 64 to be added up one after the other
int thin_part(int N) {
  const int p = (N + 63) / 64;
  return (p < 4 * COLS ? 4 * COLS : (p + COLS - 1) / COLS * COLS);
}

// Short sides from 33 on with a long one of up to 256 are quicker by one workgroup a matrix and 16-bit operands, although it pads
// them to 128: 2 of 60 x 60 take 28 us in bf16 and 48 in fp32, of 60 x 200 37 and 70, here 75 to 80, 60 of them in `steps`.
// With a short side of up to 32 these take 28 (2 of 60 x 300: 90).
bool muon_thin(int M, int N) { return M <= 32 || (M <= THIN_MAX && !muon_small(M, N)); }

hipError_t launch_muon_thin(const MuonArgs& a, int steps, int runs, hipStream_t st) {
  if (!muon_thin(a.M, a.N) || runs < 1 || runs > steps || (runs > 1 && !a.xs)) return hipErrorInvalidValue;
  if (a.M <= 32) launch_runs<32>(a, steps, runs, st);
  else launch_runs<64>(a, steps, runs, st);
  return hipGetLastError();
}

}  // namespace moe
