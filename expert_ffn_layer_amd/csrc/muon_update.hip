// What the Muon step does before its products: the momentum with the matrices' norms, and the normalised matrices.
#include "muon.h"

namespace moe {

namespace {

constexpr int THR = 256;

constexpr int PART = 16384;  // elements of a workgroup that sums

// `4` consecutive elements, or one
__device__ __forceinline__ f32x4 load_g4(const MuonArgs& a, const void* g, size_t i, float gs) {
  f32x4 v;
  if (a.g_f32) {
    v = *(const f32x4*)((const float*)g + i);
  } else {
    const u32x2 w = *(const u32x2*)((const uint16_t*)g + i);
    v = f32x4{bf16lo(w[0]), bf16hi(w[0]), bf16lo(w[1]), bf16hi(w[1])};
  }
  return a.grad_scale ? v * gs : v;
}
__device__ __forceinline__ float load_g(const MuonArgs& a, const void* g, size_t i, float gs) {
  const float v = a.g_f32 ? ((const float*)g)[i] : bf16_to_f32(((const uint16_t*)g)[i]);
  return a.grad_scale ? v * gs : v;
}

// m = mu m + g', and the sum of u^2 of this workgroup's part of a matrix, u = g' + mu m (Nesterov), m or g'. Sums are
// in 64 bits: no gradient overflows or vanishes in them. A part is always the same elements: the same bits on every run.
// Bound by memory: 10 bytes an element with a bf16 gradient, 32 matrices of 7168 x 2048 in 917 us, 5.1 TB/s.
__global__ void __launch_bounds__(THR) momentum_kernel(const MuonArgs a) {
  const int b = blockIdx.y, part = blockIdx.x;
  const MuonStack& s = muon_stack(a, a.first + b);
  const size_t n = (size_t)a.M * a.N, base = (size_t)(a.first + b - s.first) * n, from = (size_t)part * PART;
  const size_t to = from + PART < n ? from + PART : n;
  const float gs = a.grad_scale ? *a.grad_scale : 1.f;
  double sum = 0.0;
  if (n % 4 == 0) {
#pragma unroll 4
    for (size_t i = from + 4 * threadIdx.x; i < to; i += 4 * THR) {
      f32x4 u = load_g4(a, s.g, base + i, gs);
      if (s.m) {
        f32x4 m = *(const f32x4*)(s.m + base + i);
        m = a.momentum * m + u;
        *(f32x4*)(s.m + base + i) = m;
        u = a.nesterov ? u + a.momentum * m : m;
      }
#pragma unroll
      for (int z = 0; z < 4; ++z) sum += (double)u[z] * u[z];
    }
  } else {
    // eight loads of each at a time; behind the end the first of them, which does not count
    auto all = [&](auto get) __attribute__((always_inline)) {
      for (size_t i = from + threadIdx.x; i < to; i += 8 * THR) {
        float u[8], m[8];
#pragma unroll
        for (int z = 0; z < 8; ++z) {
          const size_t at = base + (i + z * THR < to ? i + z * THR : i);
          u[z] = get(at);
          if (s.m) m[z] = s.m[at];
        }
#pragma unroll
        for (int z = 0; z < 8; ++z) {
          if (i + z * THR >= to) break;
          if (a.grad_scale) u[z] *= gs;
          if (s.m) {
            m[z] = a.momentum * m[z] + u[z];
            s.m[base + i + z * THR] = m[z];
            u[z] = a.nesterov ? u[z] + a.momentum * m[z] : m[z];
          }
          sum += (double)u[z] * u[z];
        }
      }
    };
    if (a.g_f32) all([&](size_t at) { return ((const float*)s.g)[at]; });
    else all([&](size_t at) { return bf16_to_f32(((const uint16_t*)s.g)[at]); });
  }
  __shared__ double part_sum[THR / 64];
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
  if ((threadIdx.x & 63) == 0) part_sum[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) a.sums[(size_t)b * a.parts + part] = part_sum[0] + part_sum[1] + part_sum[2] + part_sum[3];
}

// A tile of X, 64 of the short side x 64 of the long one, through LDS: the user's rows are read 16 bytes a lane, X's written so.
// Bound by memory: 10 bytes an element with a bf16 gradient and momentum; of 32 matrices of 7168 x 2048 without, 6 bytes in
// 0.70 ms, 4.0 TB/s (0.94 with loads that waited for the sums and for each other).
__global__ void __launch_bounds__(THR) normalize_kernel(const MuonArgs a) {
  __shared__ float tile[64][65];
  const int b = blockIdx.z, n0 = blockIdx.x * 64, j0 = blockIdx.y * 64;
  const MuonStack& s = muon_stack(a, a.first + b);
  const size_t base = (size_t)(a.first + b - s.first) * a.M * a.N;
  const float gs = a.grad_scale ? *a.grad_scale : 1.f;
  const int cols = s.wide ? a.N : a.M, rows = s.wide ? a.M : a.N, c0 = s.wide ? n0 : j0, r0 = s.wide ? j0 : n0;
  const int c = 4 * (threadIdx.x & 15);
  // the elements, all loads before the first use; what lies outside reads the matrix's first
  f32x4 u[4], m[4];
  auto inside = [&](int it) { return r0 + it * 16 + (int)(threadIdx.x >> 4) < rows && c0 + c < cols; };
  auto place = [&](int it) { return base + (inside(it) ? (size_t)(r0 + it * 16 + (threadIdx.x >> 4)) * cols + c0 + c : 0); };
  if (cols % 4 == 0) {
#pragma unroll
    for (int it = 0; it < 4; ++it) u[it] = load_g4(a, s.g, place(it), gs);
    if (s.m) {
#pragma unroll
      for (int it = 0; it < 4; ++it) m[it] = *(const f32x4*)(s.m + place(it));
    }
  } else {
#pragma unroll
    for (int it = 0; it < 4; ++it)
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const size_t at = place(it) + (inside(it) && c0 + c + z < cols ? z : 0);
        u[it][z] = load_g(a, s.g, at, gs);
        if (s.m) m[it][z] = s.m[at];
      }
  }
  __shared__ double part_sum[THR / 64];
  double sum = 0.0;
#pragma unroll 4
  for (int i = threadIdx.x; i < a.parts; i += THR) sum += a.sums[(size_t)b * a.parts + i];
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
  if ((threadIdx.x & 63) == 0) part_sum[threadIdx.x >> 6] = sum;
  __syncthreads();
  const double norm = sqrt(part_sum[0] + part_sum[1] + part_sum[2] + part_sum[3]) + a.eps;
  // a matrix of zeros stays one without an eps, too
  const double f = norm == 0.0 ? 0.0 : (double)MUON_SCALE / norm;
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int r = it * 16 + (threadIdx.x >> 4);
    f32x4 v = u[it];
    if (s.m) v = a.nesterov ? u[it] + a.momentum * m[it] : m[it];
#pragma unroll
    for (int z = 0; z < 4; ++z) v[z] = inside(it) && c0 + c + z < cols ? (float)(v[z] * f) : 0.f;
#pragma unroll
    for (int z = 0; z < 4; ++z) {
      if (s.wide) tile[r][c + z] = v[z];
      else tile[c + z][r] = v[z];
    }
  }
  __syncthreads();
  const size_t at = (size_t)b * a.Mp * a.Np;
  const int n = 8 * (threadIdx.x & 7);
#pragma unroll
  for (int it = 0; it < 2; ++it) {
    const int j = it * 32 + (threadIdx.x >> 3);
    typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;
    f16x8 hi, lo;
#pragma unroll
    for (int z = 0; z < 8; ++z) {
      const float v = tile[j][n + z];
      hi[z] = (_Float16)v;
      lo[z] = (_Float16)(v - (float)hi[z]);
    }
    const size_t i = at + (size_t)(j0 + j) * a.Np + n0 + n;
    *(u32x4*)(a.x + i) = __builtin_bit_cast(u32x4, hi);
    *(u32x4*)(a.x_lo + i) = __builtin_bit_cast(u32x4, lo);
  }
}

}  // namespace

int muon_parts(long long elements) { return (int)((elements + PART - 1) / PART); }

hipError_t launch_muon_momentum(const MuonArgs& a, hipStream_t st) {
  momentum_kernel<<<dim3(a.parts, a.count), THR, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_muon_normalize(const MuonArgs& a, hipStream_t st) {
  normalize_kernel<<<dim3(a.Np / 64, a.Mp / 64, a.count), THR, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace moe
