// What the Muon step does before its products: the momentum with the matrices' norms, and the normalised matrices.
#include "muon.h"

namespace moe {

namespace {

constexpr int THR = 256;

__device__ __forceinline__ float load_g(const MuonArgs& a, const void* g, size_t i, float gs) {
  const float v = a.g_f32 ? ((const float*)g)[i] : bf16_to_f32(((const uint16_t*)g)[i]);
  return a.grad_scale ? v * gs : v;
}

// m = mu m + g', and the sum of u^2 of this workgroup's part of a matrix, u = g' + mu m (Nesterov), m or g'. Sums are
// in 64 bits: no gradient overflows or vanishes in them. Part p of MUON_SUMS, always the same elements: the same bits
// on every run.
__global__ void __launch_bounds__(THR) momentum_kernel(const MuonArgs a) {
  const int b = blockIdx.y, part = blockIdx.x;
  const MuonStack& s = muon_stack(a, a.first + b);
  const size_t n = (size_t)a.M * a.N, base = (size_t)(a.first + b - s.first) * n;
  const float gs = a.grad_scale ? *a.grad_scale : 1.f;
  double sum = 0.0;
  for (size_t i = (size_t)part * THR + threadIdx.x; i < n; i += (size_t)MUON_SUMS * THR) {
    float u = load_g(a, s.g, base + i, gs);
    if (s.m) {
      const float m = a.momentum * s.m[base + i] + u;
      s.m[base + i] = m;
      u = a.nesterov ? u + a.momentum * m : m;
    }
    sum += (double)u * u;
  }
  __shared__ double part_sum[THR / 64];
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
  if ((threadIdx.x & 63) == 0) part_sum[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) a.sums[b * MUON_SUMS + part] = part_sum[0] + part_sum[1] + part_sum[2] + part_sum[3];
}

// A tile of 64 x 64 of X; matrices with the long side first are transposed through LDS.
__global__ void __launch_bounds__(THR) normalize_kernel(const MuonArgs a) {
  __shared__ float tile[64][65];
  const int b = blockIdx.z, n0 = blockIdx.x * 64, j0 = blockIdx.y * 64;
  const MuonStack& s = muon_stack(a, a.first + b);
  const size_t base = (size_t)(a.first + b - s.first) * a.M * a.N;
  double sum = a.sums[b * MUON_SUMS + (threadIdx.x & 63)];
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
  const double norm = sqrt(sum) + a.eps;
  // a matrix of zeros stays one without an eps, too
  const double f = norm == 0.0 ? 0.0 : (double)MUON_SCALE / norm;
  const float gs = a.grad_scale ? *a.grad_scale : 1.f;
  const int c = threadIdx.x & 63, r0 = threadIdx.x >> 6;
  for (int r = r0; r < 64; r += 4) {
    // n: place on the long side, j: on the short one; lanes run along the user's rows
    const int n = n0 + (s.wide ? c : r), j = j0 + (s.wide ? r : c);
    float v = 0.f;
    if (n < a.N && j < a.M) {
      const size_t i = base + (s.wide ? (size_t)j * a.N + n : (size_t)n * a.M + j);
      float u = load_g(a, s.g, i, gs);
      if (s.m) u = a.nesterov ? u + a.momentum * s.m[i] : s.m[i];
      v = (float)(u * f);
    }
    if (s.wide) tile[r][c] = v;
    else tile[c][r] = v;
  }
  __syncthreads();
  const size_t at = (size_t)b * a.Mp * a.Np;
  for (int r = r0; r < 64; r += 4) {
    const float v = tile[r][c];
    const _Float16 hi = (_Float16)v, lo = (_Float16)(v - (float)hi);
    const size_t i = at + (size_t)(j0 + r) * a.Np + n0 + c;
    a.x[i] = __builtin_bit_cast(uint16_t, hi);
    a.x_lo[i] = __builtin_bit_cast(uint16_t, lo);
  }
}

}  // namespace

hipError_t launch_muon_momentum(const MuonArgs& a, hipStream_t st) {
  momentum_kernel<<<dim3(MUON_SUMS, a.count), THR, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_muon_normalize(const MuonArgs& a, hipStream_t st) {
  normalize_kernel<<<dim3(a.Np / 64, a.Mp / 64, a.count), THR, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace moe
