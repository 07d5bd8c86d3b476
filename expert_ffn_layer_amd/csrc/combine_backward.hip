// Gradient of the weighted combine y[t] = sum_j w[t][j] y_perm[slot(t, j)]:
//   dy_perm[slot(t, j)] = w[t][j] dy[t]      dw[t][j] = dy[t] . y_perm[slot(t, j)]
//
// Bound by memory: a row of y_perm read and a row of dy_perm written per pair. One wave per pair,
// 16 bytes a lane; the k pairs of a token are neighbours, so dy[t] comes from cache after its first
// reader. The dot is summed in fp32, per lane in ascending order and then over the lanes by a fixed
// tree: no atomics, the same bits on every run.
#include "train.h"

namespace moe {

namespace {

constexpr int CBTHR = 256;

template <int ACT>
__global__ void __launch_bounds__(CBTHR) combine_backward_kernel(const uint8_t* __restrict__ dy,
                                                                const uint8_t* __restrict__ y_perm,
                                                                const int32_t* __restrict__ pair_slot,
                                                                const float* __restrict__ w,
                                                                uint8_t* __restrict__ dy_perm,
                                                                float* __restrict__ dw, int H, int k, int P) {
  constexpr int EB = ACT == MOE_F32 ? 4 : 2;
  constexpr int V = 16 / EB;
  constexpr int U = 4;  // chunks in flight per lane
  const int q = __builtin_amdgcn_readfirstlane(blockIdx.x * (CBTHR / WAVE) + (threadIdx.x >> 6));
  if (q >= P) return;
  const int lane = threadIdx.x & 63;
  const int slot = pair_slot[q];
  if ((unsigned)slot >= (unsigned)P) {
    if (lane == 0) dw[q] = 0.f;
    return;
  }
  const float wt = w[q];
  const size_t row = (size_t)H * EB;
  const uint8_t* dyr = dy + (size_t)(q / k) * row;
  const uint8_t* yr = y_perm + (size_t)slot * row;
  uint8_t* out = dy_perm + (size_t)slot * row;
  const int chunks = H / V;
  float dot = 0.f;
  for (int c0 = lane; c0 < chunks; c0 += U * WAVE) {
    u32x4 d[U], v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * WAVE;
      d[u] = v[u] = u32x4{0u, 0u, 0u, 0u};
      if (c < chunks) {
        d[u] = *(const u32x4*)(dyr + (size_t)c * 16);
        v[u] = *(const u32x4*)(yr + (size_t)c * 16);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * WAVE;
      if (c >= chunks) continue;
      u32x4 o;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (ACT == MOE_F32) {
          const float x = __uint_as_float(d[u][i]);
          dot += x * __uint_as_float(v[u][i]);
          o[i] = __float_as_uint(wt * x);
        } else {
          dot += bf16lo(d[u][i]) * bf16lo(v[u][i]);
          dot += bf16hi(d[u][i]) * bf16hi(v[u][i]);
          o[i] = pack_bf16x2(wt * bf16lo(d[u][i]), wt * bf16hi(d[u][i]));
        }
      }
      *(u32x4*)(out + (size_t)c * 16) = o;
    }
  }
#pragma unroll
  for (int s = 1; s < WAVE; s <<= 1) dot += __shfl_xor(dot, s);
  if (lane == 0) dw[q] = dot;
}

}  // namespace

hipError_t launch_combine_backward(int act, const void* dy, const void* y_perm, const int32_t* pair_slot, const float* w,
                                   void* dy_perm, float* dw, int T, int H, int k, hipStream_t st) {
  const int P = T * k;
  if (P == 0) return hipSuccess;
  const unsigned grid = (unsigned)((P + CBTHR / WAVE - 1) / (CBTHR / WAVE));
  if (act == MOE_F32)
    combine_backward_kernel<MOE_F32><<<grid, CBTHR, 0, st>>>((const uint8_t*)dy, (const uint8_t*)y_perm, pair_slot, w,
                                                            (uint8_t*)dy_perm, dw, H, k, P);
  else
    combine_backward_kernel<MOE_BF16><<<grid, CBTHR, 0, st>>>((const uint8_t*)dy, (const uint8_t*)y_perm, pair_slot, w,
                                                             (uint8_t*)dy_perm, dw, H, k, P);
  return hipGetLastError();
}

}  // namespace moe
