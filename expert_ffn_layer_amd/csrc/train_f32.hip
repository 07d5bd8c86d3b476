// The gated feed-forward block's products on fp32 matrix instructions (v_mfma_f32_16x16x4_f32),
// for fp32 activations and weights; forms as listed in train.h.
//
// C[m][n] = sum_k P(m, k) Q(n, k). A workgroup of 4 waves computes 64 x 64 of C, each wave 32 x 32
// as 2 x 2 MFMA tiles, in 32-deep steps: both operands pass through registers into LDS, the next
// step's loads in flight behind the current step's products. An operand whose reduction index is
// contiguous in memory is kept [index][k] and read 16 bytes a lane (k = 4 g + j for lane group g
// and MFMA j); one whose own index is contiguous is kept [k][index] and read 4 bytes a lane at the
// same k. Row strides of 36 and 68 floats make both reads free of bank conflicts. The column
// operand is the MFMA's A, so a lane ends with 4 consecutive columns of one row.
#include "train.h"

namespace moe {

namespace {

constexpr int TM = 64, TN = 64, TK = 32;
constexpr int LDK = 36;  // floats per row of a [index][k] tile
constexpr int LDM = 68;  // floats per row of a [k][index] tile
constexpr int TTHR = 256;

typedef __attribute__((ext_vector_type(4))) float fvec4;

template <typename T>
__device__ __forceinline__ fvec4 load4(const T* p);
template <>
__device__ __forceinline__ fvec4 load4<float>(const float* p) {
  return *(const fvec4*)p;
}
template <>
__device__ __forceinline__ fvec4 load4<uint16_t>(const uint16_t* p) {
  const u32x2 w = *(const u32x2*)p;
  return fvec4{bf16lo(w[0]), bf16hi(w[0]), bf16lo(w[1]), bf16hi(w[1])};
}
template <typename T>
__device__ __forceinline__ void store4(T* p, fvec4 v);
template <>
__device__ __forceinline__ void store4<float>(float* p, fvec4 v) {
  *(fvec4*)p = v;
}
template <>
__device__ __forceinline__ void store4<uint16_t>(uint16_t* p, fvec4 v) {
  *(u32x2*)p = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

template <typename T, int FORM>
__global__ void __launch_bounds__(TTHR) train_f32_kernel(const TrainArgs a) {
  constexpr bool P_KC = FORM != TF_DW;                       // row operand contiguous along k
  constexpr bool Q_KC = FORM == TF_DH || FORM == TF_DX;      // column operand contiguous along k
  __shared__ __align__(16) float lp[P_KC ? TM * LDK : TK * LDM];
  __shared__ __align__(16) float lq[Q_KC ? TN * LDK : TK * LDM];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wr = wave >> 1, wc = wave & 1, l16 = lane & 15, g = lane >> 4;
  const size_t H = a.H, I = a.I, HI = H * I;

  // the tile: rows [m0, m0 + 64) of C up to mend, columns [n0, ...); k in [0, K)
  int e, m0, mend, n0, K, beg = 0;
  int mat = 0;  // TF_DW: 0 gate, 1 up, 2 down
  if constexpr (FORM == TF_DW) {
    const int tm = (int)((blockIdx.z == 2 ? I : H) / TM), tn = (int)((blockIdx.z == 2 ? H : I) / TN);
    mat = blockIdx.z;
    e = blockIdx.y;
    if ((int)blockIdx.x >= tm * tn) return;
    m0 = (int)(blockIdx.x / tn) * TM;
    n0 = (int)(blockIdx.x % tn) * TN;
    mend = mat == 2 ? a.I : a.H;
    int end;
    group_rows(a.off, e, a.P, beg, end);
    K = end - beg;
  } else {
    RowTile t;
    if (!find_row_tile(a.off, a.E, a.P, TM, blockIdx.x, t)) return;
    e = t.e;
    m0 = t.row0;
    mend = t.end;
    n0 = blockIdx.y * (FORM == TF_GATE_UP ? TN / 2 : TN);
    K = FORM == TF_GATE_UP || FORM == TF_DH ? a.H : FORM == TF_DOWN ? a.I : 2 * a.I;
  }

  // chunk of 4 elements of the row operand: index i (0..63) and reduction element k
  auto load_p = [&](int i, int k) -> fvec4 {
    const fvec4 z = {0.f, 0.f, 0.f, 0.f};
    if constexpr (FORM == TF_DW) {
      if (k >= K) return z;
      const int r = beg + k;
      if (mat == 2) return load4((const T*)a.h + r * I + m0 + i);
      const int s = a.slot_token ? a.slot_token[r] : r;
      return (unsigned)s < (unsigned)a.xrows ? load4((const T*)a.x + s * H + m0 + i) : z;
    } else {
      const int r = m0 + i;
      if (r >= mend) return z;
      if constexpr (FORM == TF_GATE_UP) {
        const int s = a.slot_token ? a.slot_token[r] : r;
        return (unsigned)s < (unsigned)a.xrows ? load4((const T*)a.x + s * H + k) : z;
      } else if constexpr (FORM == TF_DOWN) {
        return load4((const T*)a.h + r * I + k);
      } else if constexpr (FORM == TF_DH) {
        return load4((const T*)a.dy + r * H + k);
      } else {
        return load4((const T*)a.dgu + r * (2 * I) + k);
      }
    }
  };
  // chunk of the column operand: index i (0..63), reduction element k
  auto load_q = [&](int i, int k) -> fvec4 {
    if constexpr (FORM == TF_DW) {
      if (k >= K) return fvec4{0.f, 0.f, 0.f, 0.f};
      const int r = beg + k;
      if (mat == 2) return load4((const T*)a.dy + r * H + n0 + i);
      return load4((const T*)a.dgu + r * (2 * I) + mat * I + n0 + i);
    } else if constexpr (FORM == TF_GATE_UP) {  // columns 0..31 gate, 32..63 up
      return load4((const T*)(i < TN / 2 ? a.gate : a.up) + e * HI + k * I + n0 + (i & (TN / 2 - 1)));
    } else if constexpr (FORM == TF_DOWN) {
      return load4((const T*)a.down + e * HI + k * H + n0 + i);
    } else if constexpr (FORM == TF_DH) {
      return load4((const T*)a.down + e * HI + (n0 + i) * H + k);
    } else {
      return k < (int)I ? load4((const T*)a.gate + e * HI + (n0 + i) * I + k)
                        : load4((const T*)a.up + e * HI + (n0 + i) * I + (k - I));
    }
  };
  // this thread's two chunks of each operand: [index][k] tiles are 64 x 8 chunks, [k][index] 32 x 16
  auto chunk = [&](bool kc, int u, int& i, int& k) {
    const int c = tid + u * TTHR;
    if (kc) {
      i = c >> 3;
      k = (c & 7) * 4;
    } else {
      i = (c & 15) * 4;
      k = c >> 4;
    }
  };
  fvec4 rp[2], rq[2];
  auto fetch = [&](int k0) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      int i, k;
      chunk(P_KC, u, i, k);
      rp[u] = load_p(i, k0 + k);
      chunk(Q_KC, u, i, k);
      rq[u] = load_q(i, k0 + k);
    }
  };

  f32x4 acc[2][2];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  auto qcol = [&](int t) { return FORM == TF_GATE_UP ? t * 32 + wc * 16 : wc * 32 + t * 16; };
  if (K > 0) fetch(0);
  for (int k0 = 0; k0 < K; k0 += TK) {
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      int i, k;
      chunk(P_KC, u, i, k);
      *(fvec4*)(P_KC ? lp + i * LDK + k : lp + k * LDM + i) = rp[u];
      chunk(Q_KC, u, i, k);
      *(fvec4*)(Q_KC ? lq + i * LDK + k : lq + k * LDM + i) = rq[u];
    }
    __syncthreads();
    if (k0 + TK < K) fetch(k0 + TK);
#pragma unroll
    for (int kk = 0; kk < TK; kk += 16) {
      fvec4 p[2], q[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int m = wr * 32 + t * 16 + l16, n = qcol(t) + l16;
        if constexpr (P_KC) {
          p[t] = *(const fvec4*)(lp + m * LDK + kk + 4 * g);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) p[t][j] = lp[(kk + 4 * g + j) * LDM + m];
        }
        if constexpr (Q_KC) {
          q[t] = *(const fvec4*)(lq + n * LDK + kk + 4 * g);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) q[t][j] = lq[(kk + 4 * g + j) * LDM + n];
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            acc[t][r] = __builtin_amdgcn_mfma_f32_16x16x4f32(q[t][j], p[r][j], acc[t][r], 0, 0, 0);
    }
  }

  // lane: columns qcol(t) + 4 g + [0, 4) of row wr * 32 + r * 16 + l16
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int m = m0 + wr * 32 + r * 16 + l16;
    if (m >= mend) continue;
    if constexpr (FORM == TF_GATE_UP) {
      const size_t at = m * I + n0 + wc * 16 + 4 * g;
      fvec4 hv;
#pragma unroll
      for (int i = 0; i < 4; ++i) hv[i] = silu(acc[0][r][i]) * acc[1][r][i];
      if (a.g) {
        store4((T*)a.g + at, acc[0][r]);
        store4((T*)a.u + at, acc[1][r]);
      }
      store4((T*)a.h + at, hv);
      continue;
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int n = n0 + qcol(t) + 4 * g;
      if constexpr (FORM == TF_DH) {
        const fvec4 gv = load4((const T*)a.g + m * I + n), uv = load4((const T*)a.u + m * I + n);
        fvec4 dg, du, hv;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float s = 1.0f / (1.0f + __expf(-gv[i])), si = gv[i] * s, dh = acc[t][r][i];
          du[i] = dh * si;
          dg[i] = dh * uv[i] * (s + si * (1.0f - s));
          hv[i] = si * uv[i];
        }
        store4((T*)a.dgu + m * (2 * I) + n, dg);
        store4((T*)a.dgu + m * (2 * I) + I + n, du);
        store4((T*)a.h + m * I + n, hv);
      } else if constexpr (FORM == TF_DW) {
        T* o = (T*)(mat == 0 ? a.dgate : mat == 1 ? a.dup : a.ddown) + e * HI;
        store4(o + m * (mat == 2 ? H : I) + n, acc[t][r]);
      } else {
        store4((T*)(FORM == TF_DOWN ? a.y : a.dx) + m * H + n, acc[t][r]);
      }
    }
  }
}

template <typename T>
hipError_t launch(TrainForm form, const TrainArgs& a, hipStream_t st) {
  const long long mt = max_row_tiles(a.P, a.E, TM);
  if (form != TF_DW && mt == 0) return hipSuccess;
  const unsigned rows = (unsigned)mt, H = (unsigned)a.H, I = (unsigned)a.I;
  switch (form) {
    case TF_GATE_UP: train_f32_kernel<T, TF_GATE_UP><<<dim3(rows, I / (TN / 2)), TTHR, 0, st>>>(a); break;
    case TF_DOWN: train_f32_kernel<T, TF_DOWN><<<dim3(rows, H / TN), TTHR, 0, st>>>(a); break;
    case TF_DH: train_f32_kernel<T, TF_DH><<<dim3(rows, I / TN), TTHR, 0, st>>>(a); break;
    case TF_DX: train_f32_kernel<T, TF_DX><<<dim3(rows, H / TN), TTHR, 0, st>>>(a); break;
    case TF_DW: train_f32_kernel<T, TF_DW><<<dim3(H / TM * (I / TN), a.E, 3), TTHR, 0, st>>>(a); break;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_train_f32(TrainForm form, const TrainArgs& a, hipStream_t st) { return launch<float>(form, a, st); }

}  // namespace moe
