// The gated feed-forward block's products on fp32 matrix instructions (v_mfma_f32_16x16x4_f32),
// for fp32 activations and weights; forms as listed in train.h.
//
// C[m][n] = sum_k P(m, k) Q(n, k). A workgroup of 4 waves computes 64 x 64 of C, each wave 32 x 32
// as 2 x 2 MFMA tiles (or 32 x 64 and 16 x 32, see choose below), in 32-deep steps: both operands
// pass through registers into LDS, four steps' loads in flight behind the products. An operand whose
// reduction index is contiguous in memory is kept [index][k] and read 16 bytes a lane (k = 4 g + j
// for lane group g and MFMA j); one whose own index is contiguous is kept [k][index] and read 4 bytes
// a lane at the same k. Row strides of N + 4 floats make both reads free of bank conflicts. The column
// operand is the MFMA's A, so a lane ends with 4 consecutive columns of one row.
//
// Bound by the matrix instructions where there are tiles enough (8192 rows, H 2048, I 4096, 8 groups: 113,
// 120, 111, 111 and 106 TFLOP/s for the five forms in order, the card's fp32 library product 140), by a chain of
// load, LDS and product per step below (16 tokens, H 256, I 128: 7.4 us and 5.1 us for the forward's two). The rows
// of x that the weight gradients reduce over are found by tokens fetched as many steps before them again.
#include "train.h"

namespace moe {

namespace {

constexpr int TN = 64, TK = 32;
constexpr int LDK = 36;  // floats per row of a [index][k] tile
constexpr int LDM = TN + 4;  // floats per row of a [k][index] column operand
constexpr int TTHR = 256;
constexpr int CUS = 256;

typedef __attribute__((ext_vector_type(4))) float fvec4;

__device__ const uint4 zero_chunk = {0u, 0u, 0u, 0u};

__device__ __forceinline__ fvec4 load4(const float* p) { return *(const __attribute__((address_space(1))) fvec4*)p; }
__device__ __forceinline__ void store4(float* p, fvec4 v) { *(fvec4*)p = v; }

constexpr int LDS_FLOATS = 2 * 64 * LDK;  // both operands of the largest tile

// One tile: x is its row tile (TF_DW: tile of the matrix), y its tile of columns (expert), z of TF_DW the matrix
template <int FORM, int TM>
__device__ __forceinline__ void tile(const TrainArgs& a, int bx, int by, int bz, float* lds) {
  constexpr int RT = TM / 32;                                // MFMA tiles of rows a wave has
  constexpr int LDP = TM + 4;                                // floats per row of a [k][index] row operand
  constexpr bool P_KC = FORM != TF_DW;                       // row operand contiguous along k
  constexpr bool Q_KC = FORM == TF_DH || FORM == TF_DX;      // column operand contiguous along k
  constexpr int PF = P_KC ? TM * LDK : TK * LDP, QF = Q_KC ? TN * LDK : TK * LDM;
  static_assert(PF + QF <= LDS_FLOATS && PF % 4 == 0, "operands fit the workgroup's LDS");
  float* const lp = lds;
  float* const lq = lds + PF;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wr = wave >> 1, wc = wave & 1, l16 = lane & 15, g = lane >> 4;
  const size_t H = a.H, I = a.I, HI = H * I;

  // the tile: rows [m0, m0 + TM) of C up to mend, columns [n0, ...); k in [0, K)
  int e, m0, mend, n0, K, beg = 0;
  int mat = 0;  // TF_DW: 0 gate, 1 up, 2 down
  if constexpr (FORM == TF_DW) {
    const int tm = (int)((bz == 2 ? I : H) / TM), tn = (int)((bz == 2 ? H : I) / TN);
    mat = bz;
    e = by;
    if (bx >= tm * tn) return;
    m0 = bx / tn * TM;
    n0 = bx % tn * TN;
    mend = mat == 2 ? a.I : a.H;
    int end;
    group_rows(a.off, e, a.P, beg, end);
    K = end - beg;
  } else {
    RowTile t;
    if (!find_row_tile(a.off, a.E, a.P, TM, bx, t)) return;
    e = t.e;
    m0 = t.row0;
    mend = t.end;
    n0 = by * (FORM == TF_GATE_UP ? TN / 2 : TN);
    K = FORM == TF_GATE_UP || FORM == TF_DH ? a.H : FORM == TF_DOWN ? a.I : 2 * a.I;
  }

  // Where 4 elements of an operand are: index i (0..63) and reduction element k. Rows past the group's end and
  // tokens outside x are zeros, by address: a load under a condition would be waited for at once.
  const float* const zeros = (const float*)&zero_chunk;
  int tok[2] = {-1, -1};  // TF_GATE_UP: row of x behind each row of the tile that this thread loads
  if constexpr (FORM == TF_GATE_UP) {
#pragma unroll
    for (int u = 0; u < RT; ++u) {
      const int r = m0 + u * 32 + (tid >> 3);
      if (r < mend) tok[u] = a.slot_token ? a.slot_token[r] : r;
      if ((unsigned)tok[u] >= (unsigned)a.xrows) tok[u] = -1;
    }
  }
  auto at_p = [&](int i, int k, int token) -> const float* {
    if constexpr (FORM == TF_DW) {
      if (k >= K) return zeros;
      if (mat == 2) return (const float*)a.h + (beg + k) * I + m0 + i;
      const int r = a.slot_token ? token : beg + k;
      return (unsigned)r < (unsigned)a.xrows ? (const float*)a.x + r * H + m0 + i : zeros;
    } else {
      const int r = m0 + i;
      if (r >= mend) return zeros;
      if constexpr (FORM == TF_GATE_UP) {
        return tok[i >= 32] >= 0 ? (const float*)a.x + tok[i >= 32] * H + k : zeros;
      } else if constexpr (FORM == TF_DOWN) {
        return (const float*)a.h + r * I + k;
      } else if constexpr (FORM == TF_DH) {
        return (const float*)a.dy + r * H + k;
      } else {
        return (const float*)a.dgu + r * (2 * I) + k;
      }
    }
  };
  auto at_q = [&](int i, int k) -> const float* {
    if constexpr (FORM == TF_DW) {
      if (k >= K) return zeros;
      const int r = beg + k;
      return mat == 2 ? (const float*)a.dy + r * H + n0 + i : (const float*)a.dgu + r * (2 * I) + mat * I + n0 + i;
    } else if constexpr (FORM == TF_GATE_UP) {  // columns 0..31 gate, 32..63 up
      return (const float*)(i < TN / 2 ? a.gate : a.up) + e * HI + k * I + n0 + (i & (TN / 2 - 1));
    } else if constexpr (FORM == TF_DOWN) {
      return (const float*)a.down + e * HI + k * H + n0 + i;
    } else if constexpr (FORM == TF_DH) {
      return (const float*)a.down + e * HI + (n0 + i) * H + k;
    } else {
      return k < (int)I ? (const float*)a.gate + e * HI + (n0 + i) * I + k
                        : (const float*)a.up + e * HI + (n0 + i) * I + (k - I);
    }
  };
  // this thread's chunks of an operand of N rows or columns: [index][k] tiles are N x 8 chunks, [k][index] 32 x N / 4
  auto chunk = [&](bool kc, int N, int u, int& i, int& k) __attribute__((always_inline)) {
    const int c = tid + u * TTHR;
    if (kc) {
      i = c >> 3;
      k = (c & 7) * 4;
    } else {
      i = c % (N / 4) * 4;
      k = c / (N / 4);
    }
  };
  // AHEAD steps' chunks wait in registers: about 1.7 us of products, more than a load takes
  constexpr int AHEAD = 4;
  fvec4 rp[AHEAD][RT], rq[AHEAD][2];
  // TF_DW: the token of reduction element k, fetched AHEAD steps before its row of x
  int tokens[AHEAD][2] = {};
  const int32_t* const token_at = FORM == TF_DW && a.slot_token && mat < 2 && K > 0 ? a.slot_token + beg : (const int32_t*)zeros;
  const int token_last = FORM == TF_DW && a.slot_token && mat < 2 ? K - 1 : 0;
  auto fetch_tokens = [&](int k0, int set) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < RT && FORM == TF_DW; ++u) {
      int i, k;
      chunk(P_KC, TM, u, i, k);
      tokens[set][u] = *(const __attribute__((address_space(1))) int32_t*)(token_at + min(k0 + k, token_last));
    }
  };
  auto fetch = [&](int k0, int set) __attribute__((always_inline)) {
    if (FORM != TF_DW) k0 = min(k0, K - TK);  // past the end the last step again, which nothing uses
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      int i, k;
      if (u < RT) {
        chunk(P_KC, TM, u, i, k);
        rp[set][u] = load4(at_p(i, k0 + k, tokens[set][u]));
      }
      chunk(Q_KC, TN, u, i, k);
      rq[set][u] = load4(at_q(i, k0 + k));
    }
    fetch_tokens(k0 + AHEAD * TK, set);
  };

  // A round's sums are added to the total at its end. On values of random sign the error of a product of K elements is
  // 0.43 sqrt(64 + K / 256) 2^-24 of its norm, where one chain's is 0.43 sqrt(K / 2): measured 3.5 2^-24 at K = 640,
  // 4.1 at 7168, 5.2 at 20000 and 10.6 at 140000, which only the weight gradients of a large group reach
  f32x4 acc[2][RT], total[2][RT];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[t][j] = total[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  auto qcol = [&](int t) { return FORM == TF_GATE_UP ? t * 32 + wc * 16 : wc * 32 + t * 16; };
  auto step = [&](int k0, int set) __attribute__((always_inline)) {
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      int i, k;
      if (u < RT) {
        chunk(P_KC, TM, u, i, k);
        *(fvec4*)(P_KC ? lp + i * LDK + k : lp + k * LDP + i) = rp[set][u];
      }
      chunk(Q_KC, TN, u, i, k);
      *(fvec4*)(Q_KC ? lq + i * LDK + k : lq + k * LDM + i) = rq[set][u];
    }
    __syncthreads();
    fetch(k0 + AHEAD * TK, set);
#pragma unroll
    for (int kk = 0; kk < TK; kk += 16) {
      fvec4 p[RT], q[2];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const int m = wr * (TM / 2) + r * 16 + l16;
        if constexpr (P_KC) {
          p[r] = *(const fvec4*)(lp + m * LDK + kk + 4 * g);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) p[r][j] = lp[(kk + 4 * g + j) * LDP + m];
        }
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int n = qcol(t) + l16;
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
          for (int r = 0; r < RT; ++r)
            acc[t][r] = __builtin_amdgcn_mfma_f32_16x16x4f32(q[t][j], p[r][j], acc[t][r], 0, 0, 0);
    }
  };
  // rounds of AHEAD steps: H and I are multiples of 128, the rows of TF_DW end anywhere and go on in zeros
  if (K > 0) {
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) fetch_tokens(u * TK, u);
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) fetch(u * TK, u);
  }
  for (int k0 = 0; k0 < K; k0 += AHEAD * TK) {
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      if (FORM == TF_DW && k0 + u * TK >= K) break;
      step(k0 + u * TK, u);
    }
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        total[t][r] += acc[t][r];
        acc[t][r] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
  }

  // lane: columns qcol(t) + 4 g + [0, 4) of row wr * TM / 2 + r * 16 + l16
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int m = m0 + wr * (TM / 2) + r * 16 + l16;
    if (m >= mend) continue;
    if constexpr (FORM == TF_GATE_UP) {
      const size_t at = m * I + n0 + wc * 16 + 4 * g;
      fvec4 hv;
#pragma unroll
      for (int i = 0; i < 4; ++i) hv[i] = silu(total[0][r][i]) * total[1][r][i];
      if (a.g) {
        store4((float*)a.g + at, total[0][r]);
        store4((float*)a.u + at, total[1][r]);
      }
      store4((float*)a.h + at, hv);
      continue;
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int n = n0 + qcol(t) + 4 * g;
      if constexpr (FORM == TF_DH) {
        const fvec4 gv = load4((const float*)a.g + m * I + n), uv = load4((const float*)a.u + m * I + n);
        fvec4 dg, du, hv;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float s = 1.0f / (1.0f + __expf(-gv[i])), si = gv[i] * s, dh = total[t][r][i];
          du[i] = dh * si;
          dg[i] = dh * uv[i] * (s + si * (1.0f - s));
          hv[i] = si * uv[i];
        }
        store4((float*)a.dgu + m * (2 * I) + n, dg);
        store4((float*)a.dgu + m * (2 * I) + I + n, du);
        store4((float*)a.h + m * I + n, hv);
      } else if constexpr (FORM == TF_DW) {
        float* o = (float*)(mat == 0 ? a.dgate : mat == 1 ? a.dup : a.ddown) + e * HI;
        store4(o + m * (mat == 2 ? H : I) + n, total[t][r]);
      } else {
        store4((float*)(FORM == TF_DOWN ? a.y : a.dx) + m * H + n, total[t][r]);
      }
    }
  }
}

// 4 waves a SIMD, so 128 registers at most: 1 to 5% faster than 3 waves with some more registers, although with tiles of
// 64 rows dx then spills 3 registers, the weight gradients 10 and the launch of both 13 (10 with 32 rows)
template <int FORM, int TM>
__global__ void __launch_bounds__(TTHR, 4) train_f32_kernel(const TrainArgs a) {
  __shared__ __align__(16) float lds[LDS_FLOATS];
  tile<FORM, TM>(a, blockIdx.x, blockIdx.y, blockIdx.z, lds);
}

// dx and the weight gradients, which both follow dh and do not need each other, in one launch: the tiles of dx
// first, each the longer chain of steps
template <int TM>
__global__ void __launch_bounds__(TTHR, 4) train_f32_gradients_kernel(const TrainArgs a, unsigned rows, unsigned dx_tiles) {
  __shared__ __align__(16) float lds[LDS_FLOATS];
  unsigned b = blockIdx.x;
  if (b < dx_tiles) {
    tile<TF_DX, TM>(a, b % rows, b / rows, 0, lds);
    return;
  }
  b -= dx_tiles;
  const unsigned per = (unsigned)(a.H / 64) * (unsigned)(a.I / TN);
  tile<TF_DW, 64>(a, b % per, b / per % a.E, b / per / a.E, lds);
}

// Rows of a tile: 64, or 32 where tiles of 64 would not give every CU one, or where groups have at most 32 rows on
// average, so that most of 64 would be empty. 512 rows by H 1024 by I 1024, down: 29.2 us in 128 tiles of 64, 21.0 in
// 256 of 32; 1024 rows: 31.2 and 32.9; 8192 rows, H 2048, I 4096, 8 groups: 1209 and 1311; 333 rows in 16 groups,
// H 4096, I 1024: 99 and 69.
int tile_rows(const TrainArgs& a, long long columns) {
  const long long tiles = (a.P / 64 + (a.E + 1) / 2) * columns;
  return tiles < CUS || a.P <= 32LL * a.E ? 32 : 64;
}

template <int FORM>
hipError_t launch(const TrainArgs& a, int tile_columns, int n, hipStream_t st) {
  const unsigned columns = (unsigned)(n / tile_columns), tm = tile_rows(a, columns);
  const dim3 grid((unsigned)max_row_tiles(a.P, a.E, tm), columns);
  if (grid.x == 0) return hipSuccess;
  if (tm == 32) train_f32_kernel<FORM, 32><<<grid, TTHR, 0, st>>>(a);
  else train_f32_kernel<FORM, 64><<<grid, TTHR, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_train_f32(TrainForm form, const TrainArgs& a, hipStream_t st) {
  const unsigned weight_tiles = (unsigned)(a.H / 64) * (unsigned)(a.I / TN);
  switch (form) {
    case TF_GATE_UP: return launch<TF_GATE_UP>(a, TN / 2, a.I, st);
    case TF_DOWN: return launch<TF_DOWN>(a, TN, a.H, st);
    case TF_DH: return launch<TF_DH>(a, TN, a.I, st);
    case TF_DX: return launch<TF_DX>(a, TN, a.H, st);
    case TF_DW:
      train_f32_kernel<TF_DW, 64><<<dim3(weight_tiles, (unsigned)a.E, 3), TTHR, 0, st>>>(a);
      return hipGetLastError();
  }
  return hipErrorInvalidValue;
}

// One launch fills the CUs that few tiles leave idle: 666 rows in 5 groups, H 1024, I 384, 45 us, and 23 + 29 in two
// (with dx's tiles of 32 rows, which are the same 45 here). Past 2^16 tiles there is nothing to fill, and the grid
// stays far from 2^32 threads.
hipError_t launch_gradients_f32(const TrainArgs& a, hipStream_t st) {
  const unsigned columns = (unsigned)(a.H / TN), tm = a.P <= 32LL * a.E ? 32 : 64;
  const long long rows = max_row_tiles(a.P, a.E, tm), weights = 3LL * a.E * (a.H / 64) * (a.I / TN), n = rows * columns + weights;
  if (n > 1 << 16) {
    const hipError_t e = launch_train_f32(TF_DX, a, st);
    return e == hipSuccess ? launch_train_f32(TF_DW, a, st) : e;
  }
  const unsigned dx_tiles = (unsigned)(rows * columns);
  if (tm == 32) train_f32_gradients_kernel<32><<<(unsigned)n, TTHR, 0, st>>>(a, (unsigned)rows, dx_tiles);
  else train_f32_gradients_kernel<64><<<(unsigned)n, TTHR, 0, st>>>(a, (unsigned)rows, dx_tiles);
  return hipGetLastError();
}

}  // namespace moe
