// Kernel launchers of the training entry points: the gated feed-forward block that keeps its
// pre-activations, its gradient, the combine's gradient and the AdamW step.
#pragma once
#include "common.h"

namespace moe {

// The products of the block. Rows are those of the grouped layout (expert e owns rows
// [off[e], off[e+1])); weights are row-major, gate and up [E][H][I], down [E][I][H].
enum TrainForm {
  TF_GATE_UP,  // g = x Wg, u = x Wu (x gathered by slot_token); writes g, u (when given) and h
  TF_DOWN,     // y = h Wd
  TF_DH,       // dh = dy Wd^T; writes dg and du side by side ([row][2 I]) and h
  TF_DX,       // dx = dg Wg^T + du Wu^T
  TF_DW        // dWg = x^T dg, dWu = x^T du, dWd = h^T dy, per expert; in bf16 x by row (slot_token NULL)
};

struct TrainArgs {
  const int32_t* off;         // [E+1], or NULL: one group of all P rows
  const int32_t* slot_token;  // [P], or NULL: row r of x belongs to row r
  int E, P, T, H, I;
  int xrows;                  // rows of x (T, or P without slot_token)
  const void *x, *gate, *up, *down;
  void *g, *u, *y;            // TF_GATE_UP / TF_DOWN outputs; g, u inputs of TF_DH
  const void* dy;
  void *dx, *dgate, *dup, *ddown;
  void *h, *dgu, *xg;         // workspace: [P][I], [P][2 I] and, for bf16, [P][H]
};

// Largest number of row tiles of bm rows that E groups of P rows in all can take.
inline long long max_row_tiles(int P, int E, int bm) {
  return E == 1 ? ((long long)P + bm - 1) / bm : P / bm + (long long)(E < P ? E : P);
}

hipError_t launch_train_f32(TrainForm form, const TrainArgs& a, hipStream_t st);
hipError_t launch_gradients_f32(const TrainArgs& a, hipStream_t st);  // TF_DX and TF_DW
hipError_t launch_gather_rows(const TrainArgs& a, hipStream_t st);     // xg = rows of x in the grouped order, bf16
hipError_t launch_train_bf16(TrainForm form, const TrainArgs& a, hipStream_t st);

hipError_t launch_combine_backward(int act, const void* dy, const void* y_perm, const int32_t* pair_slot, const float* w,
                                   void* dy_perm, float* dw, int T, int H, int k, hipStream_t st);

// One AdamW launch's tensors, passed by value (the kernel argument segment holds 4 KiB).
constexpr int ADAM_MAX = 40;
struct AdamTensor {
  void* p;
  const void* g;
  void *m, *v;
  float *ms, *vs;
  float* master;
  int64_t n;
};
struct AdamArgs {
  AdamTensor t[ADAM_MAX];
  int first[ADAM_MAX + 1];  // first workgroup of each tensor
  int count, passes;
  float lr, beta1, beta2, one_minus_beta1, one_minus_beta2, eps, wd;
  float bc1, inv_root_bc2;      // 1 - beta1^t and 1 / sqrt(1 - beta2^t), without step_dev
  float log_beta1, log_beta2;
  uint32_t seed;
  int64_t step;
  const float* lr_dev;          // each of the three may be NULL
  const int64_t* step_dev;
  const float* grad_scale;
};
hipError_t launch_adamw(int p_type, int g_type, bool master, bool q8, const AdamArgs& a, hipStream_t st);
int adamw_chunk(int64_t elements);  // elements of one workgroup, for so many in all
int adamw_passes(int chunk);

#ifdef __HIPCC__
// Place of row tile `tile` (bm rows each, groups one after the other): its group and rows. Every
// lane of a wave calls it with the same arguments and gets the same answer; false past the last
// tile. Offsets are clamped to [0, P] and a group that would end before it begins is empty, so
// no offset makes a row outside the arrays.
struct RowTile {
  int e, beg, end, row0;
};
__device__ __forceinline__ int clamp_row(int v, int P) { return v < 0 ? 0 : (v > P ? P : v); }

__device__ __forceinline__ void group_rows(const int32_t* off, int e, int P, int& beg, int& end) {
  beg = off ? clamp_row(off[e], P) : 0;
  end = off ? clamp_row(off[e + 1], P) : P;
  if (end < beg) end = beg;
}

__device__ __forceinline__ bool find_row_tile(const int32_t* off, int E, int P, int bm, int tile, RowTile& t) {
  if (!off) {
    t = RowTile{0, 0, P, tile * bm};
    return (long long)tile * bm < P;
  }
  const int lane = threadIdx.x & 63, per = (E + 63) >> 6;
  int mine = 0;
  for (int i = 0; i < per; ++i) {
    const int e = lane * per + i;
    if (e >= E) break;
    int b, n;
    group_rows(off, e, P, b, n);
    mine += (n - b + bm - 1) / bm;
  }
  int upto = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(upto, d);
    if (lane >= d) upto += o;
  }
  const unsigned long long past = __ballot(upto > tile);
  if (!past) return false;
  const int l = __builtin_ctzll(past);
  int before = __builtin_amdgcn_readlane(upto - mine, l);
  for (int e = l * per;; ++e) {
    int b, n;
    group_rows(off, e, P, b, n);
    const int tiles = (n - b + bm - 1) / bm;
    if (before + tiles > tile) {
      t = RowTile{e, b, n, b + (tile - before) * bm};
      return true;
    }
    before += tiles;
  }
}
#endif

}  // namespace moe
