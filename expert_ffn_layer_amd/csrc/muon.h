// Launchers of the orthogonalisation by Newton-Schulz products and of the Muon step (formulas in include/moe.h).
//
// Matrices of one size class (short side M, long side N) are worked on together, a chunk of them at a time. In the
// workspace matrix b of a chunk is X, [Mp][Np] with the short side first, whichever way the user's matrix lies, zeros
// beyond its size; Gram's matrix A = X X^T and the polynomial C are [Mp][Mp]. Mp and Np are multiples of 128.
//
// X, A and C are held in fp16 times SCALE. All stay in its range: X's singular values are at most the bound that the
// entry points check, and no element of a matrix exceeds its largest singular value.
#pragma once
#include "common.h"

namespace moe {

constexpr int MUON_STACKS = 40;      // stacks of one launch
constexpr float MUON_SCALE = 4096.f;
constexpr int MUON_PAD = 128;

struct MuonStack {
  const void* g;
  float* m;       // NULL: u = g
  void* out;      // parameters, or the orthogonalised matrices where m is NULL
  float* master;
  float scale;    // the update is lr scale O
  int first;      // index in the class of its first matrix
  int wide;       // rows < cols, or X is the transpose; stacks with it come first
};

struct MuonArgs {
  MuonStack s[MUON_STACKS];
  int stacks;
  int first, count;        // matrices of the chunk, as indices of the class
  int skip;                // of the chunk, those that come before the launch's
  int turned;              // MF_LAST: the launch's matrices have their long side first
  int whole_c;             // MF_POLY: C's diagonal stands in C, too
  int M, N, Mp, Np;
  int g_f32, out_f32;
  int split;               // products of fp16 pairs: fp32 results
  int nesterov;
  float momentum, lr, wd;
  const float *lr_dev, *grad_scale;
  double eps;
  double a, b, c;          // the polynomial of a step
  // workspace
  int parts;               // partial sums of squares of a matrix
  int part;                // thin matrices: columns of a part
  double* sums;            // [count][parts]
  uint16_t *x, *x_lo;      // in
  uint16_t *xo, *xo_lo;    // out; xo_lo may be x_lo without split, or NULL
  uint16_t *A, *A_lo, *C, *C_lo;
  double* q;               // thin matrices
  double* xs;              // thin matrices: [count][M][N], X between two runs of steps, or NULL
  int runs;                // workgroups that share Gram's matrix by parts of the reduction; 0: a tile is one workgroup's
  float* partial;          // [2 runs][128 * 128]
  float *da, *dc;          // [count][Mp]: the diagonals of A and of a I + C, which are zero in A, and in C but for whole_c and split
};

int muon_parts(long long elements);
hipError_t launch_muon_momentum(const MuonArgs& a, hipStream_t st);   // m, and the sums of u's squares
hipError_t launch_muon_normalize(const MuonArgs& a, hipStream_t st);  // x, x_lo = SCALE u / (|u| + eps)
enum MuonForm {
  MF_GRAM,  // A = X X^T
  MF_POLY,  // C = b A + c A^2, and its diagonal with a
  MF_STEP,  // X' = a X + C X
  MF_LAST   // the same into the user's matrices
};
// How many runs Gram's matrices of a chunk of `count` take, or 0
int muon_runs(int Mp, int Np, long long count, bool split);
hipError_t launch_muon_product(MuonForm form, const MuonArgs& a, hipStream_t st);

// All of it for matrices with a short side of at most THIN_MAX that muon_thin() names; a.part = thin_part(N) and a.parts of them, a.sums
// [count][parts][MB][MB], a.q [count][MB * MB + 1], MB the short side's 32 or 64
constexpr int THIN_MAX = 64;
inline int thin_side(int M) { return M <= 32 ? 32 : 64; }
int thin_part(int N);
bool muon_thin(int M, int N);
// the steps in `runs` runs, Gram's matrix formed anew for each
hipError_t launch_muon_thin(const MuonArgs& a, int steps, int runs, hipStream_t st);

// All of it for other small matrices, without a workspace
bool muon_small(int M, int N);
hipError_t launch_muon_small(const MuonArgs& a, int steps, hipStream_t st);

#ifdef __HIPCC__
// The stack of matrix `index` of the class
__device__ __forceinline__ const MuonStack& muon_stack(const MuonArgs& a, int index) {
  int s = a.stacks - 1;
  while (s > 0 && a.s[s].first > index) --s;
  return a.s[s];
}
#endif

}  // namespace moe
