// The products of the Newton-Schulz steps (v_mfma_f32_32x32x16_f16); forms as listed in muon.h.
//
// out[m][n] = sum_k P(m, k) Q(n, k), a tile per workgroup of 4 waves; both operands pass through a ring of D slots of 64
// reduction elements in LDS (tile_ring.h). X is held with its long side contiguous, so that the product with C, most of
// the work, reads both operands with their own index contiguous (C is symmetric), and Gram's matrix both with the
// reduction index. A and C are symmetric: their tiles on and under the diagonal are computed and written to both places.
//
// What bounds it, large: the matrix cores at the power limit, 1400 TFLOP/s (1.5 us for 64 reduction elements of a 256 x 256 tile on
// every CU; on zeros 1.15), and between them the results: of 68 us of a tile with a reduction of 2048, 2.3 fill the ring and 16
// to 20 read X, form and write the next, 512 KiB a workgroup from all CUs at once. 32 matrices of 2048 x 7168: A 0.99 ms, C 0.35,
// a step's X 1.97, the last with parameters and copies 2.19. Small: a launch's latency, 12 to 15 us for a reduction of 1000.
//
// Numerics: sums are fp32. X is a pair of fp16, x + x_lo, 22 bits; the products read x alone (11 bits) unless
// SPLIT asks for fp32 results: then x y_lo and x_lo y are added to x y, as two more runs over the reduction. The diagonals
// of A and C are kept apart in fp32: where singular values are near each other the diagonal holds most of A and C, and its
// rounding would be most of the error. C's diagonal, which holds a too, multiplies the whole of X: what rounding adds to
// directions that X lacks would grow by a = 3.4 in every step. The last step has none after it: it takes x alone, and C's
// diagonal as the fp16 that stands in C, so that it has X to read in the product only (with SPLIT every step does: the pairs
// hold all of both). That adds to what five steps are off, before the result is rounded to bf16 (1.7e-3): 512 x 256 of full rank
// 6.7e-4 for 6.2e-4, of rank 16 1.7e-3 for 1.4e-3.
#include <algorithm>
#include <type_traits>

#include "muon.h"
#include "tile_ring.h"

namespace moe {

namespace {

typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;
typedef __attribute__((ext_vector_type(2))) _Float16 f16x2;
typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
typedef __attribute__((address_space(3))) u32x2 lds_u32x2;
typedef __attribute__((address_space(3))) uint16_t lds_u16;

struct Eight {
  float v[8];
};
__device__ __forceinline__ Eight halves(const u32x4& w) {
  Eight r;
  const f16x8 h = __builtin_bit_cast(f16x8, w);
#pragma unroll
  for (int z = 0; z < 8; ++z) r.v[z] = (float)h[z];
  return r;
}
__device__ __forceinline__ u32x4 to_halves(const Eight& r) {
  f16x8 h;
#pragma unroll
  for (int z = 0; z < 8; ++z) h[z] = (_Float16)r.v[z];
  return __builtin_bit_cast(u32x4, h);
}
// what rounding to `hi` leaves
__device__ __forceinline__ u32x4 to_rest(const Eight& r, const u32x4& hi) {
  const Eight h = halves(hi);
  Eight d;
#pragma unroll
  for (int z = 0; z < 8; ++z) d.v[z] = r.v[z] - h.v[z];
  return to_halves(d);
}

// Where a product goes that is not whole in the workspace: sums over a part of the reduction; O in the matrices' type; parameters of that type; bf16 parameters with fp32 copies
enum Out { OUT_NONE, OUT_PART, OUT_O, OUT_P, OUT_MASTER };

// 8 consecutive fp32 (8 words) or bf16 (4 words) of a row
template <bool F32>
struct Row8 {
  u32x4 w[F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ Row8<F32> load8(const void* p, size_t at) {
  Row8<F32> r;
  if constexpr (F32) {
    r.w[0] = *(const u32x4*)((const float*)p + at);
    r.w[1] = *(const u32x4*)((const float*)p + at + 4);
  } else {
    r.w[0] = *(const u32x4*)((const uint16_t*)p + at);
  }
  return r;
}
template <bool F32>
__device__ __forceinline__ Eight values(const Row8<F32>& r) {
  Eight v;
#pragma unroll
  for (int z = 0; z < 8; ++z) {
    if constexpr (F32) v.v[z] = __uint_as_float(r.w[z >> 2][z & 3]);
    else v.v[z] = z & 1 ? bf16hi(r.w[0][z >> 1]) : bf16lo(r.w[0][z >> 1]);
  }
  return v;
}
__device__ __forceinline__ void store_f32(float* p, size_t at, const Eight& v) {
  *(f32x4*)(p + at) = f32x4{v.v[0], v.v[1], v.v[2], v.v[3]};
  *(f32x4*)(p + at + 4) = f32x4{v.v[4], v.v[5], v.v[6], v.v[7]};
}
__device__ __forceinline__ void store_bf16(uint16_t* p, size_t at, const Eight& v) {
  *(u32x4*)(p + at) = u32x4{pack_bf16x2(v.v[0], v.v[1]), pack_bf16x2(v.v[2], v.v[3]), pack_bf16x2(v.v[4], v.v[5]), pack_bf16x2(v.v[6], v.v[7])};
}

// The tile (tm, tn) of matrix b, over `once` steps of 64 reduction elements, an even number, from step `from`. OUT_PART: the
// sums to `part`, a 4 KiB block for each 32 x 32, which has lane l's elements 4 q + j at (64 q + l) 4 + j.
template <int FORM, int WR, int WC, int MT, int NT, int D, bool SPLIT, int OUT>
__device__ __forceinline__ void product_tile(const MuonArgs& a, const int b, const int tm, const int tn, const int from, const int once, float* part) {
  constexpr bool SYM = FORM == MF_GRAM || FORM == MF_POLY, KC = FORM == MF_GRAM;
  constexpr int BM = WR * MT * 32, BN = WC * NT * 32;
  static_assert(BM == BN, "square tiles");
  constexpr bool HV = !KC && D == 2;  // slots freed and filled by halves of 32 reduction elements
  using T = Tile<BM, KC, HV>;
  constexpr int U = T::U, L = 2 * U;  // loads per wave and stage: of an operand, of both
  using S = Share<HV, U>;
  constexpr int PART = HV ? T::BYTES / 2 : T::BYTES;
  // One array for each part that is freed and filled whole: the compiler then sees which loads to LDS a read waits for
  constexpr int MORE = HV || D == 4 ? PART : 16;
  __shared__ __align__(1024) uint8_t p0[PART], p1[PART], p2[MORE], p3[MORE], q0[PART], q1[PART], q2[MORE], q3[MORE];
#define P_PART(SLOT, B) ((lds_byte*)((SLOT) + (HV && (B) ? 2 : 0) == 0 ? p0 : (SLOT) + (HV && (B) ? 2 : 0) == 1 ? p1 : (SLOT) + (HV && (B) ? 2 : 0) == 2 ? p2 : p3))
#define Q_PART(SLOT, B) ((lds_byte*)((SLOT) + (HV && (B) ? 2 : 0) == 0 ? q0 : (SLOT) + (HV && (B) ? 2 : 0) == 1 ? q1 : (SLOT) + (HV && (B) ? 2 : 0) == 2 ? q2 : q3))
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave / WC, wc = wave % WC;
  // the user's matrices have their long side first: the last product's tiles lie as they do, with X as P
  const bool turned = FORM == MF_LAST && a.turned;

  const int m0 = tm * BM, n0 = tn * BM;
  const int mend = turned ? a.Np : a.Mp, nend = SYM || turned ? a.Mp : a.Np;
  const size_t xat = (size_t)b * a.Mp * a.Np, aat = (size_t)b * a.Mp * a.Mp;
  const int nsteps = SPLIT ? 3 * once : once;

  // --- loads: this wave's units of both operands; the lower halves of pairs lie `p_lo`, `q_lo` bytes behind the upper
  const uint8_t *psrc[U], *qsrc[U];
  const uint16_t *p, *q;
  int pld, qld;
  ptrdiff_t p_lo = 0, q_lo = 0;
  if constexpr (FORM == MF_GRAM) {
    p = q = a.x + xat + from * BK;
    pld = qld = a.Np;
    if (SPLIT) p_lo = q_lo = (const uint8_t*)a.x_lo - (const uint8_t*)a.x;
  } else if constexpr (FORM == MF_POLY) {
    p = q = a.A + aat;
    pld = qld = a.Mp;
    if (SPLIT) p_lo = q_lo = (const uint8_t*)a.A_lo - (const uint8_t*)a.A;
  } else {
    p = turned ? a.x + xat : a.C + aat;
    q = turned ? a.C + aat : a.x + xat;
    pld = turned ? a.Np : a.Mp;
    qld = turned ? a.Mp : a.Np;
    if (SPLIT) {
      const ptrdiff_t x_lo = (const uint8_t*)a.x_lo - (const uint8_t*)a.x, c_lo = (const uint8_t*)a.C_lo - (const uint8_t*)a.C;
      p_lo = turned ? x_lo : c_lo;
      q_lo = turned ? c_lo : x_lo;
    }
  }
  const ptrdiff_t pstride = KC ? BK * 2 : (ptrdiff_t)BK * 2 * pld, qstride = KC ? BK * 2 : (ptrdiff_t)BK * 2 * qld;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int un = T::unit(u, wave), r = T::row(un, lane), c = T::elem(un, lane);
    // sizes are multiples of 128: past the end, indices that exist are repeated, and not stored
    if constexpr (KC) {
      const int m = m0 + r, n = n0 + r;
      psrc[u] = (const uint8_t*)(p + (size_t)(m < mend ? m : m - 128) * pld + c);
      qsrc[u] = (const uint8_t*)(q + (size_t)(n < nend ? n : n - 128) * qld + c);
    } else {
      const int m = m0 + c, n = n0 + c;
      psrc[u] = (const uint8_t*)(p + (size_t)r * pld + (m < mend ? m : m - 128));
      qsrc[u] = (const uint8_t*)(q + (size_t)r * qld + (n < nend ? n : n - 128));
    }
  }
  // One load of stage `step`; the source moves on, from one run over the reduction to the next, and stays on the last step
  auto load_one = [&](const uint8_t*& src, lds_byte* dst, int step, ptrdiff_t stride, ptrdiff_t second, ptrdiff_t third) __attribute__((always_inline)) {
    __builtin_amdgcn_global_load_lds((const void*)src, (lds_void*)dst, 16, 0, 0);
    ptrdiff_t adv = step + 1 < nsteps ? stride : 0;
    if constexpr (SPLIT) {
      if (step + 1 == once) adv = second - (once - 1) * stride;
      if (step + 1 == 2 * once) adv = third - (once - 1) * stride;
    }
    src += adv;
    asm volatile("" : "+v"(src));  // one running pointer a load, not one per load and slot
  };
  // P runs x, x, x_lo; Q runs x, x_lo, x
  auto load_p = [&](int u, int step, auto slot) __attribute__((always_inline)) {
    const int un = T::unit(u, wave);
    load_one(psrc[u], P_PART(decltype(slot)::value, u >= U / 2) + (HV ? un % (T::UNITS / 2) : un) * 1024, step, pstride, 0, p_lo);
  };
  auto load_q = [&](int u, int step, auto slot) __attribute__((always_inline)) {
    const int un = T::unit(u, wave);
    load_one(qsrc[u], Q_PART(decltype(slot)::value, u >= U / 2) + (HV ? un % (T::UNITS / 2) : un) * 1024, step, qstride, q_lo, -q_lo);
  };

  // --- for the results
  const float inv = 1.f / MUON_SCALE, pa = (float)a.a, pb = (float)a.b, pc = (float)a.c;
  const int wrow = m0 + wr * MT * 32, wcol = n0 + wc * NT * 32, r32 = lane & 31, hi4 = lane >> 5, c8 = lane & 7, r8 = lane >> 3;
  constexpr int BLOCKS = NT / 2, ALL = MT * BLOCKS;
  const float* const diagonal = FORM == MF_GRAM ? nullptr : (FORM == MF_POLY ? a.da : a.dc) + (size_t)b * a.Mp;
  // What a block's results are formed with, the elements themselves of A or X and the diagonal, or the user's parameters, is
  // fetched AHEAD - 1 blocks before: a block takes about 1 us, a load from memory 2 to 3 while all CUs write. With tiles of
  // 128 x 128 all of it comes before the reduction.
  constexpr bool OLD_HI = FORM == MF_POLY || (FORM == MF_STEP && !SPLIT), OLD_LO = (FORM == MF_POLY && SPLIT) || (FORM == MF_STEP && !SPLIT);
  constexpr bool OLD_P = OUT == OUT_P || OUT == OUT_MASTER, P_F32 = SPLIT || OUT == OUT_MASTER;
  constexpr int AHEAD = ALL < 3 ? ALL : 3;
  const uint16_t* const old_hi = FORM == MF_POLY ? a.A + aat : a.x + xat;
  const uint16_t* const old_lo = FORM == MF_POLY ? a.A_lo + aat : a.x_lo + xat;
  const int ld = FORM == MF_POLY ? a.Mp : a.Np;
  const MuonStack* const user = FORM == MF_LAST ? &muon_stack(a, a.first + b) : nullptr;
  const int rows = turned ? a.N : a.M, cols = turned ? a.M : a.N;  // of the user's matrix
  const size_t uat = FORM == MF_LAST ? (size_t)(a.first + b - user->first) * a.M * a.N : 0;
  const bool whole = cols % 8 == 0;  // rows and matrices begin on 16 bytes, and no 8 columns pass their end
  void* const params = FORM == MF_LAST ? (OUT == OUT_MASTER ? (void*)user->master : user->out) : nullptr;
  float keep = 0.f, step = 0.f;
  if constexpr (OLD_P) {
    const float lr = a.lr_dev ? *a.lr_dev : a.lr;
    keep = 1.f - lr * a.wd;
    step = lr * user->scale;
  }
  float dm[AHEAD][OLD_HI ? 4 : 1];
  f32x4 dn[AHEAD][FORM == MF_POLY ? 2 : 1];  // at this lane's columns
  u32x4 hw[AHEAD][OLD_HI ? 4 : 1], lw[AHEAD][OLD_LO ? 4 : 1];
  Row8<P_F32> pw[AHEAD][OLD_P ? 4 : 1];
  auto fetch = [&](int blk) __attribute__((always_inline)) {
    const int n = wcol + blk % BLOCKS * 64 + c8 * 8, set = blk % AHEAD;
    if constexpr (FORM == MF_POLY) {
#pragma unroll
      for (int z = 0; z < 2; ++z) dn[set][z] = *(const f32x4*)(diagonal + (n < nend ? n : 0) + 4 * z);
    }
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int m = wrow + blk / BLOCKS * 32 + it * 8 + r8;
      // past the end an element that exists, which is not used
      const size_t at = m < mend && n < nend ? (size_t)m * ld + n : 0;
      if constexpr (OLD_HI) dm[set][it] = diagonal[m < mend ? m : 0];
      if constexpr (OLD_HI) hw[set][it] = *(const u32x4*)(old_hi + at);
      if constexpr (OLD_LO) lw[set][it] = *(const u32x4*)(old_lo + at);
      if constexpr (OLD_P)
        if (whole) pw[set][it] = load8<P_F32>(params, uat + (m < rows && n < cols ? (size_t)m * cols + n : 0));
    }
  };
  constexpr bool EARLY = ALL <= AHEAD;
  if constexpr (EARLY) {
#pragma unroll
    for (int blk = 0; blk < ALL; ++blk) fetch(blk);
  }

  f32x16 acc[NT][MT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) acc[t][i][j] = 0.f;

  {
    int pb[KC ? 4 : MT], qb[KC ? 4 : NT];
#pragma unroll
    for (int i = 0; i < (KC ? 4 : MT); ++i) pb[i] = KC ? T::kc_at(wr * MT, i, lane) : T::mc_at(wr * MT + i, lane);
#pragma unroll
    for (int t = 0; t < (KC ? 4 : NT); ++t) qb[t] = KC ? T::kc_at(wc * NT, t, lane) : T::mc_at(wc * NT + t, lane);
    bf16x8 pf[2][MT], qf[2][NT];  // two quarters: the one multiplied and the one read
    auto read_p = [&](int i, auto quarter, auto slot) __attribute__((always_inline)) {
      constexpr int h = decltype(quarter)::value;
      lds_byte* const part = P_PART(decltype(slot)::value, h >= 2);
      pf[h & 1][i] = read_frag<BM, KC>(part + (KC ? pb[h] + i * 4096 : pb[i] + (HV ? h & 1 : h) * 16 * (BM * 2)));
    };
    auto read_q = [&](int t, auto quarter, auto slot) __attribute__((always_inline)) {
      constexpr int h = decltype(quarter)::value;
      lds_byte* const part = Q_PART(decltype(slot)::value, h >= 2);
      qf[h & 1][t] = read_frag<BN, KC>(part + (KC ? qb[h] + t * 4096 : qb[t] + (HV ? h & 1 : h) * 16 * (BN * 2)));
    };
    constexpr std::integral_constant<int, 0> C0{};
    constexpr std::integral_constant<int, 1> C1{};
    constexpr std::integral_constant<int, 2> C2{};
    constexpr std::integral_constant<int, 3> C3{};
    // the n-th load of phase ph of step s; slot: that of step s
    auto load_nth = [&](auto ph_c, int n, int s, auto slot) __attribute__((always_inline)) {
      constexpr int ph = decltype(ph_c)::value, each = S::count(ph);
      constexpr std::integral_constant<int, (decltype(slot)::value + D - 1) % D> before{};
      const bool is_p = HV ? n < each : n >= each;
      const int u = S::from(ph) + (is_p != HV ? n - each : n);
      // phase 0, and phase 1 for whole slots, still bring stage s + D - 1, into the slot of step s - 1
      if constexpr (ph == 0 || (!HV && ph == 1)) {
        if (is_p) load_p(u, s + D - 1, before);
        else load_q(u, s + D - 1, before);
      } else {
        if (is_p) load_p(u, s + D, slot);
        else load_q(u, s + D, slot);
      }
    };
    // Products of quarter h, with the reads of the next quarter early behind them and the phase's loads spread over all
    auto phase = [&](auto quarter, auto rd_slot, int s, auto slot) __attribute__((always_inline)) {
      constexpr int h = decltype(quarter)::value, LOADS = 2 * S::count(h);
      constexpr std::integral_constant<int, (h + 1) % 4> next{};
      constexpr int PRODUCTS = MT * NT, READS = MT + NT, SPAN = PRODUCTS > 4 ? PRODUCTS * 3 / 4 : PRODUCTS;
#pragma unroll
      for (int n = 0; n < PRODUCTS; ++n) {
        const int t = n % NT, i = n / NT;
        acc[t][i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, qf[h & 1][t]), __builtin_bit_cast(f16x8, pf[h & 1][i]),
                                                           acc[t][i], 0, 0, 0);
#pragma unroll
        for (int r = n * READS / SPAN; r < (n + 1) * READS / SPAN && r < READS; ++r) {
          if (r < NT) read_q(r, next, rd_slot);
          else read_p(r - NT, next, rd_slot);
        }
#pragma unroll
        for (int z = n * LOADS / PRODUCTS; z < (n + 1) * LOADS / PRODUCTS; ++z) load_nth(quarter, z, s, slot);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    // Loads that may still be in flight: where the second half of a slot is wanted (after phase 0), those of one step;
    // where the next stage is wanted (after phase 2), the same, and those of D - 2 steps with whole slots
    constexpr int FLY0 = L, FLY2 = HV ? L : (D - 2) * L;
    auto body = [&](int s, auto slot) __attribute__((always_inline)) {
      constexpr std::integral_constant<int, (decltype(slot)::value + 1) % D> other{};
      // opaque in every step, so that the slot stays a constant and does not become a register per slot and fragment
#pragma unroll
      for (int i = 0; i < MT && !KC; ++i) asm volatile("" : "+v"(pb[i]));
#pragma unroll
      for (int t = 0; t < NT && !KC; ++t) asm volatile("" : "+v"(qb[t]));
      phase(C0, slot, s, slot);
      if constexpr (HV) {
        MOE_WAIT_LGKM0();
        MOE_WAIT_VMCNT(FLY0);
        __builtin_amdgcn_s_barrier();
      }
      phase(C1, slot, s, slot);
      phase(C2, slot, s, slot);
      MOE_WAIT_LGKM0();
      MOE_WAIT_VMCNT(FLY2);
      __builtin_amdgcn_s_barrier();
      phase(C3, other, s, slot);
    };
    // what the steps before the first would have loaded, stage 0 first
    auto stage = [&](int step, auto slot) __attribute__((always_inline)) {
#pragma unroll
      for (int u = 0; u < U; ++u) load_q(u, step, slot);
#pragma unroll
      for (int u = 0; u < U; ++u) load_p(u, step, slot);
    };
    stage(0, C0);
    if constexpr (D == 4) {
      stage(1, C1);
      stage(2, C2);
    }
    constexpr int FIRST = HV ? U / 2 : 0;  // of stage 1, before phase 3 of step -1
#pragma unroll
    for (int u = 0; u < FIRST; ++u) load_q(u, 1, C1);
#pragma unroll
    for (int u = 0; u < FIRST; ++u) load_p(u, 1, C1);
    constexpr std::integral_constant<int, D - 1> last{};
#pragma unroll
    for (int n = 0; n < 2 * S::count(3); ++n) load_nth(C3, n, -1, last);
    MOE_WAIT_VMCNT((D - 2) * L + 2 * FIRST + 2 * S::count(3));
    __builtin_amdgcn_s_barrier();
#pragma unroll
    for (int t = 0; t < NT; ++t) read_q(t, C0, C0);
#pragma unroll
    for (int i = 0; i < MT; ++i) read_p(i, C0, C0);
    int s = 0;
    if constexpr (D == 4) {
      for (; s + 2 < nsteps; s += 4) {
        body(s, C0);
        body(s + 1, C1);
        body(s + 2, C2);
        body(s + 3, C3);
      }
    }
    for (; s < nsteps; s += 2) {  // sizes are multiples of 128: pairs of steps
      body(s, C0);
      body(s + 1, C1);
    }
    MOE_WAIT_VMCNT(0);  // loads in flight land before the workgroup's LDS is used for other things
  }

  // --- results. Element 4 q + j of a tile is column 8 q + 4 (lane / 32) + j of row lane % 32. Each wave passes blocks of
  // 32 rows x 64 columns through 8 KiB of LDS of its own, so that a lane goes on with 8 consecutive columns of a row;
  // 16-byte chunk c of a row sits at c ^ (row % 16), which keeps both directions free of bank conflicts. Mirrored blocks pass
  // through another 4.5 KiB as 64 rows of 32, 72 bytes apart. The parts of the ring serve for both.
  __builtin_amdgcn_s_barrier();
  if constexpr (OUT == OUT_PART) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *(f32x4*)(part + ((wr * MT + i) * (WC * NT) + wc * NT + t) * 1024 + (64 * j + lane) * 4) =
              f32x4{acc[t][i][4 * j], acc[t][i][4 * j + 1], acc[t][i][4 * j + 2], acc[t][i][4 * j + 3]};
    return;
  }
  constexpr bool FOUR = HV || D == 4;  // parts of an operand
  static_assert((FOUR ? PART : PART / 2) >= 8192, "a part of the ring per wave");
  lds_byte* const ep = !FOUR ? (lds_byte*)(wave & 2 ? q1 : q0) + (wave & 1) * (PART / 2) : (lds_byte*)(wave == 0 ? q0 : wave == 1 ? q1 : wave == 2 ? q2 : q3);
  lds_byte* const mirror = !FOUR ? (lds_byte*)(wave & 2 ? p1 : p0) + (wave & 1) * (PART / 2) : (lds_byte*)(wave == 0 ? p0 : wave == 1 ? p1 : wave == 2 ? p2 : p3);
  // The lanes of a wave exchange data through LDS: its accesses run in the order in which they are issued, and this keeps
  // the compiler from changing that order.
  auto in_order = [] { __asm__ volatile("" ::: "memory"); };
  if constexpr (!EARLY) {
#pragma unroll
    for (int blk = 0; blk < AHEAD - 1; ++blk) fetch(blk);
  }
#pragma unroll
  for (int blk = 0; blk < ALL; ++blk) {
    if (!EARLY && blk + AHEAD - 1 < ALL) fetch(blk + AHEAD - 1);
    const int i = blk / BLOCKS, n = wcol + blk % BLOCKS * 64 + c8 * 8, set = blk % AHEAD;
    in_order();
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const f32x16& v = acc[2 * (blk % BLOCKS) + z][i];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *(lds_f32x4*)(ep + r32 * 256 + (((z * 8 + 2 * j + hi4) ^ (r32 & 15)) << 4)) = f32x4{v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]};
    }
    in_order();
    u32x4 low[4];
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int row = it * 8 + r8, m = wrow + i * 32 + row;
      const f32x4 v0 = *(const lds_f32x4*)(ep + row * 256 + (((2 * c8) ^ (row & 15)) << 4));
      const f32x4 v1 = *(const lds_f32x4*)(ep + row * 256 + (((2 * c8 + 1) ^ (row & 15)) << 4));
      const bool inside = m < mend && n < nend;
      Eight r;
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        r.v[z] = v0[z] * inv;
        r.v[4 + z] = v1[z] * inv;
      }
      Eight x{};
      if constexpr (OLD_HI) x = halves(hw[set][it]);
      if constexpr (OLD_LO) {
        const Eight lo = halves(lw[set][it]);
#pragma unroll
        for (int z = 0; z < 8; ++z) x.v[z] += lo.v[z];
      }
      if constexpr (SYM) {
        Eight q = r;
        if constexpr (FORM == MF_POLY) {
#pragma unroll
          for (int z = 0; z < 8; ++z) q.v[z] = pb * x.v[z] + pc * ((dm[set][it] + dn[set][z >> 2][z & 3]) * x.v[z] + r.v[z]);
        }
        if (tm == tn) {
#pragma unroll
          for (int z = 0; z < 8; ++z)
            if (m == n + z) {
              float d = r.v[z] * inv;
              if constexpr (FORM == MF_POLY) d = pa + pb * dm[set][it] + pc * (dm[set][it] * dm[set][it] + d);
              if (inside) (FORM == MF_GRAM ? a.da : a.dc)[(size_t)b * a.Mp + m] = d;
              // C keeps its diagonal where the product that reads it adds nothing to it
              q.v[z] = FORM == MF_POLY && (SPLIT || a.whole_c) ? d * MUON_SCALE : 0.f;
            }
        }
        uint16_t* const out = (FORM == MF_GRAM ? a.A : a.C) + aat;
        uint16_t* const out_lo = (FORM == MF_GRAM ? a.A_lo : a.C_lo) + aat;
        const u32x4 hi = to_halves(q);
        if constexpr (SPLIT) low[it] = to_rest(q, hi);
        if (inside) {
          *(u32x4*)(out + (size_t)m * a.Mp + n) = hi;
          if (SPLIT) *(u32x4*)(out_lo + (size_t)m * a.Mp + n) = low[it];
        }
        if (tm != tn) {
#pragma unroll
          for (int z = 0; z < 8; ++z) *(lds_u16*)(mirror + (c8 * 8 + z) * 72 + row * 2) = (uint16_t)(hi[z >> 1] >> (16 * (z & 1)));
        }
      } else if constexpr (FORM == MF_STEP) {
        if constexpr (!SPLIT) {
#pragma unroll
          for (int z = 0; z < 8; ++z) r.v[z] += dm[set][it] * x.v[z];
        }
        const u32x4 hi = to_halves(r);
        if (inside) *(u32x4*)(a.xo + xat + (size_t)m * a.Np + n) = hi;
        if (a.xo_lo) {
          const u32x4 lo = to_rest(r, hi);
          if (inside) *(u32x4*)(a.xo_lo + xat + (size_t)m * a.Np + n) = lo;
        }
      } else {
#pragma unroll
        for (int z = 0; z < 8; ++z) r.v[z] *= inv;
        const size_t at = uat + (size_t)m * cols + n;
        if (whole) {
          if constexpr (OLD_P) {
            const Eight old = values<P_F32>(pw[set][it]);
#pragma unroll
            for (int z = 0; z < 8; ++z) r.v[z] = old.v[z] * keep - step * r.v[z];
          }
          if (m < rows && n < cols) {
            if constexpr (P_F32) store_f32((float*)params, at, r);
            if constexpr (!SPLIT) store_bf16((uint16_t*)user->out, at, r);
          }
        } else if (m < rows) {
#pragma unroll
          for (int z = 0; z < 8; ++z) {
            if (n + z >= cols) break;
            float w = r.v[z];
            if constexpr (OLD_P) w = (P_F32 ? ((const float*)params)[at + z] : bf16_to_f32(((const uint16_t*)params)[at + z])) * keep - step * w;
            if constexpr (P_F32) ((float*)params)[at + z] = w;
            if constexpr (!SPLIT) ((uint16_t*)user->out)[at + z] = __builtin_bit_cast(uint16_t, (__bf16)w);
          }
        }
      }
    }
    if constexpr (SYM) {
      auto across = [&](uint16_t* out) __attribute__((always_inline)) {
        in_order();
#pragma unroll
        for (int it = 0; it < 8; ++it) {
          const int row = it * 8 + r8, mm = wcol + blk % BLOCKS * 64 + row, nn = wrow + i * 32 + c8 * 4;
          const u32x2 v = *(const lds_u32x2*)(mirror + row * 72 + c8 * 8);
          if (mm < nend && nn < mend) *(u32x2*)(out + (size_t)mm * a.Mp + nn) = v;
        }
        in_order();
      };
      if (tm != tn) {
        across((FORM == MF_GRAM ? a.A : a.C) + aat);
        if constexpr (SPLIT) {
#pragma unroll
          for (int it = 0; it < 4; ++it)
#pragma unroll
            for (int z = 0; z < 8; ++z)
              *(lds_u16*)(mirror + (c8 * 8 + z) * 72 + (it * 8 + r8) * 2) = (uint16_t)(low[it][z >> 1] >> (16 * (z & 1)));
          across((FORM == MF_GRAM ? a.A_lo : a.C_lo) + aat);
        }
      }
    }
  }
}

// Row and column of a symmetric product's tile `rest`
__device__ __forceinline__ void lower_tile(int rest, int& tm, int& tn) {
  tm = 0;
  while (rest > tm) rest -= ++tm;
  tn = rest;
}

// Workgroup b runs on XCD b % 8: each XCD gets an equal run of the chunk's tiles, matrix by matrix, so that what it runs at a
// time shares operands in its L2.
template <int FORM, int WR, int WC, int MT, int NT, int D, bool SPLIT, int OUT>
__global__ void __launch_bounds__(THR, MT * NT > 8 ? 1 : 2) product_kernel(const MuonArgs a) {
  constexpr bool SYM = FORM == MF_GRAM || FORM == MF_POLY;
  constexpr int BM = WR * MT * 32;
  const int short_tiles = (a.Mp + BM - 1) / BM, long_tiles = (a.Np + BM - 1) / BM;
  const int tiles = SYM ? short_tiles * (short_tiles + 1) / 2 : short_tiles * long_tiles;
  const long long all = (long long)a.count * tiles, run = (all + NXCD - 1) / NXCD;
  const long long id = (blockIdx.x % NXCD) * run + blockIdx.x / NXCD;
  if (blockIdx.x / NXCD >= run || id >= all) return;
  int tm, tn, rest = (int)(id % tiles);
  if constexpr (SYM) {
    lower_tile(rest, tm, tn);
  } else {
    // 4 tiles of the long side x all of the short one after each other
    const int g = rest / (4 * short_tiles), wide = min(4, long_tiles - 4 * g);
    rest -= g * 4 * short_tiles;
    tn = 4 * g + rest % wide;
    tm = rest / wide;
    // the user's matrices have their long side first: the last product's tiles lie as they do, with X as P
    if (FORM == MF_LAST && a.turned) {
      const int t = tm;
      tm = tn;
      tn = t;
    }
  }
  product_tile<FORM, WR, WC, MT, NT, D, SPLIT, OUT>(a, a.skip + (int)(id / tiles), tm, tn, 0, (FORM == MF_GRAM ? a.Np : a.Mp) / BK, nullptr);
}

// Gram's matrix of few tiles of 128 x 128 with a long reduction: the pairs of steps of all tiles, one tile's after the other's,
// go in equal runs to a.runs workgroups, at least as many as tiles, so that a run touches two tiles at most. The sums over
// its part of each go to the workspace and are added up by joined_kernel, in order.
struct Runs {
  int each, work, runs;  // pairs of steps of a tile, of all
  __device__ int start(int g) const { return (int)((unsigned)g * (unsigned)work / (unsigned)runs); }  // at most 256 * 128 * 8192
};
__device__ __forceinline__ Runs runs_of(const MuonArgs& a, int tiles) { return Runs{a.Np / 128, a.Np / 128 * tiles * a.count, a.runs}; }

template <bool SPLIT>
__global__ void __launch_bounds__(THR, 2) runs_kernel(const MuonArgs a) {
  const int side = a.Mp / 128, tiles = side * (side + 1) / 2, of_xcd = (a.runs + NXCD - 1) / NXCD;
  const int g = blockIdx.x % NXCD * of_xcd + blockIdx.x / NXCD;
  if (blockIdx.x / NXCD >= of_xcd || g >= a.runs) return;
  const Runs r = runs_of(a, tiles);
  const int end = r.start(g + 1);
  int part = 2 * g;
#pragma nounroll
  for (int at = r.start(g); at < end;) {
    const int tile = at / r.each, from = at - tile * r.each, n = min(end - at, r.each - from);
    int tm, tn;
    lower_tile(tile % tiles, tm, tn);
    product_tile<MF_GRAM, 2, 2, 2, 2, 4, SPLIT, OUT_PART>(a, tile / tiles, tm, tn, 2 * from, 2 * n, a.partial + (size_t)part++ * (128 * 128));
    at += n;
  }
}

// A workgroup adds up 32 x 32 elements, a lane four of a row, and writes them to both places of A
template <bool SPLIT>
__global__ void __launch_bounds__(256) joined_kernel(const MuonArgs a) {
  __shared__ float v[32][33];
  const int side = a.Mp / 128, tiles = side * (side + 1) / 2, tile = blockIdx.x >> 4, sub = blockIdx.x & 15;
  const Runs r = runs_of(a, tiles);
  // the runs g that meet the tile; only the first may have another tile before it
  const int begin = tile * r.each, end = begin + r.each;
  int g = (int)((unsigned)begin * (unsigned)r.runs / (unsigned)r.work), last = min((int)((unsigned)end * (unsigned)r.runs / (unsigned)r.work), r.runs - 1);
  while (r.start(g + 1) <= begin) ++g;
  while (r.start(last) >= end) --last;
  const float* from = a.partial + sub * 1024 + threadIdx.x * 4;
  f32x4 sum = *(const f32x4*)(from + (size_t)(2 * g + (r.start(g) < begin)) * (128 * 128));
  from += (size_t)(2 * g) * (128 * 128);
#pragma unroll 8
  for (++g; g <= last; ++g) sum += *(const f32x4*)(from += 2 * 128 * 128);
  int tm, tn;
  lower_tile(tile % tiles, tm, tn);
  const int b = tile / tiles, lane = threadIdx.x & 63;
  const int row = lane & 31, col = (threadIdx.x >> 6) * 8 + (lane >> 5) * 4;
  const int m0 = tm * 128 + (sub >> 2) * 32, n0 = tn * 128 + (sub & 3) * 32;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float w = sum[j] * (1.f / MUON_SCALE);
    if (m0 + row == n0 + col + j) {
      a.da[(size_t)b * a.Mp + m0 + row] = w * (1.f / MUON_SCALE);
      w = 0.f;
    }
    v[row][col + j] = w;
  }
  __syncthreads();
  const int at = threadIdx.x >> 3, c = threadIdx.x & 7;
  auto write = [&](size_t to, const f32x4& w) {
    typedef __attribute__((ext_vector_type(4))) _Float16 f16x4;
    f16x4 hi, lo;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      hi[j] = (_Float16)w[j];
      lo[j] = (_Float16)(w[j] - (float)hi[j]);
    }
    *(f16x4*)(a.A + to) = hi;
    if (SPLIT) *(f16x4*)(a.A_lo + to) = lo;
  };
  const size_t aat = (size_t)b * a.Mp * a.Mp;
  write(aat + (size_t)(m0 + at) * a.Mp + n0 + c * 4, f32x4{v[at][c * 4], v[at][c * 4 + 1], v[at][c * 4 + 2], v[at][c * 4 + 3]});
  if (tm != tn) write(aat + (size_t)(n0 + at) * a.Mp + m0 + c * 4, f32x4{v[c * 4][at], v[c * 4 + 1][at], v[c * 4 + 2][at], v[c * 4 + 3][at]});
}

template <int FORM, int WR, int WC, int MT, int NT, int D>
hipError_t launch(const MuonArgs& a, hipStream_t st) {
  constexpr int B = WR * MT * 32;
  const long long m = (a.Mp + B - 1) / B, n = (a.Np + B - 1) / B;
  const long long all = (FORM == MF_GRAM || FORM == MF_POLY ? m * (m + 1) / 2 : m * n) * a.count;
  const unsigned grid = (unsigned)((all + NXCD - 1) / NXCD * NXCD);
#define MOE_PRODUCT(SPLIT, OUT) product_kernel<FORM, WR, WC, MT, NT, D, SPLIT, OUT><<<grid, THR, 0, st>>>(a)
  if constexpr (FORM == MF_LAST) {
    const MuonStack& s = a.s[0];  // all stacks have what the first has
    if (!s.m) {
      if (a.split) MOE_PRODUCT(true, OUT_O);
      else MOE_PRODUCT(false, OUT_O);
    } else if (s.master) {
      MOE_PRODUCT(false, OUT_MASTER);
    } else if (a.split) {
      MOE_PRODUCT(true, OUT_P);
    } else {
      MOE_PRODUCT(false, OUT_P);
    }
  } else {
    if (a.split) MOE_PRODUCT(true, OUT_NONE);
    else MOE_PRODUCT(false, OUT_NONE);
  }
#undef MOE_PRODUCT
  return hipGetLastError();
}

constexpr long long CUS = 256;

// Tiles of 256 x 256 read least, one workgroup a CU; of 128 x 128, two a CU, they take a round of 256 tiles as long as 680 of
// theirs: one X of 2048 x 5632 (176 tiles, or 704) takes 67 us either way, of 2048 x 4096 (128, 512) 58 and 48, of 2048 x 7168
// (224, 896) 72 and 79; five of 2048 x 2048 (320, 1280) two rounds of 64, or 118. Where every 128 x 128 tile has a CU for
// itself, Gram's matrix, whose reduction is the long side, takes a ring of four slots: three of 771 x 1000 (84 tiles)
// 13.1 us, with two slots 15.4; one of 2048 x 7168 (136) 60 and 82. The others' operands come by halves of slots, which does
// as much: 14.6 and 15.0.
template <int FORM>
hipError_t choose(const MuonArgs& a, hipStream_t st) {
  auto tiles = [&](int b) {
    const long long m = (a.Mp + b - 1) / b, n = (a.Np + b - 1) / b;
    return (FORM == MF_GRAM || FORM == MF_POLY ? m * (m + 1) / 2 : m * n) * a.count;
  };
  if (tiles(128) >= 680 * ((tiles(256) + CUS - 1) / CUS)) return launch<FORM, 2, 2, 4, 4, 2>(a, st);
  if constexpr (FORM == MF_GRAM)
    if (tiles(128) <= CUS) return launch<FORM, 2, 2, 2, 2, 4>(a, st);
  return launch<FORM, 2, 2, 2, 2, 2>(a, st);
}

}  // namespace

// Runs are worth it where the tiles leave most CUs idle: bf16, 1 of 1024 x 4096 (36 tiles) takes 29.6 us by tiles and 13.8 + 5.6
// by runs and sums, 2 of 1024 x 2048 (72) 18.5 and 13.5 + 5.8; fp32, 2 of 79 x 4042 (2) 74 and 7.9 + 6.1, 8 of 1000 x 500 (80) 28
// and 16.2 + 6.3. With more tiles a step waits for its operands: tiles that go through the reduction together share them in
// their XCD's L2, runs do not (1 of 2048 x 7168, 136 tiles: 64 and 58 + 11). A run has two pairs of steps at least, and saves six
// (f32: a pair counts for three): 1 of 200 x 1000 (3 tiles of 8 pairs) takes 11.5 us by tiles and 5.9 + 3.4 by runs.
int muon_runs(int Mp, int Np, long long count, bool split) {
  const long long side = Mp / 128, tiles = side * (side + 1) / 2 * count, each = Np / 128, pair = split ? 3 : 1;
  if (tiles > (split ? CUS / 2 : CUS / 4)) return 0;
  const long long work = tiles * each, runs = std::max(std::min({CUS, work, work * pair / 2}), tiles);
  return (each - work / runs) * pair >= 6 ? (int)runs : 0;
}

hipError_t launch_muon_product(MuonForm form, const MuonArgs& a, hipStream_t st) {
  switch (form) {
    case MF_GRAM:
      if (a.runs) {
        const int side = a.Mp / 128, tiles = side * (side + 1) / 2 * a.count;
        const unsigned grid = (unsigned)((a.runs + NXCD - 1) / NXCD * NXCD);
        if (a.split) {
          runs_kernel<true><<<grid, THR, 0, st>>>(a);
          joined_kernel<true><<<tiles * 16, 256, 0, st>>>(a);
        } else {
          runs_kernel<false><<<grid, THR, 0, st>>>(a);
          joined_kernel<false><<<tiles * 16, 256, 0, st>>>(a);
        }
        return hipGetLastError();
      }
      return choose<MF_GRAM>(a, st);
    case MF_POLY: return choose<MF_POLY>(a, st);
    case MF_STEP: return choose<MF_STEP>(a, st);
    case MF_LAST: return choose<MF_LAST>(a, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace moe
