// The gated feed-forward block's products in bf16 (v_mfma_f32_32x32x16_bf16); forms as listed in train.h.
//
// C[m][n] = sum_k P(m, k) Q(n, k), a tile of C per workgroup of 4 waves. Both operands go from global memory
// to LDS without passing registers (global_load_lds), through a ring of D slots of 64 reduction elements, and
// from there to the matrix cores a quarter of a slot (16 elements) at a time: while the products of one quarter
// run, the next one is read, and loads for a later step go out, a few behind every quarter. Weights are read
// as they are stored: an operand whose reduction index is contiguous (dy, dg | du, and the weights in the
// gradients of h and x) is read 16 bytes a lane; one whose own index is (the weights in the forward products,
// everything in the weight gradients) by transposing reads (ds_read_b64_tr_b16). Q is the MFMA's first operand,
// so that a lane ends with 4 consecutive columns of one row.
//
// Numerics: sums, SiLU and its slope are fp32. h, dg and du are rounded to bf16 when they are written, because the
// next product's instruction takes no wider operand: y, dx and the weight gradients are off by 0.0023 of their norm,
// by 0.0017 if only they themselves were rounded.
//
// At 8192 rows, H 8192, I 4096 the forms reach 1160 (gate/up), 1280 (down), 1180 (dh), 1300 (dx) and 1380 (weight
// gradients) TFLOP/s on random data, where the library's products of 8192^3 reach 1240, 1540 (dh and dx's layout) and
// 1090 (the weight gradients' layout). On zeros, which cost little power, they reach 1540, 1850, 1290, 1480 and 1990:
// gate/up, down and the weight gradients are bound by the matrix cores under the card's power limit, dh and dx, which
// gain 9% and 14% only, are not. Both of their operands are KC: in two slots all loads of a step are out by its second
// quarter and waited for at the end of its third (FLY2 = 0), the likeliest reason by the code; no counter was taken.
#include <algorithm>
#include <type_traits>

#include "train.h"

namespace moe {

namespace {

constexpr int BK = 64;     // reduction elements per step: 128 bytes of a row, a whole cache line
constexpr int THR = 256;   // 4 waves
constexpr int NXCD = 8;
constexpr int NON_TEMPORAL = 2;                // cache policy of a load: nt
constexpr long long CACHE_BYTES = 256LL << 20;  // of the last-level cache

typedef __attribute__((address_space(3))) uint8_t lds_byte;
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) bf16x8 lds_bf16x8;
typedef __attribute__((ext_vector_type(16))) float f32x16;

#define MOE_WAIT_VMCNT(n) __builtin_amdgcn_s_waitcnt(((n) & 15) | (((n) >> 4) << 14) | 0x70 | 0xF00)
#define MOE_WAIT_LGKM0() __builtin_amdgcn_s_waitcnt(0xC07F)

__device__ const uint4 zero_chunk = {0u, 0u, 0u, 0u};

// One operand's tile in LDS: L indices x 64 reduction elements per slot, as L / 8 units of 1 KiB, each
// moved by one wave-wide 16-byte load straight to LDS. A fragment is 32 indices x 16 reduction elements
// (quarter h of the step): lane l holds index l % 32, elements 16 h + 8 (l / 32) .. + 8.
//   KC (reduction index contiguous in memory): unit u holds indices 8 u .. + 8, 128 bytes each; 16-byte
//     chunk c of row r sits at c ^ ((r >> 1) & 7), so that 16 lanes' reads cover all 64 banks.
//   MC (own index contiguous): a row of L indices per reduction element, read 4 x 16 at a time by the
//     transposing read; 32-byte chunk c of row r sits at c ^ swz(r), so that its 4 rows differ in bank.
template <int L, bool KC, bool HALVES>
struct Tile {
  static constexpr int UNITS = L / 8;
  static constexpr int BYTES = L * BK * 2;
  static constexpr int LPR = L / 8;  // MC: lanes per row
  __device__ static constexpr int swz(int r) { return L >= 128 ? ((r & 3) << 1) : (r & 2); }
  // unit that wave w of 4 moves as its q-th; with HALVES the first half of them makes the slot's first 32 rows
  static constexpr int U = UNITS / 4;
  __device__ static int unit(int q, int w) {
    return HALVES ? (q / (U / 2)) * (UNITS / 2) + w * (U / 2) + q % (U / 2) : w * U + q;
  }
  // index (KC) or reduction element (MC) that lane l of unit u moves
  __device__ static int row(int u, int l) { return KC ? u * 8 + (l >> 3) : (u * 64 + l) / LPR; }
  // first of the 8 elements it moves: reduction elements (KC) or indices (MC)
  __device__ static int elem(int u, int l) {
    if (KC) return ((l & 7) ^ ((row(u, l) >> 1) & 7)) * 8;
    const int p = l % LPR;
    return ((p >> 1) ^ swz(row(u, l))) * 16 + (p & 1) * 8;
  }
  // Lane l's byte of the fragment of indices 32 t.. + 32, quarter h: a register for each h (KC) or t (MC)
  // and a constant for the other
  __device__ static int kc_at(int t0, int h, int l) { return (t0 * 32 + (l & 31)) * 128 + (((2 * h + (l >> 5)) ^ ((l >> 1) & 7)) << 4); }
  __device__ static int mc_at(int t, int l) {
    const int r = 8 * (l >> 5) + ((l & 15) >> 2);
    return r * (L * 2) + (((2 * t + ((l >> 4) & 1)) ^ swz(r)) << 5) + (l & 3) * 8;
  }
};

__device__ __forceinline__ u32x4 pack8(const f32x4& a, const f32x4& b) {
  return u32x4{pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3])};
}

template <int L, bool KC>
__device__ __forceinline__ bf16x8 read_frag(const lds_byte* at) {
  if constexpr (KC) {
    return *(const lds_bf16x8*)at;
  } else {
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 4 * (L * 2)));
    typedef __attribute__((ext_vector_type(8))) short s16x8;
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
}

// The weight gradients' tiles, square ones of 128 or 256: 3 E matrices of `longer` x `shorter` tiles, cut along
// the longer side into `per` units of up to `len` x `shorter`
struct DwUnits {
  int longer, shorter, len, per, tiles;
};
__host__ __device__ __forceinline__ DwUnits dw_units(int H, int I, int E, int bm) {
  DwUnits u;
  const int th = (H + bm - 1) / bm, ti = (I + bm - 1) / bm;
  u.longer = th > ti ? th : ti;
  u.shorter = th > ti ? ti : th;
  // units of about 4, of 1 where the XCDs would else get few and unequal numbers of them
  const int cut = 3 * E * ((u.longer + 3) / 4) >= 64 ? (u.longer + 3) / 4 : u.longer;
  u.len = (u.longer + cut - 1) / cut;
  u.per = (u.longer + u.len - 1) / u.len;
  u.tiles = u.len * u.shorter;
  return u;
}

// Number of row tiles of bm rows that the groups take, the same for every lane of a wave
__device__ __forceinline__ int row_tiles(const int32_t* off, int E, int P, int bm) {
  if (!off) return (P + bm - 1) / bm;
  const int lane = threadIdx.x & 63;
  int n = 0;
  for (int e = lane; e < E; e += 64) {
    int b, z;
    group_rows(off, e, P, b, z);
    n += (z - b + bm - 1) / bm;
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) n += __shfl_xor(n, d);
  return __builtin_amdgcn_readfirstlane(n);
}

// Which loads go behind which phase (quarter) of a step, for a ring of D slots. Quarter h + 1 is read in phase
// h, so the first half of a slot is free after phase 0 and all of it after phase 2.
//   whole slots: phases 3 of step s and 0, 1 of s + 1 bring stage s + D.
//   halves: phases 1, 2 of step s bring the first half of stage s + D, phases 3 of s and 0 of s + 1 its second
//     half.
// U loads each per wave and stage, spread evenly: bursts lengthen the wait for all of them.
template <bool HALVES, int U>
struct Share {
  // cumulative loads before the k-th of the phases in their order: 3 0 1 2 (whole), 1 2 3 0 (halves)
  static constexpr int cum(int k) { return HALVES ? U * k / 4 : (k >= 3 ? U : (U * 3 * k + 7) / 8); }
  static constexpr int from(int ph, int past = 0) { return cum((HALVES ? (ph + 3) % 4 : (ph + 1) % 4) + past); }
  static constexpr int count(int ph) { return from(ph, 1) - from(ph); }
};

// STREAM: the weights are read once and come from memory, so they pass the caches without staying there
template <int FORM, int WR, int WC, int MT, int NT, int D, bool STREAM>
__global__ void __launch_bounds__(THR, MT * NT > 8 ? 1 : 2) train_bf16_kernel(const TrainArgs a) {
  constexpr bool P_KC = FORM != TF_DW, Q_KC = FORM == TF_DH || FORM == TF_DX;
  constexpr int BM = WR * MT * 32, BN = WC * NT * 32;
  constexpr bool P_HV = !P_KC && D == 2, Q_HV = !Q_KC && D == 2;  // slots freed and filled by halves
  using TP = Tile<BM, P_KC, P_HV>;
  using TQ = Tile<BN, Q_KC, Q_HV>;
  constexpr int UP = TP::U, UQ = TQ::U, L = UP + UQ;  // loads per wave and stage
  static_assert(WR * WC == 4, "four waves share the units");
  using SP = Share<P_HV, UP>;
  using SQ = Share<Q_HV, UQ>;
  constexpr int OUTN = FORM == TF_GATE_UP ? BN / 2 : BN;  // columns of the output (per matrix)
  // D slots for each operand; with two slots those of a MC operand are freed and filled by halves of 32 rows,
  // all others whole (a cache line of every row). One array for each such part: the compiler then sees which
  // loads to LDS a read has to wait for.
  constexpr int PA = P_HV ? TP::BYTES / 2 : TP::BYTES, QA = Q_HV ? TQ::BYTES / 2 : TQ::BYTES;
  constexpr int PX = P_HV || D == 4 ? PA : 16, QX = Q_HV || D == 4 ? QA : 16;
  __shared__ __align__(1024) uint8_t p0[PA], p1[PA], p2[PX], p3[PX], q0[QA], q1[QA], q2[QX], q3[QX];
  // part B (0 or 1, of halves) of a slot
#define P_PART(SLOT, B) ((lds_byte*)((SLOT) + (P_HV && (B) ? 2 : 0) == 0 ? p0 : (SLOT) + (P_HV && (B) ? 2 : 0) == 1 ? p1 : (SLOT) + (P_HV && (B) ? 2 : 0) == 2 ? p2 : p3))
#define Q_PART(SLOT, B) ((lds_byte*)((SLOT) + (Q_HV && (B) ? 2 : 0) == 0 ? q0 : (SLOT) + (Q_HV && (B) ? 2 : 0) == 1 ? q1 : (SLOT) + (Q_HV && (B) ? 2 : 0) == 2 ? q2 : q3))
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave / WC, wc = wave % WC;
  const size_t H = a.H, I = a.I, HI = H * I;

  // --- the tile
  int e = 0, m0, mend, n0, K, beg = 0, mat = 0;
  const int N = FORM == TF_DOWN || FORM == TF_DX ? a.H : a.I;
  {
    // Workgroup b runs on XCD b % 8. What one XCD runs at a time shares operands in its L2.
    const int xcd = blockIdx.x % NXCD, j = blockIdx.x / NXCD;
    if constexpr (FORM == TF_DW) {
      // units of `len` tiles of the longer side x all of the shorter side go to the XCDs in turn
      const DwUnits u = dw_units(a.H, a.I, a.E, BM);
      const int unit = xcd + NXCD * (j / u.tiles), in = j % u.tiles;
      if (unit >= u.per * 3 * a.E) return;
      e = unit / (3 * u.per);
      mat = unit / u.per % 3;
      const int lt = unit % u.per * u.len + in % u.len, st = in / u.len;
      if (lt >= u.longer) return;
      // gate and up have H rows, down has them as columns; the longer side may be either
      const bool rows_long = (a.H >= a.I) == (mat < 2);
      m0 = (rows_long ? lt : st) * BM;
      n0 = (rows_long ? st : lt) * BN;
      mend = mat == 2 ? a.I : a.H;
      if (m0 >= mend || n0 >= (mat == 2 ? a.H : a.I)) return;
      int end;
      group_rows(a.off, e, a.P, beg, end);
      K = end - beg;
    } else {
      // 4 row tiles x all columns after each other; each XCD gets an equal run of the tiles that exist
      const int cols = (N + OUTN - 1) / OUTN, rows = row_tiles(a.off, a.E, a.P, BM);
      const int n = rows * cols, round = j / 32, left = n - round * 32 * NXCD;
      const int chunk = left >= 32 * NXCD ? 32 : (left + NXCD - 1) / NXCD;
      const int id = round * 32 * NXCD + xcd * chunk + j % 32;
      if (j % 32 >= chunk || id >= n) return;
      const int rb = id / (4 * cols), rr = min(4, rows - 4 * rb), rem = id - rb * 4 * cols;
      RowTile t;
      if (!find_row_tile(a.off, a.E, a.P, BM, rb * 4 + rem % rr, t)) return;
      e = t.e;
      m0 = t.row0;
      mend = t.end;
      n0 = rem / rr * OUTN;
      K = FORM == TF_GATE_UP || FORM == TF_DH ? a.H : FORM == TF_DOWN ? a.I : 2 * a.I;
    }
  }
  const int nsteps = (K + BK - 1) / BK;

  // --- loads: this wave's units of both operands
  const uint8_t* psrc[UP];
  const uint8_t* qsrc[UQ];
  size_t pstride = BK * 2, qstride = BK * 2;  // bytes per step
  size_t qjump = 0;                           // TF_DX: from the end of Wg's row to the start of Wu's
#pragma unroll
  for (int u = 0; u < UP; ++u) {
    const int un = TP::unit(u, wave), r = TP::row(un, lane), c = TP::elem(un, lane);
    if constexpr (P_KC) {
      const int row = m0 + r < mend ? m0 + r : mend - 1;  // past the group's end: not read
      if constexpr (FORM == TF_GATE_UP) {
        int s = a.slot_token ? a.slot_token[row] : row;
        if ((unsigned)s >= (unsigned)a.xrows) s = 0;  // its results become zeros
        psrc[u] = (const uint8_t*)a.x + (s * H + c) * 2;
      } else if constexpr (FORM == TF_DOWN) {
        psrc[u] = (const uint8_t*)a.h + (row * I + c) * 2;
      } else if constexpr (FORM == TF_DH) {
        psrc[u] = (const uint8_t*)a.dy + (row * H + c) * 2;
      } else {
        psrc[u] = (const uint8_t*)a.dgu + (row * (2 * I) + c) * 2;
      }
    } else {
      int col = m0 + c;
      if (col >= mend) col -= 128;  // H and I are multiples of 128: repeat columns that exist
      const size_t ld = mat == 2 ? I : H;
      psrc[u] = (const uint8_t*)(mat == 2 ? a.h : a.x) + ((size_t)(beg + r) * ld + col) * 2;
      pstride = BK * ld * 2;
    }
  }
#pragma unroll
  for (int u = 0; u < UQ; ++u) {
    const int un = TQ::unit(u, wave), r = TQ::row(un, lane), c = TQ::elem(un, lane);
    if constexpr (FORM == TF_GATE_UP) {
      // 32-column chunks in the order of the waves' fragments: NT / 2 of gate, the same columns of up
      const int ch = c >> 5, t = ch % NT;
      const int col = n0 + (ch / NT) * (NT * 16) + (t % (NT / 2)) * 32 + (c & 31);
      qsrc[u] = (const uint8_t*)(t < NT / 2 ? a.gate : a.up) + (e * HI + r * I + (col < (int)I ? col : col - 128)) * 2;
      qstride = BK * I * 2;
    } else if constexpr (FORM == TF_DOWN) {
      const int col = n0 + c;
      qsrc[u] = (const uint8_t*)a.down + (e * HI + r * H + (col < (int)H ? col : col - 128)) * 2;
      qstride = BK * H * 2;
    } else if constexpr (FORM == TF_DH) {
      const int n = n0 + r;
      qsrc[u] = (const uint8_t*)a.down + (e * HI + (n < (int)I ? n : n - 128) * H + c) * 2;
    } else if constexpr (FORM == TF_DX) {
      const int n = n0 + r;
      qsrc[u] = (const uint8_t*)a.gate + (e * HI + (n < (int)H ? n : n - 128) * I + c) * 2;
      qjump = (size_t)((const uint8_t*)a.up - (const uint8_t*)a.gate) - I * 2;
    } else {
      int col = n0 + c;
      if (col >= (mat == 2 ? (int)H : (int)I)) col -= 128;
      if (mat == 2) {
        qsrc[u] = (const uint8_t*)a.dy + ((size_t)(beg + r) * H + col) * 2;
        qstride = BK * H * 2;
      } else {
        qsrc[u] = (const uint8_t*)a.dgu + ((size_t)(beg + r) * (2 * I) + mat * I + col) * 2;
        qstride = BK * 2 * I * 2;
      }
    }
  }
  // One load of stage `step` to LDS; the source moves on by one step, and stays on the last one, whose
  // repeats nothing reads. With left < 0 (rows past the group's end) zeros come instead: they keep other rows'
  // values out of the sums, and where the results are not stored they save the power of a row's products
  // (1.5 to 2% of dh and dx of the ragged V3 slice).
  const int half_steps = (int)I / BK;
  auto load_one = [&](const uint8_t*& src, lds_byte* dst, int left, size_t adv, bool weights) __attribute__((always_inline)) {
    const uint8_t* const from = left >= 0 ? src : (const uint8_t*)&zero_chunk;
    if (STREAM && weights) __builtin_amdgcn_global_load_lds((const void*)from, (lds_void*)dst, 16, 0, NON_TEMPORAL);
    else __builtin_amdgcn_global_load_lds((const void*)from, (lds_void*)dst, 16, 0, 0);
    src += adv;
    asm volatile("" : "+v"(src));  // one running pointer a load, not one per load and slot
  };
  auto load_p = [&](int q, int step, auto slot) __attribute__((always_inline)) {
    const size_t adv = FORM == TF_DW || step + 1 < nsteps ? pstride : 0;
    const int un = TP::unit(q, wave);
    lds_byte* const part = P_PART(decltype(slot)::value, q >= UP / 2);
    load_one(psrc[q], part + (P_HV ? un % (TP::UNITS / 2) : un) * 1024,
             (P_KC ? mend - m0 : K - step * BK) - 1 - TP::row(un, lane), adv, false);
  };
  auto load_q = [&](int q, int step, auto slot) __attribute__((always_inline)) {
    size_t adv = FORM == TF_DW || step + 1 < nsteps ? qstride : 0;
    if constexpr (FORM == TF_DX) adv += step + 1 == half_steps ? qjump : 0;
    const int un = TQ::unit(q, wave);
    lds_byte* const part = Q_PART(decltype(slot)::value, q >= UQ / 2);
    load_one(qsrc[q], part + (Q_HV ? un % (TQ::UNITS / 2) : un) * 1024,
             FORM == TF_DW ? K - step * BK - 1 - TQ::row(un, lane) : 0, adv, true);
  };

  f32x16 acc[NT][MT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) acc[t][i][j] = 0.f;

  if (nsteps > 0) {
    // LDS bytes of this wave's fragments within a slot: a register per quarter for a KC operand, one per
    // fragment for an MC one
    int pb[P_KC ? 4 : MT], qb[Q_KC ? 4 : NT];
#pragma unroll
    for (int i = 0; i < (P_KC ? 4 : MT); ++i) pb[i] = P_KC ? TP::kc_at(wr * MT, i, lane) : TP::mc_at(wr * MT + i, lane);
#pragma unroll
    for (int t = 0; t < (Q_KC ? 4 : NT); ++t) qb[t] = Q_KC ? TQ::kc_at(wc * NT, t, lane) : TQ::mc_at(wc * NT + t, lane);
    bf16x8 pf[2][MT], qf[2][NT];  // two quarters: the one multiplied and the one read
    auto read_p = [&](int i, auto quarter, auto slot) __attribute__((always_inline)) {
      constexpr int h = decltype(quarter)::value;
      lds_byte* const part = P_PART(decltype(slot)::value, h >= 2);
      pf[h & 1][i] = read_frag<BM, P_KC>(part + (P_KC ? pb[h] + i * 4096 : pb[i] + (P_HV ? h & 1 : h) * 16 * (BM * 2)));
    };
    auto read_q = [&](int t, auto quarter, auto slot) __attribute__((always_inline)) {
      constexpr int h = decltype(quarter)::value;
      lds_byte* const part = Q_PART(decltype(slot)::value, h >= 2);
      qf[h & 1][t] = read_frag<BN, Q_KC>(part + (Q_KC ? qb[h] + t * 4096 : qb[t] + (Q_HV ? h & 1 : h) * 16 * (BN * 2)));
    };
    constexpr std::integral_constant<int, 0> C0{};
    constexpr std::integral_constant<int, 1> C1{};
    constexpr std::integral_constant<int, 2> C2{};
    constexpr std::integral_constant<int, 3> C3{};
    // the n-th load of phase ph of step s, those of whole slots first; slot: that of step s
    auto load_nth = [&](auto ph_c, int n, int s, auto slot) __attribute__((always_inline)) {
      constexpr int ph = decltype(ph_c)::value, np = SP::count(ph), nq = SQ::count(ph);
      constexpr std::integral_constant<int, (decltype(slot)::value + D - 1) % D> before{};
      const bool p = Q_HV ? n < np : n >= nq;
      const int at = p ? SP::from(ph) + (Q_HV ? n : n - nq) : SQ::from(ph) + (Q_HV ? n - np : n);
      // phase 0, and phase 1 for whole slots, still bring stage s + D - 1, into the slot of step s - 1
      if (p) {
        if constexpr (ph == 0 || (!P_HV && ph == 1)) load_p(at, s + D - 1, before);
        else load_p(at, s + D, slot);
      } else {
        if constexpr (ph == 0 || (!Q_HV && ph == 1)) load_q(at, s + D - 1, before);
        else load_q(at, s + D, slot);
      }
    };
    // Products of quarter h, with the reads of the next quarter early behind them and the phase's loads spread
    // over all of them.
    auto phase = [&](auto quarter, auto rd_slot, int s, auto slot) __attribute__((always_inline)) {
      constexpr int h = decltype(quarter)::value, LOADS = SP::count(h) + SQ::count(h);
      constexpr std::integral_constant<int, (h + 1) % 4> next{};
      constexpr int PRODUCTS = MT * NT, READS = MT + NT, SPAN = PRODUCTS > 4 ? PRODUCTS * 3 / 4 : PRODUCTS;
#pragma unroll
      for (int n = 0; n < PRODUCTS; ++n) {
        const int t = n % NT, i = n / NT;
        acc[t][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(qf[h & 1][t], pf[h & 1][i], acc[t][i], 0, 0, 0);
#pragma unroll
        for (int r = n * READS / SPAN; r < (n + 1) * READS / SPAN && r < READS; ++r) {
          if (r < NT) read_q(r, next, rd_slot);
          else read_p(r - NT, next, rd_slot);
        }
#pragma unroll
        for (int q = n * LOADS / PRODUCTS; q < (n + 1) * LOADS / PRODUCTS; ++q) load_nth(quarter, q, s, slot);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    // Loads that may still be in flight: where the second half of a slot is wanted (after phase 0), those of one
    // step; where the next stage is wanted (after phase 2), those since the last one of a whole slot of it, or of
    // one step where there is none.
    constexpr int FLY0 = L;
    constexpr int FLY2 = P_HV && Q_HV ? L : (D - 2) * L + (P_HV ? SP::count(1) + SP::count(2) : 0) + (Q_HV ? SQ::count(1) + SQ::count(2) : 0);
    auto body = [&](int s, auto slot) __attribute__((always_inline)) {
      constexpr std::integral_constant<int, (decltype(slot)::value + 1) % D> other{};
      // opaque in every step, so that the slot stays a constant and does not become a register per slot and
      // fragment
#pragma unroll
      for (int i = 0; i < MT && !P_KC; ++i) asm volatile("" : "+v"(pb[i]));
#pragma unroll
      for (int t = 0; t < NT && !Q_KC; ++t) asm volatile("" : "+v"(qb[t]));
      phase(C0, slot, s, slot);
      if constexpr (P_HV || Q_HV) {
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
    auto whole = [&](int step, auto slot) __attribute__((always_inline)) {
#pragma unroll
      for (int q = 0; q < UQ; ++q) load_q(q, step, slot);
#pragma unroll
      for (int q = 0; q < UP; ++q) load_p(q, step, slot);
    };
    whole(0, C0);
    if constexpr (D == 4) {
      whole(1, C1);
      whole(2, C2);
    }
    constexpr int Q1 = Q_HV ? UQ / 2 : 0, P1 = P_HV ? UP / 2 : 0;  // of stage 1, before phase 3 of step -1
#pragma unroll
    for (int q = 0; q < Q1; ++q) load_q(q, 1, C1);
#pragma unroll
    for (int q = 0; q < P1; ++q) load_p(q, 1, C1);
    constexpr std::integral_constant<int, D - 1> last{};
#pragma unroll
    for (int n = 0; n < SP::count(3) + SQ::count(3); ++n) load_nth(C3, n, -1, last);
    MOE_WAIT_VMCNT((D - 2) * L + Q1 + P1 + SP::count(3) + SQ::count(3));
    __builtin_amdgcn_s_barrier();
#pragma unroll
    for (int t = 0; t < NT; ++t) read_q(t, C0, C0);
#pragma unroll
    for (int i = 0; i < MT; ++i) read_p(i, C0, C0);
    // pairs of steps: H and I are multiples of 128, the rows of TF_DW end in zeros
    int s = 0;
    if constexpr (D == 4) {
      for (; s + 2 < nsteps; s += 4) {
        body(s, C0);
        body(s + 1, C1);
        body(s + 2, C2);
        body(s + 3, C3);
      }
    }
    for (; s < nsteps; s += 2) {
      body(s, C0);
      body(s + 1, C1);
    }
    MOE_WAIT_VMCNT(0);  // loads in flight land before the workgroup's LDS is released
  }

  // --- results. Element 4 q + j of a tile is column 8 q + 4 (lane / 32) + j of row lane % 32: 16 bytes of a
  // row per pair of lanes. Each wave passes them through 8 KiB of LDS of its own, 32 rows at a time, so that
  // a lane reads and writes global memory 16 bytes at a time and neighbours share cache lines. 16-byte chunk c
  // of a row sits at c ^ (row % chunks), which keeps both directions free of bank conflicts. The parts of the
  // ring serve for it: nothing is read or loaded there any more.
  static_assert((Q_HV || D == 4 ? QA : QA / 2) >= 8192, "a part of the ring per wave");
  __builtin_amdgcn_s_barrier();
  lds_byte* ep;
  if constexpr (Q_HV || D == 4) ep = (lds_byte*)(wave == 0 ? q0 : wave == 1 ? q1 : wave == 2 ? q2 : q3);
  else ep = (lds_byte*)(wave & 2 ? q1 : q0) + (wave & 1) * (QA / 2);
  typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
  typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
  typedef __attribute__((address_space(3))) u32x2 lds_u32x2;
  const int wrow = m0 + wr * MT * 32, r32 = lane & 31, hi4 = lane >> 5;
  // The lanes of a wave exchange data through ep: its LDS accesses run in the order in which they are
  // issued, and this keeps the compiler from changing that order.
  auto in_order = [] { __asm__ volatile("" ::: "memory"); };
  if constexpr (FORM == TF_GATE_UP || FORM == TF_DH) {
    // 64 fp32 columns: 32 of g beside the same 32 of u, or 64 of dh
    constexpr int BLOCKS = NT / 2;
    auto put = [&](int i, int blk) __attribute__((always_inline)) {
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const f32x16& v = acc[FORM == TF_GATE_UP ? blk + z * (NT / 2) : 2 * blk + z][i];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *(lds_f32x4*)(ep + r32 * 256 + (((z * 8 + 2 * q + hi4) ^ (r32 & 15)) << 4)) =
              f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
      }
    };
    auto get = [&](int row, int c) __attribute__((always_inline)) { return *(const lds_f32x4*)(ep + row * 256 + ((c ^ (row & 15)) << 4)); };
    if constexpr (FORM == TF_GATE_UP) {
      const int c8 = lane & 3;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int blk = 0; blk < BLOCKS; ++blk) {
          in_order();
          put(i, blk);
          in_order();
          const int n = n0 + wc * (NT * 16) + blk * 32 + c8 * 8;
#pragma unroll
          for (int it = 0; it < 2; ++it) {
            const int row = it * 16 + (lane >> 2), m = wrow + i * 32 + row;
            f32x4 g0 = get(row, 2 * c8), g1 = get(row, 2 * c8 + 1), u0 = get(row, 8 + 2 * c8), u1 = get(row, 9 + 2 * c8);
            if (m >= mend || n >= N) continue;
            if (a.slot_token && (unsigned)a.slot_token[m] >= (unsigned)a.xrows) g0 = g1 = u0 = u1 = f32x4{0.f, 0.f, 0.f, 0.f};
            const size_t at = m * I + n;
            if (a.g) {
              *(u32x4*)((uint16_t*)a.g + at) = pack8(g0, g1);
              *(u32x4*)((uint16_t*)a.u + at) = pack8(u0, u1);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              g0[j] = silu(g0[j]) * u0[j];
              g1[j] = silu(g1[j]) * u1[j];
            }
            *(u32x4*)((uint16_t*)a.h + at) = pack8(g0, g1);
          }
        }
    } else {
      // the next block's g and u are fetched before this block's results are formed
      const int c8 = lane & 7, r8 = lane >> 3;
      u32x4 gw[2][4], uw[2][4];
      auto fetch = [&](int b, int set) __attribute__((always_inline)) {
        const int i = b / BLOCKS, n = n0 + (wc * NT + b % BLOCKS * 2) * 32 + c8 * 8;
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          const int m = wrow + i * 32 + it * 8 + r8;
          gw[set][it] = uw[set][it] = u32x4{0u, 0u, 0u, 0u};
          if (m < mend && n < N) {
            gw[set][it] = *(const u32x4*)((const uint16_t*)a.g + m * I + n);
            uw[set][it] = *(const u32x4*)((const uint16_t*)a.u + m * I + n);
          }
        }
      };
      fetch(0, 0);
#pragma unroll
      for (int b = 0; b < MT * BLOCKS; ++b) {
        if (b + 1 < MT * BLOCKS) fetch(b + 1, (b + 1) & 1);
        in_order();
        put(b / BLOCKS, b % BLOCKS);
        in_order();
        const int i = b / BLOCKS, n = n0 + (wc * NT + b % BLOCKS * 2) * 32 + c8 * 8;
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          const int row = it * 8 + r8, m = wrow + i * 32 + row;
          const f32x4 d[2] = {get(row, 2 * c8), get(row, 2 * c8 + 1)};
          f32x4 dg[2], du[2], hv[2];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t gj2 = gw[b & 1][it][j >> 1], uj2 = uw[b & 1][it][j >> 1];
            const float gj = (j & 1) ? bf16hi(gj2) : bf16lo(gj2), uj = (j & 1) ? bf16hi(uj2) : bf16lo(uj2);
            const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-gj)), si = gj * s, dh = d[j >> 2][j & 3];
            du[j >> 2][j & 3] = dh * si;
            dg[j >> 2][j & 3] = dh * uj * (s + si * (1.0f - s));
            hv[j >> 2][j & 3] = si * uj;
          }
          if (m >= mend || n >= N) continue;
          uint16_t* const o = (uint16_t*)a.dgu + m * (2 * I) + n;
          *(u32x4*)o = pack8(dg[0], dg[1]);
          *(u32x4*)(o + I) = pack8(du[0], du[1]);
          *(u32x4*)((uint16_t*)a.h + m * I + n) = pack8(hv[0], hv[1]);
        }
      }
    }
  } else {
    // all the wave's columns in bf16
    constexpr int RB = NT * 64, CH = RB / 16, RPI = 1024 / RB;  // bytes and chunks of a row, rows per access
    const size_t ld = FORM == TF_DW && mat < 2 ? I : H;
    uint16_t* const out = FORM == TF_DW ? (uint16_t*)(mat == 0 ? a.dgate : mat == 1 ? a.dup : a.ddown) + e * HI
                                        : (uint16_t*)(FORM == TF_DOWN ? a.y : a.dx);
    const int c = lane % CH, n = n0 + wc * NT * 32 + c * 8;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      in_order();
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *(lds_u32x2*)(ep + r32 * RB + (((t * 4 + q) ^ (r32 % CH)) << 4) + hi4 * 8) =
              u32x2{pack_bf16x2(acc[t][i][4 * q], acc[t][i][4 * q + 1]), pack_bf16x2(acc[t][i][4 * q + 2], acc[t][i][4 * q + 3])};
      in_order();
#pragma unroll
      for (int it = 0; it < 32 / RPI; ++it) {
        const int row = it * RPI + lane / CH, m = wrow + i * 32 + row;
        const u32x4 v = *(const lds_u32x4*)(ep + row * RB + ((c ^ (row % CH)) << 4));
        if (m < mend && n < (int)ld) *(u32x4*)(out + m * ld + n) = v;
      }
    }
  }
}

template <int FORM, int WR, int WC, int MT, int NT, int D, bool STREAM = false>
hipError_t launch(const TrainArgs& a, hipStream_t st) {
  constexpr int BM = WR * MT * 32, BN = WC * NT * 32;
  long long n;
  if (FORM == TF_DW) {
    static_assert(FORM != TF_DW || BM == BN, "square tiles");
    const DwUnits u = dw_units(a.H, a.I, a.E, BM);
    n = ((long long)u.per * 3 * a.E + NXCD - 1) / NXCD * u.tiles;
  } else {
    const int N = FORM == TF_DOWN || FORM == TF_DX ? a.H : a.I, outn = FORM == TF_GATE_UP ? BN / 2 : BN;
    n = max_row_tiles(a.P, a.E, BM) * ((N + outn - 1) / outn);
    n = n / (32 * NXCD) * 32 + (n % (32 * NXCD) + NXCD - 1) / NXCD;
  }
  if (n == 0) return hipSuccess;
  const unsigned grid = (unsigned)(n * NXCD);
  train_bf16_kernel<FORM, WR, WC, MT, NT, D, STREAM><<<grid, THR, 0, st>>>(a);
  return hipGetLastError();
}

// Which tile, by the time it would take: rounds of the card times the time of a tile, steps of 64 reduction elements
// at so many microseconds each and what does not depend on them. Fitted to runs of 110 random sizes (8 to 32768 rows,
// 1 to 48 groups, H to 7168, I to 2048), where the tile taken is 0.3% slower than the best of the four on average,
// 0.6% for the weight gradients (one CU takes one 256 x 256 or four-slot workgroup, two 128 x 128 ones).
// Large problems are bound by the matrix cores and take the tile that reads LDS least; few or thin groups
// leave CUs empty or rows unused, and there the latency of a step counts: more and smaller tiles, more stages in
// flight. Measured on gate/up, best of the others in brackets: 32768 rows in 32 groups 1.78 ms (2.49); one
// group of 1027 rows, H 4096, I 1536: 43 us (79 as 256 x 256); 440 rows in 16 groups 76 us (88).
template <int FORM>
hipError_t choose(const TrainArgs& a, hipStream_t st) {
  auto rounds = [](double tiles, int per) { return (double)(long long)((tiles + per - 1) / per); };
  if constexpr (FORM == TF_DW) {
    // the 128 x 128 tiles' shorter rows of results cost at least 5.4 us a round
    const double steps = ((double)a.P / a.E + 127) / 128 * 2;
    const auto tiles = [&](int b) { return 3.0 * a.E * ((a.H + b - 1) / b) * ((a.I + b - 1) / b); };
    const double big = rounds(tiles(256), 256) * (1.24 * steps + 12), small = rounds(tiles(128), 512) * std::max(0.8 * steps + 4.2, 5.4);
    return big <= small ? launch<FORM, 2, 2, 4, 4, 2>(a, st) : launch<FORM, 2, 2, 2, 2, 2>(a, st);
  } else {
    const int N = FORM == TF_DOWN || FORM == TF_DX ? a.H : a.I, share = FORM == TF_GATE_UP ? 2 : 1;
    auto tiles = [&](int bm, int bn) {
      const int groups = std::min(a.E, a.P);
      const double rows = a.E == 1 ? (a.P + bm - 1) / bm : std::max<double>(groups, (double)a.P / bm + groups * 0.5);
      return rows * ((N * share + bn - 1) / bn);
    };
    const double steps = (FORM == TF_GATE_UP || FORM == TF_DH ? a.H : FORM == TF_DOWN ? a.I : 2 * a.I) / BK, b = tiles(128, 128);
    const double t[4] = {rounds(tiles(256, 256), 256) * (1.1 * steps + 11),
                         b > 256 ? rounds(b, 512) * (1.0 * steps + 3.8) + 3.7 : 0.52 * steps + 6.4,
                         rounds(tiles(64, 256), 256) * (0.47 * steps + 6.4) + 1.1,
                         rounds(tiles(64, 128), 256) * (0.31 * steps + 3.9) + 2.7};
    // The layer's weights go through once, no second row tile reads them and the last-level cache could not hold
    // them from before: 440 rows, H 4096, I 1536, 16 groups, gate/up 89 us with the default policy, 78 so; 100
    // rows in 8 groups, whose 200 MB were in the cache, 41 and 66.
    const bool stream = a.P <= 64LL * a.E && 6LL * a.E * a.H * a.I > CACHE_BYTES;
    switch (std::min_element(t, t + 4) - t) {
      case 0: return launch<FORM, 2, 2, 4, 4, 2>(a, st);
      case 1: return launch<FORM, 2, 2, 2, 2, 2>(a, st);
      case 2: return stream ? launch<FORM, 1, 4, 2, 2, 4, true>(a, st) : launch<FORM, 1, 4, 2, 2, 4>(a, st);
      default: return stream ? launch<FORM, 2, 2, 1, 2, 4, true>(a, st) : launch<FORM, 2, 2, 1, 2, 4>(a, st);
    }
  }
}

}  // namespace

hipError_t launch_train_bf16(TrainForm form, const TrainArgs& a, hipStream_t st) {
  switch (form) {
    case TF_GATE_UP: return choose<TF_GATE_UP>(a, st);
    case TF_DOWN: return choose<TF_DOWN>(a, st);
    case TF_DH: return choose<TF_DH>(a, st);
    case TF_DX: return choose<TF_DX>(a, st);
    case TF_DW: return choose<TF_DW>(a, st);  // x without slot_token here: its rows are gathered before
  }
  return hipErrorInvalidValue;
}

}  // namespace moe
