// The gated feed-forward block's products in bf16 (v_mfma_f32_16x16x32_bf16); forms as listed in
// train.h.
#include <type_traits>

#include "train.h"

namespace moe {

namespace {

constexpr int BK = 32;     // reduction elements per step
constexpr int THR = 256;   // 4 waves
constexpr int NXCD = 8;

typedef __attribute__((address_space(3))) uint8_t lds_byte;
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) bf16x8 lds_bf16x8;
typedef __attribute__((ext_vector_type(16))) float f32x16;

#define MOE_WAIT_VMCNT(n) __builtin_amdgcn_s_waitcnt(((n) & 15) | (((n) >> 4) << 14) | 0x70 | 0xF00)
#define MOE_WAIT_LGKM0() __builtin_amdgcn_s_waitcnt(0xC07F)

__device__ const uint4 zero_chunk = {0u, 0u, 0u, 0u};

// One operand's tile in LDS: L indices x 32 reduction elements per stage, as L / 16 units of 1 KiB,
// each moved by one wave-wide 16-byte load straight to LDS. A fragment is 32 indices x 16 reduction
// elements (half h of the step): lane l holds index l % 32, elements 16 h + 8 (l / 32) .. + 8.
//   KC (reduction index contiguous in memory): unit u holds indices 16 u .. + 16, 64 bytes each, whose
//     16-byte chunks are permuted by the row, so that 8 lanes' 16-byte reads cover all banks.
//   MC (own index contiguous): a row of L indices per reduction element, read 4 x 16 at a time by the
//     transposing read; 32-byte chunk c of row r sits at c ^ swz(r), so that its 4 rows differ in bank.
template <int L, bool KC>
struct Tile {
  static constexpr int UNITS = L / 16;
  static constexpr int BYTES = L * BK * 2;
  static constexpr int LPR = L / 8;  // MC: lanes per row
  __device__ static constexpr int swz(int r) { return L >= 128 ? ((r & 3) << 1) : (r & 2); }
  // index (KC) or reduction element (MC) that lane l of unit u moves
  __device__ static int row(int u, int l) { return KC ? u * 16 + (l >> 2) : u * (64 / LPR) + l / LPR; }
  // first of the 8 elements it moves: reduction elements (KC) or indices (MC)
  __device__ static int elem(int u, int l) {
    if (KC) return ((l & 3) ^ ((l >> 3) & 3)) * 8;
    const int p = l % LPR;
    return ((p >> 1) ^ swz(row(u, l))) * 16 + (p & 1) * 8;
  }
  // byte of lane l's part of the fragment of 32 indices from 32 t, half h, is at(t, l) + half(h, l):
  // KC: at(0, l) + 2048 t, and half(h, l) = half(0, l) ^ 32 h; MC: at(t, l) = at(0, l) ^ 64 t, half = row offset
  __device__ static int at(int t, int l) {
    const int i = l & 31;
    if (KC) return t * 2048 + i * 64;
    const int r = 8 * (l >> 5) + ((l & 15) >> 2);
    return r * (L * 2) + (((2 * t + ((l >> 4) & 1)) ^ swz(r)) << 5) + (l & 3) * 8;
  }
  __device__ static int chunk(int h, int l) { return (((2 * h + (l >> 5)) ^ ((l >> 1) & 3)) & 3) * 16; }
};

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

template <int FORM, int WR, int WC, int MT, int NT, int D>
__global__ void __launch_bounds__(THR, 1) train_bf16_kernel(const TrainArgs a) {
  constexpr bool P_KC = FORM != TF_DW, Q_KC = FORM == TF_DH || FORM == TF_DX;
  constexpr int BM = WR * MT * 32, BN = WC * NT * 32;
  using TP = Tile<BM, P_KC>;
  using TQ = Tile<BN, Q_KC>;
  constexpr int UP = TP::UNITS / 4, UQ = TQ::UNITS / 4, L = UP + UQ;  // loads per wave and stage
  static_assert(WR * WC == 4 && TP::UNITS % 4 == 0 && TQ::UNITS % 4 == 0, "four waves share the units");
  constexpr int OUTN = FORM == TF_GATE_UP ? BN / 2 : BN;  // columns of the output (per matrix)
  // one array per slot and operand: the compiler then sees which loads to LDS a read has to wait for
  __shared__ __align__(1024) uint8_t lp0[TP::BYTES], lp1[TP::BYTES], lp2[D > 2 ? TP::BYTES : 16], lp3[D > 2 ? TP::BYTES : 16];
  __shared__ __align__(1024) uint8_t lq0[TQ::BYTES], lq1[TQ::BYTES], lq2[D > 2 ? TQ::BYTES : 16], lq3[D > 2 ? TQ::BYTES : 16];
#define P_SLOT(S) ((lds_byte*)((S) == 0 ? lp0 : (S) == 1 ? lp1 : (S) == 2 ? lp2 : lp3))
#define Q_SLOT(S) ((lds_byte*)((S) == 0 ? lq0 : (S) == 1 ? lq1 : (S) == 2 ? lq2 : lq3))
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave / WC, wc = wave % WC;
  const size_t H = a.H, I = a.I, HI = H * I;

  // --- the tile
  int e = 0, m0, mend, n0, K, beg = 0, mat = 0;
  const int N = FORM == TF_DOWN || FORM == TF_DX ? a.H : a.I;
  {
    // superblocks of 4 x 8 tiles go to the XCDs in turn, so that the tiles which one XCD runs at the
    // same time share operands in its L2
    const int b = blockIdx.x;
    const int sb = (b / (32 * NXCD)) * NXCD + b % NXCD, in = (b / NXCD) % 32;
    if constexpr (FORM == TF_DW) {
      const int tg_m = (a.H + BM - 1) / BM, tg_n = (a.I + BN - 1) / BN, td_m = (a.I + BM - 1) / BM, td_n = (a.H + BN - 1) / BN;
      const int sg_n = (tg_n + 7) / 8, sg = (tg_m + 3) / 4 * sg_n, sd_n = (td_n + 7) / 8, sd = (td_m + 3) / 4 * sd_n;
      const int per = 2 * sg + sd;
      e = sb / per;
      if (e >= a.E) return;
      int r = sb % per;
      mat = r < sg ? 0 : r < 2 * sg ? 1 : 2;
      r -= mat * sg;
      const int sn = mat == 2 ? sd_n : sg_n;
      const int tm = r / sn * 4 + in % 4, tn = r % sn * 8 + in / 4;
      if (tm >= (mat == 2 ? td_m : tg_m) || tn >= (mat == 2 ? td_n : tg_n)) return;
      m0 = tm * BM;
      n0 = tn * BN;
      mend = mat == 2 ? a.I : a.H;
      int end;
      group_rows(a.off, e, a.P, beg, end);
      K = end - beg;
    } else {
      const int tn_all = (N + OUTN - 1) / OUTN, sn = (tn_all + 7) / 8;
      const int tm = sb / sn * 4 + in % 4, tn = sb % sn * 8 + in / 4;
      if (tn >= tn_all) return;
      RowTile t;
      if (!find_row_tile(a.off, a.E, a.P, BM, tm, t)) return;
      e = t.e;
      m0 = t.row0;
      mend = t.end;
      n0 = tn * OUTN;
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
    const int un = wave * UP + u, r = TP::row(un, lane), c = TP::elem(un, lane);
    if constexpr (P_KC) {
      // rows past the group's end repeat its last one: their results are not stored
      const int row = m0 + r < mend ? m0 + r : mend - 1;
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
    const int un = wave * UQ + u, r = TQ::row(un, lane), c = TQ::elem(un, lane);
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
  // Stage `step` (loads q of the wave) into a slot; the source moves on by one step, and stays on the last
  // one, whose repeats nothing reads. TF_DW: rows past the group's end read zeros.
  const int half_steps = (int)I / BK;
  auto load = [&](const uint8_t*& src, lds_byte* dst, int row, size_t adv, int step) __attribute__((always_inline)) {
    const uint8_t* from = src;
    if constexpr (FORM == TF_DW) from = row < K - step * BK ? from : (const uint8_t*)&zero_chunk;
    __builtin_amdgcn_global_load_lds((const void*)from, (lds_void*)dst, 16, 0, 0);
    src += adv;
    asm volatile("" : "+v"(src));  // one running pointer a load, not one per load and slot
  };
  auto load_p = [&](int q, int step, auto slot) __attribute__((always_inline)) {
    const size_t adv = FORM == TF_DW || step + 1 < nsteps ? pstride : 0;
    load(psrc[q], P_SLOT(decltype(slot)::value) + (wave * UP + q) * 1024, TP::row(wave * UP + q, lane), adv, step);
  };
  auto load_q = [&](int q, int step, auto slot) __attribute__((always_inline)) {
    size_t adv = FORM == TF_DW || step + 1 < nsteps ? qstride : 0;
    if constexpr (FORM == TF_DX) adv += step + 1 == half_steps ? qjump : 0;
    load(qsrc[q], Q_SLOT(decltype(slot)::value) + (wave * UQ + q) * 1024, TQ::row(wave * UQ + q, lane), adv, step);
  };

  f32x16 acc[NT][MT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) acc[t][i][j] = 0.f;

  if (nsteps > 0) {
    auto fill = [&](auto slot) __attribute__((always_inline)) {
      constexpr int S = decltype(slot)::value;
#pragma unroll
      for (int q = 0; q < UP; ++q) load_p(q, S, slot);
#pragma unroll
      for (int q = 0; q < UQ; ++q) load_q(q, S, slot);
    };
    fill(std::integral_constant<int, 0>{});
    fill(std::integral_constant<int, 1>{});
    fill(std::integral_constant<int, 2>{});
    fill(std::integral_constant<int, 3>{});
    // LDS bytes of this wave's fragments within a slot: a register per half for a KC operand, one per
    // fragment for an MC one
    int pb[P_KC ? 2 : MT], qb[Q_KC ? 2 : NT];
#pragma unroll
    for (int i = 0; i < (P_KC ? 2 : MT); ++i)
      pb[i] = P_KC ? TP::at(wr * MT, lane) + TP::chunk(i, lane) : TP::at(wr * MT + i, lane);
#pragma unroll
    for (int t = 0; t < (Q_KC ? 2 : NT); ++t)
      qb[t] = Q_KC ? TQ::at(wc * NT, lane) + TQ::chunk(t, lane) : TQ::at(wc * NT + t, lane);
    bf16x8 pf[2][MT], qf[2][NT];  // by half
    auto read_p = [&](int i, auto half, auto slot) __attribute__((always_inline)) {
      constexpr int h = decltype(half)::value;
      pf[h][i] = read_frag<BM, P_KC>(P_SLOT(decltype(slot)::value) + (P_KC ? pb[h] + i * 2048 : pb[i] + h * 16 * (BM * 2)));
    };
    auto read_q = [&](int t, auto half, auto slot) __attribute__((always_inline)) {
      constexpr int h = decltype(half)::value;
      qf[h][t] = read_frag<BN, Q_KC>(Q_SLOT(decltype(slot)::value) + (Q_KC ? qb[h] + t * 2048 : qb[t] + h * 16 * (BN * 2)));
    };
    // products of half h, with the reads of the other half and, for LOADS, stage `step` loaded into SL
    auto phase = [&](auto half, auto rd_slot, auto slot, auto loads, int step) __attribute__((always_inline)) {
      constexpr int h = decltype(half)::value;
      constexpr std::integral_constant<int, h ^ 1> other{};
      constexpr int N_MFMA = MT * NT, READS = MT + NT, LD = decltype(loads)::value ? L : 0;
#pragma unroll
      for (int n = 0; n < N_MFMA; ++n) {
        const int t = n % NT, i = n / NT;
        acc[t][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(qf[h][t], pf[h][i], acc[t][i], 0, 0, 0);
        // reads in the order in which the next phase needs them: q, p0, then the other rows
#pragma unroll
        for (int r = n * READS / N_MFMA; r < (n + 1) * READS / N_MFMA; ++r) {
          if (r < NT) read_q(r, other, rd_slot);
          else read_p(r - NT, other, rd_slot);
        }
#pragma unroll
        for (int q = n * LD / N_MFMA; q < (n + 1) * LD / N_MFMA; ++q) {
          if (q < UP) load_p(q, step, slot);
          else load_q(q - UP, step, slot);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    constexpr std::integral_constant<int, 0> H0{};
    constexpr std::integral_constant<int, 1> H1{};
    // step s in slot SL: its second half is read during the first one's products; then every wave is done
    // with the slot, stage s + 1 is there, and stage s + D goes into the slot
    auto body = [&](int s, auto slot) __attribute__((always_inline)) {
      constexpr std::integral_constant<int, (decltype(slot)::value + 1) % D> next{};
      // opaque in every step, so that the slot stays a constant and does not become a register per slot and
      // fragment
#pragma unroll
      for (int i = 0; i < MT && !P_KC; ++i) asm volatile("" : "+v"(pb[i]));
#pragma unroll
      for (int t = 0; t < NT && !Q_KC; ++t) asm volatile("" : "+v"(qb[t]));
      phase(H0, slot, slot, std::false_type{}, 0);
      MOE_WAIT_LGKM0();
      MOE_WAIT_VMCNT((D - 2) * L);
      __builtin_amdgcn_s_barrier();
      phase(H1, next, slot, std::true_type{}, s + D);
    };
    MOE_WAIT_VMCNT((D - 1) * L);
    __builtin_amdgcn_s_barrier();
#pragma unroll
    for (int t = 0; t < NT; ++t) read_q(t, H0, H0);
#pragma unroll
    for (int i = 0; i < MT; ++i) read_p(i, H0, H0);
    // whole rounds of the ring: H and I are multiples of 128, the rows of TF_DW end in zeros
    for (int s = 0; s < nsteps; s += D) {
      body(s, H0);
      body(s + 1, H1);
      body(s + 2, std::integral_constant<int, 2>{});
      body(s + 3, std::integral_constant<int, 3>{});
    }
    MOE_WAIT_VMCNT(0);  // loads in flight land before the workgroup's LDS is released
  }

  // --- results: element 4 q + j of a tile is column 8 q + 4 (lane / 32) + j of row lane % 32
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = m0 + (wr * MT + i) * 32 + (lane & 31);
    if (m >= mend) continue;
    if constexpr (FORM == TF_GATE_UP) {
      bool ok = true;
      if (a.slot_token) ok = (unsigned)a.slot_token[m] < (unsigned)a.xrows;
#pragma unroll
      for (int t = 0; t < NT / 2; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int n = n0 + wc * (NT * 16) + t * 32 + 8 * q + 4 * (lane >> 5);
          if (n >= N) continue;
          float gv[4], uv[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            gv[j] = ok ? acc[t][i][4 * q + j] : 0.f;
            uv[j] = ok ? acc[t + NT / 2][i][4 * q + j] : 0.f;
          }
          const size_t at = (m * I + n) * 2;
          if (a.g) {
            *(u32x2*)((uint8_t*)a.g + at) = u32x2{pack_bf16x2(gv[0], gv[1]), pack_bf16x2(gv[2], gv[3])};
            *(u32x2*)((uint8_t*)a.u + at) = u32x2{pack_bf16x2(uv[0], uv[1]), pack_bf16x2(uv[2], uv[3])};
          }
          *(u32x2*)((uint8_t*)a.h + at) = u32x2{pack_bf16x2(silu(gv[0]) * uv[0], silu(gv[1]) * uv[1]),
                                                pack_bf16x2(silu(gv[2]) * uv[2], silu(gv[3]) * uv[3])};
        }
    } else {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int n = n0 + (wc * NT + t) * 32 + 8 * q + 4 * (lane >> 5);
          const f32x4 v = {acc[t][i][4 * q], acc[t][i][4 * q + 1], acc[t][i][4 * q + 2], acc[t][i][4 * q + 3]};
          if constexpr (FORM == TF_DH) {
            if (n >= N) continue;
            const u32x2 gw = *(const u32x2*)((const uint8_t*)a.g + (m * I + n) * 2);
            const u32x2 uw = *(const u32x2*)((const uint8_t*)a.u + (m * I + n) * 2);
            float dg[4], du[4], hv[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float gj = (j & 1) ? bf16hi(gw[j >> 1]) : bf16lo(gw[j >> 1]);
              const float uj = (j & 1) ? bf16hi(uw[j >> 1]) : bf16lo(uw[j >> 1]);
              const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-gj)), si = gj * s;
              du[j] = v[j] * si;
              dg[j] = v[j] * uj * (s + si * (1.0f - s));
              hv[j] = si * uj;
            }
            uint8_t* const o = (uint8_t*)a.dgu + (m * (2 * I) + n) * 2;
            *(u32x2*)o = u32x2{pack_bf16x2(dg[0], dg[1]), pack_bf16x2(dg[2], dg[3])};
            *(u32x2*)(o + I * 2) = u32x2{pack_bf16x2(du[0], du[1]), pack_bf16x2(du[2], du[3])};
            *(u32x2*)((uint8_t*)a.h + (m * I + n) * 2) = u32x2{pack_bf16x2(hv[0], hv[1]), pack_bf16x2(hv[2], hv[3])};
          } else {
            uint8_t* o;
            if constexpr (FORM == TF_DW) {
              const size_t ld = mat == 2 ? H : I;
              if (n >= (int)ld) continue;
              o = (uint8_t*)(mat == 0 ? a.dgate : mat == 1 ? a.dup : a.ddown) + (e * HI + m * ld + n) * 2;
            } else {
              if (n >= N) continue;
              o = (uint8_t*)(FORM == TF_DOWN ? a.y : a.dx) + (m * H + n) * 2;
            }
            *(u32x2*)o = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
          }
        }
    }
  }
}

// Rows of x in the grouped order, zeros for tokens outside x: TF_DW then reads its row operand by row
__global__ void __launch_bounds__(THR) gather_kernel(const TrainArgs a) {
  const int cpr = a.H / 8;
  const long long id = (long long)blockIdx.x * THR + threadIdx.x;
  if (id >= (long long)a.P * cpr) return;
  const int r = (int)(id / cpr), c = (int)(id - (long long)r * cpr), s = a.slot_token[r];
  u32x4 v = {0u, 0u, 0u, 0u};
  if ((unsigned)s < (unsigned)a.xrows) v = *((const u32x4*)a.x + (size_t)s * cpr + c);
  *((u32x4*)a.xg + id) = v;
}

template <int FORM>
hipError_t launch(const TrainArgs& a, hipStream_t st) {
  constexpr int BM = 256, BN = 256;
  long long sbs;
  if (FORM == TF_DW) {
    auto blocks = [](int m, int n) { return (long long)((m + BM - 1) / BM + 3) / 4 * (((n + BN - 1) / BN + 7) / 8); };
    sbs = (2 * blocks(a.H, a.I) + blocks(a.I, a.H)) * a.E;
  } else {
    const int N = FORM == TF_DOWN || FORM == TF_DX ? a.H : a.I, outn = FORM == TF_GATE_UP ? BN / 2 : BN;
    sbs = (max_row_tiles(a.P, a.E, BM) + 3) / 4 * (((N + outn - 1) / outn + 7) / 8);
  }
  if (sbs == 0) return hipSuccess;
  const unsigned grid = (unsigned)((sbs + NXCD - 1) / NXCD * NXCD * 32);
  train_bf16_kernel<FORM, 2, 2, 4, 4, 4><<<grid, THR, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_train_bf16(TrainForm form, const TrainArgs& a, hipStream_t st) {
  switch (form) {
    case TF_GATE_UP: return launch<TF_GATE_UP>(a, st);
    case TF_DOWN: return launch<TF_DOWN>(a, st);
    case TF_DH: return launch<TF_DH>(a, st);
    case TF_DX: return launch<TF_DX>(a, st);
    case TF_DW: {
      TrainArgs b = a;
      if (a.slot_token && a.P) {
        gather_kernel<<<(unsigned)(((long long)a.P * (a.H / 8) + THR - 1) / THR), THR, 0, st>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        b.x = a.xg;
        b.slot_token = nullptr;
      }
      return launch<TF_DW>(b, st);
    }
  }
  return hipErrorInvalidValue;
}

}  // namespace moe
