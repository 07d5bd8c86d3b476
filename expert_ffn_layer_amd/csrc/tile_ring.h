// What the tiled products of 16-bit numbers share: an operand's tile in LDS, its way there from global memory and from
// there to the matrix cores, and the order of the loads of a ring of slots.
#pragma once
#include "common.h"

namespace moe {

namespace {

constexpr int BK = 64;     // reduction elements per step: 128 bytes of a row, a whole cache line
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

}  // namespace

}  // namespace moe
