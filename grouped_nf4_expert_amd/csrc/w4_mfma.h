// 4-bit weights against a few activation rows on the matrix cores: the pieces
// shared by the int4 linear and the few-token expert layer.
//
// A wavefront holds 16 weight rows and walks K in steps of 128.  In a step
// lane l owns weight row l % 16 and the 16 bytes (32 codes) of lane group
// g = l / 16: one 16-byte load per lane, 64 contiguous bytes per row.  The
// codes become bf16 operands of v_mfma_f32_16x16x32_bf16 (weights as B, 16
// activation rows as A): the matrix core does the multiply-adds of up to 16
// rows for the price of one, so the vector ALU only decodes, and the output's
// lane l holds column l % 16 for rows 4 (l / 16) + 0..3, so a lane needs the
// scales of its own weight row only.
//
// A scale covers a block of B = 32, 64 or 128 codes of a row, and one MFMA
// sums 32 codes taken from four lanes, so the four lanes must hold codes of
// one block.  Every lane's 16 bytes lie in one 128-code block as loaded; for
// smaller blocks v_permlane32_swap and v_permlane16_swap exchange dwords
// between lane groups (2 or 4 instructions per 32 codes) until each register
// holds one block.  Where a lane's codes then come from (k_of) is where the
// activation fragment is read, so both operands agree.  The block's fp32 MFMA
// sum is multiplied by the block's scale in fp32 and added to the running sum:
// no product of a code and a scale is ever rounded.
//
// Decode: one LDS read per byte (two codes) from a table of all 256 bytes,
// replicated so that every lane has its own banks (64 copies of a 4-byte
// entry, 32 of an 8-byte one: 64 KB).  An entry's address is byte << 8 | the
// lane's copy, which one v_perm_b32 builds straight from the loaded dword.
//  * int4: the entry is the pair q - 8 as bf16, exact;
//  * NF4: a level is not a bf16 number, so the entry is two pairs, the
//    level rounded to bf16 and the rest rounded to bf16 (together within
//    2^-17 of the level), and the step issues two MFMAs;
//  * MXFP4: E2M1 values are exact in bf16 and gfx950 converts them, two per
//    instruction, with no table.
#pragma once

#include "gnf4_internal.h"

namespace gnf4 {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

enum class W4 { kNf4, kMx4, kInt4 };

constexpr int kStep = 128;          // K per step
constexpr int kLutBytes = 64 * 1024;

__device__ __forceinline__ int lane_id() {
  return (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  return (uint32_t)f32_to_bf16(lo) | ((uint32_t)f32_to_bf16(hi) << 16);
}

// E8M0 scale byte -> 2^(s - 127) in fp32 (2^-127 is a subnormal); 0xFF is NaN.
__device__ __forceinline__ float e8m0_f32(uint32_t s) {
  const uint32_t bits = s == 0u ? 0x00400000u : s == 255u ? 0x7fc00000u : s << 23;
  return __uint_as_float(bits);
}

__device__ __forceinline__ float scale_f32(float s) { return s; }
__device__ __forceinline__ float scale_f32(uint16_t s) { return bf16_to_f32(s); }
__device__ __forceinline__ float scale_f32(uint8_t s) { return e8m0_f32(s); }

// The decode table, filled by the whole workgroup (a barrier must follow).
// Thread t writes a quarter of entry t / 4.
template <W4 F>
__device__ __forceinline__ void fill_lut(char* lut) {
  if constexpr (F != W4::kMx4) {
    for (int t = threadIdx.x; t < 1024; t += blockDim.x) {
      const int b = t >> 2, q = t & 3;
      const int c0 = b >> 4, c1 = b & 15;  // first element in the high nibble
      u32x4 v;
      if constexpr (F == W4::kInt4) {
        const uint32_t p = pack_bf16x2((float)(c0 - 8), (float)(c1 - 8));
        v = u32x4{p, p, p, p};
      } else {
        float l0 = nf4_level(0), l1 = l0;
#pragma unroll
        for (int i = 1; i < 16; ++i) {
          l0 = c0 == i ? nf4_level(i) : l0;
          l1 = c1 == i ? nf4_level(i) : l1;
        }
        const uint32_t hi = pack_bf16x2(l0, l1);
        const uint32_t lo = pack_bf16x2(l0 - __uint_as_float(hi << 16),
                                        l1 - __uint_as_float(hi & 0xffff0000u));
        v = u32x4{hi, lo, hi, lo};
      }
      u32x4* row = reinterpret_cast<u32x4*>(lut + b * 256 + q * 64);
#pragma unroll
      for (int j = 0; j < 4; ++j) row[(j + b) & 3] = v;
    }
  }
}

template <W4 F>
struct Operand {
  bf16x8 hi;
};
template <>
struct Operand<W4::kNf4> {
  bf16x8 hi, lo;
};

// Eight codes of one dword as MFMA operands, in k order.
template <W4 F>
__device__ __forceinline__ Operand<F> decode8(uint32_t w, const char* lut, uint32_t copy) {
  Operand<F> o;
  if constexpr (F == W4::kMx4) {
    const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 0);
    const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 1);
    const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 2);
    const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 3);
    const u32x4 v = {__builtin_bit_cast(uint32_t, p0), __builtin_bit_cast(uint32_t, p1),
                     __builtin_bit_cast(uint32_t, p2), __builtin_bit_cast(uint32_t, p3)};
    o.hi = __builtin_bit_cast(bf16x8, v);
  } else {
    // address: the byte in bits 8..15, this lane's copy in bits 0..7
    const uint32_t a0 = __builtin_amdgcn_perm(w, copy, 0x0c0c0400u);
    const uint32_t a1 = __builtin_amdgcn_perm(w, copy, 0x0c0c0500u);
    const uint32_t a2 = __builtin_amdgcn_perm(w, copy, 0x0c0c0600u);
    const uint32_t a3 = __builtin_amdgcn_perm(w, copy, 0x0c0c0700u);
    if constexpr (F == W4::kInt4) {
      const u32x4 v = {*reinterpret_cast<const uint32_t*>(lut + a0),
                       *reinterpret_cast<const uint32_t*>(lut + a1),
                       *reinterpret_cast<const uint32_t*>(lut + a2),
                       *reinterpret_cast<const uint32_t*>(lut + a3)};
      o.hi = __builtin_bit_cast(bf16x8, v);
    } else {
      const u32x2 e0 = *reinterpret_cast<const u32x2*>(lut + a0);
      const u32x2 e1 = *reinterpret_cast<const u32x2*>(lut + a1);
      const u32x2 e2 = *reinterpret_cast<const u32x2*>(lut + a2);
      const u32x2 e3 = *reinterpret_cast<const u32x2*>(lut + a3);
      o.hi = __builtin_bit_cast(bf16x8, (u32x4{e0.x, e1.x, e2.x, e3.x}));
      o.lo = __builtin_bit_cast(bf16x8, (u32x4{e0.y, e1.y, e2.y, e3.y}));
    }
  }
  return o;
}

// This lane's copy of the table entries (the low address byte).
template <W4 F>
__device__ __forceinline__ uint32_t lut_copy(int lane) {
  return F == W4::kInt4 ? (uint32_t)lane * 4u : (uint32_t)(lane & 31) * 8u;
}

// Offset within a step of the eight codes that register i (0..3) of lane
// group g holds after arrange<B>.
template <int B>
__device__ __forceinline__ int k_of(int g, int i) {
  if constexpr (B == 128) return g * 32 + i * 8;
  if constexpr (B == 64) return (i >> 1) * 64 + (g & 1) * 32 + (g >> 1) * 16 + (i & 1) * 8;
  return i * 32 + g * 8;
}

// Exchanges dwords between lane groups so that register i lies in block
// i / (B / 32) of the step.  permlane32_swap(a, b): a's upper 32 lanes with
// b's lower 32; permlane16_swap(a, b): a's odd lane groups with b's even.
template <int B>
__device__ __forceinline__ void arrange(u32x4& d) {
  if constexpr (B != 128) {
    const auto p = __builtin_amdgcn_permlane32_swap(d.x, d.z, false, false);
    const auto q = __builtin_amdgcn_permlane32_swap(d.y, d.w, false, false);
    if constexpr (B == 64) {
      d = u32x4{p[0], q[0], p[1], q[1]};
    } else {
      const auto r = __builtin_amdgcn_permlane16_swap(p[0], q[0], false, false);
      const auto s = __builtin_amdgcn_permlane16_swap(p[1], q[1], false, false);
      d = u32x4{r[0], r[1], s[0], s[1]};
    }
  }
}

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// One lane's weight row: codes, scales and (int4) zero points, all of the
// row's K.
template <typename S>
struct WeightRow {
  const uint8_t* codes;
  const S* scales;
  const uint8_t* zeros;
};

// What one step reads of a weight row.
template <int B, typename S>
struct StepData {
  u32x4 codes;
  S scale[kStep / B];
  uint8_t zero[kStep / B];
};

// Step c of a row of K codes.  Past the end of the row a lane reads the row's
// start again and the last block's scale: the activations there are zero.
template <int B, bool ZP, typename S>
__device__ __forceinline__ void load_step(const WeightRow<S>& w, int c, int g, int K,
                                          StepData<B, S>& d) {
  const int off = c * (kStep / 2) + g * 16;
  d.codes = *reinterpret_cast<const u32x4*>(w.codes + (off < K / 2 ? off : 0));
#pragma unroll
  for (int b = 0; b < kStep / B; ++b) {
    const int blk = min(c * (kStep / B) + b, K / B - 1);
    d.scale[b] = w.scales[blk];
    if constexpr (ZP) d.zero[b] = w.zeros[blk];
  }
}

// Eight activations of one row at k, or zeros past the row's end.
__device__ __forceinline__ bf16x8 load_frag(const uint16_t* row, int k, int K) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (k < K) v = *reinterpret_cast<const u32x4*>(row + k);
  return __builtin_bit_cast(bf16x8, v);
}

// acc += (activations of the step) . (weights of the step)^T, XP operands per
// activation (1, or 2 where the activation is the sum of two bf16 numbers;
// the product of the two low parts is below fp32's last bit and left out).
template <W4 F, int B, bool ZP, int XP, typename S>
__device__ __forceinline__ f32x4 step_mac(StepData<B, S> d, const bf16x8 (&x)[XP][4],
                                          const char* lut, uint32_t copy, f32x4 acc) {
  arrange<B>(d.codes);
  constexpr int kPer = B / 32;  // MFMAs of 32 codes per block
#pragma unroll
  for (int b = 0; b < kStep / B; ++b) {
    f32x4 p = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = b * kPer + j;
      const Operand<F> o = decode8<F>(d.codes[i], lut, copy);
      if constexpr (F == W4::kNf4) p = mfma16(x[0][i], o.lo, p);
      if constexpr (XP == 2) p = mfma16(x[1][i], o.hi, p);
      p = mfma16(x[0][i], o.hi, p);
      if constexpr (ZP) {  // (q - 8) - (z - 8), both exact in bf16
        const uint32_t z = pack_bf16x2((float)(8 - (int)d.zero[b]), (float)(8 - (int)d.zero[b]));
        p = mfma16(x[0][i], __builtin_bit_cast(bf16x8, (u32x4{z, z, z, z})), p);
      }
    }
    const float s = scale_f32(d.scale[b]);
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[r] = fmaf(s, p[r], acc[r]);
  }
  return acc;
}

}  // namespace gnf4
