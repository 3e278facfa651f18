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
// replicated so that the 32 lanes an LDS cycle serves have their own banks (32
// copies of a 4-byte entry).  An entry's address is byte << 8 | the lane's
// copy, which one v_perm_b32 builds straight from the loaded dword; the other
// half of each 256-byte table row holds the workgroup's own data (lds_half).
//  * int4: the entry is the pair q - 8 as bf16, exact, and meets the bf16
//    activations as they are;
//  * NF4: the entry is the pair of levels as fp16, each rounded once (2^-11
//    of its value at most; bf16's 2^-8 would show beside the output's
//    rounding, and a second bf16 term would double the reads and products);
//  * MXFP4: E2M1 values are exact in fp16 and gfx950 converts them, two per
//    instruction, with no table.
// The fp16 formats need activations in fp16's range: see RowScale.
#pragma once

#include "gnf4_internal.h"

namespace gnf4 {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

enum class W4 { kNf4, kMx4, kInt4 };

constexpr int kStep = 128;          // K per step
constexpr int kLutBytes = 64 * 1024;

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, (half2v{(_Float16)lo, (_Float16)hi}));
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

// Byte address of the i-th 4-byte word kept in the table rows' second halves.
__device__ __forceinline__ int lds_half(int i) { return (i >> 5) * 256 + 128 + (i & 31) * 4; }

// The decode table, filled by the whole workgroup (a barrier must follow).
// Thread t writes half of entry t / 2.  decode8 reads it at LDS address 0: it
// is the first thing of the workgroup's dynamic LDS, and its kernels have no
// static LDS.
template <W4 F>
__device__ __forceinline__ void fill_lut(char* lut) {
  if constexpr (F != W4::kMx4) {
    for (int t = threadIdx.x; t < 512; t += blockDim.x) {
      const int b = t >> 1, q = t & 1;
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
        const uint32_t p = pack_f16x2(l0, l1);
        v = u32x4{p, p, p, p};
      }
      u32x4* row = reinterpret_cast<u32x4*>(lut + b * 256 + q * 64);
#pragma unroll
      for (int j = 0; j < 4; ++j) row[(j + b) & 3] = v;
    }
  }
}

// Eight codes of one dword as an MFMA operand, in k order: bf16 for int4,
// fp16 for the others.
template <W4 F>
__device__ __forceinline__ u32x4 decode8(uint32_t w, uint32_t copy) {
  if constexpr (F == W4::kMx4) {
    const half2v p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0);
    const half2v p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1);
    const half2v p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2);
    const half2v p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3);
    return u32x4{__builtin_bit_cast(uint32_t, p0), __builtin_bit_cast(uint32_t, p1),
                 __builtin_bit_cast(uint32_t, p2), __builtin_bit_cast(uint32_t, p3)};
  } else {
    // address: the byte in bits 8..15, this lane's copy in bits 0..7 (the
    // table lies at LDS address 0)
    const auto at = [](uint32_t addr) {
      return *(const __attribute__((address_space(3))) uint32_t*)addr;
    };
    return u32x4{at(__builtin_amdgcn_perm(w, copy, 0x0c0c0400u)),
                 at(__builtin_amdgcn_perm(w, copy, 0x0c0c0500u)),
                 at(__builtin_amdgcn_perm(w, copy, 0x0c0c0600u)),
                 at(__builtin_amdgcn_perm(w, copy, 0x0c0c0700u))};
  }
}

// This lane's copy of the table entries (the low address byte).
__device__ __forceinline__ uint32_t lut_copy(int lane) { return (uint32_t)(lane & 31) * 4u; }

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

// a: 16 activation rows, b: 16 weight rows; lane l holds 8 k of row l % 16.
template <W4 F>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (F == W4::kInt4)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a),
                                                  __builtin_bit_cast(half8, b), c, 0, 0, 0);
}

// Activations as fp16: a row's values are multiplied by the power of two that
// puts the largest of them in [2^14, 2^15) (bf16 values within 2^28 of it then
// convert exactly, fp32 ones keep 11 bits) and the sums by its inverse.
struct RowScale {
  int exp;  // the largest value's exponent field, biased
  // Powers of two within fp32's normal range: a row of zeros or of the
  // smallest numbers stops at 2^126, one with an infinity scales it to itself.
  __device__ __forceinline__ float up() const {
    return __uint_as_float((uint32_t)(254 - down_field()) << 23);
  }
  __device__ __forceinline__ float down() const {
    return __uint_as_float((uint32_t)down_field() << 23);
  }
  // 2^(exp - 127 - 14) as an exponent field
  __device__ __forceinline__ int down_field() const { return min(max(exp - 14, 1), 253); }
};

// A row's scales of one step, and its zero points (bytes) where the format has
// them.
template <int B, typename S, bool ZP>
struct ScaleWord {
  static constexpr int kBlocks = kStep / B;
  static constexpr int kWords = (kBlocks * (int)sizeof(S) + 3) / 4;
  uint32_t v[kWords + (ZP ? 1 : 0)];
  __device__ __forceinline__ float at(int b) const {
    if constexpr (sizeof(S) == 4) return __uint_as_float(v[b]);
    if constexpr (sizeof(S) == 2)
      return __uint_as_float((b & 1) ? v[b >> 1] & 0xffff0000u : v[b >> 1] << 16);
    return e8m0_f32((v[0] >> (8 * b)) & 255u);
  }
  __device__ __forceinline__ int zero(int b) const { return (int)(v[kWords] >> (8 * b)) & 255; }
};

// Where the scales of step c start in a row: early enough to end with the row.
template <int B>
__device__ __forceinline__ int scales_first(int c, int blocks) {
  return min(c * (kStep / B), max(blocks - kStep / B, 0));
}

// N neighbouring elements of E bytes, whatever their alignment, as words.
template <int N, int E>
__device__ __forceinline__ void load_run(const void* p, uint32_t* v) {
  if constexpr (N * E == 1) {
    v[0] = *static_cast<const uint8_t*>(p);
  } else if constexpr (N * E == 2) {
    struct __attribute__((packed, aligned(E))) Raw {
      uint16_t v;
    };
    v[0] = static_cast<const Raw*>(p)->v;
  } else {
    struct __attribute__((packed, aligned(E))) Raw {
      uint32_t v[N * E / 4];
    };
    const Raw r = *static_cast<const Raw*>(p);
#pragma unroll
    for (int i = 0; i < N * E / 4; ++i) v[i] = r.v[i];
  }
}

// A row's scales (and zero points) from element `at` on.  SHORT: the row may
// have fewer blocks than a step; then one load per block it has.
template <int B, typename S, bool ZP, bool SHORT>
__device__ __forceinline__ void load_scales(const S* scales, const uint8_t* zeros, uint32_t at,
                                            int blocks, ScaleWord<B, S, ZP>& w) {
  typedef ScaleWord<B, S, ZP> W;
  constexpr int N = W::kBlocks;
  if (SHORT && blocks < N) {
#pragma unroll
    for (int i = 0; i < W::kWords + (ZP ? 1 : 0); ++i) w.v[i] = 0u;
#pragma unroll
    for (int b = 0; b < N - 1; ++b) {
      if (b >= blocks) break;
      uint32_t e;
      load_run<1, (int)sizeof(S)>(scales + at + b, &e);
      w.v[b * sizeof(S) / 4] |= e << (b * sizeof(S) % 4 * 8);
      if constexpr (ZP) w.v[W::kWords] |= (uint32_t)zeros[at + b] << (8 * b);
    }
    return;
  }
  load_run<N, (int)sizeof(S)>(reinterpret_cast<const char*>(scales) + at * (uint32_t)sizeof(S), w.v);
  if constexpr (ZP) load_run<N, 1>(zeros + at, w.v + W::kWords);
}
// The words moved to step c's first block; what lies past the row's end becomes
// zero or a block of the row's (its activations are zero).
template <int B, typename S, bool ZP>
__device__ __forceinline__ void align_scales(ScaleWord<B, S, ZP>& w, int c, int blocks) {
  typedef ScaleWord<B, S, ZP> W;
  constexpr int N = W::kBlocks;
  if constexpr (N > 1) {
    const int late = c * N - scales_first<B>(c, blocks);  // 0 but in a row's last step
    if constexpr (sizeof(S) == 4) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int l = 1; l < N; ++l) w.v[i] = late == l ? w.v[min(i + l, N - 1)] : w.v[i];
      }
    } else if constexpr (W::kWords == 2) {
      const uint64_t v = (((uint64_t)w.v[1] << 32) | w.v[0]) >> (16 * late);
      w.v[0] = (uint32_t)v;
      w.v[1] = (uint32_t)(v >> 32);
    } else {
      w.v[0] >>= late * (int)sizeof(S) * 8;
    }
    if constexpr (ZP) w.v[W::kWords] >>= 8 * late;
  }
}

// The 16 bytes of step c of the rows at codes + coff (coff includes the lane
// group's 16 bytes).  A row has kb bytes; past its end a lane reads the step's
// first bytes again (the activations there are zero).  Where `mask` is zero all
// lanes read the step's first bytes of the first row.
__device__ __forceinline__ u32x4 load_codes(const uint8_t* codes, int c, uint32_t coff, int g,
                                            int kb, uint32_t mask = ~0u) {
  const uint32_t co = (c * (kStep / 2) + g * 16 < kb ? coff : coff - (uint32_t)(g * 16)) & mask;
  return __builtin_nontemporal_load(
      reinterpret_cast<const u32x4*>(codes + c * (kStep / 2) + co));
}

// acc += (activations of the step) . (weights of the step)^T.
template <W4 F, int B, typename S, bool ZP>
__device__ __forceinline__ f32x4 step_mac(u32x4 d, const ScaleWord<B, S, ZP>& scale,
                                          const u32x4 (&x)[4], uint32_t copy, f32x4 acc) {
  arrange<B>(d);
  constexpr int kPer = B / 32;  // MFMAs of 32 codes per block
#pragma unroll
  for (int b = 0; b < kStep / B; ++b) {
    f32x4 p = {0.0f, 0.0f, 0.0f, 0.0f};
    uint32_t z = 0u;
    if constexpr (ZP) z = pack_bf16x2((float)(8 - scale.zero(b)), (float)(8 - scale.zero(b)));
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = b * kPer + j;
      p = mfma16<F>(x[i], decode8<F>(d[i], copy), p);
      // the codes' pairs are q - 8: a zero point adds (8 - z) times the sum of
      // the activations, both exact in bf16
      if constexpr (ZP) p = mfma16<F>(x[i], u32x4{z, z, z, z}, p);
    }
    const float s = scale.at(b);
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[r] = fmaf(s, p[r], acc[r]);
  }
  return acc;
}

}  // namespace gnf4
