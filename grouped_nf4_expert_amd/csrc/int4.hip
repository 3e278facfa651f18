// int4 weights with group scales: the packer and the linear layer over it.

#include "w4_tiles.h"

namespace gnf4 {
namespace {

// ---------------------------------------------------------------- int4_pack

constexpr int kPackThreads = 256;

__device__ __forceinline__ float round_scale(float s, float) { return s; }
__device__ __forceinline__ uint16_t round_scale(float s, uint16_t) { return f32_to_bf16(s); }

// 8 consecutive weights as fp32
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  const u32x4 d = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = bf16_to_f32(d[j] & 0xffffu);
    v[2 * j + 1] = bf16_to_f32(d[j] >> 16);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const f32x4 a = reinterpret_cast<const f32x4*>(p)[0];
  const f32x4 b = reinterpret_cast<const f32x4*>(p)[1];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = a[j];
    v[4 + j] = b[j];
  }
}

// The code of w: the number of midpoints (m + 1/2 - z) s below it, m = 0..14,
// which is the nearest level, ties to the lower code.  An approximate quotient
// finds it to within one (its error is far below half a step), and the two
// midpoints beside the guess settle it: their products are exact in fp64 (a
// scale has 24 bits, a midpoint 5), so the comparisons are.  A NaN lies above
// nothing; among infinite midpoints every value but -inf is above the negative
// ones.
__device__ __forceinline__ int int4_code(float w, double s, double inv_s, int z) {
  const double x = (double)w, zz = (double)z;
  const double q = ceil(x * inv_s + zz - 0.5);
  const double c = fmin(fmax(q, 0.0), 15.0);
  int n = (int)c;
  n += n < 15 && x > (c + 0.5 - zz) * s ? 1 : 0;
  n -= n > 0 && n == (int)c && !(x > (c - 0.5 - zz) * s) ? 1 : 0;
  if (s == INFINITY) n = x > -INFINITY ? z : 0;
  return s == 0.0 ? z : n;
}

// Eight weights per thread, G / 8 neighbouring lanes per group.  Bound by HBM
// once the matrix is large: 5760 x 2880 fp32 weights with zero points, 77 MB, 21
// us from cold caches, 3.7 TB/s (28 us with fifteen comparisons per weight).
template <typename WT, typename S, int G, bool ZP>
__global__ __launch_bounds__(kPackThreads) void int4_pack_kernel(const WT* __restrict__ w,
                                                                 int64_t n8,
                                                                 uint8_t* __restrict__ packed,
                                                                 S* __restrict__ scales,
                                                                 uint8_t* __restrict__ zeros) {
  const int64_t stride = (int64_t)gridDim.x * kPackThreads;
  for (int64_t i = (int64_t)blockIdx.x * kPackThreads + threadIdx.x; i < n8; i += stride) {
    float v[8];
    load8(w + i * 8, v);
    float hi = 0.0f, lo = 0.0f;  // of the group's range with zero in it; symmetric: hi = max |w|
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      hi = fmaxf(hi, ZP ? v[j] : fabsf(v[j]));
      lo = fmaxf(lo, -v[j]);
    }
#pragma unroll
    for (int o = 1; o < G / 8; o *= 2) {
      hi = fmaxf(hi, __shfl_xor(hi, o, kWave));
      if constexpr (ZP) lo = fmaxf(lo, __shfl_xor(lo, o, kWave));
    }
    const float s32 = ZP ? hi / 15.0f + lo / 15.0f : hi / 7.0f;
    const S stored = round_scale(s32, S{});
    const double s = (double)scale_f32(stored), inv_s = __builtin_amdgcn_rcp(s);
    const int z = ZP ? int4_code(lo, s, inv_s, 0) : 8;
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      // byte j / 2, the first of the two in the high nibble
      word |= (uint32_t)int4_code(v[j], s, inv_s, z) << ((j >> 1) * 8 + ((j & 1) ? 0 : 4));
    reinterpret_cast<uint32_t*>(packed)[i] = word;
    if (i % (G / 8) == 0) {
      scales[i / (G / 8)] = stored;
      if constexpr (ZP) zeros[i / (G / 8)] = (uint8_t)z;
    }
  }
}

template <typename WT, typename S, int G>
void launch_pack_g(const Int4PackArgs& a, unsigned grid, hipStream_t stream) {
  const WT* w = static_cast<const WT*>(a.w);
  S* sc = static_cast<S*>(a.scales);
  const int64_t n8 = a.n_weights / 8;
  if (a.zeros)
    hipLaunchKernelGGL((int4_pack_kernel<WT, S, G, true>), dim3(grid), dim3(kPackThreads), 0,
                       stream, w, n8, a.packed, sc, a.zeros);
  else
    hipLaunchKernelGGL((int4_pack_kernel<WT, S, G, false>), dim3(grid), dim3(kPackThreads), 0,
                       stream, w, n8, a.packed, sc, a.zeros);
}

template <typename WT, typename S>
void launch_pack_s(const Int4PackArgs& a, unsigned grid, hipStream_t stream) {
  if (a.group == 32)
    launch_pack_g<WT, S, 32>(a, grid, stream);
  else if (a.group == 64)
    launch_pack_g<WT, S, 64>(a, grid, stream);
  else
    launch_pack_g<WT, S, 128>(a, grid, stream);
}

// -------------------------------------------------------------- int4_linear
//
// Up to 16 rows of activations: the weight stream bounds it, and the loop of
// w4_tiles.h runs over one entry (the rows) and the matrix's tiles of 16 U rows.
// 1 x 65537 x 8192 takes 55 us, 5.0 TB/s.  Matrices of a few megabytes are bound
// by the chain of a launch (activations and scales, first weights, sums): 1 x
// 2048 x 2048 5.0 us, 13 x 4096 x 7168 13 us.

template <typename S, int U>
struct Rows {
  typedef RawBf16 Raw;
  static constexpr bool kKeepRaw = true;
  static constexpr int kRows = 16 * U;
  const Int4LinearArgs& a;
  const uint8_t* codes;
  const S* scales;
  const uint8_t* zeros;
  const uint16_t* x;
  static constexpr size_t expert_rows = 0;
  __device__ uint32_t entry(int) const { return make_entry(0, 0, a.M); }
  __device__ int row(int r) const { return r; }
  __device__ int weight_row(int r) const { return min(r, a.N - 1); }
  // the last item ends with the matrix, over rows of the item before it
  __device__ int first_row(int item) const { return min(item * kRows, max(a.N - kRows, 0)); }
  __device__ void finish(int team, int log_wk, int, int item, const char* sums) const {
    const int n0 = first_row(item);
    for (int i = threadIdx.x & ((64 << log_wk) - 1); i < U * 256; i += 64 << log_wk) {
      const int h = i >> 8, o = i & 255;
      const int n = min(n0 + h * 16 + tile_col(o), a.N - 1);
      float y = team_sum<U>(sums, team, log_wk, h, o);
      if (a.bias) y += bf16_to_f32(a.bias[n]);
      a.y[(size_t)min(tile_row(o), a.M - 1) * a.N + n] = f32_to_bf16(y);
    }
  }
};

template <int B, typename S, bool ZP, int NST, int G, int U>
__global__ __launch_bounds__(kThreads, waves_per_simd(NST, G)) void int4_rows_kernel(
    Int4LinearArgs a, ItemGrid ig) {
  extern __shared__ __align__(256) char lut[];
  fill_lut<W4::kInt4>(lut);
  lds_barrier();
  const Rows<S, U> p = {a, a.packed, static_cast<const S*>(a.scales), a.zeros, a.x};
  expert_tiles<W4::kInt4, B, S, ZP, NST, G, U>(p, ig, 1, lut, lut + kLutBytes);
}

template <int B, typename S, bool ZP, int NST, int G, int U>
void launch_rows_n(const Int4LinearArgs& a, const Launch& l, hipStream_t stream) {
  const int lds = kLutBytes + 2 * scale_bytes<ScaleWord<B, S, ZP>, U>(NST);
  hipLaunchKernelGGL((int4_rows_kernel<B, S, ZP, NST, G, U>), dim3(l.grid), dim3(kThreads), lds,
                     stream, a, l.ig);
}

template <int B, typename S, bool ZP, int U>
void launch_rows_u(const Int4LinearArgs& a, const Launch& l, hipStream_t stream) {
  if constexpr (U == 1) {
    if (l.group > 1) return launch_rows_n<B, S, ZP, 4, kGroup, U>(a, l, stream);
    if (l.nst > 7) return launch_rows_n<B, S, ZP, 8, 1, U>(a, l, stream);
    if (l.nst > 6) return launch_rows_n<B, S, ZP, 7, 1, U>(a, l, stream);
  }
  if (l.nst == 1)
    launch_rows_n<B, S, ZP, 1, 1, U>(a, l, stream);
  else if (l.nst == 2)
    launch_rows_n<B, S, ZP, 2, 1, U>(a, l, stream);
  else if (l.nst == 3)
    launch_rows_n<B, S, ZP, 3, 1, U>(a, l, stream);
  else if (l.nst == 4)
    launch_rows_n<B, S, ZP, 4, 1, U>(a, l, stream);
  else
    launch_rows_n<B, S, ZP, 6, 1, U>(a, l, stream);
}

// Items of two column tiles share a barrier and its sums; single ones where
// they spread the columns over the CUs at least a tenth better, and for the
// longest rows, whose activations leave no registers for two.
template <int B, typename S, bool ZP>
void launch_rows(const Int4LinearArgs& a, hipStream_t stream) {
  const auto plan = [&](int u) {
    const int tiles = (a.N + 16 * u - 1) / (16 * u);
    Launch l = plan_launch(1, 1, tiles, a.K, 8);
    l.ig.tiles = (tiles + l.group - 1) / l.group * l.group;
    return l;
  };
  const Launch two = plan(2), one = plan(1);
  if (one.cost * 10 < two.cost * 2 * 9 || one.group > 1 || one.nst > 6)
    launch_rows_u<B, S, ZP, 1>(a, one, stream);
  else
    launch_rows_u<B, S, ZP, 2>(a, two, stream);
}

// More rows, few tiles: a wavefront holds 32 rows x 64 columns of the product, so
// a decoded operand serves two products and an activation fragment four, and the
// eight wavefronts of a workgroup split the steps of K; their sums meet in LDS,
// in wavefront order.  K is a step or more.
constexpr int kGemmCols = 4;  // column tiles of 16

template <int B, typename S, bool ZP>
__global__ __launch_bounds__(kThreads) void int4_gemm_kernel(Int4LinearArgs a) {
  typedef ScaleWord<B, S, ZP> Scale;
  constexpr int RT = 2;
  extern __shared__ __align__(256) char lut[];
  fill_lut<W4::kInt4>(lut);
  const int wave = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int g = lane >> 4, col = lane & 15;
  const int n0 = blockIdx.x * 64, m0 = blockIdx.y * 16 * RT;
  const int kb = a.K / 2, blocks = a.K / B, steps = (a.K + kStep - 1) / kStep;
  const uint32_t copy = lut_copy(lane);
  size_t wrow[kGemmCols];
#pragma unroll
  for (int t = 0; t < kGemmCols; ++t) wrow[t] = min(n0 + t * 16 + col, a.N - 1);
  const uint16_t* xrow[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) xrow[t] = a.x + (size_t)min(m0 + t * 16 + col, a.M - 1) * a.K;
  f32x4 acc[kGemmCols][RT];
#pragma unroll
  for (int t = 0; t < kGemmCols; ++t)
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[t][r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  u32x4 w[kGemmCols], wn[kGemmCols];
  Scale sc[kGemmCols], scn[kGemmCols];
  const auto load = [&](int c, u32x4 (&d)[kGemmCols], Scale (&s)[kGemmCols]) {
#pragma unroll
    for (int t = 0; t < kGemmCols; ++t) {
      d[t] = load_codes(a.packed + wrow[t] * kb, c, (uint32_t)(g * 16), g, kb);
      load_scales<B, S, ZP, false>(static_cast<const S*>(a.scales) + wrow[t] * blocks,
                                   ZP ? a.zeros + wrow[t] * blocks : nullptr,
                                   (uint32_t)scales_first<B>(c, blocks), blocks, s[t]);
    }
  };
  load(min(wave, steps - 1), wn, scn);
  lds_barrier();
  for (int c = wave; c < steps; c += kWaves) {
#pragma unroll
    for (int t = 0; t < kGemmCols; ++t) {
      w[t] = wn[t];
      sc[t] = scn[t];
    }
    u32x4 x[RT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = c * kStep + k_of<B>(g, i);
        x[r][i] = *reinterpret_cast<const u32x4*>(xrow[r] + (k < a.K ? k : 0));
      }
    load(min(c + kWaves, steps - 1), wn, scn);
    if ((c + 1) * kStep > a.K)  // the row's end: zero activations past it
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c * kStep + k_of<B>(g, i) >= a.K) x[r][i] = u32x4{0u, 0u, 0u, 0u};
    constexpr int kPer = B / 32;
    // the activations' sums over each block, for the zero points
    f32x4 sum[ZP ? kStep / B : 1][ZP ? RT : 1];
    if constexpr (ZP) {
#pragma unroll
      for (int b = 0; b < kStep / B; ++b)
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          f32x4 p = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int j = 0; j < kPer; ++j)
            p = mfma16<W4::kInt4>(x[r][b * kPer + j],
                                  u32x4{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u}, p);
          sum[b][r] = p;
        }
    }
#pragma unroll
    for (int t = 0; t < kGemmCols; ++t) {
      align_scales<B, S, ZP>(sc[t], c, blocks);
      arrange<B>(w[t]);
#pragma unroll
      for (int b = 0; b < kStep / B; ++b) {
        f32x4 p[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) p[r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const u32x4 d = decode8<W4::kInt4>(w[t][b * kPer + j], copy);
#pragma unroll
          for (int r = 0; r < RT; ++r) p[r] = mfma16<W4::kInt4>(x[r][b * kPer + j], d, p[r]);
        }
        const float s = sc[t].at(b);
        const float z = ZP ? (float)(8 - sc[t].zero(b)) : 0.0f;
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if constexpr (ZP) p[r][q] = fmaf(z, sum[b][r][q], p[r][q]);
            acc[t][r][q] = fmaf(s, p[r][q], acc[t][r][q]);
          }
      }
    }
  }
  lds_barrier();  // the table has been read; the sums take its place
  // one column tile at a time: [wave][row tile][register][lane]
  float* red = reinterpret_cast<float*>(lut);
#pragma unroll
  for (int t = 0; t < kGemmCols; ++t) {
    float* set = red + (t & 1) * (kWaves * RT * 256);
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int q = 0; q < 4; ++q) set[((wave * RT + r) * 4 + q) * kWave + lane] = acc[t][r][q];
    lds_barrier();
    for (int i = threadIdx.x; i < RT * 256; i += kThreads) {
      const int m = m0 + (i >> 8) * 16 + tile_row(i & 255), n = n0 + t * 16 + tile_col(i & 255);
      float y = 0.0f;
#pragma unroll
      for (int k = 0; k < kWaves; ++k) y += set[k * RT * 256 + i];
      if (m < a.M && n < a.N) {
        if (a.bias) y += bf16_to_f32(a.bias[n]);
        a.y[(size_t)m * a.N + n] = f32_to_bf16(y);
      }
    }
  }
}

// Enough rows and columns to fill the chip: a workgroup makes 16 RT rows x 128
// columns, a wavefront 16 RT x 32 over every other step of K (so two wavefronts
// share a SIMD).  The activations of a turn, two steps, lie in LDS, with their
// sums over each scale block where there are zero points; the weights of the
// turn after the next are in flight meanwhile.  Workgroups stay resident and walk
// the tiles.  SHORT: K is less than a step.
//
// 256 x 7168 x 2048 takes 23 us, 325 TFLOP/s.  Of a wavefront's cycles there 42%
// issue vector instructions (scales and zero points applied to fp32 block sums,
// addresses), 33% move LDS data and 16% are the matrix core's: with two
// wavefronts per SIMD they overlap only in part.
constexpr int kTileCols = 128;
constexpr int kTileRow = kStep * 2 + 16;  // bytes of a row's step: eight rows meet all banks

template <int B, typename S, bool ZP, int RT, bool SHORT>
__global__ __launch_bounds__(kThreads, kWaves / 4) void int4_tile_kernel(Int4LinearArgs a) {
  typedef ScaleWord<B, S, ZP> Scale;
  constexpr int kRows = 16 * RT, kBlocks = kStep / B, kPer = B / 32;
  constexpr int kXBytes = 2 * kRows * kTileRow;  // of a turn
  constexpr int kPerRow = kThreads / kRows;      // threads that stage a row
  constexpr int kPieces = 2 * kStep / 8 / kPerRow;  // 16-byte pieces of each
  extern __shared__ __align__(256) char lut[];
  char* xs = lut + kLutBytes;
  float* zs = reinterpret_cast<float*>(xs + 2 * kXBytes);  // [turn & 1][step][block][row]
  fill_lut<W4::kInt4>(lut);
  const int wave = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int g = lane >> 4, col = lane & 15;
  const int half = wave >> 2, nw = wave & 3;
  const int kb = a.K / 2, blocks = a.K / B, steps = (a.K + kStep - 1) / kStep;
  const int turns = (steps + 1) / 2;
  const uint32_t copy = lut_copy(lane);
  const int srow = threadIdx.x / kPerRow, spiece = threadIdx.x % kPerRow;
  const int mt = (a.M + kRows - 1) / kRows, nt = (a.N + kTileCols - 1) / kTileCols;
  // neighbouring workgroups go to different XCDs: the row tiles of a column
  // tile follow each other on one of them, and its L2 has the weights
  const int64_t total = (int64_t)((nt + 7) / 8 * 8) * mt;
  for (int64_t id = blockIdx.x; id < total; id += gridDim.x) {
    const int64_t q8 = id >> 3;
    const int64_t ct = q8 / mt * 8 + (id & 7);
    if (ct >= nt) continue;
    const int n0 = (int)ct * kTileCols + nw * 32, m0 = (int)(q8 % mt) * kRows;
    const uint8_t* codes[2];
    const S* scales[2];
    const uint8_t* zeros[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const size_t n = min(n0 + t * 16 + col, a.N - 1);
      codes[t] = a.packed + n * kb;
      scales[t] = static_cast<const S*>(a.scales) + n * blocks;
      zeros[t] = ZP ? a.zeros + n * blocks : nullptr;
    }
    const uint16_t* xrow = a.x + (size_t)min(m0 + srow, a.M - 1) * a.K;
    const auto load_w = [&](int turn, u32x4 (&w)[2], Scale (&sc)[2]) {
      const int c = min(2 * turn + half, steps - 1);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        w[t] = load_codes(codes[t], c, (uint32_t)(g * 16), g, kb);
        load_scales<B, S, ZP, SHORT>(scales[t], zeros[t], (uint32_t)scales_first<B>(c, blocks),
                                     blocks, sc[t]);
      }
    };
    u32x4 xr[kPieces];
    const auto load_x = [&](int turn) {
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        const int k = turn * 2 * kStep + (spiece + j * kPerRow) * 8;
        xr[j] = *reinterpret_cast<const u32x4*>(xrow + (k < a.K ? k : 0));
      }
    };
    const auto store_x = [&](int turn) {
      char* to = xs + (turn & 1) * kXBytes;
      float sum[kPieces];
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        const int p = spiece + j * kPerRow;
        if (turn * 2 * kStep + p * 8 >= a.K) xr[j] = u32x4{0u, 0u, 0u, 0u};
        *reinterpret_cast<u32x4*>(to + ((p >> 4) * kRows + srow) * kTileRow + (p & 15) * 16) = xr[j];
        if constexpr (ZP) {
          sum[j] = 0.0f;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            sum[j] += __uint_as_float(xr[j][i] << 16) + __uint_as_float(xr[j][i] & 0xffff0000u);
        }
      }
      if constexpr (ZP) {
        constexpr int kOwn = B / 8 > kPerRow ? B / 8 / kPerRow : 1;  // a block's pieces per thread
        constexpr int kLanes = B / 8 / kOwn;
#pragma unroll
        for (int j = 0; j < kPieces; j += kOwn) {
#pragma unroll
          for (int i = 1; i < kOwn; ++i) sum[j] += sum[j + i];
#pragma unroll
          for (int o = 1; o < kLanes; o *= 2) {  // the mirrors swap equal halves
            const uint32_t v = __float_as_uint(sum[j]);
            sum[j] += __uint_as_float(o == 1   ? dpp_u32<0xB1, 0xF>(0u, v)
                                      : o == 2 ? dpp_u32<0x4E, 0xF>(0u, v)
                                      : o == 4 ? dpp_u32<0x141, 0xF>(0u, v)
                                               : dpp_u32<0x140, 0xF>(0u, v));
          }
          const int p = spiece + j * kPerRow;
          if (spiece % kLanes == 0)
            zs[((turn & 1) * 2 * kBlocks + p / (B / 8)) * kRows + srow] = sum[j];
        }
      }
    };
    f32x4 acc[2][RT];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[t][r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    u32x4 w[2][2];
    Scale sc[2][2];
    load_x(0);
    load_w(0, w[0], sc[0]);
    load_w(1, w[1], sc[1]);
    lds_barrier();  // the sums of the tile before are read
    store_x(0);
    load_x(1);
    lds_barrier();
    const auto body = [&](int turn, u32x4 (&wt)[2], Scale (&st)[2]) {
      u32x4 d[2];
      Scale s[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        d[t] = wt[t];
        s[t] = st[t];
        arrange<B>(d[t]);
        align_scales<B, S, ZP>(s[t], min(2 * turn + half, steps - 1), blocks);
      }
      load_w(turn + 2, wt, st);
      const char* from = xs + (turn & 1) * kXBytes + (half * kRows + col) * kTileRow;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        f32x4 p[2][RT];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int r = 0; r < RT; ++r) p[t][r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int i = b * kPer + j;
          u32x4 x[RT];
#pragma unroll
          for (int r = 0; r < RT; ++r)
            x[r] = *reinterpret_cast<const u32x4*>(from + r * 16 * kTileRow + k_of<B>(g, i) * 2);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const u32x4 e = decode8<W4::kInt4>(d[t][i], copy);
#pragma unroll
            for (int r = 0; r < RT; ++r) p[t][r] = mfma16<W4::kInt4>(x[r], e, p[t][r]);
          }
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          f32x4 sum;
          if constexpr (ZP)
            sum = *reinterpret_cast<const f32x4*>(
                zs + (((turn & 1) * 2 + half) * kBlocks + b) * kRows + r * 16 + g * 4);
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              if constexpr (ZP) p[t][r][q] = fmaf((float)(8 - s[t].zero(b)), sum[q], p[t][r][q]);
              acc[t][r][q] = fmaf(s[t].at(b), p[t][r][q], acc[t][r][q]);
            }
        }
        if constexpr (ZP) __builtin_amdgcn_sched_barrier(0);  // registers: one block at a time
      }
      store_x(turn + 1);
      load_x(turn + 2);
      lds_barrier();
    };
    for (int turn = 0; turn < turns; turn += 2) {
      body(turn, w[0], sc[0]);
      if (turn + 1 < turns) body(turn + 1, w[1], sc[1]);
    }
    // the halves exchange a column tile each, where the activations were
    float* red = reinterpret_cast<float*>(xs) + lane;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        red[(((1 - half) * 4 + nw) * RT * 4 + r * 4 + q) * kWave] = half ? acc[0][r][q] : acc[1][r][q];
    lds_barrier();
    const int n = n0 + half * 16 + col;
    const float bias = a.bias ? bf16_to_f32(a.bias[min(n, a.N - 1)]) : 0.0f;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int m = m0 + r * 16 + g * 4 + q;
        const float y = (half ? acc[1][r][q] : acc[0][r][q]) +
                        red[((half * 4 + nw) * RT * 4 + r * 4 + q) * kWave];
        if (m < a.M && n < a.N) a.y[(size_t)m * a.N + n] = f32_to_bf16(y + bias);
      }
  }
}

template <int B, typename S, bool ZP, int RT, bool SHORT>
void launch_tile(const Int4LinearArgs& a, hipStream_t stream) {
  const int lds = kLutBytes + 2 * (2 * 16 * RT * kTileRow) +
                  (ZP ? 2 * 2 * (kStep / B) * 16 * RT * 4 : 0);
  const int64_t mt = (a.M + 16 * RT - 1) / (16 * RT);
  const int64_t nt = ((int64_t)a.N + kTileCols - 1) / kTileCols;
  const int64_t total = (nt + 7) / 8 * 8 * mt, cus = (device_cu_count() + 7) / 8 * 8;
  hipLaunchKernelGGL((int4_tile_kernel<B, S, ZP, RT, SHORT>), dim3((unsigned)(total < cus ? total : cus)),
                     dim3(kThreads), lds, stream, a);
}

template <int B, typename S, bool ZP>
void launch_gemm(const Int4LinearArgs& a, unsigned mt, unsigned nt, hipStream_t stream) {
  hipLaunchKernelGGL((int4_gemm_kernel<B, S, ZP>), dim3(nt, mt), dim3(kThreads), kLutBytes,
                     stream, a);
}

// Tiles of 32 x 64 with K split over the workgroup while there are no more of
// them than CUs (64 x 7168 x 2048 14 us against 23 with the larger tiles, 128 x
// 4096 x 7168 31 against 57); beyond that the larger tiles (256 x 7168 x 2048 22
// us against 51, 1024 x 2880 x 2880 55 against 89).  Blocks of 32 with zero points
// have the registers for 32 rows only.
template <int B, typename S, bool ZP>
void launch_linear_rt(const Int4LinearArgs& a, hipStream_t stream) {
  if (a.M <= 16) return launch_rows<B, S, ZP>(a, stream);
  const int64_t mt = (a.M + 31) / 32, nt = ((int64_t)a.N + 63) / 64;
  if (B < kStep && a.K < kStep) {
    if constexpr (B < kStep) launch_tile<B, S, ZP, 2, true>(a, stream);
  } else if (mt * nt <= device_cu_count()) {
    launch_gemm<B, S, ZP>(a, (unsigned)mt, (unsigned)nt, stream);
  } else {
    launch_tile<B, S, ZP, B == 32 && ZP ? 2 : 4, false>(a, stream);
  }
}

template <int B, typename S>
void launch_linear_zp(const Int4LinearArgs& a, hipStream_t stream) {
  if (a.zeros)
    launch_linear_rt<B, S, true>(a, stream);
  else
    launch_linear_rt<B, S, false>(a, stream);
}

template <typename S>
void launch_linear_b(const Int4LinearArgs& a, hipStream_t stream) {
  if (a.group == 32)
    launch_linear_zp<32, S>(a, stream);
  else if (a.group == 64)
    launch_linear_zp<64, S>(a, stream);
  else
    launch_linear_zp<128, S>(a, stream);
}

}  // namespace

hipError_t launch_int4_pack(const Int4PackArgs& a, hipStream_t stream) {
  const int64_t need = (a.n_weights / 8 + kPackThreads - 1) / kPackThreads;
  const int64_t cap = (int64_t)device_cu_count() * 64;
  const unsigned grid = (unsigned)(need < cap ? need : cap);
  if (a.w_bf16) {
    if (a.scale_bf16)
      launch_pack_s<uint16_t, uint16_t>(a, grid, stream);
    else
      launch_pack_s<uint16_t, float>(a, grid, stream);
  } else {
    if (a.scale_bf16)
      launch_pack_s<float, uint16_t>(a, grid, stream);
    else
      launch_pack_s<float, float>(a, grid, stream);
  }
  return hipGetLastError();
}

hipError_t launch_int4_linear(const Int4LinearArgs& a, hipStream_t stream) {
  if (a.scale_bf16)
    launch_linear_b<uint16_t>(a, stream);
  else
    launch_linear_b<float>(a, stream);
  return hipGetLastError();
}

}  // namespace gnf4
