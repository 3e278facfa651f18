// int4 weights with group scales: the packer and the linear layer over it.

#include "w4_mfma.h"

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

// Eight weights per thread, G / 8 neighbouring lanes per group.  The code of
// w is the number of midpoints (j + 1/2 - z) s below w: the nearest level,
// ties to the lower code.  The products are exact in fp64 (a scale has 24
// bits, a midpoint 5), so the comparison is exact.
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
    // fp32 quotients, correctly rounded (an fp64 quotient rounded again is)
    const float s32 = ZP ? (float)((double)hi / 15.0) + (float)((double)lo / 15.0)
                         : (float)((double)hi / 7.0);
    const S stored = round_scale(s32, S{});
    const double s = (double)scale_f32(stored);
    int z = 8;
    if constexpr (ZP) {
      z = 0;
#pragma unroll
      for (int j = 0; j < 15; ++j) z += (double)lo > (j + 0.5) * s ? 1 : 0;
      if (s == 0.0) z = 0;
    }
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const double x = (double)v[j];
      int c = 0;
#pragma unroll
      for (int m = 0; m < 15; ++m) c += x > (m + 0.5 - (double)z) * s ? 1 : 0;
      if (s == 0.0) c = z;
      // byte j / 2, the first of the two in the high nibble
      word |= (uint32_t)c << ((j >> 1) * 8 + ((j & 1) ? 0 : 4));
    }
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

constexpr int kLinWaves = 8;

// One workgroup per 16 output columns and 16 RT rows; its wavefronts take
// every kLinWaves-th step of K and their sums are added in wavefront order.
template <int B, typename S, bool ZP, int RT>
__global__ __launch_bounds__(kLinWaves* kWave) void int4_linear_kernel(Int4LinearArgs a) {
  extern __shared__ __align__(256) char lut[];
  auto& red = *reinterpret_cast<float (*)[kLinWaves][RT][256]>(lut + kLutBytes);
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const int g = lane >> 4, col = lane & 15;
  const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16 * RT;
  const int n = min(n0 + col, a.N - 1);
  const int blocks = a.K / B;
  const WeightRow<S> w = {a.packed + (size_t)n * (a.K / 2),
                          static_cast<const S*>(a.scales) + (size_t)n * blocks,
                          ZP ? a.zeros + (size_t)n * blocks : nullptr};
  const uint16_t* xrow[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t)
    xrow[t] = a.x + (size_t)min(m0 + t * 16 + col, a.M - 1) * a.K;
  fill_lut<W4::kInt4>(lut);
  __syncthreads();
  const uint32_t copy = lut_copy(lane);
  f32x4 acc[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int steps = (a.K + kStep - 1) / kStep;
  for (int c = wave; c < steps; c += kLinWaves) {
    StepData<B, S> d;
    load_step<B, ZP>(w, c, g, a.K, d);
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      u32x4 x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = load_frag(xrow[t], c * kStep + k_of<B>(g, i), a.K);
      acc[t] = step_mac_zp<B, ZP>(d, x, copy, acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) red[wave][t][(g * 4 + r) * 16 + col] = acc[t][r];
  __syncthreads();
  for (int i = threadIdx.x; i < RT * 256; i += kLinWaves * kWave) {
    const int m = m0 + (i >> 4), nn = n0 + (i & 15);
    if (m >= a.M || nn >= a.N) continue;
    float y = 0.0f;
#pragma unroll
    for (int k = 0; k < kLinWaves; ++k) y += red[k][i >> 8][i & 255];
    if (a.bias) y += bf16_to_f32(a.bias[nn]);
    a.y[(size_t)m * a.N + nn] = f32_to_bf16(y);
  }
}

template <int B, typename S, bool ZP>
void launch_linear_rt(const Int4LinearArgs& a, hipStream_t stream) {
  const unsigned nt = (unsigned)((a.N + 15) / 16);
  const dim3 block(kLinWaves * kWave);
  if (a.M <= 16)
    hipLaunchKernelGGL((int4_linear_kernel<B, S, ZP, 1>), dim3(nt, 1), block,
                       kLutBytes + kLinWaves * 1024, stream, a);
  else
    hipLaunchKernelGGL((int4_linear_kernel<B, S, ZP, 4>), dim3(nt, (a.M + 63) / 64), block,
                       kLutBytes + kLinWaves * 4096, stream, a);
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
