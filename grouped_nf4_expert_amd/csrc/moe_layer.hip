// A whole mixture-of-experts layer for a few tokens.

#include "w4_mfma.h"

namespace gnf4 {
namespace {

constexpr int kGuWaves = 8;
constexpr int kDnWaves = 16;

// gate_up and SwiGLU.  Work item: one routed expert and 16 gate rows with
// their 16 up rows; the wavefronts split K and their sums meet in LDS.  h is
// scaled by the token's routing weight here, so the down projection's sums
// over a token's experts need no further factor, and kept as a sum of two
// bf16 numbers (hi + lo, within 2^-17): one rounding to bf16 would cost as
// much accuracy as the layer's output rounding.
template <W4 F, int B, typename S>
__global__ __launch_bounds__(kGuWaves* kWave) void moe_gate_up_kernel(MoeLayerArgs a) {
  __shared__ __align__(16) char lut[F == W4::kMx4 ? 16 : kLutBytes];
  __shared__ float red[kGuWaves][2][256];
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const int g = lane >> 4, col = lane & 15;
  fill_lut<F>(lut);
  __syncthreads();
  const uint32_t copy = lut_copy<F>(lane);
  const int tiles = a.I / 16;
  const int items = a.num_groups[0] * tiles;
  const int steps = (a.H + kStep - 1) / kStep;
  const size_t kb = a.H / 2, blocks = a.H / B;
  for (int it = blockIdx.x; it < items; it += gridDim.x) {
    const int j = it / tiles, n0 = (it % tiles) * 16;
    const int e = a.group_ids[j], cnt = a.group_sizes[j], off = a.offsets[e];
    const size_t rg = (size_t)e * 2 * a.I + n0 + col, ru = rg + a.I;
    const S* sc = static_cast<const S*>(a.gu_scales);
    const WeightRow<S> wg = {a.gu_packed + rg * kb, sc + rg * blocks, nullptr};
    const WeightRow<S> wu = {a.gu_packed + ru * kb, sc + ru * blocks, nullptr};
    for (int r0 = 0; r0 < cnt; r0 += 16) {
      const int slot = a.sorted[off + min(r0 + col, cnt - 1)];
      const uint16_t* xrow = a.x + (size_t)(slot / a.top_k) * a.H;
      f32x4 ag = {0.0f, 0.0f, 0.0f, 0.0f}, au = ag;
      for (int c = wave; c < steps; c += kGuWaves) {
        StepData<B, S> dg, du;
        load_step<B, false>(wg, c, g, a.H, dg);
        load_step<B, false>(wu, c, g, a.H, du);
        bf16x8 x[1][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[0][i] = load_frag(xrow, c * kStep + k_of<B>(g, i), a.H);
        ag = step_mac<F, B, false, 1>(dg, x, lut, copy, ag);
        au = step_mac<F, B, false, 1>(du, x, lut, copy, au);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        red[wave][0][(g * 4 + r) * 16 + col] = ag[r];
        red[wave][1][(g * 4 + r) * 16 + col] = au[r];
      }
      __syncthreads();
      if (threadIdx.x < 256) {
        const int row = r0 + (threadIdx.x >> 4);
        if (row < cnt) {
          float gs = 0.0f, us = 0.0f;
#pragma unroll
          for (int k = 0; k < kGuWaves; ++k) {
            gs += red[k][0][threadIdx.x];
            us += red[k][1][threadIdx.x];
          }
          const float h = gs / (1.0f + expf(-gs)) * us * a.topk_w[a.sorted[off + row]];
          const uint16_t hi = f32_to_bf16(h);
          const size_t o = (size_t)(off + row) * a.I + n0 + (threadIdx.x & 15);
          a.h_hi[o] = hi;
          a.h_lo[o] = f32_to_bf16(h - bf16_to_f32(hi));
        }
      }
      __syncthreads();
    }
  }
}

// down and the sum over each token's experts.  A workgroup owns 16 output
// columns for every token and expert, so the sums stay on chip: the steps of
// all routed experts are dealt to the wavefronts in equal contiguous ranges,
// each wavefront adds into its own [token][column] sums in LDS, and the
// wavefronts' sums are added in order.  No atomics, the same bits every run.
template <W4 F, int B, typename S, int TMAX>
__global__ __launch_bounds__(kDnWaves* kWave) void moe_down_kernel(MoeLayerArgs a) {
  __shared__ __align__(16) char lut[F == W4::kMx4 ? 16 : kLutBytes];
  __shared__ float sum[kDnWaves][TMAX * 16];
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const int g = lane >> 4, col = lane & 15;
  const int n0 = blockIdx.x * 16;
  fill_lut<F>(lut);
  for (int i = lane; i < TMAX * 16; i += kWave) sum[wave][i] = 0.0f;
  __syncthreads();
  const uint32_t copy = lut_copy<F>(lane);
  const int steps = (a.I + kStep - 1) / kStep;
  const int total = a.num_groups[0] * steps;
  int s0 = (int)((int64_t)total * wave / kDnWaves);
  const int s1 = (int)((int64_t)total * (wave + 1) / kDnWaves);
  const size_t kb = a.I / 2, blocks = a.I / B;
  while (s0 < s1) {
    const int j = s0 / steps, c0 = s0 % steps;
    const int c1 = min(steps, c0 + s1 - s0);
    s0 += c1 - c0;
    const int e = a.group_ids[j], cnt = a.group_sizes[j], off = a.offsets[e];
    const size_t rn = (size_t)e * a.H + n0 + col;
    const WeightRow<S> w = {a.dn_packed + rn * kb, static_cast<const S*>(a.dn_scales) + rn * blocks,
                            nullptr};
    for (int r0 = 0; r0 < cnt; r0 += 16) {
      const size_t hr = (size_t)(off + min(r0 + col, cnt - 1)) * a.I;
      f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int c = c0; c < c1; ++c) {
        StepData<B, S> d;
        load_step<B, false>(w, c, g, a.I, d);
        bf16x8 x[2][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[0][i] = load_frag(a.h_hi + hr, c * kStep + k_of<B>(g, i), a.I);
          x[1][i] = load_frag(a.h_lo + hr, c * kStep + k_of<B>(g, i), a.I);
        }
        acc = step_mac<F, B, false, 2>(d, x, lut, copy, acc);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = r0 + g * 4 + r;
        if (row < cnt) sum[wave][(a.sorted[off + row] / a.top_k) * 16 + col] += acc[r];
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * 16; i += kDnWaves * kWave) {
    const size_t o = (size_t)(i >> 4) * a.H + n0 + (i & 15);
    float y = a.residual ? bf16_to_f32(a.residual[o]) : 0.0f;
#pragma unroll
    for (int k = 0; k < kDnWaves; ++k) y += sum[k][i];
    a.out[o] = f32_to_bf16(y);
  }
}

template <W4 F, int B, typename S>
void launch_layer(const MoeLayerArgs& a, hipStream_t stream) {
  const int64_t groups = a.E < a.T * a.top_k ? a.E : a.T * a.top_k;
  const int64_t items = groups * (a.I / 16);
  const int64_t cap = 2 * (int64_t)device_cu_count();
  hipLaunchKernelGGL((moe_gate_up_kernel<F, B, S>), dim3((unsigned)(items < cap ? items : cap)),
                     dim3(kGuWaves * kWave), 0, stream, a);
  if (a.T <= 16)
    hipLaunchKernelGGL((moe_down_kernel<F, B, S, 16>), dim3(a.H / 16), dim3(kDnWaves * kWave), 0,
                       stream, a);
  else
    hipLaunchKernelGGL((moe_down_kernel<F, B, S, kMoeLayerMaxTokens>), dim3(a.H / 16),
                       dim3(kDnWaves * kWave), 0, stream, a);
}

}  // namespace

hipError_t launch_moe_layer(const MoeLayerArgs& a, int scale_kind, hipStream_t stream) {
  if (scale_kind == GNF4_SCALE_E8M0)
    launch_layer<W4::kMx4, 32, uint8_t>(a, stream);
  else if (scale_kind == GNF4_DTYPE_BF16)
    launch_layer<W4::kNf4, 64, uint16_t>(a, stream);
  else
    launch_layer<W4::kNf4, 64, float>(a, stream);
  return hipGetLastError();
}

}  // namespace gnf4
