// A whole mixture-of-experts layer for a few tokens: three launches
// (four for more than eight tokens).
//
//  1. moe_gate_up_kernel: routing, gate_up and SwiGLU.  Every workgroup routes
//     all tokens itself and then takes its share of the work items.  Up to one
//     token per wavefront it also picks each token's experts (a launch of its
//     own would cost more than the work); for more, moe_pick_kernel comes first;
//  2. moe_down_kernel: the down projection, one fp32 row per routed slot;
//  3. moe_sum_kernel: each token's sum over its slots, and the residual.
//
// Both projections run the loop of w4_tiles.h: an entry is up to 16 routed rows
// of one expert, an item 32 rows of its weights (16 where rows are long).  The
// routing is made once per workgroup, like the decode table.
//
// Few tokens wait for the chain of the launches: 1 token, 8 of 64 experts of 2048
// x 1024 (28 MB), 25 us, of which each launch costs about 4 before its weights
// stream.  Many experts are bound by the weight stream: 16 tokens over 256 experts
// of 7168 x 2048 (2.5 GB) 577 us, 4.4 TB/s from cold caches; 64 tokens over 64
// experts of 2048 x 1024 (227 MB) 78 us, 2.9 TB/s.

#include <limits.h>
#include <math.h>

#include "route_core.h"
#include "w4_tiles.h"

namespace gnf4 {
namespace {

constexpr int kMaxE = 1024;
constexpr int kMaxRows = kMoeLayerMaxTokens * 32;  // top_k <= 32

// The routing of every token, in LDS behind the decode table: room for
// max_entries entries and the call's rows.
struct Routing {
  uint32_t* entry;
  float* row_w;       // routing weight of a grouped row
  uint8_t* row_tok;   // token of a grouped row
};
// What only the routing itself needs (it lies where the table will be).
struct RouteScratch {
  uint32_t mask[kMaxE][2];     // tokens that picked the expert
  uint16_t off[kMaxE];         // first grouped row of the expert
  uint16_t pick[kMaxRows];     // expert of slot t * top_k + j
  float pick_w[kMaxRows];
  int n_entries;
};

// One wavefront's top-k of token t.  The picks are the k largest keys, equal
// logits to the lower id: the k-th largest key is found bit by bit from the
// top with ballot counts, stopping as soon as exactly k keys reach it.
// Entry s of a lane is expert lane + 64 s.  pick(slot, expert, weight) takes
// each pick, in rank order if `ranked`, else in expert order.
template <int EPL, typename Pick>
__device__ __forceinline__ void top_k_token(const float (&val)[EPL], int E, int top_k, int lane,
                                            bool ranked, const Pick& pick) {
  uint32_t key[EPL];
  uint32_t best = 0;
#pragma unroll
  for (int s = 0; s < EPL; ++s) {
    // an entry that exists keeps a key above the absent ones' 0
    key[s] = lane + kWave * s < E ? max(float_key(val[s]), 1u) : 0u;
    best = max(best, key[s]);
  }
  best = wave_max_u32(best);
  uint32_t th = 0;
  for (int b = 31; b >= 0; --b) {
    const uint32_t cand = th | (1u << b);
    int cnt = 0;
#pragma unroll
    for (int s = 0; s < EPL; ++s) cnt += __popcll(__builtin_amdgcn_ballot_w64(key[s] >= cand));
    if (cnt >= top_k) {
      th = cand;
      if (cnt == top_k) break;
    }
  }
  int need = top_k;  // of the keys equal to th, the lowest ids
#pragma unroll
  for (int s = 0; s < EPL; ++s) need -= __popcll(__builtin_amdgcn_ballot_w64(key[s] > th));
  const float vbest = __uint_as_float((best & 0x80000000u) ? best ^ 0x80000000u : ~best);
  const auto below = [](uint64_t m) {  // of m's lanes, those below this one
    return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32),
                                          __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0u));
  };
  bool sel[EPL];
  float ex[EPL];
  float part = 0.0f;
#pragma unroll
  for (int s = 0; s < EPL; ++s) {
    const uint64_t eq = __builtin_amdgcn_ballot_w64(key[s] == th);
    sel[s] = key[s] > th || (key[s] == th && below(eq) < need);
    need = max(need - __popcll(eq), 0);
    ex[s] = sel[s] ? expf(val[s] - vbest) : 0.0f;
    part += ex[s];
  }
  const float sum = wave_sum_f32(part);
  int slot[EPL];
  if (ranked) {
#pragma unroll
    for (int s = 0; s < EPL; ++s) slot[s] = 0;
#pragma unroll
    for (int s2 = 0; s2 < EPL; ++s2) {
      uint64_t m = __builtin_amdgcn_ballot_w64(sel[s2]);
      while (m) {
        const int src = __builtin_ctzll(m);
        m &= m - 1;
        const uint32_t kj = (uint32_t)__builtin_amdgcn_readlane((int)key[s2], src);
        const int ej = src + kWave * s2;
#pragma unroll
        for (int s = 0; s < EPL; ++s)
          slot[s] += (kj > key[s] || (kj == key[s] && ej < lane + kWave * s)) ? 1 : 0;
      }
    }
  } else {
    int at = 0;
#pragma unroll
    for (int s = 0; s < EPL; ++s) {
      const uint64_t m = __builtin_amdgcn_ballot_w64(sel[s]);
      slot[s] = at + below(m);
      at += __popcll(m);
    }
  }
#pragma unroll
  for (int s = 0; s < EPL; ++s)
    if (sel[s]) pick(slot[s], lane + kWave * s, ex[s] / sum);
}

template <int EPL>
__device__ __forceinline__ void load_logits(const MoeLayerArgs& a, int t, int lane,
                                            float (&val)[EPL]) {
  const float* row = a.logits + (size_t)t * a.E;
#pragma unroll
  for (int s = 0; s < EPL; ++s) val[s] = row[min(lane + kWave * s, a.E - 1)];
}

// The top-k of a batch too large for moe_gate_up_kernel to repeat in every
// workgroup (more than a token per wavefront): one wavefront per token.
template <int EPL>
__global__ __launch_bounds__(kWave) void moe_pick_kernel(MoeLayerArgs a) {
  const int t = blockIdx.x, lane = threadIdx.x;
  float val[EPL];
  load_logits<EPL>(a, t, lane, val);
  top_k_token<EPL>(val, a.E, a.top_k, lane, true, [&](int slot, int e, float w) {
    a.topk_ids[t * a.top_k + slot] = e;
    a.topk_w[t * a.top_k + slot] = w;
  });
}

__device__ __forceinline__ void set_pick(RouteScratch& R, int top_k, int t, int slot, int e,
                                         float w) {
  R.pick[t * top_k + slot] = (uint16_t)e;
  R.pick_w[t * top_k + slot] = w;
  atomicOr(&R.mask[e][t >> 5], 1u << (t & 31));
}

template <int EPL>
__device__ void pick_own(const MoeLayerArgs& a, RouteScratch& R, int wave, int lane, bool writer) {
  float val[EPL];
  load_logits<EPL>(a, min(wave, a.T - 1), lane, val);
  for (int i = threadIdx.x; i < a.E; i += kThreads) R.mask[i][0] = R.mask[i][1] = 0u;
  lds_barrier();
  if (wave < a.T)
    top_k_token<EPL>(val, a.E, a.top_k, lane, writer, [&](int slot, int e, float w) {
      set_pick(R, a.top_k, wave, slot, e, w);
      if (writer) {
        a.topk_ids[wave * a.top_k + slot] = e;
        a.topk_w[wave * a.top_k + slot] = w;
      }
    });
}

// Routes every token into LDS, and as the writing workgroup also into the
// route's outputs and the lists the later launches read.
__device__ int route_all(const MoeLayerArgs& a, const Routing& L, RouteScratch& R, int wave,
                         int lane, bool writer) {
  if (a.T > kWaves) {  // moe_pick_kernel has picked
    const int rows = a.T * a.top_k;
    int e[kMaxRows / kThreads];
    float w[kMaxRows / kThreads];
#pragma unroll
    for (int i = 0; i < kMaxRows / kThreads; ++i) {
      const int s = min((int)threadIdx.x + i * kThreads, rows - 1);
      e[i] = a.topk_ids[s];
      w[i] = a.topk_w[s];
    }
    for (int i = threadIdx.x; i < a.E; i += kThreads) R.mask[i][0] = R.mask[i][1] = 0u;
    lds_barrier();
#pragma unroll
    for (int i = 0; i < kMaxRows / kThreads; ++i) {
      const int s = (int)threadIdx.x + i * kThreads;
      if (s < rows) set_pick(R, a.top_k, s / a.top_k, s % a.top_k, e[i], w[i]);
    }
  } else if (a.E <= 64) {
    pick_own<1>(a, R, wave, lane, writer);
  } else if (a.E <= 128) {
    pick_own<2>(a, R, wave, lane, writer);
  } else if (a.E <= 256) {
    pick_own<4>(a, R, wave, lane, writer);
  } else {
    pick_own<16>(a, R, wave, lane, writer);
  }
  lds_barrier();
  if (wave == 0) {  // experts in ascending order: first rows and entries
    int rows = 0, entries = 0;
    for (int e0 = 0; e0 < a.E; e0 += kWave) {
      const int e = e0 + lane;
      const int cnt = e < a.E ? __popc(R.mask[e][0]) + __popc(R.mask[e][1]) : 0;
      const int tiles = (cnt + 15) >> 4;
      const int cinc = wave_incl_scan(cnt), tinc = wave_incl_scan(tiles);
      const int row = rows + cinc - cnt;
      if (e < a.E) R.off[e] = (uint16_t)row;
      for (int i = 0; i < tiles; ++i) {
        const uint32_t v = make_entry(e, row + 16 * i, min(cnt - 16 * i, 16));
        const int at = entries + tinc - tiles + i;
        L.entry[at] = v;
        if (writer) a.entries[1 + at] = v;
      }
      rows += __builtin_amdgcn_readlane(cinc, kWave - 1);
      entries += __builtin_amdgcn_readlane(tinc, kWave - 1);
    }
    if (lane == 0) {
      R.n_entries = entries;
      if (writer) a.entries[0] = (uint32_t)entries;
    }
  }
  lds_barrier();
  const int n_entries = uniform(R.n_entries);
  for (int s = threadIdx.x; s < a.T * a.top_k; s += kThreads) {
    const int t = s / a.top_k, e = R.pick[s];
    const uint64_t m = (uint64_t)R.mask[e][0] | ((uint64_t)R.mask[e][1] << 32);
    const int row = R.off[e] + __popcll(m & ((1ull << t) - 1ull));
    L.row_tok[row] = (uint8_t)t;
    L.row_w[row] = R.pick_w[s];
    if (writer) a.slot_rows[s] = row;
  }
  lds_barrier();
  return n_entries;
}

__device__ __forceinline__ float silu(float g) {  // through exp2 and rcp, a few units of 2^-24
  return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504f));
}

// The projections' ends (finish).  Every thread takes part and stores.  A tile's
// rows beyond its entry's repeat the entry's last row (the activations of that
// row are in them), and a team that has run out of items repeats its last
// item: the same bits go to the same place, and no store is in a branch, where
// it would make the compiler wait for loads in flight that it cannot count.

// gate_up: 8 U gate rows and their up rows; SwiGLU, scaled by the row's
// routing weight (so the sums over a token's experts need no further factor)
// and kept in fp32: one rounding to bf16 would cost as much accuracy as the
// layer's output rounding.
template <typename S, int U>
struct GateUp {
  typedef RawBf16 Raw;
  static constexpr bool kKeepRaw = true;
  static constexpr int kCols = 8 * U;  // outputs per item and token
  const MoeLayerArgs& a;
  const Routing& L;
  const uint8_t* codes;
  const S* scales;
  size_t expert_rows;
  const uint16_t* x;
  static constexpr const uint8_t* zeros = nullptr;
  __device__ int first_row(int tile) const { return tile * kCols; }
  __device__ int weight_row(int r) const { return r < kCols ? r : a.I + r - kCols; }
  __device__ uint32_t entry(int j) const { return L.entry[j]; }
  __device__ int row(int r) const { return L.row_tok[r]; }
  __device__ void finish(int team, int log_wk, int j, int tile, const char* sums) const {
    const Entry en = read_entry(L.entry[j]);
    // neighbouring lanes hold an output's gate and up
    for (int i = threadIdx.x & ((64 << log_wk) - 1); i < 256 * U; i += 64 << log_wk) {
      // two tiles: gates in the first; one: in its first eight columns
      const int q = i >> 1, o = U == 2 ? q : (q >> 3) * 16 + (i & 1) * 8 + (q & 7);
      const float v = team_sum<U>(sums, team, log_wk, U == 2 ? i & 1 : 0, o);
      const float g = __uint_as_float(dpp_u32<0xA0, 0xF>(0u, __float_as_uint(v)));  // even lane's
      const float u = __uint_as_float(dpp_u32<0xF5, 0xF>(0u, __float_as_uint(v)));  // odd lane's
      const int r = en.row0 + min(tile_row(o), en.cnt - 1);
      a.h[(uint32_t)(r * a.I + tile * kCols + (q & (kCols - 1)))] = silu(g) * u * L.row_w[r];
    }
  }
};

// down: 16 U weight rows, fp32 sums per grouped row.
template <typename S, int U>
struct Down {
  typedef RawF32 Raw;
  static constexpr bool kKeepRaw = false;  // fp32 values of all steps do not fit; read twice
  const MoeLayerArgs& a;
  const uint32_t* entries;
  const uint8_t* codes;
  const S* scales;
  size_t expert_rows;
  const float* x;
  static constexpr const uint8_t* zeros = nullptr;
  __device__ int first_row(int tile) const { return tile * 16 * U; }
  __device__ int weight_row(int r) const { return r; }
  __device__ uint32_t entry(int j) const { return entries[j]; }
  __device__ int row(int r) const { return r; }
  __device__ void finish(int team, int log_wk, int j, int tile, const char* sums) const {
    const Entry en = read_entry(entries[j]);
    for (int i = threadIdx.x & ((64 << log_wk) - 1); i < 256 * U; i += 64 << log_wk) {
      const int h = i >> 8, o = i & 255;
      const int r = en.row0 + min(tile_row(o), en.cnt - 1);
      a.y[(size_t)r * a.H + tile * 16 * U + h * 16 + tile_col(o)] =
          team_sum<U>(sums, team, log_wk, h, o);
    }
  }
};

template <W4 F, int B, typename S, int NST, int U>
__global__ __launch_bounds__(kThreads, waves_per_simd(NST, 1)) void moe_gate_up_kernel(
    MoeLayerArgs a, ItemGrid ig, int max_entries) {
  extern __shared__ __align__(256) char lut[];
  static_assert(sizeof(RouteScratch) <= kLutBytes, "the routing's scratch lies in the table");
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  char* slds = lut + kLutBytes;
  Routing L;
  L.entry = reinterpret_cast<uint32_t*>(slds + 2 * scale_bytes<ScaleWord<B, S, false>, U>(NST));
  L.row_w = reinterpret_cast<float*>(L.entry + max_entries);
  L.row_tok = reinterpret_cast<uint8_t*>(L.row_w + a.T * a.top_k);
  const int n_entries =
      route_all(a, L, *reinterpret_cast<RouteScratch*>(lut), wave, lane, blockIdx.x == 0);
  fill_lut<F>(lut);
  lds_barrier();
  const GateUp<S, U> p = {a, L, a.gu_packed, static_cast<const S*>(a.gu_scales),
                          2 * (size_t)a.I, a.x};
  expert_tiles<F, B, S, false, NST, 1, U>(p, ig, n_entries, lut, slds);
}

template <W4 F, int B, typename S, int NST, int U>
__global__ __launch_bounds__(kThreads, waves_per_simd(NST, 1)) void moe_down_kernel(
    MoeLayerArgs a, ItemGrid ig, int max_entries) {
  extern __shared__ __align__(256) char lut[];
  char* slds = lut + kLutBytes;
  uint32_t* entries =
      reinterpret_cast<uint32_t*>(slds + 2 * scale_bytes<ScaleWord<B, S, false>, U>(NST));
  // the first of the list travels while the table is made
  const uint32_t own = a.entries[min((int)threadIdx.x, max_entries)];
  fill_lut<F>(lut);
  if ((int)threadIdx.x <= max_entries) entries[threadIdx.x] = own;
  for (int i = threadIdx.x + kThreads; i <= max_entries; i += kThreads) entries[i] = a.entries[i];
  lds_barrier();
  const Down<S, U> p = {a, entries + 1, a.dn_packed, static_cast<const S*>(a.dn_scales),
                        (size_t)a.H, a.h};
  expert_tiles<F, B, S, false, NST, 1, U>(p, ig, uniform((int)entries[0]), lut, slds);
}

// out[t] = residual[t] + the fp32 rows of the token's slots, in slot order.
constexpr int kSumThreads = 64, kSumSlots = 8;

__global__ __launch_bounds__(kSumThreads) void moe_sum_kernel(MoeLayerArgs a) {
  const int q = blockIdx.x * kSumThreads + threadIdx.x;  // four columns each
  if (q >= a.H / 4) return;
  const int t = blockIdx.y;
  const size_t o = (size_t)t * a.H + q * 4;
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  if (a.residual)
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = bf16_to_f32(a.residual[o + i]);
  for (int j0 = 0; j0 < a.top_k; j0 += kSumSlots) {  // requested together, added in slot order
    int row[kSumSlots];
#pragma unroll
    for (int j = 0; j < kSumSlots; ++j)
      row[j] = a.slot_rows[t * a.top_k + min(j0 + j, a.top_k - 1)];
    f32x4 y[kSumSlots];
#pragma unroll
    for (int j = 0; j < kSumSlots; ++j)
      y[j] = *reinterpret_cast<const f32x4*>(a.y + (size_t)row[j] * a.H + q * 4);
#pragma unroll
    for (int j = 0; j < kSumSlots; ++j)
      if (j0 + j < a.top_k) v += y[j];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) a.out[o + i] = f32_to_bf16(v[i]);
}

template <W4 F, int B, typename S, bool kDown, int NST, int U>
void launch_projection(const MoeLayerArgs& a, const Launch& l, int max_entries, hipStream_t stream) {
  int lds = kLutBytes + 2 * scale_bytes<ScaleWord<B, S, false>, U>(NST) + 4 * (1 + max_entries);
  if constexpr (!kDown) lds += 5 * a.T * a.top_k;
  const auto kernel = kDown ? moe_down_kernel<F, B, S, NST, U> : moe_gate_up_kernel<F, B, S, NST, U>;
  hipLaunchKernelGGL(kernel, dim3(l.grid), dim3(kThreads), lds, stream, a, l.ig, max_entries);
}

// Rows of up to 4096: items of two column tiles, whose sums share a barrier.
// Longer rows: of one, with up to eight steps of activations per wavefront.
template <W4 F, int B, typename S, bool kDown>
void project(const MoeLayerArgs& a, int experts, int max_entries, hipStream_t stream) {
  const int K = kDown ? a.I : a.H, cols = kDown ? a.H : 2 * a.I;
  if (K <= 4 * kWaves * kStep) {
    const Launch l = plan_launch(experts, max_entries, cols / 32, K, 4);
    if (l.nst == 1)
      launch_projection<F, B, S, kDown, 1, 2>(a, l, max_entries, stream);
    else if (l.nst == 2)
      launch_projection<F, B, S, kDown, 2, 2>(a, l, max_entries, stream);
    else if (l.nst == 3)
      launch_projection<F, B, S, kDown, 3, 2>(a, l, max_entries, stream);
    else
      launch_projection<F, B, S, kDown, 4, 2>(a, l, max_entries, stream);
  } else {
    const Launch l = plan_launch(experts, max_entries, cols / 16, K, 8);
    if (l.nst <= 6)
      launch_projection<F, B, S, kDown, 6, 1>(a, l, max_entries, stream);
    else if (l.nst == 7)
      launch_projection<F, B, S, kDown, 7, 1>(a, l, max_entries, stream);
    else
      launch_projection<F, B, S, kDown, 8, 1>(a, l, max_entries, stream);
  }
}

template <W4 F, int B, typename S>
void launch_layer(const MoeLayerArgs& a, hipStream_t stream) {
  if (a.T > kWaves) {
    const auto pick = a.E <= 64    ? moe_pick_kernel<1>
                      : a.E <= 128 ? moe_pick_kernel<2>
                      : a.E <= 256 ? moe_pick_kernel<4>
                                   : moe_pick_kernel<16>;
    hipLaunchKernelGGL(pick, dim3(a.T), dim3(kWave), 0, stream, a);
  }
  const int rows = a.T * a.top_k;
  const int experts = a.E < rows ? a.E : rows, max_entries = experts + rows / 16;
  project<F, B, S, false>(a, experts, max_entries, stream);
  project<F, B, S, true>(a, experts, max_entries, stream);
  hipLaunchKernelGGL(moe_sum_kernel, dim3((a.H / 4 + kSumThreads - 1) / kSumThreads, a.T),
                     dim3(kSumThreads), 0, stream, a);
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
