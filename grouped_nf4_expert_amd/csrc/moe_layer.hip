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
// Both projections share one shape (expert_tiles).  A work item is an entry --
// up to 16 routed rows of one expert, one matrix-core tile -- and 32 weight
// rows.  The eight wavefronts of a workgroup form teams; a team owns an item, its
// wavefronts take every wk-th step of K and their sums meet in LDS.  One
// workgroup per CU stays resident and each team walks a contiguous range of
// items, so
//  * the decode table and the routing are made once;
//  * a wavefront always meets the same steps of K, and its activations (the
//    entry's rows at those steps) stay in registers until the entry changes:
//    read per item, they cost the address units four times what the weights
//    do;
//  * each wavefront loads weights ahead, across items and barriers: a CU must
//    keep tens of kilobytes in flight to draw its share of the HBM stream.

#include <math.h>

#include "route_core.h"
#include "w4_mfma.h"

namespace gnf4 {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = kWaves * kWave;
constexpr int kGroup = 2;  // items of a group that shares the activations of a pass
constexpr int kMaxE = 1024;
constexpr int kMaxRows = kMoeLayerMaxTokens * 32;  // top_k <= 32
constexpr int kMaxEntries = kMoeLayerMaxEntries;

// A value that is the same in every lane, in a scalar register.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// An entry: up to 16 grouped rows of one expert.
__device__ __forceinline__ uint32_t make_entry(int e, int row0, int cnt) {
  return (uint32_t)e | ((uint32_t)row0 << 10) | ((uint32_t)(cnt - 1) << 21);
}
struct Entry {
  int e, row0, cnt;
};
__device__ __forceinline__ Entry read_entry(uint32_t v) {
  return Entry{(int)(v & 1023u), (int)((v >> 10) & 2047u), (int)(v >> 21) + 1};
}

// The routing of every token, in LDS behind the decode table: room for
// max_entries entries and the call's rows.
struct Routing {
  uint32_t* entry;
  float* row_w;       // routing weight of a grouped row, and 0 behind them
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
  if (threadIdx.x == 0) L.row_w[a.T * a.top_k] = 0.0f;
  lds_barrier();
  return n_entries;
}

// The work items of a projection: entry j's tiles, then entry j + 1's.
struct ItemGrid {
  int tiles;    // items per entry
  int K;        // codes per weight row
  int log_wk;   // wavefronts per team, as a power of two
  int passes;   // over K, where an item's activations do not fit at once
};

// One set of the wavefronts' sums: 512 words per wavefront in the second halves
// of the decode table's rows; two sets fill them.
constexpr int kSumBytes = kWaves * 512 / 32 * 256;
static_assert(2 * kSumBytes == kLutBytes, "two sets of sums beside the table");

// Eight activations of a row at k, from the layer's input (bf16) or from h
// (fp32): the largest magnitude's bits, and the values as scaled fp16.
struct RawBf16 {
  u32x4 v;
  __device__ __forceinline__ void load(const uint16_t* x, uint32_t at) {
    v = *reinterpret_cast<const u32x4*>(x + at);
  }
  __device__ __forceinline__ uint32_t max_bits() const {  // as fp32 bits
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      m = max(m, max((v[i] << 16) & 0x7fff0000u, v[i] & 0x7fff0000u));
    return m;
  }
  __device__ __forceinline__ u32x4 half(float up) const {
    u32x4 h;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      h[i] = pack_f16x2(__uint_as_float(v[i] << 16) * up, __uint_as_float(v[i] & 0xffff0000u) * up);
    return h;
  }
};
struct RawF32 {
  f32x4 a, b;
  __device__ __forceinline__ void load(const float* x, uint32_t at) {
    a = *reinterpret_cast<const f32x4*>(x + at);
    b = *reinterpret_cast<const f32x4*>(x + at + 4);
  }
  __device__ __forceinline__ uint32_t max_bits() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      m = max(m, max(__float_as_uint(a[i]) & 0x7fffffffu, __float_as_uint(b[i]) & 0x7fffffffu));
    return m;
  }
  __device__ __forceinline__ u32x4 half(float up) const {
    return u32x4{pack_f16x2(a[0] * up, a[1] * up), pack_f16x2(a[2] * up, a[3] * up),
                 pack_f16x2(b[0] * up, b[1] * up), pack_f16x2(b[2] * up, b[3] * up)};
  }
};

// The scales of a turn in LDS: step s of row r (0..31) of a team, rows side by
// side, each step's a word further on so that a fetch's stores (neighbouring
// lanes hold neighbouring steps) meet different banks.
template <typename Scale>
__device__ __forceinline__ int scale_at(int s, int r) {
  return s * (32 * (int)sizeof(Scale) + 4 * Scale::kWords) + r * (int)sizeof(Scale);
}
template <typename Scale>
__device__ __forceinline__ int team_scales(int nst, int team, int wk) {
  return team * scale_at<Scale>(nst * wk, 0);
}
template <typename Scale>
__host__ __device__ constexpr int scale_bytes(int nst) {
  return kWaves * nst * (32 * (int)sizeof(Scale) + 4 * Scale::kWords);
}

// Workgroups per CU: two where a wavefront's activations leave its registers
// room (their barriers then fall apart: one computes while the other waits).
constexpr int groups_per_cu(int nst, int g) { return nst <= 2 && g == 1 ? 2 : 1; }
constexpr int waves_per_simd(int nst, int g) { return groups_per_cu(nst, g) * kWaves / 4; }

// The loop shared by the projections (see the head of the file); P says where
// an item's weights and activations are and what becomes of its sums.  NST:
// steps per wavefront and item whose activations fit the registers.  Longer
// rows (G > 1) are walked in passes: G neighbouring items share each pass's
// activations and keep their sums in registers from pass to pass.  Weight
// addresses are a scalar base that the item and the step move and a lane offset
// that never moves.
template <W4 F, int B, typename S, int NST, int G, typename P>
__device__ __forceinline__ void expert_tiles(const P& p, const ItemGrid ig, int n_entries,
                                             char* lut, char* slds) {
  typedef ScaleWord<B, S> Scale;
  constexpr int kBufs = NST == 3 ? 3 : 4, kAhead = kBufs - 1;
  constexpr int kUnroll = NST == 1 ? 4 : 2;  // items per turn of the loop
  static_assert(G == 1 || G == kUnroll, "a turn is a group's items");
  static_assert(NST * kUnroll % kBufs == 0 && kUnroll % 2 == 0,
                "the buffers of a step and of an item must be known when compiling");
  const int wave = uniform(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int g = lane >> 4, col = lane & 15;
  const int wk = 1 << ig.log_wk, teams = kWaves >> ig.log_wk;
  const int team = wave >> ig.log_wk, kw = wave & (wk - 1);
  const int K = ig.K, kb = K / 2, blocks = K / B;
  const int steps = (K + kStep - 1) / kStep;
  const uint32_t copy = lut_copy(lane);
  // this team's groups of G items; every team makes as many rounds as the longest
  const int groups = n_entries * (ig.tiles / G), n_teams = (int)gridDim.x * teams;
  const int share = uniform(groups / n_teams), extra = groups - share * n_teams;
  const int tid = (int)blockIdx.x * teams + team;
  const int i0 = min(tid * share + min(tid, extra), groups - 1) * G;
  const int n_mine = share + (tid < extra ? 1 : 0);
  const int rounds = share + ((int)blockIdx.x * teams < extra ? 1 : 0);
  if (rounds == 0) return;

  // load side: the group, pass and item that the next loads belong to
  int lj = uniform(i0 / ig.tiles), lt = i0 - lj * ig.tiles;
  int cj = lj, ct = lt;   // and the group whose sums are being formed
  int left = n_mine - 1;  // groups after it
  int lp = 0, lg = 0;
  const uint32_t coff = (uint32_t)(col * kb + g * 16);
  const uint8_t* cbase;
  const auto weight_row = [&](int j, int tile) {  // of the stack
    const uint32_t ev = (uint32_t)uniform((int)p.entry(j));
    return (size_t)read_entry(ev).e * p.expert_rows + (size_t)(tile * P::kTileRows);
  };
  const auto set_item = [&]() { cbase = p.codes + weight_row(lj, lt + lg) * (size_t)kb; };
  // one item (of a pass) on; past the last group, the last one again
  const auto step_on = [&](int& j, int& t, int& pass, int& item, int& rest) {
    if constexpr (G > 1) {
      if (++item < G) return;
      item = 0;
      if (++pass < ig.passes) return;
      pass = 0;
    }
    if (rest > 0) {
      --rest;
      t += G;
      if (t == ig.tiles) {
        t = 0;
        j = uniform(j + 1);
      }
    }
  };
  const auto load = [&](u32x4 (&w)[2], int i) {
    const int c = min((lp * wk + kw) * NST + i, steps - 1);
#pragma unroll
    for (int u = 0; u < 2; ++u)
      w[u] = load_codes(cbase + (size_t)u * p.second * kb, c, coff, g, kb);
    if (i == NST - 1) {
      step_on(lj, lt, lp, lg, left);
      set_item();
    }
  };
  // Scales go through LDS: read by each lane from its own row they would cost
  // as many cache lines as the codes.  The team's threads fetch the item's
  // 2 x 16 rows of wk * NST steps in row order, two items ahead.
  constexpr int kSteps = 32 * NST, kFetch = (kSteps + 63) / 64;  // words per wavefront, per thread
  int fj = lj, ft = lt, fp = 0, fg = 0, fleft = left;
  uint32_t foff[kFetch];
  int fstep[kFetch], fat[kFetch];
#pragma unroll
  for (int i = 0; i < kFetch; ++i) {  // row, then step; threads left over repeat the last
    const int id = min(kw * kWave + lane + i * (wk * kWave), (32 * NST << ig.log_wk) - 1);
    const int row = id / NST >> ig.log_wk;
    fstep[i] = id - ((row * NST) << ig.log_wk);
    foff[i] = (uint32_t)(((row & 15) + (row & 16 ? p.second : 0)) * blocks * (int)sizeof(S));
    if constexpr (G == 1) foff[i] += scales_first<B>(min(fstep[i], steps - 1), blocks) * sizeof(S);
    fat[i] = team_scales<Scale>(NST, team, wk) + scale_at<Scale>(fstep[i], row);
  }
  Scale fetched[2][kFetch];
  int fsteps[2] = {0, 0};  // the first step of a fetch
  const auto fetch = [&](int buf) {
    const char* sb = reinterpret_cast<const char*>(p.scales) +
                     weight_row(fj, ft + fg) * (size_t)blocks * sizeof(S);
    if constexpr (G > 1) fsteps[buf] = fp * wk * NST;
#pragma unroll
    for (int i = 0; i < kFetch; ++i) {
      uint32_t at = foff[i];
      if constexpr (G > 1)
        at += scales_first<B>(min(fsteps[buf] + fstep[i], steps - 1), blocks) * sizeof(S);
      load_scales<B, S>(sb, at, NST == 1 && blocks < kStep / B, fetched[buf][i]);
    }
    step_on(fj, ft, fp, fg, fleft);
  };
  const auto put = [&](int buf) {
#pragma unroll
    for (int i = 0; i < kFetch; ++i) {
      align_scales<B, S>(fetched[buf][i], min(fsteps[buf] + fstep[i], steps - 1), blocks);
      *reinterpret_cast<Scale*>(slds + buf * scale_bytes<Scale>(NST) + fat[i]) = fetched[buf][i];
    }
  };
  // The entry's activations at this wavefront's steps of a pass, each row
  // scaled by its largest value there; `down` undoes it for the rows whose sums
  // the lane holds (the row of lane l here is l % 16, of its sums
  // 4 (l / 16) + r).
  u32x4 x[NST][4];
  f32x4 down;
  constexpr bool kKeep = P::kKeepRaw || NST == 1;
  typename P::Raw keep[kKeep ? NST : 1][4];
  uint32_t xrow = 0;
  // Register i of a step lies in a block that is in the row or past it as a
  // whole (K is a multiple of the block); past it, the row's start is read and
  // multiplied by zero.
  const auto inside = [&](int pass, int n, int i) {
    return ((pass * wk + kw) * NST + n) * kStep + (B == 64 ? (i >> 1) * 64 : i * B) < K;
  };
  const auto raw = [&](int pass, int n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = ((pass * wk + kw) * NST + n) * kStep + (k_of<B>(0, i) - k_of<B>(0, 0));
      keep[kKeep ? n : 0][i].load(p.x + (inside(pass, n, i) ? k : 0), xrow);
    }
  };
  const auto issue_x = [&](int j, int pass) {
    const Entry en = read_entry((uint32_t)uniform((int)p.entry(j)));
    xrow = (uint32_t)p.row(en.row0 + min(col, en.cnt - 1)) * (uint32_t)K + k_of<B>(g, 0);
    raw(pass, 0);
    if constexpr (kKeep)
#pragma unroll
      for (int n = 1; n < NST; ++n) raw(pass, n);
  };
  const auto take_x = [&](int pass) {
    uint32_t top = 0;
#pragma unroll
    for (int n = 0; n < NST; ++n) {
      if (!kKeep && n > 0) raw(pass, n);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t m = keep[kKeep ? n : 0][i].max_bits();
        top = max(top, inside(pass, n, i) ? m : 0u);
      }
    }
    top = max(top, (uint32_t)__shfl_xor((int)top, 16, kWave));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32, kWave));
    const RowScale rs = {(int)(top >> 23)};
    const float up = rs.up();
#pragma unroll
    for (int n = 0; n < NST; ++n) {
      if (!kKeep) raw(pass, n);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[n][i] = keep[kKeep ? n : 0][i].half(inside(pass, n, i) ? up : 0.0f);
      if constexpr (!kKeep) __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) down[r] = __shfl(rs.down(), g * 4 + r, kWave);
  };

  // the first activations and scales go ahead of the weights
  issue_x(cj, 0);
  fetch(0);
  set_item();
  __builtin_amdgcn_sched_barrier(0);
  u32x4 w[kBufs][2];
#pragma unroll
  for (int n = 0; n < kAhead; ++n) load(w[n], n % NST);
  fetch(1);
  __builtin_amdgcn_sched_barrier(0);
  take_x(0);
  put(0);
  lds_barrier();
  // an item's steps of a pass; `it` is its position within a turn of the loop
  const auto item_steps = [&](int it, f32x4 (&acc)[2]) {
    acc[0] = acc[1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    fetch(it & 1);
    const char* mine = slds + (it & 1) * scale_bytes<Scale>(NST) +
                       team_scales<Scale>(NST, team, wk) + scale_at<Scale>(kw * NST, col);
#pragma unroll
    for (int n = 0; n < NST; ++n) {
      const int q = it * NST + n;
      load(w[(q + kAhead) % kBufs], (n + kAhead) % NST);
      __builtin_amdgcn_sched_barrier(0);  // the loads go first
      // idle steps past the row's end have zero activations
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const Scale sc = *reinterpret_cast<const Scale*>(mine + scale_at<Scale>(n, h * 16));
        acc[h] = step_mac<F, B, S>(w[q % kBufs][h], sc, x[n], copy, acc[h]);
        // where registers are short, one tile's decode at a time
        if constexpr (G > 1 || F == W4::kMx4 || groups_per_cu(NST, G) > 1)
          __builtin_amdgcn_sched_barrier(0);
      }
    }
    put((it + 1) & 1);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[h][r] *= down[r];
  };
  // the wavefronts' sums of an item meet: [wave][tile][register][lane]
  int turn = 0;
  const auto meet = [&](const f32x4 (&acc)[2], int tile) {
    char* sums = lut + (turn & 1) * kSumBytes;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        *reinterpret_cast<float*>(
            sums + lds_half(((wave * 2 + h) * 4 + r) * kWave) + lds_half(lane) - 128) = acc[h][r];
    lds_barrier();
    p.finish(team, ig.log_wk, cj, tile, sums);
    ++turn;
  };
  if constexpr (G == 1) {
    for (;;) {
#pragma unroll
      for (int it = 0; it < kUnroll; ++it) {
        f32x4 acc[2];
        item_steps(it, acc);
        meet(acc, ct);
        if (turn == rounds) return;
        if (turn < n_mine && ++ct == ig.tiles) {
          ct = 0;
          cj = uniform(cj + 1);
          issue_x(cj, 0);
          take_x(0);
        }
      }
    }
  } else {
    for (int round = 0; round < rounds; ++round) {
      f32x4 total[G][2];
#pragma unroll
      for (int it = 0; it < G; ++it) total[it][0] = total[it][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      for (int pass = 0; pass < ig.passes; ++pass) {
        if (round + pass > 0) {
          issue_x(cj, pass);
          take_x(pass);
        }
#pragma unroll
        for (int it = 0; it < G; ++it) {
          f32x4 acc[2];
          item_steps(it, acc);
          total[it][0] += acc[0];
          total[it][1] += acc[1];
          lds_barrier();  // the next scales are in place, the last ones free
        }
      }
#pragma unroll
      for (int it = 0; it < G; ++it) meet(total[it], ct + it);
      if (round + 1 < n_mine) {
        ct += G;
        if (ct == ig.tiles) {
          ct = 0;
          ++cj;
        }
      }
    }
  }
}

// Output o (0..255) of a tile: register o / 64 of lane o % 64.
__device__ __forceinline__ int tile_row(int o) { return ((o & 63) >> 4) * 4 + (o >> 6); }
__device__ __forceinline__ int tile_col(int o) { return o & 15; }

// The sum of a team's wavefronts, in wavefront order.
__device__ __forceinline__ float team_sum(const char* sums, int team, int log_wk, int tile, int o) {
  const char* p = sums + lds_half((((team << log_wk) * 2 + tile) << 8) + o);
  const auto at = [p](int k) { return *reinterpret_cast<const float*>(p + k * (512 / 32 * 256)); };
  float v = at(0) + at(1);
  if (log_wk > 1) v = v + at(2) + at(3);
  if (log_wk > 2) v = v + at(4) + at(5) + at(6) + at(7);
  return v;
}

__device__ __forceinline__ float silu(float g) {  // through exp2 and rcp, a few units of 2^-24
  return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504f));
}

// The projections' ends (finish).  Every thread takes part and stores, rows an
// entry does not have to a row kept for them, and a team that has run out of
// items repeats its last one's: a store in a branch would make the compiler
// wait for loads in flight that it cannot count.

// gate_up: 16 gate rows and their 16 up rows; SwiGLU, scaled by the row's
// routing weight (so the sums over a token's experts need no further factor)
// and kept in fp32: one rounding to bf16 would cost as much accuracy as the
// layer's output rounding.
template <typename S>
struct GateUp {
  typedef RawBf16 Raw;
  static constexpr bool kKeepRaw = true;
  static constexpr int kTileRows = 16;
  const MoeLayerArgs& a;
  const Routing& L;
  const uint8_t* codes;
  const S* scales;
  size_t expert_rows;
  int second;  // rows from an item's first tile to its second
  const uint16_t* x;
  __device__ uint32_t entry(int j) const { return L.entry[j]; }
  __device__ int row(int r) const { return L.row_tok[r]; }
  __device__ void finish(int team, int log_wk, int j, int tile, const char* sums) const {
    const Entry en = read_entry(L.entry[j]);
    // neighbouring lanes hold an output's gate and up
    for (int i = threadIdx.x & ((64 << log_wk) - 1); i < 512; i += 64 << log_wk) {
      const int o = i >> 1, row = tile_row(o);
      const float v = team_sum(sums, team, log_wk, i & 1, o);
      const float g = __uint_as_float(dpp_u32<0xA0, 0xF>(0u, __float_as_uint(v)));  // even lane's
      const float u = __uint_as_float(dpp_u32<0xF5, 0xF>(0u, __float_as_uint(v)));  // odd lane's
      const int r = row < en.cnt ? en.row0 + row : a.T * a.top_k;
      a.h[(uint32_t)(r * a.I + tile * 16 + tile_col(o))] = silu(g) * u * L.row_w[r];
    }
  }
};

// down: 32 weight rows, fp32 sums per grouped row.
template <typename S>
struct Down {
  typedef RawF32 Raw;
  static constexpr bool kKeepRaw = false;  // fp32 values of all steps do not fit; read twice
  static constexpr int kTileRows = 32;
  const MoeLayerArgs& a;
  const uint32_t* entries;
  const uint8_t* codes;
  const S* scales;
  size_t expert_rows;
  int second;
  const float* x;
  __device__ uint32_t entry(int j) const { return entries[j]; }
  __device__ int row(int r) const { return r; }
  __device__ void finish(int team, int log_wk, int j, int tile, const char* sums) const {
    const Entry en = read_entry(entries[j]);
    for (int i = threadIdx.x & ((64 << log_wk) - 1); i < 512; i += 64 << log_wk) {
      const int h = i >> 8, o = i & 255, row = tile_row(o);
      const int r = row < en.cnt ? en.row0 + row : a.T * a.top_k;
      a.y[(size_t)r * a.H + tile * 32 + h * 16 + tile_col(o)] = team_sum(sums, team, log_wk, h, o);
    }
  }
};

template <W4 F, int B, typename S, int NST, int G>
__global__ __launch_bounds__(kThreads, waves_per_simd(NST, G)) void moe_gate_up_kernel(MoeLayerArgs a, ItemGrid ig,
                                                               int max_entries) {
  extern __shared__ __align__(256) char lut[];
  static_assert(sizeof(RouteScratch) <= kLutBytes, "the routing's scratch lies in the table");
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  char* slds = lut + kLutBytes;
  Routing L;
  L.entry = reinterpret_cast<uint32_t*>(slds + 2 * scale_bytes<ScaleWord<B, S>>(NST));
  L.row_w = reinterpret_cast<float*>(L.entry + max_entries);
  L.row_tok = reinterpret_cast<uint8_t*>(L.row_w + a.T * a.top_k + 1);
  const int n_entries =
      route_all(a, L, *reinterpret_cast<RouteScratch*>(lut), wave, lane, blockIdx.x == 0);
  fill_lut<F>(lut);
  lds_barrier();
  const GateUp<S> p = {a, L, a.gu_packed, static_cast<const S*>(a.gu_scales),
                       2 * (size_t)a.I, a.I, a.x};
  expert_tiles<F, B, S, NST, G>(p, ig, n_entries, lut, slds);
}

template <W4 F, int B, typename S, int NST, int G>
__global__ __launch_bounds__(kThreads, waves_per_simd(NST, G)) void moe_down_kernel(MoeLayerArgs a, ItemGrid ig,
                                                            int max_entries) {
  extern __shared__ __align__(256) char lut[];
  char* slds = lut + kLutBytes;
  uint32_t* entries =
      reinterpret_cast<uint32_t*>(slds + 2 * scale_bytes<ScaleWord<B, S>>(NST));
  for (int i = threadIdx.x; i <= max_entries; i += kThreads) entries[i] = a.entries[i];
  fill_lut<F>(lut);
  lds_barrier();
  const Down<S> p = {a, entries + 1, a.dn_packed, static_cast<const S*>(a.dn_scales),
                     (size_t)a.H, 16, a.h};
  expert_tiles<F, B, S, NST, G>(p, ig, uniform((int)entries[0]), lut, slds);
}

// out[t] = residual[t] + the fp32 rows of the token's slots, in slot order.
constexpr int kSumThreads = 256;

__global__ __launch_bounds__(kSumThreads) void moe_sum_kernel(MoeLayerArgs a) {
  const int q = blockIdx.x * kSumThreads + threadIdx.x;  // four columns each
  if (q >= a.H / 4) return;
  const int t = blockIdx.y;
  const size_t o = (size_t)t * a.H + q * 4;
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  if (a.residual)
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = bf16_to_f32(a.residual[o + i]);
  for (int j = 0; j < a.top_k; ++j)
    v += *reinterpret_cast<const f32x4*>(a.y + (size_t)a.slot_rows[t * a.top_k + j] * a.H + q * 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) a.out[o + i] = f32_to_bf16(v[i]);
}

// Wavefronts per team, hence steps per wavefront: the widest team, with the
// fewest activations to load and hold per wavefront, unless a narrower one
// takes at least an eighth fewer steps in all when `entries` are routed (a team
// wider than the row's steps has idle wavefronts).  A wavefront holds the
// activations of at most four steps; longer rows take passes of four by the
// whole workgroup.
struct Launch {
  unsigned grid;
  int nst, group;
  ItemGrid ig;
};
Launch plan_launch(int entries, int max_entries, int tiles, int K) {
  const int steps = (K + kStep - 1) / kStep;
  const int64_t cus = device_cu_count(), items = (int64_t)entries * tiles;
  int best = 3, nst = (steps + 7) / 8, group = 1, passes = 1;
  if (nst > 4) {
    passes = (nst + 3) / 4;
    nst = 4;
    group = kGroup;
  } else {
    int64_t best_cost = INT64_MAX;
    for (int l = 3; l >= 1; --l) {
      const int n = (steps + (1 << l) - 1) >> l;
      const int64_t teams = cus * groups_per_cu(n, 1) * (kWaves >> l);
      const int64_t cost = (items + teams - 1) / teams * n * groups_per_cu(n, 1);
      if (n <= 4 && cost < best_cost) {
        best = l;
        nst = n;
        best_cost = cost * 7 / 8;
      }
    }
  }
  const int teams = kWaves >> best;
  const int64_t need = ((int64_t)max_entries * (tiles / group) + teams - 1) / teams;
  const int64_t room = cus * groups_per_cu(nst, group);
  return Launch{(unsigned)(need < room ? need : room), nst, group, ItemGrid{tiles, K, best, passes}};
}

template <W4 F, int B, typename S, int NST, int G>
void launch_gate_up(const MoeLayerArgs& a, const Launch& l, int max_entries, hipStream_t stream) {
  const int lds = kLutBytes + 2 * scale_bytes<ScaleWord<B, S>>(NST) + 4 * max_entries +
                  4 + 5 * a.T * a.top_k;
  hipLaunchKernelGGL((moe_gate_up_kernel<F, B, S, NST, G>), dim3(l.grid), dim3(kThreads), lds,
                     stream, a, l.ig, max_entries);
}
template <W4 F, int B, typename S, int NST, int G>
void launch_down(const MoeLayerArgs& a, const Launch& l, int max_entries, hipStream_t stream) {
  const int lds = kLutBytes + 2 * scale_bytes<ScaleWord<B, S>>(NST) + 4 * (1 + max_entries);
  hipLaunchKernelGGL((moe_down_kernel<F, B, S, NST, G>), dim3(l.grid), dim3(kThreads), lds,
                     stream, a, l.ig, max_entries);
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
  const Launch gu = plan_launch(experts, max_entries, a.I / 16, a.H);
  if (gu.group > 1)
    launch_gate_up<F, B, S, 4, kGroup>(a, gu, max_entries, stream);
  else if (gu.nst == 1)
    launch_gate_up<F, B, S, 1, 1>(a, gu, max_entries, stream);
  else if (gu.nst == 2)
    launch_gate_up<F, B, S, 2, 1>(a, gu, max_entries, stream);
  else if (gu.nst == 3)
    launch_gate_up<F, B, S, 3, 1>(a, gu, max_entries, stream);
  else
    launch_gate_up<F, B, S, 4, 1>(a, gu, max_entries, stream);
  const Launch dn = plan_launch(experts, max_entries, a.H / 32, a.I);
  if (dn.group > 1)
    launch_down<F, B, S, 4, kGroup>(a, dn, max_entries, stream);
  else if (dn.nst == 1)
    launch_down<F, B, S, 1, 1>(a, dn, max_entries, stream);
  else if (dn.nst == 2)
    launch_down<F, B, S, 2, 1>(a, dn, max_entries, stream);
  else if (dn.nst == 3)
    launch_down<F, B, S, 3, 1>(a, dn, max_entries, stream);
  else
    launch_down<F, B, S, 4, 1>(a, dn, max_entries, stream);
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
