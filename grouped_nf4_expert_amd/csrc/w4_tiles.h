// The loop over 4-bit weight tiles that the int4 linear and the expert layer's
// projections share.
//
// A work item is an entry -- up to 16 activation rows against one weight
// matrix, one matrix-core tile -- and U tiles of 16 weight rows.  The eight wavefronts of
// a workgroup form teams; a team owns an item, its wavefronts split the steps
// of K between them and their sums meet in LDS.  Workgroups stay resident (one
// or two per CU) and each team walks a contiguous range of items, so
//  * the decode table is made once;
//  * a wavefront always meets the same steps of K, and its activations (the
//    entry's rows at those steps) stay in registers until the entry changes:
//    read per item, they cost the address units four times what the weights
//    do;
//  * each wavefront loads weights ahead, across items and barriers: a CU must
//    keep tens of kilobytes in flight to draw its share of the HBM stream.  (More
//    is not better: five and seven steps of two tiles ahead instead of two and
//    three cost 5-9% of calls with a few items per team.)
// Measured on the gate_up of 64 experts' 4096 x 2048 matrices (49 us then): without
// the products 45, without scales 46, without both 42, without the ends of items
// 45: no single part bounds it but the stream and its start.
#pragma once

#include "w4_mfma.h"

namespace gnf4 {
namespace {

constexpr int kWaves = 8;
constexpr int kGroup = 2;  // items of a group that shares the activations of a pass
constexpr int kThreads = kWaves * kWave;

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

// The scales of an item in LDS: step s of row r (of 16 U) of a team, rows side by
// side, each step's a word further on so that a fetch's stores (neighbouring
// lanes hold neighbouring steps) meet different banks.
template <typename Scale, int U>
__device__ __forceinline__ int scale_at(int s, int r) {
  return s * (16 * U * (int)sizeof(Scale) + 4 * Scale::kWords) + r * (int)sizeof(Scale);
}
template <typename Scale, int U>
__device__ __forceinline__ int team_scales(int nst, int team, int wk) {
  return team * scale_at<Scale, U>(nst * wk, 0);
}
template <typename Scale, int U>
__host__ __device__ constexpr int scale_bytes(int nst) {
  return kWaves * nst * (16 * U * (int)sizeof(Scale) + 4 * Scale::kWords);
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
template <W4 F, int B, typename S, bool ZP, int NST, int G, int U, typename P>
__device__ __forceinline__ void expert_tiles(const P& p, const ItemGrid ig, int n_entries,
                                             char* lut, char* slds) {
  typedef ScaleWord<B, S, ZP> Scale;
  // steps held or in flight: 2 KB each with two tiles, 1 KB with one
  constexpr int kBufs =
      U == 1 && NST > 2 ? (NST % 3 == 0 ? 6 : NST == 7 ? 7 : 8) : NST == 3 ? 3 : 4;
  constexpr int kAhead = kBufs - 1;
  constexpr int kUnroll = G > 1 ? G : NST == 1 ? 4 : 2;  // items per turn of the loop
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
  uint32_t coff[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    coff[u] = (uint32_t)p.weight_row(u * 16 + col) * (uint32_t)kb + g * 16;
  const uint8_t* cbase;
  const auto first_row = [&](int j, int tile) {  // of the stack
    const uint32_t ev = (uint32_t)uniform((int)p.entry(j));
    return (size_t)read_entry(ev).e * p.expert_rows + (size_t)p.first_row(tile);
  };
  const auto set_item = [&]() { cbase = p.codes + first_row(lj, lt + lg) * (size_t)kb; };
  // One item (of a pass) on; past the last group the last one again.  A team with
  // a group less than its workgroup's other teams stores that one twice, so its
  // loads stay whole; past the last round, where nothing is used, a zero mask
  // leaves one line to read (1 token over 64 experts 27.7 -> 25.2 us).
  const auto step_on = [&](int& j, int& t, int& pass, int& item, int& rest, int& more,
                           uint32_t& mask) {
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
    if (more > 0)
      --more;
    else
      mask = 0u;
  };
  uint32_t lmask = ~0u, fmask = ~0u;
  int lmore = rounds - 1, fmore = rounds - 1;
  const auto load = [&](u32x4 (&w)[U], int i) {
    const int c = min((lp * wk + kw) * NST + i, steps - 1);
#pragma unroll
    for (int u = 0; u < U; ++u)
      w[u] = load_codes(cbase, c, coff[u], g, kb, lmask);
    if (i == NST - 1) {
      step_on(lj, lt, lp, lg, left, lmore, lmask);
      set_item();
    }
  };
  // Scales go through LDS: read by each lane from its own row they would cost
  // as many cache lines as the codes.  The team's threads fetch the item's
  // 2 x 16 rows of wk * NST steps in row order, two items ahead.
  constexpr int kSteps = 16 * U * NST, kFetch = (kSteps + 63) / 64;  // words per wavefront, per thread
  int fj = lj, ft = lt, fp = 0, fg = 0, fleft = left;
  uint32_t foff[kFetch];
  int fstep[kFetch], fat[kFetch];
#pragma unroll
  for (int i = 0; i < kFetch; ++i) {  // row, then step; threads left over repeat the last
    const int id = min(kw * kWave + lane + i * (wk * kWave), (kSteps << ig.log_wk) - 1);
    const int row = id / NST >> ig.log_wk;
    fstep[i] = id - ((row * NST) << ig.log_wk);
    foff[i] = (uint32_t)p.weight_row(row) * (uint32_t)blocks;
    if constexpr (G == 1) foff[i] += scales_first<B>(min(fstep[i], steps - 1), blocks);
    fat[i] = team_scales<Scale, U>(NST, team, wk) + scale_at<Scale, U>(fstep[i], row);
  }
  Scale fetched[2][kFetch];
  int fsteps[2] = {0, 0};  // the first step of a fetch
  const auto fetch = [&](int buf) {
    const size_t first = first_row(fj, ft + fg) * (size_t)blocks;
    if constexpr (G > 1) fsteps[buf] = fp * wk * NST;
#pragma unroll
    for (int i = 0; i < kFetch; ++i) {
      uint32_t at = foff[i];
      if constexpr (G > 1)
        at += scales_first<B>(min(fsteps[buf] + fstep[i], steps - 1), blocks);
      at &= fmask;
      load_scales<B, S, ZP, NST == 1>(p.scales + first, ZP ? p.zeros + first : nullptr, at, blocks,
                                      fetched[buf][i]);
    }
    step_on(fj, ft, fp, fg, fleft, fmore, fmask);
  };
  const auto put = [&](int buf) {
#pragma unroll
    for (int i = 0; i < kFetch; ++i) {
      align_scales<B, S, ZP>(fetched[buf][i], min(fsteps[buf] + fstep[i], steps - 1), blocks);
      *reinterpret_cast<Scale*>(slds + buf * scale_bytes<Scale, U>(NST) + fat[i]) = fetched[buf][i];
    }
  };
  // The entry's activations at this wavefront's steps of a pass, each row
  // scaled by its largest value there; `down` undoes it for the rows whose sums
  // the lane holds (the row of lane l here is l % 16, of its sums
  // 4 (l / 16) + r).
  u32x4 x[NST][4];
  f32x4 down;
  // kept as read until they are scaled, where the registers hold both
  constexpr bool kKeep = F == W4::kInt4 || (P::kKeepRaw && NST <= 4) || NST == 1;
  typename P::Raw keep[kKeep ? NST : 1][4];
  uint32_t xrow = 0;
  // Register i of a step lies in a block that is in the row or past it as a
  // whole (K is a multiple of the block); past it, the row's start is read and
  // multiplied by zero.
  // The positions are worked out where they are used: as constants of the loop
  // they would fill the scalar registers.
  const auto first_k = [&](int pass, int n) {
    int k = ((pass * wk + kw) * NST + n) * kStep;
    asm volatile("" : "+s"(k));
    return k;
  };
  const auto inside = [&](int k, int i) { return k + i / (B / 32) * B < K; };
  const auto raw = [&](int pass, int n) {
    const int first = first_k(pass, n);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = first + (k_of<B>(0, i) - k_of<B>(0, 0));
      keep[kKeep ? n : 0][i].load(p.x + (inside(first, i) ? k : 0), xrow);
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
    if constexpr (F == W4::kInt4) {  // bf16 as it is
#pragma unroll
      for (int n = 0; n < NST; ++n) {
        const int first = first_k(pass, n);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) x[n][i][q] = inside(first, i) ? keep[n][i].v[q] : 0u;
      }
      return;
    }
    uint32_t top = 0;
#pragma unroll
    for (int n = 0; n < NST; ++n) {
      if (!kKeep && n > 0) raw(pass, n);
      const int first = first_k(pass, n);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t m = keep[kKeep ? n : 0][i].max_bits();
        top = max(top, inside(first, i) ? m : 0u);
      }
      if constexpr (!kKeep && NST > 4) __builtin_amdgcn_sched_barrier(0);
    }
    top = max(top, (uint32_t)__shfl_xor((int)top, 16, kWave));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32, kWave));
    const RowScale rs = {(int)(top >> 23)};
    const float up = rs.up();
#pragma unroll
    for (int n = 0; n < NST; ++n) {
      if (!kKeep) raw(pass, n);
      const int first = first_k(pass, n);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[n][i] = keep[kKeep ? n : 0][i].half(inside(first, i) ? up : 0.0f);
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
  u32x4 w[kBufs][U];
#pragma unroll
  for (int n = 0; n < kAhead; ++n) load(w[n], n % NST);
  fetch(1);
  __builtin_amdgcn_sched_barrier(0);
  take_x(0);
  put(0);
  lds_barrier();
  // an item's steps of a pass; `it` is its position within a turn of the loop
  const auto item_steps = [&](int it, f32x4 (&acc)[U]) {
#pragma unroll
    for (int h = 0; h < U; ++h) acc[h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    fetch(it & 1);
    const char* mine = slds + (it & 1) * scale_bytes<Scale, U>(NST) +
                       team_scales<Scale, U>(NST, team, wk) + scale_at<Scale, U>(kw * NST, col);
#pragma unroll
    for (int n = 0; n < NST; ++n) {
      const int q = it * NST + n;
      load(w[(q + kAhead) % kBufs], (n + kAhead) % NST);
      __builtin_amdgcn_sched_barrier(0);  // the loads go first
      // idle steps past the row's end have zero activations
#pragma unroll
      for (int h = 0; h < U; ++h) {
        const Scale sc = *reinterpret_cast<const Scale*>(mine + scale_at<Scale, U>(n, h * 16));
        acc[h] = step_mac<F, B, S, ZP>(w[q % kBufs][h], sc, x[n], copy, acc[h]);
        // where registers are short, one tile's decode at a time
        if constexpr (G > 1 || F == W4::kMx4 || ZP || groups_per_cu(NST, G) > 1)
          __builtin_amdgcn_sched_barrier(0);
      }
    }
    put((it + 1) & 1);
#pragma unroll
    for (int h = 0; h < U; ++h)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if constexpr (F != W4::kInt4) acc[h][r] *= down[r];
  };
  // the wavefronts' sums of an item meet: [wave][tile][register][lane]
  int turn = 0;
  const auto meet = [&](const f32x4 (&acc)[U], int tile) {
    char* sums = lut + (turn & 1) * kSumBytes;
#pragma unroll
    for (int h = 0; h < U; ++h)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        *reinterpret_cast<float*>(
            sums + lds_half(((wave * U + h) * 4 + r) * kWave) + lds_half(lane) - 128) = acc[h][r];
    lds_barrier();
    p.finish(team, ig.log_wk, cj, tile, sums);
    ++turn;
  };
  if constexpr (G == 1) {
    for (;;) {
#pragma unroll
      for (int it = 0; it < kUnroll; ++it) {
        f32x4 acc[U];
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
      f32x4 total[G][U];
#pragma unroll
      for (int it = 0; it < G; ++it)
#pragma unroll
        for (int h = 0; h < U; ++h) total[it][h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      for (int pass = 0; pass < ig.passes; ++pass) {
        if (round + pass > 0) {
          issue_x(cj, pass);
          take_x(pass);
        }
#pragma unroll
        for (int it = 0; it < G; ++it) {
          f32x4 acc[U];
          item_steps(it, acc);
#pragma unroll
          for (int h = 0; h < U; ++h) total[it][h] += acc[h];
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
template <int U>
__device__ __forceinline__ float team_sum(const char* sums, int team, int log_wk, int tile, int o) {
  const char* p = sums + lds_half((((team << log_wk) * U + tile) << 8) + o);
  const auto at = [p](int k) {
    return *reinterpret_cast<const float*>(p + k * (U * 256 / 32 * 256));
  };
  float v = at(0) + at(1);
  if (log_wk > 1) v = v + at(2) + at(3);
  if (log_wk > 2) v = v + at(4) + at(5) + at(6) + at(7);
  return v;
}

// How a projection is launched.  Wavefronts per team, hence steps per
// wavefront: the widest team, with the fewest activations to load and hold per
// wavefront, unless a narrower one takes at least an eighth fewer steps in all
// when there are `entries` (a team wider than the row's steps has idle
// wavefronts).  Two steps per wavefront, two workgroups per CU, count a quarter
// more: they stream slower than four steps of one workgroup (64 experts' 4096 x
// 2048 matrices 49 against 43 us, 100 experts' 7168 x 2048 ones 243 against
// 217 us); one step of two workgroups does not (29 against 35 us with two steps
// over rows of 1024).  A wavefront holds the activations of at most max_nst
// steps; longer rows take passes of four steps by the whole workgroup.
struct Launch {
  unsigned grid;
  int nst, group;
  ItemGrid ig;
  int64_t cost;  // of the busiest CU's wavefronts, in quarter steps
};
inline Launch plan_launch(int entries, int max_entries, int tiles, int K, int max_nst) {
  const int steps = (K + kStep - 1) / kStep;
  const int64_t cus = device_cu_count(), items = (int64_t)entries * tiles;
  int best = 3, nst = (steps + 7) / 8, group = 1, passes = 1;
  int64_t cost = INT64_MAX;
  if (nst > max_nst) {
    passes = (nst + 3) / 4;
    nst = 4;
    group = kGroup;
    cost = (items + cus * group - 1) / (cus * group) * group * passes * nst * 4;
  } else {
    int64_t limit = INT64_MAX;
    for (int l = 3; l >= 1; --l) {
      const int n = (steps + (1 << l) - 1) >> l;
      const int64_t one = cus * (kWaves >> l), all = one * groups_per_cu(n, 1);
      const int64_t rounds = (items + all - 1) / all;
      const int64_t c = rounds * n * (items > one ? groups_per_cu(n, 1) * (n == 2 ? 5 : 4) : 4);
      if (n <= max_nst && c < limit) {
        best = l;
        nst = n;
        cost = c;
        limit = c * 7 / 8;
      }
    }
  }
  const int teams = kWaves >> best;
  const int64_t need = ((int64_t)max_entries * ((tiles + group - 1) / group) + teams - 1) / teams;
  const int64_t room = cus * groups_per_cu(nst, group);
  return Launch{(unsigned)(need < room ? need : room), nst, group,
                ItemGrid{tiles, K, best, passes}, cost};
}

}  // namespace
}  // namespace gnf4
