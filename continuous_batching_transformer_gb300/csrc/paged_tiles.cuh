// paged_tiles.cuh -- attention of ragged runs of query tokens over pages, in tiles of 128 tensor-core
// rows: units of work, how CTAs find theirs, how long rows are cut and their partial outputs joined.
// Shared by the kernels over bf16 and over 8-bit pages.
#pragma once
#include <math.h>

#include "paged_attn.cuh"

namespace {

constexpr int kRows = 128;      // tensor-core rows of a tile
constexpr int kStep = 64;       // keys of a step
constexpr int kLag = 2;         // V of a step is multiplied with the scores of the step kLag behind it

// 32 consecutive 32-bit columns of this thread's TMEM lane
CBT_D void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
CBT_D void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 2^-n for a whole n >= 0 (n NaN or beyond the range: 0)
CBT_D float pow2_down(float n) { return n <= 126.f ? __int_as_float((127 - (int)n) << 23) : 0.f; }
// 32 bytes to 16-byte aligned global memory; wide: 32-byte aligned
CBT_D void store32(void* p, const uint32_t (&v)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    static_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}
CBT_D float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
struct Unit {
  int b, t0, n;  // row; its query tokens [t0, t0 + n) of this unit
  int p0;        // position of token t0 (may be negative)
  int g;         // kv head
  int s0, s1;    // the steps [s0, s1) of the unit that this item takes
  int run;       // which of the unit's runs they are
};
constexpr int kUnits = 48;   // most units of a CTA
constexpr int kRanked = 64;  // rows up to which they are ranked
constexpr int kScratch = 16 * kRanked;

// Few units over long contexts: a unit's steps are cut into up to `runs` runs of kRunSteps steps or
// more, taken by different CTAs and joined by k_prefill_merge (runs_for decides).
// Whole and cut, rows of 4 tokens, 32 q and 8 kv heads of 128: one over 2000 positions 28 and 17 us, over
// 131072 1454 and 98 us (5.4 TB/s of K and V); ten over 8192 100 and 77 us.  One row of 512 tokens over
// 16384: 202 and 121 us.  With runs of 16 steps the first takes 21 us.
constexpr int kRunSteps = 8;
constexpr int kSms = 152, kMostRuns = 64;
constexpr int kMostItems = 4 * kSms;  // that the runs may make
CBT_HD int ceil_div(int n, int d) { return (n + d - 1) / d; }
// The steps of each run of a unit, the last one's aside, and how many runs hold any: every one of them
// is written, and those behind are not read.
CBT_HD int run_length(int steps, int runs) {
  const int most = ceil_div(steps, kRunSteps);
  return most <= 1 ? (steps > 0 ? steps : 1) : ceil_div(steps, runs < most ? runs : most);
}
CBT_HD int run_count(int steps, int runs) {
  return steps > 0 ? ceil_div(steps, run_length(steps, runs)) : 1;
}

// What the roles derive from a unit.  Its steps are the 64-key chunks that any of its queries sees; a
// tile takes part in those that its own see.
template <class A>
struct Work {
  Unit u;
  int pl, lo_win;  // positions of the last token and of the first token's window
  Seen seen;
  int steps, stages;  // steps of the item, and kLag more
  CBT_D Work(const Unit* s, const A& a)
      : u{uniform(s->b), uniform(s->t0), uniform(s->n), uniform(s->p0), uniform(s->g), uniform(s->s0),
          uniform(s->s1)} {
    pl = u.p0 + u.n - 1;
    lo_win = first_in_window(max(0, u.p0), a.window);
    seen = seen_chunks<kStep>(u.p0, pl, a.window, a.sinks);
    steps = u.s1 - u.s0;
    stages = steps > 0 ? steps + kLag : 0;
  }
  CBT_D int key(int i) const { return seen.chunk(u.s0 + i) * kStep; }  // the first of step i
};
struct TileKeys {
  int last, lo;  // positions of the tile's last token and of its first token's window
  template <class A>
  CBT_D TileKeys(const Work<A>& w, const A& a, int x, int TQ) {
    const int first = w.u.p0 + x * TQ;
    last = x * TQ < w.u.n ? min(w.pl, first + TQ - 1) : -1;
    lo = first_in_window(max(0, first), a.window);
  }
  CBT_D bool need(int key, int sinks) const { return key <= last && (key + kStep > lo || key < sinks); }
};

// This CTA's units, found by all of its THREADS threads; returns how many (the caller's barrier comes
// next).  scratch: kScratch bytes, where Q lands later; warp_sums: a word a warp.
//
// Items are (unit, kv head), dealt to the CTAs forth and back.  With few rows the units are ranked by
// their last position (the longest first), each by a thread that counts the units before it; with many
// they are taken as they come, the rows' last units first: there are enough of them then to even out.
// (Four 1024-token prompts over bf16 pages: 56 us unranked.)
// Rows whose ranges of tokens overlap may hold more units than the `most` that the launch and the
// counters here are sized for: none is done then (some range runs backwards, which is reported).
template <int THREADS, class A>
CBT_D int find_units(const A& a, Unit* units, uint8_t* scratch, int* warp_sums, int TQ, int runs, int most) {
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31, Hkv = a.kv.n_kv_heads;
  const int grid = gridDim.x;
  auto item_of = [&](int round) {  // items are below 2^31, one round past them in 32 bits too
    return (unsigned)round * grid + (round & 1 ? grid - 1 - blockIdx.x : blockIdx.x);
  };
  // tokens / (2 TQ), by multiplication where that is exact (a dividend below 2^24, a divisor of 256
  // at most): a division a row and unit was a third of the search
  const unsigned inv = 0xFFFFFFFFu / (2 * TQ) + 1;
  auto in_units = [&](int n) { return n >> 24 ? n / (2 * TQ) : 2 * TQ == 1 ? n : (int)__umulhi(n, inv); };
  int total = 0;
  auto units_of = [&](int n) { return n > 0 ? in_units(n - 1) + 1 : 0; };
  if (a.rows <= kRanked) {
    struct Row {
      int t0, n, p0, k;  // query tokens, their number, the first one's position, units
    };
    Row* rows = reinterpret_cast<Row*>(scratch);  // before Q lands there
    static_assert(sizeof(Row) * kRanked == kScratch, "what the scratch holds");
    if (tid < a.rows) {
      const RowTokens row = row_tokens(a, tid);
      if (row.bad && blockIdx.x == 0) set_device_error(a.err, CBT_DEV_LENGTH, tid);
      rows[tid] = Row{row.t0, max(0, row.n), row.len - row.n, units_of(row.n)};
    }
    __syncthreads();
#pragma unroll 1
    for (int r = 0; r < a.rows; ++r) total += rows[r].k;
    if (total > most) total = 0;
#pragma unroll 1
    for (int q = tid; q < total; q += THREADS) {
      int r = 0, first = q;  // unit `first` of row r
      for (; first >= rows[r].k; ++r) first -= rows[r].k;
      const Row me = rows[r];
      const int end = min(me.n, (first + 1) * 2 * TQ), last = me.p0 + end - 1;
      int rank = 0;
#pragma unroll 1
      for (int o = 0; o < a.rows; ++o) {
        const Row w = rows[o];
        // units of row o that end at position t or later
        auto from = [&](int t) {
          const int d = t - w.p0 + 1;  // tokens up to t
          return d > w.n ? 0 : w.k - (d > 0 ? in_units(d - 1) : 0);
        };
        rank += from(last + (o < r ? 0 : 1));
      }
      const int p0 = me.p0 + first * 2 * TQ;
      const int steps = seen_chunks<kStep>(p0, last, a.window, a.sinks).n;
      const int per = run_length(steps, runs), cuts = run_count(steps, runs);
      unsigned round = (unsigned)rank * (Hkv * runs) / grid;
      int at = rank * (Hkv * runs) - round * grid;
#pragma unroll 1
      for (int e = 0; e < Hkv * runs; ++e, ++at) {
        if (at == grid) {
          at = 0;
          ++round;
        }
        if (at == (round & 1 ? grid - 1 - (int)blockIdx.x : (int)blockIdx.x) && round < kUnits) {
          const int g = e / runs, run = e - g * runs;  // past the unit's last run: no tokens, no steps
          units[round] = Unit{r, me.t0 + first * 2 * TQ, run < cuts ? end - first * 2 * TQ : 0, p0, g,
                              min(run * per, steps), min((run + 1) * per, steps), run};
        }
      }
    }
    tc::fence_proxy_async_smem();  // Q is written over the rows by the async proxy
  } else {
    const int per = (a.rows + THREADS - 1) / THREADS;
    const int r0 = min(a.rows, tid * per), r1 = min(a.rows, r0 + per);
    int mine = 0;
#pragma unroll 1
    for (int r = r0; r < r1; ++r) {
      const RowTokens row = row_tokens(a, r);
      if (row.bad && blockIdx.x == 0) set_device_error(a.err, CBT_DEV_LENGTH, r);
      mine = min(mine + units_of(row.n), most + 1);
    }
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    const int ws = lane < THREADS / 32 ? warp_sums[lane] : 0;  // lane w: warp w's sum
    total = __reduce_add_sync(0xffffffffu, ws);
    const int begin = __reduce_add_sync(0xffffffffu, lane < warp ? ws : 0) + inc - mine;
    if (total > most) total = 0;
#pragma unroll 1
    for (int round = 0; round < kUnits; ++round) {
      const unsigned it = item_of(round);
      if (it >= (unsigned)(total * Hkv)) break;
      const int u = total - 1 - (int)(it / Hkv);
      int at = begin;
      if (u >= begin && u < begin + mine) {
#pragma unroll 1
        for (int r = r0; r < r1; ++r) {
          const RowTokens row = row_tokens(a, r);
          const int k = units_of(row.n), first = (u - at) * 2 * TQ;
          if (u >= at && u < at + k) {
            const int n = min(2 * TQ, row.n - first), p0 = row.len - row.n + first;
            units[round] = Unit{r, row.t0 + first, n, p0, (int)(it % Hkv), 0,
                                seen_chunks<kStep>(p0, p0 + n - 1, a.window, a.sinks).n, 0};
          }
          at += k;
        }
      }
    }
  }
  int count = 0;  // only the last round is not full
  while (count < kUnits && item_of(count) < (unsigned)(total * Hkv * runs)) ++count;
  return count;
}

// Joins the runs of a (token, q head), W warps each: every warp finds the common reference and sum, a
// lane per run, then takes every W-th run's O, HD / 32 dims a lane; four warps' sums are added in
// order.  Four where few pairs have many runs and each one's chain of loads counts: 20 pairs of 12 runs
// 15.6 us with four and 17.2 with one, 2880 of 12 37.1 and 39.1.  One otherwise: 4096 pairs of 9 runs 30.7
// and 27.6, 512 pairs of 4 22.5 and 20.2, 19200 of 5 176 and 156.
template <int HD, int W, class A>
__global__ void __launch_bounds__(128)
    k_prefill_merge(const __grid_constant__ A a, const int runs, const float* __restrict__ part_o,
                    const float2* __restrict__ part_ml) {
  constexpr int R = HD / 32;
  __shared__ float sums[4][HD];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = W == 4 ? warp : 0;
  const unsigned pair = W == 4 ? blockIdx.x : blockIdx.x * 4 + warp;
  const int t = (int)(pair / a.n_heads), h = (int)(pair - (unsigned)t * a.n_heads);
  // The row that holds t, among kRanked or fewer: a lane looks at two of them (the ranges need not lie in
  // the rows' order, and some may be no ranges).  Before the wait: the blocks that hand over their runs
  // have themselves waited for whatever wrote the rows, before they let this launch begin.  (4 tokens over 2000
  // positions, bf16 pages: 16.1 us so, 16.5 behind the wait; ten rows of 4 over 8192 76.5 and 77.2.)
  auto look = [&](int r) { return r < a.rows ? row_tokens<true>(a, r) : RowTokens{0, -1, 0, true}; };
  const RowTokens lo = look(lane), hi = look(lane + 32);
  pdl_wait();
  pdl_launch();
  if (t >= a.tokens) return;
  const unsigned in_lo = __ballot_sync(0xffffffffu, lo.n > 0 && t >= lo.t0 && t - lo.t0 < lo.n);
  const unsigned in_hi = __ballot_sync(0xffffffffu, hi.n > 0 && t >= hi.t0 && t - hi.t0 < hi.n);
  if (!(in_lo | in_hi)) return;  // all warps of the pair
  const int src = __ffs(in_lo ? in_lo : in_hi) - 1;
  RowTokens row{};
  row.t0 = __shfl_sync(0xffffffffu, in_lo ? lo.t0 : hi.t0, src);
  row.n = __shfl_sync(0xffffffffu, in_lo ? lo.n : hi.n, src);
  row.len = __shfl_sync(0xffffffffu, in_lo ? lo.len : hi.len, src);
  const int width = 2 * (kRows / (a.n_heads / a.kv.n_kv_heads)), first = (t - row.t0) / width * width;
  const int p0 = row.len - row.n + first, pl = row.len - row.n + min(row.n, first + width) - 1;
  const int count = run_count(seen_chunks<kStep>(p0, pl, a.window, a.sinks).n, runs);
  const size_t base = (size_t)pair * runs;
  float m = -INFINITY, l = 0.f, acc[R];
  for (int i = lane; i < count; i += 32) m = fmaxf(m, __ldcg(part_ml + base + i).x);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
  for (int r = 0; r < R; ++r) acc[r] = 0.f;
#pragma unroll 1
  for (int i0 = 0; i0 < count; i0 += 32) {
    const float2 v = i0 + lane < count ? __ldcg(part_ml + base + i0 + lane) : make_float2(-INFINITY, 0.f);
    const float mine = v.x == -INFINITY ? 0.f : ex2(v.x - m);  // 0: a run of which the token sees nothing
    l += mine == 0.f ? 0.f : v.y * mine;
    const int n = min(32, count - i0);
#pragma unroll 4
    for (int j = sub; j < n; j += W) {
      const float wgt = __shfl_sync(0xffffffffu, mine, j);
      const float* o = part_o + (base + i0 + j) * HD + lane * R;
      float x[R];
      if (R == 4) {
        const float4 f = __ldcg(reinterpret_cast<const float4*>(o));
        x[0] = f.x;
        x[1] = f.y;
        x[R - 2] = f.z;
        x[R - 1] = f.w;
      } else {
        const float2 f = __ldcg(reinterpret_cast<const float2*>(o));
        x[0] = f.x;
        x[1] = f.y;
      }
#pragma unroll
      for (int r = 0; r < R; ++r)
        acc[r] = wgt == 0.f ? acc[r] : fmaf(x[r], wgt, acc[r]);  // what such a run left is not a number
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (W == 4) {
#pragma unroll
    for (int r = 0; r < R; ++r) sums[warp][lane * R + r] = acc[r];
    __syncthreads();
    if (warp) return;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int d = lane * R + r;
      acc[r] = (sums[0][d] + sums[1][d]) + (sums[2][d] + sums[3][d]);
    }
  }
  // a token before the row's first position sees nothing
  const bool nothing = row.len - row.n + t - row.t0 < 0;
  const long long at = t * a.out_ld + (long long)h * HD + lane * R;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float y = nothing ? 0.f : acc[r] / l;
    if (a.f32) static_cast<float*>(a.out)[at + r] = y;
    else static_cast<uint16_t*>(a.out)[at + r] = round_bf16(y);
  }
}
constexpr int kFewPairs = 20 * kSms, kManyRuns = 8;  // up to, and above which, they have four warps

// The most runs a unit is cut into (1: none), from rows, max_q and max_kv alone: the number that should
// take the least time, counted in steps (0.75 us).  Items go to the SMs in rounds; each costs its steps,
// 5 more to start and end, and the writing of its partial outputs (45 bytes a ns); the join costs 6
// and the reading of them all (5000 bytes a ns).  Over 25 shapes whose bounds were the rows' own the cut so
// chosen was at worst 2 % behind whole (two rows of 700 tokens over 6000: 157 and 155 us).  Bounds above
// the rows mislead it: one prompt of 512 tokens takes 15 us, 27 with max_kv 8192 and 31 with 131072; and
// rows of one token over 65536 next to that prompt stay whole, 735 us.  One item for each SM instead:
// ten rows of 4 over 8192 stay whole, 100 for 77 us.  (All of these over bf16 pages.)  Over 8-bit pages, where
// a step takes 0.97 us, the same counts chose a cut that was nowhere behind whole in 25 shapes, up to 5.8 times
// faster (4 tokens over 16000 positions: 31 and 181 us), and at worst 7 % behind the best of nine (the same: 29).
template <class A>
int runs_for(const A& a) {
  const int G = a.n_heads / a.kv.n_kv_heads, width = 2 * (kRows / G);  // tokens of a unit
  const long long units = (long long)a.rows * (((long long)a.max_q + width - 1) / width) * a.kv.n_kv_heads;
  if (a.rows > kRanked || units <= 0 || units > kMostItems / 2) return 1;
  double keys = a.max_kv;  // that a unit sees at most
  if (a.window) keys = fmin(keys, (double)a.window + width + a.sinks + 2 * kStep);
  const int steps = (int)((keys + kStep - 1) / kStep);
  const double step_ns = 750, row_bytes = a.kv.head_dim * sizeof(float);
  const double item = 5 + fmin((double)a.max_q * G, 2 * kRows) * row_bytes / 45 / step_ns;
  // (not a.tokens: a call of fewer tokens must not need more workspace)
  const double join = (double)a.rows * a.max_q * a.n_heads * row_bytes / 5000 / step_ns;
  int best = 1;
  double least = (double)((units + kSms - 1) / kSms) * (steps + 5);
  for (int n = 2; n <= kMostRuns && n * units <= kMostItems && (n - 1) * kRunSteps < steps; ++n) {
    const double t = (double)((n * units + kSms - 1) / kSms) * ((double)steps / n + item) + 6 + n * join;
    if (t < least) {
      least = t;
      best = n;
    }
  }
  return best;
}

}  // namespace
