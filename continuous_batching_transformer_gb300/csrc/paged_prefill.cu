// paged_prefill.cu -- attention of ragged runs of query tokens over a paged KV cache.
//
// A unit is a run of query tokens of one row and one kv head, as two tiles of 128 tensor-core rows.
// A tile's rows are (token, q head) pairs: the q heads that read the kv head lie next to each other,
// so a tile holds 128 / G tokens with all G of their heads, a decode row or a short chunk fills its
// tile with heads, and one K and V tile serves all of them.  Per step of 64 keys and tile:
//   S = Q K^T       tcgen05.mma 128 x 64 x head_dim into tensor memory
//   softmax         one thread per row: the whole row of S in registers, running maximum and sum
//   O += P V        tcgen05.mma 128 x head_dim x 64, P read from tensor memory as bf16 where S was
// O stays in tensor memory for the whole unit.  A row's reference is its maximum so far, rounded up to
// a whole number of powers of two and raised (with a rescaling of O, exact) only when a step exceeds
// it by more than 2^kSlack: O is rarely touched, and weights stay below 2^kSlack.  P is rounded to
// bf16 once (at most 2^-8 of each weight, as the tensor cores take it), everything else is fp32.
//
// Long units are bound by the tensor cores and, close behind, the exponentials; a unit of one tile
// by its own chain of S, softmax and P V (0.7 to 0.8 us a step).  Each tile has an issuer warp and a
// softmax warpgroup of its own and two buffers of S, so that one step's MMAs run under another's
// softmax.  K and V come through two TMA maps over the whole pool (64 keys a request, each from its own
// page) into one ring of stages; a stage holds K of a step and V of the step kLag before it, which is
// when that is needed, so that an issuer waits once a step.  A warp of its own clears V of keys that
// no query of the unit sees (what lies there may not be finite) before the MMA reads it.  CTAs stay
// for several units, which they find from the rows' lengths: the longest first, dealt back and forth.
// Measured, 32 q and 8 kv heads of 128: four prompts of 1024 tokens 40.7 to 41.1 us (840 TFLOP/s);
// four chunks of 500 to 1030 tokens over 3000 to 9000 positions, window 4096, 168.5 to 169.8 us (1095
// TFLOP/s).
#include <math.h>

#include "paged_attn.cuh"

namespace {

constexpr int kRows = 128;      // tensor-core rows of a tile
constexpr int kStep = 64;       // keys of a step
constexpr int kBox = 16384;     // [128 rows][64 bf16], swizzled
constexpr int kStages = 5;
constexpr int kLag = 2;         // a stage holds K of a step and V of the step kLag before it
constexpr int kThreads = 384;   // warps: tiles, issuer 0, issuer 1, V; 4..7 and 8..11 softmax
constexpr float kSlack = 8.f;

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
CBT_D void tma_load_q(void* dst, const CUtensorMap* m, uint64_t* bar, int x, int head, int tok) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(tc::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(tc::smem_u32(bar)), "r"(x), "r"(head), "r"(tok)
      : "memory");
}

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
// A shared-memory matrix descriptor (tc::sdesc_sw128) as two words: the high one is the same for
// every tile, the low one counts in 16-byte units and is moved by additions.
CBT_D uint32_t desc_lo(const void* p) { return (uint32_t)tc::sdesc_sw128(tc::smem_u32(p)); }
CBT_D uint64_t desc(uint32_t lo) {
  constexpr uint32_t hi = (uint32_t)((((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61)) >> 32);
  return ((uint64_t)hi << 32) | lo;
}
// the k-th 16-deep step of a tile whose 64-column boxes are `box` bytes apart
CBT_HD constexpr uint32_t step_of(int k, int box) { return (uint32_t)((k >> 2) * (box >> 4) + 2 * (k & 3)); }

struct Unit {
  int b, t0, n;  // row; its query tokens [t0, t0 + n) of this unit
  int p0;        // position of token t0 (may be negative)
  int g;         // kv head
  int s0, s1;    // the steps [s0, s1) of the unit that this item takes
  int run;       // which of the unit's runs they are
};
constexpr int kUnits = 48;   // most units of a CTA
constexpr int kRanked = 64;  // rows up to which they are ranked

// Shared memory: the tiles of Q, K and V, then this
constexpr int kBars = 2 + 3 * kStages + 12;
struct Tail {
  uint64_t bars[kBars];
  uint32_t tmem_slot;
  int abort_flag;
  int warp_sums[kThreads / 32];
  Unit units[kUnits];
};
template <int HD>
constexpr size_t smem_bytes() {  // 1024: the base is rounded up to the tiles' alignment
  return 1024 + 2 * (HD / 64) * kBox + 2 * kStages * kStep * HD * 2 + sizeof(Tail);
}
static_assert(smem_bytes<64>() <= 227 * 1024 && smem_bytes<128>() <= 227 * 1024, "shared memory");

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
struct Work {
  Unit u;
  int pl, lo_win;  // positions of the last token and of the first token's window
  Seen seen;
  int steps, stages;  // steps of the item, and kLag more
  CBT_D Work(const Unit* s, const PagedAttn& a)
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
  CBT_D TileKeys(const Work& w, const PagedAttn& a, int x, int TQ) {
    const int first = w.u.p0 + x * TQ;
    last = x * TQ < w.u.n ? min(w.pl, first + TQ - 1) : -1;
    lo = first_in_window(max(0, first), a.window);
  }
  CBT_D bool need(int key, int sinks) const { return key <= last && (key + kStep > lo || key < sinks); }
};

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
    k_paged_prefill(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                    const __grid_constant__ CUtensorMap tv, const __grid_constant__ PagedAttn a,
                    const int runs, const int most, float* __restrict__ part_o,
                    float2* __restrict__ part_ml) {
  constexpr int nKh = HD / 64;
  constexpr uint32_t kTile = nKh * kBox;     // a Q tile
  constexpr uint32_t kKV = kStep * HD * 2;   // K or V of a step
  constexpr uint32_t kIdescS = tc::idesc_bf16(128, kStep), kIdescO = tc::idesc_bf16(128, HD);
  constexpr uint32_t kTmem = 512;  // S (P over it): tile x, buffer b at 128 x + 64 b; O: 256 + HD x
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sQ = smem;                     // [tile][64-dim half][128 rows]
  uint8_t* sK = sQ + 2 * kTile;           // [stage][64-dim half][64 keys]
  uint8_t* sV = sK + kStages * kKV;       // [stage][HD dims][64 keys]
  Tail& tail = *reinterpret_cast<Tail*>(sV + kStages * kKV);
  uint64_t* bars = tail.bars;
  // a stage has landed, its V is clean, both tiles are done with it
  uint64_t *qfull = bars, *full = bars + 1, *ready = full + kStages, *empty = ready + kStages;
  // [tile][buffer]: S is there, P is there, P has been read (and its product is in O)
  uint64_t *s_full = empty + kStages, *p_full = s_full + 4, *pv_done = p_full + 4;
  uint64_t* qempty = pv_done + 4;         // both tiles' S of a unit are done
  uint32_t* tmem_slot = &tail.tmem_slot;
  volatile int* abort_flag = &tail.abort_flag;
  int* wsum = tail.warp_sums;
  Unit* units = tail.units;

  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const int H = a.n_heads, Hkv = a.kv.n_kv_heads, G = H / Hkv;
  const int TQ = kRows / G;  // tokens per tile
  if (tid == 0) {
    for (int i = 0; i < kBars; ++i) tc::mbar_init(&bars[i], 1);
    for (int i = 0; i < kStages; ++i) tc::mbar_init(&empty[i], 2);  // both issuers
    for (int i = 0; i < 4; ++i) tc::mbar_init(&p_full[i], 4);       // a tile's softmax warps
    tc::mbar_init(qempty, 2);
    *abort_flag = 0;
    tc::mbar_fence_init();
    tc::tma_prefetch_desc(&tq);
    tc::tma_prefetch_desc(&tk);
    tc::tma_prefetch_desc(&tv);
  }
  if (warp == 1) tc::tmem_alloc(tmem_slot, kTmem);
  pdl_wait();
  const int grid = gridDim.x;
  auto item_of = [&](int round) {  // items are below 2^31, one round past them in 32 bits too
    return (unsigned)round * grid + (round & 1 ? grid - 1 - blockIdx.x : blockIdx.x);
  };
  // tokens / (2 TQ), by multiplication where that is exact (a dividend below 2^24, a divisor of 256
  // at most): a division a row and unit was a third of the search
  const unsigned inv = 0xFFFFFFFFu / (2 * TQ) + 1;
  auto in_units = [&](int n) { return n >> 24 ? n / (2 * TQ) : 2 * TQ == 1 ? n : (int)__umulhi(n, inv); };
  // ---- this CTA's units.  Items are (unit, kv head), dealt to the CTAs forth and back.  With few rows
  // the units are ranked by their last position (the longest first), each by a thread that counts
  // the units before it; with many they are taken as they come, the rows' last units first: there
  // are enough of them then to even out.  (Four 1024-token prompts: 56 us unranked.)
  // Rows whose ranges of tokens overlap may hold more units than the `most` that the launch and the
  // counters here are sized for: none is done then (some range runs backwards, which is reported).
  int total = 0;
  auto units_of = [&](int n) { return n > 0 ? in_units(n - 1) + 1 : 0; };
  if (a.rows <= kRanked) {
    struct Row {
      int t0, n, p0, k;  // query tokens, their number, the first one's position, units
    };
    Row* rows = reinterpret_cast<Row*>(sQ);  // before Q lands there
    static_assert(kRanked * sizeof(Row) <= 2 * kTile, "rows fit where Q goes");
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
    for (int q = tid; q < total; q += kThreads) {
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
    const int per = (a.rows + kThreads - 1) / kThreads;
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
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    const int ws = lane < kThreads / 32 ? wsum[lane] : 0;  // lane w: warp w's sum
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
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  count = uniform(count);
  const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);
  const int sinks = a.window ? a.sinks : 0;

  if (warp == 0) {
    // ---- tile requests: per stage K of a step and V of the step kLag before.  The pages of 32 steps
    // are looked up at once, a lane each (one dependent load a step was as long as the step).
    const uint64_t pol = tc::policy_evict_last();
    const int P = a.kv.page_tokens;
    int st = 0, n = 0;  // stage, stages requested
    uint32_t ph = 0, qp = 0;
    int qn = 0;         // units whose Q was requested
    bool ok = true;
#pragma unroll 1
    for (int k = 0; k < count && ok; ++k) {
      const Work w(units + k, a);
      if (!w.stages) continue;
      int krow = 0, vrow = 0, vlag[kLag] = {0, 0};
      const int q_at = qn ? kLag : 0;  // the step before which Q is asked for
#pragma unroll 1
      for (int i = 0; i < w.stages; ++i) {
        if ((i & 31) == 0 && i + lane < w.steps) {
          const int key = w.key(i + lane), pg = key / P, o = key - pg * P;
          int id = a.table[(size_t)w.u.b * a.max_pages + pg];
          if (id < 0 || id >= a.kv.n_pages) {
            set_device_error(a.err, CBT_DEV_PAGE_ID, w.u.b);
            id = 0;  // a page that exists: the row's outputs are unspecified
          }
          krow = (int)(paged_k(a.kv, id, w.u.g, o, 0) / HD);
          vrow = (int)(paged_v(a.kv, id, w.u.g, o, 0) / 64);
        }
        // Q once both tiles have had the last unit's.  K of the first steps needs only stages that the last
        // unit has left, so after the first unit it is asked for before (four prompts of 1024 tokens
        // 41.5 to 40.7 us; for the first unit it would only be in Q's way).
        if (i == q_at) {
          ok = __all_sync(0xffffffffu, wait_or_abort(qempty, qp ^ 1, abort_flag));
          if (!ok) break;
          qp ^= 1;
          ++qn;
          if (lane == 0) {
            const int tiles = w.u.n > TQ ? 2 : 1;
            tc::mbar_expect_tx(qfull, tiles * nKh * G * TQ * 128);
#pragma unroll 1
            for (int x = 0; x < tiles; ++x)
              for (int h = 0; h < nKh; ++h)
                tma_load_q(sQ + x * kTile + h * kBox, &tq, qfull, h * 64, w.u.g * G, w.u.t0 + x * TQ);
          }
          __syncwarp();
        }
        const int kr = __shfl_sync(0xffffffffu, krow, i & 31), vr = __shfl_sync(0xffffffffu, vrow, i & 31);
        ok = __all_sync(0xffffffffu, wait_or_abort(&empty[st], ph ^ 1, abort_flag));
        if (!ok) break;
        const bool has_k = i < w.steps, has_v = i >= kLag;
        if (elect_one()) {
          tc::mbar_expect_tx(&full[st], (has_k ? kKV : 0) + (has_v ? kKV : 0));
          if (has_k) {
#pragma unroll
            for (int h = 0; h < nKh; ++h)
              tc::tma_load_2d(sK + st * kKV + h * (kBox / 2), &tk, &full[st], h * 64, kr, pol);
          }
          if (has_v) tc::tma_load_2d(sV + st * kKV, &tv, &full[st], 0, vlag[0], pol);
        }
        ++n;
        st = st + 1 == kStages ? 0 : st + 1;
        ph ^= st == 0;
        vlag[0] = vlag[1];
        vlag[1] = vr;
      }
    }
    if (lane == 0) {
      if (!ok) wait_timeout(a.err, abort_flag, 11);
      // no copies in flight at exit
      if (qn) wait_landed(qfull, (qn - 1) & 1);
#pragma unroll 1
      for (int i = max(0, n - kStages); i < n; ++i) wait_landed(&full[i % kStages], (i / kStages) & 1);
    }
  } else if (warp <= 2) {
    // ---- MMA issue of tile x: per stage P V of the step kLag before, then S of the step into the
    // buffer this freed.  So a step's scores are there before the softmax asks for them, and it
    // never waits for its own P V.
    const int x = warp - 1;
    const uint32_t s_tm = tmem + x * 128, o_tm = tmem + 256 + x * HD;
    const uint32_t dq = desc_lo(sQ + x * kTile), dk = desc_lo(sK), dv = desc_lo(sV);
    int st = 0;
    uint32_t ph = 0, pp = 0, qp = 0;  // phases of the stages, of p_full (bit b: buffer b) and of Q
    bool ok = true;
#pragma unroll 1
    for (int k = 0; k < count && ok; ++k) {
      const Work w(units + k, a);
      if (!w.stages) continue;
      const TileKeys mine(w, a, x, TQ);
      uint32_t took = 0;  // bit j: the tile took part in the step j before this one
      uint32_t acc = 0;   // O holds something of this unit
      ok = __all_sync(0xffffffffu, wait_or_abort(qfull, qp, abort_flag));
      qp ^= 1;
#pragma unroll 1
      for (int i = 0; i < w.stages && ok; ++i) {
        const int b = i & 1;
        const bool need = i < w.steps && mine.need(w.key(i), sinks);
        const bool due = took >> (kLag - 1) & 1;
        ok = __all_sync(0xffffffffu, wait_or_abort(&ready[st], ph, abort_flag));
        if (due) ok = ok && __all_sync(0xffffffffu, wait_or_abort(&p_full[2 * x + b], pp >> b & 1, abort_flag));
        if (!ok) break;
        tc::tc_fence_after();
        if (elect_one()) {
          if (due) {
            const uint32_t v = dv + st * (kKV >> 4);
#pragma unroll
            for (int e = 0; e < kStep / 16; ++e)
              tc::mma_bf16_ta(o_tm, s_tm + 64 * b + 8 * e, desc(v + 2 * e), kIdescO, (acc || e > 0) ? 1u : 0u);
            tc::mma_commit(&pv_done[2 * x + b]);
          }
          if (need) {
            const uint32_t kd = dk + st * (kKV >> 4);
#pragma unroll
            for (int e = 0; e < HD / 16; ++e)
              tc::mma_bf16(s_tm + 64 * b, desc(dq + step_of(e, kBox)), desc(kd + step_of(e, kBox / 2)), kIdescS,
                           e > 0 ? 1u : 0u);
            tc::mma_commit(&s_full[2 * x + b]);
          }
          tc::mma_commit(&empty[st]);
          if (i == w.steps - 1) tc::mma_commit(qempty);
        }
        if (due) {
          pp ^= 1u << b;
          acc = 1;
        }
        took = took << 1 | (need ? 1u : 0u);
        st = st + 1 == kStages ? 0 : st + 1;
        ph ^= st == 0;
      }
    }
    if (!ok && lane == 0) wait_timeout(a.err, abort_flag, 12);
  } else if (warp == 3) {
    // ---- V of keys that no query of the unit sees is cleared
    bool ok = true;
    int st = 0;
    uint32_t ph = 0;
#pragma unroll 1
    for (int k = 0; k < count && ok; ++k) {
      const Work w(units + k, a);
#pragma unroll 1
      for (int i = 0; i < w.stages && ok; ++i) {
        ok = __all_sync(0xffffffffu, wait_or_abort(&full[st], ph, abort_flag));
        if (!ok) break;
        uint32_t bits[2] = {~0u, ~0u};
        if (i >= kLag) seen_bits(w.key(i - kLag), w.pl, w.lo_win, sinks, bits);
        if ((bits[0] & bits[1]) != 0xFFFFFFFFu) {
          uint8_t* v = sV + st * kKV;
#pragma unroll 1
          for (int u = 0; u < 8; ++u) {  // 8 keys
            const uint32_t m8 = ((u < 4 ? bits[0] : bits[1]) >> (8 * (u & 3))) & 0xFFu;
            if (m8 == 0xFFu) continue;
            const uint4 mk = key_mask(m8);
            for (int d = lane; d < HD; d += 32) {
              uint4* p = reinterpret_cast<uint4*>(v + d * 128 + ((u ^ (d & 7)) << 4));
              uint4 z = make_uint4(0, 0, 0, 0);
              if (m8) z = *p;
              *p = make_uint4(z.x & mk.x, z.y & mk.y, z.z & mk.z, z.w & mk.w);
            }
          }
          tc::fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0) tc::mbar_arrive(&ready[st]);
        st = st + 1 == kStages ? 0 : st + 1;
        ph ^= st == 0;
      }
    }
    if (!ok && lane == 0) wait_timeout(a.err, abort_flag, 13);
  } else {
    // ---- softmax of tile x: thread = row
    const int x = (warp - 4) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_tm = tmem + x * 128 + lane_off, o_tm = tmem + 256 + x * HD + lane_off;
    // Scores in units of log2.  A negative scale negates them first, so that the largest product is
    // the largest score's; a zero scale stands for one that leaves every weight 1 (a masked -inf
    // must stay -inf).
    const bool negate = a.scale < 0.f;
    const float scale2 = fmaxf(fabsf(a.scale) * kLog2e, 1e-37f);
    uint32_t sp = 0;  // phases of s_full to come (bit b: buffer b)
    bool ok = true;
    // rows of out on 32-byte boundaries: whole sectors a store
    const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0 && a.out_ld % (a.f32 ? 8 : 16) == 0;
#pragma unroll 1
    for (int unit = 0; unit < count && ok; ++unit) {
      const Work w(units + unit, a);
      const TileKeys mine(w, a, x, TQ);
      const int tok = x * TQ + row / G;  // token of the unit
      const bool live = row < TQ * G && tok < w.u.n;
      const int p = live ? w.u.p0 + tok : -1;  // -1: sees nothing
      // rows that hold no token are left unmasked: what they compute is not stored
      const int hi = live ? p : 0x3FFFFFFF, lo = live ? first_in_window(max(0, p), a.window) : 0;
      float m = -INFINITY, l = 0.f;  // the reference (a maximum so far, rounded up) and the sum
      int done = -1;                 // the last step done
#pragma unroll 1
      for (int i = 0; i < w.steps && ok; ++i) {
        const int k0 = w.key(i);
        if (!mine.need(k0, sinks)) continue;
        const int b = i & 1;
        ok = __all_sync(0xffffffffu, wait_or_abort(&s_full[2 * x + b], sp >> b & 1, abort_flag));
        if (!ok) break;
        sp ^= 1u << b;
        tc::tc_fence_after();
        uint32_t s[64];
        tmem_ld32(s_tm + 64 * b, s);
        tmem_ld32(s_tm + 64 * b + 32, s + 32);
        tc::tmem_ld_wait();
        if (negate) {
#pragma unroll
          for (int e = 0; e < 64; ++e) s[e] ^= 0x80000000u;
        }
        // every row sees every key of the step, or keys are masked one by one
        if (!__all_sync(0xffffffffu, hi >= k0 + 63 && (lo <= k0 || sinks >= k0 + 64))) {
          uint32_t bits[2];
          seen_bits(k0, hi, lo, sinks, bits);
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if (!((bits[e >> 5] >> (e & 31)) & 1)) s[e] = 0xFF800000u;  // -inf
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 32; ++e)
          mx[e & 3] = max3(mx[e & 3], __uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]));
        const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * scale2;
        const bool up = m == -INFINITY ? top > -INFINITY : top > m + kSlack;
        if (__any_sync(0xffffffffu, up)) {
          // Rows that exceed their reference by more than 2^kSlack, or see their first keys, raise
          // it, to a whole number: what the old one has scaled is multiplied by a power of two,
          // which rounds nothing.
          const float next = up ? ceilf(top) : m;
          const float f = m == -INFINITY ? 0.f : pow2_down(next - m);  // m = -inf: l and O are zero
          m = next;
          l *= f;
          if (done >= 0) {
            // O is at rest once the last step's product is in it (S of this step, there already, was
            // issued after those before)
            const int d = done & 1;
            ok = __all_sync(0xffffffffu, wait_or_abort(&pv_done[2 * x + d], (sp >> d & 1) ^ (d != b), abort_flag));
            if (!ok) break;
            tc::tc_fence_after();
#pragma unroll 1
            for (int d = 0; d < HD; d += 16) {
              uint32_t o[16];
              tc::tmem_ld16(o_tm + d, o);
              tc::tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st16(o_tm + d, o);
            }
          }
        }
        const float ref = m == -INFINITY ? 0.f : m;
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float p0 = ex2(fmaf(__uint_as_float(s[2 * e]), scale2, -ref));
          const float p1 = ex2(fmaf(__uint_as_float(s[2 * e + 1]), scale2, -ref));
          part[e & 3] += p0;
          part[(e + 2) & 3] += p1;
          s[e] = pack_bf16(p0, p1);
        }
        tc::tmem_st32(s_tm + 64 * b, s);  // over the scores
        tc::tmem_st_wait();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&p_full[2 * x + b]);
        l += (part[0] + part[1]) + (part[2] + part[3]);
        done = i;
      }
      // The row goes straight out (through shared memory and in whole lines it took as long).  O is
      // not written again before this tile hands in weights of the next unit.
      if (ok && done >= 0) {
        const int d = done & 1;
        ok = __all_sync(0xffffffffu, wait_or_abort(&pv_done[2 * x + d], (sp >> d & 1) ^ 1, abort_flag));
        tc::tc_fence_after();
      }
      if (!ok) break;
      // a run of several hands over O as it is, with its reference and sum
      const int head = w.u.g * G + row % G;
      const size_t part = ((size_t)(w.u.t0 + tok) * H + head) * runs + units[unit].run;
      const float inv = runs > 1 ? 1.f : p >= 0 ? 1.f / l : 0.f;
      if (runs > 1 && live) part_ml[part] = make_float2(m, l);
      const long long at = (long long)(w.u.t0 + tok) * a.out_ld + (long long)head * HD;
#pragma unroll 1
      for (int k = 0; k < HD; k += 16) {
        uint32_t o[16];
        if (done >= 0) {
          tc::tmem_ld16(o_tm + k, o);
          tc::tmem_ld_wait();
        }
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = p >= 0 ? __uint_as_float(o[e]) * inv : 0.f;
        if (!live) continue;
        if (a.f32 || runs > 1) {
          float* dst = runs > 1 ? part_o + part * HD + k : static_cast<float*>(a.out) + at + k;
#pragma unroll
          for (int e = 0; e < 16; e += 8) {
            uint32_t h[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) h[j] = __float_as_uint(v[e + j]);
            store32(dst + e, h, wide || runs > 1);
          }
        } else {
          uint32_t h[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) h[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
          store32(static_cast<uint16_t*>(a.out) + at + k, h, wide);
        }
      }
      tc::tc_fence_before();
    }
    if (!ok && lane == 0) wait_timeout(a.err, abort_flag, 14);
    tc::tc_fence_before();
  }
  pdl_launch();
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, kTmem);
  }
}

// Joins the runs of a (token, q head), W warps each: every warp finds the common reference and sum, a
// lane per run, then takes every W-th run's O, HD / 32 dims a lane; four warps' sums are added in
// order.  Four where few pairs have many runs and each one's chain of loads counts: 20 pairs of 12 runs
// 15.6 us with four and 17.2 with one, 2880 of 12 37.1 and 39.1.  One otherwise: 4096 pairs of 9 runs 30.7
// and 27.6, 512 pairs of 4 22.5 and 20.2, 19200 of 5 176 and 156.
template <int HD, int W>
__global__ void __launch_bounds__(128)
    k_prefill_merge(const __grid_constant__ PagedAttn a, const int runs, const float* __restrict__ part_o,
                    const float2* __restrict__ part_ml) {
  constexpr int R = HD / 32;
  __shared__ float sums[4][HD];
  pdl_wait();
  pdl_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = W == 4 ? warp : 0;
  const unsigned pair = W == 4 ? blockIdx.x : blockIdx.x * 4 + warp;
  const int t = (int)(pair / a.n_heads), h = (int)(pair - (unsigned)t * a.n_heads);
  if (t >= a.tokens) return;
  // the row that holds t, among kRanked or fewer: a lane looks at two of them (the ranges need not lie in
  // the rows' order, and some may be no ranges)
  auto look = [&](int r) { return r < a.rows ? row_tokens(a, r) : RowTokens{0, -1, 0, true}; };
  const RowTokens lo = look(lane), hi = look(lane + 32);
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
// ten rows of 4 over 8192 stay whole, 100 for 77 us.
int runs_for(const PagedAttn& a) {
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

template <int HD>
cudaError_t launch_hd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                      const PagedAttn& a, int num_sms, cudaStream_t s) {
  constexpr size_t smem = smem_bytes<HD>();
  const cudaError_t rc = cudaFuncSetAttribute(k_paged_prefill<HD>,
                                              cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (rc != cudaSuccess) return rc;
  const int G = a.n_heads / a.kv.n_kv_heads, run = 2 * (kRows / G);
  // most units: every row may end in a partly filled one
  const long long by_tokens = (long long)a.tokens / run + a.rows;
  const long long by_rows = (long long)a.rows * ((a.max_q + run - 1) / run);
  const long long units = by_tokens < by_rows ? by_tokens : by_rows;
  const int runs = runs_for(a);
  const long long items = units * a.kv.n_kv_heads * runs, least = (items + kUnits - 1) / kUnits;
  const long long grid = items < num_sms ? items : least > num_sms ? least : num_sms;
  float* po = reinterpret_cast<float*>(a.ws);
  const size_t parts = (size_t)a.tokens * a.n_heads * runs;
  float2* pml = reinterpret_cast<float2*>(a.ws + parts * HD * sizeof(float));
  const cudaError_t launched = launch_pdl(k_paged_prefill<HD>, dim3((unsigned)grid), dim3(kThreads), smem, s,
                                          tq, tk, tv, a, runs, (int)units, po, pml);
  if (launched != cudaSuccess || runs == 1) return launched;
  const long long pairs = (long long)a.tokens * a.n_heads;
  if (pairs <= kFewPairs && runs > kManyRuns)
    return launch_pdl(k_prefill_merge<HD, 4>, dim3((unsigned)pairs), dim3(128), 0, s, a, runs, po, pml);
  return launch_pdl(k_prefill_merge<HD, 1>, dim3((unsigned)((pairs + 3) / 4)), dim3(128), 0, s, a, runs, po, pml);
}

}  // namespace

size_t paged_prefill_workspace(const PagedAttn& a) {
  const int runs = runs_for(a);
  return runs == 1 ? 0 : (size_t)a.tokens * a.n_heads * runs * (a.kv.head_dim * sizeof(float) + sizeof(float2));
}

cudaError_t launch_paged_prefill(const PagedAttn& a, int num_sms, cudaStream_t s) {
  CUtensorMap tq, tk, tv;
  const int G = a.n_heads / a.kv.n_kv_heads;
  if (!paged_maps(a.kv, &tk, &tv) ||
      !make_tmap_rows(&tq, a.q, a.kv.head_dim, a.n_heads, a.tokens, a.q_ld, G, kRows / G))
    return cudaErrorInvalidValue;
  return a.kv.head_dim == 128 ? launch_hd<128>(tq, tk, tv, a, num_sms, s)
                              : launch_hd<64>(tq, tk, tv, a, num_sms, s);
}
