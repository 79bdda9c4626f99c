// paged_prefill_fp8.cu -- attention of ragged runs of query tokens over a paged cache in 8 bits.
//
// Units, tiles and steps are those of the kernel over bf16 pages (paged_prefill.cu, paged_tiles.cuh): two
// tiles of 128 (token, q head) rows, steps of 64 keys.  Per step and tile
//   S = Q K^T     K as the codes it is, Q as the sum of two tiles of codes (q has eight bits of mantissa, a
//                 code four: exact down to 2^-10 of the row's largest element, off by at most 2^-18 of it
//                 below), e4m3 at twice the rate of bf16: what a product of bf16 would take
//   softmax       one thread per row
//   O += P V      P as fp16 in tensor memory (2^-11 of each weight, 2^-25 of what a weight of 1 stands for),
//                 V turned from codes to fp16 in shared memory, which is exact
// The step is a scale's block, and scales are powers of two: K's multiplies the row's score unit, V's
// exponent e is added to the scores, in units of log2: the weights are 2^(s + e - m) with m a whole number
// near the largest s + e so far, and the sum takes a step's weights times 2^-e.  Where a block's scale lies so far
// below others that a key there would lose bits of a weight as large as any, m is lowered: m <= s_max + e + kLow
// in every step, so that what is lost of a weight is 2^-22 of the row's largest at most, and of weight times scale
// 2^-25 of the largest of those.
//
// The codes of K and V come through TMA into a ring of stages.  A warpgroup of its own turns V into fp16
// (into a ring of its own), clearing keys that no query of the unit sees, and splits the units' Q; it
// has the registers that requester and issuers do not need.  S has one buffer a tile: the softmax takes it
// into registers and gives it back at once, so the next step's scores are formed under its exponentials;
// P has two, so that its product is never waited for.
//
// Neither pipe is full (issue 53 %, tensor 49 % in long units): a step takes what the softmax warps' own chain
// of waits, loads and exponentials takes, 0.97 us, next to the conversion's instructions; a unit another 3
// us to write out its rows and begin.  Measured, 32 q and 8 kv heads of 128: four prompts of 1024 tokens 51.7 us
// (665 TFLOP/s; over bf16 pages 41); four chunks of 500 to 1030 tokens over 3000 to 9000 positions, window
// 4096, 198 us (936 TFLOP/s; 169.5); 19 rows of 64 tokens over 16000 positions 241 us (1325 TFLOP/s; 224).
// To look whether a reference is to be lowered is 2 % of that; where references are, at every other step (scales 2^12
// apart from two steps to the next two), four rows of 512 tokens over 3584 take 151 us for 116.
// Tried: the largest score of a step not looked for unless the weights add up to too much (243 us for 236), Q as
// fp16 with K turned into it as well (not built: as much conversion again), a third tile of Q (261 us: two
// stages fewer).
#include <type_traits>

#include "fp8_tc.cuh"
#include "paged_tiles.cuh"

namespace {

using Attn = PagedAttnFp8;
constexpr int kStages = 5;
constexpr int kVSlots = 4;      // of V in fp16
// warps: issuers of S of tile 0, S of tile 1 and P V of both, requester of tiles; 4..7 and 8..11 softmax;
// 12..15 conversion
constexpr int kThreads = 512;
// Registers of a thread of the four warpgroups, out of what a block's threads have at launch (kRegs each)
constexpr int kRegs = 128, kRegsIssue = 64, kRegsSoftmax = 168, kRegsConvert = 112;
static_assert(kRegsIssue + 2 * kRegsSoftmax + kRegsConvert <= 4 * kRegs, "registers");
// A row's weights are below 2^kHead when its reference is set, and the reference is raised once they pass
// 2^(kHead + kSlack): far from the largest fp16, 2^16, and small ones as far from the smallest
constexpr float kHead = 6.f, kSlack = 9.f;
constexpr float kLow = 3.f;
// A reference goes no further than this below its highest, so that O (65504 * 448 for each of 2^31 positions at
// most, at the highest) stays in fp32's range
constexpr float kReach = 64.f;

// Shared memory: the tiles of Q, K and V, then this
constexpr int kBars = 5 + 2 * kStages + 2 * kVSlots + 12;
struct Tail {
  uint64_t bars[kBars];
  uint32_t tmem_slot;
  int abort_flag;
  int warp_sums[kThreads / 32];
  int2 exps[kStages];          // of K's and V's scale of a stage's step
  int2 s_exps[2][2];           // [tile]: of its last steps
  float row_unit[2][kRows];    // of each row's scores, in log2 units
  float most[2][kRows];        // a row's highest reference; its thread's own
  Unit units[kUnits];
};
template <int HD>
constexpr size_t smem_bytes() {  // 1024: the base is rounded up to the tiles' alignment
  return 1024 + 4 * kRows * HD + kStages * 2 * kStep * HD + kVSlots * HD * 128 + sizeof(Tail);
}
static_assert(smem_bytes<128>() <= 227 * 1024, "shared memory");

// every key of the step from k0 on is seen, by queries up to hi whose windows start at lo
CBT_D bool sees_all(int k0, int hi, int lo, int sinks) {
  return k0 + kStep - 1 <= hi && (lo <= k0 || sinks >= k0 + kStep);
}
// The steps of an item that tile x of its unit takes part in: those before `end`, without [hole0, hole1)
// (behind the sinks, before the window of the tile's first token)
struct TileSteps {
  int end, hole0, hole1;
  CBT_D TileSteps(const Work<Attn>& w, const Attn& a, int x, int TQ, int sinks) {
    const TileKeys t(w, a, x, TQ);
    const int last = t.last >= 0 ? t.last / kStep : -1, lo = t.lo / kStep, sink = (sinks + kStep - 1) / kStep;
    const Seen& s = w.seen;
    end = min(s.ns, last + 1) + max(0, last - s.ws + 1) - w.u.s0;
    hole0 = s.ns + max(0, sink - s.ws) - w.u.s0;
    hole1 = s.ns + lo - s.ws - w.u.s0;
  }
  CBT_D bool need(int i) const { return i < end && !(i >= hole0 && i < hole1); }
};

CBT_D uint32_t sub_f16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// of each of two pairs the larger magnitude (some sign; NaN where one is)
CBT_D uint32_t largest_bf16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// A row of Q on its way: pairs of q; then, of every 8 elements, two words of codes of either part.  A tile
// lands as rows of q, boxes of 64 dims, [128 rows][128 bytes], swizzled.  A row's codes take the bytes that
// its q took: the parts one box each, or (head_dim 64) either half of a row.
constexpr int kQBox = kRows * 128;
template <int HD>
struct QRow {
  uint32_t c[HD / 2];
  float unit;  // of the row's scores, in log2 units
  CBT_D void load(const uint8_t* q, int row) {
#pragma unroll
    for (int j = 0; j < HD / 8; ++j) {
      const uint4 v = *reinterpret_cast<const uint4*>(q + j / 8 * kQBox + tc::swz<128>(row, 16 * (j % 8)));
      c[4 * j] = v.x;
      c[4 * j + 1] = v.y;
      c[4 * j + 2] = v.z;
      c[4 * j + 3] = v.w;
    }
  }
  CBT_D void split(const Attn& a) {
    uint32_t top2 = 0;
#pragma unroll
    for (int j = 0; j < HD / 2; ++j) top2 = largest_bf16(top2, c[j]);
    const uint32_t top = max(top2 >> 16 & 0x7FFFu, top2 & 0x7FFFu);
    const bool finite = top < 0x7F80u;
    const int fit = fit_exponent(bf16_lo(finite ? top : 0));
    const float f = a.scale < 0.f ? -pow2_of(fit) : pow2_of(fit);  // the sign of the scale is q's
    unit = fabsf(a.scale) * kLog2e * pow2_of(-fit);
#pragma unroll
    for (int j = 0; j < HD / 8; ++j) {
      uint32_t part[2][2];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // in fp16 from here, which the scaled element's eight bits fit: the first four of them, and the rest
        const uint32_t y = pack_f16(bf16_lo(c[4 * j + e]) * f, bf16_hi(c[4 * j + e]) * f), y_hi = y & 0xFF80FF80u;
        const uint16_t hi = f16_to_e4m3(y_hi), lo = f16_to_e4m3(sub_f16(y, y_hi));
        part[0][e >> 1] = e & 1 ? part[0][e >> 1] | (uint32_t)hi << 16 : hi;
        part[1][e >> 1] = e & 1 ? part[1][e >> 1] | (uint32_t)lo << 16 : lo;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) c[4 * j + e] = part[e >> 1][e & 1];
    }
    if (!finite) {  // its scores are not numbers
#pragma unroll
      for (int j = 0; j < HD / 2; ++j) c[j] = 0x7F7F7F7Fu;
    }
  }
  CBT_D void store(uint8_t* q, int row) const {
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int j = 0; j < HD / 16; ++j)
        *reinterpret_cast<uint4*>(q + (HD == 128 ? p * kQBox : 0) + tc::swz<128>(row, (HD == 128 ? 0 : 64 * p) + 16 * j)) =
            make_uint4(c[8 * j + 2 * p], c[8 * j + 2 * p + 1], c[8 * j + 4 + 2 * p], c[8 * j + 5 + 2 * p]);
  }
};
// the 32-deep step `step` of a part, from the tile's start in 16-byte units
template <int HD>
CBT_HD constexpr uint32_t q_step(int part, int step) {
  return (uint32_t)(HD == 128 ? part * (kQBox >> 4) + 2 * step : 4 * part + 2 * step);
}
// a tile of Q from q to codes, by 128 threads, thread = row
template <int HD>
CBT_D void split_tile(const Attn& a, uint8_t* tile, float* row_unit, int row) {
  QRow<HD> q;
  q.load(tile, row);
  q.split(a);
  q.store(tile, row);
  row_unit[row] = q.unit;
  tc::fence_proxy_async_smem();
  __syncwarp();
}
CBT_D void tma_load_q(void* dst, const CUtensorMap* m, uint64_t* bar, int x, int head, int tok) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(tc::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(tc::smem_u32(bar)), "r"(x), "r"(head), "r"(tok)
      : "memory");
}
// the first unit behind k that has steps, or count
CBT_D int next_with_steps(const Unit* units, int k, int count) {
  do ++k;
  while (k < count && units[k].s1 <= units[k].s0);
  return k;
}
// a * b + c and a + b on two numbers, one instruction
CBT_D void fma2(float& x, float& y, float a, float b, float2 m, float2 c) {
  asm("{\n .reg .b64 p, q, r;\n mov.b64 p, {%2, %3};\n mov.b64 q, {%4, %5};\n mov.b64 r, {%6, %7};\n"
      " fma.rn.f32x2 p, p, q, r;\n mov.b64 {%0, %1}, p;\n}\n"
      : "=f"(x), "=f"(y)
      : "f"(a), "f"(b), "f"(m.x), "f"(m.y), "f"(c.x), "f"(c.y));
}
CBT_D void add2(float2& s, float a, float b) {
  asm("{\n .reg .b64 p, q;\n mov.b64 p, {%0, %1};\n mov.b64 q, {%2, %3};\n add.rn.f32x2 p, p, q;\n"
      " mov.b64 {%0, %1}, p;\n}\n"
      : "+f"(s.x), "+f"(s.y)
      : "f"(a), "f"(b));
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
    k_prefill_fp8(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                  const __grid_constant__ CUtensorMap tv,
                  const __grid_constant__ Attn a, const int runs, const int most, float* __restrict__ part_o,
                  float2* __restrict__ part_ml) {
  constexpr uint32_t kTile = kRows * HD * 2; // of Q
  constexpr uint32_t kKV = kStep * HD;       // codes of K or V of a step
  constexpr uint32_t kV16 = HD * 128;        // V of a step in fp16
  constexpr uint32_t kIdescS = tc::idesc_e4m3(128, kStep), kIdescO = tc::idesc_f16(128, HD);
  constexpr uint32_t kTmem = 512;  // tile x: S at 128 x, P of buffer b at 128 x + 64 + 32 b; O: 256 + HD x
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sQ = smem;                     // [tile]
  uint8_t* sK = sQ + 2 * kTile;           // [stage][64 keys][HD]
  uint8_t* sV = sK + kStages * kKV;       // [stage][HD dims][64 keys]
  uint8_t* sV16 = sV + kStages * kKV;     // [slot][HD dims][64 keys]
  Tail& tail = *reinterpret_cast<Tail*>(sV16 + kVSlots * kV16);
  uint64_t* bars = tail.bars;
  // q of a tile has landed, it is split, all are done with Q; a stage has landed, both tiles and the
  // conversion are done with it; V in fp16 is there, both tiles are done with it
  uint64_t *q_in = bars, *qfull = bars + 2, *qempty = bars + 4, *full = bars + 5, *empty = full + kStages;
  uint64_t *v_full = empty + kStages, *v_empty = v_full + kVSlots;
  // [tile]: S is there, S has been taken; [tile][buffer]: P is there, P has been read (and its product is
  // in O)
  uint64_t *s_full = v_empty + kVSlots, *s_free = s_full + 2, *p_full = s_free + 2, *pv_done = p_full + 4;
  uint32_t* tmem_slot = &tail.tmem_slot;
  volatile int* abort_flag = &tail.abort_flag;
  Unit* units = tail.units;

  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const int H = a.n_heads, Hkv = a.kv.n_kv_heads, G = H / Hkv;
  const int TQ = kRows / G;  // tokens per tile
  if (tid == 0) {
    auto init = [](uint64_t* b, int n, int arrivals) {
      for (int i = 0; i < n; ++i) tc::mbar_init(b + i, arrivals);
    };
    init(q_in, 2, 1);
    init(qfull, 2, 4);             // the warps that split it
    init(qempty, 1, 2 + 8);        // issuers, softmax warps
    init(full, kStages, 1);
    init(empty, kStages, 2 + 4);   // issuers, converting warps
    init(v_full, kVSlots, 4);
    init(v_empty, kVSlots, 1);
    init(s_full, 2, 1 + 1);        // the product, and the issuer has stored the step's exponents
    init(s_free, 2, 4);            // a tile's softmax warps
    init(p_full, 4, 4);
    init(pv_done, 4, 1);
    *abort_flag = 0;
    tc::mbar_fence_init();
    tc::tma_prefetch_desc(&tq);
    tc::tma_prefetch_desc(&tk);
    tc::tma_prefetch_desc(&tv);
  }
  if (warp == 1) tc::tmem_alloc(tmem_slot, kTmem);
  pdl_wait();
  static_assert(kScratch <= 2 * kTile, "the search fits where Q goes");
  int count = find_units<kThreads>(a, units, sQ, tail.warp_sums, TQ, runs, most);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  count = uniform(count);
  const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);
  const int sinks = a.window ? a.sinks : 0;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    bool ok = true;
    if (warp < 2) {
      // ---- S of tile x, as soon as the softmax has taken the last one
      const int x = warp;
      const uint32_t s_tm = tmem + x * 128;
      const uint32_t dq = tc::rows_lo<128>(sQ + x * kTile), dk = tc::rows_lo<HD>(sK);
      int st = 0, n = 0;  // stage, steps that the tile took part in
      uint32_t ph = 0, qp = 0;
#pragma unroll 1
      for (int k = 0; k < count && ok; ++k) {
        const Work<Attn> w(units + k, a);
        if (!w.steps) continue;
        const TileSteps mine(w, a, x, TQ, sinks);
        ok = __all_sync(0xffffffffu, wait_or_abort(&qfull[x], qp, abort_flag));
        if (!ok) break;
        qp ^= 1;
#pragma unroll 1
        for (int i = 0; i < w.steps; ++i) {
          const bool need = mine.need(i);
          // K has landed; S has been taken; P of the step two before has been read, so that the softmax may
          // write there again
          bool got = wait_or_abort(&full[st], ph, abort_flag);
          if (need)
            got = got && wait_or_abort(&pv_done[2 * x + (n & 1)], (n >> 1 & 1) ^ 1, abort_flag) &&
                  wait_or_abort(&s_free[x], (n & 1) ^ 1, abort_flag);
          ok = __all_sync(0xffffffffu, got);
          if (!ok) break;
          tc::tc_fence_after();
          if (elect_one()) {
            if (need) {
              tail.s_exps[x][n & 1] = tail.exps[st];
              tc::mbar_arrive(&s_full[x]);
              const uint32_t kd = dk + st * (kKV >> 4);
#pragma unroll
              for (int e = 0; e < 2 * (HD / 32); ++e) {
                const int part = e / (HD / 32), step = e % (HD / 32);
                tc::mma_e4m3(s_tm, tc::rows_desc<128>(dq + q_step<HD>(part, step)),
                             tc::rows_desc<HD>(kd + 2 * step), kIdescS, e > 0 ? 1u : 0u);
              }
              tc::mma_commit(&s_full[x]);
            }
            tc::mma_commit(&empty[st]);
            if (i == w.steps - 1) tc::mma_commit(qempty);
          }
          n += need;
          st = st + 1 == kStages ? 0 : st + 1;
          ph ^= st == 0;
        }
      }
      if (!ok && lane == 0) wait_timeout(a.err, abort_flag, 32);
    } else if (warp == 2) {
      // ---- P V of both tiles
      const uint32_t dv = tc::rows_lo<128>(sV16);
      int slot = 0, n[2] = {0, 0};
      uint32_t vp = 0;
#pragma unroll 1
      for (int k = 0; k < count && ok; ++k) {
        const Work<Attn> w(units + k, a);
        const TileSteps tile[2] = {TileSteps(w, a, 0, TQ, sinks), TileSteps(w, a, 1, TQ, sinks)};
        uint32_t acc[2] = {0, 0};  // O holds something of this unit
#pragma unroll 1
        for (int i = 0; i < w.steps && ok; ++i) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const bool need = tile[x].need(i);
            const int b = n[x] & 1;
            if (x == 0 || need) {
              bool got = x > 0 || wait_or_abort(&v_full[slot], vp, abort_flag);
              if (need) got = got && wait_or_abort(&p_full[2 * x + b], n[x] >> 1 & 1, abort_flag);
              ok = __all_sync(0xffffffffu, got);
              if (!ok) break;
              tc::tc_fence_after();
            }
            if (need && elect_one()) {
              const uint32_t v = dv + slot * (kV16 >> 4);
#pragma unroll
              for (int e = 0; e < kStep / 16; ++e)
                tc::mma_bf16_ta(tmem + 256 + x * HD, tmem + 128 * x + 64 + 32 * b + 8 * e, tc::rows_desc<128>(v + 2 * e),
                                kIdescO, (acc[x] || e > 0) ? 1u : 0u);
              tc::mma_commit(&pv_done[2 * x + b]);
            }
            if (need) {
              acc[x] = 1;
              ++n[x];
            }
          }
          if (ok && elect_one()) tc::mma_commit(&v_empty[slot]);
          slot = slot + 1 == kVSlots ? 0 : slot + 1;
          vp ^= slot == 0;
        }
      }
      if (!ok && lane == 0) wait_timeout(a.err, abort_flag, 35);
    } else {
      // ---- tile requests.  The pages and scales of 32 steps are looked up at once, a lane each.
      const uint64_t pol = tc::policy_evict_last();
      const int P = a.kv.page_tokens;
      int st = 0, n = 0;  // stage, steps requested
      uint32_t ph = 0;
#pragma unroll 1
      for (int k = 0; k < count && ok; ++k) {
        const Work<Attn> w(units + k, a);
        int kat = 0, vat = 0;
        float ks = 0.f, vs = 0.f;
#pragma unroll 1
        for (int i = 0; i < w.steps; ++i) {
          if ((i & 31) == 0 && i + lane < w.steps) {
            const int key = w.key(i + lane), pg = key / P, o = key - pg * P;
            int id = a.table[(size_t)w.u.b * a.max_pages + pg];
            if (id < 0 || id >= a.kv.n_pages) {
              set_device_error(a.err, CBT_DEV_PAGE_ID, w.u.b);
              id = 0;  // a page that exists: the row's outputs are unspecified
            }
            kat = (int)(fp8_k(a.kv, id, w.u.g, o, 0) >> 8);
            vat = (int)(fp8_v(a.kv, id, w.u.g, o, 0) >> 8);
            ks = *fp8_scale(a.kv, id, 0, w.u.g, o);
            vs = *fp8_scale(a.kv, id, 1, w.u.g, o);
          }
          const int ka = __shfl_sync(0xffffffffu, kat, i & 31), va = __shfl_sync(0xffffffffu, vat, i & 31);
          ok = __all_sync(0xffffffffu, wait_or_abort(&empty[st], ph ^ 1, abort_flag));
          if (!ok) break;
          if (elect_one()) {
            tc::tma_load_rows(sK + st * kKV, &tk, &full[st], ka, pol);
            tc::tma_load_rows(sV + st * kKV, &tv, &full[st], va, pol);
          }
          // (the bytes may land before they are expected: the phase waits for the arrival)
          if (lane == (i & 31)) tail.exps[st] = make_int2(fp8_exponent(ks), fp8_exponent(vs));
          __syncwarp();
          if (elect_one()) tc::mbar_expect_tx(&full[st], 2 * kKV);
          ++n;
          st = st + 1 == kStages ? 0 : st + 1;
          ph ^= st == 0;
        }
      }
      if (lane == 0) {
        if (!ok) wait_timeout(a.err, abort_flag, 31);
        // no copies in flight at exit
#pragma unroll 1
        for (int i = max(0, n - kStages); i < n; ++i) wait_landed(&full[i % kStages], (i / kStages) & 1);
      }
    }
  } else if (warp >= 12) {
    // ---- Q into two parts of codes, V into fp16.  Thread = row of Q; of V, 16 keys of HD / 32 dims.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConvert));
    const int row = tid - 384;
    int st = 0, slot = 0;
    uint32_t ph = 0, vp = 0, qp = 0;
    bool ok = true;
    uint32_t qi = 0, asked = 0;  // phases of q_in, and which have been asked for
    const int first = next_with_steps(units, -1, count);
#pragma unroll 1
    for (int k = first; k < count && ok; k = uniform(next_with_steps(units, k, count))) {
      const Work<Attn> w(units + k, a);
      const int tiles = w.u.n > TQ ? 2 : 1;
      if (k != first) ok = __all_sync(0xffffffffu, wait_or_abort(qempty, qp, abort_flag));
      if (!ok) break;
      if (k != first) qp ^= 1;
      if (warp == 12 && elect_one()) {
#pragma unroll 1
        for (int x = 0; x < tiles; ++x) {
          tc::mbar_expect_tx(&q_in[x], HD / 64 * G * TQ * 128);
#pragma unroll
          for (int h = 0; h < HD / 64; ++h)
            tma_load_q(sQ + x * kTile + h * kQBox, &tq, &q_in[x], h * 64, w.u.g * G, w.u.t0 + x * TQ);
        }
      }
      qi ^= tiles == 2 ? 3 : 1;
      asked |= tiles == 2 ? 3 : 1;
      // the first unit's are split by the softmax's warps, which have nothing else to do
#pragma unroll 1
      for (int x = 0; x < 2 && k != first && ok; ++x) {
        if (x < tiles) {
          ok = __all_sync(0xffffffffu, wait_or_abort(&q_in[x], (qi >> x & 1) ^ 1, abort_flag));
          if (!ok) break;
          split_tile<HD>(a, sQ + x * kTile, tail.row_unit[x], row);
        }
        if (lane == 0) tc::mbar_arrive(&qfull[x]);
      }
#pragma unroll 1
      for (int i = 0; i < w.steps && ok; ++i) {
        // the step has landed, and its slot is free again
        ok = __all_sync(0xffffffffu, wait_or_abort(&full[st], ph, abort_flag) &&
                                         wait_or_abort(&v_empty[slot], vp ^ 1, abort_flag));
        if (!ok) break;
        const uint8_t* v = sV + st * kKV;
        uint4 in[HD / 32];
#pragma unroll
        for (int j = 0; j < HD / 32; ++j)
          in[j] = *reinterpret_cast<const uint4*>(v + tc::swz<64>((row >> 2) + 32 * j, 16 * (row & 3)));
        const int k0 = w.key(i);
        if (!sees_all(k0, w.pl, w.lo_win, sinks)) {  // keys that no query of the unit sees
          uint32_t bits[2];
          seen_bits(k0, w.pl, w.lo_win, sinks, bits);
          const uint4 m = code_mask((row & 2 ? bits[1] : bits[0]) >> (16 * (row & 1)));
#pragma unroll
          for (int j = 0; j < HD / 32; ++j)
            in[j] = make_uint4(in[j].x & m.x, in[j].y & m.y, in[j].z & m.z, in[j].w & m.w);
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&empty[st]);
        uint8_t* out = sV16 + slot * kV16;
#pragma unroll
        for (int j = 0; j < HD / 32; ++j) {
          const uint32_t u[4] = {in[j].x, in[j].y, in[j].z, in[j].w};
#pragma unroll
          for (int e = 0; e < 2; ++e)
            *reinterpret_cast<uint4*>(out + tc::swz<128>((row >> 2) + 32 * j, 32 * (row & 3) + 16 * e)) =
                make_uint4(e4m3_to_f16((uint16_t)u[2 * e]), e4m3_to_f16((uint16_t)(u[2 * e] >> 16)),
                           e4m3_to_f16((uint16_t)u[2 * e + 1]), e4m3_to_f16((uint16_t)(u[2 * e + 1] >> 16)));
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&v_full[slot]);
        slot = slot + 1 == kVSlots ? 0 : slot + 1;
        vp ^= slot == 0;
        st = st + 1 == kStages ? 0 : st + 1;
        ph ^= st == 0;
      }
    }
    if (!ok && lane == 0) wait_timeout(a.err, abort_flag, 33);
    // no copies in flight at exit
    if (warp == 12 && lane < 2 && asked >> lane & 1) wait_landed(&q_in[lane], (qi >> lane & 1) ^ 1);
  } else {
    // ---- softmax of tile x: thread = row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int x = (warp - 4) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_tm = tmem + x * 128 + lane_off, o_tm = tmem + 256 + x * HD + lane_off;
    uint32_t qp = 0;  // phase of Q
    int done = 0;     // steps that the tile took part in
    bool ok = true;
    if (const int first = next_with_steps(units, -1, count); first < count) {  // the first unit's Q
      if (x * TQ < units[first].n) {
        ok = __all_sync(0xffffffffu, wait_or_abort(&q_in[x], 0, abort_flag));
        if (ok) split_tile<HD>(a, sQ + x * kTile, tail.row_unit[x], row);
      }
      if (lane == 0) tc::mbar_arrive(&qfull[x]);
    }
    // rows of out on 32-byte boundaries: whole sectors a store
    const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0 && a.out_ld % (a.f32 ? 8 : 16) == 0;
#pragma unroll 1
    for (int unit = 0; unit < count && ok; ++unit) {
      const Work<Attn> w(units + unit, a);
      const TileSteps mine(w, a, x, TQ, sinks);
      const int tok = x * TQ + row / G;  // token of the unit
      const bool live = row < TQ * G && tok < w.u.n;
      const int p = live ? w.u.p0 + tok : -1;  // -1: sees nothing
      // rows that hold no token are left unmasked: what they compute is not stored
      const int hi = live ? p : 0x3FFFFFFF, lo = live ? first_in_window(max(0, p), a.window) : 0;
      const int hi_all = __reduce_min_sync(0xffffffffu, hi), lo_all = __reduce_max_sync(0xffffffffu, lo);
      float m = -INFINITY, l = 0.f;  // the reference (near the largest so far, a whole number) and the sum
      float s_max = -INFINITY;       // the largest score so far
      const int before = done;
      float row_unit = 0.f;
      if (w.steps) {
        ok = __all_sync(0xffffffffu, wait_or_abort(&qfull[x], qp, abort_flag));
        if (!ok) break;
        qp ^= 1;
        row_unit = tail.row_unit[x][row];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(qempty);
      }
#pragma unroll 1
      for (int i = 0; i < w.steps && ok; ++i) {
        if (!mine.need(i)) continue;
        ok = __all_sync(0xffffffffu, wait_or_abort(&s_full[x], done & 1, abort_flag));
        if (!ok) break;
        tc::tc_fence_after();
        const int2 exps = tail.s_exps[x][done & 1];
        uint32_t s[64];
        tmem_ld32(s_tm, s);
        tmem_ld32(s_tm + 32, s + 32);
        // a score's unit (kept where a masked -inf stays -inf and a zero is one) and the addition to it
        const float cs = fminf(fmaxf(row_unit * pow2_of(exps.x), 1e-37f), 3e38f), ve = (float)exps.y;
        tc::tmem_ld_wait();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&s_free[x]);
        const int k0 = w.key(i);
        auto weights = [&](auto masked) {
          if (masked.value) {
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
          const float top = fmaf(fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]), cs, ve);
          s_max = fmaxf(s_max, top - ve);
          const bool up = m == -INFINITY ? top > -INFINITY : top > m + (kHead + kSlack), down = m > s_max + (ve + kLow);
          if (__any_sync(0xffffffffu, up || down)) {
            // Rows that exceed their reference, or see their first keys, raise it, to a whole number: what
            // the old one has scaled is multiplied by a power of two, which rounds nothing.
            float& most = tail.most[x][row];
            float next = up ? ceilf(top) - kHead : m;
            if (down) next = fmaxf(ceilf(s_max + ve) - kHead, most - kReach);
            // m = -inf: l and O are zero
            const float f = m == -INFINITY ? 0.f : next < m ? pow2_of((int)(m - next)) : pow2_down(next - m);
            most = m == -INFINITY ? next : fmaxf(most, next);
            m = next;
            l *= f;
            if (done > before) {
              // O is at rest once the last step's product is in it
              const int d = done - 1;
              ok = __all_sync(0xffffffffu, wait_or_abort(&pv_done[2 * x + (d & 1)], d >> 1 & 1, abort_flag));
              if (!ok) return;
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
          const float add = ve - (m == -INFINITY ? 0.f : m);
          float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          const float2 cs2 = make_float2(cs, cs), add_2 = make_float2(add, add);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float p0, p1;
            fma2(p0, p1, __uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]), cs2, add_2);
            p0 = ex2(p0);
            p1 = ex2(p1);
            add2(part[e & 1], p0, p1);
            s[e] = pack_f16(p0, p1);
          }
          tc::tmem_st32(s_tm + 64 + 32 * (done & 1), s);
          tc::tmem_st_wait();
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&p_full[2 * x + (done & 1)]);
          l = fmaf((part[0].x + part[0].y) + (part[1].x + part[1].y), pow2_of(-exps.y), l);
        };
        // every row sees every key of the step, or keys are masked one by one.  (Two copies of the code: with the
        // masks in a branch of one, never taken, 251 steps took 250 us for 228.)
        if (__any_sync(0xffffffffu, !sees_all(k0, hi_all, lo_all, sinks))) weights(std::true_type());
        else weights(std::false_type());
        if (!ok) break;
        ++done;
      }
      // The row goes straight out.  O is not written again before this tile hands in weights of the next
      // unit.
      if (ok && done > before) {
        const int d = done - 1;
        ok = __all_sync(0xffffffffu, wait_or_abort(&pv_done[2 * x + (d & 1)], d >> 1 & 1, abort_flag));
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
        if (done > before) {
          tc::tmem_ld16(o_tm + k, o);
          tc::tmem_ld_wait();
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = p >= 0 ? __float_as_uint(__uint_as_float(o[e]) * inv) : 0u;
        if (!live) continue;
        if (a.f32 || runs > 1) {
          float* dst = runs > 1 ? part_o + part * HD + k : static_cast<float*>(a.out) + at + k;
#pragma unroll
          for (int e = 0; e < 16; e += 8) {
            uint32_t h[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) h[j] = o[e + j];
            store32(dst + e, h, wide || runs > 1);
          }
        } else {
          uint32_t h[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) h[j] = pack_bf16(__uint_as_float(o[2 * j]), __uint_as_float(o[2 * j + 1]));
          store32(static_cast<uint16_t*>(a.out) + at + k, h, wide);
        }
      }
      tc::tc_fence_before();
    }
    if (!ok && lane == 0) wait_timeout(a.err, abort_flag, 34);
    tc::tc_fence_before();
  }
  pdl_launch();
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, kTmem);
  }
}

template <int HD>
cudaError_t launch_hd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const Attn& a, int num_sms,
                      cudaStream_t s) {
  constexpr size_t smem = smem_bytes<HD>();
  cudaError_t rc = cudaFuncSetAttribute(k_prefill_fp8<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (rc != cudaSuccess) return rc;
  // the warpgroups' shares come out of what a block is launched with: with less the kernel would wait
  static const int regs = [] {
    cudaFuncAttributes attr;
    return cudaFuncGetAttributes(&attr, k_prefill_fp8<HD>) == cudaSuccess ? attr.numRegs : 0;
  }();
  if (regs < kRegs) return cudaErrorInvalidConfiguration;
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
  rc = launch_pdl(k_prefill_fp8<HD>, dim3((unsigned)grid), dim3(kThreads), smem, s, tq, tk, tv, a, runs, (int)units,
                  po, pml);
  if (rc != cudaSuccess || runs == 1) return rc;
  const long long pairs = (long long)a.tokens * a.n_heads;
  if (pairs <= kFewPairs && runs > kManyRuns)
    return launch_pdl(k_prefill_merge<HD, 4, Attn>, dim3((unsigned)pairs), dim3(128), 0, s, a, runs, po, pml);
  return launch_pdl(k_prefill_merge<HD, 1, Attn>, dim3((unsigned)((pairs + 3) / 4)), dim3(128), 0, s, a, runs, po, pml);
}

}  // namespace

size_t prefill_fp8_workspace(const Attn& a) {
  const int runs = runs_for(a);
  return runs == 1 ? 0 : (size_t)a.tokens * a.n_heads * runs * (a.kv.head_dim * sizeof(float) + sizeof(float2));
}

cudaError_t launch_prefill_fp8(const Attn& a, int num_sms, cudaStream_t s) {
  CUtensorMap tq, tk, tv;
  const int G = a.n_heads / a.kv.n_kv_heads;
  if (!fp8_maps(a.kv, &tk, &tv) ||
      !make_tmap_rows(&tq, a.q, a.kv.head_dim, a.n_heads, a.tokens, a.q_ld, G, kRows / G))
    return cudaErrorInvalidValue;
  return a.kv.head_dim == 128 ? launch_hd<128>(tq, tk, tv, a, num_sms, s) : launch_hd<64>(tq, tk, tv, a, num_sms, s);
}
