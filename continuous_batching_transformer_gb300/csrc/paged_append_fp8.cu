// paged_append_fp8.cu -- per-head RMS norm, rotary positions and the append of K and V to a paged cache
// in 8 bits, one launch over QKV rows.
//
// Every element is read once and written once, q as bf16 and k and v as codes.  q is rotated as for a
// bf16 cache (a warp per token and run of heads).  A scale belongs to the 64 positions of a block, so k
// and v go by blocks: a thread block takes the runs (tokens next to each other in the call that lie in
// one cache block) that begin among its chunk of tokens, to their ends, for K or V of a kv head, or of two
// one after the other.  For each it
//   1. forms the tokens' values, kept in shared memory as 16 bits rounded to odd, and each run's largest
//      magnitude;
//   2. settles each run's exponent from that and the scale that the cache block has;
//   3. where it grows, moves the codes held there down (rare: once a block has a few tokens, most of
//      those that follow are below its largest);
//   4. rounds the values to codes; V, whose layout runs along the positions of a dim, is turned around
//      on the way and written 16 positions at a time where a run fills them.
// No thread block shares a cache block with another, so nothing is exchanged through memory.
//
// HBM is the floor.  8192 tokens of 32 q and 8 kv heads of 128 with norms take 52 us, 2.8 TB/s, over bf16
// pages 40: issue slots (67 % taken) and the chains of loads and barriers of a block bound it together, DRAM is
// 34 % busy.  8 tokens of them take 4 us, 800 tokens of 12 and 4 heads of 64 in runs of up to 177 7.3 us: one
// such chain.
#include "paged_fp8.h"
#include "paged_rope.cuh"

namespace {

// sin and cos of the 256 whole fractions of a turn, for turn_sincos
struct Circle {
  float2 at[256];
};
// One entry: within an eighth of a turn of a whole number of quarters, the Taylor series (first terms left
// out: x^11 / 11! and x^12 / 12!, below 2^-28).
CBT_D float2 circle_at(int k) {
  const int quarter = (k + 32) >> 6;
  const float x = (float)(k - 64 * quarter) * 0x1.921fb6p-6f;  // 2 pi / 256
  const float z = x * x;
  float s = fmaf(z, 1.f / 362880, -1.f / 5040);
  s = fmaf(z, s, 1.f / 120);
  s = fmaf(z, s, -1.f / 6);
  s = fmaf(x * z, s, x);
  float c = fmaf(z, -1.f / 3628800, 1.f / 40320);
  c = fmaf(z, c, -1.f / 720);
  c = fmaf(z, c, 1.f / 24);
  c = fmaf(z, c, -0.5f);
  c = fmaf(z, c, 1.f);
  const float a = quarter & 1 ? c : s, b = quarter & 1 ? s : c;
  return make_float2(quarter & 2 ? -a : a, (quarter + 1) & 2 ? -b : b);
}
// sin and cos of pos * turns (a fraction of a turn, 2^64 a whole) to fp32's last place or so: the nearest
// entry, turned by the rest (at most pi / 256, where two terms of the series are enough).  (The hardware's sine,
// off by 2^-21, takes 1.5 us less for 8192 tokens of 8 heads of 128, and with it 45 codes of 8.4 million lie beside
// the formula's for 6.)
CBT_D void turn_sincos(const Circle& circle, uint32_t pos, uint64_t turns, float* sn, float* cs) {
  const uint32_t ph = pos * (uint32_t)(turns >> 32) + __umulhi(pos, (uint32_t)turns);  // 2^32 a turn
  const uint32_t k = ph + (1u << 23);
  const float r = (float)(int)((k & 0xFFFFFFu) - (1u << 23)) * 0x1.921fb6p-30f;  // 2 pi / 2^32
  const float2 e = circle.at[k >> 24];
  const float z = r * r;
  const float s = r * fmaf(z, -1.f / 6, 1.f), c1 = z * fmaf(z, 1.f / 24, -0.5f);  // sin r, cos r - 1
  *sn = e.x + fmaf(e.x, c1, e.y * s);
  *cs = e.y + fmaf(e.y, c1, -e.x * s);
}

// Two numbers' first 16 bits each, the last of them set where anything is behind it ("rounded to odd"):
// what is rounded from that to a code's four bits is rounded as the number itself.
CBT_D uint32_t pack_odd(float lo, float hi) {
  const uint32_t a = __float_as_uint(lo), b = __float_as_uint(hi);
  return __byte_perm(a, b, 0x7632) | __vminu2(__byte_perm(a, b, 0x5410), 0x00010001u);
}
// of each of two pairs of bf16 the larger magnitude (some sign; a NaN only where both are)
CBT_D uint32_t larger_bf16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// the exponent of the smallest scale that values up to `top` (finite, >= 0) are within 448 times of
CBT_D int exponent_for(float top) {
  const uint32_t u = __float_as_uint(top);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u);  // 448 = 1.75 * 2^8
  return min(max(e, kLowExp), kHighExp);
}

// four codes times f, each rounded again
CBT_D uint32_t move_codes(uint32_t w, float f) {
  const uint32_t lo = e4m3_to_f16((uint16_t)w), hi = e4m3_to_f16((uint16_t)(w >> 16));
  return pack_e4m3(f16_lo(lo) * f, f16_hi(lo) * f) | (uint32_t)pack_e4m3(f16_lo(hi) * f, f16_hi(hi) * f) << 16;
}

// How far above the start of the range around the middle between two codes (of any scale: a code's last bit is
// the fourth of its mantissa) in which what fp32 is off by may decide where it is rounded to.
// Such values are formed again from pairs of fp32 (a warp has one in 500 of its steps): what is left are a few small
// members of their pairs, where fp32 is off by more steps.  8.4 million codes: 6 beside the formula's for 13, at 2 us
// of 62 for the look at each value.
constexpr uint32_t kNear = 4;  // steps of fp32 on either side
CBT_D uint32_t above_middle(float x) { return __float_as_uint(x) * 4096u + ((kNear - 0x80000u) << 12); }
CBT_D bool near_middle(uint32_t above) { return above < (2 * kNear) << 12; }
template <bool F32>
CBT_D float element(const void* p, long long i) {
  return F32 ? static_cast<const float*>(p)[i] : bf16_lo(static_cast<const uint16_t*>(p)[i]);
}
// A value as the sum of two fp32, some 44 bits: settle's arithmetic, which in 64 bits waits for that pipe
// (with the read-back a call of 256 tokens takes 10.9 us without settle, 14.5 with it in 64 bits, 12.0 so).
struct Pair {
  float hi, lo;
};
CBT_D Pair both(float a, float b) {  // a + b
  const float s = a + b, v = s - a;
  return {s, (a - (s - v)) + (b - v)};
}
CBT_D Pair plus(Pair a, Pair b) {
  const Pair s = both(a.hi, b.hi);
  return both(s.hi, s.lo + (a.lo + b.lo));
}
CBT_D Pair times(Pair a, Pair b) {
  const float p = a.hi * b.hi;
  return both(p, fmaf(a.hi, b.hi, -p) + fmaf(a.hi, b.lo, a.lo * b.hi));
}
// sin and cos of a phase of 2^64 a turn: Taylor's series around the nearest quarter, x within pi / 4.  The terms
// from x^4 on are below 2^-5 and are summed in fp32; first ones left out: x^13 / 13! and x^12 / 12!.  Off by less
// than 2^-28.
CBT_D void turn_pairs(uint64_t ph, Pair* sn, Pair* cs) {
  const uint64_t up = ph + (1ull << 61);
  const int64_t rest = (int64_t)(up & ((1ull << 62) - 1)) - (1ll << 61);
  const float top = (float)rest;
  const Pair x = times({top, (float)(rest - (int64_t)top)}, {0x1.921fb6p-62f, -0x1.777a5cp-87f});  // 2 pi / 2^64
  const Pair z = times(x, x);
  const float w = z.hi;
  const float s = w * w * fmaf(w, fmaf(w, fmaf(w, -1.f / 39916800, 1.f / 362880), -1.f / 5040), 1.f / 120);
  const float c = w * w * fmaf(w, fmaf(w, fmaf(w, -1.f / 3628800, 1.f / 40320), -1.f / 720), 1.f / 24);
  const Pair sixth = times(z, {-0x1.555556p-3f, 0x1.555556p-28f});  // -1 / 6
  const Pair sine = times(x, plus({1.f, 0.f}, plus(sixth, {s, 0.f})));
  const Pair cosine = plus({1.f, 0.f}, plus({-0.5f * z.hi, -0.5f * z.lo}, {c, 0.f}));
  const int quarter = (int)(up >> 62);
  const Pair p = quarter & 1 ? cosine : sine, q = quarter & 1 ? sine : cosine;
  const float ps = quarter & 2 ? -1.f : 1.f, qs = (quarter + 1) & 2 ? -1.f : 1.f;
  *sn = {ps * p.hi, ps * p.lo};
  *cs = {qs * q.hi, qs * q.lo};
}
// The values of K head g of token t that lie so, formed anew and rounded to odd; by all lanes of a warp
template <int HD, bool F32, int MODE>
CBT_D void settle(const RopeAppendFp8& a, int t, int g, int l, const LaneDims& dims, bool on, float (&x)[8]) {
  unsigned near = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (on && near_middle(above_middle(x[k]))) near |= 1u << k;
  const long long row = t * a.qkv_ld + (long long)(a.n_heads + g) * HD;
  Pair r = {1.f, 0.f};
  if (a.k_gain) {
    float y[8];
    load4<F32>(a.qkv, row + 8 * l, y);
    load4<F32>(a.qkv, row + 8 * l + 4, y + 4);
    Pair s = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 8; ++k) s = plus(s, times({y[k], 0.f}, {y[k], 0.f}));
#pragma unroll 1
    for (int w = HD / 16; w > 0; w >>= 1)
      s = plus(s, {__shfl_xor_sync(0xffffffffu, s.hi, w), __shfl_xor_sync(0xffffffffu, s.lo, w)});
    s = plus({s.hi * (1.f / HD), s.lo * (1.f / HD)}, {a.eps, 0.f});
    const float r0 = rsqrtf(s.hi);
    const Pair off = plus({1.f, 0.f}, times(s, times({-r0, 0.f}, {r0, 0.f})));  // Newton: twice the places
    r = both(r0, 0.5f * r0 * off.hi);
  }
  const int rot = MODE == kNone ? 0 : a.rope.rot_dim;
  auto value = [&](int d) {
    const float y = element<F32>(a.qkv, row + d);
    return a.k_gain ? times({y, 0.f}, {element<false>(a.k_gain, d), 0.f}) : Pair{y, 0.f};
  };
#pragma unroll 1
  for (; near; near &= near - 1) {
    const int k = __ffs(near) - 1, d = k < 4 ? dims.e0 + k : dims.e1 + k - 4;
    Pair y = value(d);
    if (d < rot) {
      const bool second = MODE == kInter ? d & 1 : d >= rot / 2;
      const int pair = MODE == kInter ? d / 2 : second ? d - rot / 2 : d;
      const int other = MODE == kInter ? d ^ 1 : second ? pair : d + rot / 2;
      Pair sn, cs;
      turn_pairs((uint64_t)a.positions[t] * a.rope.turns[pair], &sn, &cs);
      if (!second) sn = {-sn.hi, -sn.lo};
      y = times(plus(times(y, cs), times(value(other), sn)), {a.rope.mscale, 0.f});
    }
    y = times(y, r);
    uint32_t f = __float_as_uint(y.hi);
    if (y.lo != 0.f) f = (f - ((y.lo < 0.f) != (y.hi < 0.f) ? 1u : 0u)) | 1u;
#pragma unroll
    for (int q = 0; q < 8; ++q)  // (a product on the way may pass fp32's range where the value does not)
      x[q] = q == k && y.lo - y.lo == 0.f ? __uint_as_float(f) : x[q];
  }
}

constexpr int kMostChunk = 64;             // tokens whose runs a thread block takes
constexpr int kTokens = 2 * kMostChunk;    // with the last run's further ones (of 64 positions at most)
constexpr int kResident = 4 * 152;         // thread blocks that the SMs hold
struct Runs {
  int slot[kTokens];               // of each token, -1: not this block's
  short run[kMostChunk];           // of each of the chunk's tokens, -1: none that begins here
  int first_slot[kMostChunk];      // of each run
  uint8_t* block[kMostChunk];      // its cache block's codes
  int top[kMostChunk];             // its largest magnitude, as bits
  int anew[kMostChunk];            // it holds its cache block's first position
  int exponent[kMostChunk];
  int grown[kMostChunk], down[kMostChunk];  // runs whose cache block moves, and by how much
  int count, lead, n_grown, last_block;
  int warp_runs[2], warp_lead[2], scan[kWarps];
  int part[kTokens], warp_parts[kTokens / 32];  // tokens next to each other in 16 aligned slots
};

// Shared memory of a block for k and v: the runs, the tokens' values (rows padded by 16 bytes), the circle,
// and what heads with odd pairs exchange through
template <int HD>
constexpr int kRowBytes = 2 * HD + 16;
constexpr size_t kRunsBytes = (sizeof(Runs) + 15) / 16 * 16;
template <int HD, int MODE>
constexpr size_t kv_smem() {
  return kRunsBytes + (size_t)kTokens * kRowBytes<HD> + (MODE == kNone ? 0 : sizeof(Circle)) +
         (MODE == kHalfOdd ? kWarps * 256 * sizeof(float) : 0);
}

// runs that begin in tokens [t0, t0 + chunk), of kv heads [g0, g1), of K or of V
template <int HD, bool F32, int MODE, bool V>
CBT_D void append_runs(const RopeAppendFp8& a, int t0, int chunk, int g0, int g1, uint8_t* sm) {
  constexpr int LPH = HD / 8, NH = 32 / LPH;  // lanes of a token, tokens of a warp
  constexpr int kPlaces = kWarps * NH;        // tokens in flight
  constexpr int kRow = kRowBytes<HD>;
  Runs& r = *reinterpret_cast<Runs*>(sm);
  uint8_t* tile = sm + kRunsBytes;
  Circle& circle = *reinterpret_cast<Circle*>(tile + kTokens * kRow);
  float* xs = reinterpret_cast<float*>(&circle + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, l = lane % LPH, sub = lane / LPH;
  const int page = a.kv.page_tokens;
  auto slot_of = [&](int t) {
    if (t < 0 || t >= a.tokens) return -1;
    const int s = a.slots[t];
    return slot_ok(a, s, a.positions[t]) ? s : -1;
  };
  // ---- the runs: a token begins one where the token before it lies in another cache block
  if (tid < kMostChunk) {
    const int s = tid < chunk ? slot_of(t0 + tid) : -1;
    const int before = tid < chunk ? slot_of(t0 + tid - 1) : -1;
    const bool first = s >= 0 && (before < 0 || before / kBlock != s / kBlock);
    const unsigned m = __ballot_sync(0xffffffffu, first);
    if (lane == 0) {
      r.warp_runs[warp] = __popc(m);
      r.warp_lead[warp] = m ? 32 * warp + __ffs(m) - 1 : kMostChunk;
    }
    r.slot[tid] = s;
    r.run[tid] = s < 0 ? -1 : (short)(__popc(m & (0xffffffffu >> (31 - lane))) - 1);  // in its warp
    r.top[tid] = 0;
    r.anew[tid] = 0;
  }
  if (!V && MODE != kNone) circle.at[tid] = circle_at(tid);
  __syncthreads();
  if (tid < chunk) {
    const int run = r.run[tid] + (warp == 1 && r.slot[tid] >= 0 ? r.warp_runs[0] : 0);
    r.run[tid] = (short)run;
    if (run >= 0) {
      const int before = tid == 0 ? -2 : r.slot[tid - 1];
      if (tid == 0 || before < 0 || before / kBlock != r.slot[tid] / kBlock) r.first_slot[run] = r.slot[tid];
    }
    if (tid == chunk - 1) r.last_block = run >= 0 ? r.slot[tid] / kBlock : -1;
    if (tid == 0) {
      r.count = r.warp_runs[0] + r.warp_runs[1];
      r.lead = min(r.warp_lead[0], r.warp_lead[1]);
    }
  }
  __syncthreads();
  const int count = r.count, last_block = r.last_block;
  const int lead = r.lead;  // the tokens before belong to a run that began earlier
  if (count == 0) return;
  // the last run's tokens behind the chunk (more than 64 only where slots come twice)
  int tail = 0;
  if (last_block >= 0) {
    int seen = 0;
#pragma unroll 1
    for (;;) {
      const int t = t0 + chunk + tail + tid, s = slot_of(t);
      const bool in = s >= 0 && s / kBlock == last_block;
      const int at = chunk + tail + tid;
      if (in && at < kTokens) r.slot[at] = s;
      const unsigned out = __ballot_sync(0xffffffffu, !in);
      if (lane == 0) r.scan[warp] = out ? __ffs(out) - 1 : 32;
      __syncthreads();
      seen = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const int n = r.scan[w];
        if (seen == 32 * w) seen += n;
      }
      __syncthreads();
      tail += seen;
      if (seen < kThreads) break;
    }
  }
  const int total = chunk + tail;
  const int held_tokens = min(total, kTokens);
  // what each run's cache block has so far
  float held = 0.f;
  float* scale_at = nullptr;
  if (tid < count) {
    const int s = r.first_slot[tid], id = s / page, o = (s - id * page) & ~(kBlock - 1);
    scale_at = fp8_scale(a.kv, id, V, g0, o);
    held = *scale_at;
    r.block[tid] = a.kv.pool + (V ? fp8_v(a.kv, id, g0, o, 0) : fp8_k(a.kv, id, g0, o, 0));
  }
  auto run_at = [&](int i) { return i >= total ? -1 : i < chunk ? (int)r.run[i] : count - 1; };
  // V is turned around where runs are long enough to fill stores, by the parts of the runs that lie in 16
  // aligned slots.  (Calls with and without, read-back included: runs of 64 tokens 60 and 88 us, of 32 29.7 and 30.0,
  // of 16 25.4 and 23.1, of 4 15.4 and 13.0.)
  const bool turned = V && total >= 24 * count;
  if (turned) {
    if (tid < held_tokens && run_at(tid) < 0) r.slot[tid] = -1;
    __syncthreads();
    bool first = false;
    int len = 0;
    unsigned m = 0;
    if (tid < kTokens) {
      const int n = held_tokens, s = tid < n ? r.slot[tid] : -1;
      first = s >= 0 && (tid == 0 || s % 16 == 0 || r.slot[tid - 1] != s - 1);
      if (first) {
        len = 1;
        while (tid + len < n && (s + len) % 16 && r.slot[tid + len] == s + len) ++len;
      }
      m = __ballot_sync(0xffffffffu, first);
      if (lane == 0) r.warp_parts[warp] = __popc(m);
    }
    __syncthreads();
    if (first) {
      int at = __popc(m & ((1u << lane) - 1));
      for (int w = 0; w < warp; ++w) at += r.warp_parts[w];
      r.part[at] = tid | (len << 16);
    }
  }

  // ---- values: lane l of a token holds eight dims
  const int rot = V ? 0 : a.rope.rot_dim;
  const LaneDims dims = lane_dims<V ? kNone : MODE>(l, rot);
  long long src = (long long)(a.n_heads + (V ? a.kv.n_kv_heads : 0) + g0) * HD;
  // a lane's pairs (kHalfOdd: the pair of each of its dims) and gains are the same for all of its tokens
  constexpr int kAngles = V || MODE == kNone ? 1 : MODE == kHalfOdd ? 8 : 4;
  uint64_t turns[kAngles];
  float gain[8];
  if (!V) {
#pragma unroll
    for (int k = 0; k < kAngles; ++k) {
      const int d = 8 * l + k, pair = MODE == kHalfOdd ? (d < rot / 2 ? d : d - rot / 2) : 4 * l + k;
      const bool turn = MODE == kHalfOdd ? d < rot : MODE != kNone && k < dims.turned;
      turns[k] = turn ? a.rope.turns[pair] : 0;
    }
    if (a.k_gain) load_gain(a.k_gain, dims, gain);
  }
  auto load = [&](int i, bool on, float (&x)[8]) {  // returns the position
    const int t = t0 + (on ? i : 0);
    load4<F32>(a.qkv, t * a.qkv_ld + src + dims.e0, x);
    load4<F32>(a.qkv, t * a.qkv_ld + src + dims.e1, x + 4);
    return !V && MODE != kNone && on ? a.positions[t] : 0;
  };
  auto turn = [&](float (&x)[8], int pos) {  // by all lanes
    if (V) return;
    if (a.k_gain) scale_head<HD>(x, head_squares<HD>(x), a.eps, gain);
    if (MODE == kNone) return;
    float cs[kAngles], sn[kAngles];
#pragma unroll
    for (int k = 0; k < kAngles; ++k) {  // dims that are not turned: by no angle, and not scaled either
      turn_sincos(circle, pos, turns[k], &sn[k], &cs[k]);
      sn[k] *= a.rope.mscale;
      cs[k] *= a.rope.mscale;
    }
    turn_head<HD, V ? kNone : MODE>(x, cs, sn, l, dims.turned, rot, xs + (warp * NH + sub) * HD);
  };
  auto note_top = [&](float top, int run, int slot) {  // of a token, at its first lane
    if (l == 0 && run >= 0) {
      atomicMax(&r.top[run], __float_as_int(top));
      if (slot % kBlock == 0) r.anew[run] = 1;
    }
  };
  auto top_of = [&](const float (&x)[8]) {  // the largest finite magnitude of a token, by all lanes
    auto over_lanes = [&](float y) {
#pragma unroll
      for (int o = LPH / 2; o > 0; o >>= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, o));
      return y;
    };
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(x[k]));  // (NaN are passed over)
    top = over_lanes(top);
    if (__any_sync(0xffffffffu, top == INFINITY)) {
      float y = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) y = fmaxf(y, fabsf(x[k]) == INFINITY ? 0.f : fabsf(x[k]));
      top = over_lanes(y);
    }
    return top;
  };
  // ---- one head after the other
#pragma unroll 1
  for (int g = g0; g < g1; ++g, src += HD) {
    const long long head_at = (long long)(g - g0) * page * HD;
    if (g != g0) __syncthreads();  // the values of the head before have been read
    if (tid == 0) r.n_grown = 0;
    // V's chain is short, so that its loads decide: four tokens' at once (8192 tokens in all 62.1 us with one, 60.0
    // with four; two of K, which is bound by its instructions, gain nothing, four cost 2.6)
    constexpr int kAtOnce = V && !F32 ? 4 : 1;
#pragma unroll 1
    for (int base = lead + warp * NH + sub; base - sub < held_tokens; base += kAtOnce * kPlaces) {
      int run[kAtOnce], pos[kAtOnce];
      uint4 v[kAtOnce];
      float x[kAtOnce][8];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const int i = base + u * kPlaces;
        run[u] = i < held_tokens ? run_at(i) : -1;
        if (V && !F32)  // as it lies there
          v[u] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.qkv) +
                                                      (t0 + (run[u] >= 0 ? i : 0)) * a.qkv_ld + src + 8 * l));
        else pos[u] = load(i, run[u] >= 0, x[u]);
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const int i = base + u * kPlaces;
        if (i - sub >= held_tokens) break;
        float top;
        if (V && !F32) {
          uint32_t m = larger_bf16(larger_bf16(v[u].x, v[u].y), larger_bf16(v[u].z, v[u].w));
#pragma unroll
          for (int o = LPH / 2; o > 0; o >>= 1) m = larger_bf16(m, __shfl_xor_sync(0xffffffffu, m, o));
          top = fmaxf(fmaxf(0.f, fabsf(bf16_lo(m))), fabsf(bf16_hi(m)));
          if (__any_sync(0xffffffffu, top == INFINITY)) {
            const float y[8] = {bf16_lo(v[u].x), bf16_hi(v[u].x), bf16_lo(v[u].y), bf16_hi(v[u].y),
                                bf16_lo(v[u].z), bf16_hi(v[u].z), bf16_lo(v[u].w), bf16_hi(v[u].w)};
            top = top_of(y);
          }
        } else {
          turn(x[u], pos[u]);
          if (!V && (MODE != kNone || a.k_gain)) {
            uint32_t least = above_middle(x[u][0]);
#pragma unroll
            for (int k = 1; k < 8; ++k) least = min(least, above_middle(x[u][k]));
            if (__any_sync(0xffffffffu, near_middle(least)))
              settle<HD, F32, MODE>(a, t0 + (run[u] >= 0 ? i : 0), g, l, dims, run[u] >= 0, x[u]);
          }
          top = top_of(x[u]);
          v[u] = make_uint4(pack_odd(x[u][0], x[u][1]), pack_odd(x[u][2], x[u][3]), pack_odd(x[u][4], x[u][5]),
                            pack_odd(x[u][6], x[u][7]));
        }
        note_top(top, run[u], run[u] >= 0 ? r.slot[i] : 1);
        if (i < held_tokens) *reinterpret_cast<uint4*>(tile + i * kRow + 16 * l) = v[u];
      }
    }
    auto values = [&](int i, bool on, float (&x)[8]) {  // by all lanes: `on` may differ between tokens
      const int pos = load(i, on, x);
      turn(x, pos);
    };
#pragma unroll 1
    for (int base = kTokens + warp * NH; base < total; base += kPlaces) {  // slots came twice
      float y[8];
      const int i = base + sub, run = run_at(i);
      values(i, run >= 0, y);
      note_top(top_of(y), run, run >= 0 ? a.slots[t0 + i] : 1);
    }
    __syncthreads();

    // ---- exponents
    if (tid < count) {
      const int e_call = exponent_for(__int_as_float(r.top[tid])), e_held = fp8_exponent(held);
      const bool anew = r.anew[tid] != 0;
      const int e = anew ? e_call : max(e_call, e_held);
      r.exponent[tid] = e;
      const float scale = pow2_of(e);
      if (scale != held) *scale_at = scale;
      r.top[tid] = 0;
      if (!anew && e > e_held) {
        const int k = atomicAdd(&r.n_grown, 1);
        r.grown[k] = tid;
        r.down[k] = e_held - e;
      }
      scale_at += page / kBlock;
      if (g + 1 < g1) held = *scale_at;
    }
    __syncthreads();
    const int n_grown = r.n_grown;
    if (n_grown) {
      constexpr int kVecs = kBlock * HD / 16;
#pragma unroll 1
      for (int k = tid; k < n_grown * kVecs; k += kThreads) {
        const int which = k / kVecs, run = r.grown[which];
        uint4* p = reinterpret_cast<uint4*>((r.block[run] + head_at)) + k % kVecs;
        const float f = pow2_of(r.down[which]);
        uint4 c = *p;
        c.x = move_codes(c.x, f);
        c.y = move_codes(c.y, f);
        c.z = move_codes(c.z, f);
        c.w = move_codes(c.w, f);
        *p = c;
      }
      __syncthreads();
    }

    // ---- codes
    auto codes = [&](const float (&y)[8], int run, uint32_t* w) {
      const float f = pow2_of(-r.exponent[run]);
#pragma unroll
      for (int k = 0; k < 2; ++k)
        w[k] = pack_e4m3(y[4 * k] * f, y[4 * k + 1] * f) | (uint32_t)pack_e4m3(y[4 * k + 2] * f, y[4 * k + 3] * f) << 16;
    };
    auto put = [&](const uint32_t* w, int run, int s) {  // straight to the token's slot
      const int o = s % kBlock;
      if (!V) {
        uint8_t* dst = (r.block[run] + head_at) + o * HD;
        *reinterpret_cast<uint32_t*>(dst + dims.e0) = w[0];
        *reinterpret_cast<uint32_t*>(dst + dims.e1) = w[1];
      } else {
        uint8_t* dst = (r.block[run] + head_at) + 8 * l * kBlock + o;
#pragma unroll
        for (int k = 0; k < 8; ++k) dst[k * kBlock] = (uint8_t)(w[k >> 2] >> (8 * (k & 3)));
      }
    };
    if (!turned) {
#pragma unroll 2
      for (int base = lead + warp * NH; base < held_tokens; base += kPlaces) {
        const int i = base + sub, run = i < held_tokens ? run_at(i) : -1;
        if (run < 0) continue;
        const uint4 v = *reinterpret_cast<const uint4*>(tile + i * kRow + 16 * l);
        const float y[8] = {bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y),
                            bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w)};
        uint32_t w[2];
        codes(y, run, w);
        put(w, run, r.slot[i]);
      }
    }
#pragma unroll 1
    for (int base = kTokens + warp * NH; base < total; base += kPlaces) {
      float y[8];
      const int i = base + sub, run = run_at(i);
      values(i, run >= 0, y);
      if (run < 0) continue;
      uint32_t w[2];
      codes(y, run, w);
      put(w, run, a.slots[t0 + i]);
    }
    // V: four dims of a part a thread; 16 positions in one store where a part fills them
    const int parts = turned ? r.warp_parts[0] + r.warp_parts[1] + r.warp_parts[2] + r.warp_parts[3] : 0;
    constexpr int kEights = HD / 32;  // groups of 8 lanes' 4 dims; with 4 parts a warp's stores fill 64-byte rows
#pragma unroll 1
    for (int k = warp; k < (parts + 3) / 4 * kEights; k += kWarps) {
      const int p = k / kEights * 4 + (lane & 3), d = ((k % kEights) * 8 + (lane >> 2)) * 4;
      if (p >= parts) continue;
      const int i = r.part[p] & 0xFFFF, size = r.part[p] >> 16;
      const int run = run_at(i);
      uint8_t* dst = (r.block[run] + head_at) + d * kBlock + r.slot[i] % kBlock;
      const float f = pow2_of(-r.exponent[run]);
      auto row = [&](int j) {
        const uint2 v = *reinterpret_cast<const uint2*>(tile + (i + j) * kRow + 2 * d);
        return pack_e4m3(bf16_lo(v.x) * f, bf16_hi(v.x) * f) | (uint32_t)pack_e4m3(bf16_lo(v.y) * f, bf16_hi(v.y) * f) << 16;
      };
      if (size == 16) {
        uint32_t w[4][4];  // [dim][positions 4j..]
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t q[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) q[e] = row(4 * j + e);
          transpose4(q);
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e][j] = q[e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<uint4*>(dst + e * kBlock) = make_uint4(w[e][0], w[e][1], w[e][2], w[e][3]);
      } else {
#pragma unroll 1
        for (int j = 0; j < size; ++j) {
          const uint32_t w = row(j);
#pragma unroll
          for (int e = 0; e < 4; ++e) dst[e * kBlock + j] = (uint8_t)(w >> (8 * e));
        }
      }
    }  }
}

// Blocks [0, kv_blocks): runs that begin in `chunk` tokens, of the K or V of `some` kv heads; then warps over (token,
// run of `per` q heads), `cuts` of them a token.  (Dealt among one another they took as long.)
template <int HD, bool F32, int MODE>
__global__ void __launch_bounds__(kThreads, 4)
    k_append_fp8(const __grid_constant__ RopeAppendFp8 a, int kv_blocks, int chunk, int some, int cuts, int per) {
  extern __shared__ __align__(16) uint8_t sm[];
  pdl_wait();
  const int warp = threadIdx.x >> 5;
  if ((int)blockIdx.x < kv_blocks) {
    const int heads = a.kv.n_kv_heads, groups = (heads + some - 1) / some;
    const int k = blockIdx.x % (2 * groups), t0 = blockIdx.x / (2 * groups) * chunk;
    const int g0 = k % groups * some, g1 = min(heads, g0 + some);
    if (k < groups) append_runs<HD, F32, MODE, false>(a, t0, chunk, g0, g1, sm);
    else append_runs<HD, F32, MODE, true>(a, t0, chunk, g0, g1, sm);
  } else {
    const long long w = (long long)(blockIdx.x - kv_blocks) * kWarps + warp;
    const int t = (int)(w / cuts), h0 = (int)(w - (long long)t * cuts) * per;
    if (t < a.tokens && h0 < a.n_heads)
      rotate_heads<HD, F32, MODE>(a, t, h0, min(a.n_heads, h0 + per), reinterpret_cast<float*>(sm) + warp * 256);
  }
  pdl_launch();
}

template <int HD, bool F32, int MODE>
cudaError_t launch(const RopeAppendFp8& a, cudaStream_t s) {
  constexpr int kStep = 32 / (HD / 8) * kUnroll;  // heads a warp has in flight
  constexpr size_t smem = kv_smem<HD, MODE>();
  static_assert(smem >= kWarps * 256 * sizeof(float) && smem <= 48 * 1024, "shared memory");
  const int steps = (a.n_heads + kStep - 1) / kStep;
  int cuts = (kTargetWarps + a.tokens - 1) / a.tokens;
  cuts = cuts < steps ? cuts : steps;
  const int per = (steps + cuts - 1) / cuts * kStep;
  cuts = (a.n_heads + per - 1) / per;
  const long long q = ((long long)a.tokens * cuts + kWarps - 1) / kWarps;
  // A block's runs are set up once, so that many tokens and two heads a block save instructions; with fewer there
  // are more blocks.  8192 tokens of 8 heads of 128 (read-back included) 79.5 us with 16 tokens a block, 65.5 with
  // 64, 59.9 with two heads of them, 65.3 with four; 4096 42.5, 35.2, 33.4; 1024 15.4, 13.3, 16.7; 256 rows of one
  // token 25.5, 32.3, 45.3; 8 of them 7.0, 8.4, 11.
  const int heads = a.kv.n_kv_heads;
  auto blocks = [&](int chunk, int some) {
    return (long long)((a.tokens + chunk - 1) / chunk) * 2 * ((heads + some - 1) / some);
  };
  const int chunk = blocks(kMostChunk, 1) >= kResident / 4 ? kMostChunk : 16;
  const int some = blocks(chunk, 2) >= kResident ? 2 : 1;
  const long long kv = blocks(chunk, some);
  if (q + kv > 0x7FFFFFFF) return cudaErrorInvalidValue;
  return launch_pdl(k_append_fp8<HD, F32, MODE>, dim3((unsigned)(q + kv)), dim3(kThreads), smem, s, a,
                    (int)kv, chunk, some, cuts, per);
}

template <int HD, bool F32>
cudaError_t launch_mode(const RopeAppendFp8& a, cudaStream_t s) {
  if (a.rope.rot_dim == 0) return launch<HD, F32, kNone>(a, s);
  if (a.rope.layout == CBT_ROPE_INTERLEAVED) return launch<HD, F32, kInter>(a, s);
  return a.rope.rot_dim % 8 ? launch<HD, F32, kHalfOdd>(a, s) : launch<HD, F32, kHalf>(a, s);
}

}  // namespace

cudaError_t launch_append_fp8(const RopeAppendFp8& a, cudaStream_t s) {
  if (a.kv.head_dim == 128) return a.f32 ? launch_mode<128, true>(a, s) : launch_mode<128, false>(a, s);
  return a.f32 ? launch_mode<64, true>(a, s) : launch_mode<64, false>(a, s);
}
