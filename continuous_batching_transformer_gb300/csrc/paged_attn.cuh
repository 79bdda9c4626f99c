// paged_attn.cuh -- what the attention kernels over a paged cache share: which keys a query sees,
// the row checks, and small device helpers.
#pragma once
#include <cuda_bf16.h>

#include "paged.h"
#include "tc_common.cuh"

constexpr float kLog2e = 1.4426950408889634f;

// Keys the query at position p sees: j <= p with j > p - window or j < sinks (window 0: all).
// They lie in the C-key chunks [0, ns) (sinks below the window's first chunk) and [ws, last].
struct Seen {
  int ns, ws, n;  // n chunks in all
  CBT_HD int chunk(int i) const { return i < ns ? i : ws + i - ns; }
};
CBT_HD int first_in_window(int p, int window) { return window && p >= window ? p - window + 1 : 0; }
// chunks that any of the queries at positions [p0, p1] sees (p1 < 0: none)
template <int C>
CBT_HD Seen seen_chunks(int p0, int p1, int window, int sinks) {
  Seen s{0, 0, 0};
  if (p1 < 0) return s;
  s.ws = first_in_window(p0 < 0 ? 0 : p0, window) / C;
  const int sc = (int)(((long long)sinks + C - 1) / C);
  s.ns = sc < s.ws ? sc : s.ws;
  s.n = s.ns + p1 / C - s.ws + 1;
  return s;
}
CBT_HD bool sees(int j, int p, int window, int sinks) {
  return j <= p && (!window || j > p - window || j < sinks);
}

// 2^x in fp32 (the hardware approximation: 2 ulp, results below 2^-126 become 0)
CBT_D float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two floats to a packed bf16 pair (lo in the low half), each rounded to nearest even
CBT_D uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
CBT_D uint16_t round_bf16(float x) {
  uint16_t r;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(x));
  return r;
}

// AND mask of 8 bf16 keys (one 16-byte unit) from their 8 visibility bits
CBT_D uint4 key_mask(uint32_t bits) {
  uint4 m;
  m.x = ((bits & 1) ? 0xFFFFu : 0u) | ((bits & 2) ? 0xFFFF0000u : 0u);
  m.y = ((bits & 4) ? 0xFFFFu : 0u) | ((bits & 8) ? 0xFFFF0000u : 0u);
  m.z = ((bits & 16) ? 0xFFFFu : 0u) | ((bits & 32) ? 0xFFFF0000u : 0u);
  m.w = ((bits & 64) ? 0xFFFFu : 0u) | ((bits & 128) ? 0xFFFF0000u : 0u);
  return m;
}

// What follows lets the compiler see that a value is the same in the whole warp, and that one
// thread runs a branch: matrix instructions take their operands from uniform registers, and moving
// them there from a lane's costs more than the instruction.
CBT_D int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }
CBT_D bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}

CBT_D void wait_timeout(int* err, volatile int* abort_flag, int where) {
  *abort_flag = 1;
  set_device_error(err, CBT_DEV_TIMEOUT, 400 + where);
}
// Bounded wait for a phase.  While it is incomplete the thread is suspended for up to a microsecond
// a poll: spinning warps take issue slots from those that work.
CBT_D bool wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
#pragma unroll 1
  for (uint32_t i = 0; i < 1u << 22; ++i) {
    if (tc::mbar_try_wait_sleep(bar, parity, 1000)) return true;
    if (*abort_flag) return false;
  }
  return false;
}

// The same for the copies in flight at exit, which an abort does not call off
CBT_D void wait_landed(uint64_t* bar, uint32_t parity) {
#pragma unroll 1
  for (uint32_t i = 0; i < 1u << 22; ++i)
    if (tc::mbar_try_wait_sleep(bar, parity, 1000)) return;
}

// The query tokens of row b: [t0, t0 + n) of the call's rows, the last at position len - 1.
// n = -1: the row cannot be taken (bad is set).
struct RowTokens {
  int t0, n, len;
  bool bad;
};
template <bool L2 = false, class Kv>  // L2: what this SM holds of them is not asked
CBT_D RowTokens row_tokens(const PagedAttnOn<Kv>& a, int b) {
  auto at = [](const int32_t* p) { return L2 ? __ldcg(p) : *p; };
  RowTokens r{b, 1, at(a.lens + b), false};
  if (a.cu) {
    r.t0 = at(a.cu + b);
    const int t1 = at(a.cu + b + 1);
    r.bad = r.t0 < 0 || t1 < r.t0 || t1 > a.tokens || t1 - r.t0 > a.max_q;
    r.n = t1 - r.t0;
  }
  r.bad = r.bad || r.len < 0 || r.len > a.max_kv ||
          r.len > (long long)a.max_pages * a.kv.page_tokens;
  if (r.bad) r.n = -1;
  return r;
}

// Visible keys among the 32 W from k0 on, as W words of bits, for a query at position hi whose
// window starts at lo (for a run of queries: the last one's position, the first one's window)
CBT_D uint32_t ones_below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; }
template <int W>
CBT_D void seen_bits(int k0, int hi, int lo, int sinks, uint32_t (&w)[W]) {
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const int b = k0 + 32 * i;
    w[i] = ones_below(hi + 1 - b) & (~ones_below(lo - b) | ones_below(sinks - b));
  }
}

// The pool as K rows of head_dim and as V^T rows of 64 keys (128 bytes)
bool paged_maps(const PagedKv& kv, CUtensorMap* tk, CUtensorMap* tv);
