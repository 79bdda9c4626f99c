// paged_decode_fp8.cu -- attention of one new token per row over a paged cache in 8 bits, split over the
// cache's length and joined.
//
// The contraction is turned around as over bf16 pages (paged_decode.cu): per 128-key chunk, S^T[key]
// [head] = K . Q^T and O^T[dim][head] = V^T . P^T, with K and V taken by the tensor cores as the codes
// they are (e4m3, M = 128).  What multiplies them is split into codes too, each part in columns of its
// own, so that nothing but a last rounding is lost:
//   q   two parts (bf16 has eight bits of mantissa, a part four): exact down to 2^-12 of the head's largest
//       element, off by at most 2^-22 of it below;
//   p   four, of the weight in fp16: 2^-11 of each weight, and 2^-24 of what the reference stands for.
// A block's scales are powers of two.  K's multiplies its scores; V's is an addition to them, in units of
// log2: the weights are 2^(s_j + e_j - u - m), e_j the exponent of j's block, u a unit that O is summed in and m a
// reference, and the sum l takes them times 2^(u - e_j).
//
// The reference is the item's first chunk's largest s_j + e_j - u, and is raised where one passes it by kSlack: so
// most chunks look for no maximum, the sums stay with the keys' threads, and O stays in tensor memory until the
// item ends or reference or unit move.  The unit follows V's exponents, 0 <= u - e_j <= kSpread: a weight beside a
// block of a far larger scale has the bits that it has alone.  Where a chunk's exponents leave that, O goes to
// registers first, and a reference that stood above what it needs for the scales so far is lowered as the unit
// rises: a block of small weights and large values keeps its bits as well.  (m <= s_max and m + u <= the largest
// s + e: what is lost of a weight is 2^-20 of the row's largest at most, of weight times scale 2^-20 of
// the largest of those.)  A chunk whose two halves lie further apart than kSpread takes them one after the other.
//
// Bound by HBM: 2 head_dim bytes of K and V per position and kv head, while a chunk's instructions hide under
// them (up to 8 q heads of 128 on a kv head; heads of 64 have half the bytes for as many).  Items, runs and
// their join are those of paged_split.cuh.  Measured (graph replays, join included): 32 rows of 8192 to 16384
// positions, 32 / 8 heads of 128, 125 us = 6.5 TB/s, 97 % of the measured copy rate; with 64 q heads 138, with
// heads of 64 91 us (67 %), 64 of them 128 (47 %); 16 rows through a window of 4096 27.8 us (72 %); 8 rows of
// 512 to 4096 11.7 us; one row of 100 4.9 us.  Where every chunk's halves lie apart 32 rows of 12288 take 155 us
// for 127, where every other chunk's scales lie far from the last one's as long as with one scale.
#include <type_traits>

#include "fp8_tc.cuh"
#include "paged_split.cuh"

namespace {

constexpr int kCompute = 128;  // warps 0..3; warp 4 requests tiles
constexpr int kParts = 4;      // of a weight
using Attn = PagedAttnFp8;

template <int HD, int GT>
struct Shape {
  static constexpr int kNQ = 16, kNP = kParts * GT <= 16 ? 16 : 32;  // columns of S^T and of O^T
  static constexpr int kK = kSub * HD, kVHalf = kBlock * HD, kQ = kNQ * HD, kP = kNP * kSub;
  static constexpr uint32_t kCols = kNQ + kNP <= 32 ? 32 : 64;  // of tensor memory: S^T, then O^T
  // V^T's halves span M = 128 rows: for head_dim 64 the second one's rows past 64 lie in what follows
  static constexpr int kTiles = kK + 2 * kVHalf + kQ + kP;
  static constexpr size_t kSmem = 1024 + (kTiles > kK + 3 * kVHalf ? kTiles : kK + 3 * kVHalf) + 1024;
  static constexpr int kCtas = 4;  // of an SM (five, with fewer registers, took up to 11 % longer, three 3 %)
  static_assert(kCtas * (kSmem + 1024) <= 228 * 1024 && kCtas * kCols <= 512, "shared and tensor memory");
};

// By how many powers of two weights may pass 1 (one whose score is the reference) before the reference is
// raised: 2^8 is below the largest code.
constexpr float kSlack = 8.f;
// How far V's exponents may lie below the unit: see above; the parts lose 2^-24 and fp16 2^-25.  (Real blocks differ
// by less, so that the unit rarely moves.)
constexpr int kSpread = 3;
constexpr float kPart = 16.f;  // of one part of q to the next one's unit
// ... of a weight: a code leaves a rest of a 16th of its power of two, of eleven bits the second one a 32nd of its
// unit's and the third one nothing, or 2^-10 each.  (Weights up to 2^8: parts of at most 256, 128, 128 and 1/4,
// whose sum is off by 2^-24 at most.)
CBT_HD constexpr float part_unit(int k) { return k == 0 ? 16.f : k == 1 ? 32.f : 256.f; }

// part_unit(k) (a - b), of two pairs of fp16
CBT_D uint32_t rest_of(uint32_t a, uint32_t b, int k) {
  uint32_t r;
  asm("{\n .reg .b32 d;\n sub.rn.f16x2 d, %1, %2;\n mul.rn.f16x2 %0, d, %3;\n}\n"
      : "=r"(r)
      : "r"(a), "r"(b), "r"(k == 0 ? 0x4C004C00u : k == 1 ? 0x50005000u : 0x5C005C00u));
  return r;
}

// What a chunk's requester hands to the softmax of each half's K and V scales, and V's unit
struct Scales {
  struct Half {
    float k_unit;  // K's scale
    float ve;      // V's exponent, from the unit
    float v_down;  // 2^-ve
  } half[2];
  int unit[2];  // V's, of the chunk; where the halves lie too far apart for one, of either
  int moves;    // 0: the unit is that of the chunk before, or an item begins with it; kMoves, or kApart
};
constexpr int kMoves = 1, kApart = 2;

// GT: the group's q heads rounded up to 1, 2, 4 or 8
template <int HD, int GT>
__global__ void __launch_bounds__(kCompute + 32, (Shape<HD, GT>::kCtas))
    k_decode_fp8(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                 const __grid_constant__ Attn a, float* __restrict__ part_o, float2* __restrict__ part_ml) {
  using S = Shape<HD, GT>;
  constexpr uint32_t kIdescS = tc::idesc_e4m3(128, S::kNQ), kIdescO = tc::idesc_e4m3(128, S::kNP);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sK = smem;                   // [128 keys][HD]
  uint8_t* sV = sK + S::kK;             // [64-key half][HD dims][64 keys]
  uint8_t* sP = sV + 2 * S::kVHalf;     // [part, head][128 keys]
  uint8_t* sQ = sP + S::kP;             // [part, head][HD]
  uint8_t* end = smem + S::kSmem - 2048;
  uint64_t* bars = reinterpret_cast<uint64_t*>(end);
  uint64_t *kfull = bars, *vfull = bars + 1, *kempty = bars + 2, *vempty = bars + 3;
  uint64_t *bar_s = bars + 4, *bar_o = bars + 5;
  Scales* scales = reinterpret_cast<Scales*>(bars + 6);  // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(scales + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* red = reinterpret_cast<float*>(tmem_slot + 2); // [4 warps][8 heads]
  float* l_run = red + 32;                              // [8]
  float* q_unit = l_run + 8;                            // [8] a score's unit, in log2 units
  float* most = q_unit + 8;                             // [8] the highest m + u before the unit moved

  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const Layout lay = layout_of(a);
  const int per_row = a.kv.n_kv_heads * lay.groups;
  if (tid == 0) {
    // kempty: the MMAs, and every warp has seen that the tile was full
    for (int i = 0; i < 6; ++i) tc::mbar_init(&bars[i], &bars[i] == kempty ? 1 + 4 : 1);
    *abort_flag = 0;
    tc::mbar_fence_init();
    tc::tma_prefetch_desc(&tk);
    tc::tma_prefetch_desc(&tv);
  }
  if (warp == 0) tc::tmem_alloc(tmem_slot, S::kCols);
  // heads and parts that no item fills stay zero
  for (int i = tid; i < (S::kP + S::kQ) / 16; i += kCompute + 32)
    reinterpret_cast<uint4*>(sP)[i] = make_uint4(0, 0, 0, 0);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);
  pdl_wait();
  Cursor<Attn> cur;
  cur.load(a, per_row, 0, 0);

  if (warp == 4) {
    // ---- tile requests: K, then V of each chunk.  The next chunk's pages and scales are looked up while
    // V's buffer is awaited, so that K's stays empty for a wait only.
    const uint64_t pol = tc::policy_evict_first();
    uint32_t n = 0, nk = 0, nv = 0;  // chunks, and tiles of K and of V requested
    // what is handed over of the next chunk's scales: V's unit and its first half's, and, lane 0 and 1, a half's own
    int unit = 0, unit0 = 0, moves = 0;
    float k_unit = 0.f, v_down = 0.f, ve = 0.f;
    bool ok = true;
    const int P = a.kv.page_tokens;
    // a chunk's halves of 64 keys that hold a key the query sees, and where they lie; lane e has half
    // e's scales
    struct Chunk {
      unsigned halves;
      bool first;  // of an item: any unit will do, since nothing has been summed
      int k[2], v[2];
      float ks, vs;
    };
    int it = blockIdx.x, i = 0;
    bool have = cur.seek(a, per_row, it);
    Item w{};
    if (have) {
      w = item_at(cur, a, lay.groups, it);
      i = w.i0;
    }
    auto next = [&]() {  // halves 0: no chunk is left
      Chunk c{};
      while (have && i >= w.i1) {
        it += gridDim.x;
        have = cur.seek(a, per_row, it);
        if (have) {
          w = item_at(cur, a, lay.groups, it);
          i = w.i0;
        }
      }
      if (!have) return c;
      c.first = i == w.i0;
      // lanes 0 and 1: a half each
      const int k0 = w.seen.chunk(i++) * kSub + kBlock * lane;
      int kat = 0, vat = 0;
      const bool want = lane < 2 && k0 <= w.p && (sees(k0, w.p, a.window, a.sinks) ||
                                                   sees(min(k0 + 63, w.p), w.p, a.window, a.sinks));
      if (want) {
        const int pg = k0 / P, o = k0 - pg * P;
        int id = a.table[(size_t)w.b * a.max_pages + pg];
        if (id < 0 || id >= a.kv.n_pages) {
          set_device_error(a.err, CBT_DEV_PAGE_ID, w.b);
          id = 0;  // a page that exists: the row's outputs are unspecified
        }
        kat = (int)(fp8_k(a.kv, id, w.g, o, 0) >> 8);
        vat = (int)(fp8_v(a.kv, id, w.g, o, 0) >> 8);
        c.ks = *fp8_scale(a.kv, id, 0, w.g, o);
        c.vs = *fp8_scale(a.kv, id, 1, w.g, o);
      }
      c.halves = __ballot_sync(0xffffffffu, want);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        c.k[e] = __shfl_sync(0xffffffffu, kat, e);
        c.v[e] = __shfl_sync(0xffffffffu, vat, e);
      }
      return c;
    };
    // (where its scales are awaited: behind the requests for the chunk before)
    auto scales_of = [&](const Chunk& c) {
      const int e = fp8_exponent(c.vs);
      // a half that is not there has the other one's scale
      const int v0 = __shfl_sync(0xffffffffu, e, c.halves == 2), v1 = __shfl_sync(0xffffffffu, e, c.halves != 1);
      const int lo = min(v0, v1), hi = max(v0, v1);
      moves = hi - lo > kSpread ? kApart : !c.first && (hi > unit || lo < unit - kSpread) ? kMoves : 0;
      if (moves || c.first) unit = min(lo + kSpread, hi + 1);
      unit0 = unit;
      int off = (lane ? v1 : v0) - unit;
      if (moves == kApart) {
        unit0 = v0;
        unit = v1;
        off = 0;
      }
      k_unit = pow2_of(fp8_exponent(c.ks));
      ve = (float)off;
      v_down = pow2_of(-off);
    };
    Chunk c = next();
    scales_of(c);
#pragma unroll 1
    for (; c.halves; ++n) {
      const uint32_t bytes = __popc(c.halves) * S::kVHalf;
      ok = __all_sync(0xffffffffu, wait_or_abort(kempty, (n & 1) ^ 1, abort_flag));
      if (!ok) break;
      if (elect_one()) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (c.halves >> e & 1) tc::tma_load_rows(sK + e * S::kVHalf, &tk, kfull, c.k[e], pol);
      }
      // (the tile's bytes may land before they are expected: the phase waits for the arrival)
      Scales& out = scales[n & 1];
      if (lane < 2) {
        out.half[lane] = {k_unit, ve, v_down};
        out.unit[lane] = lane ? unit : unit0;
      } else if (lane == 2) {
        out.moves = moves;
      }
      __syncwarp();
      if (elect_one()) tc::mbar_expect_tx(kfull, bytes);
      ++nk;
      const Chunk nxt = next();
      ok = __all_sync(0xffffffffu, wait_or_abort(vempty, (n & 1) ^ 1, abort_flag));
      if (!ok) break;
      if (elect_one()) {
        tc::mbar_expect_tx(vfull, bytes);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (c.halves >> e & 1) tc::tma_load_rows(sV + e * S::kVHalf, &tv, vfull, c.v[e], pol);
      }
      ++nv;
      c = nxt;
      if (c.halves) scales_of(c);
    }
    if (!ok && lane == 0) wait_timeout(a.err, abort_flag, 21);
    // no copies in flight at exit
    if (nk) wait_landed(kfull, (nk - 1) & 1);
    if (nv) wait_landed(vfull, (nv - 1) & 1);
  } else {
    uint32_t n = 0, no = 0;     // chunks done, products with V asked for
    int unit = 0;               // V's, of the product in tensor memory
    bool ok = true;
    const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
    const float scale2 = a.scale * kLog2e;  // scores in units of log2
    constexpr int kQUnits = HD / 8;         // 16-byte pieces of a head
    const int qh = tid / kQUnits, qu = tid % kQUnits;
    // this thread's piece of the next item's q
    auto load_q = [&](const Item& w) {
      return qh < w.heads
                 ? *reinterpret_cast<const uint4*>(a.q + w.t * a.q_ld + (long long)(w.head0 + qh) * HD + qu * 8)
                 : make_uint4(0, 0, 0, 0);
    };
    // ... as two parts of codes; by all lanes (a head's pieces lie with lanes next to each other)
    auto store_q = [&](const uint4& v) {
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
      float x[8], top = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[2 * e] = bf16_lo(u[e]);
        x[2 * e + 1] = bf16_hi(u[e]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fabsf(x[e]) <= 3.4028235e38f ? fmaxf(top, fabsf(x[e])) : top;
#pragma unroll
      for (int o = kQUnits / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int fit = fit_exponent(top);
      const float f = pow2_of(fit);
      uint32_t part[2][2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        part[0][e] = part[1][e] = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float y[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float z = x[4 * e + 2 * j + k];
            y[k] = fabsf(z) <= 3.4028235e38f ? z * f : __int_as_float(0x7FC00000);  // infinities: NaN
          }
          const uint16_t hi = pack_e4m3(y[0], y[1]);
          const uint32_t back = e4m3_to_f16(hi);
          const uint16_t lo = pack_e4m3((y[0] - f16_lo(back)) * kPart, (y[1] - f16_hi(back)) * kPart);
          part[0][e] |= (uint32_t)hi << (16 * j);
          part[1][e] |= (uint32_t)lo << (16 * j);
        }
      }
      if (qh < GT) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
          *reinterpret_cast<uint2*>(sQ + tc::swz<HD>(k * GT + qh, qu * 8)) = make_uint2(part[k][0], part[k][1]);
        if (qu == 0) q_unit[qh] = scale2 * pow2_of(-fit);
      }
    };
    int it = blockIdx.x;
    bool have = cur.seek(a, per_row, it);
    Item w{}, nxt{};
    uint4 qv = make_uint4(0, 0, 0, 0);
    if (have) {
      nxt = item_at(cur, a, lay.groups, it);
      qv = load_q(nxt);
    }
    while (have && ok) {
      w = nxt;
      // the MMAs that read the last item's Q have completed (bar_s)
      store_q(qv);
      it += gridDim.x;
      have = cur.seek(a, per_row, it);
      if (have) {
        nxt = item_at(cur, a, lay.groups, it);
        qv = load_q(nxt);
      }
      // m_run is kept by every thread, each from the same values in the same order; l_own are its own keys'
      float m_run[GT], oacc[GT], l_own[GT];
      uint32_t acc = 0;  // O in tensor memory holds something
#pragma unroll
      for (int h = 0; h < GT; ++h) {
        m_run[h] = -INFINITY;
        oacc[h] = l_own[h] = 0.f;
      }
      if (tid < GT) most[tid] = -INFINITY;
      // this thread's dim of O, from its parts
      auto add_o = [&]() {
        constexpr int kAtOnce = 16 / GT < kParts ? 16 / GT : kParts;  // parts in 16 columns
        float o[GT];
#pragma unroll
        for (int k0 = kParts - kAtOnce; k0 >= 0; k0 -= kAtOnce) {
          uint32_t part[16];
          tc::tmem_ld16(lane_base + S::kNQ + k0 * GT, part);
          tc::tmem_ld_wait();
#pragma unroll
          for (int h = 0; h < GT; ++h) {
#pragma unroll
            for (int k = kAtOnce - 1; k >= 0; --k) {
              const float x = __uint_as_float(part[k * GT + h]);
              o[h] = k0 + k == kParts - 1 ? x : fmaf(o[h], 1.f / part_unit(k0 + k), x);
            }
          }
        }
#pragma unroll
        for (int h = 0; h < GT; ++h) oacc[h] = fmaf(o[h], pow2_of(unit), oacc[h]);
      };
      tc::fence_proxy_async_smem();
      tc::named_bar_sync(1, kCompute);

      for (int i = w.i0; i < w.i1; ++i, ++n) {
        if (!__all_sync(0xffffffffu, wait_or_abort(kfull, n & 1, abort_flag))) {
          if (lane == 0) wait_timeout(a.err, abort_flag, 22);
        } else {
          if (lane == 0) tc::mbar_arrive(kempty);
          if (warp == 0 && elect_one()) {
            tc::tc_fence_after();
#pragma unroll
            for (int k = 0; k < HD / 32; ++k)
              tc::mma_e4m3(tmem, tc::sdesc_rows<HD>(tc::smem_u32(sK)) + 2 * k,
                           tc::sdesc_rows<HD>(tc::smem_u32(sQ)) + 2 * k, kIdescS, k > 0 ? 1u : 0u);
            tc::mma_commit(bar_s);
            tc::mma_commit(kempty);
          }
        }
        const int k0 = w.seen.chunk(i) * kSub;
        const bool valid = sees(k0 + tid, w.p, a.window, a.sinks);
        const uint32_t vb = __ballot_sync(0xffffffffu, valid);
        const Scales& sc = scales[n & 1];
        const Scales::Half& mine = sc.half[tid >> 6];
        const float k_unit = mine.k_unit, ve = mine.ve;
        const int moves = sc.moves;
        bool bad = !wait_or_abort(bar_s, n & 1, abort_flag);
        __syncwarp();
        tc::tc_fence_after();
        uint32_t raw[16];
        tc::tmem_ld16(lane_base, raw);
        tc::tmem_ld_wait();
        tc::tc_fence_before();
        float s[GT];
#pragma unroll
        for (int h = 0; h < GT; ++h) {
          const float both = fmaf(__uint_as_float(raw[GT + h]), 1.f / kPart, __uint_as_float(raw[h]));
          s[h] = valid ? fmaf(both * k_unit, q_unit[h], ve) : -INFINITY;
        }
        // the weights of the product before have been read
        if (no) bad = bad || !wait_or_abort(bar_o, (no - 1) & 1, abort_flag);
        __syncwarp();
        if (vb != 0xffffffffu) {
          // masked keys: their V may hold anything, so it is zeroed (their weights are zero), each warp its own
          bad = bad || !wait_or_abort(vfull, n & 1, abort_flag);
          __syncwarp();
          uint8_t* v = sV + (warp >> 1) * S::kVHalf;
#pragma unroll 1
          for (int u = 0; u < 2; ++u) {  // 16 keys
            const uint32_t bits = (vb >> (16 * u)) & 0xFFFFu;
            if (bits == 0xFFFFu) continue;
            const uint4 mk = code_mask(bits);
            for (int d = lane; d < HD; d += 32) {
              uint4* at = reinterpret_cast<uint4*>(v + tc::swz<64>(d, 32 * (warp & 1) + 16 * u));
              uint4 z = make_uint4(0, 0, 0, 0);
              if (bits) z = *at;
              *at = make_uint4(z.x & mk.x, z.y & mk.y, z.z & mk.z, z.w & mk.w);
            }
          }
        }
        // O += P V, by one thread; `last`: of the chunk
        auto multiply = [&](bool last) {
          if (warp == 0) {
            if (!__all_sync(0xffffffffu, wait_or_abort(vfull, n & 1, abort_flag))) {
              if (lane == 0) wait_timeout(a.err, abort_flag, 24);
            } else if (elect_one()) {
              tc::tc_fence_after();
#pragma unroll
              for (int k = 0; k < kSub / 32; ++k)
                tc::mma_e4m3(tmem + S::kNQ, tc::sdesc_rows<64>(tc::smem_u32(sV + (k >> 1) * S::kVHalf)) + 2 * (k & 1),
                             tc::sdesc_rows<128>(tc::smem_u32(sP)) + 2 * k, kIdescO, acc || k > 0 ? 1u : 0u);
              tc::mma_commit(bar_o);
              if (last) tc::mma_commit(vempty);
            }
          }
          acc = 1;
          ++no;
        };
        // O leaves tensor memory
        auto take_o = [&]() {
          if (!acc) return;
          tc::tc_fence_after();
          add_o();
          tc::tc_fence_before();
          acc = 0;
        };
        // The chunk's weights and their product.  (Two copies of the code: with the unit's moves in the one that most
        // chunks take, that one had a tenth more instructions.)
        auto weigh = [&](auto moving) {
          bool raise = i == w.i0 || moving.value, second = false;  // second: half's turn, of two
#pragma unroll 1
          for (;;) {
            const bool turn = valid && (!moving.value || moves != kApart || tid >> 6 == (int)second);
            if (raise) {
              float mx[GT];
#pragma unroll
              for (int h = 0; h < GT; ++h) mx[h] = !moving.value || turn ? s[h] : -INFINITY;
              warp_reduce_n<GT, true>(mx);
              if (lane == 0) {
#pragma unroll
                for (int h = 0; h < GT; ++h) red[warp * 8 + h] = mx[h];
              }
              if (moving.value && tid == 0) {
#pragma unroll
                for (int h = 0; h < GT; ++h) most[h] = fmaxf(most[h], m_run[h] + (float)unit);
              }
              tc::named_bar_sync(1, kCompute);
              take_o();
              unit = sc.unit[second];
#pragma unroll
              for (int h = 0; h < GT; ++h) {
                // (O and l, in units of 2^m, stay in fp32's range: O's elements are below 2^(most - m + 18 + kSlack))
                const float mo = m_run[h], low = moving.value ? fminf(mo, most[h] - (float)unit) : mo;
                const float mn = fmaxf(low, fmaxf(fmaxf(red[h], red[8 + h]), fmaxf(red[16 + h], red[24 + h])));
                const float scl = mo == -INFINITY ? 0.f : ex2(mo - mn);
                oacc[h] *= scl;
                l_own[h] *= scl;
                m_run[h] = mn;
              }
            }
            bool over = false;
            uint8_t* dst = sP + (tid & 15);
            float p[GT];
#pragma unroll
            for (int h = 0; h < GT; ++h) {
              // (scores of -inf, as masked keys have, alone so far: weights of 0, not of exp(-inf + inf))
              p[h] = moving.value && !turn ? 0.f : ex2(s[h] - (m_run[h] == -INFINITY ? 0.f : m_run[h]));
              over = over || s[h] > m_run[h] + kSlack;
            }
#pragma unroll
            for (int h = 0; h < GT; h += 2) {
              uint32_t y = pack_f16(p[h], h + 1 < GT ? p[h + 1 < GT ? h + 1 : h] : 0.f);
#pragma unroll
              for (int k = 0; k < kParts; ++k) {
                const uint16_t code = f16_to_e4m3(y);
                dst[tc::swz<128>(k * GT + h, tid & ~15)] = (uint8_t)code;
                if (h + 1 < GT) dst[tc::swz<128>(k * GT + h + 1, tid & ~15)] = (uint8_t)(code >> 8);
                if (k + 1 < kParts) y = rest_of(y, e4m3_to_f16(code), k);
              }
            }
            tc::fence_proxy_async_smem();
            if (!tc::named_bar_any(2, kCompute, bad || (over && !raise))) {
#pragma unroll
              for (int h = 0; h < GT; ++h) l_own[h] = fmaf(p[h], mine.v_down, l_own[h]);
              if (!moving.value || moves != kApart || second) break;
              // the second half's turn, once the first one's weights have been read
              multiply(false);
              bad = !wait_or_abort(bar_o, (no - 1) & 1, abort_flag);
              __syncwarp();
              second = true;
              continue;
            }
            // something has passed a reference, or has failed
            if (tc::named_bar_any(2, kCompute, bad)) {
              ok = false;
              break;
            }
            raise = true;
          }
          if (ok) multiply(true);
        };
        if (moves) weigh(std::true_type());
        else weigh(std::false_type());
        if (!ok) break;
      }
      if (!ok) break;
      if (acc) {
        const bool bad = !wait_or_abort(bar_o, (no - 1) & 1, abort_flag);
        if (tc::named_bar_any(2, kCompute, bad)) {
          ok = false;
          break;
        }
        tc::tc_fence_after();
        add_o();
        tc::tc_fence_before();
      }
      warp_reduce_n<GT, false>(l_own);
      if (lane == 0) {
#pragma unroll
        for (int h = 0; h < GT; ++h) red[warp * 8 + h] = l_own[h];
      }
      tc::named_bar_sync(1, kCompute);
      if (tid < GT) l_run[tid] = (red[tid] + red[8 + tid]) + (red[16 + tid] + red[24 + tid]);
      tc::named_bar_sync(1, kCompute);
      if (w.runs == 1) {
        if (tid < HD) {
#pragma unroll
          for (int h = 0; h < GT; ++h) {
            if (h >= w.heads) break;
            const float o = w.seen.n ? oacc[h] / l_run[h] : 0.f;
            const long long at = w.t * a.out_ld + (long long)(w.head0 + h) * HD + tid;
            if (a.f32) static_cast<float*>(a.out)[at] = o;
            else static_cast<uint16_t*>(a.out)[at] = round_bf16(o);
          }
        }
      } else {
        const size_t base = ((size_t)w.b * a.n_heads + w.head0) * lay.max_runs + w.run;
        if (tid < HD) {
#pragma unroll
          for (int h = 0; h < GT; ++h)
            if (h < w.heads) part_o[(base + (size_t)h * lay.max_runs) * HD + tid] = oacc[h];
        }
        if (tid < w.heads) {
          float mm = m_run[0];
#pragma unroll
          for (int h = 1; h < GT; ++h)
            if (h == tid) mm = m_run[h];
          part_ml[base + (size_t)tid * lay.max_runs] = make_float2(mm, l_run[tid]);
        }
      }
      tc::named_bar_sync(1, kCompute);
    }
  }
  // only now: the join's blocks, resident early, would take room from those that stream
  pdl_launch();
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, S::kCols);
  }
}

template <int HD, int GT>
cudaError_t launch_gt(const CUtensorMap& tk, const CUtensorMap& tv, const Attn& a, long long items, int num_sms,
                      float* po, float2* pml, cudaStream_t s) {
  using Sh = Shape<HD, GT>;
  const cudaError_t rc = cudaFuncSetAttribute(k_decode_fp8<HD, GT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                              (int)Sh::kSmem);
  if (rc != cudaSuccess) return rc;
  const int most = Sh::kCtas * num_sms;
  return launch_pdl(k_decode_fp8<HD, GT>, dim3((unsigned)(items < most ? items : most)), dim3(kCompute + 32), Sh::kSmem,
                    s, tk, tv, a, po, pml);
}

template <int HD>
cudaError_t launch_hd(const CUtensorMap& tk, const CUtensorMap& tv, const Attn& a, int num_sms, cudaStream_t s) {
  const Layout lay = layout_of(a);
  if (lay.max_runs > 1 && !a.ws) return cudaErrorInvalidValue;
  const size_t n = (size_t)a.rows * a.n_heads * lay.max_runs;
  float* po = reinterpret_cast<float*>(a.ws);
  float2* pml = reinterpret_cast<float2*>(a.ws + n * HD * sizeof(float));
  const long long items = (long long)a.rows * a.kv.n_kv_heads * lay.groups * lay.max_runs;
  const int G = a.n_heads / a.kv.n_kv_heads;
  const cudaError_t rc = G <= 1   ? launch_gt<HD, 1>(tk, tv, a, items, num_sms, po, pml, s)
                         : G <= 2 ? launch_gt<HD, 2>(tk, tv, a, items, num_sms, po, pml, s)
                         : G <= 4 ? launch_gt<HD, 4>(tk, tv, a, items, num_sms, po, pml, s)
                                  : launch_gt<HD, 8>(tk, tv, a, items, num_sms, po, pml, s);
  if (rc != cudaSuccess || lay.max_runs == 1) return rc;
  return launch_pdl(k_paged_merge<HD, Attn>, dim3(a.n_heads, a.rows), dim3(128), 0, s, a, po, pml);
}

}  // namespace

size_t decode_fp8_workspace(const Attn& a) {
  const Layout lay = layout_of(a);
  if (lay.max_runs == 1) return 0;
  return (size_t)a.rows * a.n_heads * lay.max_runs * (a.kv.head_dim * sizeof(float) + sizeof(float2));
}

cudaError_t launch_decode_fp8(const Attn& a, int num_sms, cudaStream_t s) {
  CUtensorMap tk, tv;
  if (!fp8_maps(a.kv, &tk, &tv)) return cudaErrorInvalidValue;
  return a.kv.head_dim == 128 ? launch_hd<128>(tk, tv, a, num_sms, s) : launch_hd<64>(tk, tv, a, num_sms, s);
}
