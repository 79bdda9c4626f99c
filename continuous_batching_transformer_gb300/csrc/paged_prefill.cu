// paged_prefill.cu -- attention of ragged runs of query tokens over a paged KV cache.
//
// A unit is a run of query tokens of one row and one kv head, as two tiles of 128 tensor-core rows.
// A tile's rows are (token, q head) pairs: the q heads that read the kv head lie next to each other,
// so a tile holds 128 / G tokens with all G of their heads, a decode row or a short chunk fills its
// tile with heads, and one K and V tile serves all of them.  Per 128-key block and tile:
//   S = Q K^T       tcgen05.mma 128 x 128 x head_dim into tensor memory
//   softmax         one thread per row: the whole row of S in registers, running maximum and sum
//   O += P V        tcgen05.mma 128 x head_dim x 128, P read from tensor memory as bf16 where S was
// O stays in tensor memory for the whole unit.  A row's reference maximum is raised (and its O
// rescaled) only when a block exceeds it by more than 2^kSlack, so O is rarely touched; the weights
// stay below 2^kSlack, exact in what they are divided by.  P is rounded to bf16 once (2^-9 of each
// weight on average less), everything else is fp32.
//
// Bound by the tensor cores and, close behind, the exponentials.  The two tiles of a unit run half
// a block out of step, each with an issuer thread and a softmax warpgroup of its own: one's MMAs
// run under the other's softmax.  K and V tiles come through two TMA maps over the whole pool (64
// keys a request, each from its own page) into rings of three and two stages.  A warp of its own
// clears V of keys that no query of the unit sees (what lies there may not be finite) before the
// MMA reads it.  One CTA per unit; units are found on the device from the rows' lengths, the rows'
// last units (the longest) first.
#include "paged_attn.cuh"

namespace {

constexpr int kBlk = 128;
constexpr int kBox = 16384;     // [128 rows][64 bf16], swizzled
constexpr int kKStages = 3, kVStages = 2;
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
CBT_D void tma_load_q(void* dst, const CUtensorMap* m, uint64_t* bar, int x, int head, int tok) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(tc::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(tc::smem_u32(bar)), "r"(x), "r"(head), "r"(tok)
      : "memory");
}

struct Unit {
  int b, t0, n;  // row; its query tokens [t0, t0 + n) of this unit, n = -1: no unit
  int p0;        // position of token t0 (may be negative)
};

// Blocks the tile with tokens at positions [p0, p1] needs
CBT_D bool needs(const Seen& s, int p1, int c) {
  return s.n > 0 && (c < s.ns || (c >= s.ws && c <= p1 / kBlk));
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
    k_paged_prefill(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                    const __grid_constant__ CUtensorMap tv, const __grid_constant__ PagedAttn a) {
  constexpr int nKh = HD / 64;
  constexpr uint32_t kTile = nKh * kBox;     // a Q, K or V tile
  constexpr int kVBox = HD * 128;            // V^T of 64 keys
  constexpr uint32_t kIdescS = tc::idesc_bf16(128, 128), kIdescO = tc::idesc_bf16(128, HD);
  constexpr uint32_t kTmem = 512;            // S0, S1 (P over them) in columns 0..255, O0, O1
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sQ = smem;                     // [tile][64-dim half][128 rows]
  uint8_t* sK = sQ + 2 * kTile;           // [stage][64-dim half][128 keys]
  uint8_t* sV = sK + kKStages * kTile;    // [stage][64-key half][HD dims]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sV + kVStages * kTile);
  uint64_t *qfull = bars, *kfull = bars + 1, *kempty = kfull + kKStages;
  uint64_t *vfull = kempty + kKStages, *vready = vfull + kVStages, *vempty = vready + kVStages;
  uint64_t *s_full = vempty + kVStages, *p_full = s_full + 2, *o_full = p_full + 2;
  constexpr int kBars = 1 + 2 * kKStages + 3 * kVStages + 6;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  Unit* unit = reinterpret_cast<Unit*>(tmem_slot + 2);
  int* wsum = reinterpret_cast<int*>(unit + 1);  // [12]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int H = a.n_heads, Hkv = a.kv.n_kv_heads, G = H / Hkv;
  const int TQ = kBlk / G;  // tokens per tile
  const int g = blockIdx.x % Hkv;
  if (tid == 0) {
    for (int i = 0; i < kBars; ++i) tc::mbar_init(&bars[i], 1);
    for (int i = 0; i < kKStages; ++i) tc::mbar_init(&kempty[i], 2);
    for (int i = 0; i < kVStages; ++i) tc::mbar_init(&vempty[i], 2);
    for (int i = 0; i < 2; ++i) tc::mbar_init(&p_full[i], 4);
    *abort_flag = 0;
    unit->n = -1;
    tc::mbar_fence_init();
    tc::tma_prefetch_desc(&tq);
    tc::tma_prefetch_desc(&tk);
    tc::tma_prefetch_desc(&tv);
  }
  pdl_wait();
  pdl_launch();
  // ---- this CTA's unit: units are counted over the rows, thread by thread
  {
    const int per = (a.rows + kThreads - 1) / kThreads;
    const int r0 = min(a.rows, tid * per), r1 = min(a.rows, r0 + per);
    int mine = 0;
    for (int r = r0; r < r1; ++r) {
      const RowTokens row = row_tokens(a, r);
      if (row.bad && blockIdx.x == 0) set_device_error(a.err, CBT_DEV_LENGTH, r);
      if (row.n > 0) mine += (row.n + 2 * TQ - 1) / (2 * TQ);
    }
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += wsum[w];
      total += wsum[w];
    }
    int at = before + inc - mine;
    const int u = total - 1 - (int)(blockIdx.x / Hkv);  // last units first
    if (u >= at && u < at + mine) {
      for (int r = r0; r < r1; ++r) {
        const RowTokens row = row_tokens(a, r);
        const int k = row.n > 0 ? (row.n + 2 * TQ - 1) / (2 * TQ) : 0;
        if (u < at + k) {
          const int first = (u - at) * 2 * TQ;
          *unit = Unit{r, row.t0 + first, min(2 * TQ, row.n - first), row.len - row.n + first};
          break;
        }
        at += k;
      }
    }
  }
  __syncthreads();
  const Unit un = *unit;
  if (un.n < 0) return;  // more CTAs than units (the whole block leaves)
  if (warp == 1) tc::tmem_alloc(tmem_slot, kTmem);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // positions of the unit's and of each tile's last token, and the blocks they need
  const int pl = un.p0 + un.n - 1;
  const Seen seen = seen_chunks(un.p0, pl, a.window, a.sinks);
  auto tile_first = [&](int x) { return un.p0 + x * TQ; };
  auto tile_last = [&](int x) { return min(pl, un.p0 + (x + 1) * TQ - 1); };
  auto tile_seen = [&](int x) {
    return tile_last(x) < tile_first(x) ? Seen{0, 0, 0}
                                        : seen_chunks(tile_first(x), tile_last(x), a.window, a.sinks);
  };
  const int lo_win = first_in_window(max(0, un.p0), a.window);

  if (warp == 0) {
    // ---- tile requests
    const uint64_t pol = tc::policy_evict_last();
    const int P = a.kv.page_tokens;
    uint32_t nk = 0, nv = 0;
    bool ok = true;
    if (lane == 0 && seen.n) {
      const int tiles = un.n > TQ ? 2 : 1;
      tc::mbar_expect_tx(qfull, tiles * nKh * G * TQ * 128);
      for (int x = 0; x < tiles; ++x)
#pragma unroll
        for (int h = 0; h < nKh; ++h)
          tma_load_q(sQ + x * kTile + h * kBox, &tq, qfull, h * 64, g * G, un.t0 + x * TQ);
    }
    // the tile rows of block i's halves: lanes 0 and 1 look the pages up
    struct Where {
      unsigned halves;
      int k0, k1, v0, v1;
    };
    auto where = [&](int i) {
      const int key = seen.chunk(i) * kBlk + 64 * lane;
      int krow = 0, vrow = 0;
      bool want = false;
      if (lane < 2) {
        const int last = min(key + 63, pl);
        want = key <= pl && (!a.window || last >= lo_win || key < a.sinks);
        if (want) {
          const int pg = key / P, o = key - pg * P;
          int id = a.table[(size_t)un.b * a.max_pages + pg];
          if (id < 0 || id >= a.kv.n_pages) {
            set_device_error(a.err, CBT_DEV_PAGE_ID, un.b);
            id = 0;  // a page that exists: the row's outputs are unspecified
          }
          krow = (int)(paged_k(a.kv, id, g, o, 0) / HD);
          vrow = (int)(paged_v(a.kv, id, g, o, 0) / 64);
        }
      }
      Where w;
      w.halves = __ballot_sync(0xffffffffu, want);
      w.k0 = krow;
      w.v0 = vrow;
      w.k1 = __shfl_sync(0xffffffffu, krow, 1);
      w.v1 = __shfl_sync(0xffffffffu, vrow, 1);
      return w;
    };
    auto load_k = [&](int i, const Where& w) {  // lane 0
      const int st = i % kKStages;
      if (!wait_or_abort(&kempty[st], ((i / kKStages) & 1) ^ 1, abort_flag)) return false;
      tc::mbar_expect_tx(&kfull[st], __popc(w.halves) * 64 * HD * 2);
      ++nk;
      uint8_t* dst = sK + st * kTile;
#pragma unroll
      for (int h = 0; h < nKh; ++h) {
        if (w.halves & 1) tc::tma_load_2d(dst + h * kBox, &tk, &kfull[st], h * 64, w.k0, pol);
        if (w.halves & 2) tc::tma_load_2d(dst + h * kBox + 8192, &tk, &kfull[st], h * 64, w.k1, pol);
      }
      return true;
    };
    auto load_v = [&](int i, const Where& w) {
      const int st = i % kVStages;
      if (!wait_or_abort(&vempty[st], ((i / kVStages) & 1) ^ 1, abort_flag)) return false;
      tc::mbar_expect_tx(&vfull[st], __popc(w.halves) * 64 * HD * 2);
      ++nv;
      uint8_t* dst = sV + st * kTile;
      if (w.halves & 1) tc::tma_load_2d(dst, &tv, &vfull[st], 0, w.v0, pol);
      if (w.halves & 2) tc::tma_load_2d(dst + kVBox, &tv, &vfull[st], 0, w.v1, pol);
      return true;
    };
    // K runs one block ahead of V
    Where cur{}, nxt{};
    if (seen.n) {
      cur = where(0);
      if (lane == 0) ok = load_k(0, cur);
    }
    for (int i = 0; i < seen.n && ok; ++i) {
      if (i + 1 < seen.n) {
        nxt = where(i + 1);
        if (lane == 0) ok = load_k(i + 1, nxt);
      }
      if (lane == 0 && ok) ok = load_v(i, cur);
      cur = nxt;
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    if (lane == 0) {
      if (!ok) wait_timeout(a.err, abort_flag, 11);
      // no copies in flight at exit
      if (seen.n) tc::mbar_wait(qfull, 0);
      for (uint32_t i = 0; i < (uint32_t)kKStages && i < nk; ++i)
        tc::mbar_wait(&kfull[(nk - 1 - i) % kKStages], ((nk - 1 - i) / kKStages) & 1);
      for (uint32_t i = 0; i < (uint32_t)kVStages && i < nv; ++i)
        tc::mbar_wait(&vfull[(nv - 1 - i) % kVStages], ((nv - 1 - i) / kVStages) & 1);
    }
  } else if (warp <= 2) {
    // ---- MMA issue of tile x
    if (lane == 0) {
      const int x = warp - 1;
      const Seen mine = tile_seen(x);
      const int last = tile_last(x);
      const uint32_t s_tm = tmem + x * 128, o_tm = tmem + 256 + x * HD;
      bool ok = seen.n == 0 || wait_or_abort(qfull, 0, abort_flag);
      uint32_t acc = 0, np = 0;
      for (int i = 0; i < seen.n && ok; ++i) {
        const int ks = i % kKStages, vs = i % kVStages;
        const bool need = needs(mine, last, seen.chunk(i));
        ok = wait_or_abort(&kfull[ks], (i / kKStages) & 1, abort_flag);
        if (!ok) break;
        if (!need) {  // this tile sees nothing of the block: pass its stages on
          tc::mbar_arrive(&kempty[ks]);
          ok = wait_or_abort(&vready[vs], (i / kVStages) & 1, abort_flag);
          if (ok) tc::mbar_arrive(&vempty[vs]);
          continue;
        }
        tc::tc_fence_after();
#pragma unroll
        for (int k = 0; k < HD / 16; ++k) {
          const uint64_t ad =
              tc::sdesc_sw128(tc::smem_u32(sQ + x * kTile + (k >> 2) * kBox)) + 2 * (k & 3);
          const uint64_t bd =
              tc::sdesc_sw128(tc::smem_u32(sK + ks * kTile + (k >> 2) * kBox)) + 2 * (k & 3);
          tc::mma_bf16(s_tm, ad, bd, kIdescS, k > 0 ? 1u : 0u);
        }
        tc::mma_commit(&s_full[x]);
        tc::mma_commit(&kempty[ks]);
        ok = wait_or_abort(&p_full[x], np & 1, abort_flag) &&
             wait_or_abort(&vready[vs], (i / kVStages) & 1, abort_flag);
        if (!ok) break;
        ++np;
        tc::tc_fence_after();
#pragma unroll
        for (int k = 0; k < kBlk / 16; ++k) {
          const uint64_t bd =
              tc::sdesc_sw128(tc::smem_u32(sV + vs * kTile + (k >> 2) * kVBox)) + 2 * (k & 3);
          tc::mma_bf16_ta(o_tm, s_tm + 8 * k, bd, kIdescO, (acc || k > 0) ? 1u : 0u);
        }
        acc = 1;
        tc::mma_commit(&vempty[vs]);
      }
      if (ok) tc::mma_commit(&o_full[x]);
      else wait_timeout(a.err, abort_flag, 12);
    }
  } else if (warp == 3) {
    // ---- V of keys that no query of the unit sees is cleared
    bool ok = true;
    for (int i = 0; i < seen.n && ok; ++i) {
      const int st = i % kVStages;
      ok = wait_or_abort(&vfull[st], (i / kVStages) & 1, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      uint32_t bits[4];
      seen_bits(seen.chunk(i) * kBlk, pl, lo_win, a.window ? a.sinks : 0, bits);
      if ((bits[0] & bits[1] & bits[2] & bits[3]) != 0xFFFFFFFFu) {
        uint8_t* v = sV + st * kTile;
#pragma unroll 1
        for (int u = 0; u < 16; ++u) {  // 8 keys
          const uint32_t m8 = ((u < 4 ? bits[0] : u < 8 ? bits[1] : u < 12 ? bits[2] : bits[3]) >>
                               (8 * (u & 3))) & 0xFFu;
          if (m8 == 0xFFu) continue;
          const uint4 mk = key_mask(m8);
          for (int d = lane; d < HD; d += 32) {
            uint4* p = reinterpret_cast<uint4*>(v + (u >> 3) * kVBox + d * 128 + (((u & 7) ^ (d & 7)) << 4));
            uint4 z = make_uint4(0, 0, 0, 0);
            if (m8) z = *p;
            *p = make_uint4(z.x & mk.x, z.y & mk.y, z.z & mk.z, z.w & mk.w);
          }
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
      }
      if (lane == 0) tc::mbar_arrive(&vready[st]);
    }
    if (!ok && lane == 0) wait_timeout(a.err, abort_flag, 13);
  } else {
    // ---- softmax of tile x: thread = row
    const int x = (warp - 4) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const Seen mine = tile_seen(x);
    const int last = tile_last(x);
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_tm = tmem + x * 128 + lane_off, o_tm = tmem + 256 + x * HD + lane_off;
    const int tok = x * TQ + row / G;          // token of the unit
    const bool live = row < TQ * G && tok < un.n;
    const int p = live ? un.p0 + tok : -1;     // -1: sees nothing
    // rows that hold no token are left unmasked: what they compute is not stored
    const int hi = live ? p : 0x3FFFFFFF, lo = live ? first_in_window(max(0, p), a.window) : 0;
    const int sinks = a.window ? a.sinks : 0;
    const float scale2 = a.scale * kLog2e;
    float m = -INFINITY, l = 0.f;
    uint32_t ns = 0;
    bool ok = true;
    for (int i = 0; i < seen.n && ok; ++i) {
      const int c = seen.chunk(i);
      if (!needs(mine, last, c)) continue;
      ok = wait_or_abort(&s_full[x], ns & 1, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc::tc_fence_after();
      uint32_t s[128];
#pragma unroll
      for (int k = 0; k < 4; ++k) tmem_ld32(s_tm + 32 * k, s + 32 * k);
      tc::tmem_ld_wait();
      const int k0 = c * kBlk;
      uint32_t bits[4];
      seen_bits(k0, hi, lo, sinks, bits);
      const bool whole = __all_sync(0xffffffffu, (bits[0] & bits[1] & bits[2] & bits[3]) == 0xFFFFFFFFu);
      float mx = -INFINITY;
      if (whole) {
#pragma unroll
        for (int k = 0; k < 128; ++k) {
          const float v = __uint_as_float(s[k]) * scale2;
          s[k] = __float_as_uint(v);
          mx = fmaxf(mx, v);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 128; ++k) {
          const float v = (bits[k >> 5] >> (k & 31)) & 1 ? __uint_as_float(s[k]) * scale2 : -INFINITY;
          s[k] = __float_as_uint(v);
          mx = fmaxf(mx, v);
        }
      }
      if (ns == 0) {
        m = mx;
      } else {
        const bool up = mx > m + kSlack;  // m = -inf: the row's first visible keys
        if (__any_sync(0xffffffffu, up)) {
          // the MMAs into O have completed: S of this block was issued after them
          const float f = up ? ex2(m - mx) : 1.f;
          if (up) m = mx;
          l *= f;
#pragma unroll 1
          for (int k = 0; k < HD; k += 16) {
            uint32_t o[16];
            tc::tmem_ld16(o_tm + k, o);
            tc::tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st16(o_tm + k, o);
          }
        }
      }
      const float ref = m == -INFINITY ? 0.f : m;
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < 128; k += 32) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float p0 = ex2(__uint_as_float(s[k + 2 * e]) - ref);
          const float p1 = ex2(__uint_as_float(s[k + 2 * e + 1]) - ref);
          sum += p0 + p1;
          pk[e] = pack_bf16(p0, p1);
        }
        tmem_st16(s_tm + k / 2, pk);
      }
      l += sum;
      tc::tmem_st_wait();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&p_full[x]);
      ++ns;
    }
    if (ok && ns) {
      ok = wait_or_abort(&o_full[x], 0, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      tc::tc_fence_after();
    }
    if (!ok && lane == 0) wait_timeout(a.err, abort_flag, 14);
    if (ok) {
      const float inv = p >= 0 ? 1.f / l : 0.f;
      const long long at = (long long)(un.t0 + tok) * a.out_ld + (long long)(g * G + row % G) * HD;
#pragma unroll 1
      for (int k = 0; k < HD; k += 16) {
        uint32_t o[16];
        if (ns) {
          tc::tmem_ld16(o_tm + k, o);
          tc::tmem_ld_wait();
        }
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = p >= 0 ? __uint_as_float(o[e]) * inv : 0.f;
        if (!live) continue;
        if (a.f32) {
          float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.out) + at + k);
#pragma unroll
          for (int e = 0; e < 4; ++e) dst[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at + k);
#pragma unroll
          for (int e = 0; e < 2; ++e)
            dst[e] = make_uint4(pack_bf16(v[8 * e], v[8 * e + 1]), pack_bf16(v[8 * e + 2], v[8 * e + 3]),
                                pack_bf16(v[8 * e + 4], v[8 * e + 5]), pack_bf16(v[8 * e + 6], v[8 * e + 7]));
        }
      }
    }
    tc::tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, kTmem);
  }
}

template <int HD>
cudaError_t launch_hd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                      const PagedAttn& a, cudaStream_t s) {
  constexpr size_t smem = 1024 + (2 + kKStages + kVStages) * (HD / 64) * kBox + 512;
  static_assert(smem <= 227 * 1024, "shared memory budget");
  const cudaError_t rc = cudaFuncSetAttribute(k_paged_prefill<HD>,
                                              cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (rc != cudaSuccess) return rc;
  const int G = a.n_heads / a.kv.n_kv_heads, run = 2 * (kBlk / G);
  // most units: every row may end in a partly filled one
  const long long by_tokens = (long long)a.tokens / run + a.rows;
  const long long by_rows = (long long)a.rows * ((a.max_q + run - 1) / run);
  const long long units = by_tokens < by_rows ? by_tokens : by_rows;
  return launch_pdl(k_paged_prefill<HD>, dim3((unsigned)(units * a.kv.n_kv_heads)), dim3(kThreads), smem, s,
                    tq, tk, tv, a);
}

}  // namespace

cudaError_t launch_paged_prefill(const PagedAttn& a, cudaStream_t s) {
  CUtensorMap tq, tk, tv;
  const int G = a.n_heads / a.kv.n_kv_heads;
  if (!paged_maps(a.kv, &tk, &tv) ||
      !make_tmap_rows(&tq, a.q, a.kv.head_dim, a.n_heads, a.tokens, a.q_ld, G, kBlk / G))
    return cudaErrorInvalidValue;
  return a.kv.head_dim == 128 ? launch_hd<128>(tq, tk, tv, a, s) : launch_hd<64>(tq, tk, tv, a, s);
}
