// paged_decode.cu -- attention of one new token per row over a paged KV cache, split over the
// cache's length and joined.
//
// The contraction is turned around so that the long axis fills the tensor core's rows, as in the
// engine's decode attention (attn_tc.cu): per 128-key chunk, S^T[key][head] = K . Q^T and
// O^T[dim][head] = V^T . P^T, tcgen05.mma with M = 128 and N = 16 (the up to 8 q heads that read
// one kv head, so K and V are read once for all of them; rows 8..15 hold the remainders of the
// weights' rounding to bf16, so the weights carry 16 bits and only q, K and V are as rough as
// their type).  One thread owns a key in the softmax and a dim in the output.
//
// Bound by HBM: 4 head_dim bytes of K and V per position and kv head.  Three CTAs share an SM, each
// with one K and one V tile buffer of its own (192 KB in flight an SM), and their latency chains
// overlap; a warp of its own requests tiles through two TMA maps over the whole pool, 64 keys a
// request, so a chunk may lie in two pages and a page may end inside it.
//
// Work is dealt on the device from the rows' lengths, so a captured launch stays valid while they
// grow: a persistent grid walks items (row, kv head, group of 8 q heads, run of chunks), each warp
// finding its item's row from prefix sums over 32 rows at a time kept in registers.  A run's length
// depends on the row alone, and so does the order in which k_paged_merge adds the runs' (max, sum,
// output).  Rows of one run are finished here.
//
// Measured on one GB300 (graph replays): 32 rows of 8192 to 16384 positions, 32 / 8 heads of 128, 244
// to 252 us = 6.5 to 6.7 TB/s, 95 to 99 % of the measured copy rate; 16 of them through a window of
// 4096 47.4 us (5.7 TB/s); 8 rows of 512 to 4096 15.6 us, where 2.5 chunks a CTA
// do not divide evenly and the join takes 3 us.
#include "paged_split.cuh"

namespace {

constexpr int kBox = 16384;    // [128 rows][64 bf16], swizzled
constexpr int kCompute = 128;  // warps 0..3; warp 4 requests tiles
constexpr int kCtasPerSm = 3;
constexpr int kIssuers = 2;    // threads that issue half of each contraction's MMAs
constexpr uint32_t kTmemCols = 64;

// GT: the group's q heads rounded up to 1, 2, 4 or 8
template <int HD, int GT>
__global__ void __launch_bounds__(kCompute + 32, kCtasPerSm)
    k_paged_decode(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                   const __grid_constant__ PagedAttn a, float* __restrict__ part_o,
                   float2* __restrict__ part_ml) {
  constexpr int nKh = HD / 64;
  constexpr uint32_t kIdesc = tc::idesc_bf16(128, 16);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sK = smem;                  // [64-dim half][128 keys]
  // [64-key half][HD dims]: the MMA's M is 128, so a half spans 128 rows for HD = 64 too (the
  // rows past HD hold anything; their outputs are not read)
  uint8_t* sV = sK + nKh * kBox;
  uint8_t* sQ = sV + 2 * kBox;         // [64-dim half][16 heads]
  uint8_t* sP = sQ + nKh * 2048;       // [64-key half][16 heads: 8 weights, 8 remainders]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sP + 2 * 2048);
  uint64_t *kfull = bars, *vfull = bars + 1, *kempty = bars + 2, *vempty = bars + 3;
  uint64_t *bar_s = bars + 4, *bar_o = bars + 5;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 6);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* vis = tmem_slot + 2;                        // [4] visible keys of the chunk
  float* red = reinterpret_cast<float*>(tmem_slot + 6); // [4 warps][8 heads]
  float* red2 = red + 32;
  float* l_run = red2 + 32;                             // [8]

  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const Layout lay = layout_of(a);
  const int per_row = a.kv.n_kv_heads * lay.groups;
  if (tid == 0) {
    for (int i = 0; i < 6; ++i) tc::mbar_init(&bars[i], i < 2 ? 1 : kIssuers);
    *abort_flag = 0;
    tc::mbar_fence_init();
    tc::tma_prefetch_desc(&tk);
    tc::tma_prefetch_desc(&tv);
  }
  if (warp == 0) tc::tmem_alloc(tmem_slot, kTmemCols);
  // heads that no item fills stay zero
  for (int i = tid; i < (nKh + 2) * 2048 / 16; i += kCompute + 32)
    reinterpret_cast<uint4*>(sQ)[i] = make_uint4(0, 0, 0, 0);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);
  pdl_wait();
  Cursor<PagedAttn> cur;
  cur.load(a, per_row, 0, 0);

  if (warp == 4) {
    // ---- tile requests: K, then V of each chunk.  The next chunk's pages are looked up while V's
    // buffer is awaited, so that K's stays empty for a wait only.
    const uint64_t pol = tc::policy_evict_first();
    uint32_t n = 0, nk = 0, nv = 0;  // chunks, and tiles of K and of V requested
    bool ok = true;
    const int P = a.kv.page_tokens;
    // a chunk's halves of 64 keys that hold a key the query sees, and their rows in the two maps
    struct Chunk {
      unsigned halves;
      int k[2], v[2];
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
      // lanes 0 and 1: a half each
      const int k0 = w.seen.chunk(i++) * kSub + 64 * lane;
      int krow = 0, vrow = 0;
      const bool want = lane < 2 && k0 <= w.p && (sees(k0, w.p, a.window, a.sinks) ||
                                                   sees(min(k0 + 63, w.p), w.p, a.window, a.sinks));
      if (want) {
        const int pg = k0 / P, o = k0 - pg * P;
        int id = a.table[(size_t)w.b * a.max_pages + pg];
        if (id < 0 || id >= a.kv.n_pages) {
          set_device_error(a.err, CBT_DEV_PAGE_ID, w.b);
          id = 0;  // a page that exists: the row's outputs are unspecified
        }
        krow = (int)(paged_k(a.kv, id, w.g, o, 0) / HD);
        vrow = (int)(paged_v(a.kv, id, w.g, o, 0) / 64);
      }
      c.halves = __ballot_sync(0xffffffffu, want);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        c.k[e] = __shfl_sync(0xffffffffu, krow, e);
        c.v[e] = __shfl_sync(0xffffffffu, vrow, e);
      }
      return c;
    };
    Chunk c = next();
#pragma unroll 1
    for (; c.halves; ++n) {
      const uint32_t bytes = __popc(c.halves) * 64 * HD * 2;
      ok = __all_sync(0xffffffffu, wait_or_abort(kempty, (n & 1) ^ 1, abort_flag));
      if (!ok) break;
      if (elect_one()) {
        tc::mbar_expect_tx(kfull, bytes);
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int h = 0; h < nKh; ++h)
            if (c.halves >> e & 1)
              tc::tma_load_2d(sK + h * kBox + e * (kBox / 2), &tk, kfull, h * 64, c.k[e], pol);
      }
      ++nk;
      const Chunk nxt = next();
      ok = __all_sync(0xffffffffu, wait_or_abort(vempty, (n & 1) ^ 1, abort_flag));
      if (!ok) break;
      if (elect_one()) {
        tc::mbar_expect_tx(vfull, bytes);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (c.halves >> e & 1) tc::tma_load_2d(sV + e * kBox, &tv, vfull, 0, c.v[e], pol);
      }
      ++nv;
      c = nxt;
    }
    if (!ok && lane == 0) wait_timeout(a.err, abort_flag, 1);
    // no copies in flight at exit
    if (nk) wait_landed(kfull, (nk - 1) & 1);
    if (nv) wait_landed(vfull, (nv - 1) & 1);
  } else {
    uint32_t n = 0;  // chunks done
    bool ok = true;
    const float scale2 = a.scale * kLog2e;  // scores in units of log2
    constexpr int kQUnits = HD / 8;         // 16-byte pieces of a head
    const int qh = tid / kQUnits, qu = tid % kQUnits;
    // this thread's piece of the next item's q
    auto load_q = [&](const Item& w) {
      return qh < w.heads
                 ? *reinterpret_cast<const uint4*>(a.q + w.t * a.q_ld + (long long)(w.head0 + qh) * HD + qu * 8)
                 : make_uint4(0, 0, 0, 0);
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
      if (qh < kGroup) *reinterpret_cast<uint4*>(sQ + sw128_offset(qh, qu * 8, 2048)) = qv;
      it += gridDim.x;
      have = cur.seek(a, per_row, it);
      if (have) {
        nxt = item_at(cur, a, lay.groups, it);
        qv = load_q(nxt);
      }
      if (tid < 8) l_run[tid] = 0.f;
      float m_run[GT], oacc[GT];
#pragma unroll
      for (int h = 0; h < GT; ++h) {
        m_run[h] = -INFINITY;  // kept by every thread, each from the same values in the same order
        oacc[h] = 0.f;
      }
      tc::fence_proxy_async_smem();
      tc::named_bar_sync(1, kCompute);

      for (int i = w.i0; i < w.i1; ++i, ++n) {
        if (warp < kIssuers) {
          const int iss = warp;
          if (!__all_sync(0xffffffffu, wait_or_abort(kfull, n & 1, abort_flag))) {
            if (lane == 0) wait_timeout(a.err, abort_flag, 2);
          } else if (elect_one()) {
            tc::tc_fence_after();
            constexpr int kSteps = HD / 16 / kIssuers;
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
              const int kk = iss * kSteps + k;
              const uint64_t ad = tc::sdesc_sw128(tc::smem_u32(sK + (kk >> 2) * kBox)) + 2 * (kk & 3);
              const uint64_t bd = tc::sdesc_sw128(tc::smem_u32(sQ + (kk >> 2) * 2048)) + 2 * (kk & 3);
              tc::mma_bf16(tmem + 32 * iss, ad, bd, kIdesc, k > 0 ? 1u : 0u);
            }
            tc::mma_commit(bar_s);
            tc::mma_commit(kempty);
          }
        }
        const int k0 = w.seen.chunk(i) * kSub;
        const bool valid = sees(k0 + tid, w.p, a.window, a.sinks);
        const uint32_t vb = __ballot_sync(0xffffffffu, valid);
        if (lane == 0) vis[warp] = vb;
        const bool bad_s = !wait_or_abort(bar_s, n & 1, abort_flag);
        if (tc::named_bar_any(2, kCompute, bad_s)) {
          ok = false;
          break;
        }
        tc::tc_fence_after();
        uint32_t raw[8], raw2[8];
        const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
        tc::tmem_ld8(lane_base, raw);
        tc::tmem_ld8(lane_base + 32, raw2);
        tc::tmem_ld_wait();
        float s[GT], mx[GT];
#pragma unroll
        for (int h = 0; h < GT; ++h) {
          s[h] = valid ? (__uint_as_float(raw[h]) + __uint_as_float(raw2[h])) * scale2 : -INFINITY;
          mx[h] = s[h];
        }
        warp_reduce_n<GT, true>(mx);
        if (lane == 0) {
#pragma unroll
          for (int h = 0; h < GT; ++h) red[warp * 8 + h] = mx[h];
        }
        tc::named_bar_sync(1, kCompute);
        float scl[GT];
#pragma unroll
        for (int h = 0; h < GT; ++h) {
          const float mloc = fmaxf(fmaxf(red[h], red[8 + h]), fmaxf(red[16 + h], red[24 + h]));
          const float mo = m_run[h];
          const float mn = fmaxf(mo, mloc);
          scl[h] = mo == -INFINITY ? 0.f : ex2(mo - mn);
          m_run[h] = mn;
        }
        float ps[GT];
#pragma unroll
        for (int h = 0; h < GT; ++h) {
          // (scores of -inf alone so far: weights of 0, not of exp(-inf + inf))
          const float p = valid ? ex2(s[h] - (m_run[h] == -INFINITY ? 0.f : m_run[h])) : 0.f;
          const uint16_t hi = round_bf16(p);
          *reinterpret_cast<uint16_t*>(sP + sw128_offset(h, tid, 2048)) = hi;
          *reinterpret_cast<uint16_t*>(sP + sw128_offset(8 + h, tid, 2048)) =
              round_bf16(p - bf16_to_f32(hi));
          ps[h] = p;
        }
        warp_reduce_n<GT, false>(ps);
        if (lane == 0) {
#pragma unroll
          for (int h = 0; h < GT; ++h) red2[warp * 8 + h] = ps[h];
        }
        if (vis[0] + 1 != 0 || vis[1] + 1 != 0 || vis[2] + 1 != 0 || vis[3] + 1 != 0) {
          // masked keys: their V may hold anything, so it is zeroed (their weights are zero)
          const bool bad_v = !wait_or_abort(vfull, n & 1, abort_flag);
          if (tc::named_bar_any(2, kCompute, bad_v)) {
            if (tid == 0) wait_timeout(a.err, abort_flag, 3);
            ok = false;
            break;
          }
          if (tid < HD) {
#pragma unroll 1
            for (int u = 0; u < 16; ++u) {  // 8 keys of this thread's dim
              const uint32_t bits = (vis[u >> 2] >> (8 * (u & 3))) & 0xFFu;
              if (bits == 0xFFu) continue;
              uint4* at = reinterpret_cast<uint4*>(sV + (u >> 3) * kBox + tid * 128 +
                                                   (((u & 7) ^ (tid & 7)) << 4));
              const uint4 mk = key_mask(bits);
              uint4 v = make_uint4(0, 0, 0, 0);
              if (bits) v = *at;
              *at = make_uint4(v.x & mk.x, v.y & mk.y, v.z & mk.z, v.w & mk.w);
            }
          }
        }
        tc::fence_proxy_async_smem();
        tc::tc_fence_before();
        tc::named_bar_sync(1, kCompute);
        if (tid < GT) {
          float sc = scl[0];
#pragma unroll
          for (int h = 1; h < GT; ++h)
            if (h == tid) sc = scl[h];
          l_run[tid] = l_run[tid] * sc + red2[tid] + red2[8 + tid] + red2[16 + tid] + red2[24 + tid];
        }
        if (warp < kIssuers) {
          const int iss = warp;
          if (!__all_sync(0xffffffffu, wait_or_abort(vfull, n & 1, abort_flag))) {
            if (lane == 0) wait_timeout(a.err, abort_flag, 4);
          } else if (elect_one()) {
            tc::tc_fence_after();
            constexpr int kSteps = kSub / 16 / kIssuers;
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
              const int kk = iss * kSteps + k;
              const uint64_t ad = tc::sdesc_sw128(tc::smem_u32(sV + (kk >> 2) * kBox)) + 2 * (kk & 3);
              const uint64_t bd = tc::sdesc_sw128(tc::smem_u32(sP + (kk >> 2) * 2048)) + 2 * (kk & 3);
              tc::mma_bf16(tmem + 32 * iss + 16, ad, bd, kIdesc, k > 0 ? 1u : 0u);
            }
            tc::mma_commit(bar_o);
            tc::mma_commit(vempty);
          }
        }
        const bool bad_o = !wait_or_abort(bar_o, n & 1, abort_flag);
        if (tc::named_bar_any(2, kCompute, bad_o)) {
          ok = false;
          break;
        }
        tc::tc_fence_after();
        uint32_t o1[16], o2[16];
        tc::tmem_ld16(lane_base + 16, o1);
        tc::tmem_ld16(lane_base + 48, o2);
        tc::tmem_ld_wait();
#pragma unroll
        for (int h = 0; h < GT; ++h)
          oacc[h] = oacc[h] * scl[h] + ((__uint_as_float(o1[h]) + __uint_as_float(o1[8 + h])) +
                                        (__uint_as_float(o2[h]) + __uint_as_float(o2[8 + h])));
        tc::tc_fence_before();
      }
      if (!ok) break;
      tc::named_bar_sync(1, kCompute);  // l_run is complete
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
  // Only now: the join's blocks, resident early, slowed the streaming down by a fifth (301 us for 250)
  pdl_launch();
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

template <int HD, int GT>
cudaError_t launch_gt(const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttn& a, int grid,
                      float* po, float2* pml, cudaStream_t s) {
  constexpr int nKh = HD / 64;
  constexpr size_t smem = 1024 + (nKh + 2) * kBox + (nKh + 2) * 2048 + 512;
  static_assert(smem * kCtasPerSm <= 228 * 1024 - kCtasPerSm * 1024, "shared memory budget");
  const cudaError_t rc = cudaFuncSetAttribute(k_paged_decode<HD, GT>,
                                              cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (rc != cudaSuccess) return rc;
  return launch_pdl(k_paged_decode<HD, GT>, dim3(grid), dim3(kCompute + 32), smem, s, tk, tv, a, po, pml);
}

template <int HD>
cudaError_t launch_hd(const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttn& a, int num_sms,
                      cudaStream_t s) {
  const Layout lay = layout_of(a);
  if (lay.max_runs > 1 && !a.ws) return cudaErrorInvalidValue;
  const size_t n = (size_t)a.rows * a.n_heads * lay.max_runs;
  float* po = reinterpret_cast<float*>(a.ws);
  float2* pml = reinterpret_cast<float2*>(a.ws + n * HD * sizeof(float));
  const long long items = (long long)a.rows * a.kv.n_kv_heads * lay.groups * lay.max_runs;
  const int grid = (int)(items < (long long)kCtasPerSm * num_sms ? items : kCtasPerSm * num_sms);
  const int G = a.n_heads / a.kv.n_kv_heads;
  const cudaError_t rc = G <= 1   ? launch_gt<HD, 1>(tk, tv, a, grid, po, pml, s)
                         : G <= 2 ? launch_gt<HD, 2>(tk, tv, a, grid, po, pml, s)
                         : G <= 4 ? launch_gt<HD, 4>(tk, tv, a, grid, po, pml, s)
                                  : launch_gt<HD, 8>(tk, tv, a, grid, po, pml, s);
  if (rc != cudaSuccess || lay.max_runs == 1) return rc;
  return launch_pdl(k_paged_merge<HD, PagedAttn>, dim3(a.n_heads, a.rows), dim3(128), 0, s, a, po, pml);
}

}  // namespace

bool paged_maps(const PagedKv& kv, CUtensorMap* tk, CUtensorMap* tv) {
  return make_tmap_bf16(tk, kv.pool, kv.head_dim, kv.pool_elems / kv.head_dim, 64, 64) &&
         make_tmap_bf16(tv, kv.pool, 64, kv.pool_elems / 64, 64, kv.head_dim);
}

size_t paged_decode_workspace(const PagedAttn& a) {
  const Layout lay = layout_of(a);
  if (lay.max_runs == 1) return 0;
  return (size_t)a.rows * a.n_heads * lay.max_runs * (a.kv.head_dim * sizeof(float) + sizeof(float2));
}

cudaError_t launch_paged_decode(const PagedAttn& a, int num_sms, cudaStream_t s) {
  CUtensorMap tk, tv;
  if (!paged_maps(a.kv, &tk, &tv)) return cudaErrorInvalidValue;
  return a.kv.head_dim == 128 ? launch_hd<128>(tk, tv, a, num_sms, s)
                              : launch_hd<64>(tk, tv, a, num_sms, s);
}
