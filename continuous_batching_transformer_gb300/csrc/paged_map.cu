// paged_map.cu -- block tables and slot maps from request lengths, on the device.
//
// One launch of one thread-block cluster.  Every CTA computes the same three prefix sums over the
// rows (new tokens, pages to take, pages to return) from the lengths, so no CTA waits for another
// to know where its share goes; the shares are then dealt over the cluster: returned pages are
// pushed, and, after one cluster barrier (which also orders the reads of the lengths and the count
// before they are overwritten), pages are popped into the table and every token finds its row by
// binary search in the prefix sums in shared memory.
//
// Bound by latency: some KB are read and 8 bytes a token written, all of it one dependent chain of
// loads, scans and the barrier: 3.0 us for 8 rows with a token each, 7.4 us for 256 rows, 24 prompts
// and 9 retiring rows among them, with 32768 tokens of room (7.0 us without the check of the returned
// ids across the cluster).  Eight CTAs once the tokens or rows would keep one CTA for several passes,
// one CTA (no cluster barrier) below that.
#include <cooperative_groups.h>

#include <limits.h>

#include "paged.h"

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 1024;
constexpr int kCluster = 8;

// Sums that stop at kFull instead of overflowing: the lengths are checked row by row, their sums are
// not yet
constexpr unsigned kFull = 0x7FFFFFFFu;
struct Sums {
  unsigned tok, take, back;
};
CBT_D unsigned add_full(unsigned a, unsigned b) { return min(a + b, kFull); }
CBT_D Sums operator+(Sums a, Sums b) {
  return {add_full(a.tok, b.tok), add_full(a.take, b.take), add_full(a.back, b.back)};
}
CBT_D Sums shfl_up(Sums v, int o) {
  return {__shfl_up_sync(0xffffffffu, v.tok, o), __shfl_up_sync(0xffffffffu, v.take, o),
          __shfl_up_sync(0xffffffffu, v.back, o)};
}
CBT_D Sums warp_scan(Sums v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums u = shfl_up(v, o);
    if (lane >= o) v = u + v;
  }
  return v;
}

// the row r < n whose range [pre[r], pre[r + 1]) holds i (0 <= i < pre[n])
CBT_D int find_row(const int* pre, int n, int i) {
  int lo = 0, hi = n;  // pre[lo] <= i < pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// n / d for 0 <= n < 2^31 as a multiplication: with 2^(s - 1) < d <= 2^s and m = ceil(2^(31 + s) / d),
// n m / 2^(31 + s) exceeds n / d by less than n / 2^31 / d, too little to reach the next whole number
struct Divide {
  unsigned m, s;
};
Divide divide_by(unsigned d) {
  unsigned s = 0;
  while ((1ull << s) < d) ++s;
  return {(unsigned)(((1ull << (31 + s)) + d - 1) / d), s};
}
CBT_D int quotient(int n, Divide d) { return d.s ? (int)(__umulhi(n, d.m) >> (d.s - 1)) : n; }

template <int C>
__global__ void __launch_bounds__(kThreads) k_page_map(const cbt_page_map_args a, const Divide page) {
  extern __shared__ int sm[];
  const int B = a.rows, P = a.page_tokens;
  // pages of n positions; the most a row may have, max_pages * P, is below 2^31
  auto pages = [&](int n) { return n > 0 ? quotient(n - 1, page) + 1 : 0; };
  int* cu = sm;              // [B + 1] new tokens
  int* take = sm + B + 1;    // [B + 1] pages to take
  int* back = take + B + 1;  // [B + 1] pages to return
  int* len = back + B + 1;   // [B] lengths before the call
  int* held = len + B;       // [B] and pages
  __shared__ Sums wtot[kThreads / 32];
  __shared__ int bad_row, bad_page;  // the first row with a bad length, and with a bad page to return
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = C > 1 ? (int)blockIdx.x : 0;
  const bool pool = a.free_pages != nullptr;
  if (tid == 0) bad_row = bad_page = INT_MAX;
  pdl_wait();
  pdl_launch();
  __syncthreads();

  // each thread takes a run of rows; the runs' sums are scanned over the block
  const int per = (B + kThreads - 1) / kThreads;
  const int r0 = min(B, tid * per), r1 = min(B, r0 + per);
  const long long most = (long long)a.max_pages * P;
  auto row_sums = [&](int n, int w) {
    const int h = pages(n);
    return Sums{w > 0 ? (unsigned)w : 0u, pool && w > 0 ? (unsigned)(pages(n + w) - h) : 0u,
                pool && w < 0 ? (unsigned)h : 0u};
  };
  Sums mine = {0, 0, 0};
  for (int r = r0; r < r1; ++r) {
    const int n = a.kv_lens[r], w = a.new_lens[r];
    if (n < 0 || n > most || (w > 0 && n + (long long)w > most)) {
      atomicMin(&bad_row, r);
      continue;
    }
    mine = mine + row_sums(n, w);
  }
  Sums inc = warp_scan(mine, lane);
  if (lane == 31) wtot[warp] = inc;
  __syncthreads();
  if (warp == 0) wtot[lane] = warp_scan(wtot[lane], lane);
  __syncthreads();
  const Sums tot = wtot[kThreads / 32 - 1];
  // the sums before this thread's rows (used only where none is full)
  Sums run = warp ? wtot[warp - 1] + inc : inc;
  run = {run.tok - mine.tok, run.take - mine.take, run.back - mine.back};
  const int count = pool ? *a.free_count : 0;
  int code = 0, info = 0;
  if (bad_row != INT_MAX) {
    code = CBT_DEV_LENGTH;
    info = bad_row;
  } else if (tot.tok > (unsigned)a.max_tokens || tot.tok == kFull) {
    code = CBT_DEV_TOKENS;
    info = a.max_tokens;
  } else if (pool && (count < 0 || count + (long long)tot.back > a.n_pages ||
                      (long long)tot.take > count + (long long)tot.back)) {
    code = CBT_DEV_PAGES;
    info = (int)min((long long)INT_MAX, max(0ll, (long long)tot.take - count - tot.back));
  }
  if (code == 0) {
    for (int r = r0; r < r1; ++r) {
      const int n = a.kv_lens[r], w = a.new_lens[r];
      cu[r] = (int)run.tok;
      take[r] = (int)run.take;
      back[r] = (int)run.back;
      len[r] = n;
      held[r] = pages(n);
      run = run + row_sums(n, w);
    }
    if (tid == 0) {
      cu[B] = (int)tot.tok;
      take[B] = (int)tot.take;
      back[B] = (int)tot.back;
    }
  }
  __syncthreads();
  const int t0 = rank * kThreads + tid;
  constexpr int kStep = C * kThreads;
  const bool returns = code == 0 && tot.back > 0;  // the same in the whole cluster
  if (returns) {  // push the retiring rows' pages, above the count: a bad one undoes them by leaving that
    for (int i = t0; i < (int)tot.back; i += kStep) {
      const int r = find_row(back, B, i);
      const int id = a.block_table[(size_t)r * a.max_pages + (i - back[r])];
      if (id < 0 || id >= a.n_pages) atomicMin(&bad_page, r);
      a.free_pages[count + i] = id;
    }
  }
  // every CTA has read the lengths and the count; pushed pages are visible to the whole cluster
  if (C > 1) cg::this_cluster().sync();
  else __syncthreads();
  if (returns) {
    if (warp == 0) {
      const int r = lane >= C ? INT_MAX : C > 1 ? *cg::this_cluster().map_shared_rank(&bad_page, lane) : bad_page;
      bad_row = __reduce_min_sync(0xffffffffu, r);
    }
    __syncthreads();
    if (bad_row != INT_MAX) {
      code = CBT_DEV_PAGE_ID;
      info = bad_row;
    }
    if (C > 1) cg::this_cluster().barrier_arrive();  // awaited before the CTA, and bad_page, go
  }
  auto leave = [&] {
    if (C > 1 && returns) cg::this_cluster().barrier_wait();
  };

  if (rank == 0) {  // the state afterwards
    for (int r = r0; r < r1; ++r) {
      const int w = code ? 0 : a.new_lens[r];
      const int n = code ? a.kv_lens[r] : len[r];
      a.kv_lens_out[r] = w < 0 ? 0 : n + w;
      a.cu_q[r] = code ? 0 : cu[r];
    }
    if (tid == 0) {
      a.cu_q[B] = code ? 0 : cu[B];
      if (pool) a.free_count_out[0] = code ? count : (int)(count + tot.back - tot.take);
      if (code) set_device_error(a.err, code, info);
    }
  }
  if (code) {
    for (int t = t0; t < a.max_tokens; t += kStep) a.positions[t] = a.slots[t] = -1;
    leave();
    return;
  }
  const int top = (int)(count + tot.back) - 1;
  if (pool) {
    for (int i = t0; i < (int)tot.take; i += kStep) {
      const int r = find_row(take, B, i);
      a.block_table[(size_t)r * a.max_pages + held[r] + (i - take[r])] = __ldcg(a.free_pages + top - i);
    }
  }
  // tokens, four of a thread's at a time: their searches and page loads overlap
  const int n_tok = cu[B];
  int step0 = 1;
  while (2 * step0 < B) step0 *= 2;
  constexpr int kAtOnce = 4;
  for (int tb = t0; tb < a.max_tokens; tb += kAtOnce * kStep) {
    int r[kAtOnce] = {}, pos[kAtOnce], off[kAtOnce], id[kAtOnce];
    for (int s = step0; s > 0; s >>= 1) {
#pragma unroll
      for (int e = 0; e < kAtOnce; ++e)
        if (r[e] + s < B && cu[r[e] + s] <= tb + e * kStep) r[e] += s;
    }
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e) {
      const int t = tb + e * kStep;
      pos[e] = id[e] = -1;
      off[e] = 0;
      if (t < n_tok) {
        const int n = len[r[e]];
        pos[e] = n + t - cu[r[e]];
        const int pg = quotient(pos[e], page), h = held[r[e]];
        off[e] = pos[e] - pg * P;
        // a page taken by this call is read from the stack, not from the table being written
        id[e] = __ldcg(pool && pg >= h ? a.free_pages + top - (take[r[e]] + pg - h)
                                       : a.block_table + (size_t)r[e] * a.max_pages + pg);
      }
    }
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e) {
      const int t = tb + e * kStep;
      if (t >= a.max_tokens) break;
      const bool good = id[e] >= 0 && id[e] < a.n_pages;
      if (t < n_tok && !good) set_device_error(a.err, CBT_DEV_PAGE_ID, r[e]);
      a.positions[t] = pos[e];
      a.slots[t] = good ? id[e] * P + off[e] : -1;
    }
  }
  leave();
}

template <int C>
cudaError_t launch(const cbt_page_map_args& a, cudaStream_t s) {
  const size_t smem = ((size_t)a.rows * 5 + 3) * sizeof(int);
  if (smem > 48 * 1024) {
    cudaError_t rc = cudaFuncSetAttribute(k_page_map<C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          (5 * CBT_PAGE_MAP_MAX_ROWS + 3) * (int)sizeof(int));
    if (rc != cudaSuccess) return rc;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 2 : 1;
  count_launch();
  return cudaLaunchKernelEx(&cfg, k_page_map<C>, a, divide_by(a.page_tokens));
}

}  // namespace

cudaError_t launch_page_map(const cbt_page_map_args& a, cudaStream_t s) {
  return a.max_tokens > 2 * kThreads || a.rows > kThreads ? launch<kCluster>(a, s) : launch<1>(a, s);
}
