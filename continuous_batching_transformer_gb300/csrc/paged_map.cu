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
// loads, scans and the barrier.  Eight CTAs once the tokens or pages would keep one CTA for several
// passes, one CTA (no cluster barrier) below that.
#include <cooperative_groups.h>

#include <limits.h>

#include "paged.h"

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 1024;
constexpr int kCluster = 8;

struct Sums {  // 64-bit: the lengths are checked row by row, their sums are not yet
  long long tok, take, back;
};
CBT_D Sums operator+(Sums a, Sums b) { return {a.tok + b.tok, a.take + b.take, a.back + b.back}; }
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

template <int C>
__global__ void __launch_bounds__(kThreads) k_page_map(const cbt_page_map_args a) {
  extern __shared__ int sm[];
  const int B = a.rows, P = a.page_tokens;
  int* cu = sm;              // [B + 1] new tokens
  int* take = sm + B + 1;    // [B + 1] pages to take
  int* back = take + B + 1;  // [B + 1] pages to return
  int* len = back + B + 1;   // [B] lengths before the call
  __shared__ Sums wtot[kThreads / 32];
  __shared__ int bad_row;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = C > 1 ? (int)blockIdx.x : 0;
  const bool pool = a.free_pages != nullptr;
  if (tid == 0) bad_row = INT_MAX;
  pdl_wait();
  pdl_launch();
  __syncthreads();

  // each thread takes a run of rows; the runs' sums are scanned over the block
  const int per = (B + kThreads - 1) / kThreads;
  const int r0 = min(B, tid * per), r1 = min(B, r0 + per);
  const long long most = (long long)a.max_pages * P;
  Sums mine = {0, 0, 0};
  for (int r = r0; r < r1; ++r) {
    const int n = a.kv_lens[r], w = a.new_lens[r];
    if (n < 0 || n > most || (w > 0 && n + (long long)w > most)) {
      atomicMin(&bad_row, r);
      continue;
    }
    const int held = (int)(((long long)n + P - 1) / P);
    mine.tok += w > 0 ? w : 0;
    mine.take += pool && w > 0 ? (int)(((long long)n + w + P - 1) / P) - held : 0;
    mine.back += pool && w < 0 ? held : 0;
  }
  Sums inc = warp_scan(mine, lane);
  if (lane == 31) wtot[warp] = inc;
  __syncthreads();
  if (warp == 0) wtot[lane] = warp_scan(wtot[lane], lane);
  __syncthreads();
  Sums run = warp ? wtot[warp - 1] + inc : inc;
  run = {run.tok - mine.tok, run.take - mine.take, run.back - mine.back};
  const Sums tot = wtot[kThreads / 32 - 1];
  const int count = pool ? *a.free_count : 0;
  int code = 0, info = 0;
  if (bad_row != INT_MAX) {
    code = CBT_DEV_LENGTH;
    info = bad_row;
  } else if (tot.tok > a.max_tokens) {
    code = CBT_DEV_TOKENS;
    info = a.max_tokens;
  } else if (pool && (count < 0 || count + tot.back > a.n_pages || tot.take > count + tot.back)) {
    code = CBT_DEV_PAGES;
    info = (int)min((long long)INT_MAX, max(0ll, tot.take - count - tot.back));
  }
  if (code == 0) {
    for (int r = r0; r < r1; ++r) {
      const int n = a.kv_lens[r], w = a.new_lens[r];
      const int held = (int)(((long long)n + P - 1) / P);
      cu[r] = (int)run.tok;
      take[r] = (int)run.take;
      back[r] = (int)run.back;
      len[r] = n;
      run.tok += w > 0 ? w : 0;
      run.take += pool && w > 0 ? (int)(((long long)n + w + P - 1) / P) - held : 0;
      run.back += pool && w < 0 ? held : 0;
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
  if (code == 0 && pool) {  // push the retiring rows' pages
    for (int i = t0; i < tot.back; i += kStep) {
      const int r = find_row(back, B, i);
      const int id = a.block_table[(size_t)r * a.max_pages + (i - back[r])];
      if (id < 0 || id >= a.n_pages) set_device_error(a.err, CBT_DEV_PAGE_ID, r);
      a.free_pages[count + i] = id;
    }
  }
  // every CTA has read the lengths and the count; pushed pages are visible to the whole cluster
  if (C > 1) cg::this_cluster().sync();
  else __syncthreads();

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
    return;
  }
  const int top = (int)(count + tot.back) - 1;
  if (pool) {
    for (int i = t0; i < tot.take; i += kStep) {
      const int r = find_row(take, B, i);
      const int held = (int)(((long long)len[r] + P - 1) / P);
      a.block_table[(size_t)r * a.max_pages + held + (i - take[r])] = __ldcg(a.free_pages + top - i);
    }
  }
  for (int t = t0; t < a.max_tokens; t += kStep) {
    int pos = -1, slot = -1;
    if (t < cu[B]) {
      const int r = find_row(cu, B, t);
      pos = len[r] + t - cu[r];
      const int pg = pos / P;
      const int held = (int)(((long long)len[r] + P - 1) / P);
      // a page taken by this call is read from the stack, not from the table being written
      const int id = pool && pg >= held ? __ldcg(a.free_pages + top - (take[r] + pg - held))
                                        : a.block_table[(size_t)r * a.max_pages + pg];
      if (id < 0 || id >= a.n_pages) set_device_error(a.err, CBT_DEV_PAGE_ID, r);
      else slot = id * P + (pos - pg * P);
    }
    a.positions[t] = pos;
    a.slots[t] = slot;
  }
}

template <int C>
cudaError_t launch(const cbt_page_map_args& a, cudaStream_t s) {
  const size_t smem = ((size_t)a.rows * 4 + 3) * sizeof(int);
  if (smem > 48 * 1024) {
    cudaError_t rc = cudaFuncSetAttribute(k_page_map<C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          (4 * CBT_PAGE_MAP_MAX_ROWS + 3) * (int)sizeof(int));
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
  return cudaLaunchKernelEx(&cfg, k_page_map<C>, a);
}

}  // namespace

cudaError_t launch_page_map(const cbt_page_map_args& a, cudaStream_t s) {
  return a.max_tokens > 2 * kThreads || a.rows > kThreads ? launch<kCluster>(a, s) : launch<1>(a, s);
}
