// paged_split.cuh -- attention of one token per row, split over the cache's length: which runs of
// 128-key chunks a row makes, the walk over them on the device, and the join of their partial outputs.
// Shared by the kernels over bf16 and over 8-bit pages.
#pragma once
#include "paged_attn.cuh"

namespace {

constexpr int kSub = 128;      // keys of a chunk
constexpr int kGroup = 8;      // q heads per item

// Chunks of a run, by the chunks n that the row sees alone (so that its result does not depend on the
// other rows).  Longer runs halve the partial outputs and their join; shorter ones spread a few rows
// over the SMs.  Over bf16 pages, in us: 32 rows of 64 to 128 chunks 244 by fours, 251 by twos; one row of 64
// chunks 11.3 by fours, 10.4 by twos; 16 rows of 33 chunks 47.0 by twos, 48.3 singly; one row of two chunks
// 6.4 in one run, which needs no join, against 7.4.
// Over 8-bit pages a chunk takes half the time and its partial output as long.  Rows alike, 32 q and 8 kv heads of
// 128, all in one run / singly / by twos / by fours:
//   chunks   1 row                   8 rows                  32 rows                 128 rows
//   4        8.9   6.6  7.6  8.7     9.1   7.6  8.0  8.9     10.3  14.4 11.5 10.0    24.4  37.1  32.6  24.3
//   8        13.2  6.7  7.6  9.9     13.4  9.2  8.7  10.3    15.7  19.7 16.3 14.8    43.9  62.5  54.5  50.6
//   16       22.2  7.4  7.7  9.9     22.3  13.1 11.0 11.2    26.7  33.3 28.1 26.9    81.8  114   96.9  90.5
//   32       40.0  8.7  8.4  10.1    40.9  20.0 16.1 14.2    49.2  58.8 50.6 47.8    157   216   184   171
//   64       75.9  10.9 10.0 10.7    80.2  34.1 29.8 27.2    93.8  106  93.7 87.6
// No rule on the row alone has the best of every column.  One run of up to four, twos from 5 and fours from 33 on
// are within 5 % of the best of the four ways in half of 120 such shapes and within 20 % in nine tenths; the
// furthest behind are a row of four chunks (8.9 for 6.6 singly) and 64 rows of five (22.6 for 14.6 in one run).
template <class A>
CBT_HD int chunks_per_run(int n) {
  constexpr RunRule r = decltype(A::kv)::kRuns;
  return n >= r.four ? 4 : n >= r.two ? 2 : n > r.one ? 1 : n > 0 ? n : 1;
}
template <class A>
CBT_HD int runs_of(int n) {  // a row that sees nothing has one run, which writes its zeros
  const int per = chunks_per_run<A>(n);
  return n <= 0 ? 1 : (n + per - 1) / per;
}
template <class A>
CBT_HD int most_runs(int n) {  // of any row that sees n chunks or fewer
  constexpr RunRule rule = decltype(A::kv)::kRuns;
  int r = runs_of<A>(n);
  for (const int below : {rule.two, rule.four})
    if (n >= below && runs_of<A>(below - 1) > r) r = runs_of<A>(below - 1);
  return r;
}

struct Layout {
  int groups;    // groups of kGroup q heads per kv head
  int max_runs;  // most runs of a row
};
template <class A>
__host__ __device__ inline Layout layout_of(const A& a) {
  const int G = a.n_heads / a.kv.n_kv_heads;
  int n = (int)(((long long)a.max_kv + kSub - 1) / kSub);
  if (a.window && a.window < a.max_kv) {
    // sink chunks, and a window that may start anywhere in a chunk
    const long long w = ((long long)a.sinks + kSub - 1) / kSub + (a.window + kSub - 2) / kSub + 1;
    n = w < n ? (int)w : n;
  }
  return {(G + kGroup - 1) / kGroup, most_runs<A>(n)};
}

// The rows' items in flat order, walked forward by a whole warp: lane i keeps row w0 + i and the
// items before it.
template <class A>
struct Cursor {
  int w0;         // first row of the window
  int lane;
  int begin, end; // items [begin, end) of this lane's row
  int total;      // items up to the window's last row
  RowTokens row;
  Seen seen;

  CBT_D void load(const A& a, int per_row, int first, int before) {
    w0 = first;
    lane = threadIdx.x & 31;
    const int b = w0 + lane;
    int n = 0;
    if (b < a.rows) {
      row = row_tokens(a, b);
      if (row.bad && blockIdx.x == 0) set_device_error(a.err, CBT_DEV_LENGTH, b);
      if (row.n == 1) {
        seen = seen_chunks<kSub>(row.len - 1, row.len - 1, a.window, a.sinks);
        n = runs_of<A>(seen.n) * per_row;
      }
    }
    int inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    end = before + inc;
    begin = end - n;
    total = __shfl_sync(0xffffffffu, end, 31);
  }
  // moves to the window holding item `it`; false past the last item
  CBT_D bool seek(const A& a, int per_row, int it) {
    while (it >= total) {
      if (w0 + 32 >= a.rows) return false;
      load(a, per_row, w0 + 32, total);
    }
    return true;
  }
};

struct Item {
  int b, g, head0, heads;  // row, kv head, its first q head and their number
  int run, runs, t;        // run `run` of `runs`; the row's token
  int p;                   // the token's position
  int i0, i1;              // chunks [i0, i1) of `seen`
  Seen seen;
};

template <class A>
CBT_D Item item_at(const Cursor<A>& c, const A& a, int groups, int it) {
  const unsigned hit = __ballot_sync(0xffffffffu, it >= c.begin && it < c.end);
  const int src = __ffs(hit) - 1;
  Item w;
  w.b = c.w0 + src;
  int k = it - __shfl_sync(0xffffffffu, c.begin, src);
  w.t = __shfl_sync(0xffffffffu, c.row.t0, src);
  w.p = __shfl_sync(0xffffffffu, c.row.len, src) - 1;
  w.seen.ns = __shfl_sync(0xffffffffu, c.seen.ns, src);
  w.seen.ws = __shfl_sync(0xffffffffu, c.seen.ws, src);
  w.seen.n = __shfl_sync(0xffffffffu, c.seen.n, src);
  w.runs = runs_of<A>(w.seen.n);
  w.run = k % w.runs;
  k /= w.runs;
  const int G = a.n_heads / a.kv.n_kv_heads, j = k % groups;
  w.g = k / groups;
  w.head0 = w.g * G + j * kGroup;
  w.heads = min(kGroup, G - j * kGroup);
  const int per = chunks_per_run<A>(w.seen.n);
  w.i0 = w.run * per;
  w.i1 = min(w.seen.n, w.i0 + per);
  return w;
}

template <int N, bool MAX>
__device__ __forceinline__ void warp_reduce_n(float (&v)[N]) {  // level by level: latencies overlap
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    float t[N];
#pragma unroll
    for (int h = 0; h < N; ++h) t[h] = __shfl_xor_sync(0xffffffffu, v[h], o);
#pragma unroll
    for (int h = 0; h < N; ++h) v[h] = MAX ? fmaxf(v[h], t[h]) : v[h] + t[h];
  }
}

// Joins the runs of each (row, q head): o = sum_i o_i 2^(m_i - M) / sum_i l_i 2^(m_i - M).  One
// block per pair; warp w takes runs w, w + 4, ... in order with a running maximum, lane = head_dim /
// 32 dims, then the four warps' sums are added in a fixed order.
template <int HD, class A>
__global__ void __launch_bounds__(128)
    k_paged_merge(const __grid_constant__ A a, const float* __restrict__ part_o,
                  const float2* __restrict__ part_ml) {
  constexpr int R = HD / 32;
  __shared__ float wm[4], wl[4], wo[4][HD];
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // What the row asks for, before the wait: the blocks that hand over their runs have themselves waited for
  // whatever wrote it, before they let this launch begin.  (8 rows of 512 to 4096: 11.5 us for 12.0, over bf16
  // pages 14.7 for 15.3; one row of 4096 8.0 for 8.4.)
  const RowTokens row = row_tokens<true>(a, b);
  const Seen seen = seen_chunks<kSub>(row.len - 1, row.len - 1, a.window, a.sinks);
  const int runs = row.n == 1 ? runs_of<A>(seen.n) : 1;
  const size_t base = ((size_t)b * a.n_heads + h) * layout_of(a).max_runs;
  pdl_wait();
  pdl_launch();
  if (runs == 1) return;
  float m = -INFINITY, l = 0.f, acc[R];
#pragma unroll
  for (int r = 0; r < R; ++r) acc[r] = 0.f;
#pragma unroll 4
  for (int i = warp; i < runs; i += 4) {
    const float2 v = __ldcg(part_ml + base + i);
    float o[R];
    const float* po = part_o + (base + i) * HD + lane * R;
    if (R == 4) {
      const float4 f = __ldcg(reinterpret_cast<const float4*>(po));
      o[0] = f.x;
      o[1] = f.y;
      o[R - 2] = f.z;
      o[R - 1] = f.w;
    } else {
      const float2 f = __ldcg(reinterpret_cast<const float2*>(po));
      o[0] = f.x;
      o[1] = f.y;
    }
    const float mn = fmaxf(m, v.x);
    // m = -inf: no run yet, or runs whose scores are all -inf
    const float sc = m == -INFINITY ? 0.f : ex2(m - mn), wgt = v.x == -INFINITY ? 0.f : ex2(v.x - mn);
    l = fmaf(l, sc, v.y * wgt);
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = fmaf(acc[r], sc, o[r] * wgt);
    m = mn;
  }
  if (lane == 0) {
    wm[warp] = m;
    wl[warp] = l;
  }
#pragma unroll
  for (int r = 0; r < R; ++r) wo[warp][lane * R + r] = acc[r];
  __syncthreads();
  if (tid < HD) {
    const float M = fmaxf(fmaxf(wm[0], wm[1]), fmaxf(wm[2], wm[3]));
    float L = 0.f, o = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {  // a warp without runs has m = -inf and adds nothing
      const float sc = wm[w] == -INFINITY ? 0.f : ex2(wm[w] - M);
      L = fmaf(wl[w], sc, L);
      o = fmaf(wo[w][tid], sc, o);
    }
    o /= L;
    const long long at = row.t0 * a.out_ld + (long long)h * HD + tid;
    if (a.f32) static_cast<float*>(a.out)[at] = o;
    else static_cast<uint16_t*>(a.out)[at] = round_bf16(o);
  }
}

}  // namespace
