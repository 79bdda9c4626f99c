// paged_attn.cu -- attention of ragged runs of query tokens over a paged KV cache, causal, with an
// optional sliding window and first tokens that stay visible.
#include "paged_attn.cuh"

namespace {

// One warp per (token, q head): every lane holds head_dim / 32 dims of q and the output.
template <int HD>
__global__ void k_paged_attn(const PagedAttn a) {
  constexpr int R = HD / 32;
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x, h = blockIdx.y * 4 + (threadIdx.x >> 5);
  if (a.cu && t == 0 && blockIdx.y == 0) {  // the rows' query ranges
    for (int r = threadIdx.x; r < a.rows; r += blockDim.x)
      if (a.cu[r] < 0 || a.cu[r + 1] < a.cu[r] || a.cu[r + 1] > a.tokens || a.cu[r + 1] - a.cu[r] > a.max_q)
        set_device_error(a.err, CBT_DEV_LENGTH, r);
  }
  if (h >= a.n_heads) return;
  int b = t, c0 = t, c1 = t + 1;
  if (a.cu) {
    int lo = 0, hi = a.rows;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.cu[mid] <= t) lo = mid;
      else hi = mid;
    }
    b = lo;
    c0 = a.cu[b];
    c1 = a.cu[b + 1];
    if (t < c0 || t >= c1 || c1 > a.tokens) return;
  }
  const int n = a.lens[b];
  if (n < 0 || n > a.max_kv || n > (long long)a.max_pages * a.kv.page_tokens) {
    if (lane == 0) set_device_error(a.err, CBT_DEV_LENGTH, b);
    return;
  }
  const int p = n - (c1 - c0) + (t - c0), g = h / (a.n_heads / a.kv.n_kv_heads);
  float q[R], o[R], m = -INFINITY, l = 0.f;
  for (int r = 0; r < R; ++r) {
    q[r] = bf16_to_f32(a.q[t * a.q_ld + h * HD + lane * R + r]);
    o[r] = 0.f;
  }
  for (int j = 0; j <= p; ++j) {
    if (a.window && j <= p - a.window && j >= a.sinks) {
      j = p - a.window;
      continue;
    }
    const int id = a.table[(size_t)b * a.max_pages + j / a.kv.page_tokens], off = j % a.kv.page_tokens;
    if (id < 0 || id >= a.kv.n_pages) {
      if (lane == 0) set_device_error(a.err, CBT_DEV_PAGE_ID, b);
      return;
    }
    float s = 0.f;
    for (int r = 0; r < R; ++r)
      s = fmaf(q[r], bf16_to_f32(a.kv.pool[paged_k(a.kv, id, g, off, lane * R + r)]), s);
    s = warp_sum(s) * a.scale;
    const float mn = fmaxf(m, s), sc = m == -INFINITY ? 0.f : __expf(m - mn), w = __expf(s - mn);
    l = fmaf(l, sc, w);
    for (int r = 0; r < R; ++r)
      o[r] = fmaf(o[r], sc, w * bf16_to_f32(a.kv.pool[paged_v(a.kv, id, g, off, lane * R + r)]));
    m = mn;
  }
  for (int r = 0; r < R; ++r) {
    const float v = p >= 0 ? o[r] / l : 0.f;
    const long long at = t * a.out_ld + h * HD + lane * R + r;
    if (a.f32) static_cast<float*>(a.out)[at] = v;
    else static_cast<uint16_t*>(a.out)[at] = f32_to_bf16(v);
  }
}

}  // namespace

size_t paged_attn_workspace(const PagedAttn& a) {
  return a.max_q == 1 ? paged_decode_workspace(a) : 0;
}

cudaError_t launch_paged_attn(const PagedAttn& a, cudaStream_t s) {
  int dev = 0, num_sms = 0;
  cudaError_t rc = cudaGetDevice(&dev);
  if (rc == cudaSuccess) rc = cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, dev);
  if (rc != cudaSuccess) return rc;
  if (a.max_q == 1) return launch_paged_decode(a, num_sms, s);
  const dim3 grid(a.tokens, (a.n_heads + 3) / 4);
  return a.kv.head_dim == 128 ? launch_pdl(k_paged_attn<128>, grid, dim3(128), 0, s, a)
                              : launch_pdl(k_paged_attn<64>, grid, dim3(128), 0, s, a);
}
