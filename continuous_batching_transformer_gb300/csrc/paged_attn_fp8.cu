// paged_attn_fp8.cu -- attention over a paged cache in 8 bits, the simple form: a warp takes one query
// token and head and walks the keys it sees, 32 at a time.
#include "paged_attn.cuh"
#include "paged_fp8.h"

namespace {

constexpr int kWarps = 4;

template <int HD>
__global__ void __launch_bounds__(32 * kWarps) k_attn_fp8(const __grid_constant__ PagedAttnFp8 a) {
  constexpr int R = HD / 32;
  __shared__ float sq[kWarps][HD];
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, H = a.n_heads;
  const int b = blockIdx.y, G = H / a.kv.n_kv_heads;
  const RowTokens row = row_tokens(a, b);
  if (row.bad) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_device_error(a.err, CBT_DEV_LENGTH, b);
    return;
  }
  const int page = a.kv.page_tokens;
#pragma unroll 1
  for (long long w = (long long)blockIdx.x * kWarps + warp; w < (long long)row.n * H; w += (long long)gridDim.x * kWarps) {
    const int i = (int)(w / H), h = (int)(w - (long long)i * H), g = h / G;
    const int p = row.len - row.n + i;
    const uint16_t* q = a.q + (long long)(row.t0 + i) * a.q_ld + (long long)h * HD;
    __syncwarp();
    for (int d = lane; d < HD; d += 32) sq[warp][d] = bf16_to_f32(q[d]);
    __syncwarp();
    float m = -INFINITY, l = 0.f, acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = 0.f;
    const Seen seen = seen_chunks<32>(p, p, a.window, a.sinks);
#pragma unroll 1
    for (int c = 0; c < seen.n; ++c) {
      const int k0 = seen.chunk(c) * 32, pg = k0 / page, o = k0 - pg * page;
      int id = a.table[(size_t)b * a.max_pages + pg];
      if (id < 0 || id >= a.kv.n_pages) {
        set_device_error(a.err, CBT_DEV_PAGE_ID, b);
        id = 0;
      }
      const bool on = sees(k0 + lane, p, a.window, a.sinks);
      float s = -INFINITY;
      if (on) {
        const uint32_t* k = reinterpret_cast<const uint32_t*>(a.kv.pool + fp8_k(a.kv, id, g, o + lane, 0));
        float dot = 0.f;
#pragma unroll 4
        for (int d = 0; d < HD / 4; ++d) {
          const uint32_t x = __ldg(k + d), lo = e4m3_to_f16((uint16_t)x), hi = e4m3_to_f16((uint16_t)(x >> 16));
          dot = fmaf(f16_lo(lo), sq[warp][4 * d], dot);
          dot = fmaf(f16_hi(lo), sq[warp][4 * d + 1], dot);
          dot = fmaf(f16_lo(hi), sq[warp][4 * d + 2], dot);
          dot = fmaf(f16_hi(hi), sq[warp][4 * d + 3], dot);
        }
        s = dot * pow2_of(fp8_exponent(*fp8_scale(a.kv, id, 0, g, o))) * (a.scale * kLog2e);
      }
      const float mn = fmaxf(m, warp_max(s));
      const float ref = mn == -INFINITY ? 0.f : mn, sc = m == -INFINITY ? 0.f : ex2(m - ref);
      const float wgt = on ? ex2(s - ref) : 0.f;
      m = mn;
      l = l * sc + warp_sum(wgt);
#pragma unroll
      for (int r = 0; r < R; ++r) acc[r] *= sc;
      const float vs = pow2_of(fp8_exponent(*fp8_scale(a.kv, id, 1, g, o)));
      const unsigned bits = __ballot_sync(0xffffffffu, on);
#pragma unroll 1
      for (int j = 0; j < 32; ++j) {
        const float wj = __shfl_sync(0xffffffffu, wgt, j) * vs;
        if (!(bits >> j & 1)) continue;
#pragma unroll
        for (int r = 0; r < R; ++r)
          acc[r] = fmaf(f16_lo(e4m3_to_f16(a.kv.pool[fp8_v(a.kv, id, g, o + j, lane * R + r)])), wj, acc[r]);
      }
    }
    const long long at = (long long)(row.t0 + i) * a.out_ld + (long long)h * HD + lane * R;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float y = seen.n ? acc[r] / l : 0.f;
      if (a.f32) static_cast<float*>(a.out)[at + r] = y;
      else static_cast<uint16_t*>(a.out)[at + r] = round_bf16(y);
    }
  }
}

}  // namespace

size_t attn_fp8_workspace(const PagedAttnFp8& a) { return a.max_q == 1 ? decode_fp8_workspace(a) : 0; }

cudaError_t launch_attn_fp8(const PagedAttnFp8& a, int num_sms, cudaStream_t s) {
  if (attn_fp8_workspace(a) > a.ws_bytes) return cudaErrorInvalidValue;
  if (a.max_q == 1) return launch_decode_fp8(a, num_sms, s);
  const long long pairs = (long long)a.max_q * a.n_heads, most = (pairs + kWarps - 1) / kWarps;
  const dim3 grid((unsigned)(most < 64 * num_sms ? most : 64 * num_sms), a.rows);
  return a.kv.head_dim == 128 ? launch_pdl(k_attn_fp8<128>, grid, dim3(32 * kWarps), 0, s, a)
                              : launch_pdl(k_attn_fp8<64>, grid, dim3(32 * kWarps), 0, s, a);
}
