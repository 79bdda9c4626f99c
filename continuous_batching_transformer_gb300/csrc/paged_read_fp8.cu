// paged_read_fp8.cu -- positions of a paged cache in 8 bits read back as K and V rows.
//
// One byte in and two (bf16) or four out an element: HBM is the floor.  A thread block takes 64
// positions of a row that share their scales, for one kv head, and K or V.  K's rows leave as they come;
// V's codes, which lie along the positions of a dim, go through shared memory and are turned around four
// by four, so that a warp stores whole rows of a position.
#include "paged_attn.cuh"
#include "paged_fp8.h"

namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;

// four codes of consecutive dims times a scale, to out[0 .. 3]
template <bool F32>
CBT_D void store_values(void* out, long long at, uint32_t w, float f) {
  const uint32_t lo = e4m3_to_f16((uint16_t)w), hi = e4m3_to_f16((uint16_t)(w >> 16));
  const float a = f16_lo(lo) * f, b = f16_hi(lo) * f, c = f16_lo(hi) * f, d = f16_hi(hi) * f;
  if (F32) *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = make_float4(a, b, c, d);
  else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = make_uint2(pack_bf16(a, b), pack_bf16(c, d));
}

// Row b's blocks are given the items from cu[b] / 64 + 2 b on: as many as it can have, wherever its
// first position lies in a block, and the row of an item is found by search.
CBT_D long long first_item(const PagedReadFp8& a, int b) {
  return (long long)(max(0, min(a.cu[b], a.tokens)) / kBlock) + 2 * b;
}

CBT_D bool bad_row(const PagedReadFp8& a, int b) {
  const int t0 = a.cu[b], t1 = a.cu[b + 1], from = a.first ? a.first[b] : 0, len = a.lens[b];
  return t0 < 0 || t1 < t0 || t1 > a.tokens || from < 0 || (long long)from + (t1 - t0) > len ||
         len > (long long)a.max_pages * a.kv.page_tokens;
}

template <int HD, bool F32>
__global__ void __launch_bounds__(kThreads) k_read_fp8(const __grid_constant__ PagedReadFp8 a) {
  // V's codes [dim][64 positions] as words, a dim's 16 turned by its quad, so that a warp's reads along
  // the dims fall into different banks (but for two lanes)
  __shared__ uint32_t tile[HD * 16];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int KV = a.kv.n_kv_heads, g = blockIdx.y % KV, v = blockIdx.y / KV;
  pdl_wait();
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    for (int r = tid; r < a.rows; r += kThreads)
      if (bad_row(a, r)) set_device_error(a.err, CBT_DEV_LENGTH, r);
  }
  if (!(v ? a.v_out : a.k_out)) return;
  const long long item = blockIdx.x;
  // the last row whose items begin at or before this one
  int lo = 0, n = a.rows;
#pragma unroll 1
  while (n > 1) {  // 32 rows at a time
    const int step = (n + 31) / 32, b = lo + lane * step;
    const unsigned in = __ballot_sync(0xffffffffu, lane * step < n && first_item(a, b) <= item);
    const int k = 31 - __clz(in | 1);
    lo += k * step;
    n = min(step, n - k * step);
  }
  const int b = lo, t0 = a.cu[b], t1 = a.cu[b + 1], from = a.first ? a.first[b] : 0;
  const long long nth = item - first_item(a, b);  // block of the row (below 0: before the first row)
  if (nth < 0 || bad_row(a, b)) return;
  const int count = t1 - t0;
  const long long p0 = (from / kBlock + nth) * kBlock;
  if (count == 0 || p0 >= (long long)from + count) return;
  const int begin = max(from, (int)p0), end = min(from + count, (int)p0 + kBlock);  // positions
  const int page = a.kv.page_tokens, pg = (int)p0 / page, o = (int)p0 - pg * page;
  int id = a.table[(size_t)b * a.max_pages + pg];
  if (id < 0 || id >= a.kv.n_pages) {
    if (tid == 0) set_device_error(a.err, CBT_DEV_PAGE_ID, b);
    return;
  }
  const float scale = pow2_of(fp8_exponent(*fp8_scale(a.kv, id, v, g, o)));
  void* out = v ? a.v_out : a.k_out;
  const long long row0 = (long long)t0 - from;  // position p is row row0 + p
  constexpr int kQuads = HD / 4;                // lanes of a position
  if (!v) {
    const uint32_t* src = reinterpret_cast<const uint32_t*>(a.kv.pool + fp8_k(a.kv, id, g, o, 0));
    uint32_t w[kBlock * kQuads / kThreads];
#pragma unroll
    for (int k = 0; k < kBlock * kQuads / kThreads; ++k) {
      const int p = (int)p0 + (k * kThreads + tid) / kQuads;
      w[k] = p >= begin && p < end ? __ldg(src + k * kThreads + tid) : 0;
    }
#pragma unroll
    for (int k = 0; k < kBlock * kQuads / kThreads; ++k) {
      const int p = (int)p0 + (k * kThreads + tid) / kQuads, d = (k * kThreads + tid) % kQuads * 4;
      if (p >= begin && p < end) store_values<F32>(out, (row0 + p) * a.out_ld + (long long)g * HD + d, w[k], scale);
    }
    return;
  }
  const uint4* src = reinterpret_cast<const uint4*>(a.kv.pool + fp8_v(a.kv, id, g, o, 0));
  uint4 in[HD * 4 / kThreads];
#pragma unroll
  for (int k = 0; k < HD * 4 / kThreads; ++k) in[k] = __ldg(src + k * kThreads + tid);
  auto at = [](int d, int word) { return d * 16 + ((word + (d >> 2)) & 15); };
#pragma unroll
  for (int k = 0; k < HD * 4 / kThreads; ++k) {
    const int d = (k * kThreads + tid) / 4, q = (k * kThreads + tid) % 4 * 4;
    tile[at(d, q)] = in[k].x;
    tile[at(d, q + 1)] = in[k].y;
    tile[at(d, q + 2)] = in[k].z;
    tile[at(d, q + 3)] = in[k].w;
  }
  __syncthreads();
  constexpr int kPer = 32 / kQuads;  // words of positions that a warp takes at once
#pragma unroll
  for (int k = 0; k < 16 / (kWarps * kPer); ++k) {
    const int word = (k * kWarps + warp) * kPer + lane / kQuads, d = lane % kQuads * 4;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = tile[at(d + e, word)];
    transpose4(w);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int p = (int)p0 + word * 4 + e;
      if (p >= begin && p < end) store_values<F32>(out, (row0 + p) * a.out_ld + (long long)g * HD + d, w[e], scale);
    }
  }
}

template <int HD, bool F32>
cudaError_t launch(const PagedReadFp8& a, cudaStream_t s) {
  const long long items = (long long)a.tokens / kBlock + 2ll * a.rows + 1;
  return launch_pdl(k_read_fp8<HD, F32>, dim3((unsigned)items, 2 * a.kv.n_kv_heads), dim3(kThreads), 0, s, a);
}

}  // namespace

cudaError_t launch_read_fp8(const PagedReadFp8& a, cudaStream_t s) {
  if (a.kv.head_dim == 128) return a.f32 ? launch<128, true>(a, s) : launch<128, false>(a, s);
  return a.f32 ? launch<64, true>(a, s) : launch<64, false>(a, s);
}
