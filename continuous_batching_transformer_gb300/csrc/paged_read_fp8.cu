// paged_read_fp8.cu -- positions of a paged cache in 8 bits read back as K and V rows.
//
// One byte in and two (bf16) or four out an element: HBM is the floor.  A thread block takes 64
// positions of a row that share their scales, for one kv head, and K or V.  K's rows leave as they come;
// V's codes, which lie along the positions of a dim, go through shared memory and are turned around four
// by four, so that a warp stores whole rows of positions.  Measured: four rows of 8192 to 16384 positions, 8
// heads of 128, 38.9 us = 6.2 TB/s, 93 % of the measured copy rate; three short rows 2.4 us.
#include "paged_attn.cuh"
#include "paged_fp8.h"

namespace {

constexpr int kThreads = 128;

// eight codes of consecutive dims times a scale, to out
template <bool F32>
CBT_D void store_values(void* out, uint32_t w0, uint32_t w1, float f) {
  const uint32_t h[4] = {e4m3_to_f16((uint16_t)w0), e4m3_to_f16((uint16_t)(w0 >> 16)), e4m3_to_f16((uint16_t)w1),
                         e4m3_to_f16((uint16_t)(w1 >> 16))};
  float x[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = f16_lo(h[e]) * f;
    x[2 * e + 1] = f16_hi(h[e]) * f;
  }
  if (F32) {
    static_cast<float4*>(out)[0] = make_float4(x[0], x[1], x[2], x[3]);
    static_cast<float4*>(out)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *static_cast<uint4*>(out) =
        make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  }
}

// What row b asks for: rows [t0, t1) of the output, from position `from` on
struct Range {
  int t0, t1, from, len;
};
CBT_D Range range_of(const PagedReadFp8& a, int b) {
  return {a.cu[b], a.cu[b + 1], a.first ? a.first[b] : 0, a.lens[b]};
}
CBT_D bool bad(const PagedReadFp8& a, const Range& r) {
  return r.t0 < 0 || r.t1 < r.t0 || r.t1 > a.tokens || r.from < 0 || (long long)r.from + (r.t1 - r.t0) > r.len ||
         r.len > (long long)a.max_pages * a.kv.page_tokens;
}
// Row b's blocks are given the items from t0 / 64 + 2 b on: as many as it can have, wherever its first
// position lies in a block, and the row of an item is found by search.
CBT_D long long first_item(const PagedReadFp8& a, int b, int t0) {
  return (long long)(max(0, min(t0, a.tokens)) / kBlock) + 2 * b;
}

template <int HD, bool F32>
__global__ void __launch_bounds__(kThreads) k_read_fp8(const __grid_constant__ PagedReadFp8 a) {
  // V's codes [dim][64 positions] as words, a dim's 16 turned by its eighth, so that reads along the dims
  // fall into different banks
  __shared__ uint32_t tile[HD * 16];
  const int tid = threadIdx.x, lane = tid & 31;
  const int KV = a.kv.n_kv_heads, g = blockIdx.y % KV, v = blockIdx.y / KV;
  pdl_wait();
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    for (int r = tid; r < a.rows; r += kThreads)
      if (bad(a, range_of(a, r))) set_device_error(a.err, CBT_DEV_LENGTH, r);
  }
  if (!(v ? a.v_out : a.k_out)) return;
  const long long item = blockIdx.x;
  // the last row whose items begin at or before this one
  int b = 0;
  Range r{};
  if (a.rows <= 32) {  // all of them at once, with what they ask for
    const Range mine = lane < a.rows ? range_of(a, lane) : Range{};
    const unsigned in = __ballot_sync(0xffffffffu, lane < a.rows && first_item(a, lane, mine.t0) <= item);
    b = 31 - __clz(in | 1);
    r = Range{__shfl_sync(0xffffffffu, mine.t0, b), __shfl_sync(0xffffffffu, mine.t1, b),
              __shfl_sync(0xffffffffu, mine.from, b), __shfl_sync(0xffffffffu, mine.len, b)};
  } else {
    int n = a.rows;
#pragma unroll 1
    while (n > 1) {  // 32 rows at a time
      const int step = (n + 31) / 32, at = b + lane * step;
      const unsigned in = __ballot_sync(0xffffffffu, lane * step < n && first_item(a, at, a.cu[at]) <= item);
      const int k = 31 - __clz(in | 1);
      b += k * step;
      n = min(step, n - k * step);
    }
    r = range_of(a, b);
  }
  const long long nth = item - first_item(a, b, r.t0);  // block of the row (below 0: before the first row)
  if (nth < 0 || bad(a, r)) return;
  const int t0 = r.t0, from = r.from, count = r.t1 - r.t0;
  const long long p0 = (from / kBlock + nth) * kBlock;
  if (count == 0 || p0 >= (long long)from + count) return;
  const int page = a.kv.page_tokens, pg = (int)p0 / page, o = (int)p0 - pg * page;
  int id = a.table[(size_t)b * a.max_pages + pg];
  if (id < 0 || id >= a.kv.n_pages) {
    if (tid == 0) set_device_error(a.err, CBT_DEV_PAGE_ID, b);
    return;
  }
  const float scale = pow2_of(fp8_exponent(*fp8_scale(a.kv, id, v, g, o)));
  constexpr int kLanes = HD / 8, kAtOnce = kThreads / kLanes;  // threads of a position, positions at once
  constexpr int kSize = F32 ? 4 : 2;
  const int part = tid % kLanes;                               // of a position: 8 dims
  // row of the block's first position (its own may be another row's, or none: only those asked for are written)
  uint8_t* out = static_cast<uint8_t*>(v ? a.v_out : a.k_out) +
                 ((t0 - from + p0) * a.out_ld + (long long)g * HD + 8 * part) * kSize;
  const long long step = a.out_ld * kSize;
  // the block's positions (the last block's end, as one, may be past 32 bits)
  const int lo_p = max(from - (int)p0, 0), hi_p = min(from + count - (int)p0, kBlock);
  if (!v) {
    const uint2* src = reinterpret_cast<const uint2*>(a.kv.pool + fp8_k(a.kv, id, g, o, 0)) + tid;
    uint2 w[kBlock / kAtOnce];
#pragma unroll
    for (int k = 0; k < kBlock / kAtOnce; ++k) w[k] = __ldg(src + k * kThreads);
    uint8_t* dst = out + tid / kLanes * step;
#pragma unroll
    for (int k = 0; k < kBlock / kAtOnce; ++k) {
      const int p = k * kAtOnce + tid / kLanes;
      if (p >= lo_p && p < hi_p) store_values<F32>(dst, w[k].x, w[k].y, scale);
      dst += kAtOnce * step;
    }
    return;
  }
  const uint4* src = reinterpret_cast<const uint4*>(a.kv.pool + fp8_v(a.kv, id, g, o, 0));
  uint4 in[HD * 4 / kThreads];
#pragma unroll
  for (int k = 0; k < HD * 4 / kThreads; ++k) in[k] = __ldg(src + k * kThreads + tid);
  auto at = [](int d, int word) { return d * 16 + ((word + (d >> 3)) & 15); };
#pragma unroll
  for (int k = 0; k < HD * 4 / kThreads; ++k) {
    const int d = (k * kThreads + tid) / 4, q = (k * kThreads + tid) % 4 * 4;
    tile[at(d, q)] = in[k].x;
    tile[at(d, q + 1)] = in[k].y;
    tile[at(d, q + 2)] = in[k].z;
    tile[at(d, q + 3)] = in[k].w;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kBlock / 4 / kAtOnce; ++k) {  // four positions of 8 dims
    const int word = k * kAtOnce + tid / kLanes;
    uint32_t w[2][4];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e >> 2][e & 3] = tile[at(8 * part + e, word)];
    transpose4(w[0]);
    transpose4(w[1]);
    uint8_t* dst = out + 4 * word * step;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int p = 4 * word + e;
      if (p >= lo_p && p < hi_p) store_values<F32>(dst, w[0][e], w[1][e], scale);
      dst += step;
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
