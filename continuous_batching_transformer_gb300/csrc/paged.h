// paged.h -- launchers of the operators on a paged KV cache (host side) and the index helpers
// their kernels share.  The same operators on a cache in 8 bits: paged_fp8.h.
#pragma once
#include "kernels.h"

// How attention of single tokens cuts a row of n 128-key chunks into runs: up to `one` chunks are one run;
// below `two` they go singly, below `four` by twos, from there on by fours (paged_split.cuh).
struct RunRule {
  int one, two, four;
};

// One layer's K and V in a pool of pages (cbt_paged_kv with every offset in bf16 elements)
struct PagedKv {
  static constexpr RunRule kRuns{3, 32, 96};
  uint16_t* pool;
  long long pool_elems, page_elems, k_off, v_off;
  int n_pages, page_tokens, n_kv_heads, head_dim;
};

// element offsets of (page id, kv head, position o of the page, dim d)
CBT_HD long long paged_k(const PagedKv& c, int id, int head, int o, int d) {
  return id * c.page_elems + c.k_off + ((long long)head * c.page_tokens + o) * c.head_dim + d;
}
CBT_HD long long paged_v(const PagedKv& c, int id, int head, int o, int d) {
  return id * c.page_elems + c.v_off + (long long)head * c.page_tokens * c.head_dim +
         ((long long)(o >> 6) * c.head_dim + d) * 64 + (o & 63);
}

cudaError_t launch_page_map(const cbt_page_map_args& a, cudaStream_t s);

template <class Kv>
struct RopeAppendOn {
  Kv kv;
  cbt_rope rope;  // rot_dim 0: no rotation
  const void* qkv;
  bool f32;
  long long qkv_ld;
  int tokens, n_heads;
  const uint16_t *q_gain, *k_gain;
  float eps;
  const int32_t *positions, *slots;
  uint16_t* q_out;
  long long q_ld;
  int* err;
};
using RopeAppend = RopeAppendOn<PagedKv>;
cudaError_t launch_paged_rope(const RopeAppend& a, cudaStream_t s);

template <class Kv>
struct PagedAttnOn {
  Kv kv;
  const int32_t* table;
  int max_pages, rows;
  const int32_t* lens;
  const int32_t* cu;  // NULL: one token per row
  int tokens, max_q, max_kv, n_heads;
  const uint16_t* q;
  long long q_ld;
  float scale;
  int window, sinks;
  void* out;
  bool f32;
  long long out_ld;
  uint8_t* ws;
  size_t ws_bytes;
  int* err;
};
using PagedAttn = PagedAttnOn<PagedKv>;
size_t paged_attn_workspace(const PagedAttn& a);
cudaError_t launch_paged_attn(const PagedAttn& a, int num_sms, cudaStream_t s);
// its two forms: one query token per row (max_q == 1), split over the cache's length, and ragged
// runs of them
size_t paged_decode_workspace(const PagedAttn& a);
cudaError_t launch_paged_decode(const PagedAttn& a, int num_sms, cudaStream_t s);
size_t paged_prefill_workspace(const PagedAttn& a);
cudaError_t launch_paged_prefill(const PagedAttn& a, int num_sms, cudaStream_t s);
