// paged_fp8.h -- launchers of the operators on a paged KV cache in 8 bits, and what their kernels share:
// where codes and scales lie, and how the scales' exponents are read.
#pragma once
#include "paged.h"

// One layer's K and V in a pool of pages (cbt_paged_kv_fp8)
struct PagedKvFp8 {
  static constexpr RunRule kRuns{4, 5, 33};
  uint8_t* pool;
  long long pool_bytes, page_bytes, k_off, v_off, s_off;
  int n_pages, page_tokens, n_kv_heads, head_dim;
};

constexpr int kBlock = CBT_FP8_BLOCK;      // positions of a scale
constexpr int kLowExp = -56, kHighExp = 56;  // a scale's exponents

// byte offsets of (page id, kv head, position o of the page, dim d)
CBT_HD long long fp8_k(const PagedKvFp8& c, int id, int head, int o, int d) {
  return id * c.page_bytes + c.k_off + ((long long)head * c.page_tokens + o) * c.head_dim + d;
}
CBT_HD long long fp8_v(const PagedKvFp8& c, int id, int head, int o, int d) {
  return id * c.page_bytes + c.v_off + (long long)head * c.page_tokens * c.head_dim +
         ((long long)(o >> 6) * c.head_dim + d) * kBlock + (o & 63);
}
// the scale of K (v = 0) or V (v = 1) of the block with position o of the page
CBT_HD float* fp8_scale(const PagedKvFp8& c, int id, int v, int head, int o) {
  return reinterpret_cast<float*>(c.pool + id * c.page_bytes + c.s_off) +
         ((long long)v * c.n_kv_heads + head) * (c.page_tokens / kBlock) + o / kBlock;
}
// the exponent that a stored scale stands for
CBT_D int fp8_exponent(float scale) {
  const int e = (int)(__float_as_uint(scale) >> 23 & 255) - 127;
  return min(max(e, kLowExp), kHighExp);
}
// 2^e for a whole e in [-126, 127]
CBT_D float pow2_of(int e) { return __int_as_float((e + 127) << 23); }

// two values to e4m3 codes (lo in the low byte): nearest even, beyond 448 the largest, NaN stays
CBT_D uint16_t pack_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// two codes to two fp16 (exact)
CBT_D uint32_t e4m3_to_f16(uint16_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(codes));
  return r;
}
CBT_D uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
CBT_D uint16_t f16_to_e4m3(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
CBT_D float f16_lo(uint32_t h) {
  float f;
  asm("{\n .reg .b16 l, u;\n mov.b32 {l, u}, %1;\n cvt.f32.f16 %0, l;\n}\n" : "=f"(f) : "r"(h));
  return f;
}
CBT_D float f16_hi(uint32_t h) {
  float f;
  asm("{\n .reg .b16 l, u;\n mov.b32 {l, u}, %1;\n cvt.f32.f16 %0, u;\n}\n" : "=f"(f) : "r"(h));
  return f;
}

// the 4 x 4 bytes of four words (row i: word i) with rows and columns exchanged
CBT_D void transpose4(uint32_t (&w)[4]) {
  const uint32_t a = __byte_perm(w[0], w[1], 0x5140), b = __byte_perm(w[2], w[3], 0x5140);
  const uint32_t c = __byte_perm(w[0], w[1], 0x7362), d = __byte_perm(w[2], w[3], 0x7362);
  w[0] = __byte_perm(a, b, 0x5410);
  w[1] = __byte_perm(a, b, 0x7632);
  w[2] = __byte_perm(c, d, 0x5410);
  w[3] = __byte_perm(c, d, 0x7632);
}

using RopeAppendFp8 = RopeAppendOn<PagedKvFp8>;
cudaError_t launch_append_fp8(const RopeAppendFp8& a, cudaStream_t s);

struct PagedReadFp8 {
  PagedKvFp8 kv;
  const int32_t* table;
  int max_pages, rows;
  const int32_t *lens, *first, *cu;
  int tokens;
  void *k_out, *v_out;
  bool f32;
  long long out_ld;
  int* err;
};
cudaError_t launch_read_fp8(const PagedReadFp8& a, cudaStream_t s);

using PagedAttnFp8 = PagedAttnOn<PagedKvFp8>;
size_t attn_fp8_workspace(const PagedAttnFp8& a);
cudaError_t launch_attn_fp8(const PagedAttnFp8& a, int num_sms, cudaStream_t s);
// its two forms: one query token per row (max_q == 1), and ragged runs of them
size_t decode_fp8_workspace(const PagedAttnFp8& a);
cudaError_t launch_decode_fp8(const PagedAttnFp8& a, int num_sms, cudaStream_t s);
size_t prefill_fp8_workspace(const PagedAttnFp8& a);
cudaError_t launch_prefill_fp8(const PagedAttnFp8& a, int num_sms, cudaStream_t s);
