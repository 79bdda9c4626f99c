// paged_rope.cu -- per-head RMS norm, rotary positions and the append of K and V to a paged cache,
// one pass over QKV rows.
#include "paged.h"

namespace {

CBT_D float load_elem(const void* p, long long i, bool f32) {
  return f32 ? static_cast<const float*>(p)[i] : bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}

// One block per (token, head), one thread per dim.
__global__ void k_rope_append(const RopeAppend a) {
  __shared__ float xs[128], red[4];
  pdl_wait();
  const int t = blockIdx.x, h = blockIdx.y, d = threadIdx.x;
  const int hd = a.kv.head_dim, Hq = a.n_heads, Hk = a.kv.n_kv_heads;
  const int slot = a.slots[t], pos = a.positions[t];
  if (slot < 0 || pos < 0) return;
  if (slot >= a.kv.n_pages * a.kv.page_tokens) {
    if (d == 0 && h == 0) set_device_error(a.err, CBT_DEV_PAGE_ID, t);
    return;
  }
  const int id = slot / a.kv.page_tokens, o = slot % a.kv.page_tokens;
  float x = load_elem(a.qkv, t * a.qkv_ld + (long long)h * hd + d, a.f32);
  if (h >= Hq + Hk) {
    a.kv.pool[paged_v(a.kv, id, h - Hq - Hk, o, d)] = f32_to_bf16(x);
    return;
  }
  const uint16_t* gain = h < Hq ? a.q_gain : a.k_gain;
  if (gain) {
    const float s = warp_sum(x * x);
    if ((d & 31) == 0) red[d >> 5] = s;
    __syncthreads();
    float tot = 0.f;
    for (int w = 0; w < hd / 32; ++w) tot += red[w];
    x = x * rsqrtf(tot / (float)hd + a.eps) * bf16_to_f32(gain[d]);
  }
  xs[d] = x;
  __syncthreads();
  const int rot = a.rope.rot_dim, half = rot / 2;
  if (d < rot) {
    const bool second = a.rope.layout == CBT_ROPE_HALF ? d >= half : d & 1;
    const int pair = a.rope.layout == CBT_ROPE_HALF ? (second ? d - half : d) : d / 2;
    const int other = a.rope.layout == CBT_ROPE_HALF ? (second ? d - half : d + half) : d ^ 1;
    const uint64_t ph = (uint64_t)pos * a.rope.turns[pair];
    float sn, cs;
    sincospif((float)(int32_t)(ph >> 32) * 0x1p-31f, &sn, &cs);
    sn *= a.rope.mscale;
    cs *= a.rope.mscale;
    x = second ? fmaf(x, cs, xs[other] * sn) : fmaf(x, cs, -xs[other] * sn);
  }
  if (h < Hq) a.q_out[t * a.q_ld + (long long)h * hd + d] = f32_to_bf16(x);
  else a.kv.pool[paged_k(a.kv, id, h - Hq, o, d)] = f32_to_bf16(x);
}

}  // namespace

cudaError_t launch_paged_rope(const RopeAppend& a, cudaStream_t s) {
  return launch_pdl(k_rope_append, dim3(a.tokens, a.n_heads + 2 * a.kv.n_kv_heads),
                    dim3(a.kv.head_dim), 0, s, a);
}
