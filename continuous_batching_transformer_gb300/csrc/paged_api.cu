// paged_api.cu -- the C entries of the operators on a paged KV cache: argument checks, then the
// launch.  Nothing here touches the device before every check has passed.
#include <math.h>

#include "paged_fp8.h"

namespace {

// most tokens or pages of a call: the kernels' 32-bit counters step past the last by less than this
constexpr int32_t kMostTokens = 1 << 30;

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// checks a descriptor and converts it to elements
cbt_status paged_kv(const cbt_paged_kv& k, PagedKv* out) {
  if (!k.pool) return CBT_ERR_NULL;
  if (k.head_dim != 64 && k.head_dim != 128) return CBT_ERR_UNSUPPORTED;
  if (k.n_pages <= 0 || k.page_tokens <= 0 || k.page_tokens % 64 || k.n_kv_heads <= 0 ||
      k.page_bytes <= 0 || k.page_bytes % 256 || k.k_offset < 0 || k.k_offset % 256 ||
      k.v_offset < 0 || k.v_offset % 256 || !aligned(k.pool, 256))
    return CBT_ERR_INVALID;
  if ((int64_t)k.n_pages * k.page_tokens > INT32_MAX || k.pool_bytes >= (size_t)128 << 31)
    return CBT_ERR_LIMIT;
  // pool_bytes < 2^38, so with both factors checked against it no product below overflows
  if ((uint64_t)k.page_bytes > k.pool_bytes || (uint64_t)k.k_offset > k.pool_bytes ||
      (uint64_t)k.v_offset > k.pool_bytes)
    return CBT_ERR_INVALID;
  const double block = 2.0 * k.n_kv_heads * k.page_tokens * k.head_dim;
  const double last = (double)(k.n_pages - 1) * (double)k.page_bytes;
  const double off = (double)(k.k_offset > k.v_offset ? k.k_offset : k.v_offset);
  if (last + off + block > (double)k.pool_bytes) return CBT_ERR_INVALID;
  out->pool = static_cast<uint16_t*>(k.pool);
  out->pool_elems = (long long)(k.pool_bytes / 2);
  out->page_elems = k.page_bytes / 2;
  out->k_off = k.k_offset / 2;
  out->v_off = k.v_offset / 2;
  out->n_pages = k.n_pages;
  out->page_tokens = k.page_tokens;
  out->n_kv_heads = k.n_kv_heads;
  out->head_dim = k.head_dim;
  return CBT_OK;
}

cbt_status paged_kv(const cbt_paged_kv_fp8& k, PagedKvFp8* out) {
  if (!k.pool) return CBT_ERR_NULL;
  if (k.head_dim != 64 && k.head_dim != 128) return CBT_ERR_UNSUPPORTED;
  if (k.n_pages <= 0 || k.page_tokens <= 0 || k.page_tokens % kBlock || k.n_kv_heads <= 0 || k.page_bytes <= 0 ||
      k.page_bytes % 256 || k.k_offset < 0 || k.k_offset % 256 || k.v_offset < 0 || k.v_offset % 256 ||
      k.s_offset < 0 || k.s_offset % 256 || !aligned(k.pool, 256))
    return CBT_ERR_INVALID;
  // 256: what the tensor maps count in
  if ((int64_t)k.n_pages * k.page_tokens > INT32_MAX || k.pool_bytes >= (size_t)256 << 31)
    return CBT_ERR_LIMIT;
  if ((uint64_t)k.page_bytes > k.pool_bytes || (uint64_t)k.k_offset > k.pool_bytes ||
      (uint64_t)k.v_offset > k.pool_bytes || (uint64_t)k.s_offset > k.pool_bytes)
    return CBT_ERR_INVALID;
  const double block = (double)k.n_kv_heads * k.page_tokens * k.head_dim;
  const double scales = 8.0 * k.n_kv_heads * (k.page_tokens / kBlock);
  const double off = (double)(k.k_offset > k.v_offset ? k.k_offset : k.v_offset) + block;
  const double end = (double)k.s_offset + scales > off ? (double)k.s_offset + scales : off;
  if ((double)(k.n_pages - 1) * (double)k.page_bytes + end > (double)k.pool_bytes) return CBT_ERR_INVALID;
  *out = PagedKvFp8{static_cast<uint8_t*>(k.pool), (long long)k.pool_bytes, k.page_bytes, k.k_offset, k.v_offset,
                    k.s_offset, k.n_pages, k.page_tokens, k.n_kv_heads, k.head_dim};
  return CBT_OK;
}

bool rope_ok(const cbt_rope& r, int head_dim) {
  return (r.layout == CBT_ROPE_HALF || r.layout == CBT_ROPE_INTERLEAVED) && r.head_dim == head_dim &&
         r.rot_dim >= 2 && r.rot_dim <= head_dim && r.rot_dim % 2 == 0;
}

// the sizes of an attention call, without its pointers
template <class Args>
cbt_status attn_sizes(const Args& a) {
  if (a.kv.head_dim != 64 && a.kv.head_dim != 128) return CBT_ERR_UNSUPPORTED;
  if (a.rows < 0 || a.tokens < 0 || a.max_pages <= 0 || a.max_q <= 0 || a.max_kv < 0 ||
      a.n_heads <= 0 || a.kv.n_kv_heads <= 0 || a.n_heads % a.kv.n_kv_heads || a.window < 0 ||
      a.sinks < 0 || !(fabsf(a.scale) <= 3.4e38f) || a.kv.page_tokens <= 0 ||
      a.kv.page_tokens % 64 || (a.out_dtype != CBT_DTYPE_BF16 && a.out_dtype != CBT_DTYPE_F32))
    return CBT_ERR_INVALID;
  if (a.n_heads / a.kv.n_kv_heads > 64) return CBT_ERR_UNSUPPORTED;
  if (a.rows > CBT_PAGED_ATTENTION_MAX_ROWS || (int64_t)a.max_kv + a.window > INT32_MAX ||
      (int64_t)a.max_kv + a.sinks > INT32_MAX ||
      (int64_t)a.n_heads * a.kv.head_dim > INT32_MAX / 4 ||
      // work items and grid dimensions stay below 2^31; one token per row: an item for every 128 keys
      ((double)a.rows + a.tokens) * a.n_heads >= (double)(1 << 29) ||
      (a.max_q == 1 &&
       ((double)a.rows + a.tokens) * a.n_heads * (a.max_kv / 128.0 + 2) > (double)INT32_MAX))
    return CBT_ERR_LIMIT;
  return CBT_OK;
}

template <class Args, class Kv>
PagedAttnOn<Kv> attn_args(const Args& a, const Kv& kv) {
  PagedAttnOn<Kv> p{};
  p.kv = kv;
  p.table = a.block_table;
  p.max_pages = a.max_pages;
  p.rows = a.rows;
  p.lens = a.kv_lens;
  p.cu = a.cu_q;
  p.tokens = a.tokens;
  p.max_q = a.max_q;
  p.max_kv = a.max_kv;
  p.n_heads = a.n_heads;
  p.q = static_cast<const uint16_t*>(a.q);
  p.q_ld = a.q_stride;
  p.scale = a.scale;
  p.window = a.window;
  p.sinks = a.sinks;
  p.out = a.out;
  p.f32 = a.out_dtype == CBT_DTYPE_F32;
  p.out_ld = a.out_stride;
  p.ws = static_cast<uint8_t*>(a.workspace);
  p.ws_bytes = a.workspace_bytes;
  p.err = a.err;
  return p;
}

// SMs of the current device
cudaError_t sm_count(int* n) {
  int dev = 0;
  const cudaError_t rc = cudaGetDevice(&dev);
  return rc == cudaSuccess ? cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev) : rc;
}

// an append's checks, then its launch
template <class Kv, class Args>
cbt_status rope_append(const Args* a, cudaError_t (*launch)(const RopeAppendOn<Kv>&, cudaStream_t), void* stream) {
  if (!a) return CBT_ERR_NULL;
  RopeAppendOn<Kv> p{};
  const cbt_status st = paged_kv(a->kv, &p.kv);
  if (st != CBT_OK) return st;
  const int hd = a->kv.head_dim;
  const int64_t width = ((int64_t)a->n_heads + 2 * (int64_t)a->kv.n_kv_heads) * hd;
  if (a->tokens < 0 || a->n_heads <= 0 || !(a->eps >= 0.f) || !(a->eps <= 3.4e38f) ||
      (a->qkv_dtype != CBT_DTYPE_BF16 && a->qkv_dtype != CBT_DTYPE_F32) || a->qkv_stride < width ||
      a->qkv_stride % 8 || a->q_stride < (int64_t)a->n_heads * hd || a->q_stride % 8 ||
      (a->rope && !rope_ok(*a->rope, hd)))
    return CBT_ERR_INVALID;
  // 65535: the launch's limit on its second grid dimension, far above any head count in use
  if (a->tokens > kMostTokens || width > INT32_MAX / 4 || (int64_t)a->n_heads + 2 * (int64_t)a->kv.n_kv_heads > 65535)
    return CBT_ERR_LIMIT;
  if (a->tokens == 0) return CBT_OK;
  if (!a->qkv || !a->q_out || !a->positions || !a->slots || !a->err) return CBT_ERR_NULL;
  if (!aligned(a->qkv, 16) || !aligned(a->q_out, 16) || !aligned(a->q_gain, 16) ||
      !aligned(a->k_gain, 16))
    return CBT_ERR_INVALID;
  if (a->rope) p.rope = *a->rope;
  p.qkv = a->qkv;
  p.f32 = a->qkv_dtype == CBT_DTYPE_F32;
  p.qkv_ld = a->qkv_stride;
  p.tokens = a->tokens;
  p.n_heads = a->n_heads;
  p.q_gain = static_cast<const uint16_t*>(a->q_gain);
  p.k_gain = static_cast<const uint16_t*>(a->k_gain);
  p.eps = a->eps;
  p.positions = a->positions;
  p.slots = a->slots;
  p.q_out = static_cast<uint16_t*>(a->q_out);
  p.q_ld = a->q_stride;
  p.err = a->err;
  return launch(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? CBT_OK : CBT_ERR_CUDA;
}

template <class Kv, class Args>
size_t attn_workspace(const Args* a, size_t (*need)(const PagedAttnOn<Kv>&)) {
  if (!a || attn_sizes(*a) != CBT_OK) return 0;
  Kv kv{};
  kv.n_pages = a->kv.n_pages;
  kv.page_tokens = a->kv.page_tokens;
  kv.n_kv_heads = a->kv.n_kv_heads;
  kv.head_dim = a->kv.head_dim;
  return need(attn_args(*a, kv));
}

// an attention's checks, then its launch
template <class Kv, class Args>
cbt_status attention(const Args* a, size_t (*workspace)(const PagedAttnOn<Kv>&),
                     cudaError_t (*launch)(const PagedAttnOn<Kv>&, int, cudaStream_t), void* stream) {
  if (!a) return CBT_ERR_NULL;
  Kv kv{};
  cbt_status st = paged_kv(a->kv, &kv);
  if (st == CBT_OK) st = attn_sizes(*a);
  if (st != CBT_OK) return st;
  const int64_t width = (int64_t)a->n_heads * a->kv.head_dim;
  if (a->q_stride < width || a->q_stride % 8 || a->out_stride < width || a->out_stride % 8 ||
      (!a->cu_q && (a->tokens != a->rows || a->max_q != 1)))
    return CBT_ERR_INVALID;
  if (a->rows == 0 || a->tokens == 0) return CBT_OK;
  if (!a->q || !a->out || !a->block_table || !a->kv_lens || !a->err) return CBT_ERR_NULL;
  if (!aligned(a->q, 16) || !aligned(a->out, 16)) return CBT_ERR_INVALID;
  const PagedAttnOn<Kv> p = attn_args(*a, kv);
  const size_t need = workspace(p);
  if (need && !a->workspace) return CBT_ERR_NULL;
  if (need > a->workspace_bytes || !aligned(a->workspace, 256)) return CBT_ERR_INVALID;
  int num_sms = 0;
  if (sm_count(&num_sms) != cudaSuccess) return CBT_ERR_CUDA;
  return launch(p, num_sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? CBT_OK : CBT_ERR_CUDA;
}

}  // namespace

size_t paged_attn_workspace(const PagedAttn& a) {
  return a.max_q == 1 ? paged_decode_workspace(a) : paged_prefill_workspace(a);
}

cudaError_t launch_paged_attn(const PagedAttn& a, int num_sms, cudaStream_t s) {
  if (paged_attn_workspace(a) > a.ws_bytes) return cudaErrorInvalidValue;
  return a.max_q > 1 ? launch_paged_prefill(a, num_sms, s) : launch_paged_decode(a, num_sms, s);
}

size_t attn_fp8_workspace(const PagedAttnFp8& a) {
  return a.max_q == 1 ? decode_fp8_workspace(a) : prefill_fp8_workspace(a);
}

cudaError_t launch_attn_fp8(const PagedAttnFp8& a, int num_sms, cudaStream_t s) {
  if (attn_fp8_workspace(a) > a.ws_bytes) return cudaErrorInvalidValue;
  return a.max_q > 1 ? launch_prefill_fp8(a, num_sms, s) : launch_decode_fp8(a, num_sms, s);
}

extern "C" cbt_status cbt_page_map(const cbt_page_map_args* a, void* stream) {
  if (!a) return CBT_ERR_NULL;
  if (a->rows < 0 || a->max_pages <= 0 || a->page_tokens <= 0 || a->n_pages <= 0 || a->max_tokens < 0)
    return CBT_ERR_INVALID;
  if (a->rows > CBT_PAGE_MAP_MAX_ROWS || (int64_t)a->max_pages * a->page_tokens > INT32_MAX ||
      (int64_t)a->n_pages * a->page_tokens > INT32_MAX ||
      a->max_tokens > kMostTokens || a->n_pages > kMostTokens)
    return CBT_ERR_LIMIT;
  if (a->rows == 0) return CBT_OK;
  if (!a->block_table || !a->kv_lens || !a->new_lens || !a->kv_lens_out || !a->cu_q || !a->err ||
      (a->max_tokens && (!a->positions || !a->slots)) ||
      (a->free_pages && (!a->free_count || !a->free_count_out)))
    return CBT_ERR_NULL;
  return launch_page_map(*a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? CBT_OK : CBT_ERR_CUDA;
}

extern "C" cbt_status cbt_rope_init(const cbt_rope_config* c, int32_t head_dim, cbt_rope* out) {
  if (!c || !out) return CBT_ERR_NULL;
  double fast = c->beta_fast, slow = c->beta_slow;
  if (fast == 0 && slow == 0) {
    fast = 32;
    slow = 1;
  }
  if ((head_dim != 64 && head_dim != 128) || c->rot_dim < 2 || c->rot_dim > head_dim ||
      c->rot_dim % 2 || (c->layout != CBT_ROPE_HALF && c->layout != CBT_ROPE_INTERLEAVED) ||
      c->scaling < CBT_ROPE_NONE || c->scaling > CBT_ROPE_BY_PARTS || !(c->theta > 1) ||
      !(c->theta <= 1e300) || !(c->mscale >= 0) || !(c->mscale <= 1e30) ||
      (c->scaling != CBT_ROPE_NONE && (!(c->factor >= 1) || !(c->factor <= 1e9))) ||
      (c->scaling == CBT_ROPE_BY_PARTS &&
       (c->original_len <= 0 || !(slow > 0) || !(fast > slow) || !(fast <= 1e30))))
    return CBT_ERR_INVALID;
  const double kPi = 3.14159265358979323846;
  const int rot = c->rot_dim, half = rot / 2;
  const double s = c->scaling == CBT_ROPE_NONE ? 1.0 : c->factor;
  double theta = c->theta;
  if (c->scaling == CBT_ROPE_BASE && rot > 2) theta *= pow(s, (double)rot / (rot - 2));
  double lo = 0, hi = 1;
  if (c->scaling == CBT_ROPE_BY_PARTS) {
    lo = fmax(0.0, floor(rot * log(c->original_len / (fast * 2 * kPi)) / (2 * log(theta))));
    hi = fmin(rot - 1.0, ceil(rot * log(c->original_len / (slow * 2 * kPi)) / (2 * log(theta))));
    if (!(hi > lo)) hi = lo + 0.001;
  }
  cbt_rope r{};
  for (int i = 0; i < half; ++i) {
    double f = pow(theta, -2.0 * i / rot);
    if (c->scaling == CBT_ROPE_LINEAR) f /= s;
    if (c->scaling == CBT_ROPE_BY_PARTS) {
      const double ramp = fmin(1.0, fmax(0.0, (i - lo) / (hi - lo)));
      f = f / s * ramp + f * (1 - ramp);
    }
    // f <= 1 radian, so under a sixth of a turn: in range for the conversion
    r.turns[i] = (uint64_t)ldexp(f / (2 * kPi), 64);
  }
  const double own = c->scaling == CBT_ROPE_BY_PARTS && s > 1 ? 0.1 * log(s) + 1 : 1.0;
  r.mscale = (float)(c->mscale > 0 ? c->mscale : own);
  r.layout = c->layout;
  r.rot_dim = rot;
  r.head_dim = head_dim;
  *out = r;
  return CBT_OK;
}

extern "C" cbt_status cbt_rope_append(const cbt_rope_append_args* a, void* stream) {
  return rope_append(a, launch_paged_rope, stream);
}
extern "C" cbt_status cbt_rope_append_fp8(const cbt_rope_append_fp8_args* a, void* stream) {
  return rope_append(a, launch_append_fp8, stream);
}

extern "C" size_t cbt_paged_attention_workspace(const cbt_paged_attention_args* a) {
  return attn_workspace(a, paged_attn_workspace);
}
extern "C" size_t cbt_paged_attention_fp8_workspace(const cbt_paged_attention_fp8_args* a) {
  return attn_workspace(a, attn_fp8_workspace);
}

extern "C" cbt_status cbt_paged_attention(const cbt_paged_attention_args* a, void* stream) {
  return attention(a, paged_attn_workspace, launch_paged_attn, stream);
}
extern "C" cbt_status cbt_paged_attention_fp8(const cbt_paged_attention_fp8_args* a, void* stream) {
  return attention(a, attn_fp8_workspace, launch_attn_fp8, stream);
}

extern "C" cbt_status cbt_paged_read_fp8(const cbt_paged_read_fp8_args* a, void* stream) {
  if (!a) return CBT_ERR_NULL;
  PagedReadFp8 p{};
  const cbt_status st = paged_kv(a->kv, &p.kv);
  if (st != CBT_OK) return st;
  const int64_t width = (int64_t)a->kv.n_kv_heads * a->kv.head_dim;
  if (a->rows < 0 || a->tokens < 0 || a->max_pages <= 0 || a->out_stride < width || a->out_stride % 8 ||
      (a->out_dtype != CBT_DTYPE_BF16 && a->out_dtype != CBT_DTYPE_F32))
    return CBT_ERR_INVALID;
  // 32767: the launch's limit on its second grid dimension, K's heads and V's
  if (a->rows > CBT_PAGED_ATTENTION_MAX_ROWS || a->tokens > kMostTokens || a->kv.n_kv_heads > 32767)
    return CBT_ERR_LIMIT;
  if (a->rows == 0 || a->tokens == 0 || (!a->k_out && !a->v_out)) return CBT_OK;
  if (!a->block_table || !a->kv_lens || !a->cu || !a->err) return CBT_ERR_NULL;
  if (!aligned(a->k_out, 16) || !aligned(a->v_out, 16)) return CBT_ERR_INVALID;
  p.table = a->block_table;
  p.max_pages = a->max_pages;
  p.rows = a->rows;
  p.lens = a->kv_lens;
  p.first = a->first;
  p.cu = a->cu;
  p.tokens = a->tokens;
  p.k_out = a->k_out;
  p.v_out = a->v_out;
  p.f32 = a->out_dtype == CBT_DTYPE_F32;
  p.out_ld = a->out_stride;
  p.err = a->err;
  return launch_read_fp8(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? CBT_OK : CBT_ERR_CUDA;
}
