// paged_rope.cu -- per-head RMS norm, rotary positions and the append of K and V to a paged cache,
// one pass over QKV rows.
//
// Every element is read once and written once as bf16: HBM is the floor.  8192 tokens of 32 q and 8
// kv heads of 128 take 39.4 us = 5.1 TB/s, three quarters of the measured copy rate; 8 tokens of them
// 3.4 us; 777 tokens of 12 and 4 heads of 64 5.1 us.  What keeps it from the rest is each token's
// chain (load, norm's reductions, store) over the warps that fit: issue slots are 72 % taken, yet a
// form with a fifth fewer instructions (gains held, two products an instruction) took 41 us, its
// registers having cost warps.  Two kinds of block share a launch:
// - q and k: a warp takes one token and a run of its heads.  A head is spread over head_dim / 8
//   lanes, each with two groups of four dims chosen so that both members of its rotated pairs are
//   its own (half layout: dims 4l.. of the first and of the second half), so the rotation needs no
//   exchange; the angles are formed once per token and kept in registers over its heads.
// - v: its cache layout runs along the positions of a dim, so 128 tokens of one head are turned
//   around in shared memory and written as whole 16-byte runs of 8 positions wherever 8 tokens
//   fill an aligned run of slots, wherever in the tile that run starts.
// Angles: position * turns[i] modulo 2^64 is the fraction of a turn, exact for any position; its
// top 32 bits become an fp32 angle in [-pi, pi) for the hardware's sine and cosine, which are off by
// some 2^-21 there: small next to the 2^-9 that the results are rounded by.
#include "paged.h"

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kVTokens = 128;  // tokens of a v tile
constexpr int kUnroll = 2;     // heads (or pairs of heads) in flight per warp
constexpr int kTargetWarps = 152 * 32;  // warps that fill the SMs

enum Mode { kNone, kHalf, kHalfOdd, kInter };  // kHalfOdd: rot_dim not a multiple of 8

// four elements of a row as they lie there
template <bool F32>
struct Four {
  float4 v;
  CBT_D void load(const void* p, long long i) {
    v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i));
  }
  CBT_D void to(float* x) const {
    x[0] = v.x;
    x[1] = v.y;
    x[2] = v.z;
    x[3] = v.w;
  }
};
template <>
struct Four<false> {
  uint2 v;
  CBT_D void load(const void* p, long long i) {
    v = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i));
  }
  CBT_D void to(float* x) const {
    x[0] = bf16_lo(v.x);
    x[1] = bf16_hi(v.x);
    x[2] = bf16_lo(v.y);
    x[3] = bf16_hi(v.y);
  }
};
template <bool F32>
CBT_D void load4(const void* p, long long i, float* x) {
  Four<F32> f;
  f.load(p, i);
  f.to(x);
}
CBT_D uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
CBT_D void store4(uint16_t* p, const float* x) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack2(x[0], x[1]), pack2(x[2], x[3]));
}

CBT_D bool slot_ok(const RopeAppend& a, int slot, int pos) {
  return slot >= 0 && pos >= 0 && slot < a.kv.n_pages * a.kv.page_tokens;
}

// q and k heads [h0, h1) of one token, by one warp
template <int HD, bool F32, int MODE>
CBT_D void rotate_heads(const RopeAppend& a, int t, int h0, int h1, float* xs) {
  constexpr int LPH = HD / 8, NH = 32 / LPH;  // lanes per head, heads per warp step
  constexpr int kAngles = MODE == kHalfOdd ? 8 : 4;
  const int lane = threadIdx.x & 31, l = lane % LPH, sub = lane / LPH;
  const int rot = a.rope.rot_dim, half = rot / 2;
  // this lane's dims: four from e0, four from e1; its first `turned` pairs are rotated
  int e0 = 8 * l, e1 = 8 * l + 4, turned = MODE == kInter ? half - 4 * l : 0;
  if (MODE == kHalf && l < rot / 8) {
    e0 = 4 * l;
    e1 = half + 4 * l;
    turned = 4;
  }
  const long long src = t * a.qkv_ld;
  Four<F32> in[kUnroll][2];
  auto load = [&](int hb) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long long at = src + min(hb + u * NH + sub, h1 - 1) * HD;  // the last head again past the end
      in[u][0].load(a.qkv, at + e0);
      in[u][1].load(a.qkv, at + e1);
    }
  };
  load(h0);
  const int slot = a.slots[t], pos = a.positions[t];
  if (!slot_ok(a, slot, pos)) {
    if (lane == 0 && h0 == 0 && slot >= 0 && pos >= 0) set_device_error(a.err, CBT_DEV_PAGE_ID, t);
    return;
  }
  // this lane's i-th pair (kHalfOdd: the pair of its i-th dim) is turned by (cs[i], sn[i])
  float cs[kAngles], sn[kAngles];
#pragma unroll
  for (int i = 0; i < (MODE == kNone ? 0 : kAngles); ++i) {
    int pair = 4 * l + i;
    bool on = i < turned;
    if (MODE == kHalfOdd) {
      const int d = 8 * l + i;
      on = d < rot;
      pair = d < half ? d : d - half;
    }
    float c = 1.f, s = 0.f;
    // the lanes of the NH heads form a share of the angles each and pass them on
    if (on && (MODE == kHalfOdd || i % NH == sub)) {
      const uint64_t ph = (uint64_t)pos * a.rope.turns[pair];
      const float rad = (float)(int32_t)(ph >> 32) * 0x1.921fb6p-30f;  // pi / 2^31
      __sincosf(rad, &s, &c);
      s *= a.rope.mscale;
      c *= a.rope.mscale;
    }
    if (MODE != kHalfOdd) {
      c = __shfl_sync(0xffffffffu, c, (i % NH) * LPH + l);
      s = __shfl_sync(0xffffffffu, s, (i % NH) * LPH + l);
    }
    cs[i] = c;
    sn[i] = s;
  }
  const int page = a.kv.page_tokens, id = slot / page, o = slot - id * page, H = a.n_heads;
  uint16_t* qdst = a.q_out + t * a.q_ld;
  uint16_t* kdst = a.kv.pool + paged_k(a.kv, id, 0, o, 0);
  const bool norm = a.q_gain || a.k_gain;
  for (int hb = h0; hb < h1; hb += NH * kUnroll) {
    Four<F32> now[kUnroll][2];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      now[u][0] = in[u][0];
      now[u][1] = in[u][1];
    }
    if (hb + NH * kUnroll < h1) load(hb + NH * kUnroll);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = hb + u * NH + sub;
      float x[8];
      now[u][0].to(x);
      now[u][1].to(x + 4);
      if (norm) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(x[i], x[i], s);
#pragma unroll
        for (int w = LPH / 2; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
        const uint16_t* gain = h < H ? a.q_gain : a.k_gain;
        if (gain) {
          const float r = rsqrtf(s * (1.f / HD) + a.eps);
          float g[8];
          load4<false>(gain, e0, g);
          load4<false>(gain, e1, g + 4);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = x[i] * r * g[i];
        }
      }
      if (MODE == kHalf || MODE == kInter) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float& p = MODE == kHalf ? x[i] : x[2 * i];
          float& q = MODE == kHalf ? x[4 + i] : x[2 * i + 1];
          if (i < turned) {
            const float y = fmaf(p, cs[i], -q * sn[i]);
            q = fmaf(q, cs[i], p * sn[i]);
            p = y;
          }
        }
      } else if (MODE == kHalfOdd) {  // the other member of a pair lies with any lane
        float* hx = xs + sub * HD;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) hx[8 * l + i] = x[i];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int d = 8 * l + i;
          if (d < half) x[i] = fmaf(x[i], cs[i], -hx[d + half] * sn[i]);
          else if (d < rot) x[i] = fmaf(x[i], cs[i], hx[d - half] * sn[i]);
        }
      }
      if (h < h1) {
        uint16_t* to = h < H ? qdst + h * HD : kdst + (long long)(h - H) * page * HD;
        store4(to + e0, x);
        store4(to + e1, x + 4);
      }
    }
  }
}

// v of tokens [t0, t0 + 128) of kv head g, by the block
template <int HD, bool F32>
CBT_D void append_v(const RopeAppend& a, int t0, int g, uint8_t* sm) {
  constexpr int kRow = HD + 2;  // padded: a column of tokens falls into different banks
  uint16_t* tile = reinterpret_cast<uint16_t*>(sm);
  int* slots = reinterpret_cast<int*>(sm + kVTokens * kRow * 2);  // [128], -1: skipped
  int* runs = slots + kVTokens;                                   // first token and length of each run
  __shared__ int n_runs[5];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid < kVTokens) {
    const int t = t0 + tid;
    int s = -1;
    if (t < a.tokens) {
      s = a.slots[t];
      if (!slot_ok(a, s, a.positions[t])) s = -1;
    }
    slots[tid] = s;
  }
  const long long src = (long long)(a.n_heads + a.kv.n_kv_heads + g) * HD;
#pragma unroll 8
  for (int i = tid; i < kVTokens * HD / 8; i += kThreads) {
    const int r = i / (HD / 8), d = (i % (HD / 8)) * 8;
    if (t0 + r < a.tokens) {
      uint4 v;
      const long long at = (t0 + r) * a.qkv_ld + src + d;
      if (F32) {
        float x[8];
        load4<F32>(a.qkv, at, x);
        load4<F32>(a.qkv, at + 4, x + 4);
        v = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
      } else {
        v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.qkv) + at));
      }
      uint32_t* dst = reinterpret_cast<uint32_t*>(tile + r * kRow + d);
      dst[0] = v.x;
      dst[1] = v.y;
      dst[2] = v.z;
      dst[3] = v.w;
    }
  }
  __syncthreads();
  // runs of tokens in consecutive slots of one aligned group of 8
  bool first = false;
  int len = 0;
  if (tid < kVTokens) {
    const int s = slots[tid];
    first = s >= 0 && (tid == 0 || s % 8 == 0 || slots[tid - 1] != s - 1);
    if (first) {
      len = 1;
      while (tid + len < kVTokens && (s + len) % 8 && slots[tid + len] == s + len) ++len;
    }
  }
  const unsigned m = __ballot_sync(0xffffffffu, first);
  if (warp < 4 && lane == 0) n_runs[warp] = __popc(m);
  __syncthreads();
  if (first) {
    int at = __popc(m & ((1u << lane) - 1));
    for (int w = 0; w < warp; ++w) at += n_runs[w];
    runs[at] = tid | (len << 16);
  }
  const int total = n_runs[0] + n_runs[1] + n_runs[2] + n_runs[3];
  __syncthreads();
  // 8 runs x 4 pairs of dims per warp: a warp's 16-byte stores fill whole 128-byte lines
  constexpr int kPairs = HD / 2;
  const int page = a.kv.page_tokens;
  const int ru = lane & 7, dp = lane >> 3;
  for (int w = warp; w < (total + 7) / 8 * (kPairs / 4); w += kWarps) {
    const int r = (w / (kPairs / 4)) * 8 + ru, d = 2 * ((w % (kPairs / 4)) * 4 + dp);
    if (r >= total) continue;
    const int k = runs[r] & 0xFFFF, n = runs[r] >> 16;
    const int s = slots[k], id = s / page, o = s - id * page;
    uint16_t* dst = a.kv.pool + paged_v(a.kv, id, g, o, d);
    if (n == 8) {
      uint32_t v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = *reinterpret_cast<const uint32_t*>(tile + (k + j) * kRow + d);
      uint4 lo, hi;
      lo.x = __byte_perm(v[0], v[1], 0x5410);
      lo.y = __byte_perm(v[2], v[3], 0x5410);
      lo.z = __byte_perm(v[4], v[5], 0x5410);
      lo.w = __byte_perm(v[6], v[7], 0x5410);
      hi.x = __byte_perm(v[0], v[1], 0x7632);
      hi.y = __byte_perm(v[2], v[3], 0x7632);
      hi.z = __byte_perm(v[4], v[5], 0x7632);
      hi.w = __byte_perm(v[6], v[7], 0x7632);
      *reinterpret_cast<uint4*>(dst) = lo;
      *reinterpret_cast<uint4*>(dst + 64) = hi;
    } else {
      for (int j = 0; j < n; ++j) {
        const uint32_t v = *reinterpret_cast<const uint32_t*>(tile + (k + j) * kRow + d);
        dst[j] = (uint16_t)v;
        dst[64 + j] = (uint16_t)(v >> 16);
      }
    }
  }
}

// Blocks [0, qk_blocks): warps over (token, run of `per` q and k heads), `runs` of them a token; then
// one block per (128 tokens, kv head) for v.
template <int HD, bool F32, int MODE>
__global__ void __launch_bounds__(kThreads, F32 ? 3 : 5)
    k_rope_append(const __grid_constant__ RopeAppend a, int qk_blocks, int runs, int per) {
  extern __shared__ __align__(16) uint8_t sm[];
  pdl_wait();
  if ((int)blockIdx.x < qk_blocks) {
    const int warp = threadIdx.x >> 5;
    const long long w = (long long)blockIdx.x * kWarps + warp;
    const int t = (int)(w / runs), h0 = (int)(w - (long long)t * runs) * per;
    const int heads = a.n_heads + a.kv.n_kv_heads;
    if (t < a.tokens && h0 < heads)
      rotate_heads<HD, F32, MODE>(a, t, h0, min(heads, h0 + per),
                                  reinterpret_cast<float*>(sm) + warp * 256);
  } else {
    const int b = blockIdx.x - qk_blocks;
    append_v<HD, F32>(a, b / a.kv.n_kv_heads * kVTokens, b % a.kv.n_kv_heads, sm);
  }
  pdl_launch();
}

template <int HD, bool F32, int MODE>
cudaError_t launch(const RopeAppend& a, cudaStream_t s) {
  constexpr int kStep = 32 / (HD / 8) * kUnroll;  // heads a warp has in flight
  constexpr size_t smem = kVTokens * (HD + 2) * 2 + 2 * kVTokens * sizeof(int);
  static_assert(smem >= kWarps * 256 * sizeof(float) && smem <= 48 * 1024, "shared memory");
  // A token's heads are split over more warps only while tokens alone would leave the SMs idle: the
  // angles are formed again by every warp that takes some of them (8192 tokens of 32 + 8 heads: 40
  // us in one run a token, 45 in two).
  const int heads = a.n_heads + a.kv.n_kv_heads, steps = (heads + kStep - 1) / kStep;
  int runs = (kTargetWarps + a.tokens - 1) / a.tokens;
  runs = runs < steps ? runs : steps;
  const int per = (steps + runs - 1) / runs * kStep;
  runs = (heads + per - 1) / per;
  const long long qk = ((long long)a.tokens * runs + kWarps - 1) / kWarps;
  const long long v = (long long)((a.tokens + kVTokens - 1) / kVTokens) * a.kv.n_kv_heads;
  if (qk + v > 0x7FFFFFFF) return cudaErrorInvalidValue;
  return launch_pdl(k_rope_append<HD, F32, MODE>, dim3((unsigned)(qk + v)), dim3(kThreads), smem, s, a,
                    (int)qk, runs, per);
}

template <int HD, bool F32>
cudaError_t launch_mode(const RopeAppend& a, cudaStream_t s) {
  if (a.rope.rot_dim == 0) return launch<HD, F32, kNone>(a, s);
  if (a.rope.layout == CBT_ROPE_INTERLEAVED) return launch<HD, F32, kInter>(a, s);
  return a.rope.rot_dim % 8 ? launch<HD, F32, kHalfOdd>(a, s) : launch<HD, F32, kHalf>(a, s);
}

}  // namespace

cudaError_t launch_paged_rope(const RopeAppend& a, cudaStream_t s) {
  if (a.kv.head_dim == 128) return a.f32 ? launch_mode<128, true>(a, s) : launch_mode<128, false>(a, s);
  return a.f32 ? launch_mode<64, true>(a, s) : launch_mode<64, false>(a, s);
}
