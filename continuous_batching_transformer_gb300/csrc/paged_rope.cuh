// paged_rope.cuh -- per-head norm and rotary positions of QKV rows: what the appends to a bf16 and to an
// 8-bit paged cache share.
#pragma once
#include <type_traits>

#include "paged.h"

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
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

template <class Kv>
CBT_D bool slot_ok(const RopeAppendOn<Kv>& a, int slot, int pos) {
  return slot >= 0 && pos >= 0 && slot < a.kv.n_pages * a.kv.page_tokens;
}

// The dims of lane l of a head's HD / 8 lanes: four from e0, four from e1, of which the first `turned`
// pairs are rotated.  Both members of a pair are one lane's (but for kHalfOdd).
struct LaneDims {
  int e0, e1, turned;
};
template <int MODE>
CBT_D LaneDims lane_dims(int l, int rot) {
  LaneDims d{8 * l, 8 * l + 4, MODE == kInter ? rot / 2 - 4 * l : 0};
  if (MODE == kHalf && l < rot / 8) {
    d.e0 = 4 * l;
    d.e1 = rot / 2 + 4 * l;
    d.turned = 4;
  }
  return d;
}
// sum of squares of a head, over its lanes
template <int HD>
CBT_D float head_squares(const float (&x)[8]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(x[i], x[i], s);
#pragma unroll
  for (int w = HD / 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
  return s;
}
template <int HD>
CBT_D void scale_head(float (&x)[8], float squares, float eps, const float (&g)[8]) {
  const float r = rsqrtf(squares * (1.f / HD) + eps);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = x[i] * r * g[i];
}
CBT_D void load_gain(const uint16_t* gain, const LaneDims& d, float (&g)[8]) {
  load4<false>(gain, d.e0, g);
  load4<false>(gain, d.e1, g + 4);
}
// turns a head's pairs; kHalfOdd exchanges through hx, HD floats of shared memory of the head's own
template <int HD, int MODE>
CBT_D void turn_head(float (&x)[8], const float* cs, const float* sn, int l, int turned, int rot, float* hx) {
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
    const int half = rot / 2;
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
}
// where k of head 0 goes; a cache in 8 bits has its own way
CBT_D uint16_t* k_row(const RopeAppend& a, int id, int o) { return a.kv.pool + paged_k(a.kv, id, 0, o, 0); }
template <class A>
CBT_D uint16_t* k_row(const A&, int, int) { return nullptr; }

// q and k heads [h0, h1) of one token, by one warp (k heads of a bf16 cache alone)
template <int HD, bool F32, int MODE, class A>
CBT_D void rotate_heads(const A& a, int t, int h0, int h1, float* xs) {
  constexpr int LPH = HD / 8, NH = 32 / LPH;  // lanes per head, heads per warp step
  constexpr int kAngles = MODE == kHalfOdd ? 8 : 4;
  const int lane = threadIdx.x & 31, l = lane % LPH, sub = lane / LPH;
  const int rot = a.rope.rot_dim, half = rot / 2;
  const LaneDims dims = lane_dims<MODE>(l, rot);
  const int e0 = dims.e0, e1 = dims.e1, turned = dims.turned;
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
  uint16_t* kdst = k_row(a, id, o);
  // One gain for all heads is held; two take their turns (held, their registers cost more than the loads:
  // 41 us for 39.4 in the append to bf16 pages).
  constexpr bool kQOnly = !std::is_same<A, RopeAppend>::value;
  const bool norm = a.q_gain || (!kQOnly && a.k_gain);
  float g[8];
  if (kQOnly && a.q_gain) load_gain(a.q_gain, dims, g);
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
        const float s = head_squares<HD>(x);
        const uint16_t* gain = h < H ? a.q_gain : a.k_gain;
        if (gain) {
          if (!kQOnly) load_gain(gain, dims, g);
          scale_head<HD>(x, s, a.eps, g);
        }
      }
      turn_head<HD, MODE>(x, cs, sn, l, turned, rot, xs + sub * HD);
      if (h < h1) {
        uint16_t* to = h < H ? qdst + h * HD : kdst + (long long)(h - H) * page * HD;
        store4(to + e0, x);
        store4(to + e1, x + 4);
      }
    }
  }
}

}  // namespace
