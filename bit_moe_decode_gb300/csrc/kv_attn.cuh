// kv_attn.cuh -- what the two attention kernels over the 4-bit paged KV cache (kv_attn.cu, kv_attn_wide.cu) share.
#pragma once
#include <cfloat>

#include "kv.cuh"

namespace moe {
namespace kv {

constexpr int kSmemMax = 232448;
constexpr int kPExp = 12;               // weights are carried times 2^12
constexpr float kLazy = 2.f;            // a score may pass the running maximum by this (base 2)
constexpr float kHeavy = 0.25f, kLight = 0.000244140625f;   // 2^12 times 2^-14 and 2^-24

struct AttnArgs {
  const uint16_t* q;
  int64_t q_stride;
  int32_t q_heads, group, window, row_groups, stages;
  uint32_t group_inv;               // floor(row / group) = row * group_inv >> 16 for rows below 128
  int32_t rings;                    // bytes of the warps' rings; the tables follow
  float scale_log2;                 // scale * log2(e)
  uint16_t* out;
  float* lse;
  uint32_t* counters;               // [CTAs], by the CTA in which a pair begins that others go on with (one pair at most)
  float* warp_parts;                // [CTAs][warps] partials of runs that end inside a warp's range
  float* cta_parts;                 // [CTAs][2]
  uint32_t* redo;                   // [n_seqs] sequences that kv_attn_wide.cu leaves to kv_attn.cu, whether any, CTAs that know
};

__device__ __forceinline__ bool rarely(bool x) { return __builtin_expect(x, 0); }   // (keeps rare code out of the loop's lines)

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {   // NaN loses, as in fmaxf
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t hadd2_bits(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {   // (selector bit 3: the byte's sign fill)
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}
__device__ __forceinline__ uint32_t hmul2_bits(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], const uint8_t* p) {   // N = 1, 2 or 4 words
  if (N == 4) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[0] = u.x; w[1 % N] = u.y; w[2 % N] = u.z; w[3 % N] = u.w;
  } else if (N == 2) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x; w[1 % N] = u.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// the scales of one token's blocks in fp32
template <int FMT, int NB>
__device__ __forceinline__ void load_scales(float (&s)[NB], const uint8_t* p) {
  if (FMT == MOE_FMT_MXFP4) {   // 2^(e - 127), e = 0 is zero: the byte is the exponent field
    const uint32_t w = NB == 4 ? *reinterpret_cast<const uint32_t*>(p) : *reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const uint32_t v = b == 0 ? w << 23 : b == 1 ? w << 15 : b == 2 ? w << 7 : w >> 1;
      s[b] = __uint_as_float(b == 0 ? v & 0x7F800000u : v & 0x7F800000u);
    }
  } else {
    uint32_t w[NB / 2];
    load_words<NB / 2>(w, p);
#pragma unroll
    for (int b = 0; b < NB; ++b) s[b] = __uint_as_float(b & 1 ? w[b / 2] & 0xFFFF0000u : w[b / 2] << 16);
  }
}

struct SeqInfo { int q0, qn, len, sub0; };   // sub0: first sub-block that a row sees

// x * W / n without 64-bit division where it is not needed
__device__ __forceinline__ long long share(long long x, long long W, long long n) {
  const unsigned long long p = (unsigned long long)x * W;
  return p >> 32 ? (long long)(p / (unsigned long long)n) : (long long)((uint32_t)p / (uint32_t)n);
}

// The CTA whose share has place x of the list
__device__ __forceinline__ int first_cta(long long x, long long W, int G) { return (int)(((x + 1) * G - 1) / W); }

// A row's joined values of four dimensions, written out
template <int D>
__device__ __forceinline__ void write_row4(const AttnArgs& g, int64_t row, int d, float4 o, float m, float l) {
  const bool some = l > 0.f || l != l;
  const float inv = some ? 1.f / l : 0.f;
  const __nv_bfloat162 p = some ? __floats2bfloat162_rn(o.x * inv, o.y * inv) : __floats2bfloat162_rn(0.f, 0.f);
  const __nv_bfloat162 q = some ? __floats2bfloat162_rn(o.z * inv, o.w * inv) : __floats2bfloat162_rn(0.f, 0.f);
  *reinterpret_cast<uint2*>(g.out + row * D + d) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&p), *reinterpret_cast<const uint32_t*>(&q));
  if (g.lse && d == 0) g.lse[row] = some ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// Value scales of a sub-block's tokens t, t + 1 (t even, `p` their first) times 2^-E as binary16 pairs. Exponents outside
// E - 14 .. E + 1 show in `off` & kOff. A token whose bit of `drop` is set counts as 2^-14, whatever bytes it has.
template <int FMT>
constexpr uint32_t kOff = FMT == MOE_FMT_MXFP4 ? 0xF0F0F0F0u : 0xF800F800u;
template <int FMT, int NB, int NVC>
__device__ __forceinline__ void scale_pair(const uint8_t* p, const uint32_t (&vc)[NVC], uint32_t (&u)[NB], uint32_t& off,
                                           uint32_t drop) {
  if (FMT == MOE_FMT_MXFP4) {
    uint32_t w[NB / 2];                // NB = 4: a token each; NB = 2: two tokens
    load_words<NB / 2>(w, p);
    if (drop) {
      const uint32_t low = 0u - vc[0];
#pragma unroll
      for (int i = 0; i < NB / 2; ++i) {
        const uint32_t k = NB == 4 ? 0u - ((drop >> i) & 1u) : ((drop & 1u) * 0xFFFFu) | ((drop >> 1 & 1u) * 0xFFFF0000u);
        w[i] = (w[i] & ~k) | (low & k);
      }
    }
    const uint32_t vc4 = vc[0] * 4u + 0x04040404u;
#pragma unroll
    for (int i = 0; i < NB / 2; ++i) {
      // bytes e - E + 14: 0 .. 15 in the window (8 bits: nothing aliases; a borrow comes from a byte that shows itself).
      // 4 (that + 1) is the high byte of binary16's 2^(e - E).
      off |= w[i] + vc[0];
      w[i] = w[i] * 4u + vc4;
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      // bytes (the sign fill of a byte below 128: 0; token t's; 0; token t + 1's)
      const int t = NB == 4 ? 4 + b : 2 + b;
      const uint32_t sel = (8u | b) | (uint32_t)b << 4 | (8u | t) << 8 | (uint32_t)t << 12;
      u[b] = prmt(w[0], w[NB / 2 - 1], sel);
    }
  } else {
    // bf16 and binary16 differ in the exponent's width and bias: (bits - ((E + 113) << 7) + (1 << 7)) << 3
    uint32_t w[NB];
    load_words<NB>(w, p);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      u[b] = prmt(w[b / 2], w[NB / 2 + b / 2], b & 1 ? 0x7632u : 0x5410u);
      if (drop) {
        const uint32_t k = ((drop & 1u) * 0xFFFFu) | ((drop >> 1 & 1u) * 0xFFFF0000u);
        u[b] = (u[b] & ~k) | ((0u - vc[b % NVC]) & k);
      }
      off |= u[b] + vc[b % NVC];
      u[b] = u[b] * 8u + (vc[b % NVC] * 8u + 0x04000400u);
    }
  }
}
// the same for tokens 2 c, 2 c + 1 (u0) and 2 c + 8, 2 c + 9 (u1)
template <int FMT, int NB, int NVC>
__device__ __forceinline__ void scale_pairs(const uint8_t* scales, int c, const uint32_t (&vc)[NVC], uint32_t (&u0)[NB],
                                            uint32_t (&u1)[NB], uint32_t& off, uint32_t drop) {
  constexpr int TOKEN = NB * (FMT == MOE_FMT_MXFP4 ? 1 : 2);
  scale_pair<FMT, NB, NVC>(scales + 2 * c * TOKEN, vc, u0, off, drop & 3u);
  scale_pair<FMT, NB, NVC>(scales + (2 * c + 8) * TOKEN, vc, u1, off, drop >> 2);
}

// Many query rows of a KV head over long sequences (kv_attn_wide.cu); what needs the other kernel is marked in g.redo.
moe_status_t attn_wide(const Args& a, AttnArgs g, int fmt, int D, int ctas, cudaStream_t stream);

}  // namespace kv
}  // namespace moe
