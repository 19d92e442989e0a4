// kv_append.cu -- appending keys and values to the 4-bit paged cache, with the rotation of q and k on the way, and
// reading the cached values back.
//
// Per row of D values (one token, one head): y = rotate(x) in fp32, then either one rounding to bf16 (q) or the encoder
// of 32-value blocks (k, v): MXFP4 keeps the smallest power of two that covers the block's largest |y| with 6 steps,
// INT4 the best of six scales by squared error; the rules are moe_encode_blocks'. The kernel is bound by latency in
// decode (q_start -> length -> table -> store, a chain of four L2 trips) and by HBM for prompts.
//
// D / 4 lanes hold a row, four values each, so that a block is 8 neighbouring lanes: its maximum is three shuffles, a K
// word is two lanes' codes, a V word is one lane's. A warp takes 128 / D rows of one kind (q, k or v) at a time, and
// several such groups of its token in turn when there are many tokens: the token's lookups and rotation are then
// shared, and four groups' loads are in flight.
#include "kv.cuh"

namespace moe {
namespace kv {

constexpr int kAppendThreads = 128;
constexpr float kClamp = 18446744073709551616.0f;   // 2^64: what the attention's arithmetic is sure to carry

struct AppendArgs {
  const uint16_t *k, *v, *q;
  int64_t k_stride, v_stride, q_stride;
  uint16_t* q_out;
  const float *cos, *sin;
  int32_t q_heads, rope_dim, rope_rows, interleaved;
  int32_t per_warp;   // row groups a warp handles
  int32_t chunks;     // warps a token is spread over
};

// The sequence of token t: the last b with q_start[b] <= t (q_start is increasing), found 32 boundaries at a time; the last
// step brings its rows and length along (one L2 trip for up to 32 sequences, two for 1024).
__device__ __forceinline__ Seq find_seq(const Args& a, int t, int& b) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = a.n_seqs;        // the answer lies in [lo, lo + n)
  while (n > 32) {
    const int step = (n + 31) >> 5;
    const bool le = lane * step < n && __ldg(a.q_start + lo + lane * step) <= t;
    const int c = __popc(__ballot_sync(0xFFFFFFFFu, le));
    if (c > 1) lo += (c - 1) * step;
    n = min(step, a.n_seqs - lo);
  }
  const bool in = lane < n;
  const int q0 = in ? __ldg(a.q_start + lo + lane) : 0x7FFFFFFF, q1 = in ? __ldg(a.q_start + lo + lane + 1) : 0,
            len = in ? __ldg(a.seq_len + lo + lane) : 0;
  const int k = max(0, __popc(__ballot_sync(0xFFFFFFFFu, q0 <= t)) - 1);
  b = lo + k;
  return check_seq(a, __shfl_sync(0xFFFFFFFFu, q0, k), __shfl_sync(0xFFFFFFFFu, q1, k), __shfl_sync(0xFFFFFFFFu, len, k),
                   0x7FFFFFFF);
}

__device__ __forceinline__ float4 load4_bf16(const uint16_t* p) {
  const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xFFFF0000u));
}

// The rotation of a token's rows as a lane applies it: y = x c + partner s, the same for every row. `from`: the lane that
// holds the partners (half-split pairs), or the lane itself (interleaved pairs lie in one lane).
struct Turn { float c[4], s[4]; int from; bool in, inter; };
__device__ __forceinline__ Turn load_turn(int l, int R, bool inter, const float* cs, const float* sn) {
  Turn t;
  const int d = 4 * l, lane = threadIdx.x & 31;
  t.inter = inter;
  t.in = d < R;
  t.from = lane;
#pragma unroll
  for (int j = 0; j < 4; ++j) { t.c[j] = 1.f; t.s[j] = 0.f; }
  if (!t.in) return t;
  if (inter) {
    const float2 c = __ldg(reinterpret_cast<const float2*>(cs + 2 * l)), s = __ldg(reinterpret_cast<const float2*>(sn + 2 * l));
    t.c[0] = t.c[1] = c.x; t.c[2] = t.c[3] = c.y;
    t.s[0] = -s.x; t.s[1] = s.x; t.s[2] = -s.y; t.s[3] = s.y;
  } else {
    const bool first = d < R / 2;
    const int i = first ? d : d - R / 2;
    const float4 c = __ldg(reinterpret_cast<const float4*>(cs + i)), s = __ldg(reinterpret_cast<const float4*>(sn + i));
    t.from = first ? lane + R / 8 : lane - R / 8;
    t.c[0] = c.x; t.c[1] = c.y; t.c[2] = c.z; t.c[3] = c.w;
    t.s[0] = first ? -s.x : s.x; t.s[1] = first ? -s.y : s.y; t.s[2] = first ? -s.z : s.z; t.s[3] = first ? -s.w : s.w;
  }
  return t;
}
// y of dimensions 4 l .. 4 l + 3 of a row: each product and the sum are rounded (no contraction), as the call promises
// (x_a c - x_b s is x_a c + x_b (-s): a sign does not round)
__device__ __forceinline__ float4 rotate(float4 x, const Turn& t) {
  float4 p = make_float4(x.y, x.x, x.w, x.z);
  if (!t.inter)
    p = make_float4(__shfl_sync(0xFFFFFFFFu, x.x, t.from), __shfl_sync(0xFFFFFFFFu, x.y, t.from),
                    __shfl_sync(0xFFFFFFFFu, x.z, t.from), __shfl_sync(0xFFFFFFFFu, x.w, t.from));
  if (!t.in) return x;
  return make_float4(__fadd_rn(__fmul_rn(x.x, t.c[0]), __fmul_rn(p.x, t.s[0])), __fadd_rn(__fmul_rn(x.y, t.c[1]), __fmul_rn(p.y, t.s[1])),
                     __fadd_rn(__fmul_rn(x.z, t.c[2]), __fmul_rn(p.z, t.s[2])), __fadd_rn(__fmul_rn(x.w, t.c[3]), __fmul_rn(p.w, t.s[3])));
}

__device__ __forceinline__ float sane(float v) { return v != v ? 0.f : fminf(fmaxf(v, -kClamp), kClamp); }

// clamp(rint(w / s), -8, 7) of the rounded quotient, |w / s| < 8.2, without dividing where the product with the reciprocal
// (off by less than 3e-6) is not that near to a tie
__device__ __forceinline__ float quotient(float w, float s, float inv) {
  const float t = w * inv;
  float r = rintf(t);
  if (fabsf(t - r) > 0.499996f) r = rintf(__fdiv_rn(w, s));
  return fminf(fmaxf(r, -8.f), 7.f);
}

// Block of 32 values in 8 neighbouring lanes -> this lane's four codes (code j in bits 4 j ..) and the block's scale bits.
template <int FMT>
__device__ __forceinline__ uint32_t encode(float4 y, uint32_t& scale) {
  float w[4] = {sane(y.x), sane(y.y), sane(y.z), sane(y.w)};
  float amax = fmaxf(fmaxf(fabsf(w[0]), fabsf(w[1])), fmaxf(fabsf(w[2]), fabsf(w[3])));
#pragma unroll
  for (int o = 4; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  uint32_t codes = 0;
  if (FMT == MOE_FMT_MXFP4) {
    // e = clamp(k + 127, 1, 254), k the smallest integer with amax <= 6 * 2^k: from the exponent, one more if the
    // mantissa exceeds 1.5
    const uint32_t ab = __float_as_uint(amax);
    int e = (int)(ab >> 23) - 2 + ((ab & 0x7FFFFFu) > 0x400000u ? 1 : 0);
    e = e < 1 ? 1 : e;   // e <= 190 for |w| <= 2^64
    const int h = (127 - e) >> 1;
    const float s1 = exp2i(h), s2 = exp2i(127 - e - h);   // w 2^(127 - e) by two exact powers of two
    // nearest magnitude, ties to the even code, signs kept: the hardware's rounding to E2M1 (the second operand goes low)
    asm("{\n\t.reg .b8 a, b, z;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "mov.b32 %0, {a, b, a, b};\n\t}"
        : "=r"(codes)
        : "f"(w[0] * s1 * s2), "f"(w[1] * s1 * s2), "f"(w[2] * s1 * s2), "f"(w[3] * s1 * s2));
    codes &= 0xFFFFu;
    scale = (uint32_t)e;
  } else {
    // Six candidate scales: each lane forms its four squared errors for all (two padding candidates never win), then
    // three exchanges add the 8 lanes' in the promised order (i with i + 16, + 8, + 4) while halving the candidates a
    // lane holds, so that lane l of the block ends with candidate l: 28 shuffles instead of 72.
    const float grid[6] = {6.0f / 7.0f, 0.9f, 0.95f, 1.0f, 1.05f, 1.1f};
    const float am = fmaxf(amax, 1e-8f);
    const int l = threadIdx.x & 7;
    float s[6], inv[6], m[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i < 6) {
        s[i] = __fdiv_rn(__fmul_rn(am, grid[i]), 7.0f);
        inv[i] = 1.f / s[i];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (i < 6) {
          const float q = quotient(w[j], s[i], inv[i]);
          const float d = __fsub_rn(w[j], __fmul_rn(q, s[i]));
          m[i][j] = __fmul_rn(d, d);
        } else {
          m[i][j] = __int_as_float(0x7f800000);
        }
      }
    }
#pragma unroll
    for (int o = 4; o; o >>= 1) {
      const bool up = l & o;   // the upper lanes keep the upper half of the candidates
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i < o) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float keep = up ? m[i + o][j] : m[i][j], give = up ? m[i][j] : m[i + o][j];
            m[i][j] = __fadd_rn(keep, __shfl_xor_sync(0xFFFFFFFFu, give, o));
          }
        }
      }
    }
    float err = __fadd_rn(__fadd_rn(m[0][0], m[0][2]), __fadd_rn(m[0][1], m[0][3]));
    int best = l;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      const float e2 = __shfl_xor_sync(0xFFFFFFFFu, err, o);
      const int b2 = __shfl_xor_sync(0xFFFFFFFFu, best, o);
      if (e2 < err || (e2 == err && b2 < best)) { err = e2; best = b2; }
    }
    float bs = s[0], bi = inv[0];
#pragma unroll
    for (int i = 1; i < 6; ++i) {
      bs = best == i ? s[i] : bs;
      bi = best == i ? inv[i] : bi;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int q = (int)quotient(w[j], bs, bi);
      codes |= (uint32_t)(q & 15) << (4 * j);
    }
    scale = __bfloat16_as_ushort(__float2bfloat16_rn(bs));
  }
  return codes;
}

template <int FMT>
__device__ __forceinline__ void store_scale(uint8_t* p, uint32_t s) {
  if (FMT == MOE_FMT_MXFP4) *p = (uint8_t)s;
  else *reinterpret_cast<uint16_t*>(p) = (uint16_t)s;
}

__device__ __forceinline__ uint32_t spread_nibbles(uint32_t c) {   // 16 bits of four codes -> one code per byte
  return (c & 0xFu) | ((c & 0xF0u) << 4) | ((c & 0xF00u) << 8) | ((c & 0xF000u) << 12);
}

template <int FMT, int D>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(Args a, AppendArgs g) {
  using S = Sub<FMT, D>;
  constexpr int LPR = D / 4, RPW = 32 / LPR;   // lanes per row, rows per warp
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  const int t = (int)(w / g.chunks), chunk = (int)(w % g.chunks);
  if (t >= a.n_tokens) return;
  const int l = lane % LPR, sub = lane / LPR, blk = l >> 3, r = l & 7;   // this lane's place in its row
  // row groups: first q's, then k's, then v's
  const int gq = (g.q_heads + RPW - 1) / RPW, gk = (a.kv_heads + RPW - 1) / RPW;
  const int g0 = chunk * g.per_warp;
  int g1 = min(gq + 2 * gk, g0 + g.per_warp);
  const uint16_t* qp = g.q + (int64_t)t * g.q_stride + 4 * l;
  const uint16_t* kp = g.k + (int64_t)t * g.k_stride + 4 * l;
  const uint16_t* vp = g.v + (int64_t)t * g.v_stride + 4 * l;
  constexpr int U = 4;   // row groups whose loads are in flight
  float4 xs[U];
  auto load_rows = [&](int gb) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int gi = gb + u;
      const int h = (gi < gq ? gi : gi < gq + gk ? gi - gq : gi - gq - gk) * RPW + sub;
      const uint16_t* p = gi < gq ? qp : gi < gq + gk ? kp : vp;
      xs[u] = gi < g1 && h < (gi < gq ? g.q_heads : a.kv_heads) ? load4_bf16(p + h * D) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  load_rows(g0);         // (on the way during the lookups)
  int b;
  const Seq sq = find_seq(a, t, b);
  const int j = t - sq.q0;
  const bool in_seq = j >= 0 && j < sq.qn;                 // a row past the last sequence's is nobody's: q is copied
  const int pos = in_seq ? sq.len - sq.qn + j : -1;
  int at = pos < 0 ? 0 : pos;
  if (g.rope_dim && at >= g.rope_rows) {
    record_error(a.status, MOE_ERR_INVALID_ARG);
    at = 0;
  }
  const float *cs = g.cos + (int64_t)at * (g.rope_dim / 2), *sn = g.sin + (int64_t)at * (g.rope_dim / 2);
  bool there = false;
  uint8_t* base = a.pages;
  const int slot = pos & 15;
  if (pos >= 0) {
    const int pg = pos / a.page_tokens;
    const int id = check_page(a, __ldg(a.block_table + (int64_t)b * a.table_stride + pg), there);
    base += (int64_t)id * a.page_stride + (int64_t)((pos - pg * a.page_tokens) >> 4) * S::BYTES;
  }
  const int64_t head_stride = (int64_t)(a.page_tokens / 16) * S::BYTES;
  // MXFP4 V bytes hold an even and an odd token. If both are new in this call, the even token's warp writes both;
  // otherwise the neighbour's half is read and kept.
  const bool odd = slot & 1;
  const bool mate_new = FMT == MOE_FMT_MXFP4 && pos >= 0 && (odd ? j > 0 && pos > 0 : j + 1 < sq.qn);
  const Turn turn = load_turn(l, g.rope_dim, g.interleaved, cs, sn);
  if (there && odd && mate_new) g1 = min(g1, gq + gk);   // the even token's warp writes v
  const int k_word = slot * (D / 2) + ((r >> 1) * S::NB + blk) * 4, scale_at = (slot * S::NB + blk) * S::SB;
  const int v_word = S::VC + ((((slot >> 3) * 8 + r) * 4 + ((slot >> 1) & 3)) * S::NB + blk) * 4;
  for (int gb = g0; gb < g1; gb += U) {
    if (gb > g0) load_rows(gb);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int gi = gb + u;
      if (gi >= g1) break;
      if (gi < gq) {
        const int h = gi * RPW + sub;
        const float4 y = g.rope_dim ? rotate(xs[u], turn) : xs[u];
        const __nv_bfloat162 lo = __floats2bfloat162_rn(y.x, y.y), hi = __floats2bfloat162_rn(y.z, y.w);
        if (h < g.q_heads)
          *reinterpret_cast<uint2*>(g.q_out + ((int64_t)t * g.q_heads + h) * D + 4 * l) =
              make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
        continue;
      }
      if (!there) break;
      uint32_t scale;
      if (gi < gq + gk) {
        const int h = (gi - gq) * RPW + sub;
        const float4 y = g.rope_dim ? rotate(xs[u], turn) : xs[u];
        const uint32_t codes = encode<FMT>(y, scale);
        // a lane pair's 32-bit word (dimensions 32 blk + 8 c .. + 7, c = r / 2)
        const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, codes, 1);
        if (h < a.kv_heads) {
          uint8_t* sb = base + (int64_t)h * head_stride;
          if (!(r & 1)) *reinterpret_cast<uint32_t*>(sb + k_word) = codes | (other << 16);
          if (r == 0) store_scale<FMT>(sb + S::KS + scale_at, scale);
        }
        continue;
      }
      const int h = (gi - gq - gk) * RPW + sub;
      const bool have = h < a.kv_heads;
      uint8_t* sb = base + (int64_t)(have ? h : 0) * head_stride;
      uint32_t* word = reinterpret_cast<uint32_t*>(sb + v_word);
      if (FMT == MOE_FMT_INT4G32) {
        const uint32_t codes = encode<FMT>(xs[u], scale);
        if (have) reinterpret_cast<uint16_t*>(word)[odd] = (uint16_t)codes;
      } else if (mate_new) {   // (this is the even token)
        const float4 z = have ? load4_bf16(vp + g.v_stride + h * D) : make_float4(0.f, 0.f, 0.f, 0.f);
        const uint32_t codes = encode<FMT>(xs[u], scale);
        uint32_t scale2;
        const uint32_t codes2 = encode<FMT>(z, scale2);
        if (have) {
          *word = spread_nibbles(codes) | (spread_nibbles(codes2) << 4);
          if (r == 0) store_scale<FMT>(sb + S::VS + scale_at + S::NB * S::SB, scale2);
        }
      } else {
        const uint32_t old = *word;   // the neighbour's half, on the way while this row is encoded
        const uint32_t codes = encode<FMT>(xs[u], scale);
        if (have) *word = odd ? (old & 0x0F0F0F0Fu) | (spread_nibbles(codes) << 4) : (old & 0xF0F0F0F0u) | spread_nibbles(codes);
      }
      if (have && r == 0) store_scale<FMT>(sb + S::VS + scale_at, scale);
    }
  }
}

template <int FMT>
__device__ __forceinline__ float4 decode4(uint32_t c, float s) {
  if (FMT == MOE_FMT_MXFP4) {
    const uint32_t a = e2m1x2_to_f16x2(c, 0), b = e2m1x2_to_f16x2(c, 1);
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a)), y = __half22float2(*reinterpret_cast<const __half2*>(&b));
    return make_float4(x.x * s, x.y * s, y.x * s, y.y * s);
  }
  return make_float4((float)((int)(c << 28) >> 28) * s, (float)((int)(c << 24) >> 28) * s, (float)((int)(c << 20) >> 28) * s,
                     (float)((int)(c << 16) >> 28) * s);
}

template <int FMT, int D>
__global__ void __launch_bounds__(kAppendThreads) read_kernel(Args a, float* k_out, float* v_out, int chunks, int per_warp) {
  using S = Sub<FMT, D>;
  constexpr int LPR = D / 4, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  const int t = (int)(w / chunks), chunk = (int)(w % chunks);
  if (t >= a.n_tokens) return;
  int b;
  const Seq sq = find_seq(a, t, b);
  const int j = t - sq.q0;
  const int pos = j >= 0 && j < sq.qn ? sq.len - sq.qn + j : -1;
  const uint8_t* base = a.pages;
  const int slot = pos & 15;
  if (pos >= 0) {
    bool ok;
    const int pg = pos / a.page_tokens;
    const int id = check_page(a, __ldg(a.block_table + (int64_t)b * a.table_stride + pg), ok);
    base += (int64_t)id * a.page_stride + (int64_t)((pos - pg * a.page_tokens) >> 4) * S::BYTES;
  }
  const int64_t head_stride = (int64_t)(a.page_tokens / 16) * S::BYTES;
  const int l = lane % LPR, sub = lane / LPR, blk = l >> 3, r = l & 7;
  const int groups = (2 * a.kv_heads + RPW - 1) / RPW;
  const int g0 = chunk * per_warp, g1 = min(groups, g0 + per_warp);
  constexpr int U = 4;   // row groups whose loads are in flight
  for (int gb = g0; gb < g1; gb += U) {
    uint32_t c[U];
    float sc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = (gb + u) * RPW + sub;
      c[u] = 0;
      sc[u] = 0.f;
      if (gb + u >= g1 || row >= 2 * a.kv_heads || pos < 0) continue;
      const bool is_k = row < a.kv_heads;
      const uint8_t* sb = base + (int64_t)(is_k ? row : row - a.kv_heads) * head_stride;
      const uint8_t* word = sb + S::VC + ((((slot >> 3) * 8 + r) * 4 + ((slot >> 1) & 3)) * S::NB + blk) * 4;
      if (is_k) c[u] = *reinterpret_cast<const uint16_t*>(sb + slot * (D / 2) + ((r >> 1) * S::NB + blk) * 4 + 2 * (r & 1));
      else c[u] = FMT == MOE_FMT_MXFP4 ? *reinterpret_cast<const uint32_t*>(word) : reinterpret_cast<const uint16_t*>(word)[slot & 1];
      sc[u] = load_scale<FMT>(sb + (is_k ? S::KS : S::VS) + (slot * S::NB + blk) * S::SB);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = (gb + u) * RPW + sub;
      if (gb + u >= g1 || row >= 2 * a.kv_heads) continue;
      const bool is_k = row < a.kv_heads;
      float* out = is_k ? k_out : v_out;
      if (!out) continue;
      if (FMT == MOE_FMT_MXFP4 && !is_k) {
        const uint32_t w = c[u] >> (4 * (slot & 1));
        c[u] = (w & 0xFu) | ((w >> 4) & 0xF0u) | ((w >> 8) & 0xF00u) | ((w >> 12) & 0xF000u);
      }
      __stcs(reinterpret_cast<float4*>(out + ((int64_t)t * a.kv_heads + (is_k ? row : row - a.kv_heads)) * D + 4 * l),
             decode4<FMT>(c[u], sc[u]));
    }
  }
}

// Row groups a warp handles in turn: one while the launch is small (every row its own warp: latency), more once there
// are twice as many row groups as resident warps (the token's lookups, three dependent L2 trips, are then shared).
static void split(int64_t tokens, int groups, int* per_warp, int* chunks) {
  const int64_t resident = 152 * 64, n = tokens * groups / resident;
  *per_warp = (int)(n < 1 ? 1 : n > groups ? groups : n);
  *chunks = (groups + *per_warp - 1) / *per_warp;
}

}  // namespace kv
}  // namespace moe

using namespace moe;

extern "C" size_t moe_kv_page_bytes(moe_format_t fmt, int32_t head_dim, int32_t kv_heads, int32_t page_tokens) {
  const moe_kv_cache_t c{fmt, head_dim, kv_heads, page_tokens, 1, 0, nullptr};
  if (kv::check_cache(&c) != MOE_OK) return 0;
  return (size_t)kv_heads * (page_tokens / 16) * kv::sub_bytes(fmt, head_dim);
}

extern "C" moe_status_t moe_kv_append(const moe_kv_cache_t* cache, const moe_kv_batch_t* batch, const void* k,
                                      int64_t k_stride, const void* v, int64_t v_stride, const void* q, int64_t q_stride,
                                      int32_t q_heads, void* q_out, const float* cos, const float* sin, int32_t rope_dim,
                                      int32_t rope_rows, int32_t interleaved, void* ws, size_t ws_bytes, void* stream) {
  MOE_NVTX("moe_kv_append");
  if (moe_internal::fault("kv_append")) return MOE_ERR_FAULT_INJECTED;
  kv::Args a;
  moe_status_t st = kv::check(cache, batch, &a);
  if (st != MOE_OK) return st;
  const int D = cache->head_dim;
  if (!k || !v || !ws || !kv::aligned(k, 16) || !kv::aligned(v, 16) || !kv::aligned(ws, 256)) return MOE_ERR_INVALID_ARG;
  if (q && (!q_out || !kv::aligned(q, 16) || !kv::aligned(q_out, 16))) return MOE_ERR_INVALID_ARG;
  if (rope_dim > 0 && (!cos || !sin || !kv::aligned(cos, 16) || !kv::aligned(sin, 16))) return MOE_ERR_INVALID_ARG;
  const int64_t kv_row = (int64_t)cache->kv_heads * D;
  if (k_stride % 8 || v_stride % 8 || k_stride < kv_row || v_stride < kv_row) return MOE_ERR_SHAPE;
  if (q && (q_heads < 1 || q_heads > 4096 || q_stride % 8 || q_stride < (int64_t)q_heads * D)) return MOE_ERR_SHAPE;
  if (rope_dim < 0 || rope_dim > D || rope_dim % 8 || (rope_dim > 0 && rope_rows < 1)) return MOE_ERR_SHAPE;
  if (ws_bytes < sizeof(WsHeader)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if ((st = moe_check_device()) != MOE_OK) return st;
  a.status = &((WsHeader*)ws)->status;
  kv::AppendArgs g{(const uint16_t*)k, (const uint16_t*)v, (const uint16_t*)q, k_stride, v_stride, q_stride,
                   (uint16_t*)q_out, cos, sin, q ? q_heads : 0, rope_dim, rope_rows, interleaved ? 1 : 0, 0, 0};
  const int rpw = 128 / D;   // rows of a group
  kv::split(batch->n_tokens, (g.q_heads + rpw - 1) / rpw + 2 * ((cache->kv_heads + rpw - 1) / rpw), &g.per_warp, &g.chunks);
  const int64_t warps = (int64_t)batch->n_tokens * g.chunks, ctas = (warps + 3) / 4;
  if (ctas > 0x7FFFFFFF) return MOE_ERR_SHAPE;
#define KV_CALL(F, DD) kv::append_kernel<F, DD><<<(unsigned)ctas, kv::kAppendThreads, 0, (cudaStream_t)stream>>>(a, g)
  KV_DISPATCH(KV_CALL);
#undef KV_CALL
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" moe_status_t moe_kv_read(const moe_kv_cache_t* cache, const moe_kv_batch_t* batch, float* k_out, float* v_out,
                                    void* ws, size_t ws_bytes, void* stream) {
  MOE_NVTX("moe_kv_read");
  if (moe_internal::fault("kv_read")) return MOE_ERR_FAULT_INJECTED;
  kv::Args a;
  moe_status_t st = kv::check(cache, batch, &a);
  if (st != MOE_OK) return st;
  if ((!k_out && !v_out) || !kv::aligned(k_out, 16) || !kv::aligned(v_out, 16) || !ws || !kv::aligned(ws, 256))
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < sizeof(WsHeader)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if ((st = moe_check_device()) != MOE_OK) return st;
  a.status = &((WsHeader*)ws)->status;
  int per_warp, chunks;
  kv::split(batch->n_tokens, (2 * cache->kv_heads * cache->head_dim + 127) / 128, &per_warp, &chunks);
  const int64_t warps = (int64_t)batch->n_tokens * chunks, ctas = (warps + 3) / 4;
  if (ctas > 0x7FFFFFFF) return MOE_ERR_SHAPE;
#define KV_CALL(F, DD) \
  kv::read_kernel<F, DD><<<(unsigned)ctas, kv::kAppendThreads, 0, (cudaStream_t)stream>>>(a, k_out, v_out, chunks, per_warp)
  KV_DISPATCH(KV_CALL);
#undef KV_CALL
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
