// kv_append.cu -- appending keys and values to the 4-bit paged cache, with the rotation of q and k on the way, and
// reading the cached values back.
//
// Per row of D values (one token, one head): y = rotate(x) in fp32, then either one rounding to bf16 (q) or the encoder
// of 32-value blocks (k, v): MXFP4 keeps the smallest power of two that covers the block's largest |y| with 6 steps,
// INT4 the best of six scales by squared error; the rules are moe_encode_blocks'. The kernel is bound by latency in
// decode (q_start and length -> table -> store, a chain of three L2 trips) and by HBM for prompts.
//
// D / E lanes hold a row, E values each. MXFP4, E = 8: a block is 4 neighbouring lanes, its maximum two shuffles, a K word one
// lane's codes, two V words one lane's. INT4, E = 4: its six candidates' sums are spread over 8 lanes. (MXFP4 has E = 4 too, for
// halves of the rotated part that are no multiple of 8.) A warp takes 32 E / D rows of one kind (q, k or v) at a time, and several
// such groups of its token in turn when there are many tokens: the token's lookups and rotation are then shared, and two
// groups' loads are in flight.
// (4 prompts of up to 5459 tokens, 16 + 2 x 16 heads of 64, MXFP4: append 69 us, read 34 us; 48 sequences of 8 tokens: 14 us.)
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

template <int E>
struct Vals { float v[E]; };      // E = 4 or 8 neighbouring dimensions of a row

__device__ __forceinline__ void unpack2(uint32_t u, float& a, float& b) {
  a = __uint_as_float(u << 16);
  b = __uint_as_float(u & 0xFFFF0000u);
}
template <int E>
__device__ __forceinline__ Vals<E> load_bf16(const uint16_t* p) {
  Vals<E> x;
  if (E == 8) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    unpack2(u.x, x.v[0], x.v[1]);
    unpack2(u.y, x.v[2], x.v[3]);
    unpack2(u.z, x.v[4 % E], x.v[5 % E]);
    unpack2(u.w, x.v[6 % E], x.v[7 % E]);
  } else {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
    unpack2(u.x, x.v[0], x.v[1]);
    unpack2(u.y, x.v[2], x.v[3]);
  }
  return x;
}
template <int E>
__device__ __forceinline__ Vals<E> no_values() {
  Vals<E> x;
#pragma unroll
  for (int j = 0; j < E; ++j) x.v[j] = 0.f;
  return x;
}
template <int E>
__device__ __forceinline__ void store_bf16(uint16_t* p, const Vals<E>& y) {
  uint32_t u[E / 2];
#pragma unroll
  for (int j = 0; j < E / 2; ++j) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(y.v[2 * j], y.v[2 * j + 1]);
    u[j] = *reinterpret_cast<const uint32_t*>(&b);
  }
  if (E == 8) *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2 % (E / 2)], u[3 % (E / 2)]);
  else *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
}

// The rotation of a token's rows as a lane applies it: y = x c + partner s, the same for every row. `from`: the lane that
// holds the partners (half-split pairs), or the lane itself (interleaved pairs lie in one lane).
template <int E>
struct Turn { float c[E], s[E]; int from; bool in, inter; };
template <int E>
__device__ __forceinline__ Turn<E> load_turn(int l, int R, bool inter, const float* cs, const float* sn) {
  Turn<E> t;
  const int d = E * l, lane = threadIdx.x & 31;
  t.inter = inter;
  t.in = d < R;
  t.from = lane;
#pragma unroll
  for (int j = 0; j < E; ++j) { t.c[j] = 1.f; t.s[j] = 0.f; }
  if (!t.in) return t;
  if (inter) {
#pragma unroll
    for (int j = 0; j < E; j += 4) {
      const float2 c = __ldg(reinterpret_cast<const float2*>(cs + (d + j) / 2)), s = __ldg(reinterpret_cast<const float2*>(sn + (d + j) / 2));
      t.c[j] = t.c[j + 1] = c.x; t.c[j + 2] = t.c[j + 3] = c.y;
      t.s[j] = -s.x; t.s[j + 1] = s.x; t.s[j + 2] = -s.y; t.s[j + 3] = s.y;
    }
  } else {
    const bool first = d < R / 2;
    const int i = first ? d : d - R / 2;
    t.from = first ? lane + R / (2 * E) : lane - R / (2 * E);
#pragma unroll
    for (int j = 0; j < E; j += 4) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(cs + i + j)), s = __ldg(reinterpret_cast<const float4*>(sn + i + j));
      t.c[j] = c.x; t.c[j + 1] = c.y; t.c[j + 2] = c.z; t.c[j + 3] = c.w;
      t.s[j] = first ? -s.x : s.x; t.s[j + 1] = first ? -s.y : s.y;
      t.s[j + 2] = first ? -s.z : s.z; t.s[j + 3] = first ? -s.w : s.w;
    }
  }
  return t;
}
// y of dimensions E l .. E l + E - 1 of a row: each product and the sum are rounded (no contraction), as the call promises
// (x_a c - x_b s is x_a c + x_b (-s): a sign does not round)
template <int E>
__device__ __forceinline__ Vals<E> rotate(const Vals<E>& x, const Turn<E>& t) {
  Vals<E> p, y;
#pragma unroll
  for (int j = 0; j < E; ++j) p.v[j] = t.inter ? x.v[j ^ 1] : x.v[j];
  if (!t.inter) {
#pragma unroll
    for (int j = 0; j < E; ++j) p.v[j] = __shfl_sync(0xFFFFFFFFu, p.v[j], t.from);
  }
#pragma unroll
  for (int j = 0; j < E; ++j) y.v[j] = t.in ? __fadd_rn(__fmul_rn(x.v[j], t.c[j]), __fmul_rn(p.v[j], t.s[j])) : x.v[j];
  return y;
}

__device__ __forceinline__ float sane(float v) { return v != v ? 0.f : fminf(fmaxf(v, -kClamp), kClamp); }
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// clamp(rint(w / s), -8, 7) of the rounded quotient, |w / s| < 8.2, without dividing where the product with the reciprocal
// (off by less than 3e-6) is not that near to a tie
__device__ __forceinline__ float quotient(float w, float s, float inv) {
  const float t = w * inv;
  float r = rintf(t);
  if (fabsf(t - r) > 0.499996f) r = rintf(__fdiv_rn(w, s));
  return fminf(fmaxf(r, -8.f), 7.f);
}

// Block of 32 values in 32 / E neighbouring lanes -> this lane's codes (code j in bits 4 j ..) and the block's scale bits.
template <int FMT, int E>
__device__ __forceinline__ uint32_t encode(const Vals<E>& y, uint32_t& scale) {
  float w[E], amax = fabsf(y.v[0]);
#pragma unroll
  for (int j = 0; j < E; ++j) w[j] = y.v[j];
#pragma unroll
  for (int j = 1; j < E; ++j) amax = max_or_nan(amax, fabsf(w[j]));
  if (!(amax <= kClamp)) {            // (NaN too)
    amax = 0.f;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      w[j] = sane(w[j]);
      amax = fmaxf(amax, fabsf(w[j]));
    }
  }
#pragma unroll
  for (int o = 16 / E; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  uint32_t codes = 0;
  if (FMT == MOE_FMT_MXFP4) {
    // e = clamp(k + 127, 1, 254), k the smallest integer with amax <= 6 * 2^k: from the exponent, one more if the
    // mantissa exceeds 1.5
    const uint32_t ab = __float_as_uint(amax);
    int e = (int)(ab >> 23) - 2 + ((ab & 0x7FFFFFu) > 0x400000u ? 1 : 0);
    e = e < 1 ? 1 : e;                // e <= 190 for |w| <= 2^64: 2^(127 - e) is a normal number, the products exact
    const float s = exp2i(127 - e);
    // nearest magnitude, ties to the even code, signs kept: the hardware's rounding to E2M1 (the second operand goes low)
#pragma unroll
    for (int j = 0; j < E; j += 4) {
      uint32_t c;
      asm("{\n\t.reg .b8 a, b, z;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
          "mov.b32 %0, {a, b, a, b};\n\t}"
          : "=r"(c)
          : "f"(w[j] * s), "f"(w[j + 1] * s), "f"(w[j + 2] * s), "f"(w[j + 3] * s));
      codes |= j ? c << 16 : c & 0xFFFFu;
    }
    scale = (uint32_t)e;
  } else {
    static_assert(FMT == MOE_FMT_MXFP4 || E == 4, "the INT4 sums are laid out over 8 lanes");
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

__device__ __forceinline__ uint32_t spread_nibbles(uint32_t c) {   // the low 16 bits' four codes -> one code per byte
  return (c & 0xFu) | ((c & 0xF0u) << 4) | ((c & 0xF00u) << 8) | ((c & 0xF000u) << 12);
}

template <int FMT, int D, int E>
__global__ void __launch_bounds__(kAppendThreads, 8) append_kernel(Args a, AppendArgs g) {
  using S = Sub<FMT, D>;
  constexpr int LPR = D / E, RPW = 32 / LPR, LPB = 32 / E;   // lanes per row, rows per warp, lanes per block
  constexpr int W = E / 4;                                   // V words of a lane
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  const int t = (int)(w / g.chunks), chunk = (int)(w % g.chunks);
  if (t >= a.n_tokens) return;
  const int l = lane % LPR, sub = lane / LPR, blk = l / LPB, r = l % LPB;   // this lane's place in its row
  // row groups: first q's, then k's, then v's
  const int gq = (g.q_heads + RPW - 1) / RPW, gk = (a.kv_heads + RPW - 1) / RPW;
  const int g0 = chunk * g.per_warp;
  int g1 = min(gq + 2 * gk, g0 + g.per_warp);
  const uint16_t* qp = g.q + (int64_t)t * g.q_stride + E * l;
  const uint16_t* kp = g.k + (int64_t)t * g.k_stride + E * l;
  const uint16_t* vp = g.v + (int64_t)t * g.v_stride + E * l;
  uint16_t* qo = g.q_out + (int64_t)t * g.q_heads * D + E * l;
  // Row groups whose loads are in flight; with 64 registers 32 warps fit an SM. Prompt of 18344 tokens, with the read back:
  // 2 in 32 warps 104 us, 1 in 32 108, 4 in 24 118, 4 in 16 warps of 115 registers 116, 2 in 40 warps (spilling) 120.
  constexpr int U = 2;
  Vals<E> xs[U];
  auto load_rows = [&](int gb) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int gi = gb + u;
      const int h = (gi < gq ? gi : gi < gq + gk ? gi - gq : gi - gq - gk) * RPW + sub;
      const uint16_t* p = gi < gq ? qp : gi < gq + gk ? kp : vp;
      xs[u] = gi < g1 && h < (gi < gq ? g.q_heads : a.kv_heads) ? load_bf16<E>(p + h * D) : no_values<E>();
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
  const uint32_t head_stride = (uint32_t)(a.page_tokens / 16) * S::BYTES;   // (a page has less than 2^31 bytes)
  // MXFP4 V bytes hold an even and an odd token. If both are new in this call, the even token's warp writes both;
  // otherwise the neighbour's half is read and kept.
  const bool odd = slot & 1;
  const bool mate_new = FMT == MOE_FMT_MXFP4 && pos >= 0 && (odd ? j > 0 && pos > 0 : j + 1 < sq.qn);
  const Turn<E> turn = load_turn<E>(l, g.rope_dim, g.interleaved, cs, sn);
  if (there && odd && mate_new) g1 = min(g1, gq + gk);   // the even token's warp writes v
  const int k_word = slot * (D / 2) + ((r * E / 8) * S::NB + blk) * 4, scale_at = (slot * S::NB + blk) * S::SB;
  const int v_word = S::VC + ((((slot >> 3) * 8 + r * W) * 4 + ((slot >> 1) & 3)) * S::NB + blk) * 4;
  constexpr int V_STEP = 4 * S::NB;                        // words from one of a lane's V words to the next
  for (int gb = g0; gb < g1; gb += U) {
    if (gb > g0) load_rows(gb);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int gi = gb + u;
      if (gi >= g1) break;
      if (gi < gq) {
        const int h = gi * RPW + sub;
        const Vals<E> y = g.rope_dim ? rotate(xs[u], turn) : xs[u];
        if (h < g.q_heads) store_bf16<E>(qo + h * D, y);
        continue;
      }
      if (!there) break;
      uint32_t scale;
      if (gi < gq + gk) {
        const int h = (gi - gq) * RPW + sub;
        const Vals<E> y = g.rope_dim ? rotate(xs[u], turn) : xs[u];
        const uint32_t codes = encode<FMT, E>(y, scale);
        // a 32-bit word is dimensions 32 blk + 8 c .. + 7: one lane's, or a lane pair's
        const uint32_t other = E == 4 ? __shfl_xor_sync(0xFFFFFFFFu, codes, 1) : 0u;
        if (h < a.kv_heads) {
          uint8_t* sb = base + (uint32_t)h * head_stride;
          if (E == 8) *reinterpret_cast<uint32_t*>(sb + k_word) = codes;
          else if (!(r & 1)) *reinterpret_cast<uint32_t*>(sb + k_word) = codes | (other << 16);
          if (r == 0) store_scale<FMT>(sb + S::KS + scale_at, scale);
        }
        continue;
      }
      const int h = (gi - gq - gk) * RPW + sub;
      const bool have = h < a.kv_heads;
      uint8_t* sb = base + (uint32_t)(have ? h : 0) * head_stride;
      uint32_t* word = reinterpret_cast<uint32_t*>(sb + v_word);
      if (FMT == MOE_FMT_INT4G32) {
        const uint32_t codes = encode<FMT, E>(xs[u], scale);
        if (have) reinterpret_cast<uint16_t*>(word)[odd] = (uint16_t)codes;
      } else if (mate_new) {   // (this is the even token)
        const Vals<E> z = have ? load_bf16<E>(vp + g.v_stride + h * D) : no_values<E>();
        const uint32_t codes = encode<FMT, E>(xs[u], scale);
        uint32_t scale2;
        const uint32_t codes2 = encode<FMT, E>(z, scale2);
        if (have) {
#pragma unroll
          for (int i = 0; i < W; ++i) word[i * V_STEP] = spread_nibbles(codes >> (16 * i)) | (spread_nibbles(codes2 >> (16 * i)) << 4);
          if (r == 0) store_scale<FMT>(sb + S::VS + scale_at + S::NB * S::SB, scale2);
        }
      } else {
        uint32_t old[W];       // the neighbour's half, on the way while this row is encoded
#pragma unroll
        for (int i = 0; i < W; ++i) old[i] = word[i * V_STEP];
        const uint32_t codes = encode<FMT, E>(xs[u], scale);
        if (have) {
#pragma unroll
          for (int i = 0; i < W; ++i) {
            const uint32_t c = spread_nibbles(codes >> (16 * i));
            word[i * V_STEP] = odd ? (old[i] & 0x0F0F0F0Fu) | (c << 4) : (old[i] & 0xF0F0F0F0u) | c;
          }
        }
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
  const bool eight = cache->fmt == MOE_FMT_MXFP4 && (interleaved || rope_dim % 16 == 0);   // (half a rotation is whole lanes)
  const int rpw = 32 * (eight ? 8 : 4) / D;   // rows of a group
  kv::split(batch->n_tokens, (g.q_heads + rpw - 1) / rpw + 2 * ((cache->kv_heads + rpw - 1) / rpw), &g.per_warp, &g.chunks);
  const int64_t warps = (int64_t)batch->n_tokens * g.chunks, ctas = (warps + 3) / 4;
  if (ctas > 0x7FFFFFFF) return MOE_ERR_SHAPE;
  const cudaStream_t s = (cudaStream_t)stream;
#define KV_CALL(F, DD)                                                                                              \
  if (eight) kv::append_kernel<F, DD, F == MOE_FMT_MXFP4 ? 8 : 4><<<(unsigned)ctas, kv::kAppendThreads, 0, s>>>(a, g); \
  else kv::append_kernel<F, DD, 4><<<(unsigned)ctas, kv::kAppendThreads, 0, s>>>(a, g)
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
