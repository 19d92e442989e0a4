// kv_append.cu -- appending keys and values to the 4-bit paged cache, with the rotation of q and k on the way, and
// reading the cached values back.
//
// Per row of D values (one token, one head): y = rotate(x) in fp32, then either one rounding to bf16 (q) or the encoder
// of 32-value blocks (k, v): MXFP4 keeps the smallest power of two that covers the block's largest |y| with 6 steps,
// INT4 the best of six scales by squared error; the rules are moe_encode_blocks'. The kernel is bound by latency in
// decode (q_start -> length -> table -> store, a chain of four L2 trips) and by HBM for prompts.
//
// D / 4 lanes hold a row, four values each, so that a block is 8 neighbouring lanes: its maximum is three shuffles, a K
// word is two lanes' codes, a V word is one lane's. A warp takes 128 / D rows at a time.
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
  int32_t rows;       // head rows of a token: q_heads + 2 kv_heads
  int32_t per_warp;   // row groups a warp handles
  int32_t chunks;     // warps a token is spread over
};

// The sequence of token t: the last b with q_start[b] <= t, found 32 boundaries at a time (q_start is increasing).
__device__ __forceinline__ int find_seq(const Args& a, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = a.n_seqs;        // the answer lies in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) >> 5, i = lo + lane * step;
    const bool le = lane * step < n && __ldg(a.q_start + i) <= t;
    const int c = __popc(__ballot_sync(0xFFFFFFFFu, le));
    if (c > 1) lo += (c - 1) * step;
    n = min(step, a.n_seqs - lo);
  }
  return lo;
}

__device__ __forceinline__ float4 load4_bf16(const uint16_t* p) {
  const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xFFFF0000u));
}

// y of dimensions 4 l .. 4 l + 3 of a row; every product and sum is rounded (no contraction), as the call promises
__device__ __forceinline__ float4 rotate(float4 x, int l, int R, bool inter, const float* cs, const float* sn) {
  const int d = 4 * l;
  if (inter) {
    if (d >= R) return x;
    const float2 c = __ldg(reinterpret_cast<const float2*>(cs + 2 * l)), s = __ldg(reinterpret_cast<const float2*>(sn + 2 * l));
    return make_float4(__fsub_rn(__fmul_rn(x.x, c.x), __fmul_rn(x.y, s.x)), __fadd_rn(__fmul_rn(x.y, c.x), __fmul_rn(x.x, s.x)),
                       __fsub_rn(__fmul_rn(x.z, c.y), __fmul_rn(x.w, s.y)), __fadd_rn(__fmul_rn(x.w, c.y), __fmul_rn(x.z, s.y)));
  }
  // the pair's other half is R / 8 lanes away (all lanes shuffle; those past R read themselves)
  const bool first = d < R / 2, in = d < R;
  const int lane = threadIdx.x & 31, from = in ? (first ? lane + R / 8 : lane - R / 8) : lane;
  const float4 p = make_float4(__shfl_sync(0xFFFFFFFFu, x.x, from), __shfl_sync(0xFFFFFFFFu, x.y, from),
                               __shfl_sync(0xFFFFFFFFu, x.z, from), __shfl_sync(0xFFFFFFFFu, x.w, from));
  if (!in) return x;
  const int i = first ? d : d - R / 2;
  const float4 c = __ldg(reinterpret_cast<const float4*>(cs + i)), s = __ldg(reinterpret_cast<const float4*>(sn + i));
  if (first)
    return make_float4(__fsub_rn(__fmul_rn(x.x, c.x), __fmul_rn(p.x, s.x)), __fsub_rn(__fmul_rn(x.y, c.y), __fmul_rn(p.y, s.y)),
                       __fsub_rn(__fmul_rn(x.z, c.z), __fmul_rn(p.z, s.z)), __fsub_rn(__fmul_rn(x.w, c.w), __fmul_rn(p.w, s.w)));
  return make_float4(__fadd_rn(__fmul_rn(x.x, c.x), __fmul_rn(p.x, s.x)), __fadd_rn(__fmul_rn(x.y, c.y), __fmul_rn(p.y, s.y)),
                     __fadd_rn(__fmul_rn(x.z, c.z), __fmul_rn(p.z, s.z)), __fadd_rn(__fmul_rn(x.w, c.w), __fmul_rn(p.w, s.w)));
}

__device__ __forceinline__ float sane(float v) { return v != v ? 0.f : fminf(fmaxf(v, -kClamp), kClamp); }

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
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float v = w[j] * s1 * s2, a = fabsf(v);
      // nearest magnitude, ties to the even code: strict where the tie goes down
      uint32_t c = (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) + (a > 5.0f);
      c |= (__float_as_uint(v) >> 28) & 8u;
      codes |= c << (4 * j);
    }
    scale = (uint32_t)e;
  } else {
    // Six candidate scales: each lane forms its four squared errors for all (two padding candidates never win), then
    // three exchanges add the 8 lanes' in the promised order (i with i + 16, + 8, + 4) while halving the candidates a
    // lane holds, so that lane l of the block ends with candidate l: 28 shuffles instead of 72.
    const float grid[6] = {6.0f / 7.0f, 0.9f, 0.95f, 1.0f, 1.05f, 1.1f};
    const float am = fmaxf(amax, 1e-8f);
    const int l = threadIdx.x & 7;
    float s[6], m[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i < 6) s[i] = __fdiv_rn(__fmul_rn(am, grid[i]), 7.0f);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (i < 6) {
          const float q = fminf(fmaxf(rintf(__fdiv_rn(w[j], s[i])), -8.f), 7.f);
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
    float bs = s[0];
#pragma unroll
    for (int i = 1; i < 6; ++i) bs = best == i ? s[i] : bs;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int q = (int)fminf(fmaxf(rintf(__fdiv_rn(w[j], bs)), -8.f), 7.f);
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
  const int b = find_seq(a, t);
  const Seq sq = load_seq(a, b, 0x7FFFFFFF);
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
  const int l = lane % LPR, sub = lane / LPR, blk = l >> 3, r = l & 7;   // this lane's place in its row
  // MXFP4 V bytes hold an even and an odd token. If both are new in this call, the even token's warp writes both;
  // otherwise the neighbour's half is read and kept.
  const bool odd = slot & 1;
  const bool mate_new = FMT == MOE_FMT_MXFP4 && pos >= 0 && (odd ? j > 0 && pos > 0 : j + 1 < sq.qn);
  const int groups = (g.rows + RPW - 1) / RPW;
  const int g0 = chunk * g.per_warp, g1 = min(groups, g0 + g.per_warp);
  for (int gi = g0; gi < g1; ++gi) {
    const int row = gi * RPW + sub;
    const bool have = row < g.rows;
    const int is_q = row < g.q_heads, is_k = !is_q && row < g.q_heads + a.kv_heads;
    const int h = is_q ? row : is_k ? row - g.q_heads : row - g.q_heads - a.kv_heads;
    const uint16_t* src = is_q ? g.q + (int64_t)t * g.q_stride : is_k ? g.k + (int64_t)t * g.k_stride : g.v + (int64_t)t * g.v_stride;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (have) x = load4_bf16(src + (int64_t)h * D + 4 * l);
    const float4 y = g.rope_dim ? rotate(x, l, g.rope_dim, g.interleaved, cs, sn) : x;
    const bool is_v = have && !is_q && !is_k;
    if (have && is_q) {
      __nv_bfloat162 lo = __floats2bfloat162_rn(y.x, y.y), hi = __floats2bfloat162_rn(y.z, y.w);
      uint2 o = make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
      *reinterpret_cast<uint2*>(g.q_out + ((int64_t)t * g.q_heads + h) * D + 4 * l) = o;
    }
    if (__all_sync(0xFFFFFFFFu, !have || is_q)) continue;
    uint32_t scale;
    const uint32_t codes = encode<FMT>(is_v ? x : y, scale);
    uint8_t* sb = base + (int64_t)h * head_stride;
    // K: a lane pair's 32-bit word (dimensions 32 blk + 8 c .. + 7, c = r / 2)
    const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, codes, 1);
    const bool put = have && !is_q && there;
    if (put && is_k) {
      if (!(r & 1)) *reinterpret_cast<uint32_t*>(sb + slot * (D / 2) + ((r >> 1) * S::NB + blk) * 4) = codes | (other << 16);
      if (r == 0) store_scale<FMT>(sb + S::KS + (slot * S::NB + blk) * S::SB, scale);
    }
    uint32_t codes2 = 0, scale2 = 0;
    if (FMT == MOE_FMT_MXFP4 && mate_new && !odd && __any_sync(0xFFFFFFFFu, is_v)) {   // (mate_new is the warp's)
      float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
      if (is_v) z = load4_bf16(src + g.v_stride + (int64_t)h * D + 4 * l);
      codes2 = encode<FMT>(z, scale2);
    }
    if (put && is_v) {
      uint8_t* word = sb + S::VC + ((((slot >> 3) * 8 + r) * 4 + ((slot >> 1) & 3)) * S::NB + blk) * 4;
      if (FMT == MOE_FMT_MXFP4) {
        uint32_t* w32 = reinterpret_cast<uint32_t*>(word);
        if (mate_new) {
          if (!odd) *w32 = spread_nibbles(codes) | (spread_nibbles(codes2) << 4);
        } else if (odd) {
          *w32 = (*w32 & 0x0F0F0F0Fu) | (spread_nibbles(codes) << 4);
        } else {
          *w32 = (*w32 & 0xF0F0F0F0u) | spread_nibbles(codes);
        }
      } else {
        reinterpret_cast<uint16_t*>(word)[odd] = (uint16_t)codes;
      }
      if (r == 0) store_scale<FMT>(sb + S::VS + (slot * S::NB + blk) * S::SB, scale);
    }
  }
}

template <int FMT>
__device__ __forceinline__ float4 decode4(uint32_t c, float s) {
  return make_float4(code_value<FMT>(c & 15u) * s, code_value<FMT>((c >> 4) & 15u) * s, code_value<FMT>((c >> 8) & 15u) * s,
                     code_value<FMT>((c >> 12) & 15u) * s);
}

template <int FMT, int D>
__global__ void __launch_bounds__(kAppendThreads) read_kernel(Args a, float* k_out, float* v_out, int chunks, int per_warp) {
  using S = Sub<FMT, D>;
  constexpr int LPR = D / 4, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  const int t = (int)(w / chunks), chunk = (int)(w % chunks);
  if (t >= a.n_tokens) return;
  const int b = find_seq(a, t);
  const Seq sq = load_seq(a, b, 0x7FFFFFFF);
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
  for (int gi = g0; gi < g1; ++gi) {
    const int row = gi * RPW + sub;
    if (row >= 2 * a.kv_heads) continue;
    const bool is_k = row < a.kv_heads;
    const int h = is_k ? row : row - a.kv_heads;
    float* out = is_k ? k_out : v_out;
    if (!out) continue;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    if (pos >= 0) {
      const uint8_t* sb = base + (int64_t)h * head_stride;
      uint32_t c;
      if (is_k) {
        c = *reinterpret_cast<const uint16_t*>(sb + slot * (D / 2) + ((r >> 1) * S::NB + blk) * 4 + 2 * (r & 1));
      } else {
        const uint8_t* word = sb + S::VC + ((((slot >> 3) * 8 + r) * 4 + ((slot >> 1) & 3)) * S::NB + blk) * 4;
        if (FMT == MOE_FMT_MXFP4) {
          const uint32_t u = *reinterpret_cast<const uint32_t*>(word) >> (4 * (slot & 1));
          c = (u & 0xFu) | ((u >> 4) & 0xF0u) | ((u >> 8) & 0xF00u) | ((u >> 12) & 0xF000u);
        } else {
          c = reinterpret_cast<const uint16_t*>(word)[slot & 1];
        }
      }
      y = decode4<FMT>(c, load_scale<FMT>(sb + (is_k ? S::KS : S::VS) + (slot * S::NB + blk) * S::SB));
    }
    *reinterpret_cast<float4*>(out + ((int64_t)t * a.kv_heads + h) * D + 4 * l) = y;
  }
}

// Row groups a warp handles in turn: one while the launch is small (every row its own warp: latency), more once there
// are several warps for each of an SM's 64 slots anyway (the token's lookups are then shared).
static void split(int64_t tokens, int groups, int* per_warp, int* chunks) {
  const int64_t slots = 152 * 64;
  int64_t n = (tokens * groups + slots - 1) / slots;
  *per_warp = (int)(n < 1 ? 1 : n > 8 ? 8 : n);
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
                   (uint16_t*)q_out, cos, sin, q ? q_heads : 0, rope_dim, rope_rows, interleaved ? 1 : 0, 0, 0, 0};
  g.rows = g.q_heads + 2 * cache->kv_heads;
  kv::split(batch->n_tokens, (g.rows * D + 127) / 128, &g.per_warp, &g.chunks);
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
