// kv_attn.cu -- attention of a decode or verify step over the 4-bit paged KV cache.
//
// For each query row: x_s = scale q . k_s over the visible keys s, out = sum_s softmax(x)_s v_s, lse = log sum_s exp(x_s), in
// one pass over the keys with a running maximum m and sum l: when m grows to m', l and the output so far are multiplied by
// exp(m - m').
#include "kv.cuh"

namespace moe {
namespace kv {

constexpr int kThreads = 128;

// One CTA per (row, query head); its warps take keys in turn, a lane holds D / 32 dimensions.
template <int FMT, int D>
__global__ void __launch_bounds__(kThreads) attn_kernel(Args a, const uint16_t* q, int64_t q_stride, int q_heads, float scale,
                                                        int window, uint16_t* out, float* lse) {
  using S = Sub<FMT, D>;
  constexpr int E = D / 32;
  __shared__ float sm[kThreads / 32], sl[kThreads / 32], so[kThreads / 32][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = blockIdx.x, n = blockIdx.y;
  int b = 0;
  while (b + 1 < a.n_seqs && a.q_start[b + 1] <= t) ++b;
  const Seq sq = load_seq(a, b, a.max_q);
  const int j = t - sq.q0;
  const int pos = j >= 0 && j < sq.qn && sq.len > 0 ? sq.len - sq.qn + j : -1;
  const int h = n / (q_heads / a.kv_heads);
  const int lo = window > 0 && pos - window + 1 > 0 ? pos - window + 1 : 0;
  float qv[E], o[E] = {0.f}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e)   // dimension 32 e + lane
    qv[e] = __uint_as_float((uint32_t)q[(int64_t)t * q_stride + (int64_t)n * D + 32 * e + lane] << 16) * scale;
  for (int s = lo + warp; s <= pos; s += kThreads / 32) {
    bool ok;
    const int pg = s / a.page_tokens, slot = s & 15;
    const int id = check_page(a, a.block_table[(int64_t)b * a.table_stride + pg], ok);
    const uint8_t* sb = a.pages + (int64_t)id * a.page_stride +
                        (int64_t)(h * (a.page_tokens / 16) + ((s - pg * a.page_tokens) >> 4)) * S::BYTES;
    float x = 0.f, v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const uint32_t kc = sb[slot * (D / 2) + ((lane >> 3) * S::NB + e) * 4 + ((lane & 7) >> 1)] >> (4 * (lane & 1)) & 15u;
      const uint8_t* word = sb + S::VC + ((((slot >> 3) * 8 + (lane >> 2)) * 4 + ((slot >> 1) & 3)) * S::NB + e) * 4;
      const uint32_t vc = FMT == MOE_FMT_MXFP4 ? word[lane & 3] >> (4 * (slot & 1)) & 15u
                                               : word[(slot & 1) * 2 + ((lane & 3) >> 1)] >> (4 * (lane & 1)) & 15u;
      x += qv[e] * (code_value<FMT>(kc) * load_scale<FMT>(sb + S::KS + (slot * S::NB + e) * S::SB));
      v[e] = code_value<FMT>(vc) * load_scale<FMT>(sb + S::VS + (slot * S::NB + e) * S::SB);
    }
#pragma unroll
    for (int i = 16; i; i >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, i);
    const float mn = fmaxf(m, x), c = expf(m - mn), p = expf(x - mn);
    l = l * c + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * c + p * v[e];
    m = mn;
  }
  if (lane == 0) { sm[warp] = m; sl[warp] = l; }
#pragma unroll
  for (int e = 0; e < E; ++e) so[warp][32 * e + lane] = o[e];
  __syncthreads();
  float mm = -INFINITY, ll = 0.f;
  for (int w = 0; w < kThreads / 32; ++w) mm = fmaxf(mm, sm[w]);
  for (int w = 0; w < kThreads / 32; ++w) ll += sl[w] > 0.f ? sl[w] * expf(sm[w] - mm) : 0.f;
  for (int d = threadIdx.x; d < D; d += kThreads) {
    float y = 0.f;
    for (int w = 0; w < kThreads / 32; ++w) y += sl[w] > 0.f ? so[w][d] * expf(sm[w] - mm) : 0.f;
    out[((int64_t)t * q_heads + n) * D + d] = __bfloat16_as_ushort(__float2bfloat16_rn(ll > 0.f ? y / ll : 0.f));
  }
  if (lse && threadIdx.x == 0) lse[(int64_t)t * q_heads + n] = ll > 0.f ? mm + logf(ll) : -INFINITY;
}

}  // namespace kv
}  // namespace moe

using namespace moe;

extern "C" size_t moe_kv_workspace_bytes(const moe_kv_cache_t* cache, const moe_kv_batch_t* batch, int32_t q_heads) {
  if (kv::check_cache(cache) != MOE_OK || kv::check_sizes(batch) != MOE_OK) return 0;
  if (q_heads < 1 || q_heads > 4096 || q_heads % cache->kv_heads) return 0;
  return sizeof(WsHeader);
}

extern "C" moe_status_t moe_kv_attention(const moe_kv_cache_t* cache, const moe_kv_batch_t* batch, const void* q,
                                         int64_t q_stride, int32_t q_heads, float scale, int32_t window, void* out, float* lse,
                                         void* ws, size_t ws_bytes, void* stream) {
  MOE_NVTX("moe_kv_attention");
  if (moe_internal::fault("kv_attention")) return MOE_ERR_FAULT_INJECTED;
  kv::Args a;
  moe_status_t st = kv::check(cache, batch, &a);
  if (st != MOE_OK) return st;
  if (!q || !out || !ws || !kv::aligned(q, 16) || !kv::aligned(out, 16) || !kv::aligned(lse, 4) || !kv::aligned(ws, 256))
    return MOE_ERR_INVALID_ARG;
  if (q_heads < 1 || q_heads > 4096 || q_heads % cache->kv_heads || batch->max_q > 8 ||
      (int64_t)batch->max_q * (q_heads / cache->kv_heads) > kv::kMaxRows || q_stride % 8 ||
      q_stride < (int64_t)q_heads * cache->head_dim || window < 0)
    return MOE_ERR_SHAPE;
  if (!(scale - scale == 0.f)) return MOE_ERR_INVALID_ARG;   // NaN or infinite
  const size_t need = moe_kv_workspace_bytes(cache, batch, q_heads);
  if (need == 0 || ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if ((st = moe_check_device()) != MOE_OK) return st;
  a.status = &((WsHeader*)ws)->status;
  const dim3 grid(batch->n_tokens, q_heads);
#define KV_CALL(F, DD)                                                                                                   \
  kv::attn_kernel<F, DD><<<grid, kv::kThreads, 0, (cudaStream_t)stream>>>(a, (const uint16_t*)q, q_stride, q_heads, scale, \
                                                                          window, (uint16_t*)out, lse)
  KV_DISPATCH(KV_CALL);
#undef KV_CALL
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
