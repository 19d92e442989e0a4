// logits.cu -- from the last layer's logits to the probabilities that moe_spec_accept reads: penalties for repeated tokens,
// biases, the allowed-token mask, temperature and softmax, one row per CTA.
#include <cmath>

#include "common.cuh"
#include "api_internal.h"

namespace moe {
namespace logits {

constexpr int kThreads = 1024;

struct Args {
  const void* x;
  int64_t stride;
  int32_t V, rows_per_seq;
  const float* params;
  const int32_t *counts, *draft, *bias_start, *bias_id;
  const float* bias_value;
  const uint32_t* allowed;
  int64_t allowed_stride;
  float* probs;
  int32_t* top;
};

template <int T>
__device__ __forceinline__ float load(const void* x, int64_t i) {
  const float v = T == MOE_LOGITS_F32 ? ((const float*)x)[i] : __uint_as_float((uint32_t)((const uint16_t*)x)[i] << 16);
  return v != v ? -INFINITY : v;
}

__device__ __forceinline__ float penalise(float x, int c, float rep, float pres, float freq) {
  if (c > 0) {
    x = x > 0.f ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
    x = __fsub_rn(__fsub_rn(x, __fmul_rn(freq, (float)c)), pres);
  }
  return x;
}

template <typename Op>
__device__ __forceinline__ float reduce(float v, float* part, Op op) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = part[0];
  for (int w = 1; w < kThreads / 32; ++w) t = op(t, part[w]);
  return t;
}

template <int T>
__global__ void __launch_bounds__(kThreads) probs_kernel(Args a) {
  __shared__ float part[kThreads / 32];
  __shared__ int s_top;
  const int r = blockIdx.x, i = r / a.rows_per_seq, j = r % a.rows_per_seq, V = a.V;
  const float rep = a.params[4 * i], pres = a.params[4 * i + 1], freq = a.params[4 * i + 2], temp = a.params[4 * i + 3];
  float* p = a.probs + (int64_t)r * V;
  for (int v = threadIdx.x; v < V; v += kThreads) {
    float x = load<T>(a.x, (int64_t)r * a.stride + v);
    if (a.counts) {
      int c = a.counts[(int64_t)i * V + v];
      if (a.draft)
        for (int d = 0; d < j; ++d) c += a.draft[(int64_t)i * (a.rows_per_seq - 1) + d] == v;
      x = penalise(x, c, rep, pres, freq);
    }
    p[v] = x;
  }
  __syncthreads();
  if (a.bias_start)
    for (int e = a.bias_start[i] + threadIdx.x; e < a.bias_start[i + 1]; e += kThreads) {
      const int v = a.bias_id[e];
      if (v >= 0 && v < V) p[v] += a.bias_value[e];
    }
  if (threadIdx.x == 0) s_top = V;
  __syncthreads();
  float m = -INFINITY;
  for (int v = threadIdx.x; v < V; v += kThreads) {
    if (a.allowed && !((a.allowed[(int64_t)r * a.allowed_stride + v / 32] >> (v % 32)) & 1u)) p[v] = -INFINITY;
    m = fmaxf(m, p[v]);
  }
  m = reduce(m, part, [](float x, float y) { return fmaxf(x, y); });
  for (int v = threadIdx.x; v < V; v += kThreads)
    if (p[v] == m) { atomicMin(&s_top, v); break; }
  __syncthreads();
  const int top = m == -INFINITY ? -1 : s_top;
  if (a.top && threadIdx.x == 0) a.top[r] = top;
  const float mt = temp > 0.f ? __fdiv_rn(m, temp) : 0.f;
  float s = 0.f;
  for (int v = threadIdx.x; v < V; v += kThreads) {
    float e;
    if (m == -INFINITY) e = 0.f;
    else if (!(temp > 0.f)) e = v == top ? 1.f : 0.f;
    else if (m == INFINITY) e = p[v] == INFINITY ? 1.f : 0.f;
    else e = expf(__fdiv_rn(p[v], temp) - mt);
    p[v] = e;
    s += e;
  }
  s = reduce(s, part, [](float x, float y) { return x + y; });
  for (int v = threadIdx.x; v < V; v += kThreads) p[v] = s > 0.f ? __fdiv_rn(p[v], s) : 0.f;
}

}  // namespace logits
}  // namespace moe

using namespace moe;

static bool al4(const void* p) { return ((uintptr_t)p & 3) == 0; }

extern "C" moe_status_t moe_logits_probs(const moe_logits_t* l, float* probs, int32_t* top, void* stream) {
  MOE_NVTX("moe_logits_probs");
  if (moe_internal::fault("logits")) return MOE_ERR_FAULT_INJECTED;
  if (!l || !l->logits || !l->params || !probs) return MOE_ERR_INVALID_ARG;
  if (l->type != MOE_LOGITS_F32 && l->type != MOE_LOGITS_BF16) return MOE_ERR_INVALID_ARG;
  if (!al4(probs) || !al4(top) || !al4(l->params) || !al4(l->counts) || !al4(l->draft) || !al4(l->bias_start) ||
      !al4(l->bias_id) || !al4(l->bias_value) || !al4(l->allowed) ||
      ((uintptr_t)l->logits & (l->type == MOE_LOGITS_F32 ? 3 : 1)))
    return MOE_ERR_INVALID_ARG;
  if (l->bias_start && (!l->bias_id || !l->bias_value)) return MOE_ERR_INVALID_ARG;
  if (l->n_seqs < 1 || l->rows_per_seq < 1 || l->rows_per_seq > 64 || (int64_t)l->n_seqs * l->rows_per_seq >= 65536 ||
      l->vocab < 1 || l->vocab > (1 << 22) || l->logits_stride < l->vocab ||
      (l->allowed && l->allowed_stride < (l->vocab + 31) / 32))
    return MOE_ERR_SHAPE;
  if ((const void*)probs == l->logits && (l->type != MOE_LOGITS_F32 || l->logits_stride != l->vocab)) return MOE_ERR_INVALID_ARG;
  moe_status_t st = moe_check_device();
  if (st != MOE_OK) return st;
  const logits::Args a{l->logits, l->logits_stride, l->vocab, l->rows_per_seq, l->params, l->counts,
                       l->rows_per_seq > 1 ? l->draft : nullptr, l->bias_start, l->bias_id, l->bias_value, l->allowed,
                       l->allowed_stride, probs, top};
  const int rows = l->n_seqs * l->rows_per_seq;
  if (l->type == MOE_LOGITS_F32)
    logits::probs_kernel<MOE_LOGITS_F32><<<rows, logits::kThreads, 0, (cudaStream_t)stream>>>(a);
  else
    logits::probs_kernel<MOE_LOGITS_BF16><<<rows, logits::kThreads, 0, (cudaStream_t)stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
