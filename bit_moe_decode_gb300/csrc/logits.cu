// logits.cu -- from the last layer's logits to the probabilities that moe_spec_accept reads: penalties for repeated tokens,
// biases, the allowed-token mask, temperature and softmax.
//
// Per value: x = penalised logit + bias, masked; p = exp(x / T - max / T) / sum. Bound by HBM when there are many rows (the
// logits, the counts and the mask are read once, the probabilities written once: 12 bytes a value with fp32 logits),
// by latency when there are few.
//
// A row is split over a cluster of C CTAs; each holds its slice of x in shared memory between the passes, so that every
// value is read and written once: x, then exponentials relative to the slice's maximum, then, after one exchange of
// (maximum, first place, sum) through distributed shared memory, the output. 256 x 131071 with counts: 125 us, 3.2 TB/s, the
// phases of three CTAs an SM overlapping in part (512 threads in two CTAs 121, in three 128 to 148, and 1.3 us more for one
// row); 4 x 8 x 32768: 8.8 us; 1 x 32768: 6.4 us, latency. C is the smallest of 1 .. 16 whose slices
// fit kSlice and that gives the GPU enough CTAs. Only a vocabulary above 16 kSlice is walked in chunks that are formed
// twice (once for the statistics, once for the output).
// The few tokens that need more than their own element (earlier drafts, biases) are patched in shared memory, by the
// thread that owns the entry; what that takes is loaded ahead of the slice.
#include <cmath>
#include <cstring>

#include "common.cuh"
#include "api_internal.h"

namespace moe {
namespace logits {

constexpr int kThreads = 256;
constexpr int kSlice = 16384;      // values a CTA holds: 64 KB, three CTAs on an SM
constexpr int kMaxCluster = 16;
constexpr int kMaxRows = 64;       // rows_per_seq

struct Args {
  const void* x;
  int64_t stride;
  int32_t V, rows_per_seq, slice;  // slice: values per CTA, a multiple of 32; more than kSlice: in chunks
  const float* params;
  const int32_t *counts, *draft, *bias_start, *bias_id;
  const float* bias_value;
  const uint32_t* allowed;
  int64_t allowed_stride;
  float* probs;
  int32_t* top;
};

template <int T>
__device__ __forceinline__ float logit_at(const void* x, int64_t i) {
  return T == MOE_LOGITS_F32 ? __ldcs((const float*)x + i) : __uint_as_float((uint32_t)((const uint16_t*)x)[i] << 16);
}

__device__ __forceinline__ float number(float x) { return x != x ? -INFINITY : x; }   // (NaN is never chosen)

// x / repetition or x * repetition, then (x - frequency c) - presence, each operation rounded (no contraction)
__device__ __forceinline__ float penalise(float x, int c, float rep, float pres, float freq) {
  if (c > 0) {
    x = x > 0.f ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
    x = __fsub_rn(__fsub_rn(x, __fmul_rn(freq, (float)c)), pres);
  }
  return x;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
template <typename V>
__device__ __forceinline__ V peer(const V* p, uint32_t rank) {   // a 4-byte value of another CTA of the cluster
  uint32_t a, v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  V out;
  memcpy(&out, &v, 4);
  return out;
}

// 2^x for x <= 0, 2^-22 relative; below 2^-126 it gives 0
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct Stat { float m; int at; float sum; };   // a CTA's largest x, the first place that has it, its sum of exponentials

template <int T, bool CHUNKED>
__global__ void __launch_bounds__(kThreads, 3) probs_kernel(Args a, uint32_t C) {
  extern __shared__ __align__(16) float xs[];          // one slice, or one chunk of it
  __shared__ Stat s_stat;
  __shared__ float s_m[kThreads / 32];
  __shared__ int s_at[kThreads / 32];
  __shared__ uint32_t s_mask[kSlice / 32 + 2];         // from word 1 on; a word of padding at either end
  __shared__ int s_draft[kMaxRows];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = C > 1 ? cluster_rank() : 0u;
  const int r = blockIdx.x / C, i = r / a.rows_per_seq, j = r - i * a.rows_per_seq, V = a.V;
  const int v0 = min(V, (int)rank * a.slice), v1 = min(V, v0 + a.slice);
  const float rep = __ldg(a.params + 4 * i), pres = __ldg(a.params + 4 * i + 1), freq = __ldg(a.params + 4 * i + 2),
              temp = __ldg(a.params + 4 * i + 3);
  const int64_t x_row = (int64_t)r * a.stride, c_row = (int64_t)i * V;
  const uint32_t* mask = a.allowed ? a.allowed + (int64_t)r * a.allowed_stride : nullptr;
  // this thread's draft (with its logit and count) and its first bias
  const int drafts = a.draft ? j : 0;
  int d_id = -1, d_count = 0, b_id = -1;
  float d_x = 0.f, b_val = 0.f;
  if (tid < drafts) {
    d_id = __ldg(a.draft + (int64_t)i * (a.rows_per_seq - 1) + tid);
    s_draft[tid] = d_id;
    if (d_id >= 0 && d_id < V) {
      d_x = logit_at<T>(a.x, x_row + d_id);
      d_count = __ldg(a.counts + c_row + d_id);
    } else {
      d_id = -1;
    }
  }
  const int b0 = a.bias_start ? __ldg(a.bias_start + i) : 0, b1 = a.bias_start ? __ldg(a.bias_start + i + 1) : 0;
  if (b0 + tid < b1) {
    b_id = __ldg(a.bias_id + b0 + tid);
    b_val = __ldg(a.bias_value + b0 + tid);
  }

  // Place of value k of [lo, ..): xs[mis + k], with mis the logits' place within a 16-byte group (8 bytes of bf16), so that
  // rows of an odd vocabulary move in whole groups too.
  auto misplaced = [&](const void* p, int64_t i, int size) { return (int)(((uintptr_t)p / size + i) & 3); };
  constexpr int kLogitBytes = T == MOE_LOGITS_F32 ? 4 : 2;

  // x of [lo, hi) into xs, the places around them in their groups -inf; returns the thread's largest and its first value
  // (a thread's values ascend)
  auto form = [&](int lo, int hi, float& m, int& at) {
    const int n = hi - lo, mis = misplaced(a.x, x_row + lo, kLogitBytes), groups = (mis + n + 3) / 4;
    const bool whole = !a.counts || misplaced(a.counts, c_row + lo, 4) == mis;
    if (mask) {   // (lo is a multiple of 32)
      const int words = (n + 31) / 32;
      for (int k = tid; k < words + 2; k += kThreads) s_mask[k] = k > 0 && k <= words ? __ldg(mask + lo / 32 + k - 1) : 0u;
    }
    const char* xp = (const char*)a.x + (x_row + lo - mis) * kLogitBytes;
    const int32_t* cp = a.counts ? a.counts + c_row + lo - mis : nullptr;
    constexpr int U = 4;   // groups whose loads are in flight
    for (int q0 = tid; q0 < groups; q0 += U * kThreads) {
      float x[U][4];
      int4 c[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int q = q0 + u * kThreads, k = 4 * q - mis;
        c[u] = make_int4(0, 0, 0, 0);
        if (whole && k >= 0 && k + 3 < n) {
          if (T == MOE_LOGITS_F32) {
            const float4 v = __ldcs(reinterpret_cast<const float4*>(xp) + q);
            x[u][0] = v.x; x[u][1] = v.y; x[u][2] = v.z; x[u][3] = v.w;
          } else {
            const uint2 v = __ldcs(reinterpret_cast<const uint2*>(xp) + q);
            x[u][0] = __uint_as_float(v.x << 16); x[u][1] = __uint_as_float(v.x & 0xFFFF0000u);
            x[u][2] = __uint_as_float(v.y << 16); x[u][3] = __uint_as_float(v.y & 0xFFFF0000u);
          }
          if (cp) c[u] = __ldg(reinterpret_cast<const int4*>(cp) + q);
        } else {
          int ce[4] = {0, 0, 0, 0};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool in = k + e >= 0 && k + e < n;
            x[u][e] = in ? logit_at<T>(a.x, x_row + lo + k + e) : -INFINITY;
            if (in && cp) ce[e] = __ldg(cp + 4 * q + e);
          }
          c[u] = make_int4(ce[0], ce[1], ce[2], ce[3]);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int q = q0 + u * kThreads;
        float4 y = make_float4(number(x[u][0]), number(x[u][1]), number(x[u][2]), number(x[u][3]));
        if ((c[u].x | c[u].y | c[u].z | c[u].w) != 0) {   // few tokens have occurred
          y.x = penalise(y.x, c[u].x, rep, pres, freq);
          y.y = penalise(y.y, c[u].y, rep, pres, freq);
          y.z = penalise(y.z, c[u].z, rep, pres, freq);
          y.w = penalise(y.w, c[u].w, rep, pres, freq);
        }
        if (q < groups) reinterpret_cast<float4*>(xs)[q] = y;
      }
    }
    __syncthreads();
    if (drafts > 0) {
      // a token of earlier drafts: from the logit again, with all their occurrences, by the first that names it
      if (d_id >= lo && d_id < hi) {
        int c = 0, first = tid;
        for (int k = drafts - 1; k >= 0; --k)
          if (s_draft[k] == d_id) { ++c; first = k; }
        if (first == tid) xs[mis + d_id - lo] = penalise(number(d_x), d_count + c, rep, pres, freq);
      }
      __syncthreads();
    }
    if (b1 > b0) {
      if (b_id >= lo && b_id < hi) xs[mis + b_id - lo] = __fadd_rn(xs[mis + b_id - lo], b_val);
      for (int e = b0 + kThreads + tid; e < b1; e += kThreads) {
        const int v = __ldg(a.bias_id + e);
        if (v >= lo && v < hi) xs[mis + v - lo] = __fadd_rn(xs[mis + v - lo], __ldg(a.bias_value + e));
      }
      __syncthreads();
    }
    // the mask, and the largest; the place among a group's four is found at the end
    m = -INFINITY;
    int at4 = -1;
#pragma unroll 4
    for (int q = tid; q < groups; q += kThreads) {
      float4 x = reinterpret_cast<const float4*>(xs)[q];
      if (mask) {
        const int k = 4 * q - mis + 32;                // bits k .. k + 3 from the padding word on
        const uint32_t w = __funnelshift_r(s_mask[k >> 5], s_mask[(k >> 5) + 1], k & 31);
        x.x = w & 1u ? x.x : -INFINITY;
        x.y = w & 2u ? x.y : -INFINITY;
        x.z = w & 4u ? x.z : -INFINITY;
        x.w = w & 8u ? x.w : -INFINITY;
        reinterpret_cast<float4*>(xs)[q] = x;
      }
      const float big = fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w));
      if (big > m) { m = big; at4 = q; }
    }
    at = 0x7FFFFFFF;
    if (at4 >= 0) {
      const float4 x = reinterpret_cast<const float4*>(xs)[at4];
      at = lo + 4 * at4 - mis + (x.x == m ? 0 : x.y == m ? 1 : x.z == m ? 2 : 3);
    }
  };

  float m = -INFINITY;                                 // the slice's largest and its first place
  int at = 0x7FFFFFFF;
  for (int lo = v0; lo < v1; lo += kSlice) {
    float cm;
    int ca;
    form(lo, min(v1, lo + kSlice), cm, ca);
    if (cm > m) { m = cm; at = ca; }
    if (CHUNKED) __syncthreads();
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xFFFFFFFFu, m, o);
    const int at2 = __shfl_xor_sync(0xFFFFFFFFu, at, o);
    if (m2 > m || (m2 == m && at2 < at)) { m = m2; at = at2; }
  }
  if (lane == 0) { s_m[warp] = m; s_at[warp] = at; }
  __syncthreads();
  m = s_m[lane % (kThreads / 32)];
  at = s_at[lane % (kThreads / 32)];
#pragma unroll
  for (int o = kThreads / 64; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xFFFFFFFFu, m, o);
    const int at2 = __shfl_xor_sync(0xFFFFFFFFu, at, o);
    if (m2 > m || (m2 == m && at2 < at)) { m = m2; at = at2; }
  }
  __syncthreads();                                     // s_m is reused

  // Exponentials relative to the slice's maximum, in place: 2^((x - m) log2(e) / T); the difference first, so that its
  // error is relative to itself. A temperature whose reciprocal overflows acts as 0: the first largest takes all. One that is
  // infinite: the smallest scale there is (0 times the -inf of tokens that are not allowed, or not there, is not a number).
  const float by_temp = 1.4426950408889634f / temp, scale = by_temp == 0.f ? __int_as_float(1) : by_temp;
  const bool greedy = !(temp > 0.f && scale < INFINITY);
  float sum = 0.f;
  auto exponentials = [&](int lo, int hi) {
    if (greedy || m == -INFINITY) return;
    const int groups = (misplaced(a.x, x_row + lo, kLogitBytes) + hi - lo + 3) / 4;
    const bool top = m == INFINITY;                    // those at +inf share equally
#pragma unroll 4
    for (int q = tid; q < groups; q += kThreads) {
      float4 x = reinterpret_cast<const float4*>(xs)[q];
      if (top)
        x = make_float4(x.x == m ? 1.f : 0.f, x.y == m ? 1.f : 0.f, x.z == m ? 1.f : 0.f, x.w == m ? 1.f : 0.f);
      else
        x = make_float4(ex2((x.x - m) * scale), ex2((x.y - m) * scale), ex2((x.z - m) * scale), ex2((x.w - m) * scale));
      reinterpret_cast<float4*>(xs)[q] = x;
      sum += (x.x + x.y) + (x.z + x.w);
    }
  };
  for (int lo = v0; lo < v1; lo += kSlice) {
    float cm;
    int ca;
    if (CHUNKED) {
      __syncthreads();
      form(lo, min(v1, lo + kSlice), cm, ca);
    }
    exponentials(lo, min(v1, lo + kSlice));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (lane == 0) s_m[warp] = sum;
  __syncthreads();
  sum = s_m[lane % (kThreads / 32)];
#pragma unroll
  for (int o = kThreads / 64; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);

  // the row's maximum M, its first place, its sum; factor: from the slice's exponentials to probabilities
  float M = m;
  int first = at;
  if (C > 1) {
    if (tid == 0) s_stat = Stat{m, at, sum};
    cluster_arrive();
    cluster_wait();
    // every warp reads all CTAs' values itself: lane k those of CTA k
    float pm = -INFINITY, ps = 0.f;
    int pa = 0x7FFFFFFF;
    if (lane < C) { pm = peer(&s_stat.m, lane); pa = peer(&s_stat.at, lane); ps = peer(&s_stat.sum, lane); }
    cluster_arrive();   // this CTA has read its peers' shared memory (waited for before it ends)
    M = pm;
    first = pa;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float m2 = __shfl_xor_sync(0xFFFFFFFFu, M, o);
      const int at2 = __shfl_xor_sync(0xFFFFFFFFu, first, o);
      if (m2 > M || (m2 == M && at2 < first)) { M = m2; first = at2; }
    }
    sum = pm == M ? ps : ps * ex2((pm - M) * scale);
    if (ps == 0.f) sum = 0.f;                          // (no largest in the slice: the difference is no number)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  }
  const bool none = M == -INFINITY;
  if (a.top && rank == 0 && tid == 0) a.top[r] = none ? -1 : first;
  const float factor = none || m == -INFINITY ? 0.f : (m == M ? 1.f : ex2((m - M) * scale)) / sum;

  const int64_t p_row = (int64_t)r * V;
  auto write = [&](int lo, int hi) {
    const int n = hi - lo, mis = misplaced(a.x, x_row + lo, kLogitBytes), groups = (mis + n + 3) / 4;
    if (greedy || factor == 0.f) {                     // (0 times what is not a weight is not 0)
      for (int k = tid; k < n; k += kThreads) a.probs[p_row + lo + k] = greedy && !none && lo + k == first ? 1.f : 0.f;
      return;
    }
    const bool whole = misplaced(a.probs, p_row + lo, 4) == mis;
    float* out = a.probs + p_row + lo - mis;
    if (whole) {
#pragma unroll 4
      for (int q = tid; q < groups; q += kThreads) {
        const int k = 4 * q - mis;
        float4 e = reinterpret_cast<const float4*>(xs)[q];
        e = make_float4(e.x * factor, e.y * factor, e.z * factor, e.w * factor);
        if (k >= 0 && k + 3 < n) {
          __stcs(reinterpret_cast<float4*>(out) + q, e);
        } else {
          if (k >= 0) out[4 * q] = e.x;
          if (k + 1 >= 0 && k + 1 < n) out[4 * q + 1] = e.y;
          if (k + 2 >= 0 && k + 2 < n) out[4 * q + 2] = e.z;
          if (k + 3 < n) out[4 * q + 3] = e.w;
        }
      }
    } else {
#pragma unroll 8
      for (int k = tid; k < n; k += kThreads) __stcs(a.probs + p_row + lo + k, xs[mis + k] * factor);
    }
  };
  for (int lo = v0; lo < v1; lo += kSlice) {
    if (CHUNKED) {
      float cm;
      int ca;
      __syncthreads();
      form(lo, min(v1, lo + kSlice), cm, ca);
      exponentials(lo, min(v1, lo + kSlice));
      __syncthreads();
    }
    write(lo, min(v1, lo + kSlice));
  }
  if (C > 1) cluster_wait();
}

// CTAs per row: enough to hold the row; more, down to kLeast values each, while the rows alone leave SMs idle.
static uint32_t cluster_for(int rows, int V) {
  constexpr int kLeast = 2048;
  uint32_t c = 1;
  while (c < kMaxCluster && ((int64_t)c * kSlice < V || ((int64_t)rows * c < 152 && (int64_t)c * kLeast < V))) c *= 2;
  return c;
}

template <int T, bool CHUNKED>
static moe_status_t launch(const Args& a, int rows, uint32_t C, cudaStream_t stream) {
  auto* kernel = probs_kernel<T, CHUNKED>;
  static int configured[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MOE_ERR_CUDA;
  if (!configured[dev]) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSlice * 4 + 16) != cudaSuccess ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
      return MOE_ERR_CUDA;
    configured[dev] = 1;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(rows * C);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)(a.slice < kSlice ? a.slice : kSlice) * 4 + 16;
  cfg.stream = stream;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = C;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = C > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a, C) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
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
  if (l->n_seqs < 1 || l->rows_per_seq < 1 || l->rows_per_seq > logits::kMaxRows ||
      (int64_t)l->n_seqs * l->rows_per_seq >= 65536 || l->vocab < 1 || l->vocab > (1 << 22) || l->logits_stride < l->vocab ||
      (l->allowed && l->allowed_stride < (l->vocab + 31) / 32))
    return MOE_ERR_SHAPE;
  if ((const void*)probs == l->logits && (l->type != MOE_LOGITS_F32 || l->logits_stride != l->vocab)) return MOE_ERR_INVALID_ARG;
  moe_status_t st = moe_check_device();
  if (st != MOE_OK) return st;
  const int rows = l->n_seqs * l->rows_per_seq;
  const uint32_t C = logits::cluster_for(rows, l->vocab);
  const int slice = (int)(((int64_t)l->vocab + C - 1) / C + 31) / 32 * 32;
  const logits::Args a{l->logits, l->logits_stride, l->vocab, l->rows_per_seq, slice, l->params, l->counts,
                       l->counts && l->rows_per_seq > 1 ? l->draft : nullptr, l->bias_start, l->bias_id, l->bias_value,
                       l->allowed, l->allowed_stride, probs, top};
  const bool f32 = l->type == MOE_LOGITS_F32, chunked = slice > logits::kSlice;
  cudaStream_t s = (cudaStream_t)stream;
  if (chunked)
    return f32 ? logits::launch<MOE_LOGITS_F32, true>(a, rows, C, s) : logits::launch<MOE_LOGITS_BF16, true>(a, rows, C, s);
  return f32 ? logits::launch<MOE_LOGITS_F32, false>(a, rows, C, s) : logits::launch<MOE_LOGITS_BF16, false>(a, rows, C, s);
}
