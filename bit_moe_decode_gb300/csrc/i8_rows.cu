// i8_rows.cu -- rows to 8 bits with a scale each: of any matrix (moe_i8_quantize), or of the residual stream after its
// addition and RMS norm (moe_rms_norm_i8); and the values that such rows stand for (moe_i8_values).
//
//   s = h + r,  v = s g,  rho = 1 / sqrt(mean s^2 + eps),  a = max |v|:  q = 127 v / a,  scale = a rho / 127,  x = bf16(v rho).
// rho is a row's common factor, so it cancels in q: the codes need only the row's maximum, and one pass over the data with one
// reduction of (sum of squares, maximum) does all. q is the rounding of the real quotient: fp32 gives 127 v / a within
// 2^-16, and what lies that near to a border between two codes (one value in 16,000) is compared in 64 bits, where 127 v and
// (code + 1/2) a are exact. So the codes depend on no order of sums.
//
// One CTA a row, eight values a thread and vector, held in registers between the reduction and the outputs: each byte is read
// and written once. The threads of a row follow from its length alone, so that a token's sum has the same order whatever
// the other tokens are.
#include <type_traits>

#include "i8.cuh"

namespace moe {
namespace i8 {

constexpr float kFloor = 7.888609052210118e-31f;    // 2^-100
constexpr float kNear = 3.0517578125e-05f;          // 2^-15

struct RowArgs {
  const void *h, *r;
  const float* gain;
  void* h_out;
  uint16_t* x;
  int8_t* q;
  float* scale;
  int64_t h_stride, r_stride, out_stride, q_stride;
  int cols;
  float eps;
};

template <typename T> struct Vec8;
template <> struct Vec8<float> {
  static __device__ __forceinline__ void load(const float* p, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&v)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
};
template <> struct Vec8<__nv_bfloat16> {
  static __device__ __forceinline__ void load(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
struct None {};

// The code of v in a row with maximum a; t = v (127 / a) in fp32, within 2^-16 of the real 127 v / a.
__device__ __forceinline__ int code_of(float v, float a, float t) {
  const float k = rintf(t);
  if (fabsf(fabsf(t - k) - 0.5f) >= kNear) return (int)k;
  const float f = floorf(t);
  const double x = 127.0 * (double)v, border = ((double)f + 0.5) * (double)a;   // both exact
  const int lo = (int)f;
  return x > border || (x == border && (lo & 1)) ? lo + 1 : lo;
}
__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
  uint32_t w;
  asm("{\n\t.reg .b32 t;\n\tcvt.pack.sat.s8.s32.b32 t, %4, %3, 0;\n\tcvt.pack.sat.s8.s32.b32 %0, %2, %1, t;\n\t}"
      : "=r"(w)
      : "r"(a), "r"(b), "r"(c), "r"(d));
  return w;
}

// The block's sum of `sum` (a fixed order) and maximum of `top`; part: 64 words.
__device__ __forceinline__ void reduce(float& sum, uint32_t& top, uint32_t* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();   // (an earlier reduction's values may still be read)
  if (lane == 0) {
    part[warp] = __float_as_uint(sum);
    part[32 + warp] = top;
  }
  __syncthreads();
  sum = lane < warps ? __uint_as_float(part[lane]) : 0.f;
  top = __reduce_max_sync(0xFFFFFFFFu, lane < warps ? part[32 + lane] : 0u);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
}

// TR None: no addition. NORM false: only the codes and scales of h. V vectors of eight a thread.
template <typename TH, typename TR, bool NORM, int V>
__global__ void __launch_bounds__(1024) rows_kernel(RowArgs a) {
  __shared__ uint32_t part[64];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, n = a.cols >> 3;
  const TH* h = (const TH*)a.h + row * a.h_stride;
  float v[V][8];
  float sum = 0.f, big = 0.f, small = 0.f;   // of squares: plain, of s 2^-80, of s 2^80
  uint32_t top = 0;                          // |v|'s bits: infinities and NaN are the largest
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = tid + j * blockDim.x;
    if (i < n) {
      Vec8<TH>::load(h + 8 * i, v[j]);
      if (NORM) {
        if constexpr (!std::is_same<TR, None>::value) {
          float r[8];
          Vec8<TR>::load((const TR*)a.r + row * a.r_stride + 8 * i, r);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[j][e] = __fadd_rn(v[j][e], r[e]);
        }
        if (a.h_out) Vec8<TH>::store((TH*)a.h_out + row * a.out_stride + 8 * i, v[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          sum = fmaf(v[j][e], v[j][e], sum);
          const float b = v[j][e] * 0x1p-80f, s = v[j][e] * 0x1p80f;
          big = fmaf(b, b, big);
          small = fmaf(s, s, small);
        }
        if (a.gain) {
          float g[8];
          Vec8<float>::load(a.gain + 8 * i, g);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[j][e] = __fmul_rn(v[j][e], g[e]);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[j][e]) & 0x7FFFFFFFu);
    }
  }
  reduce(sum, top, part);
  const bool bad = top >= 0x7F800000u;
  const float amax = fmaxf(__uint_as_float(top), kFloor);
  float rho = 1.f;
  if (NORM) {
    // the plain sum, unless it overflowed or lost what small squares weigh (the same choice for the whole row)
    const float n = (float)a.cols;
    if (sum > 3e38f) {
      reduce(big, top, part);
      rho = __fdiv_rn(0x1p-80f, __fsqrt_rn(__fdiv_rn(big, n) + a.eps * 0x1p-80f * 0x1p-80f));
    } else if (sum < 0x1p-100f && a.eps < 0x1p-60f) {
      reduce(small, top, part);
      rho = __fdiv_rn(0x1p80f, __fsqrt_rn(__fdiv_rn(small, n) + a.eps * 0x1p80f * 0x1p80f));
    } else {
      rho = __fdiv_rn(1.f, __fsqrt_rn(__fdiv_rn(sum, n) + a.eps));
    }
  }
  if (NORM && a.x) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = tid + j * blockDim.x;
      if (i < n) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __fmul_rn(v[j][e], rho);
        Vec8<__nv_bfloat16>::store((__nv_bfloat16*)a.x + row * a.cols + 8 * i, x);
      }
    }
  }
  if (!NORM || a.q) {
    const float inv = __fdiv_rn(127.f, amax);
    if (tid == 0) a.scale[row] = bad ? __uint_as_float(0x7FC00000u) : __fdiv_rn(NORM ? __fmul_rn(amax, rho) : amax, 127.f);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = tid + j * blockDim.x;
      if (i < n) {
        int q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = bad ? 0 : code_of(v[j][e], amax, __fmul_rn(v[j][e], inv));
        *reinterpret_cast<uint2*>(a.q + row * a.q_stride + 8 * i) =
            make_uint2(pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7]));
      }
    }
  }
}

// Rows too long for registers: the row is read twice.
template <typename T>
__global__ void __launch_bounds__(1024) long_rows_kernel(RowArgs a) {
  __shared__ uint32_t part[64];
  const int64_t row = blockIdx.x;
  const int n = a.cols >> 3;
  const T* h = (const T*)a.h + row * a.h_stride;
  float sum = 0.f;
  uint32_t top = 0;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    float v[8];
    Vec8<T>::load(h + 8 * i, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
  }
  reduce(sum, top, part);
  const bool bad = top >= 0x7F800000u;
  const float amax = fmaxf(__uint_as_float(top), kFloor), inv = __fdiv_rn(127.f, amax);
  if (threadIdx.x == 0) a.scale[row] = bad ? __uint_as_float(0x7FC00000u) : __fdiv_rn(amax, 127.f);
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    float v[8];
    int q[8];
    Vec8<T>::load(h + 8 * i, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = bad ? 0 : code_of(v[e], amax, __fmul_rn(v[e], inv));
    *reinterpret_cast<uint2*>(a.q + row * a.q_stride + 8 * i) = make_uint2(pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7]));
  }
}

// 512 codes of a row a warp
__global__ void __launch_bounds__(256) values_kernel(const int8_t* q, int64_t stride, const float* scale, float* out, int rows,
                                                    int cols) {
  const int per_row = (cols + 511) / 512, lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t row = item / per_row;
  if (row >= rows) return;
  const int first = (int)(item - row * per_row) * 512 + 4 * lane;
  const float s = scale[row];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int c = first + 128 * k;
    if (c < cols) {
      const char4 w = *reinterpret_cast<const char4*>(q + row * stride + c);
      *reinterpret_cast<float4*>(out + row * cols + c) =
          make_float4(__fmul_rn((float)w.x, s), __fmul_rn((float)w.y, s), __fmul_rn((float)w.z, s), __fmul_rn((float)w.w, s));
    }
  }
}

template <typename TH, typename TR, bool NORM>
static moe_status_t launch_rows(const RowArgs& a, int rows, cudaStream_t st) {
  const int vecs = a.cols / 8;
  const int per = vecs <= 1024 ? 1 : vecs <= 2048 ? 2 : 4;
  const int threads = ((vecs + per - 1) / per + 31) / 32 * 32;
  if (per == 1) rows_kernel<TH, TR, NORM, 1><<<rows, threads, 0, st>>>(a);
  else if (per == 2) rows_kernel<TH, TR, NORM, 2><<<rows, threads, 0, st>>>(a);
  else rows_kernel<TH, TR, NORM, 4><<<rows, threads, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

static bool type_ok(moe_type_t t) { return t == MOE_TYPE_F32 || t == MOE_TYPE_BF16; }
static int64_t size_of(moe_type_t t) { return t == MOE_TYPE_F32 ? 4 : 2; }
// a matrix's pointer and row stride: 16-byte aligned, rows at least `cols` wide
static bool rows_ok(const void* p, int64_t stride, int64_t cols, moe_type_t t) {
  return ((uintptr_t)p & 15) == 0 && stride >= cols && stride * size_of(t) % 16 == 0;
}

}  // namespace i8
}  // namespace moe

using namespace moe;
using namespace moe::i8;

extern "C" moe_status_t moe_i8_quantize(moe_type_t type, const void* src, int64_t src_stride, const moe_i8_rows_t* dst,
                                        void* stream) {
  MOE_NVTX("moe_i8_quantize");
  if (moe_internal::fault("i8_quantize")) return MOE_ERR_FAULT_INJECTED;
  if (!src || !type_ok(type)) return MOE_ERR_INVALID_ARG;
  moe_status_t st = check_rows(dst);
  if (st != MOE_OK) return st;
  if (!rows_ok(src, src_stride, dst->cols, type)) return MOE_ERR_INVALID_ARG;
  st = moe_check_device();
  if (st != MOE_OK) return st;
  RowArgs a{};
  a.h = src;
  a.h_stride = src_stride;
  a.q = dst->q;
  a.q_stride = dst->stride;
  a.scale = dst->scale;
  a.cols = dst->cols;
  cudaStream_t s = (cudaStream_t)stream;
  if (dst->cols <= 32768) {
    if (type == MOE_TYPE_F32) return launch_rows<float, None, false>(a, dst->rows, s);
    return launch_rows<__nv_bfloat16, None, false>(a, dst->rows, s);
  }
  if (type == MOE_TYPE_F32) long_rows_kernel<float><<<dst->rows, 1024, 0, s>>>(a);
  else long_rows_kernel<__nv_bfloat16><<<dst->rows, 1024, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" moe_status_t moe_i8_values(const moe_i8_rows_t* src, float* out, void* stream) {
  MOE_NVTX("moe_i8_values");
  if (moe_internal::fault("i8_values")) return MOE_ERR_FAULT_INJECTED;
  moe_status_t st = check_rows(src);
  if (st != MOE_OK) return st;
  if (!out || ((uintptr_t)out & 15)) return MOE_ERR_INVALID_ARG;
  st = moe_check_device();
  if (st != MOE_OK) return st;
  const int64_t items = (int64_t)src->rows * ((src->cols + 511) / 512);
  values_kernel<<<(unsigned)((items + 7) / 8), 256, 0, (cudaStream_t)stream>>>(src->q, src->stride, src->scale, out, src->rows,
                                                                              src->cols);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" moe_status_t moe_rms_norm_i8(const moe_norm_t* p, const moe_i8_rows_t* xq, void* stream) {
  MOE_NVTX("moe_rms_norm_i8");
  if (moe_internal::fault("norm_i8")) return MOE_ERR_FAULT_INJECTED;
  if (!p || !p->h || (!p->x_bf16 && !xq) || !type_ok(p->h_type) || (p->r && !type_ok(p->r_type))) return MOE_ERR_INVALID_ARG;
  if (p->tokens < 1 || p->tokens > kMaxRows || p->hidden < 16 || p->hidden > 32768 || p->hidden % 16 || !(p->eps >= 0.f))
    return MOE_ERR_SHAPE;
  if (xq) {
    const moe_status_t st = check_rows(xq);
    if (st != MOE_OK) return st;
    if (xq->rows != p->tokens || xq->cols != p->hidden) return MOE_ERR_SHAPE;
  }
  if (!rows_ok(p->h, p->h_stride, p->hidden, p->h_type) || (p->r && !rows_ok(p->r, p->r_stride, p->hidden, p->r_type)) ||
      (p->h_out && !rows_ok(p->h_out, p->h_out_stride, p->hidden, p->h_type)) || ((uintptr_t)p->gain & 15) ||
      ((uintptr_t)p->x_bf16 & 15))
    return MOE_ERR_INVALID_ARG;
  moe_status_t st = moe_check_device();
  if (st != MOE_OK) return st;
  RowArgs a{p->h, p->r, p->gain, p->h_out, (uint16_t*)p->x_bf16, xq ? xq->q : nullptr, xq ? xq->scale : nullptr,
            p->h_stride, p->r_stride, p->h_out_stride, xq ? xq->stride : 0, p->hidden, p->eps};
  cudaStream_t s = (cudaStream_t)stream;
  const int kind = (p->h_type == MOE_TYPE_BF16 ? 3 : 0) + (!p->r ? 0 : p->r_type == MOE_TYPE_F32 ? 1 : 2);
  switch (kind) {
    case 0: return launch_rows<float, None, true>(a, p->tokens, s);
    case 1: return launch_rows<float, float, true>(a, p->tokens, s);
    case 2: return launch_rows<float, __nv_bfloat16, true>(a, p->tokens, s);
    case 3: return launch_rows<__nv_bfloat16, None, true>(a, p->tokens, s);
    case 4: return launch_rows<__nv_bfloat16, float, true>(a, p->tokens, s);
    default: return launch_rows<__nv_bfloat16, __nv_bfloat16, true>(a, p->tokens, s);
  }
}
