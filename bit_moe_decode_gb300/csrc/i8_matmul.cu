// i8_matmul.cu -- product of 8-bit integers with scales for each token and output channel, and the gated block: the entry points,
// and the kernel for a few tokens (i8_tc.cu has the one for more).
//
// A few tokens: the weights are read once, and that is all the time there is. They go from global memory straight into registers, 16
// channels a CTA at a time, whose 8 warps share K; codes become binary16 (exactly) and mma.sync (m16n8k16) multiplies them with
// the tokens, which the CTA keeps in shared memory in binary16. fp32 adds 1024 products exactly; then the accumulators are
// added to integers. The order of k within a block is the one in which a lane gets its codes: 16 contiguous bytes of two rows.
// Gated: rows 0-7 of the 16 are gate's, 8-15 up's of the same channels, so that a thread has both.
#include "i8.cuh"

namespace moe {
namespace i8 {

constexpr int kRowThreads = 256, kRowWarps = 8;
constexpr int kAhead = 2;                     // blocks of 128 codes of 16 rows that a warp has in flight
constexpr int kExactBlocks = 8;               // blocks whose products fp32 adds exactly

__device__ __forceinline__ uint4 load_codes(const int8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// NT tiles of 8 tokens. x in shared memory: T rows of `pitch` bytes (2 K rounded up to 256, and 16).
template <bool GATED, int NT>
__global__ void __launch_bounds__(kRowThreads, NT == 1 ? 3 : 2) rows_kernel(MatArgs a, int groups) {
  extern __shared__ uint8_t smem[];
  __shared__ int part[kRowWarps][16 * 8 * NT];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int blocks = (a.K + 127) / 128, pitch = blocks * 256 + 16;
  const int mine = (blocks - warp + kRowWarps - 1) / kRowWarps;           // blocks of a group that this warp has (may be <= 0)
  const int channels = GATED ? 8 : 16;

  // ---- the next block of the warp's list (group after group): four pieces of 16 codes
  uint4 buf[kAhead][4];
  int lg = blockIdx.x, lb = 0;
  auto fetch = [&](uint4 (&v)[4]) {
    if (lg < groups && mine > 0) {
      const int n0 = lg * channels + g, k = (warp + lb * kRowWarps) * 128 + 16 * c;
      const int r0 = min(n0, a.N - 1), r1 = min(GATED ? n0 : n0 + 8, a.N - 1);
      const int8_t *p0 = a.w[0] + r0 * a.w_stride[0] + k, *p1 = a.w[GATED ? 1 : 0] + r1 * a.w_stride[GATED ? 1 : 0] + k;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool in = k + 64 * h < a.K;
        v[2 * h] = in ? load_codes(p0 + 64 * h) : make_uint4(0, 0, 0, 0);
        v[2 * h + 1] = in ? load_codes(p1 + 64 * h) : make_uint4(0, 0, 0, 0);
      }
      if (++lb == mine) { lb = 0; lg += gridDim.x; }
    }
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) fetch(buf[i]);

  // ---- the tokens, in convert4's order
  const int pieces = blocks * 8;
  for (int i = tid; i < a.T * pieces; i += kRowThreads) {
    const int t = i / pieces, k = (i - t * pieces) * 16;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (k < a.K) v = *reinterpret_cast<const uint4*>(a.x + t * a.x_stride + k);
    uint32_t h[8];
    convert4(v.x, h[0], h[1]);
    convert4(v.y, h[2], h[3]);
    convert4(v.z, h[4], h[5]);
    convert4(v.w, h[6], h[7]);
    uint4* to = reinterpret_cast<uint4*>(smem + t * pitch + k * 2);
    to[0] = make_uint4(h[0], h[1], h[2], h[3]);
    to[1] = make_uint4(h[4], h[5], h[6], h[7]);
  }
  __syncthreads();
  const uint8_t* xr[NT];                     // (columns past the last token repeat it and are not used)
#pragma unroll
  for (int t = 0; t < NT; ++t) xr[t] = smem + min(8 * t + g, a.T - 1) * pitch + c * 32;

  for (int group = blockIdx.x; group < groups; group += gridDim.x) {
    float acc[NT][4] = {};
    int sum[NT][4] = {};
    auto add = [&]() {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sum[t][e] += __float2int_rn(acc[t][e]);
          acc[t][e] = 0.f;
        }
    };
    for (int i = 0; i < mine; i += kAhead) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (i + j < mine) {
          const int at = (warp + (i + j) * kRowWarps) * 256;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t w0[8], w1[8];
            const uint4 v0 = buf[j][2 * h], v1 = buf[j][2 * h + 1];
            convert4(v0.x, w0[0], w0[1]);
            convert4(v0.y, w0[2], w0[3]);
            convert4(v0.z, w0[4], w0[5]);
            convert4(v0.w, w0[6], w0[7]);
            convert4(v1.x, w1[0], w1[1]);
            convert4(v1.y, w1[2], w1[3]);
            convert4(v1.z, w1[4], w1[5]);
            convert4(v1.w, w1[6], w1[7]);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const uint4 b0 = *reinterpret_cast<const uint4*>(xr[t] + at + 128 * h), b1 = *reinterpret_cast<const uint4*>(xr[t] + at + 128 * h + 16);
              mma_f16(acc[t], w0[0], w1[0], w0[1], w1[1], b0.x, b0.y, acc[t]);
              mma_f16(acc[t], w0[2], w1[2], w0[3], w1[3], b0.z, b0.w, acc[t]);
              mma_f16(acc[t], w0[4], w1[4], w0[5], w1[5], b1.x, b1.y, acc[t]);
              mma_f16(acc[t], w0[6], w1[6], w0[7], w1[7], b1.z, b1.w, acc[t]);
            }
          }
          fetch(buf[j]);
          if ((i + j) % kExactBlocks == kExactBlocks - 1) add();
        }
    }
    // (the ring's first place has the next group's first block only if this one's count is a multiple of the ring's)
    if (mine > 0 && mine % kAhead != 0) {
#pragma unroll
      for (int j = 0; j < kAhead - 1; ++j) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint4 v = buf[0][e];
          buf[0][e] = buf[1][e];
          buf[1][e] = v;
        }
      }
    }
    add();
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) part[warp][(8 * t + 2 * c + (e & 1)) * 16 + g + 8 * (e >> 1)] = sum[t][e];
    __syncthreads();
    for (int i = tid; i < channels * a.T; i += kRowThreads) {
      const int t = i / channels, r = i % channels, n = group * channels + r;
      int s0 = 0, s1 = 0;
#pragma unroll
      for (int w = 0; w < kRowWarps; ++w) {
        s0 += part[w][t * 16 + r];
        if (GATED) s1 += part[w][t * 16 + 8 + r];
      }
      if (n < a.N) {
        const float xs = a.xs[t], p = product(s0, xs, a.ws[0][n]);
        put(a, t, n, GATED ? silu_mul(p, product(s1, xs, a.ws[GATED ? 1 : 0][n])) : p);
      }
    }
    __syncthreads();
  }
}

// MOE_OK, or MOE_ERR_SHAPE: the tokens do not fit.
static bool rows_fit(int T, int K) { return T <= 16 && (int64_t)T * ((K + 127) / 128 * 256 + 16) <= (T <= 8 ? 72 : 100) * 1024; }
template <bool GATED, int NT>
static moe_status_t launch_rows(const MatArgs& a, int sms, cudaStream_t stream) {
  const int groups = (a.N + (GATED ? 7 : 15)) / (GATED ? 8 : 16);
  const int smem = a.T * ((a.K + 127) / 128 * 256 + 16), fit = min(NT == 1 ? 3 : 2, 220 * 1024 / (smem + 8192 * NT));
  rows_kernel<GATED, NT><<<min(groups, sms * fit), kRowThreads, smem, stream>>>(a, groups);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
static moe_status_t rows_multiply(const MatArgs& a, cudaStream_t stream) {
  static int configured[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MOE_ERR_CUDA;
  if (!configured[dev]) {
    const int most = 104 * 1024;
    if (cudaFuncSetAttribute(rows_kernel<false, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess ||
        cudaFuncSetAttribute(rows_kernel<true, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess ||
        cudaFuncSetAttribute(rows_kernel<false, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess ||
        cudaFuncSetAttribute(rows_kernel<true, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess) {
      cudaGetLastError();
      return MOE_ERR_CUDA;
    }
    configured[dev] = 1;
  }
  const int sms = moe_internal::num_sms();
  if (sms <= 0) return MOE_ERR_CUDA;
  if (a.w[1]) return a.T <= 8 ? launch_rows<true, 1>(a, sms, stream) : launch_rows<true, 2>(a, sms, stream);
  return a.T <= 8 ? launch_rows<false, 1>(a, sms, stream) : launch_rows<false, 2>(a, sms, stream);
}

static bool out_ok(const void* p, int64_t stride, int64_t cols, int size) {
  return !p || (((uintptr_t)p & (size - 1)) == 0 && stride >= cols);
}

static moe_status_t multiply(const moe_i8_rows_t* x, const moe_i8_rows_t* w, const moe_i8_rows_t* w2, const float* base,
                             int64_t base_stride, float* y, int64_t y_stride, void* y_bf16, int64_t yb_stride, void* ws,
                             size_t ws_bytes, void* stream) {
  moe_status_t st = check_rows(x);
  if (st == MOE_OK) st = check_rows(w);
  if (st == MOE_OK && w2) st = check_rows(w2);
  if (st != MOE_OK) return st;
  if ((!y && !y_bf16) || !ws || ((uintptr_t)ws & 255)) return MOE_ERR_INVALID_ARG;
  if (x->cols != w->cols || (w2 && (w2->cols != w->cols || w2->rows != w->rows))) return MOE_ERR_SHAPE;
  if (!out_ok(base, base_stride, w->rows, 4) || !out_ok(y, y_stride, w->rows, 4) || !out_ok(y_bf16, yb_stride, w->rows, 2))
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < moe_i8_workspace_bytes(w, x->rows)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  st = moe_check_device();
  if (st != MOE_OK) return st;
  MatArgs a{x->q, {w->q, w2 ? w2->q : nullptr}, x->scale, {w->scale, w2 ? w2->scale : nullptr}, base, y, (uint16_t*)y_bf16,
            x->stride, {w->stride, w2 ? w2->stride : 0}, base_stride, y_stride, yb_stride, x->rows, w->rows, x->cols, (int32_t*)ws};
  return rows_fit(a.T, a.K) ? rows_multiply(a, (cudaStream_t)stream) : tc_multiply(a, (cudaStream_t)stream);
}

}  // namespace i8
}  // namespace moe

using namespace moe;
using namespace moe::i8;

extern "C" size_t moe_i8_workspace_bytes(const moe_i8_rows_t* w, int32_t T_max) {
  if (check_rows(w) != MOE_OK || T_max < 1 || T_max > kMaxRows) return 0;
  return sizeof(WsHeader) + tc_workspace_bytes(w->cols, T_max);
}

extern "C" moe_status_t moe_i8_matmul(const moe_i8_rows_t* x, const moe_i8_rows_t* w, const float* base, int64_t base_stride,
                                      float* y, int64_t y_stride, void* y_bf16, int64_t yb_stride, void* ws, size_t ws_bytes,
                                      void* stream) {
  MOE_NVTX("moe_i8_matmul");
  if (moe_internal::fault("i8_matmul")) return MOE_ERR_FAULT_INJECTED;
  return multiply(x, w, nullptr, base, base_stride, y, y_stride, y_bf16, yb_stride, ws, ws_bytes, stream);
}

extern "C" moe_status_t moe_i8_gated(const moe_i8_rows_t* x, const moe_i8_rows_t* gate, const moe_i8_rows_t* up, float* y,
                                     int64_t y_stride, void* y_bf16, int64_t yb_stride, void* ws, size_t ws_bytes, void* stream) {
  MOE_NVTX("moe_i8_gated");
  if (moe_internal::fault("i8_gated")) return MOE_ERR_FAULT_INJECTED;
  if (!up) return MOE_ERR_INVALID_ARG;
  return multiply(x, gate, up, nullptr, 0, y, y_stride, y_bf16, yb_stride, ws, ws_bytes, stream);
}
