// i8_matmul.cu -- product of 8-bit integers with scales for each token and output channel, and the gated block.
#include "i8.cuh"

namespace moe {
namespace i8 {

// 64 channels x 64 tokens a CTA, 64 of K at a time; a thread has 4 x 4 of them (channels tid % 16 + 16 i, tokens tid / 16 + 16 j)
template <bool GATED>
__global__ void __launch_bounds__(256) tile_kernel(MatArgs a) {
  constexpr int P = 17;   // words a row of 64 codes takes in shared memory
  __shared__ uint32_t sx[64 * P], sw[GATED ? 2 : 1][64 * P];
  const int tid = threadIdx.x, cn = tid & 15, ct = tid >> 4;
  const int n0 = blockIdx.x * 64, t0 = blockIdx.y * 64;
  int acc[GATED ? 2 : 1][4][4] = {};
  for (int k0 = 0; k0 < a.K; k0 += 64) {
    const int row = tid >> 2, k = k0 + 16 * (tid & 3);
    __syncthreads();
    auto fill = [&](uint32_t* to, const int8_t* from, int64_t stride, int r, int rows) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (r < rows && k < a.K) v = *reinterpret_cast<const uint4*>(from + r * stride + k);
      uint32_t* p = to + row * P + 4 * (tid & 3);
      p[0] = v.x; p[1] = v.y; p[2] = v.z; p[3] = v.w;
    };
    fill(sx, a.x, a.x_stride, t0 + row, a.T);
    fill(sw[0], a.w[0], a.w_stride[0], n0 + row, a.N);
    if (GATED) fill(sw[GATED], a.w[1], a.w_stride[1], n0 + row, a.N);
    __syncthreads();
#pragma unroll 4
    for (int kk = 0; kk < 16; ++kk) {
      int xv[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) xv[j] = (int)sx[(ct + 16 * j) * P + kk];
#pragma unroll
      for (int m = 0; m < (GATED ? 2 : 1); ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int wv = (int)sw[m][(cn + 16 * i) * P + kk];
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[m][i][j] = __dp4a(wv, xv[j], acc[m][i][j]);
        }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + cn + 16 * i, t = t0 + ct + 16 * j;
      if (n >= a.N || t >= a.T) continue;
      const float xs = a.xs[t], p = product(acc[0][i][j], xs, a.ws[0][n]);
      put(a, t, n, GATED ? silu_mul(p, product(acc[GATED ? 1 : 0][i][j], xs, a.ws[1][n])) : p);
    }
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
  if (a.T > 8) return tc_multiply(a, (cudaStream_t)stream);
  const dim3 grid((a.N + 63) / 64, (a.T + 63) / 64);
  if (w2) tile_kernel<true><<<grid, 256, 0, (cudaStream_t)stream>>>(a);
  else tile_kernel<false><<<grid, 256, 0, (cudaStream_t)stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
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
