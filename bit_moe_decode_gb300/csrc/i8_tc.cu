// i8_tc.cu -- product of 8-bit integers (and the gated block) for more than a few tokens, on tcgen05.
//
// GB300's tensor cores multiply 8-bit integers at a small fraction of their 16-bit rate, but binary16 holds every code
// exactly, and a product of two codes is at most 2^14: kind::f16 with fp32 accumulators adds 1024 of them without rounding
// (2^24). So codes are converted to binary16 on their way to the tensor cores, and every 1024 of K at the latest the
// accumulators are added to integers in registers: the sums are exact whatever the codes are.
//
//   D [128 channels x nt tokens] += W [128 x 64] X^T [64 x nt]: channels are the rows of the product, so that a weight's tile
//   goes from shared memory through a warpgroup's registers straight into TMEM (operand A; lane = channel) and is not written to
//   shared memory again. X is converted into a swizzled shared memory operand (B).
//
// A CTA has 256 channels: two blocks of 128 (gated: 128 of gate and the same 128 of up), each with a warpgroup that converts its
// weights, adds up its accumulators and writes its outputs, and with a warp of its own that issues its products. The blocks'
// sums are taken out 512 of K apart, so that one block's products run while the other's accumulators are read.
// One warpgroup converts X for both, one warp copies packed tiles (TMA, 128 of K a stage).
//
// Few channels: a cluster of CTAs shares a tile, each takes a part of K; the integer parts are exchanged through distributed
// shared memory, each CTA finishing some of the tokens. Many tiles: CTAs go from one to the next, outputs of one tile being
// written while the tensor cores work on the next.
#include "i8.cuh"
#include "tcgen05.cuh"

namespace moe {
namespace i8 {

constexpr int kThreads = 512;
constexpr int kMaxTokens = 128;        // of a tile
constexpr int kTileK = 128;            // K of a stage of packed codes; two steps of 64
constexpr int kSlots = 4;              // converted steps in flight
constexpr int kSegment = 16;           // steps that fp32 adds exactly
constexpr int kMaxStages = 8;
constexpr uint32_t kTmemA = 256;       // columns: accumulators of the blocks at 0 and 128, then [block][slot] 32 columns of A
constexpr int kXchgTokens = 8;         // tokens that the blocks of a gated tile exchange at a time
constexpr int kXchgBytes = 2 * 2 * kXchgTokens * 128 * 4;
constexpr int kSmemLimit = 232448 - 1024;    // (1 KB for alignment and the static part)

struct TcArgs {
  MatArgs m;
  int nt;              // tokens of a tile: a multiple of 16
  int tiles_n, tiles;  // tiles of 256 channels (gated: 128), times the tiles of nt tokens
  int split;           // CTAs (a cluster) that share a tile
  int stages;
};

__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(
          d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// binary16 x binary16 -> fp32, M = 128, B K-major
__device__ __forceinline__ uint32_t idesc_f16(uint32_t n) { return (1u << 4) | ((n >> 3) << 17) | (8u << 24); }
__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr), "r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
      "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
template <int N> __device__ __forceinline__ void regs_more() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void regs_less() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void st_peer(uint32_t addr, uint32_t rank, uint32_t v) {
  asm volatile("{\n\t.reg .b32 p;\n\tmapa.shared::cluster.u32 p, %0, %1;\n\tst.shared::cluster.u32 [p], %2;\n\t}" ::"r"(addr), "r"(rank),
               "r"(v)
               : "memory");
}
__device__ __forceinline__ uint4 ld_shared(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Four codes (one word) -> binary16, exactly: a byte under the exponent of 1024, sign bit flipped, is 1024 + 128 + code. The order
// is codes 0, 2, 1, 3 (a shift instead of two permutations); W and X have the same, so the sums are those of the same products.
__device__ __forceinline__ void convert4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t a = lop3_and_xor(w, 0x00FF00FFu, 0x64806480u), b = lop3_and_xor(w >> 8, 0x00FF00FFu, 0x64806480u);
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0xE480E480u));     // - 1152
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0xE480E480u));
}

// The rest of a wait: true if it ran out. (Inlined: a call would hold registers that the warpgroups' split has not left.)
__device__ __forceinline__ bool wait_longer(uint64_t* bar, int parity, int32_t* status) {
  const long long t0 = globaltimer_ns();
  for (uint32_t n = 1; !mbar_try_wait(bar, parity); ++n)
    if (n % 64 == 0 && globaltimer_ns() - t0 > kDefaultWaitNs) {
      record_error(status, MOE_ERR_DEVICE_TIMEOUT);
      return true;
    }
  return false;
}

// Step i of `steps` of a block ends a segment: every kSegment steps, the second block's half as many earlier, and the last
__device__ __forceinline__ bool ends_segment(int i, int steps, int block) {
  return i == steps - 1 || (i + 1 + block * (kSegment / 2)) % kSegment == 0;
}

template <bool GATED>
__global__ void __launch_bounds__(kThreads, 1) tc_kernel(TcArgs a, const __grid_constant__ CUtensorMap map_x,
                                                         const __grid_constant__ CUtensorMap map_w0,
                                                         const __grid_constant__ CUtensorMap map_w1) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023);
  __shared__ uint64_t bar_full[kMaxStages], bar_empty[kMaxStages];          // packed tiles
  __shared__ uint64_t bar_a_full[2][kSlots], bar_a_empty[2][kSlots];        // converted W
  __shared__ uint64_t bar_x_full[kSlots], bar_x_empty[kSlots];              // converted X
  __shared__ uint64_t bar_d_full[2], bar_d_empty[2];                        // accumulators
  __shared__ uint32_t s_tmem;

  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), wg = warp >> 2;
  const int nt = a.nt, stages = a.stages, T = a.m.T, N = a.m.N;
  const uint32_t stage_bytes = 32768 + nt * 128, slot_bytes = nt * 128;
  const uint32_t ring = smem_u32(smem), xring = ring + stages * stage_bytes, xchg = xring + kSlots * slot_bytes;

  // ---- this CTA's tiles and its part of K (in stages of 128)
  const int rank = a.split > 1 ? (int)cluster_rank() : 0;
  const int first = blockIdx.x / a.split, step_tiles = gridDim.x / a.split;
  const int nk = (a.m.K + kTileK - 1) / kTileK;
  const int k_begin = (int)((long long)rank * nk / a.split), k_end = (int)((long long)(rank + 1) * nk / a.split);
  const int steps = 2 * (k_end - k_begin);
  const int my_tiles = first < a.tiles ? (a.tiles - first + step_tiles - 1) / step_tiles : 0;

  if (tid == 0) {
    for (int i = 0; i < stages; ++i) { mbar_init(bar_full + i, 1); mbar_init(bar_empty + i, 12); }
    for (int i = 0; i < kSlots; ++i) {
      for (int b = 0; b < 2; ++b) { mbar_init(&bar_a_full[b][i], 4); mbar_init(&bar_a_empty[b][i], 1); }
      mbar_init(bar_x_full + i, 4);
      mbar_init(bar_x_empty + i, 2);
    }
    for (int b = 0; b < 2; ++b) { mbar_init(bar_d_full + b, 1); mbar_init(bar_d_empty + b, 4); }
    fence_mbar_init();
  }
  if (warp == 12) tc_alloc(&s_tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  // A wait that runs out is recorded; the thread then goes on without waiting, so that every barrier is still met and all
  // loops end (the results are void).
  bool dead = false;
  auto wait = [&](uint64_t* bar, int parity) {
    if (!mbar_try_wait(bar, parity) && !dead) dead = wait_longer(bar, parity, a.m.status);
  };

  if (wg == 3) {
    regs_less<40>();
    if (warp == 12) {
      // ================================================================ copies
      if (lane == 0) {
        int stage = 0, phase = 1;                              // (the first pass over the ring finds it empty)
        for (int j = 0; j < my_tiles; ++j) {
          const int tile = first + j * step_tiles, tn = tile % a.tiles_n, tt = tile / a.tiles_n;
          for (int k = k_begin; k < k_end; ++k) {
            wait(bar_empty + stage, phase);
            uint8_t* to = smem + stage * stage_bytes;
            mbar_arrive_expect_tx(bar_full + stage, stage_bytes);
            tma_load_2d(to, &map_w0, k * kTileK, tn * (GATED ? 128 : 256), bar_full + stage);
            if (GATED) tma_load_2d(to + 16384, &map_w1, k * kTileK, tn * 128, bar_full + stage);
            else tma_load_2d(to + 16384, &map_w0, k * kTileK, tn * 256 + 128, bar_full + stage);
            tma_load_2d(to + 32768, &map_x, k * kTileK, tt * nt, bar_full + stage);
            if (++stage == stages) { stage = 0; phase ^= 1; }
          }
        }
        // (where waits have run out, copies may still be in flight)
        dead = false;
        const int total = my_tiles * (k_end - k_begin);
        for (int t = max(0, total - stages); t < total; ++t) wait(bar_full + t % stages, (t / stages) & 1);
      }
    } else if (warp <= 14) {
      // ================================================================ products of block b
      const int b = warp - 13;
      if (lane == 0) {
        const uint32_t idesc = idesc_f16(nt);
        const uint64_t dx = umma_desc_sw128(xring);
        int i = 0, seg = 0;
        for (int j = 0; j < my_tiles; ++j) {
          bool fresh = true;
          for (int s = 0; s < steps; ++s, ++i) {
            const int slot = i % kSlots, phase = (i / kSlots) & 1;
            if (fresh) wait(bar_d_empty + b, (seg & 1) ^ 1);
            wait(&bar_a_full[b][slot], phase);
            wait(bar_x_full + slot, phase);
            tc_fence_after();
            const uint32_t ta = tmem + kTmemA + (b * kSlots + slot) * 32;
            const uint64_t dxs = dx + slot * (slot_bytes / 16);
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_f16_ts(tmem + b * 128, ta + 8 * k, dxs + 2 * k, idesc, k > 0 || !fresh);
            tc_commit(&bar_a_empty[b][slot]);
            tc_commit(bar_x_empty + slot);
            fresh = false;
            if (ends_segment(s, steps, b)) {
              tc_commit(bar_d_full + b);
              ++seg;
              fresh = true;
            }
          }
        }
      }
    }
    __syncwarp();
    if (a.split > 1) { cluster_sync(); cluster_sync(); }
  } else if (wg == 2) {
    // ================================================================ conversion of X
    regs_less<72>();
    const int t = tid - 256, items = nt * 4;                    // 16-byte pieces of a step
    int stage = 0, phase = 0, i = 0;
    for (int j = 0; j < my_tiles; ++j)
      for (int s = 0; s < steps; s += 2) {
        wait(bar_full + stage, phase);
        const uint32_t from = ring + stage * stage_bytes + 32768;
#pragma unroll
        for (int half = 0; half < 2; ++half, ++i) {
          const int slot = i % kSlots;
          wait(bar_x_empty + slot, ((i / kSlots) & 1) ^ 1);
          const uint32_t to = xring + slot * slot_bytes;
          // eight lanes have the four pieces of rows r and r ^ 5: their reads and their writes meet no bank twice
          for (int p = t; p < items; p += 128) {
            const int c = p & 3, pair = (p >> 3) & 3, r = (p >> 5) * 8 + ((p & 4) ? pair ^ 5 : pair);
            const uint4 v = ld_shared(from + r * 128 + (((half * 4 + c) ^ (r & 7)) << 4));
            uint32_t h[8];
            convert4(v.x, h[0], h[1]);
            convert4(v.y, h[2], h[3]);
            convert4(v.z, h[4], h[5]);
            convert4(v.w, h[6], h[7]);
            const uint32_t row = to + r * 128;
            st_shared(row + (((2 * c) ^ (r & 7)) << 4), h[0], h[1], h[2], h[3]);
            st_shared(row + (((2 * c + 1) ^ (r & 7)) << 4), h[4], h[5], h[6], h[7]);
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_x_full + slot);
        }
        if (lane == 0) mbar_arrive(bar_empty + stage);
        if (++stage == stages) { stage = 0; phase ^= 1; }
      }
    __syncwarp();
    if (a.split > 1) { cluster_sync(); cluster_sync(); }
  } else {
    // ================================================================ block wg: conversion of W, sums, outputs
    regs_more<200>();
    const int b = wg, row = tid & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;           // TMEM lane quarter
    int sum[kMaxTokens];
#pragma unroll
    for (int t = 0; t < kMaxTokens; ++t) sum[t] = 0;
    int stage = 0, phase = 0, i = 0, seg = 0;
    uint32_t from = 0;

    // converts step i: the next 64 of K
    auto convert = [&]() {
      const int half = i & 1, slot = i % kSlots;
      if (half == 0) {
        wait(bar_full + stage, phase);
        from = ring + stage * stage_bytes + b * 16384 + row * 128;
      }
      wait(&bar_a_empty[b][slot], ((i / kSlots) & 1) ^ 1);
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t h[16];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint4 v = ld_shared(from + (((half * 4 + 2 * k + c) ^ (row & 7)) << 4));
          convert4(v.x, h[8 * c], h[8 * c + 1]);
          convert4(v.y, h[8 * c + 2], h[8 * c + 3]);
          convert4(v.z, h[8 * c + 4], h[8 * c + 5]);
          convert4(v.w, h[8 * c + 6], h[8 * c + 7]);
        }
        tc_st16(tmem + lanes + kTmemA + (b * kSlots + slot) * 32 + 16 * k, h);
      }
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bar_a_full[b][slot]);
        if (half == 1) mbar_arrive(bar_empty + stage);
      }
      if (half == 1 && ++stage == stages) { stage = 0; phase ^= 1; }
      ++i;
    };
    // adds the accumulators of the segment that is done next to the sums
    auto take = [&]() {
      wait(bar_d_full + b, seg & 1);
      ++seg;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < kMaxTokens / 16; ++c)
        if (c * 16 < nt) {
          uint32_t r[16];
          tc_ld16(tmem + lanes + b * 128 + 16 * c, r);
          tc_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) sum[16 * c + e] += __float2int_rn(__uint_as_float(r[e]));
        }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_d_empty + b);
    };
    auto output = [&](int tile) {
      const int tn = tile % a.tiles_n, t0 = tile / a.tiles_n * nt;
      if (!GATED) {
        const int n = tn * 256 + b * 128 + row;
        const float ws = n < N ? a.m.ws[0][n] : 0.f;
#pragma unroll
        for (int t = 0; t < kMaxTokens; ++t) {
          if (t < nt && t0 + t < T && n < N) put(a.m, t0 + t, n, product(sum[t], __ldg(a.m.xs + t0 + t), ws));
          sum[t] = 0;
        }
      } else {
        // block 0 (gate) finishes the lower half of every 16 tokens, block 1 (up) the upper; what the other needs goes through
        // shared memory, two buffers in turn
        const int n = tn * 128 + row;
        const float ws = n < N ? a.m.ws[b][n] : 0.f;
#pragma unroll
        for (int c = 0; c < kMaxTokens / 16; ++c)
          if (c * 16 < nt) {
            const uint32_t buf = xchg + (c & 1) * (kXchgBytes / 2);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int v = b == 0 ? sum[16 * c + 8 + e] : sum[16 * c + e];
              const int t = t0 + 16 * c + 8 * (1 - b) + e;
              const float p = product(v, t < T ? __ldg(a.m.xs + t) : 0.f, ws);
              asm volatile("st.shared.f32 [%0], %1;" ::"r"(buf + (((1 - b) * 8 + e) * 128 + row) * 4), "f"(p) : "memory");
            }
            named_bar(1, 256);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int t = t0 + 16 * c + 8 * b + e;
              float other;
              asm volatile("ld.shared.f32 %0, [%1];" : "=f"(other) : "r"(buf + ((b * 8 + e) * 128 + row) * 4) : "memory");
              if (t < T && n < N) {
                const float p = product(b == 0 ? sum[16 * c + e] : sum[16 * c + 8 + e], __ldg(a.m.xs + t), ws);
                put(a.m, t, n, b == 0 ? silu_mul(p, other) : silu_mul(other, p));
              }
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) sum[16 * c + e] = 0;
          }
        named_bar(1, 256);   // the next tile's first buffer is free
      }
    };

    // A segment's sums are taken three steps after its last one has been converted, so that the tensor cores have steps to
    // go on with. d: the next segment's end; one tile's steps after another's.
    const int total = my_tiles * steps;
    int ds = 0, dtile = 0;                          // the next step whose sums may be due, within its tile
    for (int at = 0; at < total + kSlots - 1; ++at) {
      if (at < total) convert();
      if (at >= kSlots - 1) {
        if (ends_segment(ds, steps, b)) take();
        if (++ds == steps) {
          if (a.split == 1) output(first + dtile * step_tiles);
          ds = 0;
          ++dtile;
        }
      }
    }

    if (a.split > 1) {
      // every CTA of the cluster is through with its rings; token t is finished by CTA t / per
      const int per = (nt + a.split - 1) / a.split;
      cluster_sync();
#pragma unroll
      for (int t = 0; t < kMaxTokens; ++t)
        if (t < nt) st_peer(ring + ((rank * per + t % per) * 256 + (b * 128 + row)) * 4, t / per, (uint32_t)sum[t]);
      cluster_sync();
      const int tn = first % a.tiles_n, t0 = first / a.tiles_n * nt;
      const int* got = reinterpret_cast<const int*>(smem);
      const int here = min(per, nt - rank * per);
      if (!GATED) {
        const int n = tn * 256 + tid;
        if (n < N && first < a.tiles) {
          const float ws = a.m.ws[0][n];
          for (int t = 0; t < here; ++t) {
            const int tok = t0 + rank * per + t;
            if (tok >= T) break;
            int acc = 0;
            for (int s = 0; s < a.split; ++s) acc += got[(s * per + t) * 256 + tid];
            put(a.m, tok, n, product(acc, __ldg(a.m.xs + tok), ws));
          }
        }
      } else {
        const int n = tn * 128 + row;
        if (n < N && first < a.tiles) {
          const float wg_ = a.m.ws[0][n], wu = a.m.ws[1][n];
          for (int t = b; t < here; t += 2) {
            const int tok = t0 + rank * per + t;
            if (tok >= T) break;
            int g = 0, u = 0;
            for (int s = 0; s < a.split; ++s) {
              g += got[(s * per + t) * 256 + row];
              u += got[(s * per + t) * 256 + 128 + row];
            }
            const float xs = __ldg(a.m.xs + tok);
            put(a.m, tok, n, silu_mul(product(g, xs, wg_), product(u, xs, wu)));
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tc_dealloc(tmem, 512);
  }
}

struct TcPlan {
  int nt, tiles_n, tiles, split, stages;
  uint32_t smem;
};

static TcPlan plan(const MatArgs& a, bool gated, int sms) {
  TcPlan p;
  p.tiles_n = (a.N + (gated ? 127 : 255)) / (gated ? 128 : 256);
  const int nk = (a.K + kTileK - 1) / kTileK;
  // tokens of a tile: as few columns as the waves of tiles need in all
  p.nt = 16;
  if (a.T <= kMaxTokens) {
    p.nt = (a.T + 15) / 16 * 16;
  } else {
    long long best = 0;
    for (int nt = kMaxTokens; nt >= 64; nt -= 16) {
      const long long tiles = (long long)p.tiles_n * ((a.T + nt - 1) / nt), cost = (tiles + sms - 1) / sms * nt;
      if (best == 0 || cost < best) { best = cost; p.nt = nt; }
    }
  }
  p.tiles = p.tiles_n * ((a.T + p.nt - 1) / p.nt);
  p.split = 1;
  while (p.split < 8 && p.tiles * p.split * 2 <= sms && p.split * 2 <= nk) p.split *= 2;
  const int stage = 32768 + p.nt * 128, fixed = kSlots * p.nt * 128 + (gated ? kXchgBytes : 0);
  p.stages = (kSmemLimit - 1024 - fixed) / stage;
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  p.smem = 1024 + fixed + p.stages * stage;
  return p;
}

static bool map_rows(CUtensorMap* m, const int8_t* q, int rows, int cols, int64_t stride, int box_rows) {
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows}, strides[1] = {(uint64_t)stride};
  const uint32_t box[2] = {kTileK, (uint32_t)box_rows};
  return moe_internal::tmap_u8(m, q, 2, dims, strides, box);
}

moe_status_t tc_multiply(const MatArgs& a, cudaStream_t stream) {
  const bool gated = a.w[1] != nullptr;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MOE_ERR_CUDA;
  static int configured[64] = {0};
  if (!configured[dev]) {
    if (cudaFuncSetAttribute(tc_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit) != cudaSuccess ||
        cudaFuncSetAttribute(tc_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit) != cudaSuccess)
      return MOE_ERR_CUDA;
    configured[dev] = 1;
  }
  const int sms = moe_internal::num_sms();
  if (sms <= 0) return MOE_ERR_CUDA;
  const TcPlan p = plan(a, gated, sms);
  CUtensorMap mx, m0, m1;
  if (!map_rows(&mx, a.x, a.T, a.K, a.x_stride, p.nt) || !map_rows(&m0, a.w[0], a.N, a.K, a.w_stride[0], 128)) return MOE_ERR_CUDA;
  m1 = m0;
  if (gated && !map_rows(&m1, a.w[1], a.N, a.K, a.w_stride[1], 128)) return MOE_ERR_CUDA;
  TcArgs args{a, p.nt, p.tiles_n, p.tiles, p.split, p.stages};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.split > 1 ? p.tiles * p.split : min(p.tiles, sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = stream;
  cudaLaunchAttribute at;
  if (p.split > 1) {
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = p.split;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
  }
  const cudaError_t e = gated ? cudaLaunchKernelEx(&cfg, tc_kernel<true>, args, mx, m0, m1)
                              : cudaLaunchKernelEx(&cfg, tc_kernel<false>, args, mx, m0, m1);
  if (e != cudaSuccess) { cudaGetLastError(); return MOE_ERR_CUDA; }
  return MOE_OK;
}

}  // namespace i8
}  // namespace moe
