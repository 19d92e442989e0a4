// kv_attn_wide.cu -- attention of a verify step over the 4-bit paged KV cache on tcgen05: 32 or 64 query rows of a KV head
// at a time (rows that are not there count as zero; more than 64 are two groups).
//
// The mathematics and the cache are kv_attn.cu's; there a key's codes are converted once per 8 query rows, which bounds it
// when the rows are many. Here a tile of 128 keys is converted once, into shared memory operands of binary16, exactly: a
// code times its block's scale has at most 11 significant bits in either format, and the scales are taken relative to a
// power of two E so that they lie in 2^-14 .. 2^2. Then, with keys (or dimensions) as the 128 rows of the products:
//   S^T [128 keys x N] = K Q^T,  O^T [128 dimensions x N] += V^T P^T,  fp32 in TMEM.
//
// Work: as in kv_attn.cu the (sequence, KV head) pairs are laid end to end, here in tiles, and dealt out evenly over one
// CTA per SM; a pair that spans CTAs is joined by the one that finishes last.
//
// 16 warps convert and do the softmax, one copies packed tiles into a ring, one issues the products. Per tile a worker
// warp converts eight tokens' keys of the next tile, does the softmax of this one (lane = key, N / 4 rows), then converts
// the next tile's values: S of the next tile is formed during the softmax, O during the conversion. Splitting the
// workers' roles instead (8 warps converting, 16 in the softmax) took 287 us where this took 248, most of it polling; one
// hand-over to the tensor cores a tile instead of two (keys two tiles ahead) did no better.
// P is stored with its rows contiguous (B transposed): a lane's key is then one or two 16-byte stores.
//
// What bounds it: instructions. A tile at N = 64 takes 3,500 cycles for about 510 warp instructions a worker
// warp (58 % of the issue slots; the integer pipe is half, shared memory two thirds busy); its HBM share would take 800, the tensor
// cores 510. Verify step of 16 sequences of up to 32768 keys, 64 rows a KV head (8 KV heads, D = 128, MXFP4): 249 us, against
// 467 us with kv_attn.cu; the cache is read at 1.4 TB/s.
//
// What the window of scales cannot hold (set from a pair's first tile: 12 powers of two down, 3 up), and weights below
// 2^-21 (binary16 has no full precision for them) in rows that have not yet seen 12 keys of 2^-20 are left to kv_attn.cu,
// whose passes keep them: the sequence is marked, and the launch that follows does the marked ones again. Blocks of zeros,
// whose scale is the smallest there is, are not left over (a tenth of the tokens zero: 276 us instead of 2,544); looking for
// them costs 5 % where there are none.
#include "kv_attn.cuh"

namespace moe {
namespace kv {

constexpr int kTileSubs = 8;        // 128 keys
constexpr int kWorkers = 16;         // warps that convert and do the softmax; one more copies, one issues the MMAs
constexpr int kThreads = (kWorkers + 2) * 32;
// Weights are carried times 2^8, and a score may pass the running maximum by 7 (base 2) before it is raised: to raise it
// stops all 64 rows for about 2,000 cycles, a tile's whole time, and binary16 holds 2^15.
constexpr int kAnchor = 8;
constexpr float kSlack = 7.f, kHeavyW = 0.000244140625f, kLightW = 0.0001220703125f;   // 2^8 times 2^-20 and 2^-21
constexpr int kTileBatch = 4;       // tiles whose addresses the producer's lanes hold at a time

__device__ __forceinline__ void tc_mma_f16(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(
          d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// binary16 x binary16 -> fp32, both operands K-major, M = 128
__device__ __forceinline__ uint32_t idesc_f16(uint32_t n) { return (1u << 4) | ((n >> 3) << 17) | (8u << 24); }
constexpr uint32_t kBTransposed = 1u << 16;   // B with its rows contiguous (for each k)
__device__ __forceinline__ void fma2(float (&d)[2], const float (&a)[2], float b0, float b1, float c0, float c1) {
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d[0]), "=f"(d[1])
      : "f"(a[0]), "f"(a[1]), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void add2(float (&d)[2], const float (&a)[2]) {
  asm("{\n\t.reg .b64 a, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 d, {%0, %1};\n\tadd.rn.f32x2 d, d, a;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "+f"(d[0]), "+f"(d[1])
      : "f"(a[0]), "f"(a[1]));
}
// a shared memory address as a pointer (arithmetic on 32-bit addresses costs half of that on pointers)
__device__ __forceinline__ uint8_t* at_shared(uint32_t addr) { return static_cast<uint8_t*>(__cvta_shared_to_generic(addr)); }
template <int C>
__device__ __forceinline__ void tc_load(uint32_t taddr, uint32_t (&r)[C]) {
  if (C == 8) {
    uint32_t v[8];
    tc_ld8(taddr, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i % C] = v[i];
  } else {
#pragma unroll
    for (int k = 0; k < C / 16; ++k) {
      uint32_t v[16];
      tc_ld16(taddr + 16 * k, v);
#pragma unroll
      for (int i = 0; i < 16; ++i) r[(16 * k + i) % C] = v[i];
    }
  }
  tc_wait_ld();
}
__device__ __forceinline__ void tc_st4(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// barrier `id` among 128 threads; true if any of them passes true
__device__ __forceinline__ bool bar_any(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(id)
      : "memory");
  return r != 0;
}

// The largest (or the sum) over the warp's lanes of each of C values; afterwards lane x < C has column x's
template <int C, bool MAX>
__device__ __forceinline__ float across(float (&v)[C]) {
#pragma unroll
  for (int o = 16; o >= C; o >>= 1)
#pragma unroll
    for (int x = 0; x < C; ++x) {
      const float y = __shfl_xor_sync(0xFFFFFFFFu, v[x], o);
      v[x] = MAX ? fmaxf(v[x], y) : v[x] + y;
    }
#pragma unroll
  for (int o = C / 2; o > 0; o >>= 1) {
    const bool up = threadIdx.x & o;
#pragma unroll
    for (int x = 0; x < C / 2; ++x)
      if (x < o) {
        const float keep = up ? v[x + o] : v[x], give = up ? v[x] : v[x + o], y = __shfl_xor_sync(0xFFFFFFFFu, give, o);
        v[x] = MAX ? fmaxf(keep, y) : keep + y;
      }
  }
  return v[0];
}

// A K word's 8 codes times their scale (twice in s), in the operand's order
template <int FMT>
__device__ __forceinline__ uint4 convert8(uint32_t w, uint32_t s) {
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = hmul2_bits(FMT == MOE_FMT_MXFP4 ? e2m1x2_to_f16x2(w, i)
                                           : hadd2_bits(lop3_and_xor(w >> (4 * i), 0x000F000Fu, 0x64086408u), 0xE408E408u), s);
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// A pair's start counts as 3 tiles in the list of work (what its q, its first maximum and its output cost).
constexpr int kPairTiles = 3;
__device__ __forceinline__ int seq_tiles(const SeqInfo& s) {
  return s.qn > 0 && s.len > 0 ? ((s.len + 15) / 16 - s.sub0 + kTileSubs - 1) / kTileSubs : 0;
}

// A row's keys, counted until there are 12 of weight 2^-20 and more (low half); those of 2^-12 and more in the high half.
__device__ __forceinline__ bool few_keys(int cnt) { return (cnt & 0xFFFF) < 12; }

// Where scales have left the window (which spoils their neighbours in a word): one block's scale times 2^-E in binary16, for
// `codes` of that block (those a lane has, other bits 0). Blocks of zeros have the smallest scale and need none; other scales
// outside the window set `off`. minus_low: minus the window's lower end, as scale_pair takes it.
template <int FMT>
__device__ __forceinline__ uint32_t one_scale(const uint8_t* scale, uint32_t minus_low, uint32_t codes, uint32_t& off) {
  int low = FMT == MOE_FMT_MXFP4 ? (int)((0u - minus_low) & 255) : (int)((0u - minus_low) >> 7 & 511);   // -12 .. 242
  if (low > 242) low -= FMT == MOE_FMT_MXFP4 ? 256 : 512;
  const int bits = FMT == MOE_FMT_MXFP4 ? (int)*scale << 7 : (int)*reinterpret_cast<const uint16_t*>(scale);
  const int x = bits - (low << 7);
  if ((uint32_t)x < 16u << 7) return (uint32_t)(x + 128) << 3;
  if (codes & (FMT == MOE_FMT_MXFP4 ? 0x77777777u : 0xFFFFFFFFu)) off = kOff<FMT>;   // (a zero's sign does not count)
  return 0;
}

// The rest of a wait: true if it ran out.
__device__ __noinline__ bool wait_longer(uint64_t* bar, int parity, int32_t* status) {
  const long long t0 = globaltimer_ns();
  for (uint32_t n = 1; !mbar_try_wait(bar, parity); ++n)
    if (n % 64 == 0 && globaltimer_ns() - t0 > kDefaultWaitNs) {
      record_error(status, MOE_ERR_DEVICE_TIMEOUT);
      return true;
    }
  return false;
}

template <int FMT, int D, int N>
struct Wide {   // shared memory, in bytes from the 1024-byte aligned start
  static constexpr int TILE = kTileSubs * Sub<FMT, D>::BYTES;
  static constexpr int K_OP = D / 64 * 16384, V_OP = 2 * 16384;            // [keys][64 dims] slabs; [dims][64 keys] slabs
  static constexpr int P_OP = 128 * 2 * N;                                 // [keys][rows], swizzled over its 2 N bytes
  static constexpr int K = 0, V = 2 * K_OP, P = V + 2 * V_OP, Q = P + P_OP, RING = Q + D / 64 * N * 128;
  static constexpr int C = N / 4;                                          // rows of a group of 4 warps
  static constexpr int TMEM_COLS = 4 * N;                                  // S twice, O: 3 N columns, to a power of two
};

template <int FMT, int D, int N>
__global__ void __launch_bounds__(kThreads, 1) wide_kernel(Args a, AttnArgs g) {
  using S = Sub<FMT, D>;
  using L = Wide<FMT, D, N>;
  constexpr int NB = S::NB, C = L::C;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023);
  __shared__ uint64_t bar_ring_full[4], bar_ring_empty[4], bar_k[2], bar_s[2], bar_p, bar_done;
  __shared__ uint32_t s_tmem;
  __shared__ long long s_warp[kThreads / 32], s_total;
  __shared__ __align__(16) float s_neg[N], s_al[N], s_max[4][N];   // s_neg: -m
  __shared__ int s_cnt[N], s_lim[N], s_exp[kWorkers][2], s_used[2], s_tiles[2], s_last[2];
  __shared__ __align__(16) float s_f[4][N];                            // per pair (of the last four): the rows' factor of the scores,
  __shared__ int s_ev[4];                                // and V's E

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int stages = g.stages, RG = g.row_groups, Hv = a.kv_heads * RG;
  uint8_t* ring = smem + L::RING;
  long long* prefix = reinterpret_cast<long long*>(smem + g.rings);               // [n_seqs + 1]
  SeqInfo* info = reinterpret_cast<SeqInfo*>(prefix + a.n_seqs + 1 + ((a.n_seqs + 1) & 1));

  if (tid == 0) {
    for (int i = 0; i < stages; ++i) { mbar_init(bar_ring_full + i, 1); mbar_init(bar_ring_empty + i, kWorkers); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_k + i, kWorkers);
      mbar_init(bar_s + i, 2);
      s_used[i] = -1;
      s_last[i] = -1;
    }
    mbar_init(&bar_p, kWorkers);
    mbar_init(&bar_done, 1);
    prefix[0] = 0;
    s_total = 0;
  }
  // ---- the sequences, as in kv_attn.cu: a pair (sequence, KV head and row group) costs kPairTiles more than it has
  int live = 0;
  for (int base = 0; base < a.n_seqs; base += kThreads) {
    const int b = base + tid;
    long long x = 0;
    if (b < a.n_seqs) {
      const Seq sq = check_seq(a, a.q_start[b], a.q_start[b + 1], a.seq_len[b], a.max_q);
      SeqInfo si{sq.q0, sq.qn, sq.len, 0};
      if (g.window > 0 && sq.len - sq.qn - g.window + 1 > 0) si.sub0 = (sq.len - sq.qn - g.window + 1) / 16;
      info[b] = si;
      x = seq_tiles(si) ? (long long)(seq_tiles(si) + kPairTiles) * Hv : 0;
    }
    const bool some = x > 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    live += __syncthreads_count(some);
    long long add = s_total;
    for (int w = 0; w < warp; ++w) add += s_warp[w];
    if (b < a.n_seqs) prefix[b + 1] = x + add;
    __syncthreads();
    if (tid == kThreads - 1) s_total = x + add;
  }
  fence_mbar_init();
  __syncthreads();
  const long long W = prefix[a.n_seqs];
  for (int b = blockIdx.x; b < a.n_seqs; b += gridDim.x) {
    const SeqInfo si = info[b];
    if (si.qn <= 0 || seq_tiles(si) > 0) continue;
    const int64_t r0 = (int64_t)si.q0 * g.q_heads, n = (int64_t)si.qn * g.q_heads;
    for (int64_t i = tid; i < n * (D / 8); i += kThreads) reinterpret_cast<uint4*>(g.out + r0 * D)[i] = make_uint4(0, 0, 0, 0);
    if (g.lse)
      for (int64_t i = tid; i < n; i += kThreads) g.lse[r0 + i] = -INFINITY;
  }
  if (W == 0) return;
  // G: at least about four tiles a CTA, a multiple of the pairs (those that have tiles) while SMs are left over; at most W, as
  // W >= 4 pairs, so that no CTA is without a place of the list (see kv_attn.cu)
  const long long pairs = (long long)live * Hv, even = (W + 4 * pairs - 1) / (4 * pairs) * pairs;
  const int G = (int)min(even, (long long)gridDim.x);
  if (blockIdx.x >= G) return;
  const long long f_begin = share(blockIdx.x, W, G), f_end = share(blockIdx.x + 1, W, G);

  // ---- this CTA's first tile u0 (of units) of pair (b0, h0), and how many tiles it has
  int b0 = 0, h0 = 0, u0 = 0, units0 = 0, todo = 0;
  if (f_begin < f_end) {
    int lo = 0, hi = a.n_seqs;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= f_begin) lo = mid;
      else hi = mid;
    }
    b0 = lo;
    units0 = seq_tiles(info[lo]);
    const long long rem = f_begin - prefix[lo];
    h0 = (int)share(rem, 1, units0 + kPairTiles);
    int at = (int)(rem - (long long)h0 * (units0 + kPairTiles));
    u0 = max(0, at - kPairTiles);
    long long left = f_end - f_begin;
    for (int b = lo, h = h0, units = units0; left > 0;) {
      const int here = (int)min(left, (long long)(units + kPairTiles - at));
      todo += max(0, at + here - max(at, kPairTiles));
      left -= here;
      at = 0;
      if (++h < Hv) {
        const int n = (int)min(share(left, 1, units + kPairTiles), (long long)(Hv - h));
        todo += n * units;
        left -= (long long)n * (units + kPairTiles);
        h += n;
      }
      if (h == Hv && left > 0) {
        h = 0;
        do units = seq_tiles(info[++b]); while (units == 0);
      }
    }
  }
  auto next_pair = [&](int& b, int& h, int& u, int& units) {   // (there is one: tiles remain)
    u = 0;
    if (++h < Hv) return;
    h = 0;
    do units = seq_tiles(info[++b]); while (units == 0);
  };
  if (warp == kWorkers + 1) tc_alloc(&s_tmem, L::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem, tmem_o = tmem + 2 * N;

  // A wait that runs out is recorded; the thread then goes on without waiting, so that every barrier is still met and all
  // loops end (the results are void).
  bool dead = false;
  auto wait = [&](uint64_t* bar, int parity) {
    if (!mbar_try_wait(bar, parity) && !dead) dead = wait_longer(bar, parity, a.status);
  };

  if (warp == kWorkers) {
    // ================================================================ copies
    int b = b0, h = h0, u = u0, units = units0, left = todo, next_id = 0, n = 0, subs = 0, sub_first = 0, nb = 0, nh = 0;
    // the next batch's table entries: up to 4 tiles of one pair, a sub-block a lane
    auto fetch = [&]() {
      n = min(min(kTileBatch, units - u), left);
      if (n > 0) {
        sub_first = info[b].sub0 + u * kTileSubs;
        subs = min(n * kTileSubs, (info[b].len + 15) / 16 - sub_first);
        nb = b;
        nh = h / RG;
        if (lane < subs)
          next_id = __ldg(a.block_table + (int64_t)nb * a.table_stride + (sub_first + lane) / (a.page_tokens / 16));
        left -= n;
        u += n;
        if (u == units && left > 0) next_pair(b, h, u, units);
      }
    };
    fetch();
    int stage = 0, phase = 1;                            // (the first pass over the ring finds it empty)
    for (int i = 0; i < todo;) {
      const int cur_n = n, cur_subs = subs, per_page = a.page_tokens / 16;
      const uint8_t* ptr = nullptr;
      if (lane < cur_subs) {
        bool ok;
        const int id = check_page(a, next_id, ok), sub = sub_first + lane;
        ptr = a.pages + (int64_t)id * a.page_stride + (int64_t)(nh * per_page + sub % per_page) * S::BYTES;
      }
      fetch();
      for (int k = 0; k < cur_n; ++k, ++i) {
        wait(bar_ring_empty + stage, phase);
        const int here = min(kTileSubs, cur_subs - k * kTileSubs);
        if (lane == 0) mbar_arrive_expect_tx(bar_ring_full + stage, here * S::BYTES);
        __syncwarp();
        if ((lane >> 3) == k && lane < cur_subs)
          bulk_g2s_plain(ring + stage * L::TILE + (lane & 7) * S::BYTES, ptr, S::BYTES, bar_ring_full + stage);
        if (++stage == stages) { stage = 0; phase ^= 1; }
      }
    }
    // (where waits have run out, copies may still be in flight)
    dead = false;
    for (int t = max(0, todo - stages); t < todo; ++t) wait(bar_ring_full + t % stages, (t / stages) & 1);
  } else if (warp == kWorkers + 1) {
    // ================================================================ MMAs
    if (lane == 0) {
      const uint32_t idesc = idesc_f16(N);
      const uint64_t dk = umma_desc_sw128(smem_u32(smem + L::K)), dq = umma_desc_sw128(smem_u32(smem + L::Q)),
                     dv = umma_desc_sw128(smem_u32(smem + L::V)),
                     dp = umma_desc(smem_u32(smem + L::P), 16 * N, 16 * N, N == 64 ? 2 : 4);
      int b = b0, h = h0, u = u0, units = units0;
      bool first = true, first_prev = true;              // the tile begins (this CTA's part of) a pair
      for (int i = 0; i <= todo; ++i) {
        if (i < todo) {
          wait(bar_k + (i & 1), (i >> 1) & 1);
          tc_fence_after();
          const uint64_t ka = dk + (i & 1) * (L::K_OP / 16);
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            tc_mma_f16(tmem + (i & 1) * N, ka + (k >> 2) * 1024 + (k & 3) * 2, dq + (k >> 2) * (N * 8) + (k & 3) * 2, idesc, k > 0);
          tc_commit(bar_s + (i & 1));
          mbar_arrive(bar_s + (i & 1));             // (passes on what the conversion wrote)
        }
        if (i > 0) {
          const int t = i - 1;
          wait(&bar_p, t & 1);
          tc_fence_after();
          const uint64_t va = dv + (t & 1) * (L::V_OP / 16);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            tc_mma_f16(tmem_o, va + (k >> 2) * 1024 + (k & 3) * 2, dp + k * (2 * N), idesc | kBTransposed, k > 0 || !first_prev);
          tc_commit(&bar_done);
        }
        first_prev = first;
        first = false;
        if (i < todo && ++u == units && i + 1 < todo) {
          next_pair(b, h, u, units);
          first = true;
        }
      }
    }
    __syncwarp();
  } else if (warp < kWorkers) {
    // ================================================================ workers
    // Conversion: warp w has eight tokens of sub-block w / 2 of a tile. Softmax: lane = key (then dimension) 32 (w % 4) +
    // lane of the tile, rows col0 .. col0 + C - 1. A tile's iteration converts the next tile's keys, does its own softmax, then
    // converts the next tile's values, so that each product has a phase of the others' to finish in.
    const int r = lane >> 2, c = lane & 3, half = warp & 1;
    int cb = b0, ch_ = h0, cu = u0, cunits = units0, stage = 0, phase = 0, cpair = -1, key0 = 0, len = 0, min_lo = 0;
    bool cfirst = true;
    uint32_t vc[FMT == MOE_FMT_MXFP4 ? 1 : NB], kc = 0;  // minus the windows' lower ends, as scale_pair takes them
    constexpr int NVC = FMT == MOE_FMT_MXFP4 ? 1 : NB;
    uint32_t off = 0;
    // K rows: a lane writes 8 dimensions of one key per block; lanes 4 to 7 of eight have the row four on, so that eight lanes
    // fill all banks
    const int rk = (r & 1) * 4 + (r >> 1), tk = 8 * half + rk;
    const uint32_t smem_at = smem_u32(smem), sub_at = smem_at + L::RING + (warp >> 1) * S::BYTES;
    const uint32_t k_at = smem_at + L::K + (uint32_t)(8 * warp + rk) * 128 + (uint32_t)((c ^ rk) << 4);
    // V rows: dimension 32 b + 4 r + j, j = (i + r / 2) % 4 at step i (again: all banks), tokens 2 c, 2 c + 1 of the eight
    const int rot = r >> 1;
    uint32_t v_at[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = 4 * r + ((i + rot) & 3);
      v_at[i] = smem_at + L::V + (uint32_t)(warp >> 3) * 16384 + d * 128 + (((warp & 7) ^ (d & 7)) << 4) + 4 * c;
    }
    // ---- keys (and, with a new pair's first tile, its windows and its q) of tile i
    auto convert_keys = [&](int i) {
      wait(bar_ring_full + stage, phase);
      const uint8_t* sb = at_shared(sub_at + stage * L::TILE);
      if (cfirst) {
        const SeqInfo si = info[cb];
        key0 = (si.sub0 + cu * kTileSubs) * 16 + 8 * warp;
        len = si.len;
        min_lo = g.window > 0 ? si.len - si.qn + 1 - g.window : 0;
        ++cpair;
        // q's loads first: D / 8 neighbouring lanes have a row
        constexpr int QN = (N * (D / 8) + kWorkers * 32 - 1) / (kWorkers * 32);
        const int row0 = (ch_ % RG) * N, kvh = ch_ / RG;
        uint4 qs[QN];
#pragma unroll
        for (int y = 0; y < QN; ++y) {
          const int id = tid + y * kWorkers * 32, row = row0 + id / (D / 8), j = (int)((uint32_t)row * g.group_inv >> 16);
          qs[y] = make_uint4(0, 0, 0, 0);
          if (id < N * (D / 8) && j < si.qn)
            qs[y] = __ldg(reinterpret_cast<const uint4*>(g.q + (int64_t)(si.q0 + j) * g.q_stride +
                                                         (int64_t)(kvh * g.group + row - j * g.group) * D) + id % (D / 8));
        }
        // E from the first tile's largest scales (tokens past the end or before the window do not count)
        const int t = lane & 7, sel = lane >> 3 & 1;     // (lanes 16 .. 31 repeat)
        const uint8_t* p = sb + (sel ? S::VS : S::KS) + (8 * half + t) * (NB * S::SB);
        int e = 0;
#pragma unroll
        for (int x = 0; x < NB; ++x)
          e = max(e, FMT == MOE_FMT_MXFP4 ? (int)p[x] : (int)(reinterpret_cast<const uint16_t*>(p)[x] >> 7 & 255));
        if (key0 + t >= len || key0 + t < min_lo) e = 0;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) e = max(e, __shfl_xor_sync(0xFFFFFFFFu, e, o));
        if (lane == 0 || lane == 8) s_exp[warp][sel] = e;
        if (i > 0) wait(bar_s + ((i - 1) & 1), ((i - 1) >> 1) & 1);   // the pair before has used q's operand
        named_bar(15, kWorkers * 32);
        int e_k = 0, e_v = 0;
#pragma unroll
        for (int x = 0; x < kWorkers; ++x) {
          e_k = max(e_k, s_exp[x][0]);
          e_v = max(e_v, s_exp[x][1]);
        }
        e_k += 2 - 127;                                  // the window: 12 powers of two below the largest, 3 above
        e_v += 2 - 127;
        if (max(e_k, e_v) > 127 && tid == 0) g.redo[cb] = g.redo[a.n_seqs] = 1;
        // q, each row times its power of two
#pragma unroll
        for (int y = 0; y < QN; ++y) {
          const int id = tid + y * kWorkers * 32, n = id / (D / 8), ch = id % (D / 8);
          if (id >= N * (D / 8)) break;                  // (whole warps)
          const uint4 qv = qs[y];
          const uint32_t x[4] = {qv.x, qv.y, qv.z, qv.w};
          float v[8], amax = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[2 * e] = __uint_as_float(x[e] << 16);
            v[2 * e + 1] = __uint_as_float(x[e] & 0xFFFF0000u);
            amax = fmaxf(amax, fmaxf(fabsf(v[2 * e]), fabsf(v[2 * e + 1])));
          }
#pragma unroll
          for (int o = D / 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
          const int sg = rescale_exponent(amax), t = e_k - sg;
          const float up = exp2i(sg);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] *= up;
          // INT4 codes come as pairs (i, i + 4) of the 8: the same order here
          *reinterpret_cast<uint4*>(smem + L::Q + (ch >> 3) * (N * 128) + n * 128 + (((ch & 7) ^ (n & 7)) << 4)) =
              FMT == MOE_FMT_MXFP4
                  ? make_uint4(pack_f16(v[0], v[1]), pack_f16(v[2], v[3]), pack_f16(v[4], v[5]), pack_f16(v[6], v[7]))
                  : make_uint4(pack_f16(v[0], v[4]), pack_f16(v[1], v[5]), pack_f16(v[2], v[6]), pack_f16(v[3], v[7]));
          if (ch == 0) s_f[cpair & 3][n] = g.scale_log2 * exp2i(max(t / 2, -126)) * exp2i(max(t - t / 2, -126));
        }
        if (tid == 0) s_ev[cpair & 3] = e_v;
        if (FMT == MOE_FMT_MXFP4) {
          kc = 0u - (uint32_t)((e_k + 113) * 0x01010101);
          vc[0] = 0u - (uint32_t)((e_v + 113) * 0x01010101);
        } else {
          kc = 0u - (uint32_t)((e_k + 113) * 0x00800080);
#pragma unroll
          for (int x = 0; x < NB; ++x) vc[x % NVC] = 0u - (uint32_t)((e_v + 113) * 0x00800080);
        }
        named_bar(15, kWorkers * 32);                    // (s_exp is free again)
      }
      const uint32_t k_to = k_at + (i & 1) * L::K_OP;
      uint32_t wd[NB], us[NB], o = 0;
      load_words<NB>(wd, sb + S::KC + tk * (D / 2) + c * (4 * NB));
      if (FMT == MOE_FMT_MXFP4) {
        const uint8_t* p = sb + S::KS + tk * NB;
        uint32_t x = NB == 4 ? *reinterpret_cast<const uint32_t*>(p) : *reinterpret_cast<const uint16_t*>(p);
        if (NB == 2) x |= x << 16;
        o = x + kc;
        x = x * 4u + (kc * 4u + 0x04040404u);
#pragma unroll
        for (int y = 0; y < NB; ++y) {
          const uint32_t sel = (8u | y) | (uint32_t)y << 4;
          us[y] = prmt(x, x, sel | sel << 8);
        }
      } else {
        uint32_t x[NB / 2];
        load_words<NB / 2>(x, sb + S::KS + tk * (2 * NB));
#pragma unroll
        for (int y = 0; y < NB; ++y) {
          us[y] = prmt(x[y / 2], 0u, y & 1 ? 0x3232u : 0x1010u);
          o |= us[y] + kc;
          us[y] = us[y] * 8u + (kc * 8u + 0x04000400u);
        }
      }
      if (rarely(o & kOff<FMT>)) {
        o = 0;
#pragma unroll
        for (int y = 0; y < NB; ++y)
          us[y] = one_scale<FMT>(sb + S::KS + (tk * NB + y) * S::SB, kc, wd[y], o) * 0x00010001u;
      }
      off = key0 + rk < len && key0 + rk >= min_lo ? o : 0u;
#pragma unroll
      for (int y = 0; y < NB; y += 2) {
        *reinterpret_cast<uint4*>(at_shared(k_to + (y >> 1) * 16384)) = convert8<FMT>(wd[y], us[y]);
        *reinterpret_cast<uint4*>(at_shared((k_to ^ 64u) + (y >> 1) * 16384)) = convert8<FMT>(wd[y + 1], us[y + 1]);
      }
      fence_async_smem();
      tc_fence_before();                                 // (the scores of tile i - 2 have been read)
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_k + (i & 1));
    };
    // ---- values of tile i; then the conversion moves on to the next
    auto convert_values = [&](int i) {
      const uint8_t* sb = at_shared(sub_at + stage * L::TILE);
      const uint32_t v_to = (i & 1) * L::V_OP;
      uint32_t drop = 0, u[NB], wd[NB];
      if (key0 + 8 > len || key0 < min_lo) {
        const int key = key0 + 2 * c;
        drop = (key >= len || key < min_lo ? 1u : 0u) | (key + 1 >= len || key + 1 < min_lo ? 2u : 0u);
      }
      load_words<NB>(wd, sb + S::VC + (half * 32 + lane) * (4 * NB));
      uint32_t o = 0;
      scale_pair<FMT, NB, NVC>(sb + S::VS + (8 * half + 2 * c) * (NB * S::SB), vc, u, o, drop);
      if (rarely(o & kOff<FMT>)) {
        o = 0;
#pragma unroll
        for (int y = 0; y < NB; ++y) {
          u[y] = 0;
#pragma unroll
          for (int t = 0; t < 2; ++t)
            if (!(drop >> t & 1u))
              u[y] |= one_scale<FMT>(sb + S::VS + ((8 * half + 2 * c + t) * NB + y) * S::SB, vc[0],
                                     wd[y] & (FMT == MOE_FMT_MXFP4 ? 0x0F0F0F0Fu << (4 * t) : 0xFFFFu << (16 * t)), o) << (16 * t);
        }
      }
      off |= o;
#pragma unroll
      for (int y = 0; y < NB; ++y) {
        const uint32_t x = FMT == MOE_FMT_MXFP4 ? __funnelshift_r(wd[y], wd[y], 8 * rot) : wd[y];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t v = FMT == MOE_FMT_MXFP4 ? e2m1x2_to_f16x2(x, k)
                                                  : hadd2_bits(lop3_and_xor(x >> (4 * ((k + rot) & 3)), 0x000F000Fu, 0x64086408u), 0xE408E408u);
          *reinterpret_cast<uint32_t*>(at_shared(v_at[k] + v_to + y * 4096)) = hmul2_bits(v, u[y]);
        }
      }
      if (__any_sync(0xFFFFFFFFu, off & kOff<FMT>) && lane == 0) g.redo[cb] = g.redo[a.n_seqs] = 1;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_ring_empty + stage);
      if (++stage == stages) { stage = 0; phase ^= 1; }
      cfirst = false;
      key0 += 128;
      if (++cu == cunits && i + 1 < todo) {
        next_pair(cb, ch_, cu, cunits);
        cfirst = true;
      }
    };
    if (todo > 0) {
      convert_keys(0);
      convert_values(0);
    }
    const int quarter = warp & 3, group = warp >> 2, col0 = group * C, gt = tid & 127, key_in = gt;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    int b = b0, h = h0, u = u0, units = units0, pair = -1, u_first = u0;
    bool first = true, settled = false;
    float l[C / 2][2];
    int ev = 0, min_lim = 0, max_lo = 0;
    const int wnd = g.window > 0 ? g.window : 0x3FFFFFFF;
    const uint32_t p_swizzle = N == 64 ? key_in & 7 : key_in >> 1 & 3;
    const uint32_t p_row = smem_at + L::P + key_in * (2 * N) + (((uint32_t)(col0 / 8) ^ p_swizzle) << 4);
    int k0 = 0;
    for (int i = 0; i < todo; ++i) {
      if (i + 1 < todo) convert_keys(i + 1);
      if (first) {
        const SeqInfo si = info[b];
        ++pair;
        u_first = u;
        k0 = (si.sub0 + u * kTileSubs) * 16;
        min_lim = si.len - si.qn + 1;
        max_lo = si.len - wnd;
        settled = false;
#pragma unroll
        for (int x = 0; x < C; ++x) l[x / 2][x & 1] = 0.f;
        if (gt < C) {
          const int n = col0 + gt, row = (h % RG) * N + n, j = (int)((uint32_t)row * g.group_inv >> 16);
          s_lim[n] = j < si.qn ? si.len - si.qn + j + 1 : 0;
          s_neg[n] = j < si.qn ? FLT_MAX : 0.f;          // (absent rows: their scores of 0 raise nothing)
          s_cnt[n] = 0;
        }
        named_bar(1 + group, 128);
      }
      wait(bar_s + (i & 1), (i >> 1) & 1);
      tc_fence_after();
      if (first) ev = s_ev[pair & 3];
      float t[C / 2][2], big = -INFINITY;                // scores less m
      {
        uint32_t raw[C];
        tc_load<C>(tmem + lanes + (i & 1) * N + col0, raw);
#pragma unroll
        for (int x = 0; x < C; x += 4) {
          const float4 f = *reinterpret_cast<const float4*>(s_f[pair & 3] + col0 + x);
          const float4 m = *reinterpret_cast<const float4*>(s_neg + col0 + x);
          t[x / 2][0] = __uint_as_float(raw[x]); t[x / 2][1] = __uint_as_float(raw[x + 1]);
          t[x / 2 + 1][0] = __uint_as_float(raw[x + 2]); t[x / 2 + 1][1] = __uint_as_float(raw[x + 3]);
          fma2(t[x / 2], t[x / 2], f.x, f.y, m.x, m.y);
          fma2(t[x / 2 + 1], t[x / 2 + 1], f.z, f.w, m.z, m.w);
        }
      }
      const int key = k0 + key_in;
      const bool masked = k0 + 128 > min_lim || k0 < max_lo;
      if (masked) {
#pragma unroll
        for (int x = 0; x < C; ++x) {
          const int top = s_lim[col0 + x];
          if (key >= top || key < top - wnd) t[x / 2][x & 1] = -INFINITY;
        }
      }
#pragma unroll
      for (int x = 0; x < C / 2; ++x) big = max3(t[x][0], t[x][1], big);
      if (rarely(bar_any(1 + group, big > kAnchor + kSlack))) {
        // raise the maxima: over the tile's keys, then the weights, l and the output so far follow
        float v[C];
        uint32_t raw[C];
        tc_load<C>(tmem + lanes + (i & 1) * N + col0, raw);
#pragma unroll
        for (int x = 0; x < C; ++x) {
          const int top = s_lim[col0 + x];
          v[x] = key >= top || key < top - wnd ? -INFINITY : __uint_as_float(raw[x]) * s_f[pair & 3][col0 + x];
          t[x / 2][x & 1] = v[x];
        }
        const float mx = across<C, true>(v);
        if (lane < C) s_max[quarter][col0 + lane] = mx;
        named_bar(1 + group, 128);
        bool few = false;
        if (gt < C) {
          const int n = col0 + gt;
          const float m = -s_neg[n], top = fmaxf(fmaxf(s_max[0][n], s_max[1][n]), fmaxf(s_max[2][n], s_max[3][n]));
          const float m_new = fmaxf(m, top - kAnchor), al = ex2(m - m_new);
          s_neg[n] = -m_new;
          s_al[n] = al;
          // after a raise by up to 2^8 the keys of more than 2^-12 still have more than 2^-20
          const int cnt = al == 1.f ? s_cnt[n] : al < 0.00390625f ? 0 : s_cnt[n] >> 16;
          s_cnt[n] = cnt;
          few = s_lim[n] > 0 && few_keys(cnt);
        }
        settled = !bar_any(1 + group, few);
#pragma unroll
        for (int x = 0; x < C; ++x) {
          t[x / 2][x & 1] += s_neg[col0 + x];
          l[x / 2][x & 1] *= s_al[col0 + x];
        }
        if (!first) {
          wait(&bar_done, (i - 1) & 1);
          tc_fence_after();
          uint32_t ov[C];
          tc_load<C>(tmem_o + lanes + col0, ov);
#pragma unroll
          for (int x = 0; x < C; ++x) ov[x] = __float_as_uint(__uint_as_float(ov[x]) * s_al[col0 + x]);
#pragma unroll
          for (int x = 0; x < C; x += 4) tc_st4(tmem_o + lanes + col0 + x, ov + x);
          tc_wait_st();
          tc_fence_before();
        }
      }
#pragma unroll
      for (int x = 0; x < C / 2; ++x) {
        t[x][0] = ex2(t[x][0]);
        t[x][1] = ex2(t[x][1]);
        add2(l[x], t[x]);
      }
      if (rarely(!settled)) {
        // until a row has 12 keys of weight 2^-20 and more, its weights below 2^-21 go to the other kernel
        int n = 0;
#pragma unroll
        for (int x = 0; x < C; ++x) {
          const uint32_t heavy = __ballot_sync(0xFFFFFFFFu, t[x / 2][x & 1] >= kHeavyW);
          const uint32_t top = __ballot_sync(0xFFFFFFFFu, t[x / 2][x & 1] >= 256.f * kHeavyW);
          if (lane == x) n = __popc(heavy) | __popc(top) << 16;
        }
        const bool counts = few_keys(s_cnt[col0 + lane % C]);
        named_bar(1 + group, 128);                       // (whether a warp's keys count does not depend on who is first)
        if (n && counts) atomicAdd(s_cnt + col0 + lane % C, n);
        named_bar(1 + group, 128);
        bool light = false, few = false;
#pragma unroll
        for (int x = 0; x < C; ++x)
          if (s_lim[col0 + x] > 0 && few_keys(s_cnt[col0 + x])) {
            few = true;
            light |= t[x / 2][x & 1] > 0.f && t[x / 2][x & 1] < kLightW;
          }
        settled = !few;
        if (light) g.redo[b] = g.redo[a.n_seqs] = 1;
        named_bar(1 + group, 128);                       // (the counts have been read)
      }
      if (i > 0) wait(&bar_done, (i - 1) & 1);           // P and V's other operand are free
#pragma unroll
      for (int y = 0; y < C / 8; ++y)
        *reinterpret_cast<uint4*>(at_shared(p_row ^ (16u * y))) = make_uint4(pack_f16(t[4 * y][0], t[4 * y][1]), pack_f16(t[4 * y + 1][0], t[4 * y + 1][1]),
                                                                   pack_f16(t[4 * y + 2][0], t[4 * y + 2][1]), pack_f16(t[4 * y + 3][0], t[4 * y + 3][1]));
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_p);
      if (i + 1 < todo) convert_values(i + 1);
      first = false;
      k0 += 128;
      const bool done = ++u == units, last = i + 1 == todo;
      if (!done && !last) continue;
      const SeqInfo si = info[b];
      // ---- the pair's (part's) end: sums over the keys, the output's dimensions in this thread's lane
      wait(&bar_done, i & 1);
      tc_fence_after();
      uint32_t ov[C];
      tc_load<C>(tmem_o + lanes + col0, ov);
      tc_fence_before();
      {
        float v[C];
#pragma unroll
        for (int x = 0; x < C; ++x) v[x] = l[x / 2][x & 1];
        const float sum = across<C, false>(v);
        if (lane < C) s_max[quarter][col0 + lane] = sum;
      }
      named_bar(1 + group, 128);
      const float val = exp2i(min(127, max(-126, ev)));
      const bool whole = u_first == 0 && done;
      const int slot = u_first == 0 ? 1 : 0;
      float* part = g.cta_parts + ((size_t)blockIdx.x * 2 + slot) * (N * (D + 2));
      if (gt < C) {
        // per row: 1 / sum, and the output row (in s_cnt; below 0: none)
        const int n = col0 + gt, row = (h % RG) * N + n, j = (int)((uint32_t)row * g.group_inv >> 16);
        const float sum = (s_max[0][n] + s_max[1][n]) + (s_max[2][n] + s_max[3][n]), m = -s_neg[n];
        const bool some = sum > 0.f || sum != sum;
        const int at = j < si.qn ? (si.q0 + j) * g.q_heads + (h / RG) * g.group + row - j * g.group : -1;
        s_cnt[n] = at;
        s_al[n] = !some ? 0.f : 1.f / sum;
        if (at >= 0 && whole && g.lse) g.lse[at] = some ? (m + log2f(sum)) * 0.6931471805599453f : -INFINITY;
        if (at >= 0 && !whole) {
          part[N * D + n] = m;
          part[N * D + N + n] = sum;
        }
      }
      named_bar(1 + group, 128);
#pragma unroll
      for (int x = 0; x < C; ++x) {
        const int n = col0 + x, at = s_cnt[n];
        if (at < 0 || key_in >= D) continue;
        const float o = __uint_as_float(ov[x]) * val;
        if (whole)
          g.out[(int64_t)at * D + key_in] = __bfloat16_as_ushort(__float2bfloat16_rn(s_al[n] == 0.f ? 0.f : o * s_al[n]));
        else
          part[n * D + key_in] = o;
      }
      if (!whole && tid == 0) {
        // what the join needs: pair, tiles of this part
        s_used[slot] = b * Hv + h;
        s_tiles[slot] = u - u_first;
      }
      named_bar(1 + group, 128);                         // s_max, s_neg are free again
      if (done && !last) {
        next_pair(b, h, u, units);
        first = true;
      }
    }
    // ---- a pair that spans CTAs: count its tiles; the CTA that completes the count joins the parts in order
    named_bar(15, kWorkers * 32);
    if (tid < 2 && s_used[tid] >= 0) {
      const int pb = s_used[tid] / Hv;
      const uint32_t n = (uint32_t)s_tiles[tid];
      const long long p0 = prefix[pb] + (long long)(s_used[tid] % Hv) * (seq_tiles(info[pb]) + kPairTiles) + kPairTiles;
      uint32_t* cnt = g.counters + first_cta(p0, W, G);
      if (atom_acq_rel_add(cnt, n) + n == (uint32_t)seq_tiles(info[pb])) {
        *cnt = 0;
        s_last[tid] = 1;
      }
    }
    named_bar(15, kWorkers * 32);
    for (int k = 0; k < 2; ++k) {
      if (s_last[k] < 0) continue;
      const int pb = s_used[k] / Hv, ph = s_used[k] % Hv, tiles = seq_tiles(info[pb]);
      const SeqInfo sj = info[pb];
      const long long p0 = prefix[pb] + (long long)ph * (tiles + kPairTiles) + kPairTiles;
      const int c0 = first_cta(p0, W, G), n = (int)(((p0 + tiles) * G - 1) / W) - c0 + 1;
      for (int t = tid; t < N * (D / 4); t += kWorkers * 32) {
        const int d = t % (D / 4) * 4, nr = t / (D / 4), row = (ph % RG) * N + nr, j = (int)((uint32_t)row * g.group_inv >> 16);
        if (j >= sj.qn) continue;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float mx = -FLT_MAX, sum = 0.f;
        constexpr int BATCH = 4;
        for (int i0 = 0; i0 < n; i0 += BATCH) {
          float4 v[BATCH];
          float pm[BATCH], pl[BATCH];
#pragma unroll
          for (int x = 0; x < BATCH; ++x) {
            const float* p = g.cta_parts + ((size_t)(c0 + i0 + x) * 2 + (i0 + x == 0 ? 1 : 0)) * (N * (D + 2));
            const bool in = i0 + x < n;
            v[x] = in ? __ldcg(reinterpret_cast<const float4*>(p + nr * D + d)) : make_float4(0.f, 0.f, 0.f, 0.f);
            pm[x] = in ? __ldcg(p + N * D + nr) : -FLT_MAX;
            pl[x] = in ? __ldcg(p + N * D + N + nr) : 0.f;
          }
          float m_new = mx;
#pragma unroll
          for (int x = 0; x < BATCH; ++x) m_new = pm[x] > m_new || pm[x] != pm[x] ? pm[x] : m_new;
          const float al = ex2(mx - m_new);
          mx = m_new;
          sum *= al;
          acc.x *= al; acc.y *= al; acc.z *= al; acc.w *= al;
#pragma unroll
          for (int x = 0; x < BATCH; ++x) {
            const float wt = ex2(pm[x] - mx);
            sum = fmaf(wt, pl[x], sum);
            acc.x = fmaf(wt, v[x].x, acc.x); acc.y = fmaf(wt, v[x].y, acc.y);
            acc.z = fmaf(wt, v[x].z, acc.z); acc.w = fmaf(wt, v[x].w, acc.w);
          }
        }
        write_row4<D>(g, (int64_t)(sj.q0 + j) * g.q_heads + (ph / RG) * g.group + row - j * g.group, d, acc, mx, sum);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWorkers + 1) tc_dealloc(tmem, L::TMEM_COLS);
}

template <int FMT, int D, int N>
static moe_status_t launch_wide(const Args& a, AttnArgs g, int ctas, cudaStream_t stream) {
  using L = Wide<FMT, D, N>;
  const size_t meta = (size_t)(a.n_seqs + 2) * 8 + (size_t)a.n_seqs * sizeof(SeqInfo), most = kSmemMax - 4096;
  int stages = 4;
  while (stages > 1 && 1024 + L::RING + (size_t)stages * L::TILE + meta > most) --stages;
  g.stages = stages;
  g.rings = L::RING + stages * L::TILE;
  static int configured[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MOE_ERR_CUDA;
  if (!configured[dev]) {
    if (cudaFuncSetAttribute(wide_kernel<FMT, D, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most) != cudaSuccess)
      return MOE_ERR_CUDA;
    configured[dev] = 1;
  }
  wide_kernel<FMT, D, N><<<ctas, kThreads, 1024 + g.rings + meta, stream>>>(a, g);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <int FMT, int D>
static moe_status_t launch_rows(const Args& a, AttnArgs g, int ctas, cudaStream_t stream) {
  const int rows = a.max_q * g.group;
  g.row_groups = rows <= 64 ? 1 : 2;
  return rows <= 32 ? launch_wide<FMT, D, 32>(a, g, ctas, stream) : launch_wide<FMT, D, 64>(a, g, ctas, stream);
}

moe_status_t attn_wide(const Args& a, AttnArgs g, int fmt, int D, int ctas, cudaStream_t stream) {
  if (fmt == MOE_FMT_MXFP4)
    return D == 64 ? launch_rows<MOE_FMT_MXFP4, 64>(a, g, ctas, stream) : launch_rows<MOE_FMT_MXFP4, 128>(a, g, ctas, stream);
  return D == 64 ? launch_rows<MOE_FMT_INT4G32, 64>(a, g, ctas, stream) : launch_rows<MOE_FMT_INT4G32, 128>(a, g, ctas, stream);
}

}  // namespace kv
}  // namespace moe
