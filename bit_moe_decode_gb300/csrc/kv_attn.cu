// kv_attn.cu -- attention of a decode or verify step over the 4-bit paged KV cache.
//
// For each query row: x_s = scale q . k_s over the visible keys s, out = sum_s softmax(x)_s v_s, lse = log sum_s exp(x_s), in
// one pass over the keys with a running maximum m and sum l.
//
// What bounds it. A key of one KV head is 136 bytes (MXFP4, D = 128) of HBM traffic and 256 codes to convert. At the
// measured 6.7 TB/s an SM gets 44 bytes per ns, so it has about 24 issue slots per warp-wide MMA (16 keys x 16
// dimensions) and half as many in the integer pipe. Everything below serves to convert a code with as few instructions
// as possible, once per 8 query rows. What it reaches: 64 sequences of up to 8192 keys, 8 rows a KV head (4 KV heads, D = 128,
// MXFP4) 44.6 us, 3.3 TB/s (47 % of the issue slots, 44 % of the integer pipe); one of 262143 keys (8 KV heads, INT4) 77.6 us,
// 3.9 TB/s; one of 517 keys 10.5 us, latency; 256 of up to 600, 1 row a KV head (16, D = 64, INT4) 44.2 us, pairs' starts and
// ends.
//
// Work. The (sequence, KV head) pairs are laid end to end in units of 32 keys, a pair's start counting as some units more
// (what its queries and its output cost), and dealt out evenly: every warp of the grid streams one contiguous run (the
// prefix sums over the sequences are formed by each CTA from the device's lengths, so a captured graph follows them). A warp
// copies its units with bulk copies (one per 16-token sub-block, which the layout keeps contiguous) into its own ring and
// is its own consumer, so there is no barrier between warps until the end. A pair that lies in several warps is joined
// from partial results, first inside the CTA, then, if it spans CTAs, by the CTA that finishes last (a counter, left at zero); always in the order of
// the keys, so the bits do not depend on timing. More than 8 NT query rows: RG warps stream the same units, each
// for its own rows (the copies then hit L2). Above 16 rows over long sequences kv_attn_wide.cu goes first, and this kernel
// does again what that one marks.
//
// Arithmetic, for 16 keys x 8 rows at a time on mma.sync.m16n8k16 with the keys (then the dimensions) as the 16 rows,
// so that a decode step's few query rows fill the 8 columns:
//   S^T = K Q^T: a K word holds 8 codes of one key whose order in the contraction is free, so a lane's 16 bytes of a key
//     are its A fragments of all blocks. Codes become exact binary16 (E2M1: one conversion per pair; INT4: the nibble
//     + 8 as a subnormal n 2^-24 or n 2^-20 by one mask, with -8 sum q as the accumulator's start and 2^-4 in q's
//     fragments), q is scaled by a power of two into binary16, and each block's scale multiplies its fp32 partial.
//   O^T += V^T P^T: the V layout puts an even and the following odd token's codes of one dimension side by side, which
//     is what an A fragment's register holds. movmatrix turns the weights' accumulator layout into a B fragment. V's
//     scales vary along the contraction, so they go into the weights: p_s is rounded to binary16 and multiplied by vscale_s
//     there, which is exact for MXFP4's powers of two and rounds a second time for INT4's bf16 scales. (One rounding in fp32
//     would take a conversion per block and pair of keys instead of one per pair.)
//   Range: the weights are carried as 2^12 p, at most 2^14 (m is raised only when a score passes m + 2), and the value
//     scales as v 2^-E in binary16, exact within 2^-14 .. 2^2; the fp32 accumulators hold 2^(12 - E) times the output. E is set
//     by the first unit of a warp's part of a pair (its largest scale lies 2 below), and moves per block of 32 dimensions.
//     Products keep all 11 bits down to 2^-14, 2^-24 of the largest. Where scales leave the window, E moves (accumulators
//     rescaled, exactly) and the keys take passes: each adds the products of the next 26 powers of two at a scale of its own, so
//     that no ratio of scales costs precision. So do keys of weights below 2^-24 until each row has seen 12 keys of more
//     than 2^-14 (counts are halved when its maximum rises, and forgotten when that is by 2^4): a dimension whose few heavy
//     keys all have code 0 is made of such weights. E stays within 36 of the largest scale that the accumulators can hold, which
//     is what keeps them and the passes' 2^52 (2^78 within 10) in fp32's range.
#include <algorithm>

#include "kv_attn.cuh"

namespace moe {
namespace kv {

constexpr int kUnitSubs = 2;        // sub-blocks per unit
constexpr int kBatch = 16;          // units whose addresses a warp's lanes hold at a time
constexpr int kEvMin = -112;            // the smallest E (a scale byte of 0, which stands for zero, is below its window)
constexpr float kNormal = 6.103515625e-05f;   // 2^-14: binary16 products from here on keep all bits
constexpr int kPassExp = 26;            // powers of two that a pass covers

__device__ __forceinline__ uint32_t transpose8(uint32_t v) {   // 8 x 8 of 16 bits over the warp
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two keys' K words (rows r and r + 8) of one block -> the A fragments of its two k-steps.
template <int FMT>
__device__ __forceinline__ void decode_k(uint32_t w0, uint32_t w1, uint32_t (&a)[2][4]) {
  if (FMT == MOE_FMT_MXFP4) {
    a[0][0] = e2m1x2_to_f16x2(w0, 0); a[0][1] = e2m1x2_to_f16x2(w1, 0);
    a[0][2] = e2m1x2_to_f16x2(w0, 1); a[0][3] = e2m1x2_to_f16x2(w1, 1);
    a[1][0] = e2m1x2_to_f16x2(w0, 2); a[1][1] = e2m1x2_to_f16x2(w1, 2);
    a[1][2] = e2m1x2_to_f16x2(w0, 3); a[1][3] = e2m1x2_to_f16x2(w1, 3);
  } else {   // code + 8 as n 2^-24 (first of a pair of steps' registers) and n 2^-20 (second)
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      a[s][0] = lop3_and_xor(w0, 0x000F000Fu, 0x00080008u); a[s][1] = lop3_and_xor(w1, 0x000F000Fu, 0x00080008u);
      a[s][2] = lop3_and_xor(w0, 0x00F000F0u, 0x00800080u); a[s][3] = lop3_and_xor(w1, 0x00F000F0u, 0x00800080u);
      w0 >>= 8;
      w1 >>= 8;
    }
  }
}

// V words of tokens 2c, 2c + 1 (w0) and 2c + 8, 2c + 9 (w1) of one block -> the A fragments of its two 16-dimension tiles.
// INT4 values come out as q 2^-24 in the fragments' first row half, q 2^-20 in the second.
template <int FMT>
__device__ __forceinline__ void decode_v(uint32_t w0, uint32_t w1, uint32_t (&a)[2][4]) {
  if (FMT == MOE_FMT_MXFP4) {
    a[0][0] = e2m1x2_to_f16x2(w0, 0); a[0][1] = e2m1x2_to_f16x2(w0, 1);
    a[0][2] = e2m1x2_to_f16x2(w1, 0); a[0][3] = e2m1x2_to_f16x2(w1, 1);
    a[1][0] = e2m1x2_to_f16x2(w0, 2); a[1][1] = e2m1x2_to_f16x2(w0, 3);
    a[1][2] = e2m1x2_to_f16x2(w1, 2); a[1][3] = e2m1x2_to_f16x2(w1, 3);
  } else {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      a[s][0] = hadd2_bits(lop3_and_xor(w0, 0x000F000Fu, 0x00080008u), 0x80088008u);
      a[s][1] = hadd2_bits(lop3_and_xor(w0, 0x00F000F0u, 0x00800080u), 0x80808080u);
      a[s][2] = hadd2_bits(lop3_and_xor(w1, 0x000F000Fu, 0x00080008u), 0x80088008u);
      a[s][3] = hadd2_bits(lop3_and_xor(w1, 0x00F000F0u, 0x00800080u), 0x80808080u);
      w0 >>= 8;
      w1 >>= 8;
    }
  }
}

__device__ __forceinline__ int seq_units(const SeqInfo& s) {
  return s.qn > 0 && s.len > 0 ? ((s.len + 15) / 16 - s.sub0 + kUnitSubs - 1) / kUnitSubs : 0;
}

// A pair's place in the list of work: kPairCost, then its units.
// (Measured in units of a warp: decode 256 x 600 47.6, 45.6, 44.6, 45.1 us at 1, 2, 3, 4; 16 rows, 64 x 8192 with 8 KV heads,
// 124, 129, 135 us at 1, 2, 3, where two warps or more share the units.)
template <int NT>
constexpr int pair_cost = NT == 1 ? 3 : 1;
template <int NT>
__device__ __forceinline__ int seq_cost(const SeqInfo& s) {
  const int u = seq_units(s);
  return u ? u + pair_cost<NT> : 0;
}
struct Prod {        // a warp's producer: the next batch is n units (subs sub-blocks from `sub` on) at unit u of a pair; left
  int b, h, u, units, left, n, subs, sub;   // counts the units from it on
  int ev_run[4];     // and of its consumer, per block: no value scale with a weight has had a larger exponent so far,
  int ev_ref[4];     // and the E in use (units in its window have scales of up to 2^(E + 1))
};

struct Entry { int u0, u1, b, h; };   // a partial result of one warp: units [u0, u1) of pair (b, h); b < 0: none
struct Run { int u0, u1, b, h, first, n, slot, whole; };      // n consecutive entries of one pair, from list place `first`
struct Place { const float* p; int step, at; };   // an entry's values, floats from one row group's to the next's, its place

template <int FMT, int D, int NT, int NW, int SUBS>
__global__ void __launch_bounds__(NW * 32, 1) attn_kernel(Args a, AttnArgs g) {
  using S = Sub<FMT, D>;
  constexpr int NB = S::NB, UNIT = kUnitSubs * S::BYTES, ROWS = 8 * NT, THREADS = NW * 32;
  constexpr int PART = ROWS * (D + 2);                   // floats of a warp's partial: o [ROWS][D], m [ROWS], l [ROWS]
  constexpr int NVC = FMT == MOE_FMT_MXFP4 ? 1 : NB;
  constexpr float kVal = FMT == MOE_FMT_INT4G32 ? 16777216.f : 1.f;   // 2^24 of the INT4 fragments
  constexpr int kPairCost = pair_cost<NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Entry s_entry[2 * NW];
  __shared__ Run s_run[2 * NW];
  __shared__ Place s_place[2 * NW];
  __shared__ int s_runs, s_last[2];
  __shared__ float s_wt[2 * NW * ROWS], s_m[2 * NW * ROWS], s_l[2 * NW * ROWS];   // [entry or run][row]
  __shared__ long long s_warp[NW], s_total;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, c = lane & 3;
  const int stages = g.stages, RG = g.row_groups, KS = NW / RG, Hkv = a.kv_heads;
  const int stream = warp / RG, rg = warp % RG;
  uint8_t* ring = smem + (size_t)warp * stages * UNIT;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + g.rings);
  uint64_t* bar = bars + warp * stages;
  long long* prefix = reinterpret_cast<long long*>(bars + NW * stages);           // [n_seqs + 1]
  SeqInfo* info = reinterpret_cast<SeqInfo*>(prefix + a.n_seqs + 1 + ((a.n_seqs + 1) & 1));
  Prod* prods = reinterpret_cast<Prod*>(info + a.n_seqs);

  if (NT > 1 && g.redo && __ldcg(g.redo + a.n_seqs) == 0) return;   // nothing was left over
  // ---- the sequences: lengths, first visible sub-block, prefix sums of their units over all KV heads, how many have any
  int live = 0;
  if (lane < stages) mbar_init(bar + lane, 1);
  if (tid < 2 * NW) s_entry[tid].b = -1;
  if (tid == 0) { prefix[0] = 0; s_total = 0; }
  for (int base = 0; base < a.n_seqs; base += NW * 32) {
    const int b = base + tid;
    long long x = 0;
    if (b < a.n_seqs) {
      const Seq sq = check_seq(a, a.q_start[b], a.q_start[b + 1], a.seq_len[b], a.max_q);
      SeqInfo si{sq.q0, sq.qn, sq.len, 0};
      if (NT > 1 && g.redo && __ldcg(g.redo + b) == 0) si.qn = 0;
      if (g.window > 0 && sq.len - sq.qn - g.window + 1 > 0) si.sub0 = (sq.len - sq.qn - g.window + 1) / 16;
      info[b] = si;
      x = (long long)seq_cost<NT>(si) * Hkv;
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
    if (tid == NW * 32 - 1) s_total = x + add;
  }
  fence_mbar_init();
  __syncthreads();
  const long long W = prefix[a.n_seqs];
  if (NT > 1 && g.redo && tid == 0 && atom_acq_rel_add(g.redo + a.n_seqs + 1, 1) == gridDim.x - 1)
    for (int b = 0; b < a.n_seqs + 2; ++b) g.redo[b] = 0;   // every CTA has read them

  // rows of empty sequences
  for (int b = blockIdx.x; b < a.n_seqs; b += gridDim.x) {
    const SeqInfo si = info[b];
    if (si.qn <= 0 || seq_units(si) > 0) continue;
    const int64_t r0 = (int64_t)si.q0 * g.q_heads, n = (int64_t)si.qn * g.q_heads;
    for (int64_t i = tid; i < n * (D / 8); i += NW * 32) reinterpret_cast<uint4*>(g.out + r0 * D)[i] = make_uint4(0, 0, 0, 0);
    if (g.lse)
      for (int64_t i = tid; i < n; i += NW * 32) g.lse[r0 + i] = -INFINITY;
  }

  // ---- this warp's run [f_begin, f_end) of the list
  if (W == 0) return;
  // G: about two units a stream at least; where that leaves SMs over, a multiple of the pairs, so that a pair of an even
  // batch ends where a CTA does (a pair within one CTA needs no join across CTAs, 3 us). Only pairs that have units count: with
  // W >= 2 pairs, G is then at most W, so that every CTA has a place of the list. The joins rely on it: each CTA from a pair's
  // first unit's to its last unit's has written a part.
  const long long pairs = (long long)live * Hkv, even = (W + 2 * KS * pairs - 1) / (2 * KS * pairs) * pairs;
  const int G = (int)min(even, (long long)gridDim.x);
  const int N = G * KS;
  if (blockIdx.x >= G) return;
  const int sidx = blockIdx.x * KS + stream;
  const long long f_begin = share(sidx, W, N), f_end = share(sidx + 1, W, N);

  // The unit u of `units` of KV head h of sequence b that the run starts with, and how many units it holds.
  int cb = 0, ch = 0, cu = 0, cunits = 0, todo = 0;
  if (f_begin < f_end) {
    int lo = 0, hi = a.n_seqs;                 // the last b with prefix[b] <= f_begin
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= f_begin) lo = mid;
      else hi = mid;
    }
    cb = lo;
    cunits = seq_units(info[lo]);
    const int cost = cunits + kPairCost;
    const long long rem = f_begin - prefix[lo];
    ch = (int)share(rem, 1, cost);
    int at = (int)(rem - (long long)ch * cost);            // 0 .. cost - 1: the pair's start, or its unit at - kPairCost
    cu = max(0, at - kPairCost);
    // units in [f_begin, f_end): all but the pair starts; counted pair by pair, in one step within a sequence
    long long left = f_end - f_begin;
    for (int b = lo, h = ch, units = cunits; left > 0;) {
      const int here = (int)min(left, (long long)(units + kPairCost - at));
      todo += max(0, at + here - max(at, kPairCost));
      left -= here;
      at = 0;
      if (++h < Hkv) {
        const int n = (int)min(share(left, 1, units + kPairCost), (long long)(Hkv - h));
        todo += n * units;
        left -= (long long)n * (units + kPairCost);
        h += n;
      }
      if (h == Hkv && left > 0) {
        h = 0;
        do units = seq_units(info[++b]); while (units == 0);
      }
    }
  }
  // to the next pair (there is one: units remain)
  auto next_pair = [&](int& b, int& h, int& u, int& units) {
    u = 0;
    if (++h < Hkv) return;
    h = 0;
    do units = seq_units(info[++b]); while (units == 0);
  };

  // ---- producer: addresses of up to 16 units (32 sub-blocks, one a lane) at a time, the next batch's table entries
  // fetched ahead. The state that only a change of batch needs is kept in shared memory.
  Prod* pr = prods + warp;
  const uint8_t* cur_ptr = nullptr;
  int cur_n = 0, cur_subs = 0, next_id = 0;
  auto fetch = [&]() {                         // describes the next batch and loads its table entries
    Prod p = *pr;
    __syncwarp();
    if (p.n > 0) {                             // past the batch that was current
      p.left -= p.n;
      p.u += p.n;
      if (p.u == p.units && p.left > 0) next_pair(p.b, p.h, p.u, p.units);
    }
    p.n = min(min(kBatch, p.units - p.u), p.left);
    if (p.n > 0) {
      const SeqInfo s = info[p.b];
      const int sub = s.sub0 + p.u * kUnitSubs;
      p.subs = min(p.n * kUnitSubs, (s.len + 15) / 16 - sub);
      p.sub = sub;
      if (lane < p.subs)
        next_id = __ldg(a.block_table + (int64_t)p.b * a.table_stride + (sub + lane) / (a.page_tokens / 16));
    }
    if (lane == 0) {
      pr->b = p.b; pr->h = p.h; pr->u = p.u; pr->units = p.units;
      pr->left = p.left; pr->n = p.n; pr->subs = p.subs; pr->sub = p.sub;
    }
    __syncwarp();
  };
  auto take = [&]() {                          // makes the described batch the current one
    const Prod p = *pr;
    cur_n = p.n;
    cur_subs = p.subs;
    if (p.n > 0 && lane < p.subs) {
      const int per_page = a.page_tokens / 16, sub = p.sub + lane;
      bool ok;
      const int id = check_page(a, next_id, ok);
      cur_ptr = a.pages + (int64_t)id * a.page_stride + (int64_t)(p.h * per_page + sub % per_page) * S::BYTES;
    }
    __syncwarp();
    fetch();
  };
  if (lane == 0) *pr = Prod{cb, ch, cu, cunits, todo, 0, 0, 0, {0, 0, 0, 0}, {0, 0, 0, 0}};
  __syncwarp();
  fetch();
  int bi = 0, issued = 0, istage = 0;       // unit within the batch; units issued in all; stage of the next issue
  auto issue = [&]() {                      // every lane of the warp has read what the stage held
    if (issued >= todo) return;
    const bool mine = (lane >> 1) == bi && lane < cur_subs;
    if (mine && !(lane & 1)) mbar_arrive_expect_tx(bar + istage, (lane + 1 < cur_subs ? 2 : 1) * S::BYTES);
    __syncwarp();
    if (mine) bulk_g2s_plain(ring + istage * UNIT + (lane & 1) * S::BYTES, cur_ptr, S::BYTES, bar + istage);
    ++issued;
    if (++istage == stages) istage = 0;
    if (++bi == cur_n) {
      bi = 0;
      take();
    }
  };

  // ---- consumer
  uint32_t qf[NT][NB][4];
  float ci[NT][NB][2], fx[NT][2], m[NT][2], l[NT][2], o[NT][NB][2][4];   // m: the maximum - 12
  uint32_t vc[NVC];                          // E as the conversion of value scales takes it
  bool settled = false;                      // each row has had 12 keys of some weight (see above);
  int heavy = 0;                             // their counts until then, a byte a row
  int lim[NT][2];                            // a row sees keys below this
  int seg_len = 0, min_lim = 0, key0 = 0;    // the pair's keys, what all rows see, the next unit's first key
  const int wnd = g.window > 0 ? g.window : 0x3FFFFFFF;

  auto set_ref = [&]() {
    // minus the exponent of the window's lower end, E + 127 - 14, per block: in its byte (MXFP4) or at bf16's exponent's
    // place in both halves (INT4). Signed terms, so that an E near the smallest exponent works too.
    if (FMT == MOE_FMT_MXFP4) {
      int low = 0;
#pragma unroll
      for (int b = 0; b < NB; ++b) low += (pr->ev_ref[b] + 113) * (1 << (8 * b));
      if (NB == 2) low += low * 65536;
      vc[0] = 0u - (uint32_t)low;
    } else {
#pragma unroll
      for (int b = 0; b < NB; ++b) vc[b % NVC] = 0u - (uint32_t)((pr->ev_ref[b] + 113) * 0x00800080);
    }
  };
  // B fragments: this lane holds row r of the 8 and dimensions 32 b + 8 c .. + 7
  uint4 qw[NT][NB];
  auto load_q = [&]() {
    const int q0 = info[cb].q0, qn = info[cb].qn;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = (rg * NT + nt) * 8 + r, j = (int)((uint32_t)row * g.group_inv >> 16);
      const uint16_t* p = g.q + (int64_t)(q0 + j) * g.q_stride + (int64_t)(ch * g.group + row - j * g.group) * D + 8 * c;
#pragma unroll
      for (int b = 0; b < NB; ++b)
        qw[nt][b] = j < qn ? __ldg(reinterpret_cast<const uint4*>(p + 32 * b)) : make_uint4(0, 0, 0, 0);
    }
  };
  auto begin_segment = [&]() {
    const SeqInfo si = info[cb];
    seg_len = si.len;
    min_lim = si.len - si.qn + 1;
    key0 = (si.sub0 + cu * kUnitSubs) * 16;
    settled = false;
    heavy = 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float amax = 0.f;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint32_t u[4] = {qw[nt][b].x, qw[nt][b].y, qw[nt][b].z, qw[nt][b].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(u[i] << 16)), fabsf(__uint_as_float(u[i] & 0xFFFF0000u))));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
      const int sg = rescale_exponent(amax);
      const float up = exp2i(sg);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint32_t u[4] = {qw[nt][b].x, qw[nt][b].y, qw[nt][b].z, qw[nt][b].w};
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[2 * i] = __uint_as_float(u[i] << 16) * up;
          v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u) * up;
        }
        if (FMT == MOE_FMT_MXFP4) {
#pragma unroll
          for (int i = 0; i < 4; ++i) qf[nt][b][i] = pack_f16(v[2 * i], v[2 * i + 1]);
        } else {
          // pairs (i, i + 4); those that meet n 2^-20 carry 2^-4. The sum of what the fragments hold corrects the + 8.
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float w4 = i & 1 ? 0.0625f : 1.f;
            qf[nt][b][i] = pack_f16(v[i] * w4, v[i + 4] * w4);
            const __half2 hh = *reinterpret_cast<const __half2*>(&qf[nt][b][i]);
            sum += (__low2float(hh) + __high2float(hh)) * (i & 1 ? 16.f : 1.f);
          }
          sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
          sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
          const float start = -8.f / kVal * sum;
          ci[nt][b][0] = __shfl_sync(0xFFFFFFFFu, start, 8 * c);
          ci[nt][b][1] = __shfl_sync(0xFFFFFFFFu, start, 8 * c + 4);
        }
      }
      // accumulator columns: rows 2 c and 2 c + 1 of the 8
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int s_row = __shfl_sync(0xFFFFFFFFu, sg, 8 * c + 4 * e);
        fx[nt][e] = g.scale_log2 * exp2i_neg(s_row) * kVal;
        const int row_e = (rg * NT + nt) * 8 + 2 * c + e, je = (int)((uint32_t)row_e * g.group_inv >> 16);
        lim[nt][e] = je < si.qn ? si.len - si.qn + je + 1 : 0;
        m[nt][e] = -FLT_MAX;
        l[nt][e] = 0.f;
      }
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][b][x][e] = 0.f;
    }
  };

  // E from the segment's first unit: its largest scale (of tokens that some row sees) lies 2 below E, so 12 powers of two below
  // that and 3 above it are in the window. (All blocks the same: four maxima cost 0.1 us a call more than one.)
  auto first_window = [&](const uint8_t* unit) {
    const int key = key0 + lane, n = key < seg_len && key >= min_lim - wnd ? 255 : 0;
    const uint8_t* p = unit + (lane >> 4) * S::BYTES + S::VS + (lane & 15) * (NB * S::SB);
    int e = 0;
#pragma unroll
    for (int b = 0; b < NB; ++b) e = max(e, FMT == MOE_FMT_MXFP4 ? (int)p[b] : (int)(reinterpret_cast<const uint16_t*>(p)[b] >> 7));
    const int ev = max((int)__reduce_max_sync(0xFFFFFFFFu, (uint32_t)(e & n)) - 125, kEvMin);
    __syncwarp();
    if (lane < NB) {
      pr->ev_run[lane] = ev + 1;
      pr->ev_ref[lane] = ev;
    }
    __syncwarp();
    set_ref();
  };

  // The rare path: value scales outside E's window. Moves E to the largest, then adds the products of the weights s (times
  // 2^12) and the scales in passes.
  auto wide_products = [&](const uint8_t* base, const float (&s)[SUBS][NT][4]) {
    // Scales of 2^-100 of the largest so far and less count as zero: the passes do not reach them, and blocks of zeros, which
    // have the smallest scale, move nothing.
    auto value_scales = [&](const uint8_t* sb, float (&v0)[NB], float (&v1)[NB]) {
      load_scales<FMT, NB>(v0, sb + S::VS + r * (NB * S::SB));
      load_scales<FMT, NB>(v1, sb + S::VS + (r + 8) * (NB * S::SB));
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int none = (pr->ev_run[b] + 27) << 23;   // (of positive numbers, the bits order as the numbers do)
        if (__float_as_int(v0[b]) <= none) v0[b] = 0.f;
        if (__float_as_int(v1[b]) <= none) v1[b] = 0.f;
      }
    };
    float most[NB];              // (a weight of 0 has no product, whatever bytes its scale is)
#pragma unroll
    for (int b = 0; b < NB; ++b) most[b] = 0.f;
#pragma unroll 1
    for (int i = 0; i < SUBS; ++i) {
      float v0[NB], v1[NB];
      value_scales(base + i * S::BYTES, v0, v1);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if ((SUBS == 1 || i == 0 ? s[0][nt][e] : s[SUBS - 1][nt][e]) > 0.f)
#pragma unroll
            for (int b = 0; b < NB; ++b) most[b] = fmaxf(most[b], e & 2 ? v1[b] : v0[b]);
    }
    int depth = 3;               // passes after the first that the accumulators' range allows
    __syncwarp();
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float vm = most[b];
#pragma unroll
      for (int i = 1; i < 32; i <<= 1) vm = fmaxf(vm, __shfl_xor_sync(0xFFFFFFFFu, vm, i));
      const int e_old = pr->ev_ref[b];
      int run = pr->ev_run[b], e_new = e_old;
      if (vm > 0.f) {
        // Accumulators stay below 2^(38 + run - E) for a million keys: E at least run - 36 keeps two passes' 2^52 in range (run
        // covers the units of the main path too: each window's top)
        const int ev = (int)(__float_as_uint(vm) >> 23) - 127;
        run = max(run, ev);
        e_new = max(ev <= e_old + 1 && ev >= e_old - 10 ? e_old : ev, max(run - 36, kEvMin));   // (ev is -126 .. 127)
      }
      depth = min(depth, run - e_new <= 10 ? 3 : 2);
      __syncwarp();
      if (lane == 0) { pr->ev_run[b] = max(run, e_new + 1); pr->ev_ref[b] = e_new; }
      const float f1 = exp2i((e_old - e_new) >> 1), f2 = exp2i(e_old - e_new - ((e_old - e_new) >> 1));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][b][x][e] = o[nt][b][x][e] * f1 * f2;
    }
    __syncwarp();
    set_ref();
    for (int pass = 0;; ++pass) {
      const float up = exp2i(kPassExp * pass), top = pass ? kNormal * exp2i(kPassExp) : FLT_MAX;
      bool left = false;
#pragma unroll 1
      for (int i = 0; i < SUBS; ++i) {
        const uint8_t* sb = base + i * S::BYTES;
        uint32_t vw0[NB], vw1[NB];
        float v0[NB], v1[NB];
        load_words<NB>(vw0, sb + S::VC + (r * 4 + c) * (4 * NB));
        load_words<NB>(vw1, sb + S::VC + (32 + r * 4 + c) * (4 * NB));
        value_scales(sb, v0, v1);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const float fr = exp2i(-pr->ev_ref[b]);
          uint32_t f[2][4];
          decode_v<FMT>(vw0[b], vw1[b], f);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float p = SUBS == 1 || i == 0 ? s[0][nt][e] : s[SUBS - 1][nt][e];
              const float x = p == 0.f ? 0.f : p * ((e & 2 ? v1[b] : v0[b]) * fr) * up;
              left |= x > 0.f && x < kNormal;
              w[e] = x < kNormal || x >= top ? 0.f : x;      // (NaN stays)
            }
            const uint32_t p0 = transpose8(pack_f16(w[0], w[1])), p1 = transpose8(pack_f16(w[2], w[3]));
            mma(o[nt][b][0], f[0], p0, p1);
            mma(o[nt][b][1], f[1], p0, p1);
          }
        }
      }
      const bool again = pass < depth && __any_sync(0xFFFFFFFFu, left);
      if (!again && pass == 0) return;
      const float f = exp2i(again ? kPassExp : -kPassExp * pass);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][b][x][e] *= f;
      if (!again) return;
    }
  };

  // the first copies, with the first queries' loads on the way
  if (todo > 0) load_q();
  take();
  for (int i = 0; i < stages; ++i) issue();

  // SUBS sub-blocks of 16 keys, from k0 on
  auto process = [&](const uint8_t* base, int k0) {
    float s[SUBS][NT][4];
    uint32_t u0[SUBS][NB], u1[SUBS][NB], off = 0;
#pragma unroll
    for (int i = 0; i < SUBS; ++i) {
      const uint8_t* sb = base + i * S::BYTES;
      uint32_t kw0[NB], kw1[NB];
      float ks0[NB], ks1[NB];
      load_words<NB>(kw0, sb + S::KC + r * (D / 2) + c * (4 * NB));
      load_words<NB>(kw1, sb + S::KC + (r + 8) * (D / 2) + c * (4 * NB));
      load_scales<FMT, NB>(ks0, sb + S::KS + r * (NB * S::SB));
      load_scales<FMT, NB>(ks1, sb + S::KS + (r + 8) * (NB * S::SB));
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        uint32_t f[2][4];
        decode_k<FMT>(kw0[b], kw1[b], f);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float d[4] = {0.f, 0.f, 0.f, 0.f};
          if (FMT == MOE_FMT_INT4G32) { d[0] = d[2] = ci[nt][b][0]; d[1] = d[3] = ci[nt][b][1]; }
          mma(d, f[0], qf[nt][b][0], qf[nt][b][1]);
          mma(d, f[1], qf[nt][b][2], qf[nt][b][3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float ks = e & 2 ? ks1[b] : ks0[b];
            s[i][nt][e] = b == 0 ? ks * d[e] : fmaf(ks, d[e], s[i][nt][e]);
          }
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][nt][e] *= fx[nt][e & 1];
      if (rarely(k0 + 16 * (i + 1) > min_lim || k0 + 16 * i < seg_len - wnd)) {   // some row does not see some key
        const int ka = k0 + 16 * i + r;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = e & 2 ? ka + 8 : ka, top = lim[nt][e & 1];
            if (key >= top || key < top - wnd) s[i][nt][e] = -INFINITY;
          }
        // bytes past the end or before the window may be anything: their scales are replaced (their weights are 0)
        const int kt = k0 + 16 * i + 2 * c, min_lo = min_lim - wnd;
        uint32_t drop = 0;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int key = kt + (t & 1) + (t & 2 ? 8 : 0);
          drop |= (key >= seg_len || key < min_lo ? 1u : 0u) << t;
        }
        scale_pairs<FMT, NB, NVC>(sb + S::VS, c, vc, u0[i], u1[i], off, drop);
      } else {
        scale_pairs<FMT, NB, NVC>(sb + S::VS, c, vc, u0[i], u1[i], off, 0u);
      }
    }
    float tmax = -INFINITY;
#pragma unroll
    for (int i = 0; i < SUBS; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        tmax = max3(max3(s[i][nt][0] - m[nt][0], s[i][nt][1] - m[nt][1], s[i][nt][2] - m[nt][0]), s[i][nt][3] - m[nt][1], tmax);
    if (rarely(__any_sync(0xFFFFFFFFu, tmax > kPExp + kLazy))) {   // raise the maxima
      settled = false;
      heavy = heavy >> 1 & 0x7F7F7F7F;   // (some of the keys that counted no longer do; none after a large step)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = -INFINITY;
#pragma unroll
          for (int i = 0; i < SUBS; ++i) mx = max3(mx, s[i][nt][e], s[i][nt][e + 2]);
#pragma unroll
          for (int i = 4; i < 32; i <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, i));
          mx = fmaxf(m[nt][e], mx - kPExp);
          const float al = ex2(m[nt][e] - mx);
          if (al < 0.0625f) heavy &= ~(255 << (8 * (2 * nt + e)));
          m[nt][e] = mx;
          l[nt][e] *= al;
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              o[nt][b][x][e] *= al;
              o[nt][b][x][e + 2] *= al;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < SUBS; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][nt][e] = ex2(s[i][nt][e] - m[nt][e & 1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) l[nt][e] += s[i][nt][e] + s[i][nt][e + 2];
      }
    bool wide = off & kOff<FMT>;
    if (rarely(!settled)) {
      // heavy keys per row, four counts in an int, over the lanes that share the rows; and the rows with light ones
      int n = 0, light = 0;
#pragma unroll
      for (int i = 0; i < SUBS; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            n += (s[i][nt][e] >= kHeavy ? 1 : 0) << (8 * (2 * nt + (e & 1)));
            light |= (s[i][nt][e] > 0.f && s[i][nt][e] < kLight ? 1 : 0) << (2 * nt + (e & 1));
          }
#pragma unroll
      for (int i = 4; i < 32; i <<= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, i);
      bool all = true;
#pragma unroll
      for (int k = 0; k < 2 * NT; ++k) {
        const int sum = min(128, (heavy >> (8 * k) & 255) + (n >> (8 * k) & 255));
        heavy = (heavy & ~(255 << (8 * k))) | sum << (8 * k);
        const bool few = sum < 12 && lim[k / 2][k % 2] != 0;
        all = all && !few;
        wide |= few && (light >> k & 1);
      }
      settled = __all_sync(0xFFFFFFFFu, all);
    }
    if (rarely(__any_sync(0xFFFFFFFFu, wide))) {
      wide_products(base, s);
      return;
    }
#pragma unroll
    for (int i = 0; i < SUBS; ++i) {
      uint32_t vw0[NB], vw1[NB], t0[NT], t1[NT];
      load_words<NB>(vw0, base + i * S::BYTES + S::VC + (r * 4 + c) * (4 * NB));
      load_words<NB>(vw1, base + i * S::BYTES + S::VC + (32 + r * 4 + c) * (4 * NB));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        t0[nt] = transpose8(pack_f16(s[i][nt][0], s[i][nt][1]));
        t1[nt] = transpose8(pack_f16(s[i][nt][2], s[i][nt][3]));
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        uint32_t f[2][4];
        decode_v<FMT>(vw0[b], vw1[b], f);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint32_t p0 = hmul2_bits(t0[nt], u0[i][b]), p1 = hmul2_bits(t1[nt], u1[i][b]);
          mma(o[nt][b][0], f[0], p0, p1);
          mma(o[nt][b][1], f[1], p0, p1);
        }
      }
    }
  };

  // o (times 2^12, as l) in true scale relative to the maximum: dimensions 32 b + 4 r .. + 3 of row 2 c + e
  auto value4 = [&](int nt, int e, int b) {
    const float s = kVal * exp2i(pr->ev_ref[b]), s2 = FMT == MOE_FMT_INT4G32 ? s * 0.0625f : s;
    return make_float4(o[nt][b][0][e] * s, o[nt][b][0][e + 2] * s2, o[nt][b][1][e] * s, o[nt][b][1][e + 2] * s2);
  };
  auto end_segment = [&](int u0, int u1, bool last) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 4; i < 32; i <<= 1) l[nt][e] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][e], i);
    if (u0 == 0 && u1 == cunits) {
      const int q0 = info[cb].q0, qn = info[cb].qn;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = (rg * NT + nt) * 8 + 2 * c + e, j = (int)((uint32_t)row * g.group_inv >> 16);
          if (j >= qn) continue;
          const int64_t at = (int64_t)(q0 + j) * g.q_heads + ch * g.group + row - j * g.group;
#pragma unroll
          for (int b = 0; b < NB; ++b) write_row4<D>(g, at, 32 * b + 4 * r, value4(nt, e, b), m[nt][e], l[nt][e]);
        }
      return;
    }
    // a part of the pair: in this warp's ring if the warp is done, else in the workspace
    float* p = last ? reinterpret_cast<float*>(ring) : g.warp_parts + ((size_t)blockIdx.x * NW + warp) * PART;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = nt * 8 + 2 * c + e;
#pragma unroll
        for (int b = 0; b < NB; ++b) *reinterpret_cast<float4*>(p + row * D + 32 * b + 4 * r) = value4(nt, e, b);
        if (r == 0) {
          const int at = (2 * stream + (last ? 1 : 0)) * (RG * ROWS) + rg * ROWS + row;
          s_m[at] = m[nt][e];
          s_l[at] = l[nt][e];
        }
      }
    if (rg == 0 && lane == 0) s_entry[2 * stream + (last ? 1 : 0)] = Entry{u0, u1, cb, ch};
  };

  int stage = 0, phase = 0, seg_u0 = 0;
  bool fresh = true;
  for (int i = 0; i < todo; ++i) {
    if (fresh) {
      if (i > 0) load_q();
      begin_segment();
      seg_u0 = cu;
    }
    const bool ok = mbar_wait(bar + stage, phase, kDefaultWaitNs);
    if (!__all_sync(0xFFFFFFFFu, ok)) {
      // give up: record it, wait (again with a limit) for the copies that are under way, leave no part
      if (lane == 0) record_error(a.status, MOE_ERR_DEVICE_TIMEOUT);
      for (int k = i; k < issued; ++k) {
        mbar_wait(bar + stage, phase, kDefaultWaitNs);
        if (++stage == stages) { stage = 0; phase ^= 1; }
      }
      break;
    }
    const uint8_t* unit = ring + stage * UNIT;
    if (fresh) first_window(unit);
    fresh = false;
#pragma unroll 1
    for (int k = 0; k < kUnitSubs; k += SUBS)
      if (key0 + 16 * k < seg_len) process(unit + k * S::BYTES, key0 + 16 * k);
    key0 += 16 * kUnitSubs;
    __syncwarp();
    issue();
    if (++stage == stages) { stage = 0; phase ^= 1; }
    const bool done = ++cu == cunits, last = i + 1 == todo;
    if (done || last) {
      end_segment(seg_u0, cu, last);
      if (done && !last) {
        next_pair(cb, ch, cu, cunits);
        fresh = true;
      }
    }
  }
  __syncthreads();

  // ---- join the CTA's parts: entries in the order of the units, runs of one pair
  const int rows_all = RG * ROWS, row_bits = 31 - __clz(rows_all);   // (a power of two)
  auto token_of = [&](int row) { return (int)((uint32_t)row * g.group_inv >> 16); };
  if (warp == 0) {
    Entry en{0, 0, -1, 0};
    if (lane < 2 * KS) en = s_entry[lane];
    const uint32_t valid = __ballot_sync(0xFFFFFFFFu, en.b >= 0), below = (1u << lane) - 1u;
    const int before = valid & below ? 31 - __clz(valid & below) : 0;
    const int pb = __shfl_sync(0xFFFFFFFFu, en.b, before), ph = __shfl_sync(0xFFFFFFFFu, en.h, before);
    const bool lead = en.b >= 0 && (!(valid & below) || pb != en.b || ph != en.h);
    const uint32_t leads = __ballot_sync(0xFFFFFFFFu, lead), later = leads & ~below & ~(1u << lane);
    const uint32_t mine = valid & ~below & (later ? (1u << (__ffs(later) - 1)) - 1u : 0xFFFFFFFFu);
    const int u1 = __shfl_sync(0xFFFFFFFFu, en.u1, mine ? 31 - __clz(mine) : 0), place = __popc(valid & below);
    if (lane == 0) {
      s_runs = __popc(leads);
      s_last[0] = s_last[1] = -1;
    }
    if (en.b >= 0) {
      const int w = (lane >> 1) * RG;
      s_place[place] = lane & 1 ? Place{reinterpret_cast<const float*>(smem + (size_t)w * stages * UNIT), stages * UNIT / 4, lane}
                                : Place{g.warp_parts + ((size_t)blockIdx.x * NW + w) * PART, PART, lane};
    }
    if (lead)
      s_run[__popc(leads & below)] =
          Run{en.u0, u1, en.b, en.h, place, __popc(mine), en.u0 == 0 ? 1 : 0, en.u0 == 0 && u1 == seq_units(info[en.b]) ? 1 : 0};
  }
  __syncthreads();
  const int runs = s_runs;
  // each entry's weight 2^(m_e - m) per row, and each run's m and l (over its first entry's)
  for (int t = tid; t < runs << row_bits; t += THREADS) {
    const int row = t & (rows_all - 1), first = s_run[t >> row_bits].first, n = s_run[t >> row_bits].n;
    float mx = -FLT_MAX, sum = 0.f;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float x = s_m[s_place[first + i].at * rows_all + row];
      mx = x > mx || x != x ? x : mx;
    }
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const int at = s_place[first + i].at * rows_all + row;
      const float w = ex2(s_m[at] - mx);
      sum += w * s_l[at];
      s_wt[(first + i) * rows_all + row] = w;
    }
    const int at = s_place[first].at * rows_all + row;
    s_m[at] = mx;
    s_l[at] = sum;
  }
  __syncthreads();
  const size_t cta_part = (size_t)rows_all * (D + 2);
  for (int t = tid; t < (runs << row_bits) * (D / 4); t += THREADS) {
    const int d = t % (D / 4) * 4, row = t / (D / 4) & (rows_all - 1);
    const Run ru = s_run[t / (D / 4) >> row_bits];
    const int j = token_of(row), w_rg = row / ROWS, at = (row % ROWS) * D + d;
    if (j >= info[ru.b].qn) continue;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = 0; i < ru.n; ++i) {
      const Place pl = s_place[ru.first + i];
      const float4 v = *reinterpret_cast<const float4*>(pl.p + w_rg * pl.step + at);
      const float wt = s_wt[(ru.first + i) * rows_all + row];
      acc.x = fmaf(wt, v.x, acc.x); acc.y = fmaf(wt, v.y, acc.y); acc.z = fmaf(wt, v.z, acc.z); acc.w = fmaf(wt, v.w, acc.w);
    }
    const int ml = s_place[ru.first].at * rows_all + row;
    if (ru.whole) {
      write_row4<D>(g, (int64_t)(info[ru.b].q0 + j) * g.q_heads + ru.h * g.group + row - j * g.group, d, acc, s_m[ml], s_l[ml]);
    } else {
      float* p = g.cta_parts + ((size_t)blockIdx.x * 2 + ru.slot) * cta_part;
      *reinterpret_cast<float4*>(p + row * D + d) = acc;
      if (d == 0) {
        p[rows_all * D + row] = s_m[ml];
        p[rows_all * D + rows_all + row] = s_l[ml];
      }
    }
  }
  __syncthreads();
  // ---- a pair that spans CTAs: count its units; the CTA that completes the count joins the parts
  if (tid < runs) {
    const Run ru = s_run[tid];
    if (!ru.whole) {
      uint32_t* cnt = g.counters + first_cta(prefix[ru.b] + (long long)ru.h * (seq_units(info[ru.b]) + kPairCost) + kPairCost, W, G);
      const uint32_t n = (uint32_t)(ru.u1 - ru.u0);
      if (atom_acq_rel_add(cnt, n) + n == (uint32_t)seq_units(info[ru.b])) {
        *cnt = 0;
        s_last[ru.slot] = tid;
      }
    }
  }
  __syncthreads();
  for (int k = 0; k < 2; ++k) {
    if (s_last[k] < 0) continue;
    const Run ru = s_run[s_last[k]];
    const SeqInfo sj = info[ru.b];
    const int units = seq_units(sj);
    // the CTAs that hold the pair's first and last unit; CTA i's run begins at i W / G
    const long long p0 = prefix[ru.b] + (long long)ru.h * (units + kPairCost) + kPairCost;
    const int c0 = first_cta(p0, W, G), n = (int)(((p0 + units) * G - 1) / W) - c0 + 1;
    // parts in batches: a batch's loads are all in flight, then the sums move to its maximum
    for (int t = tid; t < rows_all * (D / 4); t += THREADS) {
      const int d = t % (D / 4) * 4, row = t / (D / 4), j = token_of(row);
      if (j >= sj.qn) continue;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float mx = -FLT_MAX, sum = 0.f;
      constexpr int BATCH = 4;
      for (int i0 = 0; i0 < n; i0 += BATCH) {
        float4 v[BATCH];
        float pm[BATCH], pl[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          // (the pair's first CTA holds its part as one that begins there, the others as one that goes on)
          const float* p = g.cta_parts + ((size_t)(c0 + i0 + i) * 2 + (i0 + i == 0 ? 1 : 0)) * cta_part;
          const bool in = i0 + i < n;
          v[i] = in ? __ldcg(reinterpret_cast<const float4*>(p + row * D + d)) : make_float4(0.f, 0.f, 0.f, 0.f);
          pm[i] = in ? __ldcg(p + rows_all * D + row) : -FLT_MAX;
          pl[i] = in ? __ldcg(p + rows_all * D + rows_all + row) : 0.f;
        }
        float m_new = mx;
#pragma unroll
        for (int i = 0; i < BATCH; ++i) m_new = pm[i] > m_new || pm[i] != pm[i] ? pm[i] : m_new;
        const float al = ex2(mx - m_new);
        mx = m_new;
        sum *= al;
        acc.x *= al; acc.y *= al; acc.z *= al; acc.w *= al;
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          const float wt = ex2(pm[i] - mx);
          sum = fmaf(wt, pl[i], sum);
          acc.x = fmaf(wt, v[i].x, acc.x); acc.y = fmaf(wt, v[i].y, acc.y);
          acc.z = fmaf(wt, v[i].z, acc.z); acc.w = fmaf(wt, v[i].w, acc.w);
        }
      }
      write_row4<D>(g, (int64_t)(sj.q0 + j) * g.q_heads + ru.h * g.group + row - j * g.group, d, acc, mx, sum);
    }
  }
}

// Rows a warp holds and warps per CTA. 8 rows: 12 warps of up to 168 registers. More: 16 rows in 8 warps of up to 255
// registers, as many warps on the same units as it takes.
struct Shape { int nt, warps, row_groups; };
static Shape shape_for(int rows) {
  if (rows <= 8) return {1, 12, 1};
  int rg = 1;
  while (rg * 16 < rows) rg *= 2;
  return {2, 8, rg};
}

static size_t meta_bytes(int n_seqs, int warps, int stages) {
  return (size_t)warps * stages * 8 + (size_t)(n_seqs + 2) * 8 + (size_t)n_seqs * sizeof(SeqInfo) +
         warps * sizeof(Prod);
}

template <int FMT, int D, int NT, int NW, int SUBS>
static moe_status_t launch(const Args& a, AttnArgs g, int ctas, cudaStream_t stream) {
  constexpr size_t unit = kUnitSubs * Sub<FMT, D>::BYTES, most = kSmemMax - 6144;   // (the kernel's fixed tables take the rest)
  int stages = 6;
  while (stages > 1 && NW * stages * unit + meta_bytes(a.n_seqs, NW, stages) > most) --stages;
  g.stages = stages;
  g.rings = (int32_t)(NW * stages * unit);
  const size_t smem = g.rings + meta_bytes(a.n_seqs, NW, stages);
  static int configured[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MOE_ERR_CUDA;
  if (!configured[dev]) {
    if (cudaFuncSetAttribute(attn_kernel<FMT, D, NT, NW, SUBS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most) !=
        cudaSuccess)
      return MOE_ERR_CUDA;
    configured[dev] = 1;
  }
  attn_kernel<FMT, D, NT, NW, SUBS><<<ctas, NW * 32, smem, stream>>>(a, g);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace kv
}  // namespace moe

using namespace moe;

static size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

// What a call leaves at zero (counters, marks) lies at the same place for every batch, so that batches of different sizes can
// share a workspace.
static const size_t kZeroBytes = up256((kv::kMaxCtas + kv::kMaxSeqs + 2) * 4);

extern "C" size_t moe_kv_workspace_bytes(const moe_kv_cache_t* cache, const moe_kv_batch_t* batch, int32_t q_heads) {
  if (kv::check_cache(cache) != MOE_OK || kv::check_sizes(batch) != MOE_OK) return 0;
  if (q_heads < 1 || q_heads > 4096 || q_heads % cache->kv_heads) return 0;
  // attention's part is for the most new tokens that it takes, so that a workspace for longer prompts serves decoding too
  const int group = q_heads / cache->kv_heads;
  if (group > kv::kMaxRows) return sizeof(WsHeader);   // append and read only
  const kv::Shape s = kv::shape_for(group * std::min(batch->max_q, std::min(8, kv::kMaxRows / group)));
  const size_t row_bytes = (size_t)(cache->head_dim + 2) * 4;
  return sizeof(WsHeader) + kZeroBytes + up256(kv::kMaxCtas * s.warps * 8 * s.nt * row_bytes) + up256(kv::kMaxCtas * 2 * s.row_groups * 8 * s.nt * row_bytes);
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
  // A sequence has fewer than 2^30 keys, so a window of that many hides none. Smaller ones keep the kernels' 32-bit differences
  // of positions and windows in range.
  if (window >= 1 << 30) window = 0;
  // units of 32 keys in all: a warp counts its share in 32 bits
  if ((int64_t)batch->n_seqs * cache->kv_heads * ((int64_t)batch->table_stride * cache->page_tokens / 32 + 1) >= (int64_t)1 << 37)
    return MOE_ERR_SHAPE;
  const size_t need = moe_kv_workspace_bytes(cache, batch, q_heads);
  if (need == 0 || ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if ((st = moe_check_device()) != MOE_OK) return st;
  a.status = &((WsHeader*)ws)->status;
  const int group = q_heads / cache->kv_heads, rows = batch->max_q * group;
  const kv::Shape s = kv::shape_for(rows);
  uint8_t* w = (uint8_t*)ws + sizeof(WsHeader);
  kv::AttnArgs g{(const uint16_t*)q, q_stride, q_heads, group, window, s.row_groups, 0, 65535u / (uint32_t)group + 1u, 0, scale * 1.4426950408889634f,
                 (uint16_t*)out, lse, (uint32_t*)w, nullptr, nullptr, nullptr};
  g.redo = g.counters + kv::kMaxCtas;
  w += kZeroBytes;
  g.warp_parts = (float*)w;
  w += up256(kv::kMaxCtas * s.warps * 8 * s.nt * (size_t)(cache->head_dim + 2) * 4);
  g.cta_parts = (float*)w;
  const int ctas = moe_internal::num_sms() < kv::kMaxCtas ? moe_internal::num_sms() : kv::kMaxCtas;
  if (ctas < 1) return MOE_ERR_CUDA;
  // Above 16 rows a KV head, and where the table and the window leave room for long sequences, kv_attn_wide.cu goes first; its
  // cost does not grow with the rows up to 64, but a pair's start costs it 3 tiles of 128 keys, this kernel none.
  // Measured, this kernel / that: 24 rows over 300 keys (256 sequences) 33 / 60 us; 18 rows over a window of 1024 (33)
  // 54 / 49 us, 32 rows over 16384 keys (16) 181 / 141 us; 64 rows over 600 (16) 41 / 32 us, over 100000 (1) 197 / 97 us;
  // 16 rows over 8192 (64, 8 KV heads) 124 / 178 us.
  int64_t keys = (int64_t)batch->table_stride * cache->page_tokens;
  if (window) keys = std::min(keys, (int64_t)window + batch->max_q);
  if (rows <= 16 || keys * s.row_groups < 2048) g.redo = nullptr;
  if (g.redo && (st = kv::attn_wide(a, g, cache->fmt, cache->head_dim, ctas, (cudaStream_t)stream)) != MOE_OK) return st;
#define KV_CALL(F, DD)                                                                   \
  return s.nt == 1 ? kv::launch<F, DD, 1, 12, 2>(a, g, ctas, (cudaStream_t)stream)        \
                   : kv::launch<F, DD, 2, 8, 1>(a, g, ctas, (cudaStream_t)stream)
  KV_DISPATCH(KV_CALL);
#undef KV_CALL
}
