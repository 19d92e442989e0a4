// kv.cuh -- the 4-bit paged KV cache: sub-block geometry, host-side argument checks and device-side lookups shared by
// kv_append.cu and kv_attn.cu. The layout is defined in include/moe.h; why it looks like that is in kv_attn.cu.
#pragma once
#include "common.cuh"
#include "api_internal.h"
#include "tcgen05.cuh"

namespace moe {
namespace kv {

constexpr int kMaxSeqs = 1024;
constexpr int kMaxRows = 128;    // query rows of one KV head in one attention call: max_q * (q_heads / kv_heads)
constexpr int kMaxCtas = 160;    // CTAs an attention launch uses at most (one per SM; a GB300 has 152)

// 16 tokens of one KV head
template <int FMT, int D>
struct Sub {
  static constexpr int NB = D / 32;                               // blocks of 32 values per row
  static constexpr int SB = FMT == MOE_FMT_MXFP4 ? 1 : 2;         // bytes per scale
  static constexpr int KC = 0, VC = 8 * D;                        // byte offsets of the four parts
  static constexpr int KS = 16 * D, VS = 16 * D + 16 * NB * SB;
  static constexpr int BYTES = 16 * D + 32 * NB * SB;
  static_assert(BYTES % 16 == 0, "sub-blocks are moved by 16-byte granular bulk copies");
};

__host__ __device__ inline int sub_bytes(int fmt, int D) { return 16 * D + D * (fmt == MOE_FMT_MXFP4 ? 1 : 2); }

struct Args {   // the cache and the batch as the kernels take them
  uint8_t* pages;
  int64_t page_stride, n_pages;
  const int32_t* q_start;
  const int32_t* seq_len;
  const int32_t* block_table;
  int32_t n_seqs, n_tokens, max_q, table_stride, kv_heads, page_tokens;
  int32_t* status;
};

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

inline moe_status_t check_cache(const moe_kv_cache_t* c) {
  if (!c) return MOE_ERR_INVALID_ARG;
  if (c->fmt != MOE_FMT_MXFP4 && c->fmt != MOE_FMT_INT4G32) return MOE_ERR_UNSUPPORTED_FORMAT;
  if (c->head_dim != 64 && c->head_dim != 128) return MOE_ERR_SHAPE;
  if (c->kv_heads < 1 || c->kv_heads > 256 || c->page_tokens < 16 || c->page_tokens > 1024 || c->page_tokens % 16)
    return MOE_ERR_SHAPE;
  return MOE_OK;
}

inline moe_status_t check_sizes(const moe_kv_batch_t* b) {
  if (!b) return MOE_ERR_INVALID_ARG;
  if (b->n_seqs < 1 || b->n_seqs > kMaxSeqs || b->n_tokens < 1 || b->max_q < 1 || b->table_stride < 1)
    return MOE_ERR_SHAPE;
  return MOE_OK;
}

// everything but the workspace; fills `a`
inline moe_status_t check(const moe_kv_cache_t* c, const moe_kv_batch_t* b, Args* a) {
  moe_status_t st = check_cache(c);
  if (st != MOE_OK) return st;
  if ((st = check_sizes(b)) != MOE_OK) return st;
  if (!c->pages || !aligned(c->pages, 16) || !b->q_start || !b->seq_len || !b->block_table || !aligned(b->q_start, 4) ||
      !aligned(b->seq_len, 4) || !aligned(b->block_table, 4))
    return MOE_ERR_INVALID_ARG;
  if (c->n_pages < 1 || c->page_stride % 16 ||
      c->page_stride < (int64_t)moe_kv_page_bytes(c->fmt, c->head_dim, c->kv_heads, c->page_tokens))
    return MOE_ERR_SHAPE;
  if ((int64_t)b->table_stride * c->page_tokens >= (1 << 30)) return MOE_ERR_SHAPE;
  *a = Args{(uint8_t*)c->pages, c->page_stride, c->n_pages, b->q_start, b->seq_len, b->block_table, b->n_seqs,
            b->n_tokens, b->max_q, b->table_stride, c->kv_heads, c->page_tokens, nullptr};
  return MOE_OK;
}

// One sequence's rows and length; anything out of range makes it empty and is recorded.
struct Seq { int q0, qn, len; };
__device__ __forceinline__ Seq check_seq(const Args& a, int q0, int q1, int len, int max_q) {
  if (q0 < 0 || q1 < q0 || q1 > a.n_tokens) {              // its rows are not in the call's tensors
    record_error(a.status, MOE_ERR_INVALID_ARG);
    return Seq{0, 0, 0};
  }
  if (q1 - q0 > max_q || len < 0 || len > a.table_stride * a.page_tokens) {
    record_error(a.status, MOE_ERR_INVALID_ARG);
    len = 0;
  }
  return Seq{q0, q1 - q0, len};
}

// A page id from the table; an id outside the pool is recorded and reads as page 0 (`ok` tells a writer).
__device__ __forceinline__ int check_page(const Args& a, int id, bool& ok) {
  ok = id >= 0 && id < a.n_pages;
  if (!ok) record_error(a.status, MOE_ERR_INVALID_ARG);
  return ok ? id : 0;
}

// a block's scale
template <int FMT>
__device__ __forceinline__ float load_scale(const uint8_t* p) {
  if (FMT == MOE_FMT_MXFP4) return __uint_as_float((uint32_t)*p << 23);   // 2^(e - 127); e = 0 is zero
  return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(p) << 16);
}

}  // namespace kv
}  // namespace moe

// CALL(format, head dimension) for the cache's
#define KV_DISPATCH(CALL)                                                                  \
  do {                                                                                     \
    if (cache->fmt == MOE_FMT_MXFP4) {                                                     \
      if (cache->head_dim == 64) { CALL(MOE_FMT_MXFP4, 64); } else { CALL(MOE_FMT_MXFP4, 128); }     \
    } else {                                                                               \
      if (cache->head_dim == 64) { CALL(MOE_FMT_INT4G32, 64); } else { CALL(MOE_FMT_INT4G32, 128); } \
    }                                                                                      \
  } while (0)
