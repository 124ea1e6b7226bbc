// paged_batch.hpp -- sequences over a paged cache, as the attention operators
// share them: which rows are whose, where an index of a cache lies, and the
// host's checks of the description.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "status.hpp"

namespace fluxbin {

// fluxbin_paged_batch as the kernels take it.
struct Paged {
  const int32_t *seq_starts, *kv_lens, *page_table;  // seq_starts may be null: row s is sequence s
  uint16_t *k, *v;
  int64_t table_ld, page_stride, head_stride;
  int32_t tokens, seqs, pages, table_pages, token_stride;
  int32_t heads, kv_heads, dim, page_shift;
};

// A sequence: its number (seqs: none), its first row and the next sequence's, as
// they are given, and the length of its cache.
struct Found {
  int seq, start, next, len;
};

// The number of j in [1, seqs] for which within(seq_starts[j], j) holds, which is
// true up to some j, as a sequence.  Up to 63 sequences are looked at in one round
// of loads, a lane to each; of more, 64 places at a time (4096 take two rounds).
template <typename F>
__device__ __forceinline__ Found find_sequence(const Paged &b, int lane, F within) {
  Found f;
  if (b.seqs < 64) {
    const int start = b.seq_starts ? b.seq_starts[min(lane, b.seqs)] : lane, len = b.kv_lens[min(lane, b.seqs - 1)];
    f.seq = __popcll(__ballot(lane >= 1 && lane <= b.seqs && within(start, lane)));
    const int at = min(f.seq, b.seqs - 1);
    f.start = __builtin_amdgcn_readlane(start, at);
    f.next = __builtin_amdgcn_readlane(start, at + 1);
    f.len = __builtin_amdgcn_readlane(len, at);
    return f;
  }
  int lo = 0, n = b.seqs;
  while (n > 0) {
    const int step = (n + 63) / 64, j = (lane + 1) * step;
    const int c = __popcll(__ballot(j <= n && within(b.seq_starts ? b.seq_starts[lo + j] : lo + j, lo + j)));
    lo += c * step;
    n = min(step - 1, n - c * step);
  }
  f.seq = lo;
  const int at = min(lo, b.seqs - 1);
  f.start = b.seq_starts ? b.seq_starts[at] : at;
  f.next = b.seq_starts ? b.seq_starts[at + 1] : at + 1;
  f.len = b.kv_lens[at];
  return f;
}

// The page that holds `index` (>= 0) of sequence s, or -1 where there is none.
__device__ __forceinline__ int page_of(const Paged &b, int s, int index) {
  const int i = index >> b.page_shift;
  if (i >= b.table_pages) return -1;
  const int p = b.page_table[(int64_t)s * b.table_ld + i];
  return (uint32_t)p < (uint32_t)b.pages ? p : -1;
}

// Keys of a sequence: the kernels look up to a few hundred beyond the last one, in 32 bits.
constexpr int64_t kMostKeys = ((int64_t)1 << 31) - (1 << 16);

inline fluxbin_status check_paged(const fluxbin_paged_batch *b) {
  if (!b) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "batch is NULL");
  if (b->abi_version != FLUXBIN_ABI_VERSION)
    return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "batch abi_version %d != %d", b->abi_version, FLUXBIN_ABI_VERSION);
  if (b->dtype != FLUXBIN_DT_F16 && b->dtype != FLUXBIN_DT_BF16)
    return fail(FLUXBIN_ERR_UNSUPPORTED, "dtype = %d (fp16 or bf16)", b->dtype);
  if (b->heads < 1 || b->kv_heads < 1 || b->heads % b->kv_heads)
    return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "heads = %d is no multiple of kv_heads = %d", b->heads, b->kv_heads);
  if (b->heads > 1024) return fail(FLUXBIN_ERR_UNSUPPORTED, "heads = %d (at most 1024)", b->heads);
  if (b->dim < 8 || b->dim % 8 || b->dim > 256)
    return fail(FLUXBIN_ERR_UNSUPPORTED, "dim = %d (a multiple of 8, 8 .. 256)", b->dim);
  if (b->page_size < 16 || b->page_size > 65536 || (b->page_size & (b->page_size - 1)))
    return fail(FLUXBIN_ERR_UNSUPPORTED, "page_size = %d (a power of two, 16 .. 65536)", b->page_size);
  if (b->tokens < 0 || b->seqs < 0)
    return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "tokens = %lld, seqs = %lld", (long long)b->tokens, (long long)b->seqs);
  if (b->tokens > 1 << 24 || b->seqs > 1 << 24 || b->tokens * b->heads > 1 << 30)
    return fail(FLUXBIN_ERR_UNSUPPORTED, "tokens or seqs above 2^24, or tokens * heads above 2^30");
  if (!b->seq_starts && b->tokens != b->seqs)
    return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "tokens = %lld rows of seqs = %lld sequences without seq_starts",
                (long long)b->tokens, (long long)b->seqs);
  if (b->max_kv_len < 0) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "max_kv_len = %lld", (long long)b->max_kv_len);
  if (b->table_pages < 0 || b->table_ld < b->table_pages)
    return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "table_pages = %lld, table_ld = %lld", (long long)b->table_pages, (long long)b->table_ld);
  if (b->table_pages > kMostKeys / b->page_size)
    return fail(FLUXBIN_ERR_UNSUPPORTED, "table_pages * page_size above 2^31 - 2^16");
  if (b->cache_pages < 0) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "cache_pages = %lld", (long long)b->cache_pages);
  if (b->cache_pages >= (int64_t)1 << 31) return fail(FLUXBIN_ERR_UNSUPPORTED, "cache_pages reaches 2^31");
  if (b->page_stride < 0 || b->head_stride < 0 || b->page_stride % 8 || b->head_stride % 8 || b->token_stride % 8)
    return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "the cache's strides are not multiples of 8 elements");
  if (b->token_stride < b->dim)
    return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "token_stride = %lld < dim = %d", (long long)b->token_stride, b->dim);
  if (b->token_stride > 1 << 24) return fail(FLUXBIN_ERR_UNSUPPORTED, "token_stride above 2^24");
  if (b->tokens == 0 || b->seqs == 0) return FLUXBIN_OK;
  if (!b->kv_lens || !b->page_table || !b->k_cache || !b->v_cache)
    return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "kv_lens, page_table, k_cache or v_cache is NULL");
  if (!aligned(b->kv_lens, 4) || !aligned(b->page_table, 4) || !aligned(b->seq_starts, 4))
    return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "seq_starts, kv_lens or page_table is not aligned to its elements");
  if (!aligned(b->k_cache, 16) || !aligned(b->v_cache, 16))
    return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "k_cache or v_cache is not 16-byte aligned");
  return FLUXBIN_OK;
}

// Rows of `width` elements of 16 bits, `ld` apart.
inline fluxbin_status check_rows(const char *name, const void *p, int64_t ld, int64_t width) {
  if (!p) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "%s is NULL", name);
  if (!aligned(p, 2)) return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "%s is not aligned to its elements", name);
  if (ld < width)
    return fail(FLUXBIN_ERR_INVALID_ARGUMENT, "the row stride of %s, %lld, is below %lld", name, (long long)ld, (long long)width);
  return FLUXBIN_OK;
}

inline Paged paged_of(const fluxbin_paged_batch &b) {
  Paged p{};
  p.seq_starts = b.seq_starts;
  p.kv_lens = b.kv_lens;
  p.page_table = b.page_table;
  p.k = (uint16_t *)b.k_cache;
  p.v = (uint16_t *)b.v_cache;
  p.table_ld = b.table_ld;
  p.page_stride = b.page_stride;
  p.head_stride = b.head_stride;
  p.tokens = (int32_t)b.tokens;
  p.seqs = (int32_t)b.seqs;
  p.pages = (int32_t)b.cache_pages;
  p.table_pages = (int32_t)b.table_pages;
  p.token_stride = (int32_t)b.token_stride;
  p.heads = b.heads;
  p.kv_heads = b.kv_heads;
  p.dim = b.dim;
  p.page_shift = __builtin_ctz((unsigned)b.page_size);
  return p;
}

}  // namespace fluxbin
