// The paged latent cache as the kernels see it, and the argument checks its
// calls share.
#pragma once

#include <climits>

#include "moe_common.cuh"

namespace moe {

constexpr int kMaxSeqs = 8192;   // the plan kernels keep one int per sequence in 32 KB of shared memory

struct KvView {
  __nv_bfloat16* pages;
  int32_t* table;
  int32_t* lens;
  int32_t* refs;
  int n_layers, n_pages, page_tokens, rank, row, max_seqs, max_blocks;
  int page_shift;   // page_tokens = 1 << page_shift

  __device__ size_t row_offset(int layer, int page, int slot) const {
    return (((size_t)layer * n_pages + page) * page_tokens + slot) * (size_t)row;
  }
  // tokens of a sequence, never past its blocks whatever lens holds
  __device__ int len_of(int seq) const {
    const long long cap = (long long)max_blocks << page_shift;
    const int n = lens[seq];
    return n < 0 ? 0 : n > cap ? (int)cap : n;
  }
  __device__ int blocks_of(int len) const { return (int)(((long long)len + page_tokens - 1) >> page_shift); }
};

inline bool kv_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline int check_kv(const moe_kv_cache* c) {
  if (!c || !c->pages || !c->table || !c->lens || !c->refs) return MOE_ERR_INVALID_ARG;
  if (c->n_layers < 1 || c->n_pages < 1 || c->page_tokens < 1 || c->rank < 1 || c->rope < 0 || c->max_seqs < 1 ||
      c->max_blocks < 1)
    return MOE_ERR_INVALID_ARG;
  const int pt = c->page_tokens;
  if ((pt != 16 && pt != 32 && pt != 64 && pt != 128) || (c->rank % 8) || (c->rope % 8)) return MOE_ERR_UNSUPPORTED;
  if ((long long)c->rank + c->rope > (1 << 20) || c->max_seqs > kMaxSeqs) return MOE_ERR_UNSUPPORTED;
  if ((long long)c->n_layers * c->n_pages > INT_MAX / pt || (long long)c->max_seqs * c->max_blocks > INT_MAX)
    return MOE_ERR_UNSUPPORTED;
  if (!kv_aligned(c->pages, 16) || !kv_aligned(c->table, 4) || !kv_aligned(c->lens, 4) || !kv_aligned(c->refs, 4))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

inline KvView kv_view(const moe_kv_cache& c) {
  KvView v;
  v.pages = reinterpret_cast<__nv_bfloat16*>(c.pages);
  v.table = c.table;
  v.lens = c.lens;
  v.refs = c.refs;
  v.n_layers = c.n_layers;
  v.n_pages = c.n_pages;
  v.page_tokens = c.page_tokens;
  v.rank = c.rank;
  v.row = c.rank + c.rope;
  v.max_seqs = c.max_seqs;
  v.max_blocks = c.max_blocks;
  v.page_shift = c.page_tokens == 16 ? 4 : c.page_tokens == 32 ? 5 : c.page_tokens == 64 ? 6 : 7;
  return v;
}

// what the attention kernels add to check_kv
inline int check_latent(const moe_kv_cache* c, int layer) {
  const int st = check_kv(c);
  if (st != MOE_OK) return st;
  if (layer < 0 || layer >= c->n_layers) return MOE_ERR_INVALID_ARG;
  if ((c->rank % 128) || c->rank > 512 || (c->rope % 16) || c->rope > 64) return MOE_ERR_UNSUPPORTED;
  if ((long long)c->max_blocks * c->page_tokens > (1 << 27)) return MOE_ERR_UNSUPPORTED;   // tile sums of a batch are ints
  return MOE_OK;
}

inline int check_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (need && (!ws || ws_bytes < need)) return MOE_ERR_WORKSPACE;
  return need && !kv_aligned(ws, 256) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

}  // namespace moe
