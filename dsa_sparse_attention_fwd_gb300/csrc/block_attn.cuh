// Attention over selected blocks of keys: the problem as the kernels of
// block_attn.cu, block_attn_bwd.cu and block_attn_row.cuh see it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace dsa {

struct BlockAttn {
  const __nv_bfloat16 *q;       // [S, B, H, D]
  const __nv_bfloat16 *k, *v;   // keys and values, or their paged caches
  long long k_st, k_sb, k_sh;   // element strides: token, sequence (paged:
  long long v_st, v_sb, v_sh;   // page), head
  const int32_t *blocks;        // [B, S, sel_heads, topk]
  const int32_t *q_pos;         // [B] or nullptr
  const int32_t *table;         // paged: [B, max_pages], else nullptr
  int max_pages, page_size, num_pages;
  int S, B, H, Hk, G, D, T;     // G = H / Hk heads share a key head
  int sel_heads, topk, blk, local, nblk;
  float scale;
  int *status;
};

// Ids of a row: its topk given ones, then its local ones.  Returns the block
// of candidate i, or -1 where it holds none: empty, out of range (`bad`), a
// block after the row's position, or one of the local blocks given again.
__device__ __forceinline__ int candidate(const BlockAttn &p,
                                         const int32_t *ids, long long pos,
                                         int i, bool &bad) {
  if (pos < 0) return -1;
  const long long own = pos / p.blk;
  if (i < p.topk) {
    const int n = __ldg(ids + i);
    if (n < -1 || n >= p.nblk) bad = true;
    return n < 0 || n >= p.nblk || n > own - p.local ? -1 : n;
  }
  const long long n = own - (i - p.topk);
  return n >= 0 && n < p.nblk ? (int)n : -1;
}

__device__ __forceinline__ const int32_t *row_ids(const BlockAttn &p, int b,
                                                  int s, int hk) {
  return p.blocks +
         (((size_t)b * p.S + s) * p.sel_heads + (p.sel_heads > 1 ? hk : 0)) *
             p.topk;
}

// Page of block n of sequence b (blocks lie within pages), or -1 where the
// table names none (`bad`).
__device__ __forceinline__ int block_page(const BlockAttn &p, int b, int n,
                                          bool &bad) {
  const int pg = (int)((long long)n * p.blk / p.page_size);
  const int page = __ldg(p.table + (long long)b * p.max_pages + pg);
  if (page >= 0 && page < p.num_pages) return page;
  bad = true;
  return -1;
}

}  // namespace dsa
