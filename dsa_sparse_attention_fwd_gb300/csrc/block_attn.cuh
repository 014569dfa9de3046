// Attention over selected blocks of keys: the problem as the kernels of
// block_attn.cu, block_attn_bwd.cu and block_attn_row.cuh see it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "ptx.cuh"

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
  int lb;  // log2 of blk
  float scale;
  int *status;
};

// Ids of a row: its topk given ones, then its local ones.  Returns the block
// of candidate i, or -1 where it holds none: empty, out of range (`bad`), a
// block after the row's position, or one of the local blocks given again.
__device__ __forceinline__ int candidate(const BlockAttn &p,
                                         const int32_t *ids, long long pos,
                                         int i, bool &bad) {
  if (i < p.topk) {
    const int n = __ldg(ids + i);  // (does not wait for the position)
    if (n < -1 || n >= p.nblk) bad = true;
    if (pos < 0) return -1;
    return n < 0 || n >= p.nblk || n > (pos >> p.lb) - p.local ? -1 : n;
  }
  if (pos < 0) return -1;
  const long long n = (pos >> p.lb) - (i - p.topk);
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

// Query tiles: `qt` consecutive queries of one sequence with the G heads of
// one key head are qt * G <= `rows` MMA rows (row = query * G + head); at
// most 32 queries, one bit each in a block's mask.
__host__ __device__ __forceinline__ int tile_queries(int G, int rows) {
  const int n = rows / G;
  return n > 32 ? 32 : n;
}

// The blocks that the queries s0 .. s0 + nq - 1 of sequence b attend to
// under key head hk: words[n] gets bit i where query s0 + i holds block n.
// Every thread of the CTA takes part.  The first call looks up the thread's
// first candidate (three loads in a row, that need no shared memory yet), the
// second, after the words have been cleared, marks it and the others.
struct FirstMark {
  int n, i;  // block (-1: none), query
  bool bad;
};
__device__ __forceinline__ int mark_at(const BlockAttn &p, int b, int s0,
                                       int hk, long long pos0, int i, int c,
                                       bool &bad) {
  int n = candidate(p, row_ids(p, b, s0 + i, hk), pos0 + i, c, bad);
  if (n >= 0 && p.table && block_page(p, b, n, bad) < 0) n = -1;
  return n;
}
__device__ __forceinline__ FirstMark first_mark(const BlockAttn &p, int b,
                                                int s0, int nq, int hk,
                                                int tid) {
  const int n_cand = p.topk + p.local;
  FirstMark f{-1, tid / n_cand, false};
  if (tid < nq * n_cand)
    f.n = mark_at(p, b, s0, hk, row_pos(p.q_pos, b, s0), f.i,
                  tid - f.i * n_cand, f.bad);
  return f;
}
__device__ __forceinline__ void mark_blocks(const BlockAttn &p, int b, int s0,
                                            int nq, int hk, uint32_t *words,
                                            int tid, int nthreads,
                                            FirstMark f) {
  constexpr int U = 4;  // candidates of a thread on the way together
  const int n_cand = p.topk + p.local, all = nq * n_cand;
  if (f.n >= 0) atomicOr(words + f.n, 1u << f.i);
  if (all > nthreads) {
    const long long pos0 = row_pos(p.q_pos, b, s0);
    for (int x0 = tid + nthreads; x0 < all; x0 += U * nthreads) {
      int n[U], i[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int x = x0 + u * nthreads;
        i[u] = x / n_cand;
        n[u] = x < all ? candidate(p, row_ids(p, b, s0 + i[u], hk),
                                   pos0 + i[u], x - i[u] * n_cand, f.bad)
                       : -1;
      }
      if (p.table) {
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (n[u] >= 0 && block_page(p, b, n[u], f.bad) < 0) n[u] = -1;
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (n[u] >= 0) atomicOr(words + n[u], 1u << i[u]);
    }
  }
  if (f.bad) atomicOr(p.status, kStatusIndexRange);
}

// The marked blocks in ascending order, and their masks moved to the front of
// words in the same order; one warp.  Returns their number.
__device__ __forceinline__ int list_blocks(uint32_t *words, int nblk,
                                           uint16_t *list, int lane) {
  int count = 0;
  for (int n0 = 0; n0 < nblk; n0 += 128) {
    uint32_t w[4];
    unsigned m[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int n = n0 + u * 32 + lane;
      w[u] = n < nblk ? words[n] : 0u;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) m[u] = __ballot_sync(0xffffffffu, w[u] != 0u);
    // (an entry never moves up, and these 128 have been read)
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int at = count + __popc(m[u] & ((1u << lane) - 1));
      if (w[u]) {
        words[at] = w[u];
        list[at] = (uint16_t)(n0 + u * 32 + lane);
      }
      count += __popc(m[u]);
    }
    __syncwarp();
  }
  return count;
}

// A row's position as the masks use it: capped to the last key (T is at most
// 2^21: 16384 blocks of 128), -1 before the first.
__device__ __forceinline__ int key_pos(const BlockAttn &p, int b, int s) {
  const long long pos = row_pos(p.q_pos, b, s);
  return pos < 0 ? -1 : pos < p.T ? (int)pos : p.T - 1;
}

// The first n of `width` keys, n of any size: a mask.
__device__ __forceinline__ uint32_t first_keys(int n, int width) {
  n = n < 0 ? 0 : n;
  return n >= width ? 0xffffffffu >> (32 - width) : (1u << n) - 1u;
}

// The masks of the 64 keys of step t for the row of query bit qi at `pos`:
// its units of 16, 32 or 64 keys are list[t * 4 ..], list[t * 2 ..], list[t],
// or half of list[t / 2].  `diag`: some of the keys (each 32) come after
// pos_lo.  The masks of held blocks are made key by key only then; it runs for
// every row and step.
__device__ __forceinline__ void step_masks(const uint32_t *words,
                                           const uint16_t *list, int t,
                                           int count, int lb, int qi, int pos,
                                           int pos_lo, uint32_t (&mask)[2],
                                           bool (&diag)[2]) {
  if (lb >= 6) {
    const int i = lb == 6 ? t : t >> 1;
    const uint32_t held = words[i] >> qi & 1u;
    const int j0 = ((int)list[i] << lb) + (lb == 6 ? 0 : (t & 1) * 64);
    mask[0] = mask[1] = 0u - held;
    diag[0] = j0 + 31 > pos_lo;
    diag[1] = j0 + 63 > pos_lo;
    if (diag[1]) {
      mask[0] &= first_keys(pos - j0 + 1, 32);
      mask[1] &= first_keys(pos - j0 - 31, 32);
    }
    return;
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    mask[c] = 0u;
    int end = -1;
    if (lb == 5) {
      const int i = 2 * t + c, x = min(i, count - 1);
      const int j0 = (int)list[x] * 32;
      if (i < count) {
        end = j0 + 31;
        mask[c] = 0u - (words[x] >> qi & 1u);
        if (end > pos_lo) mask[c] &= first_keys(pos - j0 + 1, 32);
      }
    } else {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int i = 4 * t + 2 * c + u, x = min(i, count - 1);
        const int j0 = (int)list[x] * 16;
        if (i < count) {
          end = j0 + 15;  // ascending: the last one stays
          uint32_t h = 0u - (words[x] >> qi & 1u);
          if (end > pos_lo) h &= first_keys(pos - j0 + 1, 16);
          mask[c] |= (h & 0xffffu) << (16 * u);
        }
      }
    }
    diag[c] = end > pos_lo;
  }
}

// A warp's 32 rows of NW words to memory, lane = row, `dst` its address
// (nullptr: not written), through NW * 128 bytes of shared memory, so that a
// store covers whole rows: written from the lanes' own rows, the output of a
// forward tile took 6000 cycles.
template <int NW>
__device__ __forceinline__ void store_rows(uint32_t buf,
                                           const uint32_t (&w)[NW], void *dst,
                                           int lane) {
  constexpr int NC = NW / 4;  // 16-byte pieces of a row
  auto at = [&](int r, int c) {
    const int sw = NC == 8 ? r & 7 : (r >> 1) & 3;
    return buf + (uint32_t)(r * NC + (c ^ sw)) * 16;
  };
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const uint32_t v[4] = {w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]};
    st_shared_v4(at(lane, c), v);
  }
  __syncwarp();
  const unsigned long long d = reinterpret_cast<unsigned long long>(dst);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int r = (i * 32 + lane) / NC, c = lane % NC;
    const float4 v = ld_shared_v4f(at(r, c));
    const unsigned long long to = __shfl_sync(0xffffffffu, d, r);
    if (to) *reinterpret_cast<float4 *>(to + c * 16) = v;
  }
  __syncwarp();
}

// TMA coordinates of block n of sequence b, for a map made with
// encode_kv_maps(): token (or slot) and sequence (or page).  A broadcast
// sequence or head has extent 1 and coordinate 0 (bc_*).
struct KvMaps {
  CUtensorMap k, v;
  int bc_ks, bc_kh, bc_vs, bc_vh;  // 0 where broadcast, else 1
};

}  // namespace dsa
