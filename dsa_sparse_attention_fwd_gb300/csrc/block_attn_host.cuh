// Host side shared by the block attention's forward and backward.
#pragma once

#include "block_attn.cuh"
#include "dsa_indexer.h"

namespace dsa {

inline bool aligned_to(const void *p, unsigned n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

int check_block_attn(BlockAttn &p);

// strides: (k token, k sequence or page, k head, v ...) in elements, or
// nullptr for the dense layout with token stride st and sequence stride sb.
void set_kv(BlockAttn &p, const void *k, const void *v,
            const int64_t *strides, long long st, long long sb);

// TMA maps of keys and values with boxes of `rows` tokens.
inline int encode_kv_maps(const BlockAttn &p, int rows, KvMaps *m) {
  const long long toks = p.table ? p.page_size : p.T;
  const long long outer = p.table ? p.num_pages : p.B;
  m->bc_ks = p.k_sb != 0, m->bc_kh = p.k_sh != 0;
  m->bc_vs = p.v_sb != 0, m->bc_vh = p.v_sh != 0;
  int rc = encode_kv(&m->k, p.k, p.D, rows, toks, p.k_st,
                     m->bc_kh ? p.Hk : 1, p.k_sh, m->bc_ks ? outer : 1,
                     p.k_sb);
  if (rc != DSA_OK) return rc;
  return encode_kv(&m->v, p.v, p.D, rows, toks, p.v_st, m->bc_vh ? p.Hk : 1,
                   p.v_sh, m->bc_vs ? outer : 1, p.v_sb);
}

}  // namespace dsa
