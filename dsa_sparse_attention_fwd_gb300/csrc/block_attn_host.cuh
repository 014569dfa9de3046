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

}  // namespace dsa
