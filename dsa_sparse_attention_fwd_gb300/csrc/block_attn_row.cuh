// One row of the block attention by one warp, from the formulas, in fp32 on
// the CUDA cores: x_j = scale q.k_j over the row's keys, the running maximum
// and sum of a softmax, o = sum p v.
#pragma once

#include "block_attn.cuh"

namespace dsa {

// Calls f(j, x_j, lane_has_key) for the keys of the row in groups of 32,
// lane l holding key j.
template <typename F>
__device__ __forceinline__ void row_keys(const BlockAttn &p, int b, int s,
                                         int hk, const float *qs, int lane,
                                         bool &bad, F f) {
  const long long pos = row_pos(p.q_pos, b, s);
  const int32_t *ids = row_ids(p, b, s, hk);
  const int n_cand = p.topk + p.local;
  for (int i = 0; i < n_cand; ++i) {
    int n = candidate(p, ids, pos, i, bad);
    if (n < 0) continue;
    bool again = false;  // a block given twice counts once
    for (int t = lane; t < i && i < p.topk; t += 32) again |= __ldg(ids + t) == n;
    if (__any_sync(0xffffffffu, again)) continue;
    long long k0, v0;
    if (p.table) {
      const int page = block_page(p, b, n, bad);
      if (page < 0) continue;
      const long long off = (long long)n * p.blk % p.page_size;
      k0 = page * p.k_sb + off * p.k_st;
      v0 = page * p.v_sb + off * p.v_st;
    } else {
      k0 = b * p.k_sb + (long long)n * p.blk * p.k_st;
      v0 = b * p.v_sb + (long long)n * p.blk * p.v_st;
    }
    k0 += hk * p.k_sh;
    v0 += hk * p.v_sh;
    for (int c = 0; c < p.blk; c += 32) {
      const int jj = c + lane;
      const long long j = (long long)n * p.blk + jj;
      const bool has = jj < p.blk && j <= pos && j < p.T;
      float x = 0.f;
      if (has) {
        const __nv_bfloat16 *kr = p.k + k0 + jj * p.k_st;
        for (int d = 0; d < p.D; d += 2) {
          const float2 kk = __bfloat1622float2(
              *reinterpret_cast<const __nv_bfloat162 *>(kr + d));
          x = fmaf(qs[d], kk.x, x);
          x = fmaf(qs[d + 1], kk.y, x);
        }
      }
      f((int)j, x * p.scale, has, k0 + jj * p.k_st, v0 + jj * p.v_st);
    }
  }
}

// The row's output and log-sum.  qs: its query in shared memory (fp32, this
// warp's own copy); lane l returns o[l + 32 i] in acc[i].
__device__ __forceinline__ void attn_row(const BlockAttn &p, int b, int s,
                                         int hk, const float *qs, int lane,
                                         bool &bad, float (&acc)[4],
                                         float &lse) {
  const float neg_inf = -__int_as_float(0x7f800000);
  float m = neg_inf, l = 0.f;
  for (int i = 0; i < 4; ++i) acc[i] = 0.f;
  row_keys(p, b, s, hk, qs, lane, bad,
           [&](int, float x, bool has, long long, long long vo) {
             float t = has ? x : neg_inf;
             for (int o = 16; o; o >>= 1)
               t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
             const float mn = fmaxf(m, t);
             const unsigned any = __ballot_sync(0xffffffffu, has);
             if (!any) return;
             // a finite stand-in while every score so far is -inf
             const float mu = mn > neg_inf ? mn : 0.f;
             const float f = m > neg_inf ? expf(m - mu) : 0.f;
             const float e = has ? expf(x - mu) : 0.f;
             float es = e;
             for (int o = 16; o; o >>= 1)
               es += __shfl_xor_sync(0xffffffffu, es, o);
             l = l * f + es;
             for (int i = 0; i < 4; ++i) acc[i] *= f;
             m = mn;
             for (int t2 = 0; t2 < 32; ++t2) {
               const long long at = __shfl_sync(0xffffffffu, vo, t2);
               const float w = __shfl_sync(0xffffffffu, e, t2);
               if (!(any >> t2 & 1u)) continue;
               for (int i = 0; i * 32 < p.D; ++i)
                 acc[i] = fmaf(w, __bfloat162float(p.v[at + lane + 32 * i]),
                               acc[i]);
             }
           });
  const bool some = l > 0.f || l != l;
  for (int i = 0; i < 4; ++i) acc[i] = some ? acc[i] / l : 0.f;
  lse = some ? m + logf(l) : neg_inf;
}

}  // namespace dsa
