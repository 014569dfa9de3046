// Attention over a paged cache held in 8 bits: the problem as the kernels of
// block_attn_q8*.cu see it, and one row from the formulas.
#pragma once

#include "block_attn.cuh"
#include "cache_q8.cuh"

namespace dsa {

struct BlockAttnQ8 : BlockAttn {  // k, v and their strides: unused
  Q8Cache c;
  __nv_bfloat16 *o;
  float *lse;
};

// TMA map of e4m3 keys or values as (d, token, head, page) with a box of D (64
// or 128) x `rows` tokens (api.cu).
int encode_kv8(CUtensorMap *m, const void *base, int D, int rows,
               long long tokens, long long st, long long heads, long long sh,
               long long outer, long long sx);

// Few rows (block_attn_q8_step.cu).
size_t attn_q8_step_workspace_bytes(int D);
int run_attn_q8_step(const BlockAttnQ8 &p, void *workspace, int num_sms,
                     cudaStream_t st);

// Many (block_attn_q8_tile.cu); workspace as for dsa_block_attn_fwd().
int run_attn_q8_tile(const BlockAttnQ8 &p, void *workspace, int num_sms,
                     cudaStream_t st);

// One row by one warp in fp32 on the CUDA cores: a running maximum and sum
// over its keys, 32 at a time, lane l holding one.  Rows whose fast result is
// not finite are computed again by it: a key that only other rows of a tile
// see may hold anything.  qs: the query times 2^-eq as fp32 in shared memory,
// this warp's own copy; lane l returns o[l + 32 i] in acc[i].
__device__ __forceinline__ void attn_row_q8(const BlockAttnQ8 &p, int b,
                                            int s, int hk, const float *qs,
                                            int eq, int lane, bool &bad,
                                            float (&acc)[4], float &lse) {
  const float neg_inf = -__int_as_float(0x7f800000);
  const long long pos = row_pos(p.q_pos, b, s);
  const int32_t *ids = row_ids(p, b, s, hk);
  const int n_cand = p.topk + p.local;
  float m = neg_inf, l = 0.f;
  for (int i = 0; i < 4; ++i) acc[i] = 0.f;
  for (int i = 0; i < n_cand; ++i) {
    if (i >= p.topk && pos < (long long)(i - p.topk) << p.lb) break;
    const int n = candidate(p, ids, pos, i, bad);
    if (n < 0) continue;
    bool again = false;  // a block given twice counts once
    for (int t = lane; t < i && i < p.topk; t += 32)
      again |= __ldg(ids + t) == n;
    if (__any_sync(0xffffffffu, again)) continue;
    const int page = block_page(p, b, n, bad);
    if (page < 0) continue;
    const int off0 =
        (int)((unsigned)n * (unsigned)p.blk % (unsigned)p.page_size);
    for (int c = 0; c < p.blk; c += 32) {
      const int jj = c + lane;
      const long long j = (long long)n * p.blk + jj;
      const bool has = jj < p.blk && j <= pos && j < p.T;
      const int off = off0 + min(jj, p.blk - 1);
      const int ek = q8_exp(__ldg(p.c.ks + q8_scale_at(p.c, page, off, hk)));
      const float sv = q8_pow2(q8_exp(__ldg(p.c.vs + q8_scale_at(p.c, page, off, hk))));
      const uint8_t *kr =
          p.c.k + page * p.c.k_p + off * p.c.k_t + hk * p.c.k_h;
      const long long vo = page * p.c.v_p + off * p.c.v_t + hk * p.c.v_h;
      float x = 0.f;
      if (has) {
        for (int d = 0; d < p.D; d += 4) {
          const uint32_t w = *reinterpret_cast<const uint32_t *>(kr + d);
          const float2 lo = q8_float2(w & 0xffffu), hi = q8_float2(w >> 16);
          x = fmaf(qs[d], lo.x, x);
          x = fmaf(qs[d + 1], lo.y, x);
          x = fmaf(qs[d + 2], hi.x, x);
          x = fmaf(qs[d + 3], hi.y, x);
        }
        x = scalbnf(x * p.scale, ek + eq);  // (the factor may pass fp32)
      }
      float t = has ? x : neg_inf;
      for (int o = 16; o; o >>= 1)
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
      const float mn = fmaxf(m, t);
      const unsigned any = __ballot_sync(0xffffffffu, has);
      if (!any) continue;
      // a finite stand-in while every score so far is -inf
      const float mu = mn > neg_inf ? mn : 0.f;
      const float f = m > neg_inf ? expf(m - mu) : 0.f;
      const float e = has ? expf(x - mu) : 0.f;
      float es = e;
      for (int o = 16; o; o >>= 1) es += __shfl_xor_sync(0xffffffffu, es, o);
      l = l * f + es;
      for (int k = 0; k < 4; ++k) acc[k] *= f;
      m = mn;
      for (int t2 = 0; t2 < 32; ++t2) {
        const long long at = __shfl_sync(0xffffffffu, vo, t2);
        const float w = __shfl_sync(0xffffffffu, e * sv, t2);
        if (!(any >> t2 & 1u)) continue;
        for (int k = 0; k * 32 < p.D; ++k) {
          const float2 v = q8_float2(p.c.v[at + lane + 32 * k]);
          acc[k] = fmaf(w, v.x, acc[k]);
        }
      }
    }
  }
  const bool some = l > 0.f || l != l;
  for (int k = 0; k < 4; ++k) acc[k] = some ? acc[k] / l : 0.f;
  lse = some ? m + logf(l) : neg_inf;
}

// The same, written to o and lse: row s, head h.  qs: 128 floats.  The query
// is brought to [1, 2) first, so that its products stay within fp32 whatever
// finite values it has.  (Inlined, rare as it is: kernels with setmaxnreg make
// no calls.)
__device__ __forceinline__ void redo_row_q8(const BlockAttnQ8 &p, int b, int s,
                                            int h, float *qs, int lane) {
  const size_t at = ((size_t)s * p.B + b) * p.H + h;
  float top = 0.f;
  for (int d = lane; d < p.D; d += 32)
    top = fmaxf(top, fabsf(__bfloat162float(p.q[at * p.D + d])));
  top = __int_as_float(__reduce_max_sync(0xffffffffu, __float_as_int(top)));
  const int eq = min(max((__float_as_int(top) >> 23) - 127, -100), 120);
  const float f = q8_pow2(-eq);
  __syncwarp();
  for (int d = lane; d < p.D; d += 32)
    qs[d] = __bfloat162float(p.q[at * p.D + d]) * f;
  __syncwarp();
  bool bad = false;
  float acc[4], lse;
  attn_row_q8(p, b, s, h / p.G, qs, eq, lane, bad, acc, lse);
  for (int i = 0; i * 32 < p.D; ++i)
    p.o[at * p.D + lane + 32 * i] = __float2bfloat16(acc[i]);
  if (lane == 0) p.lse[at] = lse;
}

}  // namespace dsa
