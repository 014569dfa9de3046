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

// Registers of a thread move between the warpgroups of a CTA: never more than
// the launch gave to all of them.
template <int R>
__device__ __forceinline__ void regs_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void regs_fewer() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// One row by one warp in fp32 on the CUDA cores: a running maximum and sum
// over its keys, 32 at a time, lane l holding one.  Rows of a tile whose fast
// result is not finite are computed again by it where a key that only other rows
// see may be the reason.  qs: the query times 2^-eq as fp32 in shared memory,
// this warp's own copy; lane l returns o[l D / 32 + i] in acc[i].
//
// A chain of loads, those of 32 keys and their values on the way together: 3
// to 5 ms for 131072 keys, 125 ms for 2^21, so that the four rows that a warp may
// have end well within the limit of the waits for it, four seconds.  (A value at a
// time it took 28 to 57 ms for 131072 keys, which is 0.9 s for 2^21; 16 at a time
// behind branches 9 to 19 ms.)
template <int D>
__device__ __forceinline__ void attn_row_q8(const BlockAttnQ8 &p, int b,
                                            int s, int hk, const float *qs,
                                            int eq, int lane, bool &bad,
                                            float (&acc)[D / 32], float &lse) {
  constexpr int C = D / 32;  // columns of a lane
  const float neg_inf = -__int_as_float(0x7f800000);
  const long long pos = row_pos(p.q_pos, b, s);
  const int32_t *ids = row_ids(p, b, s, hk);
  const int n_cand = p.topk + p.local;
  float m = neg_inf, l = 0.f;
  for (int i = 0; i < C; ++i) acc[i] = 0.f;
  // (a sum that is not a number stays one, and o with it)
  for (int i = 0; i < n_cand && l == l; ++i) {
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
      const unsigned any = __ballot_sync(0xffffffffu, has);
      if (!any) continue;
      const int off = off0 + min(jj, p.blk - 1);
      const int ek = q8_exp(__ldg(p.c.ks + q8_scale_at(p.c, page, off, hk)));
      const float sv = q8_pow2(q8_exp(__ldg(p.c.vs + q8_scale_at(p.c, page, off, hk))));
      // (keys that the row does not see lie in the page, too: read, not used)
      const uint4 *kr = reinterpret_cast<const uint4 *>(
          p.c.k + page * p.c.k_p + off * p.c.k_t + hk * p.c.k_h);
      const long long vo = page * p.c.v_p + off * p.c.v_t + hk * p.c.v_h;
      uint4 kw[D / 16];
#pragma unroll
      for (int u = 0; u < D / 16; ++u) kw[u] = __ldg(kr + u);
      uint32_t v[32];
#pragma unroll
      for (int u = 0; u < 32; ++u) {
        const uint8_t *at = p.c.v + __shfl_sync(0xffffffffu, vo, u) + lane * C;
        if constexpr (C == 4)
          v[u] = __ldg(reinterpret_cast<const uint32_t *>(at));
        else
          v[u] = __ldg(reinterpret_cast<const uint16_t *>(at));
      }
      float x = 0.f;
#pragma unroll
      for (int u = 0; u < D / 16; ++u) {
        const uint32_t w[4] = {kw[u].x, kw[u].y, kw[u].z, kw[u].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float *qd = qs + 16 * u + 4 * k;
          const float2 lo = q8_float2(w[k] & 0xffffu), hi = q8_float2(w[k] >> 16);
          x = fmaf(qd[0], lo.x, x);
          x = fmaf(qd[1], lo.y, x);
          x = fmaf(qd[2], hi.x, x);
          x = fmaf(qd[3], hi.y, x);
        }
      }
      x = scalbnf(x * p.scale, ek + eq);  // (the factor may pass fp32)
      float t = has ? x : neg_inf;
      for (int o = 16; o; o >>= 1)
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
      const float mn = fmaxf(m, t);
      // a finite stand-in while every score so far is -inf
      const float mu = mn > neg_inf ? mn : 0.f;
      const float f = m > neg_inf ? expf(m - mu) : 0.f;
      const float e = has ? expf(x - mu) : 0.f;
      float es = e;
      for (int o = 16; o; o >>= 1) es += __shfl_xor_sync(0xffffffffu, es, o);
      l = l * f + es;
      if (l != l) break;
      for (int k = 0; k < C; ++k) acc[k] *= f;
      m = mn;
#pragma unroll
      for (int u = 0; u < 32; ++u) {
        const float w = __shfl_sync(0xffffffffu, e * sv, u);
        const uint32_t y = any >> u & 1u ? v[u] : 0u;
#pragma unroll
        for (int k = 0; k < C; k += 2) {
          const float2 t2 = q8_float2(k ? y >> 16 : y & 0xffffu);
          acc[k] = fmaf(w, t2.x, acc[k]);
          acc[k + 1] = fmaf(w, t2.y, acc[k + 1]);
        }
      }
    }
  }
  const bool some = l > 0.f || l != l;
  for (int k = 0; k < C; ++k) acc[k] = some ? acc[k] / l : 0.f;
  lse = some ? m + logf(l) : neg_inf;
}

// The same, written to o and lse: row s, head h.  qs: 128 floats.  The query
// is brought to [1, 2) first, so that its products stay within fp32 whatever
// finite values it has.  (Inlined, rare as it is: kernels with setmaxnreg make
// no calls.)
template <int D>
__device__ __forceinline__ void redo_row_q8(const BlockAttnQ8 &p, int b, int s,
                                            int h, float *qs, int lane) {
  const size_t at = ((size_t)s * p.B + b) * p.H + h;
  float top = 0.f;
  for (int d = lane; d < D; d += 32)
    top = fmaxf(top, fabsf(__bfloat162float(p.q[at * D + d])));
  top = __int_as_float(__reduce_max_sync(0xffffffffu, __float_as_int(top)));
  const int eq = min(max((__float_as_int(top) >> 23) - 127, -100), 120);
  const float f = q8_pow2(-eq);
  __syncwarp();
  for (int d = lane; d < D; d += 32)
    qs[d] = __bfloat162float(p.q[at * D + d]) * f;
  __syncwarp();
  bool bad = false;
  float acc[D / 32], lse;
  attn_row_q8<D>(p, b, s, h / p.G, qs, eq, lane, bad, acc, lse);
  if constexpr (D == 128)
    reinterpret_cast<uint2 *>(p.o + at * D)[lane] = make_uint2(
        pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]));
  else
    reinterpret_cast<uint32_t *>(p.o + at * D)[lane] =
        pack_bf16x2(acc[0], acc[1]);
  if (lane == 0) p.lse[at] = lse;
}

}  // namespace dsa
