// Backward of the block attention.  With P = exp(x - lse) from the saved
// log-sums:  dv_j += P do,  dP = do.v_j,  dS = P (dP - do.o) scale,
// dq += dS k_j,  dk_j += dS q; dk and dv are sums over the heads of a group.
#include "block_attn.cuh"
#include "block_attn_host.cuh"
#include "block_attn_row.cuh"
#include "dsa_indexer.h"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kRowWarps = 8;

// One warp per (row, head); dk and dv by fp32 atomics.
__global__ void __launch_bounds__(kRowWarps * 32)
    block_attn_bwd_rows_kernel(const BlockAttn p, const __nv_bfloat16 *o,
                               const float *lse, const __nv_bfloat16 *go,
                               __nv_bfloat16 *gq, float *gk, float *gv) {
  __shared__ float qs_all[kRowWarps][128], gs_all[kRowWarps][128];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long it = (long long)blockIdx.x * kRowWarps + warp;
  if (it >= (long long)p.S * p.B * p.H) return;
  const int h = (int)(it % p.H);
  const int b = (int)(it / p.H % p.B), s = (int)(it / p.H / p.B);
  const int hk = h / p.G;
  float *qs = qs_all[warp], *gs = gs_all[warp];
  float delta = 0.f;
  for (int d = lane; d < p.D; d += 32) {
    qs[d] = __bfloat162float(p.q[it * p.D + d]);
    gs[d] = __bfloat162float(go[it * p.D + d]);
    delta = fmaf(gs[d], __bfloat162float(o[it * p.D + d]), delta);
  }
  for (int x = 16; x; x >>= 1) delta += __shfl_xor_sync(0xffffffffu, delta, x);
  __syncwarp();
  const float ls = lse[it];
  bool bad = false;
  float acc[4] = {};
  row_keys(p, b, s, hk, qs, lane, bad,
           [&](int j, float x, bool has, long long ko, long long vo) {
             float pr = 0.f, ds = 0.f;
             if (has) {
               float dp = 0.f;
               for (int d = 0; d < p.D; ++d)
                 dp = fmaf(gs[d], __bfloat162float(p.v[vo + d]), dp);
               pr = expf(x - ls);
               ds = pr * (dp - delta) * p.scale;
             }
             const unsigned any = __ballot_sync(0xffffffffu, has);
             for (int t = 0; t < 32; ++t) {
               const long long at = __shfl_sync(0xffffffffu, ko, t);
               const float w = __shfl_sync(0xffffffffu, ds, t);
               const float pw = __shfl_sync(0xffffffffu, pr, t);
               const int jt = __shfl_sync(0xffffffffu, j, t);
               if (!(any >> t & 1u)) continue;
               const size_t g0 =
                   (((size_t)jt * p.B + b) * p.Hk + hk) * p.D + lane;
               for (int i = 0; i * 32 < p.D; ++i) {
                 const int d = lane + 32 * i;
                 acc[i] = fmaf(w, __bfloat162float(p.k[at + d]), acc[i]);
                 atomicAdd(gk + g0 + 32 * i, w * qs[d]);
                 atomicAdd(gv + g0 + 32 * i, pw * gs[d]);
               }
             }
           });
  for (int i = 0; i * 32 < p.D; ++i)
    gq[it * p.D + lane + 32 * i] = __float2bfloat16(acc[i]);
  if (__any_sync(0xffffffffu, bad) && lane == 0)
    atomicOr(p.status, kStatusIndexRange);
}

__global__ void round_kernel(const float *x, __nv_bfloat16 *y, size_t n) {
  for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n;
       i += (size_t)gridDim.x * blockDim.x)
    y[i] = __float2bfloat16(x[i]);
}

}  // namespace
}  // namespace dsa

extern "C" {

size_t dsa_block_attn_bwd_workspace_size(int S, int B, int H, int Hk, int D,
                                         int T, int block_size, int topk,
                                         int local_blocks) {
  if (dsa_block_attn_workspace_size(S, B, H, Hk, D, T, block_size, topk,
                                    local_blocks) == 0)
    return 0;
  return 256 + (size_t)T * B * Hk * D * 8;
}

int dsa_block_attn_bwd(const void *q, const void *k, const void *v,
                       const int64_t *kv_strides, const void *o,
                       const float *lse, const void *grad_o, int S, int B,
                       int H, int Hk, int D, int T, const int32_t *blocks,
                       int sel_heads, int topk, int block_size,
                       int local_blocks, const int32_t *q_pos, float scale,
                       void *grad_q, void *grad_k, void *grad_v,
                       void *workspace, size_t workspace_bytes,
                       void *cuda_stream) {
  if (!o || !lse || !grad_o || !grad_q || !grad_k || !grad_v)
    return DSA_ERR_INVALID_ARG;
  dsa::BlockAttn p{};
  p.q = static_cast<const __nv_bfloat16 *>(q);
  p.S = S, p.B = B, p.H = H, p.Hk = Hk, p.D = D, p.T = T;
  dsa::set_kv(p, k, v, kv_strides, (long long)B * Hk * D, (long long)Hk * D);
  p.blocks = blocks, p.sel_heads = sel_heads, p.topk = topk;
  p.blk = block_size, p.local = local_blocks;
  p.q_pos = q_pos, p.scale = scale;
  int rc = dsa::check_block_attn(p);
  if (rc != DSA_OK) return rc;
  using dsa::aligned_to;
  if (!aligned_to(o, 16) || !aligned_to(grad_o, 16) || !aligned_to(lse, 4) ||
      !aligned_to(grad_q, 16) || !aligned_to(grad_k, 16) ||
      !aligned_to(grad_v, 16))
    return DSA_ERR_INVALID_ARG;
  const size_t need = dsa_block_attn_bwd_workspace_size(
      S, B, H, Hk, D, T, block_size, topk, local_blocks);
  if (!workspace || workspace_bytes < need) return DSA_ERR_WORKSPACE;
  if (!aligned_to(workspace, 256)) return DSA_ERR_INVALID_ARG;
  p.status = static_cast<int *>(workspace);
  int num_sms = 0;
  rc = dsa::device_num_sms(&num_sms);
  if (rc != DSA_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const size_t n = (size_t)T * B * Hk * D;
  float *gk = reinterpret_cast<float *>(static_cast<char *>(workspace) + 256);
  float *gv = gk + n;
  if (cudaMemsetAsync(gk, 0, n * 8, st) != cudaSuccess) return DSA_ERR_CUDA;
  const long long rows = (long long)S * B * H;
  dsa::block_attn_bwd_rows_kernel<<<
      (unsigned)((rows + dsa::kRowWarps - 1) / dsa::kRowWarps),
      dsa::kRowWarps * 32, 0, st>>>(
      p, static_cast<const __nv_bfloat16 *>(o), lse,
      static_cast<const __nv_bfloat16 *>(grad_o),
      static_cast<__nv_bfloat16 *>(grad_q), gk, gv);
  dsa::round_kernel<<<1024, 256, 0, st>>>(
      gk, static_cast<__nv_bfloat16 *>(grad_k), n);
  dsa::round_kernel<<<1024, 256, 0, st>>>(
      gv, static_cast<__nv_bfloat16 *>(grad_v), n);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // extern "C"
