// Attention over a paged cache held in 8 bits (cache_q8.cuh), of selected
// blocks of keys or of all keys: the rows of block_attn.cu with
//     x_j = scale s_k q.k_j,  o = sum_j softmax(x)_j s_v v_j
// where k_j, v_j are e4m3 values and s_k, s_v the powers of two of their groups.
#include "block_attn_host.cuh"
#include "block_attn_q8.cuh"
#include "dsa_indexer.h"

namespace dsa {
namespace {

// Rows of a sequence and key head that take the kernel for few rows.
bool few_rows(int S, int G) { return (long long)S * G <= 64; }

// One warp a row.
__global__ void __launch_bounds__(128) attn_q8_rows_kernel(
    const __grid_constant__ BlockAttnQ8 p) {
  __shared__ float qs[4][128];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long rows = (long long)p.S * p.B * p.H;
  for (long long r = (long long)blockIdx.x * 4 + warp; r < rows;
       r += (long long)gridDim.x * 4) {
    const int h = (int)(r % p.H), b = (int)(r / p.H % p.B);
    const int s = (int)(r / p.H / p.B);
    __syncwarp();
    for (int d = lane; d < p.D; d += 32)
      qs[warp][d] = __bfloat162float(p.q[r * p.D + d]);
    __syncwarp();
    float acc[4], lse;
    bool bad = false;
    attn_row_q8(p, b, s, h / p.G, qs[warp], lane, bad, acc, lse);
    if (bad) atomicOr(p.status, kStatusIndexRange);
    for (int i = 0; i * 32 < p.D; ++i)
      p.o[r * p.D + lane + 32 * i] = __float2bfloat16(acc[i]);
    if (lane == 0) p.lse[r] = lse;
  }
}

}  // namespace
}  // namespace dsa

extern "C" {

size_t dsa_block_attn_q8_workspace_size(int S, int B, int H, int Hk, int D,
                                        int T, int block_size, int topk,
                                        int local_blocks) {
  if (S <= 0 || B <= 0 || H <= 0 || Hk <= 0 || H % Hk != 0 || D <= 0 ||
      T <= 0 || block_size <= 0 || topk < 0 || local_blocks < 0)
    return 0;
  return dsa::few_rows(S, H / Hk) ? dsa::attn_q8_step_workspace_bytes(D) : 256;
}

int dsa_block_attn_paged_q8_fwd(
    const void *q, const void *k_cache, const void *v_cache,
    const int64_t *cache_strides, const float *k_scale, const float *v_scale,
    int group, int num_pages, int page_size, const int32_t *page_table,
    int max_pages, int S, int B, int H, int Hk, int D, const int32_t *blocks,
    int sel_heads, int topk, int block_size, int local_blocks,
    const int32_t *q_pos, float scale, void *out_o, float *out_lse,
    void *workspace, size_t workspace_bytes, void *cuda_stream) {
  if (!k_cache || !v_cache || !k_scale || !v_scale || !out_o || !out_lse)
    return DSA_ERR_INVALID_ARG;
  dsa::BlockAttnQ8 p{};
  int rc = dsa::set_q8_cache(p.c, k_cache, v_cache, cache_strides, k_scale,
                             v_scale, group, num_pages, page_size, page_table,
                             max_pages, Hk, D);
  if (rc != DSA_OK) return rc;
  p.q = static_cast<const __nv_bfloat16 *>(q);
  p.S = S, p.B = B, p.H = H, p.Hk = Hk, p.D = D;
  p.T = max_pages * page_size;
  p.table = page_table, p.max_pages = max_pages;
  p.page_size = page_size, p.num_pages = num_pages;
  // (checked as addresses and strides of 16 bytes already)
  dsa::set_kv(p, k_cache, v_cache, nullptr, (long long)Hk * D,
              (long long)page_size * Hk * D);
  p.blocks = blocks, p.sel_heads = sel_heads, p.topk = topk;
  p.blk = block_size, p.local = local_blocks;
  p.q_pos = q_pos, p.scale = scale;
  rc = dsa::check_block_attn(p);
  if (rc != DSA_OK) return rc;
  if (!dsa::aligned_to(out_o, 16) || !dsa::aligned_to(out_lse, 4))
    return DSA_ERR_INVALID_ARG;
  const size_t need = dsa_block_attn_q8_workspace_size(
      S, B, H, Hk, D, p.T, block_size, topk, local_blocks);
  if (!workspace || workspace_bytes < need) return DSA_ERR_WORKSPACE;
  if (!dsa::aligned_to(workspace, 256)) return DSA_ERR_INVALID_ARG;
  p.status = static_cast<int *>(workspace);
  p.o = static_cast<__nv_bfloat16 *>(out_o);
  p.lse = out_lse;
  int num_sms = 0;
  rc = dsa::device_num_sms(&num_sms);
  if (rc != DSA_OK) return rc;
  if (dsa::few_rows(S, p.G))
    return dsa::run_attn_q8_step(p, workspace, num_sms,
                                 static_cast<cudaStream_t>(cuda_stream));
  const long long grid = ((long long)S * B * H + 3) / 4;
  const long long most = 16ll * num_sms;
  dsa::attn_q8_rows_kernel<<<(unsigned)(grid < most ? grid : most), 128, 0,
                             static_cast<cudaStream_t>(cuda_stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // extern "C"
