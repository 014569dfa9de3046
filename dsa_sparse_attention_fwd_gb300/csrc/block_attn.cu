// Attention over selected blocks of keys, forward: contiguous and paged keys
// and values, grouped heads, a running softmax.  Row (s, b) at position
// p = q_pos[b] + s attends to the keys j <= p of its blocks: the topk given
// ids (each once) and the `local` blocks that end with its own.
//     x_j = scale q.k_j,  o = softmax(x) v,  lse = ln sum exp x
#include "block_attn.cuh"
#include "block_attn_host.cuh"
#include "block_attn_row.cuh"
#include "dsa_indexer.h"

namespace dsa {
namespace {

constexpr int kRowWarps = 8;

// One warp per (row, head).
__global__ void __launch_bounds__(kRowWarps * 32)
    block_attn_rows_kernel(const BlockAttn p, __nv_bfloat16 *out_o,
                           float *out_lse) {
  __shared__ float qs_all[kRowWarps][128];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long it = (long long)blockIdx.x * kRowWarps + warp;
  if (it >= (long long)p.S * p.B * p.H) return;
  const int h = (int)(it % p.H);
  const int b = (int)(it / p.H % p.B), s = (int)(it / p.H / p.B);
  float *qs = qs_all[warp];
  for (int d = lane; d < p.D; d += 32)
    qs[d] = __bfloat162float(p.q[it * p.D + d]);
  __syncwarp();
  bool bad = false;
  float acc[4], lse;
  attn_row(p, b, s, h / p.G, qs, lane, bad, acc, lse);
  for (int i = 0; i * 32 < p.D; ++i)
    out_o[it * p.D + lane + 32 * i] = __float2bfloat16(acc[i]);
  if (lane == 0) out_lse[it] = lse;
  if (__any_sync(0xffffffffu, bad) && lane == 0)
    atomicOr(p.status, kStatusIndexRange);
}

int run_fwd(const BlockAttn &p, void *out_o, float *out_lse, void *workspace,
            cudaStream_t st) {
  const long long rows = (long long)p.S * p.B * p.H;
  block_attn_rows_kernel<<<(unsigned)((rows + kRowWarps - 1) / kRowWarps),
                           kRowWarps * 32, 0, st>>>(
      p, static_cast<__nv_bfloat16 *>(out_o), out_lse);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

int fwd_common(BlockAttn &p, void *out_o, float *out_lse, void *workspace,
               size_t workspace_bytes, void *cuda_stream) {
  if (!out_o || !out_lse) return DSA_ERR_INVALID_ARG;
  const int rc = check_block_attn(p);
  if (rc != DSA_OK) return rc;
  if (!aligned_to(out_o, 16) || !aligned_to(out_lse, 4))
    return DSA_ERR_INVALID_ARG;
  const size_t need = dsa_block_attn_workspace_size(
      p.S, p.B, p.H, p.Hk, p.D, p.T, p.blk, p.topk, p.local);
  if (!workspace || workspace_bytes < need) return DSA_ERR_WORKSPACE;
  if (!aligned_to(workspace, 256)) return DSA_ERR_INVALID_ARG;
  p.status = static_cast<int *>(workspace);
  int num_sms = 0;
  const int rd = device_num_sms(&num_sms);
  if (rd != DSA_OK) return rd;
  return run_fwd(p, out_o, out_lse, workspace,
                 static_cast<cudaStream_t>(cuda_stream));
}

}  // namespace

// Argument checks of the forward and the backward (no device access); fills
// in the derived sizes.
int check_block_attn(BlockAttn &p) {
  if (!p.q || !p.k || !p.v || (p.topk > 0 && !p.blocks))
    return DSA_ERR_INVALID_ARG;
  if (p.S <= 0 || p.B <= 0 || p.H <= 0 || p.Hk <= 0 || p.D <= 0 ||
      p.T <= 0 || p.topk < 0 || p.local < 0 || p.topk + p.local <= 0 ||
      p.blk <= 0 || p.H % p.Hk != 0)
    return DSA_ERR_INVALID_ARG;
  if (p.sel_heads != 1 && p.sel_heads != p.Hk) return DSA_ERR_INVALID_ARG;
  if (!(p.scale > 0.f) || p.scale > 1e30f) return DSA_ERR_INVALID_ARG;
  if (p.D != 64 && p.D != 128) return DSA_ERR_UNSUPPORTED;
  if (p.blk != 16 && p.blk != 32 && p.blk != 64 && p.blk != 128)
    return DSA_ERR_UNSUPPORTED;
  p.G = p.H / p.Hk;
  if (p.G > DSA_BLOCK_ATTN_MAX_GROUP) return DSA_ERR_UNSUPPORTED;
  p.nblk = (int)(((long long)p.T + p.blk - 1) / p.blk);
  if (p.nblk > DSA_BLOCK_ATTN_MAX_BLOCKS || p.topk > DSA_BLOCK_ATTN_MAX_BLOCKS ||
      p.local > DSA_BLOCK_ATTN_MAX_BLOCKS)
    return DSA_ERR_UNSUPPORTED;
  if ((long long)p.S * p.B >= (1ll << 31) / p.H) return DSA_ERR_UNSUPPORTED;
  if (p.table) {
    if (p.page_size % p.blk != 0) return DSA_ERR_UNSUPPORTED;
    if (!aligned_to(p.table, 4)) return DSA_ERR_INVALID_ARG;
  }
  if (!aligned_to(p.q, 16) || !aligned_to(p.k, 16) || !aligned_to(p.v, 16) ||
      !aligned_to(p.blocks, 4) || !aligned_to(p.q_pos, 4))
    return DSA_ERR_INVALID_ARG;
  for (long long s : {p.k_st, p.k_sb, p.k_sh, p.v_st, p.v_sb, p.v_sh})
    if (s % 8 != 0 || s < 0 || s >= (1ll << 38)) return DSA_ERR_INVALID_ARG;
  return DSA_OK;
}

void set_kv(BlockAttn &p, const void *k, const void *v,
            const int64_t *strides, long long st, long long sb) {
  p.k = static_cast<const __nv_bfloat16 *>(k);
  p.v = static_cast<const __nv_bfloat16 *>(v);
  p.k_st = p.v_st = st;
  p.k_sb = p.v_sb = sb;
  p.k_sh = p.v_sh = p.D;
  if (strides) {
    p.k_st = strides[0], p.k_sb = strides[1], p.k_sh = strides[2];
    p.v_st = strides[3], p.v_sb = strides[4], p.v_sh = strides[5];
  }
}

}  // namespace dsa

extern "C" {

size_t dsa_block_attn_workspace_size(int S, int B, int H, int Hk, int D,
                                     int T, int block_size, int topk,
                                     int local_blocks) {
  if (S <= 0 || B <= 0 || H <= 0 || Hk <= 0 || H % Hk != 0 || D <= 0 ||
      T <= 0 || block_size <= 0 || topk < 0 || local_blocks < 0)
    return 0;
  return 256;
}

int dsa_block_attn_fwd(const void *q, const void *k, const void *v,
                       const int64_t *kv_strides, int S, int B, int H, int Hk,
                       int D, int T, const int32_t *blocks, int sel_heads,
                       int topk, int block_size, int local_blocks,
                       const int32_t *q_pos, float scale, void *out_o,
                       float *out_lse, void *workspace,
                       size_t workspace_bytes, void *cuda_stream) {
  dsa::BlockAttn p{};
  p.q = static_cast<const __nv_bfloat16 *>(q);
  p.S = S, p.B = B, p.H = H, p.Hk = Hk, p.D = D, p.T = T;
  dsa::set_kv(p, k, v, kv_strides, (long long)B * Hk * D, (long long)Hk * D);
  p.blocks = blocks, p.sel_heads = sel_heads, p.topk = topk;
  p.blk = block_size, p.local = local_blocks;
  p.q_pos = q_pos, p.scale = scale;
  return dsa::fwd_common(p, out_o, out_lse, workspace, workspace_bytes,
                         cuda_stream);
}

int dsa_block_attn_paged_fwd(
    const void *q, const void *k_cache, const void *v_cache,
    const int64_t *cache_strides, int num_pages, int page_size,
    const int32_t *page_table, int max_pages, int S, int B, int H, int Hk,
    int D, const int32_t *blocks, int sel_heads, int topk, int block_size,
    int local_blocks, const int32_t *q_pos, float scale, void *out_o,
    float *out_lse, void *workspace, size_t workspace_bytes,
    void *cuda_stream) {
  if (!page_table || num_pages <= 0 || page_size <= 0 || max_pages <= 0)
    return DSA_ERR_INVALID_ARG;
  if ((long long)max_pages * page_size >= (1ll << 31))
    return DSA_ERR_UNSUPPORTED;
  dsa::BlockAttn p{};
  p.q = static_cast<const __nv_bfloat16 *>(q);
  p.S = S, p.B = B, p.H = H, p.Hk = Hk, p.D = D;
  p.T = max_pages * page_size;
  p.table = page_table, p.max_pages = max_pages;
  p.page_size = page_size, p.num_pages = num_pages;
  // the caches' strides come as (page, slot, head)
  int64_t st[6];
  for (int i = 0; cache_strides && i < 6; ++i)
    st[i] = cache_strides[i % 3 == 0 ? i + 1 : i % 3 == 1 ? i - 1 : i];
  dsa::set_kv(p, k_cache, v_cache, cache_strides ? st : nullptr,
              (long long)Hk * D, (long long)page_size * Hk * D);
  p.blocks = blocks, p.sel_heads = sel_heads, p.topk = topk;
  p.blk = block_size, p.local = local_blocks;
  p.q_pos = q_pos, p.scale = scale;
  return dsa::fwd_common(p, out_o, out_lse, workspace, workspace_bytes,
                         cuda_stream);
}

}  // extern "C"
