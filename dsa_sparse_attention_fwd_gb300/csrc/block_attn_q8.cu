// Attention over a paged cache held in 8 bits (cache_q8.cuh), of selected
// blocks of keys or of all keys: the rows of block_attn.cu with
//     x_j = scale s_k q.k_j,  o = sum_j softmax(x)_j s_v v_j
// where k_j, v_j are e4m3 values and s_k, s_v the powers of two of their groups.
#include "block_attn_host.cuh"
#include "block_attn_q8.cuh"
#include "dsa_indexer.h"

namespace dsa {
namespace {

// Which problems take the kernel for few rows (block_attn_q8_step.cu), by the
// rows that share keys: S * G with all keys, G of a selection, whose queries it
// takes one by one.  Both kernels measured on 4 key heads at 12000 to 16000
// keys, or 34 blocks of 64 (us on the device; the other kernel joins split
// tiles in a second launch, 4 us more of the host's time up to 76 pairs of
// sequence and key head):
//   all keys, 16 rows: few 18 / 50 / 151 for 1 / 16 / 64 sequences of 128
//     dimensions, many 28 / 69 / 252; 32 rows: few 32 / 91 / 278, many 28 / 69 /
//     252.  At 64 dimensions, 32 rows: few 20 / 51 / 155, many 18 / 65 / 217;
//     64 rows: few 19 / 84 / 288, many 19 / 74 / 244.
//   a selection, one token, 16 rows: few 21 / 21 / 21 / 42 for 1 / 4 / 16 / 64
//     sequences, many 16 / 18 / 22 / 46 (two launches up to 16).  Up to 4
//     sequences the rule goes by the host's time, 21 us a call with one launch
//     and 27 with two; in a captured graph, which has none, the kernel for many
//     rows would be the faster one there.
//   a selection, four tokens of 8 heads: few 18 / 20 / 37 / 116, many 24 / 19 /
//     28 / 67, where tokens that share blocks read them once.
bool few_rows(int S, int B, int Hk, int G, int D, int topk) {
  if (topk > 0)
    return G <= 16 && (S == 1 || (long long)S * B * Hk <= 128);
  return (long long)S * G <= (D == 64 ? 32 : 16);
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
  if (dsa::few_rows(S, B, Hk, H / Hk, D, topk))
    return dsa::attn_q8_step_workspace_bytes(D);
  return dsa_block_attn_workspace_size(S, B, H, Hk, D, T, block_size, topk,
                                       local_blocks);
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
  if (dsa::few_rows(S, B, Hk, p.G, D, topk))
    return dsa::run_attn_q8_step(p, workspace, num_sms,
                                 static_cast<cudaStream_t>(cuda_stream));
  return dsa::run_attn_q8_tile(p, workspace, num_sms,
                               static_cast<cudaStream_t>(cuda_stream));
}

}  // extern "C"
