// Forward launches of the block attention: how its query tiles are shared among
// CTAs, over either cache.
#pragma once

#include "block_attn.cuh"

namespace dsa {

constexpr int kRows = 128;  // MMA rows of a query tile
constexpr int kKeys = 64;   // keys of a step

// What a launch adds to the problem.
struct FwdPlan {
  int qt;      // queries of a tile
  int tiles;   // query tiles of a sequence
  int splits;  // CTAs that share a tile's blocks
  int cap;     // entries of the block list
  __nv_bfloat16 *o;
  float *lse;
  // splits > 1: [item][split][qt * G] rows of D and of log-sums (base 2)
  float *part_o, *part_l;
};

// Room for two CTAs an SM on the largest device: a split launch has no more.
constexpr int kSplitItems = 320;
// A CTA takes some 5 us to start and end, a step 0.6 us.
constexpr int kMinSteps = 2;

// The launch of a problem; `workspace` as dsa_block_attn_workspace_size() says.
inline FwdPlan plan_fwd(const BlockAttn &p, void *out_o, float *out_lse,
                        void *workspace, int num_sms) {
  FwdPlan pl{};
  pl.qt = tile_queries(p.G, kRows);
  if (pl.qt > p.S) pl.qt = p.S;
  pl.tiles = (p.S + pl.qt - 1) / pl.qt;
  const long long most = (long long)pl.qt * (p.topk + p.local);
  pl.cap = (int)(most < p.nblk ? most : p.nblk);
  pl.o = static_cast<__nv_bfloat16 *>(out_o);
  pl.lse = out_lse;
  // Few tiles: share each among CTAs until two an SM are busy, with
  // kMinSteps steps each at least.
  const long long items = (long long)pl.tiles * p.B * p.Hk;
  long long slots = 2ll * num_sms;
  if (slots > kSplitItems) slots = kSplitItems;
  pl.splits = 1;
  if (items * 2 <= slots) {
    long long n = slots / items;
    long long steps = ((long long)pl.cap * p.blk + kKeys - 1) / kKeys;
    steps = (steps + kMinSteps - 1) / kMinSteps;
    if (n > steps) n = steps;
    if (n > 255) n = 255;  // counted in a byte
    pl.splits = (int)n;
  }
  if (pl.splits > 1) {
    char *ws = static_cast<char *>(workspace);
    pl.part_l = reinterpret_cast<float *>(ws + 256);
    const size_t rows = (size_t)items * pl.splits * pl.qt * p.G;
    pl.part_o = pl.part_l + ((rows + 63) & ~(size_t)63);
  }
  return pl;
}

}  // namespace dsa
