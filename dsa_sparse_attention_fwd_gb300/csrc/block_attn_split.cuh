// Forward launches of the block attention: how its query tiles are shared among
// CTAs, and the join of the parts of tiles that several CTAs work on.
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
  uint32_t *done;  // a byte an item: parts written; zero between calls
};

// Joins the parts of a split tile, o = sum_i w_i o_i / sum_i w_i with w_i =
// 2^(l_i - max), in the order of the splits; the CTA that finished last.  A
// thread takes four columns of a row and has kJoin parts in flight: the join
// is a chain of loads from L2.  qs: 128 floats of shared memory a warp.
constexpr int kJoin = 8;
// redo(b, s, h, qs, lane): a row with a part that is not finite, by one warp.
// (Callers that can keep it out of line do: it runs once a tile.)
template <int D, int THREADS, typename F>
__device__ __forceinline__ void join_parts(const BlockAttn &p, const FwdPlan &pl,
                                        size_t part0, int b, int s0, int nq,
                                        int hk, float *qs, int tid, F redo) {
  constexpr int kLanes = D / 4;  // threads of a row: half a warp or a warp
  const float neg_inf = -__int_as_float(0x7f800000);
  const int rows = pl.qt * p.G, lane = tid & 31, c = tid % kLanes;
  const int todo = nq * p.G;
  // (whole warps stay in the loop: they vote)
  for (int r0 = tid / 32 * (32 / kLanes); r0 < todo;
       r0 += THREADS / kLanes) {
    const int r = r0 + lane / kLanes;
    const bool mine = r < todo;
    const size_t part = part0 + (mine ? r : 0);
    float m = neg_inf, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    bool odd = false;
    for (int i0 = 0; i0 < pl.splits; i0 += kJoin) {
      float l[kJoin];
      float4 v[kJoin];
#pragma unroll
      for (int u = 0; u < kJoin; ++u) {
        const size_t at = part + (size_t)min(i0 + u, pl.splits - 1) * rows;
        l[u] = __ldcg(pl.part_l + at);
        v[u] = __ldcg(reinterpret_cast<const float4 *>(pl.part_o + at * D) + c);
        if (i0 + u >= pl.splits) l[u] = neg_inf;
      }
      float mx = m;
#pragma unroll
      for (int u = 0; u < kJoin; ++u) {
        odd |= l[u] != l[u];
        mx = fmaxf(mx, l[u]);
      }
      const float ref = mx > neg_inf ? mx : 0.f;
      const float f = ex2(m - ref);
      sum *= f, acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f;
#pragma unroll
      for (int u = 0; u < kJoin; ++u) {
        const float w = ex2(l[u] - ref);
        sum += w;
        acc.x = fmaf(w, v[u].x, acc.x);
        acc.y = fmaf(w, v[u].y, acc.y);
        acc.z = fmaf(w, v[u].z, acc.z);
        acc.w = fmaf(w, v[u].w, acc.w);
      }
      m = mx;
    }
    const int s = s0 + r / p.G, h = hk * p.G + r % p.G;
    if (mine) {
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
      const size_t at = ((size_t)s * p.B + b) * p.H + h;
      reinterpret_cast<uint2 *>(pl.o + at * D)[c] =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv),
                     pack_bf16x2(acc.z * inv, acc.w * inv));
      if (c == 0)
        pl.lse[at] =
            sum > 0.f ? (m + log2f(sum)) * 0.69314718055994531f : neg_inf;
    }
    // rows with a part that is not finite
    unsigned again = __ballot_sync(0xffffffffu, mine && odd && c == 0);
    for (; again; again &= again - 1) {
      const int ra = r0 + (__ffs(again) - 1) / kLanes;
      redo(b, s0 + ra / p.G, hk * p.G + ra % p.G, qs + tid / 32 * 128, lane);
    }
  }
}

// Room for two CTAs an SM on the largest device: a split launch has no more.
constexpr int kSplitItems = 320;
// A CTA takes some 5 us to start and end, a step 0.6 us.
constexpr int kMinSteps = 2;
// The counts of written parts, in the 256 bytes that every entry point leaves
// to the status word: no other use of a workspace touches them.
constexpr int kDoneOffset = 64;
static_assert(kDoneOffset + kSplitItems / 2 <= 256,
              "a byte for each item that is split");

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
    pl.done = reinterpret_cast<uint32_t *>(ws + kDoneOffset);
    pl.part_l = reinterpret_cast<float *>(ws + 256);
    const size_t rows = (size_t)items * pl.splits * pl.qt * p.G;
    pl.part_o = pl.part_l + ((rows + 63) & ~(size_t)63);
  }
  return pl;
}

}  // namespace dsa
