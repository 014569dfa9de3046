// Backward of the block attention.  With P = exp(x - lse) from the saved
// log-sums and delta = do.o (a sum over D):
//     dv_j = sum P do,   dP = do.v_j,   dS = P (dP - delta),
//     dq = scale sum dS k_j,   dk_j = scale sum dS q;
// dk and dv are sums over the heads of a group and over the rows that hold
// the key's block.
//   delta is read from the rounded o, e off, and every dS with it by P e.
// Where a key d has nearly all of a row's weight, dS_d is a small difference of
// which e may be most (a sink that holds 0.99 of the weights: dq 7.5% off, 39% in
// those rows).  sum dS = 0 by definition, so the sum that the dq pass finds is
// e: it corrects delta for dk and dv, and in dq it comes off dS_d where d has
// more than half of the weight.  What stays there is (1 - P_d) e, as small
// against the true dS as e is against dP; dS_d's own rounding, which the sum
// does not see, comes off with it.  dq and dk are then 0.23 to 0.25% off at any
// weight of the sink (one rounding of the exact ones: 0.17%), for 11 us of the
// training step below.  Rows without such a key at a sequence's first positions
// get delta from their keys (few_keys_delta).
//
// Two passes, each with its sums in tensor memory, so nothing is added
// atomically and the results do not change from run to run:
//   dq: a CTA takes a query tile (128 rows of queries x heads, as in the
// forward) and walks the union of its blocks, 64 keys a step: S = Q K^T, dP =
// dO V^T, dS in bf16 back into tensor memory, dQ += dS K.  Q and dO are operands
// from tensor memory: with both operands in shared memory, a product with 64
// columns is bound by reading its 128 rows again for each K step (48 cycles
// against 32).
//   dk, dv: a CTA takes 128 consecutive keys and walks the query tiles (64
// rows) that hold one of their blocks: S^T = K Q^T, dP^T = V dO^T, dV += P^T
// dO, dK += dS^T Q.  The list of these query tiles is the transpose of the
// selection: bwd_mark_kernel lists each query tile's blocks and sets a bit
// for each of its key tiles, bwd_scan_kernel turns the counts into offsets
// and cuts long lists (blocks that every query holds) into chunks of a
// quarter of an SM's share, bwd_fill_kernel writes them.  Chunks of one key
// tile leave their sums in fp32 and bwd_join_kernel adds them in order.
//   At D = 128 both run one CTA an SM with the scores of two steps in tensor
// memory: the compute warps work on one step (each of the two warpgroups on
// half of its columns) while the tensor cores run the products of its
// neighbours.  At D = 64, where the products are short, the sums and one step
// take half of tensor memory, and two CTAs share an SM.
//   Masks cost no arithmetic away from the diagonal: a (row, block) that is
// not held has a log-sum of +inf, so its weights are exp2(-inf) = 0.
//
// Measured on one GB300 (bf16 peak 1909 TFLOP/s) at 4096 tokens, 64 / 4 heads
// of 128, 17 blocks of 64: dk, dv 323 us, 1330 TFLOP/s of the lists' products;
// dq 202 us, 1190; delta 23, join 22, the transposed selection 33.  The tensor
// pipe is busy 55% and 50% of the time: dk, dv is bound by shared memory (its
// products with 64 columns read 6 KB in 48 cycles, for 32 of arithmetic; 1375
// cycles a step of 64 rows by that, 1600 to 1750 measured), dq by its chain of
// score product, exponentials and dS a step with one CTA an SM.
#include "block_attn.cuh"
#include "block_attn_host.cuh"
#include "dsa_indexer.h"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kBwdThreads = 320;  // 8 compute warps, TMA warp, MMA warp
constexpr int kTmaWarp = 8, kMmaWarp = 9;
constexpr int kKeyTile = 128;  // keys of a dk, dv item
constexpr int kRowTile = 64;   // rows of its query tiles
// A stage of 32 KB takes 1900 cycles to arrive from L2 and is held for 2900
// more, with a step every 1300 to 1500: four stages.
constexpr int kKvStages = 4;
constexpr int kMinChunk = 16;     // query tiles of a chunk at least
constexpr int kChunkUnits = 640;  // 4 chunks on each of 160 SMs
constexpr int kJoinParts = 16;    // CTAs that join a key tile's chunks
constexpr int kFewKeys = 32;      // see few_keys_delta

// The transposed selection and the other buffers in the workspace.
struct BwdPlan {
  int qt, nqt;      // queries of a 64-row tile, such tiles of a sequence
  int nkt, nqw;     // key tiles of a sequence, words of a bit row over nqt
  int bpt;          // blocks of a key tile
  int cap;          // blocks that a query tile can hold
  int rep;          // key heads that share a selection
  long long entries;  // of all lists, at most
  int items, slots;   // at most
  float2 *stat;       // [S, B, H] (lse log2 e, delta); no keys: (+inf, 0)
  uint32_t *counts;   // [B Hs nkt] entries of each key tile
  uint32_t *bits;     // [B Hs nkt][nqw]
  uint32_t *head;     // number of items
  uint32_t *lens;     // [B Hs nqt] blocks of each query tile
  uint32_t *lmask;    // [B Hs nqt][cap] query masks of its blocks
  uint16_t *lblk;     // [B Hs nqt][cap] the blocks, ascending
  uint32_t *offs;     // [B Hs nkt] first entry
  uint32_t *slot0;    // [B Hs nkt] first partial slot (chunks > 1)
  uint32_t *chunks;   // [B Hs nkt]
  uint2 *item;        // (key tile of all, chunk)
  uint32_t *chunk_len;
  uint32_t *eq;       // [entries] query tile
  uint32_t *em;       // [entries][bpt] query masks of the tile's blocks
  float *part;        // [slots][rep][2][128][D]
  size_t bytes;       // of the workspace
  size_t zero_bytes;  // from counts on: cleared by the call
};

int make_plan(const BlockAttn &p, char *ws, BwdPlan *pl) {
  pl->qt = tile_queries(p.G, kRowTile);
  if (pl->qt > p.S) pl->qt = p.S;
  pl->nqt = (p.S + pl->qt - 1) / pl->qt;
  pl->nkt = (int)(((long long)p.T + kKeyTile - 1) / kKeyTile);
  pl->nqw = (pl->nqt + 31) / 32;
  pl->bpt = kKeyTile / p.blk;
  const long long most = (long long)pl->qt * (p.topk + p.local);
  pl->cap = (int)(most < p.nblk ? most : p.nblk);
  pl->rep = p.Hk / p.sel_heads;
  const long long bh = (long long)p.B * p.sel_heads;
  const long long kts = bh * pl->nkt, qts = bh * pl->nqt;
  pl->entries = qts * (pl->nkt < pl->cap ? pl->nkt : pl->cap);
  // (the last two: grids of the marking, the dk, dv pass and its join)
  if (pl->entries >= (1ll << 31) || kts >= (1ll << 20) ||
      qts * pl->cap >= (1ll << 40) ||
      (long long)p.B * p.H * (kFewKeys / 4) + qts >= (1ll << 31) ||
      (kts + kChunkUnits) * pl->rep * kJoinParts >= (1ll << 31))
    return DSA_ERR_UNSUPPORTED;
  pl->items = (int)(kts + kChunkUnits / pl->rep + 1);
  // only lists longer than a chunk have slots: at most twice entries / chunk
  long long slots = 2 * (kChunkUnits / pl->rep) + 2;
  if (slots > pl->entries / (kMinChunk / 2) + 1)
    slots = pl->entries / (kMinChunk / 2) + 1;
  pl->slots = (int)slots;
  size_t at = 256;
  auto take = [&](size_t n) {
    char *r = ws + at;
    at = (at + n + 255) & ~(size_t)255;
    return r;
  };
  const size_t z0 = at;
  pl->counts = reinterpret_cast<uint32_t *>(take(kts * 4));
  pl->bits = reinterpret_cast<uint32_t *>(take(kts * pl->nqw * 4));
  pl->zero_bytes = at - z0;
  pl->head = reinterpret_cast<uint32_t *>(take(4));
  pl->chunk_len = reinterpret_cast<uint32_t *>(take(4));
  pl->stat = reinterpret_cast<float2 *>(take((size_t)p.S * p.B * p.H * 8));
  pl->lens = reinterpret_cast<uint32_t *>(take(qts * 4));
  pl->lmask = reinterpret_cast<uint32_t *>(take((size_t)qts * pl->cap * 4));
  pl->lblk = reinterpret_cast<uint16_t *>(take((size_t)qts * pl->cap * 2));
  pl->offs = reinterpret_cast<uint32_t *>(take(kts * 4));
  pl->slot0 = reinterpret_cast<uint32_t *>(take(kts * 4));
  pl->chunks = reinterpret_cast<uint32_t *>(take(kts * 4));
  pl->item = reinterpret_cast<uint2 *>(take((size_t)pl->items * 8));
  pl->eq = reinterpret_cast<uint32_t *>(take((size_t)pl->entries * 4));
  pl->em = reinterpret_cast<uint32_t *>(
      take((size_t)pl->entries * pl->bpt * 4));
  pl->part = reinterpret_cast<float *>(
      take((size_t)pl->slots * pl->rep * 2 * kKeyTile * p.D * 4));
  pl->bytes = at;
  return DSA_OK;
}

// ---- delta --------------------------------------------------------------------

// stat = (lse log2 e, do.o); D / 8 lanes a row, 16 bytes each, kDeltaRows
// rows in flight.  Bound by memory: 6.5 TB/s at 4096 x 64 rows of 128 (21 us).
// A row without keys gets +inf, so its weights exp2(x - inf) are zero.
constexpr int kDeltaRows = 4;
template <int D>
__global__ void __launch_bounds__(256)
    bwd_delta_kernel(const __nv_bfloat16 *o, const __nv_bfloat16 *go,
                     const float *lse, long long rows, float2 *stat) {
  constexpr int L = D / 8, kPer = 256 / L;  // lanes of a row, rows of a pass
  const int sub = threadIdx.x / L, lane = threadIdx.x % L;
  const long long r0 = (long long)blockIdx.x * kPer * kDeltaRows + sub;
  uint4 a[kDeltaRows], g[kDeltaRows];
  float l[kDeltaRows];
#pragma unroll
  for (int i = 0; i < kDeltaRows; ++i) {
    const long long r = r0 + i * kPer;
    a[i] = g[i] = make_uint4(0u, 0u, 0u, 0u);
    l[i] = 0.f;
    if (r < rows) {
      a[i] = __ldg(reinterpret_cast<const uint4 *>(o + r * D) + lane);
      g[i] = __ldg(reinterpret_cast<const uint4 *>(go + r * D) + lane);
      if (lane == 0) l[i] = __ldg(lse + r);
    }
  }
#pragma unroll
  for (int i = 0; i < kDeltaRows; ++i) {
    const uint32_t x[4] = {a[i].x, a[i].y, a[i].z, a[i].w};
    const uint32_t y[4] = {g[i].x, g[i].y, g[i].z, g[i].w};
    float t = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      t = fmaf(__uint_as_float(x[e] << 16), __uint_as_float(y[e] << 16), t);
      t = fmaf(__uint_as_float(x[e] & 0xffff0000u),
               __uint_as_float(y[e] & 0xffff0000u), t);
    }
#pragma unroll
    for (int m = L / 2; m; m >>= 1) t += __shfl_xor_sync(0xffffffffu, t, m);
    const long long r = r0 + i * kPer;
    if (lane == 0 && r < rows) {
      const float inf = __int_as_float(0x7f800000);
      stat[r] = l[i] == -inf
                    ? make_float2(inf, 0.f)
                    : make_float2(l[i] * 1.4426950408889634f, t);
    }
  }
}

// delta of a row at one of a sequence's first kFewKeys positions, by one warp,
// as sum P dP instead of do.o, whose o has been rounded.  Rows of two or three
// keys have a dS that is small against dP more often than others do: dq of
// sequences below 8 tokens is 0.32% off at worst without, 0.24% with it, for
// 4 us in the launch of bwd_mark_kernel.  The rule is the position, which needs
// no look at the selection; later rows with as few keys stay at 0.32%.
__device__ __forceinline__ void few_keys_delta(const BlockAttn &p,
                                               const __nv_bfloat16 *go,
                                               float2 *stat, int b, int h,
                                               int pos, int lane) {
  const long long s = p.q_pos ? (long long)pos - __ldg(p.q_pos + b) : pos;
  if (s < 0 || s >= p.S) return;
  const int hk = h / p.G;
  const int32_t *ids = row_ids(p, b, (int)s, hk);
  unsigned held = 0u;  // blocks of 16 or more keys: two at most
  bool bad = false;
  for (int i = lane; i < p.topk + p.local; i += 32) {
    const int n = candidate(p, ids, pos, i, bad);
    if (n >= 0) held |= 1u << n;
  }
  held = __reduce_or_sync(0xffffffffu, held);
  const size_t row = ((size_t)s * p.B + b) * p.H + h;
  const float lse = stat[row].x;
  const int n = (int)min((long long)pos + 1, (long long)p.T);
  // eight lanes a key, each 8 values of every 64: four keys a step
  const int sub = lane >> 3, l8 = lane & 7;
  auto piece = [&](const __nv_bfloat16 *at, int c) {
    return c * 64 < p.D ? __ldg(reinterpret_cast<const uint4 *>(at) + c * 8 +
                                l8)
                        : make_uint4(0u, 0u, 0u, 0u);
  };
  auto dot = [](const uint4 &u, const uint4 &w, float t) {
    const uint32_t x[4] = {u.x, u.y, u.z, u.w}, y[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t = fmaf(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16), t);
      t = fmaf(__uint_as_float(x[i] & 0xffff0000u),
               __uint_as_float(y[i] & 0xffff0000u), t);
    }
    return t;
  };
  uint4 q[2], g[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    q[c] = piece(p.q + row * p.D, c);
    g[c] = piece(go + row * p.D, c);
  }
  float sum = 0.f;
#pragma unroll 2
  for (int j0 = 0; j0 < n; j0 += 4) {
    const int j = j0 + sub;
    const bool has = j < n && (held >> (j >> p.lb) & 1u);
    const long long at = min(j, n - 1);  // (does not wait for the blocks)
    const __nv_bfloat16 *kr = p.k + b * p.k_sb + at * p.k_st + hk * p.k_sh;
    const __nv_bfloat16 *vr = p.v + b * p.v_sb + at * p.v_st + hk * p.v_sh;
    float x = 0.f, dp = 0.f;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      x = dot(q[c], piece(kr, c), x);
      dp = dot(g[c], piece(vr, c), dp);
    }
#pragma unroll
    for (int m = 4; m; m >>= 1) {
      x += __shfl_xor_sync(0xffffffffu, x, m);
      dp += __shfl_xor_sync(0xffffffffu, dp, m);
    }
    if (has)
      sum = fmaf(exp2f(x * p.scale * 1.4426950408889634f - lse), dp, sum);
  }
  sum += __shfl_xor_sync(0xffffffffu, sum, 8);
  sum += __shfl_xor_sync(0xffffffffu, sum, 16);
  // (a row without keys keeps its zero)
  if (lane == 0 && lse != __int_as_float(0x7f800000)) stat[row].y = sum;
}

// ---- the transposed selection ---------------------------------------------------

// Three short launches (15, 7 and 11 us at 4096 tokens of 64 heads): the
// order of a list must not depend on who comes first, so the filling waits for
// all counts.  (The scan needs the counts only and could be the work of the
// marking's last CTA; that has not been tried.)
// A CTA lists the blocks of one query tile and marks its key tiles.  The first
// `few` CTAs take four positions of one head each (few_keys_delta) instead.
__global__ void __launch_bounds__(128)
    bwd_mark_kernel(const BlockAttn p, const __nv_bfloat16 *go,
                    const BwdPlan pl, unsigned few) {
  if (blockIdx.x < few) {
    constexpr int kCtas = kFewKeys / 4;
    const int bh = blockIdx.x / kCtas;
    few_keys_delta(p, go, pl.stat, bh / p.H, bh % p.H,
                   blockIdx.x % kCtas * 4 + (threadIdx.x >> 5),
                   threadIdx.x & 31);
    return;
  }
  extern __shared__ uint32_t words[];
  uint16_t *list = reinterpret_cast<uint16_t *>(words + p.nblk);
  __shared__ int sCount;
  const int tid = threadIdx.x, lane = tid & 31;
  const long long it = blockIdx.x - few;
  const int tile = (int)(it % pl.nqt);
  const long long bh = it / pl.nqt;
  const int b = (int)(bh / p.sel_heads), hs = (int)(bh % p.sel_heads);
  const int s0 = tile * pl.qt, nq = min(pl.qt, p.S - s0);
  const FirstMark first = first_mark(p, b, s0, nq, hs, tid);
  for (int n = tid; n < p.nblk; n += 128) words[n] = 0u;
  __syncthreads();
  mark_blocks(p, b, s0, nq, hs, words, tid, 128, first);
  __syncthreads();
  if (tid < 32) {
    const int n = list_blocks(words, p.nblk, list, lane);
    if (lane == 0) sCount = n;
  }
  __syncthreads();
  const int count = sCount;
  if (tid == 0) pl.lens[it] = (uint32_t)count;
  for (int i = tid; i < count; i += 128) {
    const int n = list[i];
    pl.lblk[(size_t)it * pl.cap + i] = (uint16_t)n;
    pl.lmask[(size_t)it * pl.cap + i] = words[i];
    const int kt = n / pl.bpt;
    if (i == 0 || list[i - 1] / pl.bpt != kt) {
      const long long k = bh * pl.nkt + kt;
      atomicOr(pl.bits + k * pl.nqw + (tile >> 5), 1u << (tile & 31));
      atomicAdd(pl.counts + k, 1u);
    }
  }
}

// Exclusive sum of x over the 1024 threads of the CTA, and the total.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t *sums,
                                               uint32_t &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t inc = x;
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  uint32_t before = 0;
  total = 0;
  for (int w = 0; w < 32; ++w) {
    const uint32_t v = sums[w];
    if (w < warp) before += v;
    total += v;
  }
  return before + inc - x;
}

// Offsets of the lists, and the items: chunks of each list (a list without
// entries is one chunk, which writes zeros).  One CTA.
__global__ void __launch_bounds__(1024)
    bwd_scan_kernel(const BwdPlan pl, int kts) {
  __shared__ uint32_t sums[32];
  const int per = (kts + 1023) / 1024;
  const int k0 = min(kts, (int)threadIdx.x * per), k1 = min(kts, k0 + per);
  uint32_t n = 0, total;
  for (int k = k0; k < k1; ++k) n += pl.counts[k];
  uint32_t off = block_scan(n, sums, total);
  const unsigned long long share =
      ((unsigned long long)total * pl.rep + kChunkUnits - 1) / kChunkUnits;
  const uint32_t len = share > kMinChunk ? (uint32_t)share : kMinChunk;
  // whole chunks come first, the lists' ends and the empty lists after them:
  // CTAs start in this order, and the short ones fill the last round
  uint32_t whole = 0, rest = 0, slots = 0, unused, wholes, rests;
  for (int k = k0; k < k1; ++k) {
    const uint32_t c = pl.counts[k];
    const uint32_t ch = c == 0 ? 1u : (c + len - 1) / len;
    whole += c / len;
    rest += ch - c / len;
    slots += ch > 1 ? ch : 0u;
  }
  uint32_t item = block_scan(whole, sums, wholes);
  uint32_t end = block_scan(rest, sums, rests) + wholes;
  if (threadIdx.x == 0) {
    *pl.head = wholes + rests;
    *pl.chunk_len = len;
  }
  uint32_t slot = block_scan(slots, sums, unused);
  for (int k = k0; k < k1; ++k) {
    const uint32_t c = pl.counts[k];
    const uint32_t ch = c == 0 ? 1u : (c + len - 1) / len;
    pl.offs[k] = off;
    pl.chunks[k] = ch;
    pl.slot0[k] = slot;
    for (uint32_t i = 0; i < ch; ++i) {
      uint2 *to = pl.item + (i < c / len ? item++ : end++);
      *to = make_uint2(k, i);
    }
    off += c;
    slot += ch > 1 ? ch : 0u;
  }
}

// The entries of one key tile, in the order of the query tiles.
__global__ void __launch_bounds__(1024)
    bwd_fill_kernel(const BlockAttn p, const BwdPlan pl) {
  __shared__ uint32_t sums[32];
  const long long k = blockIdx.x;
  const int kt = (int)(k % pl.nkt);
  const long long bh = k / pl.nkt;
  const uint32_t off = pl.offs[k], count = pl.counts[k];
  if (count == 0) return;
  uint32_t done = 0;
  for (int w0 = 0; w0 < pl.nqw; w0 += 1024) {
    const int w = w0 + threadIdx.x;
    uint32_t m = w < pl.nqw ? pl.bits[k * pl.nqw + w] : 0u;
    uint32_t total;
    uint32_t at = off + done + block_scan(__popc(m), sums, total);
    for (; m; m &= m - 1) pl.eq[at++] = w * 32 + __ffs(m) - 1;
    done += total;
  }
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < count; i += 1024) {
    const size_t it = (size_t)bh * pl.nqt + pl.eq[off + i];
    const uint16_t *blk = pl.lblk + it * pl.cap;
    // first of the tile's blocks that is in this key tile
    int lo = 0, hi = (int)pl.lens[it];
    const int first = kt * pl.bpt, last = first + pl.bpt, n = hi;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (blk[mid] < first) lo = mid + 1;
      else hi = mid;
    }
    uint32_t *em = pl.em + (size_t)(off + i) * pl.bpt;
    for (int x = 0; x < pl.bpt; ++x) em[x] = 0u;
    for (; lo < n && blk[lo] < last; ++lo)
      em[blk[lo] - first] = pl.lmask[it * pl.cap + lo];
  }
}

// Steps in tensor memory, and CTAs an SM.
constexpr int bwd_bufs(int D) { return D == 64 ? 1 : 2; }
constexpr int bwd_ctas(int D) { return D == 64 ? 2 : 1; }

// ---- dk, dv ---------------------------------------------------------------------

template <int D>
struct KvSmem {
  static constexpr int kCh = D / 64;
  static constexpr int kTile = kCh * kKeyTile * 128;  // K or V
  static constexpr int kRow = kCh * kRowTile * 128;   // Q or dO of a stage
  static constexpr int kOffK = 0;
  static constexpr int kOffV = kTile;
  static constexpr int kOffS = 2 * kTile;  // stages: Q, dO
  static constexpr int kOffStat = kOffS + kKvStages * 2 * kRow;
  // a stage's log-sums for each block of the key tile, delta, query masks,
  // and the first query's position
  static constexpr int kStat = (8 + 1) * kRowTile * 4 + 64;
  static constexpr int kOffBar = kOffStat + kKvStages * kStat;
  // kv_full acc_full sdp_full[2] ds_full[2] st_full[] st_empty[]
  static constexpr int kOffMisc = kOffBar + (6 + 2 * kKvStages) * 8;
  static constexpr int kBytes = kOffMisc + 32 + 1024;
};

template <int D>
__global__ void __launch_bounds__(kBwdThreads, bwd_ctas(D))
    block_attn_dkv_kernel(const __grid_constant__ CUtensorMap tm_q,
                          const __grid_constant__ CUtensorMap tm_go,
                          const __grid_constant__ KvMaps maps,
                          const BlockAttn p, const BwdPlan pl,
                          __nv_bfloat16 *gk, __nv_bfloat16 *gv) {
  using L = KvSmem<D>;
  constexpr int CH = L::kCh;
  constexpr uint32_t kIdescS = idesc_bf16_f32(kKeyTile, kRowTile);
  constexpr uint32_t kIdescA = idesc_bf16_f32_mn(kKeyTile, D, false, true);
  constexpr int NB = bwd_bufs(D);
  constexpr uint32_t kTmK = 0, kTmV = D, kTmBuf = 2 * D;  // + 128 a step
  constexpr uint32_t kTmCols = 2 * D + NB * 128;

  if (blockIdx.x / pl.rep >= *pl.head) return;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (base - raw_addr);
  const uint32_t sK = base + L::kOffK, sV = base + L::kOffV;
  auto sQ = [&](int st) { return base + L::kOffS + st * 2 * L::kRow; };
  auto sG = [&](int st) { return sQ(st) + L::kRow; };
  // offsets of K step ks in the tiles of keys and of rows
  auto koff = [](int ks) {
    return (uint32_t)((ks >> 2) * (kKeyTile * 128) + (ks & 3) * 32) >> 4;
  };
  auto roff = [](int ks) {
    return (uint32_t)((ks >> 2) * (kRowTile * 128) + (ks & 3) * 32) >> 4;
  };
  auto stat = [&](int st) {
    return reinterpret_cast<float *>(smem + L::kOffStat + st * L::kStat);
  };
  const uint32_t bars = base + L::kOffBar;
  const uint32_t kv_full = bars, acc_full = bars + 8;
  auto sdp_full = [&](int i) { return bars + 16 + 8 * i; };
  auto ds_full = [&](int i) { return bars + 32 + 8 * i; };
  auto st_full = [&](int i) { return bars + 48 + 8 * i; };
  auto st_empty = [&](int i) { return bars + 48 + 8 * (kKvStages + i); };
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + L::kOffMisc);
  volatile int *abort_flag = reinterpret_cast<int *>(smem + L::kOffMisc + 4);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint2 item = pl.item[blockIdx.x / pl.rep];
  const int k = (int)item.x;
  const int kt = k % pl.nkt, bh = k / pl.nkt;
  const int b = bh / p.sel_heads;
  const int hk = bh % p.sel_heads * pl.rep + blockIdx.x % pl.rep;
  const uint32_t count = pl.counts[k], len = *pl.chunk_len;
  const uint32_t e0 = pl.offs[k] + item.y * len;
  const int n = (int)min(len, count - item.y * len);  // entries of this item

  if (tid == 0) {
    mbar_init(kv_full, 1);
    mbar_init(acc_full, 1);
    for (int i = 0; i < kKvStages; ++i) {
      mbar_init(st_full(i), 33);
      mbar_init(st_empty(i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sdp_full(i), 1);
      mbar_init(ds_full(i), 8);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_go);
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(tmem_holder), kTmCols);
    tmem_relinquish();
  }
  // rows past the query tile's are never loaded, but read as operands (times
  // zero): they must be numbers
  if (pl.qt * p.G < kRowTile) {
    for (int i = tid; i < kKvStages * 2 * L::kRow / 16; i += kBwdThreads) {
      const uint32_t z[4] = {0u, 0u, 0u, 0u};
      st_shared_v4(base + L::kOffS + i * 16, z);
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0);

  if (warp == kTmaWarp) {
    if (n > 0 && lane == 0) {
      mbar_arrive_expect_tx(kv_full, 2 * L::kTile);
      for (int c = 0; c < CH; ++c) {
        tma_load_4d(sK + c * (kKeyTile * 128), &maps.k, kv_full, c * kChunk,
                    kt * kKeyTile, hk * maps.bc_kh, b * maps.bc_ks);
        tma_load_4d(sV + c * (kKeyTile * 128), &maps.v, kv_full, c * kChunk,
                    kt * kKeyTile, hk * maps.bc_vh, b * maps.bc_vs);
      }
    }
    const float inf = __int_as_float(0x7f800000);
    const long long q0 = row_pos(p.q_pos, b, 0);
    const int qr[2] = {lane / p.G, (lane + 32) / p.G};  // queries of two rows
    const int hr[2] = {lane % p.G, (lane + 32) % p.G};
    // What a step needs from memory is asked for one step before, and the
    // query tile's number two before.
    float2 v[2], v1[2];
    uint32_t m, m1;
    auto ask = [&](int i, int tile, float2(&to)[2], uint32_t &tm) {
      const int s0 = tile * pl.qt, nq = min(pl.qt, p.S - s0);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        to[u] = make_float2(inf, 0.f);
        if (i < n && qr[u] < nq)
          to[u] = __ldg(pl.stat + ((size_t)(s0 + qr[u]) * p.B + b) * p.H +
                        hk * p.G + hr[u]);
      }
      tm = i < n && lane < pl.bpt
               ? __ldg(pl.em + (size_t)(e0 + i) * pl.bpt + lane)
               : 0u;
    };
    int tile0 = n > 0 ? (int)__ldg(pl.eq + e0) : 0;
    int tile1 = n > 1 ? (int)__ldg(pl.eq + e0 + 1) : 0;
    ask(0, tile0, v1, m1);
    int st = 0;
    uint32_t ph = 0;
    for (int i = 0; i < n; ++i) {
      const int s0 = tile0 * pl.qt;
      const int nq = min(pl.qt, p.S - s0);
      v[0] = v1[0], v[1] = v1[1], m = m1;
      ask(i + 1, tile1, v1, m1);
      tile0 = tile1;
      tile1 = i + 2 < n ? (int)__ldg(pl.eq + e0 + i + 2) : 0;
      if (!__all_sync(0xffffffffu, wait_bar_rest(st_empty(st), ph ^ 1u,
                                                 abort_flag, p.status)))
        goto done;
      float *sst = stat(st);
      for (int x = 0; x < pl.bpt; ++x) {
        const uint32_t mx = __shfl_sync(0xffffffffu, m, x);
#pragma unroll
        for (int u = 0; u < 2; ++u)
          sst[x * kRowTile + lane + 32 * u] =
              qr[u] < nq && (mx >> qr[u] & 1u) ? v[u].x : inf;
      }
      sst[8 * kRowTile + lane] = v[0].y;
      sst[8 * kRowTile + lane + 32] = v[1].y;
      uint32_t *meta = reinterpret_cast<uint32_t *>(sst + 9 * kRowTile);
      if (lane < 8) meta[lane] = m;
      if (lane == 8)
        *reinterpret_cast<long long *>(meta + 8) = q0 + s0;
      mbar_arrive(st_full(st));
      if (lane == 0) {
        mbar_arrive_expect_tx(st_full(st), 2 * CH * pl.qt * p.G * 128);
        for (int c = 0; c < CH; ++c) {
          tma_load_4d(sQ(st) + c * (kRowTile * 128), &tm_q, st_full(st),
                      c * kChunk, hk * p.G, b, s0);
          tma_load_4d(sG(st) + c * (kRowTile * 128), &tm_go, st_full(st),
                      c * kChunk, hk * p.G, b, s0);
        }
      }
      __syncwarp();
      if (++st == kKvStages) st = 0, ph ^= 1;
    }
  } else if (warp == kMmaWarp) {
    if (elect_one()) {
      auto wait = [&](uint32_t bar, uint32_t ph) -> bool {
        return wait_bar_rest(bar, ph, abort_flag, p.status);
      };
      const uint64_t kd = sdesc_k_sw128(sK), vd = sdesc_k_sw128(sV);
      bool ok = n <= 0 || wait(kv_full, 0);
      int st = 0, done = 0;  // stages of the step begun and of the one before
      uint32_t ph = 0, acc = 0;
      for (int i = 0; ok && i < n + NB - 1; ++i) {
        if (i < n) {
          if (!(ok = wait(st_full(st), ph))) break;
          tc_fence_after();
          const uint64_t qd = sdesc_k_sw128(sQ(st)),
                         gd = sdesc_k_sw128(sG(st));
          const uint32_t d = tmem + kTmBuf + i % NB * 128;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            mma_bf16(d, kd + koff(ks), qd + roff(ks), kIdescS, ks != 0);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            mma_bf16(d + 64, vd + koff(ks), gd + roff(ks), kIdescS, ks != 0);
          mma_commit(sdp_full(i % NB));
          if (++st == kKvStages) st = 0, ph ^= 1;
        }
        if (i >= NB - 1) {
          const int j = i - (NB - 1), b1 = j % NB;
          if (!(ok = wait(ds_full(b1), j / NB & 1u))) break;
          tc_fence_after();
          const uint64_t qm = sdesc_mn_sw128(sQ(done), kRowTile * 128, 1024);
          const uint64_t gm = sdesc_mn_sw128(sG(done), kRowTile * 128, 1024);
          const uint32_t a = tmem + kTmBuf + b1 * 128;
          // each warpgroup's 32 rows are 16 columns at its half's start
#pragma unroll
          for (int ks = 0; ks < kRowTile / 16; ++ks)
            mma_bf16_ta(tmem + kTmV, a + (ks >> 1) * 32 + (ks & 1) * 8,
                        gm + ((ks * 2048) >> 4), kIdescA, ks == 0 ? acc : 1u);
#pragma unroll
          for (int ks = 0; ks < kRowTile / 16; ++ks)
            mma_bf16_ta(tmem + kTmK, a + 64 + (ks >> 1) * 32 + (ks & 1) * 8,
                        qm + ((ks * 2048) >> 4), kIdescA, ks == 0 ? acc : 1u);
          mma_commit(st_empty(done));
          if (j + 1 == n) mma_commit(acc_full);
          acc = 1;
          if (++done == kKvStages) done = 0;
        }
      }
    }
    __syncwarp();
  } else {
    // ---------- one key a thread; a warpgroup takes 32 of the rows ----------
    const int wg = warp >> 2;
    const int key = (warp & 3) * 32 + lane;
    const long long j = (long long)kt * kKeyTile + key;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const float c2 = p.scale * 1.4426950408889634f;
    const int kb = key / p.blk;  // this key's block
    const long long last = (long long)kt * kKeyTile + kKeyTile - 1;
    for (int i = 0; i < n; ++i) {
      const int st = i % kKvStages;
      if (!__all_sync(0xffffffffu,
                      wait_bar_rest(sdp_full(i % NB), i / NB & 1u, abort_flag,
                                   p.status) &&
                          wait_bar_rest(st_full(st), (i / kKvStages) & 1u,
                                       abort_flag, p.status)))
        goto done;
      tc_fence_after();
      const uint32_t ts = tmem + kTmBuf + i % NB * 128 + wg * 32 + lane_off;
      uint32_t u[32], g[32];
      __syncwarp();
      tmem_ld32(ts, u);
      tmem_ld32(ts + 64, g);
      const float *sst = stat(st);
      const float4 *sl = reinterpret_cast<const float4 *>(
          sst + kb * kRowTile + wg * 32);
      const float4 *sd = reinterpret_cast<const float4 *>(
          sst + 8 * kRowTile + wg * 32);
      const uint32_t *meta =
          reinterpret_cast<const uint32_t *>(sst + 9 * kRowTile);
      const long long pos0 = *reinterpret_cast<const long long *>(meta + 8);
      tmem_ld_wait();
      reg_fence32(u);
      reg_fence32(g);
      if (last > pos0) {  // keys after some query: row by row
        uint32_t qm = meta[kb];
        const long long late = j - pos0;
        if (late > 0) qm = late >= 32 ? 0u : qm & (~0u << (int)late);
        if (j >= p.T) qm = 0u;
        int q = wg * 32 / p.G, h = wg * 32 % p.G;
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          if (q >= 32 || !(qm >> q & 1u)) u[x] = 0xff800000u;
          if (++h == p.G) h = 0, ++q;
        }
      }
      uint32_t pk[16], dk[16];
#pragma unroll
      for (int x = 0; x < 32; x += 4) {
        const float4 l4 = sl[x >> 2], d4 = sd[x >> 2];
#pragma unroll
        for (int y = 0; y < 4; y += 2) {
          const float2 l = y ? make_float2(l4.z, l4.w)
                             : make_float2(l4.x, l4.y);
          const float2 d = y ? make_float2(d4.z, d4.w)
                             : make_float2(d4.x, d4.y);
          float2 e = __ffma2_rn(
              make_float2(__uint_as_float(u[x + y]),
                          __uint_as_float(u[x + y + 1])),
              make_float2(c2, c2), make_float2(-l.x, -l.y));
          e.x = ex2(e.x);
          e.y = ex2(e.y);
          pk[(x + y) >> 1] = pack_bf16x2(e.x, e.y);
          const float2 w = __fmul2_rn(
              e, __fadd2_rn(make_float2(__uint_as_float(g[x + y]),
                                        __uint_as_float(g[x + y + 1])),
                            make_float2(-d.x, -d.y)));
          dk[(x + y) >> 1] = pack_bf16x2(w.x, w.y);
        }
      }
      __syncwarp();
      tmem_st16(ts, pk);
      tmem_st16(ts + 64, dk);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ds_full(i % NB));
    }
    // ---------------- dK (warpgroup 0), dV (1) ----------------
    if (n > 0) {
      if (!__all_sync(0xffffffffu,
                      wait_bar_rest(acc_full, 0, abort_flag, p.status)))
        goto done;
      tc_fence_after();
    }
    const float f = wg == 0 ? p.scale : 1.f;
    const bool direct = pl.chunks[k] == 1;
    float *part =
        pl.part + ((((size_t)pl.slot0[k] + item.y) * pl.rep +
                    blockIdx.x % pl.rep) * 2 + wg) * kKeyTile * D +
        (size_t)key * D;
    __nv_bfloat16 *out =
        (wg == 0 ? gk : gv) + (((size_t)j * p.B + b) * p.Hk + hk) * D;
    // K's and V's space is free for the way out
    const uint32_t out_buf = (wg == 0 ? sK : sV) + (warp & 3) * 4096;
    const bool inside = j < p.T;
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      uint32_t u[32];
      if (n > 0) {
        __syncwarp();
        tmem_ld32(tmem + (wg == 0 ? kTmK : kTmV) + lane_off + c * 32, u);
        tmem_ld_wait();
        reg_fence32(u);
      }
#pragma unroll
      for (int x = 0; x < 32; ++x)
        u[x] = n > 0 ? __float_as_uint(__uint_as_float(u[x]) * f) : 0u;
      if (!direct) {
        store_rows<32>(out_buf, u, part + c * 32, lane);
      } else {
        uint32_t w[16];
#pragma unroll
        for (int x = 0; x < 16; ++x)
          w[x] = pack_bf16x2(__uint_as_float(u[2 * x]),
                             __uint_as_float(u[2 * x + 1]));
        store_rows<16>(out_buf, w, inside ? out + c * 32 : nullptr, lane);
      }
    }
  }
done:
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmCols);
  }
}

// Adds the chunks of the key tiles that have several; kJoinParts CTAs a tile.
// Bound by memory and, where one tile has most of the chunks (a block that
// every query holds), by that tile's CTAs: 20 us for 90 MB.
template <int D>
__global__ void __launch_bounds__(256)
    bwd_join_kernel(const BlockAttn p, const BwdPlan pl, __nv_bfloat16 *gk,
                    __nv_bfloat16 *gv) {
  const int kr = blockIdx.x / kJoinParts;
  const int k = kr / pl.rep, r = kr % pl.rep;
  const uint32_t ch = pl.chunks[k];
  if (ch <= 1) return;
  const int kt = k % pl.nkt, bh = k / pl.nkt;
  const int b = bh / p.sel_heads, hk = bh % p.sel_heads * pl.rep + r;
  const size_t stride = (size_t)pl.rep * 2 * kKeyTile * D;
  const float *part = pl.part + ((size_t)pl.slot0[k] * pl.rep + r) * 2 *
                                    kKeyTile * D;
  constexpr int kPart = 2 * kKeyTile * D / 4 / kJoinParts;
  for (int x = threadIdx.x; x < kPart; x += 256) {
    const int e = (blockIdx.x % kJoinParts * kPart + x) * 4;
    const int which = e / (kKeyTile * D), key = e / D % kKeyTile, d = e % D;
    const long long j = (long long)kt * kKeyTile + key;
    if (j >= p.T) continue;
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (uint32_t c = 0; c < ch; ++c) {
      const float4 v =
          *reinterpret_cast<const float4 *>(part + c * stride + e);
      t.x += v.x, t.y += v.y, t.z += v.z, t.w += v.w;
    }
    uint2 o = make_uint2(pack_bf16x2(t.x, t.y), pack_bf16x2(t.z, t.w));
    *reinterpret_cast<uint2 *>((which ? gv : gk) +
                               (((size_t)j * p.B + b) * p.Hk + hk) * D + d) =
        o;
  }
}

// ---- dq ---------------------------------------------------------------------------

constexpr int kDqRows = 128, kDqKeys = 64;

constexpr int kDqStages = 6;
template <int D>
struct DqSmem {
  static constexpr int kCh = D / 64;
  static constexpr int kKey = kCh * kDqKeys * 128;  // K or V of a stage
  static constexpr int kOffBar = 0;
  // q_full acc_full sdp_full[2] ds_full[2] kv_full[] kv_empty[] q_here met
  static constexpr int kOffMisc = kOffBar + (8 + 2 * kDqStages) * 8;
  // a row's sum of dS by each warpgroup, its key with most weight and that
  // key's rounding
  static constexpr int kOffLeft = 512;
  static constexpr int kOffTop = kOffLeft + 2 * kDqRows * 4;
  // stages: K, V
  static constexpr int kOffS = (kOffTop + kDqRows * 8 + 1023) / 1024 * 1024;
  static_assert(kOffMisc + 32 <= kOffLeft);
  static int bytes(int stages, int nblk, int cap) {
    return kOffS + stages * 2 * kKey + nblk * 4 + ((cap * 2 + 15) & ~15) +
           1024;
  }
};

struct DqPlan {
  int qt, tiles, cap, stages;
  float2 *stat;
  __nv_bfloat16 *gq;
};

// The one of a thread's 32 keys that has more than half of its row's weight (its
// column, or -1), and what rounding this key's dS to bf16 adds to it.  Out of
// line: a row has one such key at most.
__device__ __noinline__ int top_key(uint32_t ts, uint32_t mask, float c2,
                                    float2 sd, float &fix) {
  uint32_t u[32];
  __syncwarp();
  tmem_ld32(ts, u);
  tmem_ld_wait();
  reg_fence32(u);
  int at = -1;
  float top = 0.f;
#pragma unroll
  for (int x = 0; x < 32; ++x) {
    const float e = ex2(fmaf(__uint_as_float(u[x]), c2, -sd.x));
    if ((mask >> x & 1u) && e > 0.5f) at = x, top = e;
  }
  tmem_ld32(ts + 64, u);
  tmem_ld_wait();
  reg_fence32(u);
  float dp = 0.f;
#pragma unroll
  for (int x = 0; x < 32; ++x) dp = x == at ? __uint_as_float(u[x]) : dp;
  const float w = top * (dp - sd.y);
  fix = __bfloat162float(__float2bfloat16(w)) - w;
  return at;
}

template <int D>
__global__ void __launch_bounds__(kBwdThreads, bwd_ctas(D))
    block_attn_dq_kernel(const __grid_constant__ CUtensorMap tm_q,
                         const __grid_constant__ CUtensorMap tm_go,
                         const __grid_constant__ KvMaps maps,
                         const BlockAttn p, const DqPlan pl) {
  using L = DqSmem<D>;
  constexpr int CH = L::kCh;
  constexpr uint32_t kIdescS = idesc_bf16_f32(kDqRows, kDqKeys);
  constexpr uint32_t kIdescA = idesc_bf16_f32_mn(kDqRows, D, false, true);
  // tensor memory: dQ, two steps' scores, Q and dO (bf16)
  constexpr int NB = bwd_bufs(D);
  constexpr uint32_t kTmQ = 0, kTmBuf = D, kTmA = D + NB * 128,
                     kTmG = kTmA + D / 2, kTmCols = kTmG + D / 2;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (base - raw_addr);
  auto sK = [&](int st) { return base + L::kOffS + st * 2 * L::kKey; };
  auto sV = [&](int st) { return sK(st) + L::kKey; };
  auto koff = [](int ks) {
    return (uint32_t)((ks >> 2) * (kDqKeys * 128) + (ks & 3) * 32) >> 4;
  };
  const uint32_t bars = base + L::kOffBar;
  const uint32_t q_full = bars, acc_full = bars + 8;
  const uint32_t q_here = bars + 48 + 16 * kDqStages, met = q_here + 8;
  auto sdp_full = [&](int i) { return bars + 16 + 8 * i; };
  auto ds_full = [&](int i) { return bars + 32 + 8 * i; };
  auto kv_full = [&](int i) { return bars + 48 + 8 * i; };
  auto kv_empty = [&](int i) { return bars + 48 + 8 * (kDqStages + i); };
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + L::kOffMisc);
  volatile int *abort_flag = reinterpret_cast<int *>(smem + L::kOffMisc + 4);
  int *sCount = reinterpret_cast<int *>(smem + L::kOffMisc + 8);
  float *lefts = reinterpret_cast<float *>(smem + L::kOffLeft);
  int2 *tops = reinterpret_cast<int2 *>(smem + L::kOffTop);
  uint32_t *words = reinterpret_cast<uint32_t *>(smem + L::kOffS +
                                                 pl.stages * 2 * L::kKey);
  uint16_t *list = reinterpret_cast<uint16_t *>(words + p.nblk);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int it = blockIdx.x;
  const int hk = it % p.Hk;
  it /= p.Hk;
  const int b = it % p.B;
  const int tile = pl.tiles - 1 - it / p.B;
  const int s0 = tile * pl.qt;
  const int nq = min(pl.qt, p.S - s0);

  // Q and dO pass through the last two stages on their way to tensor memory
  const uint32_t sQ = sK(pl.stages - 1), sG = sK(pl.stages - 2);
  if (tid == 0) {
    mbar_init(q_full, 8);
    mbar_init(q_here, 1);
    mbar_init(met, 8);
    mbar_init(acc_full, 1);
    for (int i = 0; i < kDqStages; ++i) {
      mbar_init(kv_full(i), 1);
      mbar_init(kv_empty(i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sdp_full(i), 1);
      mbar_init(ds_full(i), 8);
    }
    *abort_flag = 0;
    fence_mbar_init();
    mbar_arrive_expect_tx(q_here, 2 * CH * pl.qt * p.G * 128);
    for (int c = 0; c < CH; ++c) {
      tma_load_4d(sQ + c * (kDqRows * 128), &tm_q, q_here, c * kChunk,
                  hk * p.G, b, s0);
      tma_load_4d(sG + c * (kDqRows * 128), &tm_go, q_here, c * kChunk,
                  hk * p.G, b, s0);
    }
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(tmem_holder), kTmCols);
    tmem_relinquish();
  }
  const FirstMark first = first_mark(p, b, s0, nq, hk, tid);
  if (tid < kDqRows) tops[tid] = make_int2(-1, 0);
  for (int n = tid; n < p.nblk; n += kBwdThreads) words[n] = 0u;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  mark_blocks(p, b, s0, nq, hk, words, tid, kBwdThreads, first);
  __syncthreads();
  if (warp == 0) {
    const int n = list_blocks(words, p.nblk, list, lane);
    if (lane == 0) *sCount = n;
  }
  __syncthreads();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0);
  // a step takes units of up to 64 keys: whole blocks, or halves of 128
  const int count = *sCount;
  const int unit = min(p.blk, kDqKeys), per = p.blk / unit;
  const int upt = kDqKeys / unit;
  const int n = (count * per + upt - 1) / upt;

  if (warp == kTmaWarp) {
    int st = 0;
    uint32_t ph = 0;
    for (int i = 0; i < n; ++i) {
      if (i == pl.stages - 2 &&
          !__all_sync(0xffffffffu,
                      wait_bar_rest(q_full, 0, abort_flag, p.status)))
        goto done;
      const int ui = lane / CH, c = lane % CH;  // unit and chunk of this lane
      if (!__all_sync(0xffffffffu, wait_bar_rest(kv_empty(st), ph ^ 1u,
                                                abort_flag, p.status)))
        goto done;
      if (lane == 0)
        mbar_arrive_expect_tx(kv_full(st), 2 * kDqKeys * CH * 128);
      __syncwarp();
      if (ui < upt) {
        // a ragged step's end repeats the last unit: masked, but numbers
        const int x = min(i * upt + ui, count * per - 1);
        const int tok = list[x / per] * p.blk + x % per * unit;
        const uint32_t at = c * (kDqKeys * 128) + ui * unit * 128;
        tma_load_4d(sK(st) + at, &maps.k, kv_full(st), c * kChunk, tok,
                    hk * maps.bc_kh, b * maps.bc_ks);
        tma_load_4d(sV(st) + at, &maps.v, kv_full(st), c * kChunk, tok,
                    hk * maps.bc_vh, b * maps.bc_vs);
      }
      if (++st == pl.stages) st = 0, ph ^= 1;
    }
  } else if (warp == kMmaWarp) {
    if (elect_one()) {
      auto wait = [&](uint32_t bar, uint32_t ph) -> bool {
        return wait_bar_rest(bar, ph, abort_flag, p.status);
      };
      const uint32_t ta = tmem + kTmA, tg = tmem + kTmG;
      bool ok = wait(q_full, 0);
      tc_fence_after();
      int st = 0, done = 0;
      uint32_t ph = 0, acc = 0;
      for (int i = 0; ok && i < n + NB - 1; ++i) {
        if (i < n) {
          if (!(ok = wait(kv_full(st), ph))) break;
          tc_fence_after();
          const uint64_t kd = sdesc_k_sw128(sK(st)),
                         vd = sdesc_k_sw128(sV(st));
          const uint32_t d = tmem + kTmBuf + i % NB * 128;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            mma_bf16_ta(d, ta + ks * 8, kd + koff(ks), kIdescS, ks != 0);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            mma_bf16_ta(d + 64, tg + ks * 8, vd + koff(ks), kIdescS, ks != 0);
          mma_commit(sdp_full(i % NB));
          if (++st == pl.stages) st = 0, ph ^= 1;
        }
        if (i >= NB - 1) {
          const int j = i - (NB - 1), b1 = j % NB;
          if (!(ok = wait(ds_full(b1), j / NB & 1u))) break;
          tc_fence_after();
          const uint64_t km = sdesc_mn_sw128(sK(done), kDqKeys * 128, 1024);
          const uint32_t a = tmem + kTmBuf + b1 * 128;
          // each warpgroup's 32 keys are 16 columns at its half's start
#pragma unroll
          for (int ks = 0; ks < kDqKeys / 16; ++ks)
            mma_bf16_ta(tmem + kTmQ, a + (ks >> 1) * 32 + (ks & 1) * 8,
                        km + ((ks * 2048) >> 4), kIdescA, ks == 0 ? acc : 1u);
          mma_commit(kv_empty(done));
          if (j + 1 == n) mma_commit(acc_full);
          acc = 1;
          if (++done == pl.stages) done = 0;
        }
      }
    }
    __syncwarp();
  } else {
    // ---------- one row a thread; a warpgroup takes 32 of the keys ----------
    const int wg = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const int qi = row / p.G;
    const bool live = qi < nq;
    const int s = s0 + (live ? qi : 0);
    const int pos = live ? key_pos(p, b, s) : -1;
    const int pos_lo = key_pos(p, b, s0);
    const size_t at = ((size_t)s * p.B + b) * p.H + hk * p.G + row % p.G;
    const float inf = __int_as_float(0x7f800000);
    const float2 sd = live ? pl.stat[at] : make_float2(inf, 0.f);
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const float c2 = p.scale * 1.4426950408889634f;
    // Q (warpgroup 0) and dO (1) into tensor memory, each thread its row
    if (!__all_sync(0xffffffffu,
                    wait_bar_rest(q_here, 0, abort_flag, p.status)))
      goto done;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      uint32_t w[32];
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const float4 v =
            ld_shared_v4f((wg == 0 ? sQ : sG) + c * (kDqRows * 128) +
                          row * 128 + ((x ^ (row & 7)) << 4));
        w[4 * x] = __float_as_uint(v.x), w[4 * x + 1] = __float_as_uint(v.y);
        w[4 * x + 2] = __float_as_uint(v.z), w[4 * x + 3] = __float_as_uint(v.w);
      }
      __syncwarp();
      tmem_st32(tmem + (wg == 0 ? kTmA : kTmG) + lane_off + c * 32, w);
    }
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(q_full);
    float2 left = make_float2(0.f, 0.f);  // this thread's sum of dS
    for (int i = 0; i < n; ++i) {
      uint32_t masks[2];
      bool diag[2];
      step_masks(words, list, i, count, p.lb, qi & 31, pos, pos_lo, masks,
                 diag);
      const uint32_t mask = wg ? masks[1] : masks[0];
      const bool late = wg ? diag[1] : diag[0];
      const bool any = __any_sync(0xffffffffu, mask != 0u);
      if (!__all_sync(0xffffffffu, wait_bar_rest(sdp_full(i % NB), i / NB & 1u,
                                                abort_flag, p.status)))
        goto done;
      tc_fence_after();
      const uint32_t ts = tmem + kTmBuf + i % NB * 128 + wg * 32 + lane_off;
      uint32_t dk[16];
      if (!any) {
#pragma unroll
        for (int x = 0; x < 16; ++x) dk[x] = 0u;
      } else {
        uint32_t u[32], g[32];
        __syncwarp();
        tmem_ld32(ts, u);
        tmem_ld32(ts + 64, g);
        tmem_ld_wait();
        reg_fence32(u);
        reg_fence32(g);
        if (late) {  // keys after some row's position: one by one
#pragma unroll
          for (int x = 0; x < 32; ++x)
            u[x] = mask >> x & 1u ? u[x] : 0xff800000u;
        }
        float2 weight = make_float2(0.f, 0.f);
#pragma unroll
        for (int x = 0; x < 32; x += 2) {
          // a row holds 16 neighbouring keys or none, or they are hidden
          const float sub =
              mask & (x < 16 ? 0xffffu : 0xffff0000u) ? -sd.x : -inf;
          float2 e = __ffma2_rn(
              make_float2(__uint_as_float(u[x]), __uint_as_float(u[x + 1])),
              make_float2(c2, c2), make_float2(sub, sub));
          e.x = ex2(e.x);
          e.y = ex2(e.y);
          const float2 w = __fmul2_rn(
              e, __fadd2_rn(make_float2(__uint_as_float(g[x]),
                                        __uint_as_float(g[x + 1])),
                            make_float2(-sd.y, -sd.y)));
          dk[x >> 1] = pack_bf16x2(w.x, w.y);
          weight = __fadd2_rn(weight, e);
          left = __fadd2_rn(left, w);
        }
        if (__any_sync(0xffffffffu, weight.x + weight.y > 0.5f)) {
          float fix;
          const int x = top_key(ts, mask, c2, sd, fix);
          if (x >= 0) {
            const int col = wg * 32 + x, ux = i * upt + col / unit;
            tops[row] = make_int2(
                list[ux / per] * p.blk + ux % per * unit + col % unit,
                __float_as_int(fix));
          }
        }
      }
      __syncwarp();
      tmem_st16(ts, dk);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ds_full(i % NB));
    }
    // The sum of a row's dS is what delta is off by: delta is put right for the
    // dk, dv pass, and here the key with most of the weight takes it.
    lefts[wg * kDqRows + row] = left.x + left.y;
    __syncwarp();
    if (lane == 0) mbar_arrive(met);
    if (!__all_sync(0xffffffffu,
                    (n == 0 || wait_bar_rest(acc_full, 0, abort_flag,
                                             p.status)) &&
                        wait_bar_rest(met, 0, abort_flag, p.status)))
      goto done;
    tc_fence_after();
    const float off = lefts[row] + lefts[kDqRows + row];
    const int2 top = tops[row];
    const float back = off + __int_as_float(top.y);
    if (wg == 0 && live)
      reinterpret_cast<float *>(pl.stat + at)[1] = sd.y + off;
    const uint4 *kt = reinterpret_cast<const uint4 *>(
        p.k + b * p.k_sb + max(top.x, 0) * p.k_st + hk * p.k_sh + wg * (D / 2));
    // each warpgroup writes half of the columns; the first stage is free
    uint32_t ow[D / 4];
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      uint32_t u[32];
      if (n > 0) {
        __syncwarp();
        tmem_ld32(tmem + kTmQ + lane_off + wg * (D / 2) + c * 32, u);
        tmem_ld_wait();
        reg_fence32(u);
      }
      if (top.x >= 0) {
#pragma unroll
        for (int x = 0; x < 32; x += 8) {
          const uint4 v = __ldg(kt + (c * 32 + x) / 8);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int y = 0; y < 8; ++y)
            u[x + y] = __float_as_uint(
                fmaf(-back,
                     __uint_as_float(y & 1 ? w[y >> 1] & 0xffff0000u
                                           : w[y >> 1] << 16),
                     __uint_as_float(u[x + y])));
        }
      }
#pragma unroll
      for (int x = 0; x < 16; ++x)
        ow[c * 16 + x] =
            n > 0 ? pack_bf16x2(__uint_as_float(u[2 * x]) * p.scale,
                                __uint_as_float(u[2 * x + 1]) * p.scale)
                  : 0u;
    }
    store_rows<D / 4>(sK(0) + warp * (32 * D), ow,
                      live ? pl.gq + at * D + wg * (D / 2) : nullptr, lane);
  }
done:
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmCols);
  }
}

template <int D>
int launch_bwd(const BlockAttn &p, const BwdPlan &pl, const void *o,
               const float *lse, const void *go, void *gq, void *gk, void *gv,
               cudaStream_t st) {
  auto ok = [](cudaError_t e) { return e == cudaSuccess; };
  const long long rows = (long long)p.S * p.B * p.H;
  const int kts = p.B * p.sel_heads * pl.nkt;
  const long long qts = (long long)p.B * p.sel_heads * pl.nqt;
  auto bf = [](void *x) { return static_cast<__nv_bfloat16 *>(x); };
  if (!ok(cudaMemsetAsync(pl.counts, 0, pl.zero_bytes, st)))
    return DSA_ERR_CUDA;
  constexpr int kDelta = 256 / (D / 8) * kDeltaRows;
  bwd_delta_kernel<D><<<(unsigned)((rows + kDelta - 1) / kDelta), 256, 0,
                        st>>>(
      static_cast<const __nv_bfloat16 *>(o),
      static_cast<const __nv_bfloat16 *>(go), lse, rows, pl.stat);
  const unsigned few = p.B * p.H * (kFewKeys / 4);
  const int mark_smem = p.nblk * 4 + pl.cap * 2;
  if (!ok(allow_smem(bwd_mark_kernel, DSA_BLOCK_ATTN_MAX_BLOCKS * 6)))
    return DSA_ERR_CUDA;
  bwd_mark_kernel<<<few + (unsigned)qts, 128, mark_smem, st>>>(
      p, static_cast<const __nv_bfloat16 *>(go), pl, few);
  bwd_scan_kernel<<<1, 1024, 0, st>>>(pl, kts);
  bwd_fill_kernel<<<kts, 1024, 0, st>>>(p, pl);
  if (!ok(cudaGetLastError())) return DSA_ERR_CUDA;

  CUtensorMap tm_q, tm_go;
  KvMaps maps;
  const Problem qp{p.q, nullptr, nullptr, nullptr, p.S, p.B, p.H, p.D, 1, 1};
  const Problem gp{go, nullptr, nullptr, nullptr, p.S, p.B, p.H, p.D, 1, 1};
  // dq first: it puts delta right for dk, dv
  DqPlan dp{};
  dp.qt = tile_queries(p.G, kDqRows);
  if (dp.qt > p.S) dp.qt = p.S;
  dp.tiles = (p.S + dp.qt - 1) / dp.qt;
  const long long most = (long long)dp.qt * (p.topk + p.local);
  dp.cap = (int)(most < p.nblk ? most : p.nblk);
  dp.stat = pl.stat;
  dp.gq = bf(gq);
  // fewer stages where a very long context's block words need the room
  dp.stages = kDqStages;
  while (dp.stages > 2 && DqSmem<D>::bytes(dp.stages, p.nblk, dp.cap) >
                              kMaxSmem / bwd_ctas(D) - 1024)
    --dp.stages;
  const int smem = DqSmem<D>::bytes(dp.stages, p.nblk, dp.cap);
  int rc = encode_q_heads(&tm_q, qp, dp.qt, p.G);
  if (rc == DSA_OK) rc = encode_q_heads(&tm_go, gp, dp.qt, p.G);
  if (rc == DSA_OK) rc = encode_kv_maps(p, p.blk < kDqKeys ? p.blk : kDqKeys,
                                        &maps);
  if (rc != DSA_OK) return rc;
  auto dq = block_attn_dq_kernel<D>;
  if (!ok(allow_smem(dq, kMaxSmem))) return DSA_ERR_CUDA;
  const long long grid = (long long)dp.tiles * p.B * p.Hk;
  dq<<<(unsigned)grid, kBwdThreads, smem, st>>>(tm_q, tm_go, maps, p, dp);
  if (!ok(cudaGetLastError())) return DSA_ERR_CUDA;

  rc = encode_q_heads(&tm_q, qp, pl.qt, p.G);
  if (rc == DSA_OK) rc = encode_q_heads(&tm_go, gp, pl.qt, p.G);
  if (rc == DSA_OK) rc = encode_kv_maps(p, kKeyTile, &maps);
  if (rc != DSA_OK) return rc;
  auto dkv = block_attn_dkv_kernel<D>;
  if (!ok(allow_smem(dkv, KvSmem<D>::kBytes))) return DSA_ERR_CUDA;
  dkv<<<(unsigned)pl.items * pl.rep, kBwdThreads, KvSmem<D>::kBytes, st>>>(
      tm_q, tm_go, maps, p, pl, bf(gk), bf(gv));
  bwd_join_kernel<D><<<(unsigned)kts * pl.rep * kJoinParts, 256, 0, st>>>(
      p, pl, bf(gk), bf(gv));
  return ok(cudaGetLastError()) ? DSA_OK : DSA_ERR_CUDA;
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
  if (H / Hk > DSA_BLOCK_ATTN_MAX_GROUP || topk + local_blocks <= 0 ||
      (block_size != 16 && block_size != 32 && block_size != 64 &&
       block_size != 128))
    return 0;
  // the larger of the two ways to select, shared by all heads or not, that are
  // supported
  size_t most = 0;
  for (int heads : {1, Hk}) {
    dsa::BlockAttn p{};
    p.S = S, p.B = B, p.H = H, p.Hk = Hk, p.G = H / Hk, p.D = D, p.T = T;
    p.sel_heads = heads, p.topk = topk, p.blk = block_size;
    p.local = local_blocks;
    p.nblk = (int)(((long long)T + block_size - 1) / block_size);
    dsa::BwdPlan pl;
    if (dsa::make_plan(p, nullptr, &pl) == DSA_OK && pl.bytes > most)
      most = pl.bytes;
  }
  return most;
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
  // this selection's limits, then the room that any may take
  dsa::BwdPlan pl;
  rc = dsa::make_plan(p, static_cast<char *>(workspace), &pl);
  if (rc != DSA_OK) return rc;
  const size_t need = dsa_block_attn_bwd_workspace_size(
      S, B, H, Hk, D, T, block_size, topk, local_blocks);
  if (!workspace || workspace_bytes < need) return DSA_ERR_WORKSPACE;
  if (!aligned_to(workspace, 256)) return DSA_ERR_INVALID_ARG;
  p.status = static_cast<int *>(workspace);
  int num_sms = 0;
  rc = dsa::device_num_sms(&num_sms);
  if (rc != DSA_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  return D == 64 ? dsa::launch_bwd<64>(p, pl, o, lse, grad_o, grad_q, grad_k,
                                       grad_v, st)
                 : dsa::launch_bwd<128>(p, pl, o, lse, grad_o, grad_q, grad_k,
                                        grad_v, st);
}

}  // extern "C"
