// Attention over selected blocks of keys, forward: contiguous and paged keys
// and values, grouped heads, a running softmax.  Row (s, b) at position
// p = q_pos[b] + s attends to the keys j <= p of its blocks: the topk given
// ids (each once) and the `local` blocks that end with its own.
//     x_j = scale q.k_j,  o = softmax(x) v,  lse = ln sum exp x
//
// A CTA takes one query tile: up to 32 consecutive queries with the G heads
// that share a key head, 128 MMA rows.  It walks the union of its queries'
// blocks, 128 keys a step; a row's own choice is a bit in the block's mask.
// Neighbouring queries ask for much the same blocks, so the union is little
// longer than one query's list and the keys are read once for all of them;
// where they do not, an MMA over 128 rows still takes no longer than one over
// 16, so a query alone costs what it would cost in a tile of its own.
//   S = Q K^T on the tensor cores (128 x 128, fp32 in tensor memory); a
// softmax thread has half of a row in registers: maximum, moved only when a step exceeds it by
// more than 2^8 (then O is rescaled), P = exp2(S c - m) rounded to bf16 into
// columns of S that are done; O += P V with P from tensor memory.  A row holds
// 16 neighbouring keys or none of them, so its mask is a choice of m or +inf
// for each 16; only steps with keys after some row's position look at single
// keys.
//   One stage of K and V (96 KB with Q at D = 128) and 256 tensor-memory
// columns let two CTAs share an SM: one's products run under the other's
// softmax, and its next K arrives while its own softmax and second product
// run.  Few rows (single tokens) are split over their blocks, and a second
// kernel joins the parts.
//
// Masked keys: a score that is not finite in a key that only other rows hold
// spoils the row's sum, see below; a V row that no row of
// the tile sees is zeroed in shared memory (a page's unwritten end may hold
// anything).  A V row that some rows see meets a zero weight in the others,
// which a NaN or an infinity survives: rows with a sum or a result that is not
// finite are computed again on their own (block_attn_row.cuh).
//
// Warps: 0 .. 7 softmax (warp w reads tensor-memory lanes 32 (w % 4) .. + 31,
// 64 keys of a step: the two warps of a row exchange its maximum), 8 TMA
// producer, 9 MMA issuer and tensor-memory allocator.
#include "block_attn.cuh"
#include "block_attn_host.cuh"
#include "block_attn_row.cuh"
#include "dsa_indexer.h"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kRows = 128;  // MMA rows of a query tile
constexpr int kKeys = 128;  // keys of a step
constexpr int kSoftWarps = 8;  // two for each 32 rows, 64 keys each
constexpr int kFwdThreads = 32 * (kSoftWarps + 2);
constexpr int kTmaWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1;
// tensor-memory columns; P takes the second half of each 64 of S
constexpr uint32_t kTmS = 0, kTmO = 128;
constexpr float kSlack = 8.f;

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

template <int D>
struct FwdSmem {
  static constexpr int kCh = D / 64;
  static constexpr int kTile = kCh * kRows * 128;  // 128 rows of D bf16
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kTile;
  static constexpr int kOffV = 2 * kTile;
  static constexpr int kOffBar = 3 * kTile;
  // q_full k_full k_empty v_full v_empty s_full p_full o_full
  static constexpr int kOffMisc = kOffBar + 8 * 8;
  static constexpr int kOffRed = kOffMisc + 32;  // [4][128]
  static constexpr int kOffWords = kOffRed + 4 * kRows * 4;
  static int bytes(int nblk, int cap) {
    return kOffWords + nblk * 4 + ((cap * 2 + 15) & ~15) + 1024;
  }
};

// One row on its own, by one warp (qs: 128 floats of shared memory).  Out of
// line: it is rare, and inlined it costs the loop before it registers.
__device__ __noinline__ void redo_row(const BlockAttn &p, const FwdPlan &pl,
                                      int b, int s, int h, float *qs,
                                      int lane) {
  const size_t at = ((size_t)s * p.B + b) * p.H + h;
  __syncwarp();
  for (int d = lane; d < p.D; d += 32)
    qs[d] = __bfloat162float(p.q[at * p.D + d]);
  __syncwarp();
  bool bad = false;
  float acc[4], lse;
  attn_row(p, b, s, h / p.G, qs, lane, bad, acc, lse);
  for (int i = 0; i * 32 < p.D; ++i)
    pl.o[at * p.D + lane + 32 * i] = __float2bfloat16(acc[i]);
  if (lane == 0) pl.lse[at] = lse;
}

// The barrier of the two warps of 32 rows.  Its number is written out: one
// that is computed makes the compiler claim all sixteen, and a second CTA no
// longer fits the SM.
__device__ __forceinline__ bool pair_bar(int quad, bool pred) {
  switch (quad) {
    case 0: return named_bar_or(1, 64, pred);
    case 1: return named_bar_or(2, 64, pred);
    case 2: return named_bar_or(3, 64, pred);
    default: return named_bar_or(4, 64, pred);
  }
}

template <int D>
__global__ void __launch_bounds__(kFwdThreads, 2)
    block_attn_fwd_kernel(const __grid_constant__ CUtensorMap tm_q,
                          const __grid_constant__ KvMaps maps,
                          const __grid_constant__ BlockAttn p,
                          const __grid_constant__ FwdPlan pl) {
  using L = FwdSmem<D>;
  constexpr int CH = L::kCh;
  constexpr uint32_t kIdescS = idesc_bf16_f32(kRows, kKeys);
  constexpr uint32_t kIdescO = idesc_bf16_f32_mn(kRows, D, false, true);
  const float neg_inf = -__int_as_float(0x7f800000);

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (base - raw_addr);
  const uint32_t sQ = base + L::kOffQ, sK = base + L::kOffK,
                 sV = base + L::kOffV;
  const uint32_t bars = base + L::kOffBar;
  const uint32_t q_full = bars, k_full = bars + 8, k_empty = bars + 16,
                 v_full = bars + 24, v_empty = bars + 32, s_full = bars + 40,
                 p_full = bars + 48, o_full = bars + 56;
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + L::kOffMisc);
  volatile int *abort_flag = reinterpret_cast<int *>(smem + L::kOffMisc + 4);
  int *sCount = reinterpret_cast<int *>(smem + L::kOffMisc + 8);
  uint32_t *words = reinterpret_cast<uint32_t *>(smem + L::kOffWords);
  uint16_t *list = reinterpret_cast<uint16_t *>(words + p.nblk);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // later tiles have more keys: they go first
  int it = blockIdx.x;
  const int split = it % pl.splits;
  it /= pl.splits;
  const int hk = it % p.Hk;
  it /= p.Hk;
  const int b = it % p.B;
  const int tile = pl.tiles - 1 - it / p.B;
  const int s0 = tile * pl.qt;
  const int nq = min(pl.qt, p.S - s0);

  const FirstMark first = first_mark(p, b, s0, nq, hk, tid);
  if (tid == 0) {
    for (int i = 0; i < 8; ++i)
      mbar_init(bars + 8 * i, i == 6 ? kSoftWarps : 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(tmem_holder), 256);
    tmem_relinquish();
  }
  for (int n = tid; n < p.nblk; n += kFwdThreads) words[n] = 0u;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 32 * kTmaWarp) {  // Q arrives while the blocks are listed
    mbar_arrive_expect_tx(q_full, CH * pl.qt * p.G * 128);
    for (int c = 0; c < CH; ++c)
      tma_load_4d(sQ + c * (kRows * 128), &tm_q, q_full, c * kChunk,
                  hk * p.G, b, s0);
  }
  mark_blocks(p, b, s0, nq, hk, words, tid, kFwdThreads, first);
  __syncthreads();
  if (warp == 0) {
    const int n = list_blocks(words, p.nblk, list, lane);
    if (lane == 0) *sCount = n;
  }
  __syncthreads();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0);
  const int bpt = kKeys / p.blk;  // blocks of a step
  const int all = (*sCount + bpt - 1) / bpt;
  const int t0 = (int)((long long)all * split / pl.splits);
  const int t1 = (int)((long long)all * (split + 1) / pl.splits);
  const int count = *sCount;
  if (t1 - t0 == 1 && count < t1 * bpt) {
    // a single, ragged step: the rows past its blocks are read by the second
    // product (times zero) and must be numbers
    for (int i = tid; i < L::kTile / 16; i += kFwdThreads) {
      const uint32_t z[4] = {0u, 0u, 0u, 0u};
      st_shared_v4(sV + i * 16, z);
    }
    fence_proxy_async_smem();
    __syncthreads();
  }

  if (warp == kTmaWarp) {
    // ---------------- TMA producer ----------------
    for (int t = t0; t < t1; ++t) {
      const uint32_t ph = (t - t0) & 1u;
      const int nb = min(bpt, count - t * bpt);
      // lane (block, chunk) of the step
      const int bi = lane / CH, c = lane % CH;
      const bool mine = bi < nb;
      int tok = 0, outer = 0;
      if (mine) {
        const int n = list[t * bpt + bi];
        if (p.table) {
          bool bad = false;
          outer = block_page(p, b, n, bad);
          tok = (int)((long long)n * p.blk % p.page_size);
        } else {
          outer = b;
          tok = n * p.blk;
        }
      }
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint32_t full = kv ? v_full : k_full;
        if (!__all_sync(0xffffffffu,
                        wait_bar_rest(kv ? v_empty : k_empty, ph ^ 1u,
                                     abort_flag, p.status)))
          goto done;
        if (lane == 0) mbar_arrive_expect_tx(full, nb * p.blk * CH * 128);
        __syncwarp();
        if (mine)
          tma_load_4d((kv ? sV : sK) + c * (kRows * 128) + bi * p.blk * 128,
                      kv ? &maps.v : &maps.k, full, c * kChunk, tok,
                      hk * (kv ? maps.bc_vh : maps.bc_kh),
                      outer * (kv ? maps.bc_vs : maps.bc_ks));
      }
    }
  } else if (warp == kMmaWarp) {
    // ---------------- MMA issuer: one thread ----------------
    if (elect_one()) {
      auto wait = [&](uint32_t bar, uint32_t ph) -> bool {
        return wait_bar_rest(bar, ph, abort_flag, p.status);
      };
      const uint64_t qd = sdesc_k_sw128(sQ), kd = sdesc_k_sw128(sK);
      const uint64_t vd = sdesc_mn_sw128(sV, kRows * 128, 1024);
      bool ok = wait(q_full, 0);
      uint32_t ph = 0, acc = 0;
      for (int t = t0; ok && t < t1; ++t) {
        if (!(ok = wait(k_full, ph))) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t o = ((ks >> 2) * (kRows * 128) + (ks & 3) * 32) >> 4;
          mma_bf16(tmem + kTmS, qd + o, kd + o, kIdescS, ks != 0);
        }
        mma_commit(k_empty);
        mma_commit(s_full);
        if (!(ok = wait(v_full, ph) && wait(p_full, ph))) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < kKeys / 16; ++ks)
          mma_bf16_ta(tmem + kTmO, tmem + kTmS + (ks >> 2) * 64 + 32 + (ks & 3) * 8,
                      vd + ((ks * 2048) >> 4), kIdescO, ks == 0 ? acc : 1u);
        mma_commit(v_empty);
        if (t + 1 == t1) mma_commit(o_full);
        acc = 1;
        ph ^= 1;
      }
    }
    __syncwarp();
  } else {
    // ---------- softmax: a thread takes a row's keys 64 half .. + 63 ----------
    const int half = warp >> 2, quad = warp & 3;
    const int row = quad * 32 + lane;
    const int qi = row / p.G;
    const bool live = qi < nq;
    const int pos = live ? key_pos(p, b, s0 + qi) : -1;
    // the last key that the first and that any row of the tile sees
    const int pos_lo = key_pos(p, b, s0), pos_hi = key_pos(p, b, s0 + nq - 1);
    const float c2 = p.scale * 1.4426950408889634f;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t tS = tmem + kTmS + lane_off + half * 64,
                   tO = tmem + kTmO + lane_off + half * (D / 2);
    float *red = reinterpret_cast<float *>(smem + L::kOffRed);
    float m = neg_inf;
    float2 l2[2] = {};
    // the two warps of 32 rows meet at a barrier every step: a wait that
    // gave up is carried to it, so that both leave together
    bool fail = false;
    for (int t = t0; t < t1; ++t) {
      const uint32_t ph = (t - t0) & 1u;
      uint32_t mask[2];
      bool held[2], diag[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        int end;
        mask[c] = step_mask(words, list, t * bpt, count, p.lb, 2 * half + c,
                            qi & 31, pos, end);
        diag[c] = end > pos_lo;
        held[c] = __any_sync(0xffffffffu, mask[c] != 0u);
      }
      fail |= !__all_sync(0xffffffffu, wait_bar_rest(s_full, ph, abort_flag,
                                                     p.status));
      tc_fence_after();
      // the row's maximum, 32 keys at a time; the second 32 stay
      uint32_t u[32];
      float mx = neg_inf;
      auto fetch = [&](int c) {
        __syncwarp();
        tmem_ld32(tS + c * 32, u);
        tmem_ld_wait();
        reg_fence32(u);
        if (diag[c]) {  // keys after some row's position: one by one
#pragma unroll
          for (int i = 0; i < 32; ++i)
            u[i] = mask[c] >> i & 1u ? u[i] : 0xff800000u;
        }
      };
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (!held[c]) continue;
        fetch(c);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          float a = neg_inf, e = neg_inf;
#pragma unroll
          for (int i = 16 * g; i < 16 * g + 16; i += 4) {
            a = fmaxf(a, fmaxf(__uint_as_float(u[i]),
                               __uint_as_float(u[i + 1])));
            e = fmaxf(e, fmaxf(__uint_as_float(u[i + 2]),
                               __uint_as_float(u[i + 3])));
          }
          // a row holds all 16 keys or none, or they are hidden above
          if (mask[c] & (0xffffu << (16 * g))) mx = fmaxf(mx, fmaxf(a, e));
        }
      }
      red[half * kRows + row] = mx;
      if (pair_bar(quad, fail)) goto done;
      mx = fmaxf(mx, red[(half ^ 1) * kRows + row]) * c2;
      // a row without a key so far keeps m = -inf and weights of zero
      const bool move = mx > m + kSlack;
      if (__any_sync(0xffffffffu, move && t > t0)) {
        const float f = move ? ex2(m - mx) : 1.f;
        l2[0] = __fmul2_rn(l2[0], make_float2(f, f));
        l2[1] = __fmul2_rn(l2[1], make_float2(f, f));
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {  // half of O's columns
          uint32_t w[16];
          __syncwarp();
          tmem_ld16(tO + c * 16, w);
          tmem_ld_wait();
          reg_fence16(w);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            w[i] = __float_as_uint(__uint_as_float(w[i]) * f);
          tmem_st16(tO + c * 16, w);
        }
      }
      if (move) m = mx;
      const float mu = m > neg_inf ? m : 0.f;
      // P = exp2(S c2 - mu) into the second half of the 64 columns of S
#pragma unroll
      for (int c = 1; c >= 0; --c) {
        uint32_t pk[16];
        if (held[c]) {
          if (c == 0) fetch(0);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            // -inf takes the weights of keys that the row does not hold to 0
            const float sub = mask[c] & (0xffffu << (16 * g)) ? -mu : neg_inf;
#pragma unroll
            for (int i = 16 * g; i < 16 * g + 16; i += 2) {
              float2 e = __ffma2_rn(make_float2(__uint_as_float(u[i]),
                                                __uint_as_float(u[i + 1])),
                                    make_float2(c2, c2),
                                    make_float2(sub, sub));
              e.x = ex2(e.x);
              e.y = ex2(e.y);
              l2[(i >> 1) & 1] = __fadd2_rn(l2[(i >> 1) & 1], e);
              pk[i >> 1] = pack_bf16x2(e.x, e.y);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) pk[i] = 0u;
        }
        __syncwarp();
        tmem_st16(tS + 32 + c * 16, pk);
      }
      tmem_st_wait();
      tc_fence_before();
      if (diag[0] || diag[1]) {
        // V rows of this step that no row sees; each half its 64 keys
        const int kr = half * 64 + (row & 63);
        const int i = t * bpt + (kr >> p.lb);
        const bool over = row < 64 && i < count &&
                          (list[i] << p.lb) + (kr & (p.blk - 1)) > pos_hi;
        if (__any_sync(0xffffffffu, over)) {
          fail |= !__all_sync(0xffffffffu, wait_bar_rest(v_full, ph, abort_flag,
                                                         p.status));
          const uint32_t z[4] = {0u, 0u, 0u, 0u};
          if (over && !fail)
            for (int c = 0; c < CH * 8; ++c)
              st_shared_v4(sV + (c >> 3) * (kRows * 128) + kr * 128 +
                               (c & 7) * 16,
                           z);
          fence_proxy_async_smem();
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full);
    }
    float l = (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
    red[half * kRows + row] = l;
    if (pair_bar(quad, fail)) goto done;
    l += red[(half ^ 1) * kRows + row];
    // ---------------- o = O / l ----------------
    if (t1 > t0) {
      fail = !__all_sync(0xffffffffu,
                         wait_bar_rest(o_full, 0, abort_flag, p.status));
      tc_fence_after();
    }
    const bool some = l > 0.f || l != l;
    const float inv = some ? 1.f / l : 0.f;
    bool odd = l != l || l > 3e38f;  // not finite: computed again below
    const size_t at =
        ((size_t)(s0 + qi) * p.B + b) * p.H + hk * p.G + row % p.G;
    const size_t part =
        ((size_t)(blockIdx.x / pl.splits) * pl.splits + split) *
            (pl.qt * p.G) +
        row;
    // half of the columns; Q's space is free for the way out
    const uint32_t out_buf = sQ + warp * (32 * D);
    constexpr int kOut = D / 4;  // words of this half's bf16 row
    uint32_t ow[kOut];
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      const int d0 = half * (D / 2) + c * 32;
      uint32_t u[32];
      if (t1 > t0) {
        __syncwarp();
        tmem_ld32(tO + c * 32, u);
        tmem_ld_wait();
        reg_fence32(u);
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float v = some ? __uint_as_float(u[i]) * inv : 0.f;
        odd |= !(fabsf(v) < 3e38f);
        u[i] = __float_as_uint(v);
      }
      if (pl.splits > 1) {
        if (live) {
          float4 *dst = reinterpret_cast<float4 *>(pl.part_o + part * D + d0);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[i] = make_float4(
                __uint_as_float(u[4 * i]), __uint_as_float(u[4 * i + 1]),
                __uint_as_float(u[4 * i + 2]), __uint_as_float(u[4 * i + 3]));
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i)
        ow[c * 16 + i] = pack_bf16x2(__uint_as_float(u[2 * i]),
                                     __uint_as_float(u[2 * i + 1]));
    }
    if (pl.splits == 1)
      store_rows<kOut>(out_buf, ow,
                       live ? pl.o + at * D + half * (D / 2) : nullptr, lane);
    // a row that is not finite in either half
    red[(2 + half) * kRows + row] = odd && live ? 1.f : 0.f;
    if (pair_bar(quad, fail)) goto done;
    odd = live && (odd || red[(3 - half) * kRows + row] != 0.f);
    if (live && half == 0) {
      const float lse2 = some ? m + log2f(l) : neg_inf;
      if (pl.splits > 1)
        // a NaN tells the joining kernel to compute the row again
        pl.part_l[part] = odd ? __int_as_float(0x7fffffff) : lse2;
      else
        pl.lse[at] = some ? lse2 * 0.69314718055994531f : neg_inf;
    }
    unsigned todo = __ballot_sync(0xffffffffu, odd && half == 0);
    if (pl.splits == 1) {
      // K's space is free: the last product is done
      float *qs = reinterpret_cast<float *>(smem + L::kOffK) + warp * 128;
      for (; todo; todo &= todo - 1) {
        const int r = quad * 32 + __ffs(todo) - 1;
        redo_row(p, pl, b, s0 + r / p.G, hk * p.G + r % p.G, qs, lane);
      }
    }
  }
done:
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// Joins the parts of a split tile: o = sum_i w_i o_i / sum_i w_i with
// w_i = 2^(l_i - max).  One warp a row.
__global__ void __launch_bounds__(256)
    block_attn_join_kernel(const BlockAttn p, const FwdPlan pl) {
  __shared__ float qs_all[8][128];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long r = (long long)blockIdx.x * 8 + warp;
  if (r >= (long long)p.S * p.B * p.H) return;
  const float neg_inf = -__int_as_float(0x7f800000);
  const int h = (int)(r % p.H);
  const int b = (int)(r / p.H % p.B), s = (int)(r / p.H / p.B);
  const int hk = h / p.G, tile = s / pl.qt;
  const int rows = pl.qt * p.G;
  const size_t item = ((size_t)(pl.tiles - 1 - tile) * p.B + b) * p.Hk + hk;
  const size_t part =
      item * pl.splits * rows + (s - tile * pl.qt) * p.G + h % p.G;
  float mx = neg_inf;
  bool odd = false;
  for (int i = lane; i < pl.splits; i += 32) {
    const float l = pl.part_l[part + (size_t)i * rows];
    odd |= l != l;
    mx = fmaxf(mx, l);
  }
  for (int x = 16; x; x >>= 1)
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
  float acc[4] = {}, ls = neg_inf;
  if (__any_sync(0xffffffffu, odd)) {
    float *qs = qs_all[warp];
    for (int d = lane; d < p.D; d += 32)
      qs[d] = __bfloat162float(p.q[r * p.D + d]);
    __syncwarp();
    bool bad = false;
    attn_row(p, b, s, h / p.G, qs, lane, bad, acc, ls);
  } else if (mx > neg_inf) {
    float sum = 0.f;
    for (int i = 0; i < pl.splits; ++i) {
      const float w = ex2(pl.part_l[part + (size_t)i * rows] - mx);
      sum += w;
      const float *src = pl.part_o + (part + (size_t)i * rows) * p.D + lane;
#pragma unroll
      for (int d = 0; d < 4; ++d)
        if (d * 32 < p.D) acc[d] = fmaf(w, src[32 * d], acc[d]);
    }
    for (int d = 0; d < 4; ++d) acc[d] /= sum;
    ls = (mx + log2f(sum)) * 0.69314718055994531f;
  }
  for (int d = 0; d * 32 < p.D; ++d)
    pl.o[r * p.D + lane + 32 * d] = __float2bfloat16(acc[d]);
  if (lane == 0) pl.lse[r] = ls;
}

// Room for two CTAs an SM on the largest device: a split launch has no more.
constexpr int kSplitItems = 320;

template <int D>
int launch_fwd(const CUtensorMap &tm_q, const KvMaps &maps,
               const BlockAttn &p, const FwdPlan &pl, cudaStream_t st) {
  auto kern = block_attn_fwd_kernel<D>;
  const int smem = FwdSmem<D>::bytes(p.nblk, pl.cap);
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           smem) != cudaSuccess)
    return DSA_ERR_CUDA;
  const long long grid = (long long)pl.tiles * p.B * p.Hk * pl.splits;
  if (grid > 0x7fffffffll) return DSA_ERR_UNSUPPORTED;
  kern<<<(unsigned)grid, kFwdThreads, smem, st>>>(tm_q, maps, p, pl);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

int run_fwd(const BlockAttn &p, void *out_o, float *out_lse, void *workspace,
            int num_sms, cudaStream_t st) {
  FwdPlan pl{};
  pl.qt = tile_queries(p.G, kRows);
  if (pl.qt > p.S) pl.qt = p.S;
  pl.tiles = (p.S + pl.qt - 1) / pl.qt;
  const long long most = (long long)pl.qt * (p.topk + p.local);
  pl.cap = (int)(most < p.nblk ? most : p.nblk);
  pl.o = static_cast<__nv_bfloat16 *>(out_o);
  pl.lse = out_lse;
  // Few tiles: share each among CTAs until two an SM are busy, with a step
  // each at least.
  const long long items = (long long)pl.tiles * p.B * p.Hk;
  const int bpt = kKeys / p.blk;
  long long slots = 2ll * num_sms;
  if (slots > kSplitItems) slots = kSplitItems;
  pl.splits = 1;
  if (items * 2 <= slots) {
    long long n = slots / items;
    const long long steps = (pl.cap + bpt - 1) / bpt;
    if (n > steps) n = steps;
    pl.splits = (int)n;
  }
  if (pl.splits > 1) {
    pl.part_l = reinterpret_cast<float *>(static_cast<char *>(workspace) + 256);
    const size_t rows = (size_t)items * pl.splits * pl.qt * p.G;
    pl.part_o = pl.part_l + ((rows + 63) & ~(size_t)63);
  }
  CUtensorMap tm_q;
  KvMaps maps;
  Problem qp{p.q, nullptr, nullptr, nullptr, p.S, p.B, p.H, p.D, 1, 1};
  int rc = encode_q_heads(&tm_q, qp, pl.qt, p.G);
  if (rc != DSA_OK) return rc;
  rc = encode_kv_maps(p, p.blk, &maps);
  if (rc != DSA_OK) return rc;
  rc = p.D == 64 ? launch_fwd<64>(tm_q, maps, p, pl, st)
                 : launch_fwd<128>(tm_q, maps, p, pl, st);
  if (rc != DSA_OK || pl.splits == 1) return rc;
  const long long rows = (long long)p.S * p.B * p.H;
  block_attn_join_kernel<<<(unsigned)((rows + 7) / 8), 256, 0, st>>>(p, pl);
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
  return run_fwd(p, out_o, out_lse, workspace, num_sms,
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
  p.lb = p.blk == 16 ? 4 : p.blk == 32 ? 5 : p.blk == 64 ? 6 : 7;
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
    if (s < 0 || s >= (1ll << 38)) return DSA_ERR_INVALID_ARG;
  // a dimension of one element may have any other stride
  if ((p.table ? p.page_size : p.T) == 1) p.k_st = p.v_st = 0;
  if ((p.table ? p.num_pages : p.B) == 1) p.k_sb = p.v_sb = 0;
  if (p.Hk == 1) p.k_sh = p.v_sh = 0;
  // tokens of one tensor may not share their memory
  if ((p.table ? p.page_size : p.T) > 1 && (p.k_st == 0 || p.v_st == 0))
    return DSA_ERR_INVALID_ARG;
  for (long long s : {p.k_st, p.k_sb, p.k_sh, p.v_st, p.v_sb, p.v_sh})
    if (s % 8 != 0) return DSA_ERR_INVALID_ARG;
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
  // the status word, then the parts of tiles shared among CTAs
  const int G = H / Hk;
  if (G > DSA_BLOCK_ATTN_MAX_GROUP) return 256;
  long long qt = dsa::tile_queries(G, dsa::kRows);
  if (qt > S) qt = S;
  const long long items = ((S + qt - 1) / qt) * B * Hk;
  if (items * 2 > dsa::kSplitItems) return 256;
  const size_t rows = (size_t)dsa::kSplitItems * qt * G;
  return 256 + (rows + 64) * 4 + rows * D * 4;
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
