// Attention over selected blocks of keys, forward: contiguous and paged keys
// and values, grouped heads, a running softmax.  Row (s, b) at position
// p = q_pos[b] + s attends to the keys j <= p of its blocks: the topk given
// ids (each once) and the `local` blocks that end with its own.
//     x_j = scale q.k_j,  o = softmax(x) v,  lse = ln sum exp x
//
// A CTA takes one query tile: up to 32 consecutive queries with the G heads
// that share a key head, 128 MMA rows.  It walks the union of its queries'
// blocks, 64 keys a step; a row's own choice is a bit in the block's mask.
// Neighbouring queries ask for much the same blocks, so the union is little
// longer than one query's list and the keys are read once for all of them;
// where they do not, an MMA over 128 rows still takes no longer than one over
// 16, so a query alone costs what it would cost in a tile of its own.
//   A step is 64 keys: S = Q K^T on the tensor cores (128 x 64, fp32 in
// tensor memory), of which each softmax thread holds a row in registers:
// maximum, moved only when a step exceeds it by more than 2^8 (then O is
// rescaled), P = exp2(S c - m) rounded to bf16 into columns of S; O += P V
// with P from tensor memory.  A row holds 16 neighbouring keys or none of
// them, so its mask is a choice of m or +inf for each 16; only steps with keys
// after some row's position look at single keys.
//   The scores have two buffers: the next step's product runs under this
// step's softmax, and the softmax warps go from step to step without waiting
// for the second product.  Two stages each of K and V at D = 128 (96 KB with Q;
// four at D = 64) and 256 tensor-memory columns let two CTAs share an SM.  Few
// rows (single tokens) are split over their blocks; the CTA that ends last
// joins the parts.
//
// Measured on one GB300 (bf16 peak 1909 TFLOP/s, copies 6776 GB/s):
//   16384 tokens, 64 / 8 heads of 128, 18 blocks of 64: 877 to 895 us, 1160
// TFLOP/s of the unions' products (1.7 times a row's own).  The tensor pipe is
// busy 48% of the time and issue slots 45%: a step alternates between a
// product and a softmax of 64 columns, and two CTAs fill each other's gaps only
// in part.
//   3 x 777 tokens, 40 / 8 heads of 64 from pages: 289 to 300 us; unions of
// three times a row's list, and a softmax twice as long beside a product.
//   One token of 64 sequences, 34 blocks of 64, 4 heads of 128: 53 us, 5.4
// TB/s; of one sequence: 12 us, of which two steps are 3.
//   A tile has 32 queries at most (a block's mask is one word), so heads with
// keys of their own (G = 1) fill 32 of the 128 MMA rows: 4096 tokens of 16 such
// heads take 115 us, of 64 heads in groups of four 118.
//
// Masked keys: a score that is not finite in a key that only other rows hold
// spoils the row's sum, see below; a V row that no row of
// the tile sees is zeroed in shared memory (a page's unwritten end may hold
// anything).  A V row that some rows see meets a zero weight in the others,
// which a NaN or an infinity survives: rows with a sum or a result that is not
// finite are computed again on their own (block_attn_row.cuh).
//
// Warps: 0 .. 3 softmax (thread = row = tensor-memory lane), 4 TMA producer,
// 5 MMA issuer and tensor-memory allocator.
#include "block_attn.cuh"
#include "block_attn_host.cuh"
#include "block_attn_row.cuh"
#include "block_attn_split.cuh"
#include "dsa_indexer.h"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kFwdThreads = 192;
constexpr int kTmaWarp = 4, kMmaWarp = 5;
// tensor-memory columns: two steps' scores, O; P takes the second half of
// its scores
constexpr uint32_t kTmS = 0, kTmO = 128;
// Rows of Q in shared memory: tiles of up to 32 rows (single tokens) are held
// in 32, and the products read what follows as the other rows, whose results
// no one uses.  The room goes to the stages: such launches wait for memory.
constexpr int q_rows(bool few) { return few ? 32 : kRows; }
// Stages of K and of V: what two CTAs an SM have room for (16 KB each at D =
// 128, 8 KB at D = 64).
constexpr int fwd_stages(int D, bool few) {
  return D == 64 ? (few ? 5 : 4) : (few ? 3 : 2);
}
constexpr float kSlack = 8.f;
// The counts of written parts, a byte for each item that is split, in the 256
// bytes that every entry point leaves to the status word: no other use of a
// workspace touches them.  Zero between calls.
constexpr int kDoneOffset = 64;
static_assert(kDoneOffset + kSplitItems / 2 <= 256,
              "a byte for each item that is split");

template <int D, bool FEW>
struct FwdSmem {
  static constexpr int kCh = D / 64;
  static constexpr int kTile = kCh * q_rows(FEW) * 128;
  static constexpr int kKey = kCh * kKeys * 128;   // K or V of a step
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kTile;
  static constexpr int kStages = fwd_stages(D, FEW);
  static constexpr int kOffV = kOffK + kStages * kKey;
  static constexpr int kOffBar = kOffV + kStages * kKey;
  // q_full; s_full p_full o_done, two each; k_full k_empty v_full v_empty
  static constexpr int kBars = 7 + 4 * kStages;
  static constexpr int kOffMisc = kOffBar + kBars * 8;
  static constexpr int kOffWords = kOffMisc + 32;
  static constexpr int bytes(int nblk, int cap) {
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

// Joins the parts of a split tile, o = sum_i w_i o_i / sum_i w_i with w_i =
// 2^(l_i - max), in the order of the splits; the CTA that finished last.  A
// thread takes four columns of a row and has kJoin parts in flight: the join
// is a chain of loads from L2.  qs: 128 floats of shared memory a warp.
constexpr int kJoin = 8;
template <int D>
__device__ __noinline__ void join_parts(const BlockAttn &p, const FwdPlan &pl,
                                        size_t part0, int b, int s0, int nq,
                                        int hk, float *qs, int tid) {
  constexpr int kLanes = D / 4;  // threads of a row: half a warp or a warp
  const float neg_inf = -__int_as_float(0x7f800000);
  const int rows = pl.qt * p.G, lane = tid & 31, c = tid % kLanes;
  const int todo = nq * p.G;
  // (whole warps stay in the loop: they vote)
  for (int r0 = tid / 32 * (32 / kLanes); r0 < todo;
       r0 += kFwdThreads / kLanes) {
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
      redo_row(p, pl, b, s0 + ra / p.G, hk * p.G + ra % p.G,
               qs + tid / 32 * 128, lane);
    }
  }
}

template <int D, bool FEW>
__global__ void __launch_bounds__(kFwdThreads, 2)
    block_attn_fwd_kernel(const __grid_constant__ CUtensorMap tm_q,
                          const __grid_constant__ KvMaps maps,
                          const __grid_constant__ BlockAttn p,
                          const __grid_constant__ FwdPlan pl) {
  using L = FwdSmem<D, FEW>;
  constexpr int CH = L::kCh, NS = L::kStages;
  constexpr uint32_t kIdescS = idesc_bf16_f32(kRows, kKeys);
  constexpr uint32_t kIdescO = idesc_bf16_f32_mn(kRows, D, false, true);
  const float neg_inf = -__int_as_float(0x7f800000);

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (base - raw_addr);
  const uint32_t sQ = base + L::kOffQ;
  auto sK = [&](int st) { return base + L::kOffK + st * L::kKey; };
  auto sV = [&](int st) { return base + L::kOffV + st * L::kKey; };
  auto qoff = [](int ks) {  // K step ks in Q's rows, and in 64 keys
    return (uint32_t)((ks >> 2) * (q_rows(FEW) * 128) + (ks & 3) * 32) >> 4;
  };
  auto koff = [](int ks) {
    return (uint32_t)((ks >> 2) * (kKeys * 128) + (ks & 3) * 32) >> 4;
  };
  const uint32_t bars = base + L::kOffBar;
  const uint32_t q_full = bars;
  auto s_full = [&](int i) { return bars + 8 + 8 * i; };
  auto p_full = [&](int i) { return bars + 24 + 8 * i; };
  auto o_done = [&](int i) { return bars + 40 + 8 * i; };
  auto k_full = [&](int i) { return bars + 56 + 8 * i; };
  auto k_empty = [&](int i) { return bars + 56 + 8 * (NS + i); };
  auto v_full = [&](int i) { return bars + 56 + 8 * (2 * NS + i); };
  auto v_empty = [&](int i) { return bars + 56 + 8 * (3 * NS + i); };
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

  if (tid == 0) {
    for (int i = 0; i < L::kBars; ++i)
      mbar_init(bars + 8 * i, i == 3 || i == 4 ? 4 : 1);  // p_full: 4 warps
    *abort_flag = 0;
    fence_mbar_init();
    // Q arrives while the blocks are listed
    mbar_arrive_expect_tx(q_full, CH * pl.qt * p.G * 128);
    for (int c = 0; c < CH; ++c)
      tma_load_4d(sQ + c * (q_rows(FEW) * 128), &tm_q, q_full, c * kChunk, hk * p.G,
                  b, s0);
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(tmem_holder), 256);
    tmem_relinquish();
  }
  const FirstMark first = first_mark(p, b, s0, nq, hk, tid);
  for (int n = tid; n < p.nblk; n += kFwdThreads) words[n] = 0u;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  mark_blocks(p, b, s0, nq, hk, words, tid, kFwdThreads, first);
  __syncthreads();
  if (warp == 0) {
    const int n = list_blocks(words, p.nblk, list, lane);
    if (lane == 0) *sCount = n;
  }
  __syncthreads();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0);
  // a step takes units of up to 64 keys: whole blocks, or halves of 128
  const int count = *sCount;
  const int unit = min(p.blk, kKeys), per = p.blk / unit;
  const int upt = kKeys / unit, units = count * per;
  const int all = (units + upt - 1) / upt;
  const int t0 = (int)((long long)all * split / pl.splits);
  const int t1 = (int)((long long)all * (split + 1) / pl.splits);
  const int n = t1 - t0;
  if (n > 0 && n <= NS && units < t1 * upt) {
    // the first pass of a stage is ragged: the rows past its blocks are read
    // by the second product (times zero) and must be numbers
    for (int i = tid; i < L::kKey / 16; i += kFwdThreads) {
      const uint32_t z[4] = {0u, 0u, 0u, 0u};
      st_shared_v4(sV((n - 1) % NS) + i * 16, z);
    }
    fence_proxy_async_smem();
    __syncthreads();
  }

  if (warp == kTmaWarp) {
    // ---------------- TMA producer ----------------
    const int ui = lane / CH, c = lane % CH;  // unit and chunk of this lane
    for (int i = 0; i < n; ++i) {
      const int st = i % NS;
      const uint32_t ph = i / NS & 1u;
      const int nu = min(upt, units - (t0 + i) * upt);
      int tok = 0, outer = 0;
      if (ui < upt) {
        // a ragged step's end repeats the last unit's keys: their scores are
        // masked, but have to be numbers (V's rows there are zeros, see above)
        const int x = min((t0 + i) * upt + ui, units - 1);
        const int bn = list[x / per];
        tok = bn * p.blk + x % per * unit;
        outer = b;
        if (p.table) {
          bool bad = false;
          outer = block_page(p, b, bn, bad);
          tok %= p.page_size;
        }
      }
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint32_t full = kv ? v_full(st) : k_full(st);
        const int n_in = kv ? nu : upt;
        if (!__all_sync(0xffffffffu,
                        wait_bar_rest(kv ? v_empty(st) : k_empty(st), ph ^ 1u,
                                      abort_flag, p.status)))
          goto done;
        if (lane == 0) mbar_arrive_expect_tx(full, n_in * unit * CH * 128);
        __syncwarp();
        if (ui < n_in)
          tma_load_4d((kv ? sV(st) : sK(st)) + c * (kKeys * 128) +
                          ui * unit * 128,
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
      const uint64_t qd = sdesc_k_sw128(sQ);
      bool ok = wait(q_full, 0);
      auto scores = [&](int i) -> bool {
        const int st = i % NS;
        if (!wait(k_full(st), i / NS & 1u)) return false;
        tc_fence_after();
        const uint64_t kd = sdesc_k_sw128(sK(st));
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          mma_bf16(tmem + kTmS + (i & 1) * 64, qd + qoff(ks), kd + koff(ks),
                   kIdescS, ks != 0);
        mma_commit(k_empty(st));
        mma_commit(s_full(i & 1));
        return true;
      };
      if (ok && n > 0) ok = scores(0);
      uint32_t acc = 0;
      for (int i = 0; ok && i < n; ++i) {
        if (i + 1 < n && !(ok = scores(i + 1))) break;
        const int st = i % NS;
        if (!(ok = wait(v_full(st), i / NS & 1u) &&
                   wait(p_full(i & 1), (i >> 1) & 1u)))
          break;
        tc_fence_after();
        const uint64_t vd = sdesc_mn_sw128(sV(st), kKeys * 128, 1024);
#pragma unroll
        for (int ks = 0; ks < kKeys / 16; ++ks)
          mma_bf16_ta(tmem + kTmO, tmem + kTmS + (i & 1) * 64 + 32 + ks * 8,
                      vd + ((ks * 2048) >> 4), kIdescO, ks == 0 ? acc : 1u);
        mma_commit(v_empty(st));
        mma_commit(o_done(i & 1));
        acc = 1;
      }
    }
    __syncwarp();
  } else {
    // ---------------- softmax: one row a thread ----------------
    const int row = tid;
    const int qi = row / p.G;
    const bool live = qi < nq;
    const int pos = live ? key_pos(p, b, s0 + qi) : -1;
    // the last key that the first and that any row of the tile sees
    const int pos_lo = key_pos(p, b, s0), pos_hi = key_pos(p, b, s0 + nq - 1);
    const float c2 = p.scale * 1.4426950408889634f;
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    const uint32_t tO = tmem + kTmO + lane_off;
    float m = neg_inf;
    float2 l2[2] = {};
    uint32_t next[2] = {};
    bool next_diag[2] = {};
    if (n > 0)
      step_masks(words, list, t0, count, p.lb, qi & 31, pos, pos_lo, next,
                 next_diag);
    for (int i = 0; i < n; ++i) {
      const int st = i % NS;
      const uint32_t tS = tmem + kTmS + (i & 1) * 64 + lane_off;
      const int t = t0 + i;
      const uint32_t mask[2] = {next[0], next[1]};
      const bool diag[2] = {next_diag[0], next_diag[1]};
      bool held[2];
#pragma unroll
      for (int c = 0; c < 2; ++c)
        held[c] = __any_sync(0xffffffffu, mask[c] != 0u);
      if (!__all_sync(0xffffffffu, wait_bar_rest(s_full(i & 1), (i >> 1) & 1u,
                                                 abort_flag, p.status)))
        goto done;
      tc_fence_after();
      uint32_t u[2][32];
      float mx = neg_inf;
      if (held[0] || held[1]) {
        __syncwarp();
        tmem_ld32(tS, u[0]);
        tmem_ld32(tS + 32, u[1]);
        tmem_ld_wait();
        reg_fence32(u[0]);
        reg_fence32(u[1]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (diag[c]) {  // keys after some row's position: one by one
#pragma unroll
            for (int x = 0; x < 32; ++x)
              u[c][x] = mask[c] >> x & 1u ? u[c][x] : 0xff800000u;
          }
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            float a = neg_inf, e = neg_inf;
#pragma unroll
            for (int x = 16 * g; x < 16 * g + 16; x += 4) {
              a = fmaxf(a, fmaxf(__uint_as_float(u[c][x]),
                                 __uint_as_float(u[c][x + 1])));
              e = fmaxf(e, fmaxf(__uint_as_float(u[c][x + 2]),
                                 __uint_as_float(u[c][x + 3])));
            }
            // a row holds all 16 keys or none, or they are hidden above
            if (mask[c] & (0xffffu << (16 * g))) mx = fmaxf(mx, fmaxf(a, e));
          }
        }
        mx *= c2;
      }
      // a row without a key so far keeps m = -inf and weights of zero
      const bool move = mx > m + kSlack;
      if (i > 0 && __any_sync(0xffffffffu, move)) {
        // O is at rest once the last step's second product is done
        if (!__all_sync(0xffffffffu,
                        wait_bar_rest(o_done((i - 1) & 1),
                                      ((i - 1) >> 1) & 1u, abort_flag,
                                      p.status)))
          goto done;
        tc_fence_after();
        const float f = move ? ex2(m - mx) : 1.f;
        l2[0] = __fmul2_rn(l2[0], make_float2(f, f));
        l2[1] = __fmul2_rn(l2[1], make_float2(f, f));
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t w[32];
          __syncwarp();
          tmem_ld32(tO + c * 32, w);
          tmem_ld_wait();
          reg_fence32(w);
#pragma unroll
          for (int x = 0; x < 32; ++x)
            w[x] = __float_as_uint(__uint_as_float(w[x]) * f);
          tmem_st32(tO + c * 32, w);
        }
      }
      if (move) m = mx;
      const float mu = m > neg_inf ? m : 0.f;
      // the next step's masks, among the exponentials
      if (i + 1 < n)
        step_masks(words, list, t + 1, count, p.lb, qi & 31, pos, pos_lo,
                   next, next_diag);
      // P = exp2(S c2 - mu)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t pk[16];
        if (held[c]) {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            // -inf takes the weights of keys that the row does not hold to 0
            const float sub = mask[c] & (0xffffu << (16 * g)) ? -mu : neg_inf;
#pragma unroll
            for (int x = 16 * g; x < 16 * g + 16; x += 2) {
              float2 e = __ffma2_rn(make_float2(__uint_as_float(u[c][x]),
                                                __uint_as_float(u[c][x + 1])),
                                    make_float2(c2, c2),
                                    make_float2(sub, sub));
              e.x = ex2(e.x);
              e.y = ex2(e.y);
              l2[(x >> 1) & 1] = __fadd2_rn(l2[(x >> 1) & 1], e);
              pk[x >> 1] = pack_bf16x2(e.x, e.y);
            }
          }
        } else {
#pragma unroll
          for (int x = 0; x < 16; ++x) pk[x] = 0u;
        }
        __syncwarp();
        tmem_st16(tS + 32 + c * 16, pk);
      }
      tmem_st_wait();
      tc_fence_before();
      if (diag[0] || diag[1]) {
        // V rows of this step that no row sees
        const int x = t * upt + row / unit;
        const bool over =
            row < kKeys && x < units &&
            list[x / per] * p.blk + x % per * unit + row % unit > pos_hi;
        if (__any_sync(0xffffffffu, over)) {
          if (!__all_sync(0xffffffffu,
                          wait_bar_rest(v_full(st), i / NS & 1u, abort_flag,
                                        p.status)))
            goto done;
          const uint32_t z[4] = {0u, 0u, 0u, 0u};
          if (over)
            for (int c = 0; c < CH * 8; ++c)
              st_shared_v4(sV(st) + (c >> 3) * (kKeys * 128) + row * 128 +
                               (c & 7) * 16,
                           z);
          fence_proxy_async_smem();
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full(i & 1));
    }
    // ---------------- o = O / l ----------------
    // The last score product came before the second products of the last two
    // steps: both may be open or done, and a parity names one phase of two, so
    // each has a barrier of its own.
    for (int i = max(n - 2, 0); i < n; ++i)
      if (!__all_sync(0xffffffffu,
                      wait_bar_rest(o_done(i & 1), (i >> 1) & 1u, abort_flag,
                                    p.status)))
        goto done;
    tc_fence_after();
    const float l = (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
    const bool some = l > 0.f || l != l;
    const float inv = some ? 1.f / l : 0.f;
    bool odd = l != l || l > 3e38f;  // not finite: computed again below
    const size_t at =
        ((size_t)(s0 + qi) * p.B + b) * p.H + hk * p.G + row % p.G;
    const size_t part =
        ((size_t)(blockIdx.x / pl.splits) * pl.splits + split) *
            (pl.qt * p.G) +
        row;
    const uint32_t out_buf = sK(0) + warp * 4096;  // K's space is free
    // (a short loop: this runs once a CTA, and instructions that are fetched
    // to run once take longer than they save)
    float2 chk = make_float2(0.f, 0.f);  // not a number where O is not finite
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      uint32_t u[32], w[16];
      if (n > 0) {
        __syncwarp();
        tmem_ld32(tO + c * 32, u);
        tmem_ld_wait();
        reg_fence32(u);
      }
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        float2 v = __fmul2_rn(make_float2(__uint_as_float(u[2 * x]),
                                          __uint_as_float(u[2 * x + 1])),
                              make_float2(inv, inv));
        chk = __ffma2_rn(v, make_float2(0.f, 0.f), chk);
        u[2 * x] = some ? __float_as_uint(v.x) : 0u;
        u[2 * x + 1] = some ? __float_as_uint(v.y) : 0u;
        w[x] = some ? pack_bf16x2(v.x, v.y) : 0u;
      }
      if (pl.splits > 1)
        store_rows<32>(out_buf, u,
                       live ? pl.part_o + part * D + c * 32 : nullptr, lane);
      else
        store_rows<16>(out_buf, w, live ? pl.o + at * D + c * 32 : nullptr,
                       lane);
    }
    odd |= some && !(chk.x + chk.y == 0.f);
    // m is a rounded product, the weights' exponents are multiply-adds of its
    // factors: above 2^25 they are a whole power of two apart, and a row may
    // lose all its weights
    odd |= m > neg_inf && fabsf(m) > 33554432.f;
    odd &= live;
    if (live) {
      const float lse2 = some ? m + log2f(l) : neg_inf;
      if (pl.splits > 1)
        // a NaN tells the joining CTA to compute the row again
        pl.part_l[part] = odd ? __int_as_float(0x7fffffff) : lse2;
      else
        pl.lse[at] = some ? lse2 * 0.69314718055994531f : neg_inf;
    }
    unsigned todo = __ballot_sync(0xffffffffu, odd);
    if (pl.splits == 1) {
      // (store_rows is done with this warp's part of the space)
      float *qs = reinterpret_cast<float *>(smem + L::kOffK) + warp * 1024;
      for (; todo; todo &= todo - 1) {
        const int r = warp * 32 + __ffs(todo) - 1;
        redo_row(p, pl, b, s0 + r / p.G, hk * p.G + r % p.G, qs, lane);
      }
    }
  }
done:
  if (pl.splits > 1) __threadfence();  // this CTA's parts, before the count
  __syncthreads();
  if (pl.splits > 1) {
    // (also after a wait that gave up: the counts stay whole)
    const int item = blockIdx.x / pl.splits;
    if (tid == 0) {
      const int sh = 8 * (item & 3);
      uint32_t *word = reinterpret_cast<uint32_t *>(p.status) +
                       (kDoneOffset + item) / 4;
      const uint32_t before = atomicAdd(word, 1u << sh) >> sh & 0xffu;
      const bool last = before + 1 == (uint32_t)pl.splits;
      if (last) atomicAnd(word, ~(0xffu << sh));  // for the next call
      __threadfence();
      *sCount = last;
    }
    __syncthreads();
    if (*sCount)
      join_parts<D>(p, pl, (size_t)item * pl.splits * (pl.qt * p.G), b, s0, nq,
                    hk, reinterpret_cast<float *>(smem + L::kOffK), tid);
    __syncthreads();
  }
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

template <int D, bool FEW>
int launch_fwd(const CUtensorMap &tm_q, const KvMaps &maps,
               const BlockAttn &p, const FwdPlan &pl, cudaStream_t st) {
  auto kern = block_attn_fwd_kernel<D, FEW>;
  const int smem = FwdSmem<D, FEW>::bytes(p.nblk, pl.cap);
  constexpr int kMost = FwdSmem<D, FEW>::bytes(DSA_BLOCK_ATTN_MAX_BLOCKS,
                                               DSA_BLOCK_ATTN_MAX_BLOCKS);
  static_assert(kMost <= kMaxSmem);
  if (allow_smem(kern, kMost) != cudaSuccess) return DSA_ERR_CUDA;
  const long long grid = (long long)pl.tiles * p.B * p.Hk * pl.splits;
  if (grid > 0x7fffffffll) return DSA_ERR_UNSUPPORTED;
  kern<<<(unsigned)grid, kFwdThreads, smem, st>>>(tm_q, maps, p, pl);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

int run_fwd(const BlockAttn &p, void *out_o, float *out_lse, void *workspace,
            int num_sms, cudaStream_t st) {
  const FwdPlan pl = plan_fwd(p, out_o, out_lse, workspace, num_sms);
  CUtensorMap tm_q;
  KvMaps maps;
  Problem qp{p.q, nullptr, nullptr, nullptr, p.S, p.B, p.H, p.D, 1, 1};
  int rc = encode_q_heads(&tm_q, qp, pl.qt, p.G);
  if (rc != DSA_OK) return rc;
  rc = encode_kv_maps(p, p.blk < kKeys ? p.blk : kKeys, &maps);
  if (rc != DSA_OK) return rc;
  const bool few = pl.qt * p.G <= q_rows(true);
  if (p.D == 64)
    rc = few ? launch_fwd<64, true>(tm_q, maps, p, pl, st)
             : launch_fwd<64, false>(tm_q, maps, p, pl, st);
  else
    rc = few ? launch_fwd<128, true>(tm_q, maps, p, pl, st)
             : launch_fwd<128, false>(tm_q, maps, p, pl, st);
  return rc;
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
