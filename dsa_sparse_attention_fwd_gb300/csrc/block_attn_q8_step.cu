// Attention over a paged cache held in 8 bits for few rows: single tokens and
// drafts, over selected blocks or all keys.
//
// Bounded by memory: every key and value is one byte an element and is read
// once for the G heads (and, where all keys are attended to, the queries) that
// share it.  An item is up to 16 or 32 rows of one sequence and key head; all
// items' steps of 32 keys laid end to end are cut into equal slices, one a
// CTA, so that sequences of any lengths load the GPU evenly.  An item that
// spans CTAs leaves its parts in the workspace, joined by the CTA that
// finishes last in the order of the slices.
//
// Four warps walk the slice (block lists, pages, scales, queries) and fill a
// ring of shared memory by TMA, each of the eight others having its own stages:
// a step of 32 keys goes to one warp, which keeps its own running maximum, sum
// and output for the item; the warps meet only at an item's end, while the
// ring fills with the next.  The products are mma.sync m16n8k16: a tile of a
// few rows cannot fill a tcgen05 tile, whose operands would have to be
// written to shared memory again as 16-bit values (three times the bytes that
// came); here they go from the 8-bit tile to registers, two elements a
// conversion (e4m3 to fp16 is exact).
//     t_j = c q.k_j 2^ek + ev,   P_j = 2^(t_j - m),   O += P_j v_j,
//     l += P_j 2^-ev
// with 2^ek, 2^ev the group's scales: the values' scale is part of the
// exponent, so the largest P is 2^6 to 2^14 whatever the scales are, and fp16
// holds P to 2^-11 (more than bf16), down to 2^-31 of the largest.  The query
// enters as fp16 after a power of two brings its largest value to 2^14.
//
// The order of the elements in the products is free as long as both sides
// agree, and chosen for whole 16-byte loads without bank conflicts: thread (g,
// t) reads 16 neighbours of a key, and for the output product 16 neighbours of
// the keys 2t and (2t + 1) ^ 4.
//
// Values that are not finite: masked scores are replaced before use, and value
// rows that no row of the tile sees are zeroed in registers.  What is not finite
// then comes from a key that some row sees.  A row's own it keeps.  Where rows of
// a tile see different keys (several queries over all keys), or a row's factor
// may have left fp32, the row is computed again on its own (block_attn_q8.cuh).
//
// Measured on one GB300 (copies 6767 GB/s), on the device: 64 single tokens over
// all of 2048 to 32767 keys, 4 heads of 128, 1.09 GB: 186 us, 5.8 TB/s; the loop
// is 161 of 178 us of a CTA (6.7 TB/s), the start 4, the ends of its 2.7 items 6,
// the last join 5, and the last CTA ends 15 us after the mean.  One token over
// 131064 keys: 52.6 us of 39.7.  34 blocks of 64 for 64 tokens: 43 us, of which
// the loop is 23: items of 68 steps over eight warps end often.  One warp loading
// for all took 725 cycles a step (358 us); four take less than the memory's 330.
#include "block_attn_host.cuh"
#include "block_attn_q8.cuh"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kFeeders = 4;  // warps that load
// Warps that multiply, and how many registers of a thread move to them from
// those that load (setmaxnreg; 384 threads are launched with 168 each).  Twelve
// warps with 144 registers were 8% slower: the spills cost more than they hide.
constexpr int kWarps = 8, kThreads = (kWarps + kFeeders) * 32;
constexpr int mul_regs(int mt) { return mt == 1 ? 192 : 200; }
constexpr int feeder_regs(int mt) { return mt == 1 ? 120 : 104; }
static_assert(kWarps * mul_regs(1) + kFeeders * feeder_regs(1) <=
                      (kWarps + kFeeders) * 168 &&
                  kWarps * mul_regs(2) + kFeeders * feeder_regs(2) <=
                      (kWarps + kFeeders) * 168,
              "registers move, there are no more of them");
constexpr int kKeys = 32;  // of a step
// A CTA's slice has at least so many steps.
constexpr int kMinSteps = 8;
// The counts of written parts: a byte for each CTA, in the 256 bytes that
// every entry point leaves to the status word.
constexpr int kDoneOffset = 64;
constexpr int kMaxCtas = 256 - kDoneOffset;

struct StepPlan {
  bool all;     // no selection: all keys of the local blocks
  int rows;     // that share keys: S * G, of one query of a selection G
  int items_b;  // items of a sequence
  int box;      // tokens of a TMA box: 16 or 32
  int stages;   // of a warp's ring
  int cap;      // entries of the block list
  float *part_o, *part_l;  // [CTA][2][32] rows of D, and their log-sums
  uint32_t *done;
};

struct Maps8 {
  CUtensorMap k, v;
};

// In place of a part's log-sum: the row is to be computed again.  (A NaN that no
// arithmetic gives.)
constexpr int kAgain = 0x7fc0a9a1;
// c times the query's power of two up to which scores are right whatever the
// keys' scales (2^40 at most) and codes are.
constexpr float kMostFactor = 1208925819614629174706176.f;  // 2^80

// What the producer says of an item's part.
struct Entry {
  int n, g0;     // its steps, and the CTA's steps before it
  int b, hk, s;  // s: the query, of a selection
  int c0, c1;    // CTAs that share it
  int slot;      // where this one's part goes: 0, 1 or -1 (whole)
};

// Of 16 keys of a step: exponents of the scales, the first key, and how many
// of them some row of the tile sees.
struct Sub {
  int ek, ev, j0, seen;
};

// A tile's rows as the loading warps prepare them: their queries as MMA
// operands (16-bit, after a power of two), the factor c times that power's
// inverse, the last and the first key that they see.
template <int D, int MT>
struct Rows {
  uint4 q[D / 16][MT][32];
  float cr[MT * 16];
  int pos[MT * 16], lo[MT * 16];
};

template <int D, int MT>
struct StepSmem {
  static constexpr int kStage = 2 * kKeys * D;  // K, then V
  // Floats of a row when the warps' outputs are added up: 8 runs of D / 8, each
  // in an order (run_at) that keeps a warp's 16-byte pieces in different banks.
  static constexpr int kPitch = D == 128 ? 144 : 72;
  static constexpr int kSum = kWarps * 16 * kPitch * 4;
  static int bytes(int stages, int nblk, int cap) {
    return stages * kWarps * (kStage + 2 * (int)sizeof(Sub) + 16) + kSum +
           2 * (int)sizeof(Rows<D, MT>) + 4 * (int)sizeof(Entry) +
           2 * kWarps * 16 * MT * 4 + kWarps * 512 + 128 +
           (cap ? (nblk + 31) / 32 * 4 + (cap * 2 + 15) / 16 * 16 : 0) + 1024;
  }
};
// Place of the 16-byte piece k of run q (of 8) of a row.
template <int D>
__device__ __forceinline__ int run_at(int q, int k) {
  return D == 128 ? 4 * q + (k ^ (q >> 1)) : 2 * q + (k ^ (q >> 2));
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4],
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "r"(addr)
               : "memory");
  return v;
}

// First row position, last key that a row of the queries [s0, s1] sees, and
// the first key that one may see (local blocks only).
struct Span {
  int lo, hi;  // keys lo .. hi (hi < lo: none)
};
__device__ __forceinline__ Span span_of(const BlockAttnQ8 &p, int b, int s0,
                                        int s1) {
  const long long first = row_pos(p.q_pos, b, s0);
  const long long last = row_pos(p.q_pos, b, s1);
  Span r;
  r.hi = last < 0 ? -1 : (int)min(last, (long long)p.T - 1);
  const long long blk = ((max(first, 0ll) >> p.lb) - p.local + 1) << p.lb;
  r.lo = (int)min(max(blk, 0ll), (long long)p.T);
  return r;
}

// Steps that an item of sequence b may take: what slices are cut by.
// (2^shift steps count as one.)
__device__ __forceinline__ unsigned steps_bound(const BlockAttnQ8 &p,
                                                const StepPlan &pl, int b,
                                                int shift) {
  const Span r = span_of(p, b, 0, p.S - 1);
  int keys = r.hi + 1 - (pl.all ? r.lo : 0);
  if (!pl.all) keys = min(keys, (p.topk + p.local) << p.lb);
  return ((unsigned)max(keys - 1, 0) >> (5 + shift)) + 1u;
}

template <int D, int MT>
__global__ void __launch_bounds__(kThreads, 1)
    attn_q8_step_kernel(const __grid_constant__ Maps8 maps,
                        const __grid_constant__ BlockAttnQ8 p,
                        const __grid_constant__ StepPlan pl) {
  using L = StepSmem<D, MT>;
  constexpr int kRows = 16 * MT;
  const float neg_inf = -__int_as_float(0x7f800000);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t *smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  const int NS = pl.stages;
  uint8_t *at = smem + NS * kWarps * L::kStage;
  float *sums = reinterpret_cast<float *>(at);
  at += L::kSum;
  Rows<D, MT> *rows_of_entry = reinterpret_cast<Rows<D, MT> *>(at);  // [2]
  at += 2 * sizeof(Rows<D, MT>);
  Sub *subs = reinterpret_cast<Sub *>(at);
  at += NS * kWarps * 2 * sizeof(Sub);
  Entry *entries = reinterpret_cast<Entry *>(at);  // [2]
  Entry *waiting = entries + 2;                    // [2], see below
  at += 4 * sizeof(Entry);
  float *row_m = reinterpret_cast<float *>(at);  // [warp][kRows]
  float *row_l = row_m + kWarps * kRows;
  at += 2 * kWarps * kRows * 4;
  float *qs = reinterpret_cast<float *>(at) + (threadIdx.x >> 5) % kWarps * 128;
  at += kWarps * 512;
  const uint32_t bars = smem_u32(at);
  at += NS * kWarps * 16;
  volatile int *abort_flag = reinterpret_cast<int *>(at);
  int *joined = reinterpret_cast<int *>(at + 8);  // [2]
  const uint32_t item_bars = smem_u32(at + 16);
  at += 128;
  uint32_t *bitmap = reinterpret_cast<uint32_t *>(at);
  uint16_t *list = reinterpret_cast<uint16_t *>(bitmap + (p.nblk + 31) / 32);
  auto full = [&](int w, int st) { return bars + (w * NS + st) * 16; };
  auto empty = [&](int w, int st) { return bars + (w * NS + st) * 16 + 8; };
  auto item_full = [&](int e) { return item_bars + e * 16; };
  auto item_empty = [&](int e) { return item_bars + e * 16 + 8; };
  auto stage = [&](int w, int st) {
    return smem_u32(smem) + (w * NS + st) * L::kStage;
  };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < NS * kWarps; ++i) {
      mbar_init(bars + i * 16, 1);
      mbar_init(bars + i * 16 + 8, 1);
    }
    for (int e = 0; e < 2; ++e) {
      mbar_init(item_full(e), kFeeders);
      mbar_init(item_empty(e), kWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
  }
  __syncthreads();

  if (warp >= kWarps) {
    // ---------------- the warps that load ----------------
    // Each serves some of the others; all walk the slice together.
    constexpr int kServe = kWarps / kFeeders;
    const int fw = warp - kWarps, ft = tid - kWarps * 32;
    regs_fewer<feeder_regs(MT)>();
    // the sequences' steps, and this CTA's slice of them all: [u0, u1)
    const int per = (p.B + 31) / 32;
    int shift = 0;
    unsigned mine, all, before;
    for (;; ++shift) {  // (sums below 2^31: steps are counted by two, four ..)
      unsigned long long sum = 0;
      for (int b = lane * per; b < min(p.B, lane * per + per); ++b)
        sum += (unsigned long long)steps_bound(p, pl, b, shift) *
               (unsigned)pl.items_b;
      unsigned long long upto = sum;
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
      }
      const unsigned long long t = __shfl_sync(0xffffffffu, upto, 31);
      mine = (unsigned)sum, before = (unsigned)(upto - sum), all = (unsigned)t;
      if (t < (1ull << 31) || shift == 16) break;
    }
    const unsigned ctas = min(gridDim.x, max(all / kMinSteps, 1u));
    const unsigned share = all / ctas, more = all % ctas;
    // all c / ctas, rounded down.  (The first slices one longer than the rest
    // would put whole pages between CTAs now and then, all of them at one place
    // of their pages: 131072 keys of one sequence took 60 us instead of 53.)
    auto begin_of = [&](unsigned c) { return c * share + c * more / ctas; };
    const unsigned cta = blockIdx.x;
    const unsigned u0 = cta < ctas ? begin_of(cta) : all;
    const unsigned u1 = cta < ctas ? begin_of(cta + 1) : all;
    // the CTA that holds step u of them all
    auto holder = [&](unsigned u) {
      int c = (int)((float)u / (float)all * (float)ctas);
      c = min(c, (int)ctas - 1);
      while (c > 0 && begin_of(c) > u) --c;
      while (c + 1 < (int)ctas && begin_of(c + 1) <= u) ++c;
      return c;
    };
    int b = 0;
    unsigned w = u0, w_b = 0;  // position, and where sequence b begins
    if (u0 < u1) {
      const unsigned here =
          __ballot_sync(0xffffffffu, before <= u0 && u0 - before < mine);
      const int src = __ffs(here) - 1;
      b = src * per;
      w_b = __shfl_sync(0xffffffffu, before, src);
    }
    int entry = 0, g0 = 0;  // items, and steps before this item's
    bool bad = false, ok = true;
    while (w < u1) {
      const unsigned U = steps_bound(p, pl, b, shift);
      if (w - w_b >= U * pl.items_b) {
        w_b += U * pl.items_b;
        ++b;
        continue;
      }
      const int idx = (int)((w - w_b) / U);
      const unsigned w_i = w_b + idx * U;
      const unsigned x0 = w - w_i, x1 = min(U, x0 + (u1 - w));
      w += x1 - x0;
      const int hk = idx % p.Hk;
      const int s = idx / p.Hk;  // (0 without a selection)
      // the item's keys: units of `box` keys
      Span sp;
      int units;
      if (pl.all) {
        sp = span_of(p, b, 0, p.S - 1);
        units = max(0, sp.hi - sp.lo + pl.box) / pl.box;
      } else {
        // (the list of the item before has been read by all)
        if (named_bar_or(2, kFeeders * 32, !ok)) break;
        sp = span_of(p, b, s, s);
        const long long pos = row_pos(p.q_pos, b, s);
        const int32_t *ids = row_ids(p, b, s, hk);
        const int words = (p.nblk + 31) / 32, n_cand = p.topk + p.local;
        for (int i = ft; i < words; i += kFeeders * 32) bitmap[i] = 0u;
        named_bar_sync(2, kFeeders * 32);
        for (int i = ft; i < n_cand; i += kFeeders * 32) {
          const int n = candidate(p, ids, pos, i, bad);
          if (n >= 0) atomicOr(bitmap + (n >> 5), 1u << (n & 31));
        }
        named_bar_sync(2, kFeeders * 32);
        // ascending; every warp counts, the first one writes
        int count = 0;
        for (int i0 = 0; i0 < words; i0 += 32) {
          uint32_t m = i0 + lane < words ? bitmap[i0 + lane] : 0u;
          const int mn = __popc(m);
          int to = mn;
          for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, to, o);
            if (lane >= o) to += x;
          }
          const int sum = __shfl_sync(0xffffffffu, to, 31);
          to += count - mn;
          if (fw == 0)
            for (; m; m &= m - 1)
              list[to++] = (uint16_t)((i0 + lane) * 32 + __ffs(m) - 1);
          count += sum;
        }
        named_bar_sync(2, kFeeders * 32);
        units = count << (p.lb - (pl.box == 32 ? 5 : 4));
      }
      const int per_step = kKeys / pl.box;
      const unsigned steps = (units + per_step - 1) / per_step;
      // (below 2^32: an item has at most 2^16 steps)
      const int t0 = (int)(steps * x0 / U);
      const int t1 = (int)(x1 == U ? steps : steps * x1 / U);
      const int g1 = g0 + t1 - t0;
      // the queries of the first 16 rows, on the way
      const int gq = lane >> 2, tq = lane & 3;
      uint4 raw[2][D / 32];
      auto row_of = [&](int r, int &rs, int &rh) {
        rh = hk * p.G + r % p.G;
        rs = s + r / p.G;
        return r < pl.rows;
      };
      auto fetch = [&](int mt) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          int rs, rh;
          const bool live = row_of(mt * 16 + gq + 8 * i, rs, rh);
          const uint4 *src = reinterpret_cast<const uint4 *>(
              p.q + (((long long)rs * p.B + b) * p.H + rh) * D + 16 * tq);
#pragma unroll
          for (int c = 0; c < D / 32; ++c)  // elements 64 c/2 + 16 tq ..
            raw[i][c] = live ? __ldg(src + (c >> 1) * 8 + (c & 1))
                             : make_uint4(0u, 0u, 0u, 0u);
        }
      };
      fetch(0);

      // 16 steps of this warp's at a time: lane 2 i + j holds the 16 keys j of
      // the i-th; those of steps are g = 8 n + kServe fw + 0, 1
      auto step_of = [&](int k) {
        return (k / kServe) * kWarps + fw * kServe + k % kServe;
      };
      struct Look {
        int page, off, j0, seen;
        float ks, vs;
      };
      const int k0 = g0 / kWarps * kServe;
      const int k1 = (g1 + kWarps - 1) / kWarps * kServe;
      auto look = [&](int k) {
        Look r{-1, 0, 0, 0, 1.f, 1.f};
        const int g = step_of(k + (lane >> 1)), sub = lane & 1;
        if (g < g0 || g >= g1) return r;
        const int step = t0 + g - g0;
        const int unit = pl.box == 32 ? step : 2 * step + sub;
        if (unit >= units) return r;
        if (pl.all) {
          r.j0 = sp.lo + step * kKeys + sub * 16;
        } else {
          const int sh = p.lb - (pl.box == 32 ? 5 : 4);
          r.j0 = ((int)list[unit >> sh] << p.lb) +
                 (unit & ((1 << sh) - 1)) * pl.box +
                 (pl.box == 32 ? sub * 16 : 0);
        }
        r.seen = min(max(sp.hi - r.j0 + 1, 0), 16);
        if (r.seen == 0) return r;
        const int pg = r.j0 / p.page_size;
        r.off = r.j0 - pg * p.page_size;
        r.page = __ldg(p.table + (long long)b * p.max_pages + pg);
        if (r.page < 0 || r.page >= p.num_pages) {
          bad = true;
          r.seen = 0;
          r.page = -1;
        } else {
          const long long sa = q8_scale_at(p.c, r.page, r.off, hk);
          r.ks = __ldg(p.c.ks + sa);
          r.vs = __ldg(p.c.vs + sa);
        }
        return r;
      };
      Look next = look(k0);
      // tell the others: the item, and its rows
      ok = __all_sync(0xffffffffu,
                      ok && wait_bar_inl(item_empty(entry & 1),
                                         (entry >> 1 & 1) ^ 1, abort_flag,
                                         p.status));
      if (ok) {
        Rows<D, MT> &rw = rows_of_entry[entry & 1];
        if (fw == 0 && lane == 0) {
          Entry &e = entries[entry & 1];
          e.n = t1 - t0;
          e.g0 = g0;
          e.b = b, e.hk = hk, e.s = s;
          e.slot = x0 == 0 && x1 == U ? -1 : x0 == 0 ? 1 : 0;
          e.c0 = e.c1 = (int)cta;
          if (e.slot >= 0) {
            e.c0 = x0 == 0 ? (int)cta : holder(w_i);
            e.c1 = x1 == U ? (int)cta : holder(w_i + U - 1);
          }
        }
        for (int r = fw * 32 + lane; r < kRows; r += kFeeders * 32) {
          int rs, rh;
          const bool live = row_of(r, rs, rh);
          const long long ps = live ? row_pos(p.q_pos, b, rs) : -1;
          rw.pos[r] = ps < 0 ? -1 : (int)min(ps, (long long)p.T - 1);
          rw.lo[r] = pl.all && live
                         ? (int)min(max(((ps >> p.lb) - p.local + 1) << p.lb,
                                        0ll),
                                    (long long)p.T)
                         : 0;
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          if (mt > 0) fetch(mt);
          float f[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float top = 0.f;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              const uint32_t u[4] = {raw[i][c].x, raw[i][c].y, raw[i][c].z,
                                     raw[i][c].w};
#pragma unroll
              for (int k = 0; k < 4; ++k)
                top = fmaxf(top, fmaxf(fabsf(__uint_as_float(u[k] << 16)),
                                       fabsf(__uint_as_float(u[k] & 0xffff0000u))));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // the largest value to [2^14, 2^15), whatever finite value it is
            int eq = (__float_as_int(top) >> 23) - 127 - 14;
            eq = max(eq, -100);
            f[i] = q8_pow2(-eq);
            if (fw == 0 && tq == 0)
              rw.cr[mt * 16 + gq + 8 * i] =
                  p.scale * 1.4426950408889634f * q8_pow2(eq);
          }
          // operand ks: elements 64 (ks / 4) + 16 tq + 4 (ks % 4) .. + 3; two
          // words of piece ks / 2
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            if (ks % kFeeders != fw) continue;
            uint32_t a[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint4 &v = raw[i][ks >> 1];
              const uint32_t w0 = ks & 1 ? v.z : v.x, w1 = ks & 1 ? v.w : v.y;
              a[i] = pack_half2(__uint_as_float(w0 << 16) * f[i],
                                __uint_as_float(w0 & 0xffff0000u) * f[i]);
              a[2 + i] = pack_half2(__uint_as_float(w1 << 16) * f[i],
                                    __uint_as_float(w1 & 0xffff0000u) * f[i]);
            }
            rw.q[ks][mt][lane] = make_uint4(a[0], a[1], a[2], a[3]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(item_full(entry & 1));
      }
      ++entry;
      for (int k = k0; ok && k < k1; k += 16) {
        const Look cur = next;
        if (k + 16 < k1) next = look(k + 16);
        const Sub sub_s{q8_exp(cur.ks), q8_exp(cur.vs), cur.j0, cur.seen};
        for (int i = 0; i < 16; ++i) {
          const int g = step_of(k + i);
          if (g < g0) continue;
          if (g >= g1) break;
          const int wp = g % kWarps, turn = g / kWarps;
          const int st = turn % NS;
          if (!__all_sync(0xffffffffu,
                          wait_bar_inl(empty(wp, st), (turn / NS & 1) ^ 1,
                                   abort_flag, p.status))) {
            ok = false;
            break;
          }
          // lanes 2 i and 2 i + 1 hold this step's keys
          const unsigned there = __ballot_sync(0xffffffffu, cur.page >= 0);
          const bool here = (lane >> 1) == i;
          if (here) subs[(wp * NS + st) * 2 + (lane & 1)] = sub_s;
          const unsigned two = there >> (2 * i) & 3u;
          const int n_box = pl.box == 32 ? (two & 1u) * 2 : __popc(two);
          __syncwarp();
          if (lane == 2 * i)
            mbar_arrive_expect_tx(full(wp, st), n_box * 2 * 16 * D);
          __syncwarp();
          if (here && cur.page >= 0 && (pl.box == 16 || lane == 2 * i)) {
            const uint32_t dst = stage(wp, st) + (lane & 1) * 16 * D;
            tma_load_4d(dst, &maps.k, full(wp, st), 0, cur.off, hk, cur.page);
            tma_load_4d(dst + kKeys * D, &maps.v, full(wp, st), 0, cur.off, hk,
                        cur.page);
          }
        }
      }
      g0 = g1;
      if (pl.all && !ok) break;
    }
    if (bad) atomicOr(p.status, kStatusIndexRange);
    // no more
    if (ok && __all_sync(0xffffffffu,
                         wait_bar_inl(item_empty(entry & 1),
                                      (entry >> 1 & 1) ^ 1, abort_flag,
                                      p.status))) {
      if (lane == 0) {
        if (fw == 0) entries[entry & 1].n = -1;
        mbar_arrive(item_full(entry & 1));
      }
    }
  } else {
    // ---------------- the warps that multiply ----------------
    regs_more<mul_regs(MT)>();
    const int gq = lane >> 2, tq = lane & 3;
    // Joins the parts of an item that several CTAs share: the one that finished
    // last, o = sum_i w_i o_i / sum_i w_i with w_i = 2^(l_i - max).
    auto join_item = [&](const Entry &e) {
      const int parts = e.c1 - e.c0 + 1;
      const int live = pl.rows;
      constexpr int kLanes = D / 4;  // threads of a row: a warp or half of one
      const int c = tid % kLanes;
      // (whole warps stay in the loop: they vote)
      for (int r0 = tid / 32 * (32 / kLanes); r0 < live;
           r0 += kWarps * 32 / kLanes) {
        const int r = r0 + lane / kLanes;
        const bool mine = r < live;
        float M = neg_inf, sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        bool again = false;
        for (int i0 = 0; i0 < parts; i0 += 8) {
          float ls[8];
          float4 v[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int i = min(i0 + u, parts - 1);
            const size_t a = ((size_t)(e.c0 + i) * 2 + (i == 0 ? 1 : 0)) * 32 +
                             (mine ? r : 0);
            ls[u] = __ldcg(pl.part_l + a);
            v[u] = __ldcg(
                reinterpret_cast<const float4 *>(pl.part_o + a * D) + c);
            if (i0 + u >= parts) ls[u] = neg_inf;
          }
          float mx = M;
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            again |= __float_as_int(ls[u]) == kAgain;
            mx = fmaxf(mx, ls[u]);
          }
          const float ref = mx > neg_inf ? mx : 0.f;
          const float f = ex2(M - ref);
          sum *= f, acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f;
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const float wt = ex2(ls[u] - ref);
            sum += wt;
            acc.x = fmaf(wt, v[u].x, acc.x);
            acc.y = fmaf(wt, v[u].y, acc.y);
            acc.z = fmaf(wt, v[u].z, acc.z);
            acc.w = fmaf(wt, v[u].w, acc.w);
          }
          M = mx;
        }
        const int s = e.s + r / p.G, h = e.hk * p.G + r % p.G;
        const long long to = ((long long)s * p.B + e.b) * p.H + h;
        if (mine) {
          const bool some = sum > 0.f || sum != sum;
          const float inv = some ? 1.f / sum : 0.f;
          reinterpret_cast<uint2 *>(p.o + to * D)[c] =
              make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv),
                         pack_bf16x2(acc.z * inv, acc.w * inv));
          if (c == 0)
            p.lse[to] =
                some ? (M + log2f(sum)) * 0.69314718055994531f : neg_inf;
        }
        // rows with a part that says so
        unsigned odd = __ballot_sync(0xffffffffu, mine && again && c == 0);
        for (; odd; odd &= odd - 1) {
          const int src = __ffs(odd) - 1;
          redo_row_q8<D>(p, e.b, __shfl_sync(0xffffffffu, s, src),
                         __shfl_sync(0xffffffffu, h, src), qs, lane);
        }
      }
    };
    // A shared item's part is counted when all have come to the next item, and
    // joined, if it was the last, at that one's end: its count is on the way
    // meanwhile.
    bool shared_item = false;
    for (int entry = 0;; ++entry) {
      const bool got = __all_sync(
          0xffffffffu, wait_bar_inl(item_full(entry & 1), entry >> 1 & 1,
                                    abort_flag, p.status));
      // (all stop together; and the item before has left shared memory)
      if (named_bar_or(1, kWarps * 32, !got)) break;
      const Entry e = entries[entry & 1];
      if (shared_item && warp == (entry & (kWarps - 1))) {
        if (lane == 0) {
          const Entry &was = waiting[(entry - 1) & 1];
          const int sh = 8 * (was.c0 & 3);
          uint32_t *word = pl.done + (was.c0 >> 2);
          __threadfence();  // the CTA's parts, before the count
          const uint32_t had = atomicAdd(word, 1u << sh) >> sh & 0xffu;
          const bool last = had == (uint32_t)(was.c1 - was.c0);
          if (last) atomicAnd(word, ~(0xffu << sh));  // for the next call
          __threadfence();
          joined[entry & 1] = last;
        }
        __syncwarp();
      }
      if (e.n < 0) {
        if (shared_item) {
          named_bar_sync(1, kWarps * 32);
          if (joined[entry & 1]) join_item(waiting[(entry - 1) & 1]);
        }
        break;
      }
      // this thread's rows: gq and gq + 8 of each 16
      const Rows<D, MT> &rw = rows_of_entry[entry & 1];
      int pos[MT][2], lo[MT][2];
      float cr[MT][2];
      uint32_t qr[MT == 1 ? D / 16 : 1][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = mt * 16 + gq + 8 * i;
          pos[mt][i] = rw.pos[r], lo[mt][i] = rw.lo[r], cr[mt][i] = rw.cr[r];
        }
      if constexpr (MT == 1) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint4 v = rw.q[ks][0][lane];
          qr[ks][0] = v.x, qr[ks][1] = v.y, qr[ks][2] = v.z, qr[ks][3] = v.w;
        }
      }
      const int live = pl.rows;
      const bool mixed = pl.all && p.S > 1;  // rows that see different keys
      // the tile's rows see the same keys but where a step holds keys after
      // the first row's position or before the last row's first block
      int pos_lo = 0x7fffffff, lo_hi = 0;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (mt * 16 + gq + 8 * i < live) pos_lo = min(pos_lo, pos[mt][i]);
          lo_hi = max(lo_hi, lo[mt][i]);
        }
      pos_lo = __reduce_min_sync(0xffffffffu, pos_lo);
      lo_hi = __reduce_max_sync(0xffffffffu, lo_hi);

      float o[MT][D / 8][4] = {};
      float m[MT][2], l[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
        m[mt][0] = m[mt][1] = neg_inf, l[mt][0] = l[mt][1] = 0.f;
      const int g1 = e.g0 + e.n;
      int g = e.g0 + (warp - e.g0 % kWarps + kWarps) % kWarps;
      bool ok = true;
      for (; ok && g < g1; g += kWarps) {
        const int turn = g / kWarps, st = turn % NS;
        if (!__all_sync(0xffffffffu, wait_bar_inl(full(warp, st), turn / NS & 1,
                                              abort_flag, p.status))) {
          ok = false;
          break;
        }
        const uint32_t sk = stage(warp, st), sv = sk + kKeys * D;
        const Sub sub[2] = {subs[(warp * NS + st) * 2],
                            subs[(warp * NS + st) * 2 + 1]};
        // ---- scores: four tiles of 8 keys ----
        float x[MT][4][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[mt][n][j] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint4 kw[4];
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const int r = 8 * n + (gq ^ ((gq & 1) << 2));
            const int ch = c * 4 + tq;
            kw[n] = lds128(sk + r * D +
                           ((D == 128 ? ch ^ (r & 7) : ch ^ (r >> 1 & 3)) << 4));
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t a[MT][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              if constexpr (MT == 1) {
#pragma unroll
                for (int i = 0; i < 4; ++i) a[mt][i] = qr[c * 4 + j][i];
              } else {
                const uint4 v = rw.q[c * 4 + j][mt][lane];
                a[mt][0] = v.x, a[mt][1] = v.y, a[mt][2] = v.z, a[mt][3] = v.w;
              }
            }
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              const uint32_t wd = j == 0   ? kw[n].x
                                  : j == 1 ? kw[n].y
                                  : j == 2 ? kw[n].z
                                           : kw[n].w;
              uint32_t b0, b1;
              q8_half4(wd, b0, b1);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) mma_f16(x[mt][n], a[mt], b0, b1);
            }
          }
        }
        // ---- softmax ----
        uint32_t pa[MT][2][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          float mx[2] = {neg_inf, neg_inf};
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float sc = q8_pow2(sub[u].ek), ev = (float)sub[u].ev;
            const float a0 = cr[mt][0] * sc, a1 = cr[mt][1] * sc;
            const bool some = sub[u].seen < 16 || sub[u].j0 + 15 > pos_lo ||
                              sub[u].j0 < lo_hi;
#pragma unroll
            for (int n = 2 * u; n < 2 * u + 2; ++n) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                x[mt][n][j] = fmaf(x[mt][n][j], j < 2 ? a0 : a1, ev);
              if (some) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const int key = 8 * (n & 1) + ((2 * tq + (j & 1)) ^
                                                 ((j & 1) << 2));
                  const int jj = sub[u].j0 + key;
                  const bool sees = key < sub[u].seen &&
                                    jj <= pos[mt][j >> 1] &&
                                    jj >= lo[mt][j >> 1];
                  x[mt][n][j] = sees ? x[mt][n][j] : neg_inf;
                }
              }
              mx[0] = fmaxf(mx[0], fmaxf(x[mt][n][0], x[mt][n][1]));
              mx[1] = fmaxf(mx[1], fmaxf(x[mt][n][2], x[mt][n][3]));
            }
          }
          bool move = false;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
            move |= mx[i] > m[mt][i] + 14.f;
          }
          if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const bool mv = mx[i] > m[mt][i] + 14.f;
              const float to = mx[i] - 6.f;
              const float f = mv ? ex2(m[mt][i] - to) : 1.f;
              if (mv) m[mt][i] = to;
              l[mt][i] *= f;
#pragma unroll
              for (int n = 0; n < D / 8; ++n) {
                o[mt][n][2 * i] *= f;
                o[mt][n][2 * i + 1] *= f;
              }
            }
          }
          const float mu0 = m[mt][0] > neg_inf ? m[mt][0] : 0.f;
          const float mu1 = m[mt][1] > neg_inf ? m[mt][1] : 0.f;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              float *v = x[mt][2 * u + n];
              v[0] = ex2(v[0] - mu0), v[1] = ex2(v[1] - mu0);
              v[2] = ex2(v[2] - mu1), v[3] = ex2(v[3] - mu1);
              s0 += v[0] + v[1];
              s1 += v[2] + v[3];
              pa[mt][u][2 * n] = pack_half2(v[0], v[1]);
              pa[mt][u][2 * n + 1] = pack_half2(v[2], v[3]);
            }
            const float un = q8_pow2(-sub[u].ev);
            l[mt][0] = fmaf(s0, un, l[mt][0]);
            l[mt][1] = fmaf(s1, un, l[mt][1]);
          }
        }
        // ---- O += P V, 16 keys at a time ----
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          constexpr int W = D / 32;  // 32-bit words of a key that a thread has
          uint32_t vw[4][W];
#pragma unroll
          for (int r4 = 0; r4 < 4; ++r4) {
            const int key = 8 * (r4 >> 1) + ((2 * tq + (r4 & 1)) ^
                                             ((r4 & 1) << 2));
            const int r = 16 * u + key;
            if constexpr (D == 128) {
              const uint4 v = lds128(sv + r * D + ((gq ^ (r & 7)) << 4));
              vw[r4][0] = v.x, vw[r4][1] = v.y;
              vw[r4][2] = v.z, vw[r4][3] = v.w;
            } else {
              const uint2 v = lds64(sv + r * D +
                                    ((gq >> 1 ^ (r >> 1 & 3)) << 4) +
                                    (gq & 1) * 8);
              vw[r4][0] = v.x, vw[r4][1] = v.y;
            }
            if (sub[u].seen < 16 && key >= sub[u].seen) {
#pragma unroll
              for (int i = 0; i < W; ++i) vw[r4][i] = 0u;
            }
          }
#pragma unroll
          for (int i = 0; i < W; ++i) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              // elements 2 h and 2 h + 1 of word i: keys' bytes side by side
              const uint32_t sel = h ? 0x7362u : 0x5140u;
              const uint32_t w0 = __byte_perm(vw[0][i], vw[1][i], sel);
              const uint32_t w1 = __byte_perm(vw[2][i], vw[3][i], sel);
              uint32_t b00, b01, b10, b11;
              q8_half4(w0, b00, b10);
              q8_half4(w1, b01, b11);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                mma_f16(o[mt][i * 4 + 2 * h], pa[mt][u], b00, b01);
                mma_f16(o[mt][i * 4 + 2 * h + 1], pa[mt][u], b10, b11);
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty(warp, st));
      }
      // ---------------- the item's end ----------------
      // the warps' outputs side by side; one barrier, then 16 threads a row
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        if (mt > 0) named_bar_sync(1, kWarps * 32);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float t = l[mt][i];
          t += __shfl_xor_sync(0xffffffffu, t, 1);
          t += __shfl_xor_sync(0xffffffffu, t, 2);
          const int r = gq + 8 * i;
          if (tq == 0) {
            row_m[warp * kRows + mt * 16 + r] = m[mt][i];
            row_l[warp * kRows + mt * 16 + r] = t;
          }
          // columns 2 tq and 2 tq + 1 of tile n are element n of the runs 2 tq
          // and 2 tq + 1
          if (mt * 16 + r < live) {
            float4 *dst = reinterpret_cast<float4 *>(
                sums + (warp * 16 + r) * L::kPitch);
#pragma unroll
            for (int cc = 0; cc < 2; ++cc)
#pragma unroll
              for (int k = 0; k < D / 32; ++k)
                dst[run_at<D>(2 * tq + cc, k)] = make_float4(
                    o[mt][4 * k][2 * i + cc], o[mt][4 * k + 1][2 * i + cc],
                    o[mt][4 * k + 2][2 * i + cc], o[mt][4 * k + 3][2 * i + cc]);
          }
        }
        named_bar_sync(1, kWarps * 32);
        const int r = mt * 16 + (tid >> 4), j = tid & 15;
        const bool mine = r < live;
        float M = neg_inf, sum = 0.f, f[kWarps];
#pragma unroll
        for (int i = 0; i < kWarps; ++i)
          M = fmaxf(M, row_m[i * kRows + r]);
        const float mu = M > neg_inf ? M : 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
          f[i] = ex2(row_m[i * kRows + r] - mu);
          sum = fmaf(row_l[i * kRows + r], f[i], sum);
        }
        const bool some = sum > 0.f || sum != sum;
        const float inv = some ? 1.f / sum : 0.f;
        constexpr int kPer = D / 64;  // 16-byte pieces of a thread
        float4 acc[kPer];
        bool odd = sum != sum || sum > 3e38f;
        if (mine) {
#pragma unroll
          for (int k = 0; k < kPer; ++k) {
            acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            const int piece = j * kPer + k;  // of the row
            const int at4 = run_at<D>(piece / (D / 32), piece % (D / 32));
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
              const float4 v = reinterpret_cast<const float4 *>(
                  sums + (i * 16 + (tid >> 4)) * L::kPitch)[at4];
              acc[k].x = fmaf(v.x, f[i], acc[k].x);
              acc[k].y = fmaf(v.y, f[i], acc[k].y);
              acc[k].z = fmaf(v.z, f[i], acc[k].z);
              acc[k].w = fmaf(v.w, f[i], acc[k].w);
            }
            acc[k].x *= inv, acc[k].y *= inv, acc[k].z *= inv, acc[k].w *= inv;
            if (!some) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            const float top = fmaxf(fmaxf(fabsf(acc[k].x), fabsf(acc[k].y)),
                                    fmaxf(fabsf(acc[k].z), fabsf(acc[k].w)));
            odd |= !(top <= 3e38f) || acc[k].x != acc[k].x ||
                   acc[k].y != acc[k].y || acc[k].z != acc[k].z ||
                   acc[k].w != acc[k].w;
          }
        }
        odd &= mixed || rw.cr[r] > kMostFactor;
        const unsigned votes = __ballot_sync(0xffffffffu, mine && odd);
        odd = (votes >> (lane & 16) & 0xffffu) != 0u;  // any of the row's
        const float lse2 = some ? M + log2f(sum) : neg_inf;
        const int s = e.s + r / p.G, h = e.hk * p.G + r % p.G;
        const long long to = ((long long)s * p.B + e.b) * p.H + h;
        if (mine && e.slot < 0) {
#pragma unroll
          for (int k = 0; k < kPer; ++k)
            reinterpret_cast<uint2 *>(p.o + to * D)[j * kPer + k] =
                make_uint2(pack_bf16x2(acc[k].x, acc[k].y),
                           pack_bf16x2(acc[k].z, acc[k].w));
          if (j == 0) p.lse[to] = lse2 * 0.69314718055994531f;
        } else if (mine) {
          const size_t part =
              ((size_t)blockIdx.x * 2 + (e.slot > 0 ? 1 : 0)) * 32 + r;
#pragma unroll
          for (int k = 0; k < kPer; ++k)
            reinterpret_cast<float4 *>(pl.part_o + part * D)[j * kPer + k] =
                acc[k];
          if (j == 0)
            pl.part_l[part] = __int_as_float(
                odd            ? kAgain
                : lse2 != lse2 ? 0x7fffffff
                               : __float_as_int(lse2));
        }
        if (e.slot < 0) {
          unsigned again = __ballot_sync(0xffffffffu, mine && odd && j == 0);
          for (; again; again &= again - 1) {
            const int src = __ffs(again) - 1;
            redo_row_q8<D>(p, e.b, __shfl_sync(0xffffffffu, s, src),
                           __shfl_sync(0xffffffffu, h, src), qs, lane);
          }
        }
      }
      // (its count came before the barrier above)
      if (shared_item && joined[entry & 1]) join_item(waiting[(entry - 1) & 1]);
      shared_item = e.slot >= 0;
      if (tid == 0) waiting[entry & 1] = e;
      __syncwarp();
      if (lane == 0) mbar_arrive(item_empty(entry & 1));
    }
  }
}

template <int D, int MT>
int launch(const BlockAttnQ8 &p, StepPlan &pl, const Maps8 &maps, int ctas,
           cudaStream_t st) {
  using L = StepSmem<D, MT>;
  auto kern = attn_q8_step_kernel<D, MT>;
  // as many stages as there is room for beside the block list (two at 128
  // dimensions hold 128 KB; three are no faster)
  for (pl.stages = D == 64 ? 4 : 2;; --pl.stages) {
    if (L::bytes(pl.stages, p.nblk, pl.cap) <= kMaxSmem) break;
    if (pl.stages == 1) return DSA_ERR_UNSUPPORTED;
  }
  if (allow_smem(kern, kMaxSmem) != cudaSuccess) return DSA_ERR_CUDA;
  kern<<<ctas, kThreads, L::bytes(pl.stages, p.nblk, pl.cap), st>>>(maps, p,
                                                                    pl);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace

size_t attn_q8_step_workspace_bytes(int D) {
  return 256 + (size_t)kMaxCtas * 2 * 32 * (D + 1) * sizeof(float);
}

// Rows that share keys: up to 16, or 32 of all keys at 64 dimensions.
int run_attn_q8_step(const BlockAttnQ8 &p, void *workspace, int num_sms,
                     cudaStream_t st) {
  StepPlan pl{};
  pl.all = p.topk == 0;
  pl.rows = pl.all ? p.S * p.G : p.G;
  const int mt = pl.rows > 16 ? 2 : 1;
  const long long items = (long long)p.Hk * (pl.all ? 1 : p.S);
  if (items * p.B >= (1ll << 31)) return DSA_ERR_UNSUPPORTED;
  pl.items_b = (int)items;
  pl.box = p.blk >= 32 ? 32 : 16;
  if (!pl.all) {
    const long long most = (long long)p.topk + p.local;
    pl.cap = (int)(most < p.nblk ? most : p.nblk);
  }
  char *ws = static_cast<char *>(workspace);
  pl.done = reinterpret_cast<uint32_t *>(ws + kDoneOffset);
  pl.part_l = reinterpret_cast<float *>(ws + 256);
  pl.part_o = pl.part_l + kMaxCtas * 2 * 32;
  Maps8 maps;
  const Q8Cache &c = p.c;
  int rc = encode_kv8(&maps.k, c.k, p.D, pl.box, c.page_size, c.k_t, p.Hk,
                      c.k_h, c.num_pages, c.k_p);
  if (rc != DSA_OK) return rc;
  rc = encode_kv8(&maps.v, c.v, p.D, pl.box, c.page_size, c.v_t, p.Hk, c.v_h,
                  c.num_pages, c.v_p);
  if (rc != DSA_OK) return rc;
  const int ctas = num_sms < kMaxCtas ? num_sms : kMaxCtas;
  if (p.D == 64)
    return mt == 1 ? launch<64, 1>(p, pl, maps, ctas, st)
                   : launch<64, 2>(p, pl, maps, ctas, st);
  return mt == 1 ? launch<128, 1>(p, pl, maps, ctas, st)
                 : DSA_ERR_UNSUPPORTED;
}

}  // namespace dsa
