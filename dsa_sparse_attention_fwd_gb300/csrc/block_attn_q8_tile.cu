// Attention over a paged cache held in 8 bits for many rows (chunks of a
// prompt): the query tiles of block_attn.cu, 128 rows that walk the union of
// their queries' blocks in steps of 64 keys, over e4m3 keys and values.
//
// The score product takes the keys as they lie in memory (kind::f8f6f4): a
// row's query, brought to [224, 448] by a power of two, is the sum of two e4m3
// values (4 bits each: bf16 has 8), exactly but for elements below 2^-9 of the
// row's largest, which are off by half a step of the smallest e4m3 values (2^-10,
// 2^-17 of the largest) at most.  Two 8-bit products of K =
// 32 take as long as one of 16 bits, and the keys are neither converted nor
// stored twice.  The values are: softmax weights need more than e4m3's range
// and precision, so four warps turn each step's values into fp16 (exactly) in
// shared memory, next to the softmax of the step before.
//     t_j = c q.k_j 2^ek + ev,   P_j = 2^(t_j - m),   O += P_j v_j,
//     l += P_j 2^-ev
// with the scales 2^ek, 2^ev of 16 to 128 keys: one multiply-add with other
// constants for each 16 keys, nothing more than without scales.  m is chosen so
// that P lies below 2^14: fp16 holds it to 2^-11, down to 2^-31 of the
// largest (see block_attn_q8_step.cu).
//
// Measured on one GB300 (bf16 peak 1908 TFLOP/s): 2 x 512 tokens of 32 / 8 heads
// of 128 over all of 8000 to 15800 keys 227 to 249 us, 900 TFLOP/s; 3 x 777
// tokens of 40 / 8 heads of 64, 34 blocks of 64, 294 us (the bf16 tiles: 286 to
// 302).  No unit is busy more than half of the time (tcgen05 45%, issue 51%,
// exponentials 21%, ALU 40%): a step is a chain of the score product, tensor
// memory to registers, softmax, and back, which two CTAs an SM overlap twofold.
// Leaving out one part of it in a copy gave little: the conversion 0 to 3%, the
// exponentials 8%, half the score product 1 to 3%, the maximum 2 to 4%.  Two
// threads a row were slower (322 -> 378 us: a barrier of two warps a step), and
// so were tiles cut in parts where there are one to three a CTA slot (268 ->
// 287): two CTAs at work fill an SM, the parts only add their ends.
//
// Two CTAs an SM need half of its shared memory each: at 128 dimensions there are
// 7.4 KB for 4 bytes a block that the table can name and 2 a block of a list, at
// 64 dimensions 56 KB.  Over all keys that is up to 1236 blocks (79104 tokens of
// 64); with a table of more one CTA an SM remains, whatever the sequences'
// lengths: 2 x 512 tokens over up to 15500 keys 256 us with a table of 15872
// tokens, 259 with 65536, 408 with 131072, 417 with 1048576.
//
// Warps: 0 .. 3 softmax (thread = row = tensor-memory lane), 4 .. 7 convert the
// values, 8 TMA producer, 9 MMA issuer and tensor-memory allocator; two CTAs an
// SM.  Masks and rows that are not finite, or whose scores are above 2^25: as in
// block_attn.cu, the row path in block_attn_q8.cuh.
#include "block_attn_host.cuh"
#include "block_attn_q8.cuh"
#include "block_attn_split.cuh"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kTileThreads = 384;
constexpr int kTmaWarp = 8, kMmaWarp = 9;
// Registers of a thread: 80 at launch (two CTAs of 384 an SM), then moved
// from the warps that need few to the softmax: 152 + 56 + 32 = 3 x 80.
constexpr int kSoftRegs = 152, kConvRegs = 56, kIssueRegs = 32;
constexpr uint32_t kTmS = 0, kTmO = 128;  // tensor-memory columns
constexpr int kMeta = 8;                  // steps whose scales are held

template <int D>
struct TileSmem {
  static constexpr int kKStages = D == 128 ? 3 : 4;
  static constexpr int kVStages = 2;                   // 8-bit, and fp16
  static constexpr int kQ = kRows * D;                 // one of two parts
  static constexpr int kKey = kKeys * D;               // 8-bit K or V
  static constexpr int kV16 = kKeys * D * 2;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = 2 * kQ;
  static constexpr int kOffV8 = kOffK + kKStages * kKey;
  static constexpr int kOffV = kOffV8 + kVStages * kKey;
  static constexpr int kOffMeta = kOffV + kVStages * kV16;
  static constexpr int kOffBar = kOffMeta + kMeta * 4 * 16;
  // q_full, s_full p_full o_done (two each), then k_full k_empty, v8_full
  // v8_empty, v_full v_empty, meta_full
  static constexpr int kBars = 7 + 2 * kKStages + 4 * kVStages + kMeta;
  // Arrivals of a phase of barrier i: one for each warp where four arrive.
  static constexpr int arrivals(int i) {
    const int v8_empty = 7 + 2 * kKStages + kVStages;
    const bool four = i == 0 || i == 3 || i == 4 ||  // q_full, p_full
                      (i >= v8_empty && i < v8_empty + 2 * kVStages);  // v_full
    return four ? 4 : 1;
  }
  static constexpr int kOffMisc = kOffBar + kBars * 8;
  static constexpr int kOffWords = kOffMisc + 32;
  static constexpr int bytes(int nblk, int cap) {
    return kOffWords + nblk * 4 + ((cap * 2 + 15) & ~15) + 1024;
  }
};

// K-major operand of 8-bit rows of D bytes, swizzled over D: 128 or 64.
template <int D>
__device__ __forceinline__ uint64_t sdesc_k8(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(16u >> 4) << 16;
  d |= (uint64_t)((8u * D) >> 4) << 32;  // the next 8 rows
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)(D == 128 ? 2u : 4u) << 61;
  return d;
}

// D[tmem] (+)= A[smem] * B[smem]^T of e4m3 values, issued by one thread.
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t adesc,
                                         uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(
          d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// wait_bar_rest() without the call: kernels that move registers between warps
// (setmaxnreg) may not make one.
__device__ __forceinline__ bool wait_bar_rest_inl(uint32_t bar, uint32_t parity,
                                                  volatile int *abort_flag,
                                                  int *status) {
#pragma unroll 1
  for (int it = 0; it < 64; ++it)
    if (mbar_try_wait_ns(bar, parity, 1000000u)) return true;
  return wait_bar_loop(bar, parity, abort_flag, status);
}

// Both of two barriers, for a whole warp: asked for together, one vote where
// both are there.  (A wait with a vote of its own takes 150 cycles of a step's
// 1850 even then: the softmax's scales and scores, 322 -> 304 us for 3 x 777
// tokens; the loads' two stages, 304 -> 299.)
__device__ __forceinline__ bool wait_both(uint32_t bar0, uint32_t parity0,
                                          uint32_t bar1, uint32_t parity1,
                                          volatile int *abort_flag,
                                          int *status) {
  const bool there0 = mbar_try_wait_ns(bar0, parity0, 1000000u);
  const bool there1 = mbar_try_wait_ns(bar1, parity1, 1000000u);
  if (__all_sync(0xffffffffu, there0 && there1)) return true;
  return __all_sync(
      0xffffffffu,
      wait_bar_rest_inl(bar0, parity0, abort_flag, status) &&
          wait_bar_rest_inl(bar1, parity1, abort_flag, status));
}

// words[] of a tile without a selection: the local blocks of each query.
__device__ __forceinline__ void mark_local(const BlockAttnQ8 &p, int b, int s0,
                                           int nq, uint32_t *words, int tid,
                                           int nthreads) {
  const long long pos0 = row_pos(p.q_pos, b, s0), pos1 = pos0 + nq - 1;
  const uint32_t all = 0xffffffffu >> (32 - nq);
  const long long own0 = pos0 >> p.lb, own1 = pos1 >> p.lb;
  bool bad = false;
  for (int n = tid; n < p.nblk; n += nthreads) {
    uint32_t w = 0;
    if (pos1 >= 0 && n <= own1 && n > max(own0, 0ll) - p.local) {
      if (n <= own0 && n > own1 - p.local) {
        w = all;
      } else {
        for (int i = 0; i < nq; ++i) {
          const long long own = (pos0 + i) >> p.lb;
          if (pos0 + i >= 0 && n <= own && n > own - p.local) w |= 1u << i;
        }
      }
      if (w && block_page(p, b, n, bad) < 0) w = 0;
    }
    words[n] = w;
  }
  if (bad) atomicOr(p.status, kStatusIndexRange);
}

template <int D>
__global__ void __launch_bounds__(kTileThreads, 2)
    attn_q8_tile_kernel(const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ BlockAttnQ8 p,
                        const __grid_constant__ FwdPlan pl) {
  using L = TileSmem<D>;
  constexpr int NK = L::kKStages, NV = L::kVStages;
  // e4m3 x e4m3 -> fp32, both K-major; fp16 x fp16 -> fp32, B MN-major
  constexpr uint32_t kIdescS =
      (1u << 4) | ((uint32_t)(kKeys >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
  constexpr uint32_t kIdescO = (1u << 4) | (1u << 16) |
                               ((uint32_t)(D >> 3) << 17) |
                               ((uint32_t)(kRows >> 4) << 24);
  const float neg_inf = -__int_as_float(0x7f800000);

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (base - raw_addr);
  const uint32_t sQ = base + L::kOffQ;
  auto sK = [&](int st) { return base + L::kOffK + st * L::kKey; };
  auto sV8 = [&](int st) { return base + L::kOffV8 + st * L::kKey; };
  auto sV = [&](int st) { return base + L::kOffV + st * L::kV16; };
  const uint32_t bars = base + L::kOffBar;
  const uint32_t q_full = bars;
  auto s_full = [&](int i) { return bars + 8 + 8 * i; };
  auto p_full = [&](int i) { return bars + 24 + 8 * i; };
  auto o_done = [&](int i) { return bars + 40 + 8 * i; };
  auto k_full = [&](int i) { return bars + 56 + 8 * i; };
  auto k_empty = [&](int i) { return bars + 56 + 8 * (NK + i); };
  auto v8_full = [&](int i) { return bars + 56 + 8 * (2 * NK + i); };
  auto v8_empty = [&](int i) { return bars + 56 + 8 * (2 * NK + NV + i); };
  auto v_full = [&](int i) { return bars + 56 + 8 * (2 * NK + 2 * NV + i); };
  auto v_empty = [&](int i) { return bars + 56 + 8 * (2 * NK + 3 * NV + i); };
  auto meta_full = [&](int i) { return bars + 56 + 8 * (2 * NK + 4 * NV + i); };
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + L::kOffMisc);
  volatile int *abort_flag = reinterpret_cast<int *>(smem + L::kOffMisc + 4);
  int *sCount = reinterpret_cast<int *>(smem + L::kOffMisc + 8);
  // of 16 keys: 2^ek, ev, 2^-ev
  float4 *meta = reinterpret_cast<float4 *>(smem + L::kOffMeta);
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
    // (each once: a barrier that is one already may not be initialised again)
    for (int i = 0; i < L::kBars; ++i)
      mbar_init(bars + 8 * i, L::arrivals(i));
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(tmem_holder), 256);
    tmem_relinquish();
  }
  if (p.topk == 0) {
    mark_local(p, b, s0, nq, words, tid, kTileThreads);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  } else {
    const FirstMark first = first_mark(p, b, s0, nq, hk, tid);
    for (int n = tid; n < p.nblk; n += kTileThreads) words[n] = 0u;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    mark_blocks(p, b, s0, nq, hk, words, tid, kTileThreads, first);
    __syncthreads();
  }
  if (warp == 0) {
    const int n = list_blocks(words, p.nblk, list, lane);
    if (lane == 0) *sCount = n;
  }
  __syncthreads();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0);
  // a step takes units of up to 64 keys: whole blocks, or halves of 128
  const int count = *sCount;
  const int lu = min(p.lb, 6), lper = p.lb - lu;  // logarithms of a unit's
  const int lupt = 6 - lu;                        // keys, a block's and a
  const int units = count << lper;                // step's units
  const int all = (units + (1 << lupt) - 1) >> lupt;
  const int t0 = (int)((long long)all * split / pl.splits);
  const int t1 = (int)((long long)all * (split + 1) / pl.splits);
  const int n = t1 - t0;
  // key x (of 64) of step t's units, the last one instead of those behind it
  auto key_at = [&](int t, int x) {
    const int u = min((t << lupt) + (x >> lu), units - 1);
    return ((int)list[u >> lper] << p.lb) + ((u & ((1 << lper) - 1)) << lu) +
           (x & ((1 << lu) - 1));
  };
  // the last key that any row of the tile sees
  const int pos_hi = key_pos(p, b, s0 + nq - 1);

  if (warp >= kTmaWarp) {
    regs_fewer<kIssueRegs>();
    if (warp == kTmaWarp) {
      // ---------------- TMA producer ----------------
      // lanes 0 .. 3: 16 keys of a step each, their page and scales; the first
      // lane of a unit loads it
      struct Look {
        int page, off;
        float ks, vs;
      };
      auto look = [&](int i) {
        Look r{-1, 0, 1.f, 1.f};
        if (lane >= 4 || i >= n) return r;
        // a ragged step's end repeats the last unit's keys: their scores are
        // masked, but have to be numbers (its values become zeros)
        const int j = key_at(t0 + i, lane * 16);
        const int pg = j / p.page_size;
        r.off = j - pg * p.page_size;
        // (blocks without a page are not listed)
        r.page = __ldg(p.table + (long long)b * p.max_pages + pg);
        const long long at = q8_scale_at(p.c, r.page, r.off, hk);
        r.ks = __ldg(p.c.ks + at);
        r.vs = __ldg(p.c.vs + at);
        return r;
      };
      Look next = look(0);
      for (int i = 0; i < n; ++i) {
        const Look cur = next;
        next = look(i + 1);
        const bool loads = lane < 4 && (lane * 16 & ((1 << lu) - 1)) == 0;
        if (lane < 4) {
          const int ev = q8_exp(cur.vs);
          meta[(i % kMeta) * 4 + lane] =
              make_float4(q8_pow2(q8_exp(cur.ks)), (float)ev, q8_pow2(-ev), 0.f);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(meta_full(i % kMeta));
        // (what frees the values' stage, the conversion of step i - 2, waits
        // for nothing of step i)
        const int sk = i % NK, sv = i % NV;
        if (!wait_both(k_empty(sk), (i / NK & 1u) ^ 1u, v8_empty(sv),
                       (i / NV & 1u) ^ 1u, abort_flag, p.status))
          goto done;
        if (lane == 0) {
          mbar_arrive_expect_tx(k_full(sk), L::kKey);
          mbar_arrive_expect_tx(v8_full(sv), L::kKey);
        }
        __syncwarp();
        if (loads) {
          const uint32_t to = lane * 16 * D;
          tma_load_4d(sK(sk) + to, &tm_k, k_full(sk), 0, cur.off, hk, cur.page);
          tma_load_4d(sV8(sv) + to, &tm_v, v8_full(sv), 0, cur.off, hk,
                      cur.page);
        }
      }
    } else if (warp == kMmaWarp) {
      // ---------------- MMA issuer: one thread ----------------
      if (elect_one()) {
        auto wait = [&](uint32_t bar, uint32_t ph) -> bool {
          return wait_bar_rest_inl(bar, ph, abort_flag, p.status);
        };
        const uint64_t qd = sdesc_k8<D>(sQ);
        bool ok = wait(q_full, 0);
        auto scores = [&](int i) -> bool {
          const int st = i % NK;
          if (!wait(k_full(st), i / NK & 1u)) return false;
          tc_fence_after();
          const uint64_t kd = sdesc_k8<D>(sK(st));
#pragma unroll
          for (int ks = 0; ks < 2 * D / 32; ++ks) {
            const int part = ks / (D / 32), k = ks % (D / 32);
            mma_e4m3(tmem + kTmS + (i & 1) * 64,
                     qd + ((part * L::kQ + k * 32) >> 4), kd + (k * 32 >> 4),
                     kIdescS, ks != 0);
          }
          mma_commit(k_empty(st));
          mma_commit(s_full(i & 1));
          return true;
        };
        if (ok && n > 0) ok = scores(0);
        uint32_t acc = 0;
        for (int i = 0; ok && i < n; ++i) {
          if (i + 1 < n && !(ok = scores(i + 1))) break;
          const int st = i % NV;
          if (!(ok = wait(v_full(st), i / NV & 1u) &&
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
    }
  } else if (warp >= 4) {
    // ---------------- values to fp16 ----------------
    regs_fewer<kConvRegs>();
    const int ct = tid - 128;
    constexpr int kPer = D / 32;  // 16-byte pieces of a thread: half a row
    const int row = ct >> 1, half = ct & 1;
    // pieces of a row's half, the two halves in another order each: no bank
    // conflicts; a piece of 16 bytes becomes two of 8 fp16, 64 a row of 128
    // bytes
    uint32_t from[kPer], to[kPer][2];
#pragma unroll
    for (int c = 0; c < kPer; ++c) {
      const int ch = half * kPer + (D == 128 ? c ^ (half << 1) : c ^ half);
      from[c] = row * D + ((D == 128 ? ch ^ (row & 7) : ch ^ (row >> 1 & 3)) << 4);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int piece = ch * 2 + u;
        to[c][u] = (piece >> 3) * (kKeys * 128) + row * 128 +
                   (((piece & 7) ^ (row & 7)) << 4);
      }
    }
    for (int i = 0; i < n; ++i) {
      const int st = i % NV;
      const uint32_t ph = i / NV & 1u;
      // values that no row sees: only the last block can hold any (the others
      // lie before the last row's own), and what fills a ragged step up
      const bool zero = (t0 + i + 1) << lupt > units - (1 << lper) &&
                        (((t0 + i) << lupt) + (row >> lu) >= units ||
                         key_at(t0 + i, row) > pos_hi);
      if (!__all_sync(0xffffffffu, wait_bar_rest_inl(v8_full(st), ph, abort_flag,
                                                     p.status)))
        goto done;
      uint4 x[kPer];
#pragma unroll
      for (int c = 0; c < kPer; ++c) {
        const float4 v = ld_shared_v4f(sV8(st) + from[c]);
        x[c] = make_uint4(__float_as_uint(v.x), __float_as_uint(v.y),
                          __float_as_uint(v.z), __float_as_uint(v.w));
        if (zero) x[c] = make_uint4(0u, 0u, 0u, 0u);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(v8_empty(st));
      if (!__all_sync(0xffffffffu, wait_bar_rest_inl(v_empty(st), ph ^ 1u,
                                                     abort_flag, p.status)))
        goto done;
#pragma unroll
      for (int c = 0; c < kPer; ++c) {
        const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t h[4];
          q8_half4(w[2 * u], h[0], h[1]);
          q8_half4(w[2 * u + 1], h[2], h[3]);
          st_shared_v4(sV(st) + to[c][u], h);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(v_full(st));
    }
  } else {
    // ---------------- softmax: one row a thread ----------------
    regs_more<kSoftRegs>();
    const int row = tid;
    const int qi = row / p.G;
    const bool live = qi < nq;
    const size_t at =
        ((size_t)(s0 + qi) * p.B + b) * p.H + hk * p.G + row % p.G;
    const int pos = live ? key_pos(p, b, s0 + qi) : -1;
    const int pos_lo = key_pos(p, b, s0);  // of the tile's first row
    float cr;                              // c times the row's power of two
    {
      // the row's query as two e4m3 parts
      const uint4 *src = reinterpret_cast<const uint4 *>(p.q + at * D);
      float top = 0.f;
      uint32_t u[D / 2];
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        const uint4 v = live ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
        u[4 * c] = v.x, u[4 * c + 1] = v.y;
        u[4 * c + 2] = v.z, u[4 * c + 3] = v.w;
      }
#pragma unroll
      for (int k = 0; k < D / 2; ++k)
        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(u[k] << 16)),
                               fabsf(__uint_as_float(u[k] & 0xffff0000u))));
      // the largest value to [224, 448]
      const int e = top > 0.f && top < __int_as_float(0x7f800000)
                        ? (__float_as_int(top) >> 23) - 127 - 8 +
                              ((__float_as_int(top) & 0x7fffff) > 0x600000)
                        : 0;
      // (120 at most: no finite query is clamped from above.  Below -100 the
      // factor c times the scales would leave fp32.)
      const int eq = max(e, -100);
      const float f = q8_pow2(-eq);
      cr = p.scale * 1.4426950408889634f * q8_pow2(eq);
      if (!(top < __int_as_float(0x7f800000)))
        cr = __int_as_float(0x7fffffff);  // the row is computed on its own
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t a = u[8 * c + 2 * k], d = u[8 * c + 2 * k + 1];
          const float v[4] = {__uint_as_float(a << 16) * f,
                              __uint_as_float(a & 0xffff0000u) * f,
                              __uint_as_float(d << 16) * f,
                              __uint_as_float(d & 0xffff0000u) * f};
          hi[k] = q8_pack4(v[0], v[1], v[2], v[3]);
          const float2 h0 = q8_float2(hi[k] & 0xffffu);
          const float2 h1 = q8_float2(hi[k] >> 16);
          lo[k] = q8_pack4(v[0] - h0.x, v[1] - h0.y, v[2] - h1.x, v[3] - h1.y);
        }
        const uint32_t sw = D == 128 ? c ^ (row & 7) : c ^ (row >> 1 & 3);
        st_shared_v4(sQ + row * D + sw * 16, hi);
        st_shared_v4(sQ + L::kQ + row * D + sw * 16, lo);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    const uint32_t tO = tmem + kTmO + lane_off;
    float m = neg_inf, l = 0.f;
    uint32_t next[2] = {};
    bool next_diag[2] = {};
    if (n > 0)
      step_masks(words, list, t0, count, p.lb, qi & 31, pos, pos_lo, next,
                 next_diag);
    for (int i = 0; i < n; ++i) {
      const uint32_t tS = tmem + kTmS + (i & 1) * 64 + lane_off;
      const int t = t0 + i;
      const uint32_t mask[2] = {next[0], next[1]};
      const bool diag[2] = {next_diag[0], next_diag[1]};
      bool held[2];
#pragma unroll
      for (int c = 0; c < 2; ++c)
        held[c] = __any_sync(0xffffffffu, mask[c] != 0u);
      if (!wait_both(meta_full(i % kMeta), i / kMeta & 1u, s_full(i & 1),
                     (i >> 1) & 1u, abort_flag, p.status))
        goto done;
      tc_fence_after();
      const float4 *mt = meta + (i % kMeta) * 4;
      float a16[4], e16[4];  // of 16 keys: c 2^ek, ev
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
            const float4 s = mt[2 * c + g];
            a16[2 * c + g] = cr * s.x;
            e16[2 * c + g] = s.y;
            const float top = fmaf(fmaxf(a, e), a16[2 * c + g], s.y);
            if (mask[c] & (0xffffu << (16 * g))) mx = fmaxf(mx, top);
          }
        }
      }
      // a row without a key so far keeps m = -inf and weights of zero
      const bool move = mx > m + 14.f;
      if (i > 0 && __any_sync(0xffffffffu, move)) {
        // O is at rest once the last step's second product is done
        if (!__all_sync(0xffffffffu,
                        wait_bar_rest_inl(o_done((i - 1) & 1),
                                          ((i - 1) >> 1) & 1u, abort_flag,
                                      p.status)))
          goto done;
        tc_fence_after();
        const float f = move ? ex2(m - (mx - 6.f)) : 1.f;
        l *= f;
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
      if (move) m = mx - 6.f;  // the largest weight is 2^6, and may grow to 2^14
      const float mu = m > neg_inf ? m : 0.f;
      // the next step's masks, among the exponentials
      if (i + 1 < n)
        step_masks(words, list, t + 1, count, p.lb, qi & 31, pos, pos_lo,
                   next, next_diag);
      // P = exp2(S cr 2^ek + ev - mu)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t pk[16];
        if (held[c]) {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const float a = a16[2 * c + g];
            // -inf takes the weights of keys that the row does not hold to 0
            const float sub =
                mask[c] & (0xffffu << (16 * g)) ? e16[2 * c + g] - mu
                                                : neg_inf;
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int x = 16 * g; x < 16 * g + 16; x += 2) {
              float2 e = __ffma2_rn(make_float2(__uint_as_float(u[c][x]),
                                                __uint_as_float(u[c][x + 1])),
                                    make_float2(a, a), make_float2(sub, sub));
              e.x = ex2(e.x);
              e.y = ex2(e.y);
              sum = __fadd2_rn(sum, e);
              asm("cvt.rn.f16x2.f32 %0, %1, %2;"
                  : "=r"(pk[x >> 1])
                  : "f"(e.y), "f"(e.x));
            }
            l = fmaf(sum.x + sum.y, mt[2 * c + g].z, l);
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
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full(i & 1));
    }
    // ---------------- o = O / l ----------------
    for (int i = max(n - 2, 0); i < n; ++i)
      if (!__all_sync(0xffffffffu,
                      wait_bar_rest_inl(o_done(i & 1), (i >> 1) & 1u,
                                        abort_flag, p.status)))
        goto done;
    tc_fence_after();
    const bool some = l > 0.f || l != l;
    const float inv = some ? 1.f / l : 0.f;
    bool odd = l != l || l > 3e38f;  // not finite: computed again below
    const size_t part =
        ((size_t)(blockIdx.x / pl.splits) * pl.splits + split) *
            (pl.qt * p.G) +
        row;
    const uint32_t out_buf = sQ + warp * 4096;  // Q's space is free
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
    odd |= n > 0 && cr != cr;
    // m is rounded, the multiply-adds that it is taken from are not: above 2^25
    // they are a whole power of two apart, and a row may lose all its weights
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
      float *qs = reinterpret_cast<float *>(smem + L::kOffQ) + warp * 1024;
      for (; todo; todo &= todo - 1) {
        const int r = warp * 32 + __ffs(todo) - 1;
        redo_row_q8<D>(p, b, s0 + r / p.G, hk * p.G + r % p.G, qs, lane);
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

// Joins the parts of split tiles, o = sum_i w_i o_i / sum_i w_i with w_i =
// 2^(l_i - max), in the order of the splits: a warp a row, in a launch of its
// own.  A tile has 128 rows of up to 255 parts: the CTA that ended last took 190
// us for 38 of them (one token of 128 heads' rows: 800 us instead of 30).
template <int D>
__global__ void __launch_bounds__(256)
    attn_q8_join_kernel(const __grid_constant__ BlockAttnQ8 p,
                        const __grid_constant__ FwdPlan pl) {
  constexpr int kEl = D / 32;  // columns of a lane
  __shared__ float qs[8][128];
  const float neg_inf = -__int_as_float(0x7f800000);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = pl.qt * p.G;
  const long long all = (long long)pl.tiles * p.B * p.Hk * rows;
  for (long long x = (long long)blockIdx.x * 8 + warp; x < all;
       x += (long long)gridDim.x * 8) {
    const int row = (int)(x % rows);
    const long long item = x / rows;
    int it = (int)item;
    const int hk = it % p.Hk;
    it /= p.Hk;
    const int b = it % p.B;
    const int s = (pl.tiles - 1 - it / p.B) * pl.qt + row / p.G;
    if (s >= p.S) continue;
    float m = neg_inf, sum = 0.f, acc[kEl] = {};
    bool odd = false;
    for (int i0 = 0; i0 < pl.splits; i0 += 8) {
      float l[8], v[8][kEl];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const long long at =
            (item * pl.splits + min(i0 + u, pl.splits - 1)) * rows + row;
        l[u] = i0 + u < pl.splits ? __ldcg(pl.part_l + at) : neg_inf;
        if constexpr (kEl == 4) {
          const float4 t = __ldcg(
              reinterpret_cast<const float4 *>(pl.part_o + at * D) + lane);
          v[u][0] = t.x, v[u][1] = t.y, v[u][2] = t.z, v[u][3] = t.w;
        } else {
          const float2 t = __ldcg(
              reinterpret_cast<const float2 *>(pl.part_o + at * D) + lane);
          v[u][0] = t.x, v[u][1] = t.y;
        }
      }
      float mx = m;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        odd |= l[u] != l[u];
        mx = fmaxf(mx, l[u]);
      }
      const float ref = mx > neg_inf ? mx : 0.f;
      const float f = ex2(m - ref);
      sum *= f;
#pragma unroll
      for (int c = 0; c < kEl; ++c) acc[c] *= f;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float w = ex2(l[u] - ref);
        sum += w;
#pragma unroll
        for (int c = 0; c < kEl; ++c) acc[c] = fmaf(w, v[u][c], acc[c]);
      }
      m = mx;
    }
    const int h = hk * p.G + row % p.G;
    if (odd) {  // (all lanes of the warp)
      redo_row_q8<D>(p, b, s, h, qs[warp], lane);
      continue;
    }
    const size_t at = ((size_t)s * p.B + b) * p.H + h;
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    if constexpr (kEl == 4)
      reinterpret_cast<uint2 *>(p.o + at * D)[lane] =
          make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv),
                     pack_bf16x2(acc[2] * inv, acc[3] * inv));
    else
      reinterpret_cast<uint32_t *>(p.o + at * D)[lane] =
          pack_bf16x2(acc[0] * inv, acc[1] * inv);
    if (lane == 0)
      p.lse[at] = sum > 0.f ? (m + log2f(sum)) * 0.69314718055994531f : neg_inf;
  }
}

template <int D>
int launch_tile(const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                const BlockAttnQ8 &p, const FwdPlan &pl, cudaStream_t st) {
  auto kern = attn_q8_tile_kernel<D>;
  const int smem = TileSmem<D>::bytes(p.nblk, pl.cap);
  constexpr int kMost = TileSmem<D>::bytes(DSA_BLOCK_ATTN_MAX_BLOCKS,
                                           DSA_BLOCK_ATTN_MAX_BLOCKS);
  static_assert(kMost <= kMaxSmem);
  if (allow_smem(kern, kMost) != cudaSuccess) return DSA_ERR_CUDA;
  const long long grid = (long long)pl.tiles * p.B * p.Hk * pl.splits;
  if (grid > 0x7fffffffll) return DSA_ERR_UNSUPPORTED;
  kern<<<(unsigned)grid, kTileThreads, smem, st>>>(tm_k, tm_v, p, pl);
  if (cudaGetLastError() != cudaSuccess) return DSA_ERR_CUDA;
  if (pl.splits == 1) return DSA_OK;
  const long long rows = (long long)pl.tiles * p.B * p.Hk * pl.qt * p.G;
  attn_q8_join_kernel<D><<<(unsigned)((rows + 7) / 8), 256, 0, st>>>(p, pl);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace

int run_attn_q8_tile(const BlockAttnQ8 &p, void *workspace, int num_sms,
                     cudaStream_t st) {
  const FwdPlan pl = plan_fwd(p, p.o, p.lse, workspace, num_sms);
  CUtensorMap tm_k, tm_v;
  const Q8Cache &c = p.c;
  const int rows = p.blk < kKeys ? p.blk : kKeys;
  int rc = encode_kv8(&tm_k, c.k, p.D, rows, c.page_size, c.k_t, p.Hk, c.k_h,
                      c.num_pages, c.k_p);
  if (rc != DSA_OK) return rc;
  rc = encode_kv8(&tm_v, c.v, p.D, rows, c.page_size, c.v_t, p.Hk, c.v_h,
                  c.num_pages, c.v_p);
  if (rc != DSA_OK) return rc;
  return p.D == 64 ? launch_tile<64>(tm_k, tm_v, p, pl, st)
                   : launch_tile<128>(tm_k, tm_v, p, pl, st);
}

}  // namespace dsa
