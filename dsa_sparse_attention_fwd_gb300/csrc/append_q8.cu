// Append to a paged cache held in 8 bits (cache_q8.cuh), the keys normed and
// rotated on the way (norm_rope.cuh), the queries too; and the read back.
//
// Sequence b appends its first n = count[b] rows at positions p = start[b] ..
// start[b] + n - 1.  For each group of the cache that they reach and each head,
//     s = 2^e, the smallest with max |x| <= 448 s over the group's new rows x;
// where the group holds earlier tokens (it begins before start[b]), s is not
// smaller than the scale s0 that it has, and their codes c become
// round(c s0 / s) where it is larger.  New codes are round(x / s).
//
// Bounded by loads in flight.  Measured on one GB300 (copies 6767 GB/s), on the
// device: a ragged chunk of 4 x 2048 tokens of 40 + 2 x 8 heads of 64 27 us (103
// MB, 15 us; the queries alone take 17.5, keys and values alone 13), one token of
// 64 sequences of 64 + 2 x 4 heads of 128 5.1 us.  Read back: two prefixes of up
// to 30000 tokens of 8 heads of 128 62.6 us, 5.6 TB/s, 70% of it writes.
#include "cache_q8.cuh"
#include "norm_rope.cuh"

namespace dsa {
namespace {

struct AppendQ8 {
  RopeArgs a;  // a.k, a.v: inputs only
  Q8Cache c;
  const int32_t *start, *count;  // [B]; count nullptr: all S rows
  int groups;                    // groups that a sequence's rows can reach
  unsigned kv;                   // CTAs that take keys and values
  bool by_warp;                  // a warp an item, else a CTA
  int heads;                     // of a CTA's item
  int angles;                    // angles of a warp's, in shared memory
};

// The rows of a sequence that are appended: [0, n).
__device__ __forceinline__ int rows_of(const AppendQ8 &p, int b, int start) {
  const int n = p.count ? __ldg(p.count + b) : p.a.S;
  return start < 0 ? 0 : min(max(n, 0), p.a.S);
}

// cos and sin (times m) of an angle of pos * fr turns: the top 32 bits of the
// fraction, rounded to fp32, and what that rounds off as a first-order term.
// A code of the cache may be a whole step off where its value falls on the
// border between two: the fewer, the closer the angle.
__device__ __forceinline__ float2 turn_of(const RopeArgs &a, long long pos,
                                          unsigned long long fr) {
  const int t = (int)(((unsigned long long)pos * fr) >> 32);
  const float x = (float)t;
  const float d = (float)(t - (int)x) * 1.4629180792671596e-9f;  // pi 2^-31
  float sn, co;
  sincospif(x * 4.656612873077393e-10f, &sn, &co);
  return make_float2(a.mscale * fmaf(-sn, d, co), a.mscale * fmaf(co, d, sn));
}

// Keys or values of one group and head by `nw` warps (one, or the CTA's four):
// rows s0 .. s0 + n - 1 of the sequence go to the group's tokens from `to` on,
// `early` tokens before them are there already.  A thread holds 8 neighbouring
// values of up to RW rows as they came, and works them out twice, for the
// scale and for the codes: that costs less than fp32 registers for them.
template <int LPR, int RW, bool KEYS>
__device__ __forceinline__ void store_group(
    const AppendQ8 &p, const RopeRows &r, int nw, const __nv_bfloat16 *src,
    int n, int early, uint8_t *group_at, long long st, float *scale, int e0, int sub,
    int unit, Turn<__nv_bfloat16, false> &turn, const float2 *cs, const float *w,
    float *buf, float *red) {
  constexpr int RPW = 32 / LPR;
  const RopeArgs &a = p.a;
  const bool norm = KEYS && r.w != nullptr;
  const int half = a.R / 2;
  Chunk<__nv_bfloat16, false> x[RW];
#pragma unroll
  for (int u = 0; u < RW; ++u) {
    const int row = (u * nw + unit) * RPW + sub;
    if (u * nw * RPW >= n) break;  // (the same for all warps)
    x[u].load(src + row * r.ss, e0, row < n ? a.D : 0);
  }
  auto values = [&](int u, float2 (&y)[4]) {
    asm volatile("" ::: "memory");  // one row's coefficients at a time
    const int row = (u * nw + unit) * RPW + sub;
    if constexpr (KEYS) {
      float2 v[4];
      x[u].get(v);
      const float sq = squares(v);
      turn.set(a, e0, false, cs + (row < n ? row : 0) * half,
               norm ? w : nullptr);
      turn.apply(a, x[u], v, y, e0, buf, sq < 3e38f);
      if (norm) {
        const float r2 = rsqrtf(row_sum<LPR>(sq) * (1.f / a.D) + a.eps);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          y[i] = __fmul2_rn(y[i], make_float2(r2, r2));
      }
    } else {
      x[u].get(y);
    }
  };
  const float had = early > 0 ? *scale : 0.f;
  float top = 0.f;
#pragma unroll
  for (int u = 0; u < RW; ++u) {
    if (u * nw * RPW >= n) break;
    const int row = (u * nw + unit) * RPW + sub;
    float2 y[4];
    values(u, y);
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      t = fmaxf(t, fmaxf(q8_mag(y[i].x), q8_mag(y[i].y)));
    // (padding of the last rows may hold what eps = 0 makes of zeros)
    if (row < n && e0 < a.D) top = fmaxf(top, t);
  }
  // non-negative floats compare as integers
  top = __int_as_float(__reduce_max_sync(0xffffffffu, __float_as_int(top)));
  if (nw > 1) {
    if ((threadIdx.x & 31) == 0) red[unit] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRopeWarps; ++i) top = fmaxf(top, red[i]);
  }
  __syncwarp();
  int e = q8_exp_for(top);
  if (early > 0) {
    const int e_old = q8_exp(had);
    if (e > e_old && e0 < a.D) {
      const float f = q8_pow2(e_old - e);
      for (int t = unit * RPW + sub; t < early; t += nw * RPW) {
        uint2 *at = reinterpret_cast<uint2 *>(group_at + t * st + e0);
        const uint2 c = *at;
        const float2 v0 = q8_float2(c.x & 0xffffu), v1 = q8_float2(c.x >> 16);
        const float2 v2 = q8_float2(c.y & 0xffffu), v3 = q8_float2(c.y >> 16);
        *at = make_uint2(q8_pack4(v0.x * f, v0.y * f, v1.x * f, v1.y * f),
                         q8_pack4(v2.x * f, v2.y * f, v3.x * f, v3.y * f));
      }
    }
    e = max(e, e_old);
  }
  if (unit == 0 && (threadIdx.x & 31) == 0) *scale = q8_pow2(e);
  const float inv = q8_pow2(-e);
#pragma unroll
  for (int u = 0; u < RW; ++u) {
    if (u * nw * RPW >= n) break;
    const int row = (u * nw + unit) * RPW + sub;
    float2 y[4];
    values(u, y);
    if (row < n && e0 < a.D)
      *reinterpret_cast<uint2 *>(group_at + (early + row) * st + e0) =
          make_uint2(q8_pack4(y[0].x * inv, y[0].y * inv, y[1].x * inv,
                              y[1].y * inv),
                     q8_pack4(y[2].x * inv, y[2].y * inv, y[3].x * inv,
                              y[3].y * inv));
  }
}

// Rows that cannot be read in 16-byte pieces (odd strides or pointers, halves
// that do not fall on them): element loads, the partners of the rotation through
// shared memory.  A thread holds up to 16 rows as they came, which spills 252 to
// 276 bytes of it: one token of 64 sequences takes 12.7 us instead of 4.9, the
// ragged chunk above 234 instead of 27.  It is there for layouts that are rare.  CTAs 0 .. kv - 1 take keys and values, the others queries as
// norm_rope_kernel() does.  Keys and values: an item is a group that a
// sequence's rows can reach and one head (by a warp, where a group gets few new
// rows) or several (by a CTA, the angles of the group's tokens in shared
// memory for all of them).
template <int LPR, int RW>
__global__ void __launch_bounds__(kRopeThreads, RW <= 8 ? 5 : 3)
    append_q8_kernel(const __grid_constant__ AppendQ8 p) {
  constexpr int RPW = 32 / LPR;
  using T = __nv_bfloat16;
  __shared__ __align__(16) float xch[kRopeWarps * RPW * LPR * 8];
  __shared__ unsigned long long fr[kRopeMaxD / 2];
  __shared__ __align__(16) float sw[2][kRopeMaxD];
  __shared__ float red[2][kRopeWarps];
  extern __shared__ __align__(16) float2 angles[];
  const RopeArgs &a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / LPR, e0 = (lane % LPR) * 8;
  float *buf = xch + (warp * RPW + sub) * LPR * 8;
  load_weights(a, sw);
  for (int i = threadIdx.x; i < a.R / 2; i += kRopeThreads) {
    double t = a.inv_freq[i] * 0.15915494309189535;  // 1 / (2 pi)
    t -= floor(t);
    fr[i] = __double2ull_rn(t * 18446744073709551616.0);
  }
  const int half = a.R / 2;
  // lanes outside the rotated part multiply the first coefficients by zero
  float2 *cs = angles + (blockIdx.x < p.kv && !p.by_warp
                             ? 0
                             : warp * p.angles);
  if (half == 0 && threadIdx.x < kRopeWarps * 8)
    angles[(threadIdx.x / 8) * p.angles + threadIdx.x % 8] =
        make_float2(0.f, 0.f);
  __syncthreads();
  Turn<T, false> turn;
  turn.init(a, e0, lane, false);

  if (blockIdx.x >= p.kv) {
    // ---------------- queries ----------------
    const unsigned items = (unsigned)a.S * a.B * a.chunks;
    const unsigned stride = (gridDim.x - p.kv) * kRopeWarps;
    const int nq = a.q.heads;
    for (unsigned item = (blockIdx.x - p.kv) * kRopeWarps + warp; item < items;
         item += stride) {
      const unsigned tk = item / (unsigned)a.chunks;
      const int s = (int)(tk / (unsigned)a.B), b = (int)(tk % (unsigned)a.B);
      const int h0 = (int)(item % (unsigned)a.chunks) * a.heads_per_item;
      const long long pos = (long long)__ldg(p.start + b) + s;
      __syncwarp();
      for (int i = lane; i < half; i += 32) cs[i] = turn_of(a, pos, fr[i]);
      __syncwarp();
      rope_heads<T, false, LPR, 0>(
          a, a.q, static_cast<const T *>(a.q.in) + s * a.q.ss + b * a.q.sb,
          static_cast<T *>(a.q.out) + tk * (long long)nq * a.D, a.D, h0,
          min(h0 + a.heads_per_item, nq), sub, e0, turn, cs, sw[0], buf);
    }
    return;
  }
  // ---------------- keys and values ----------------
  const int hc = p.by_warp ? 1 : p.heads;  // heads of an item
  const int nh = (a.k.heads + hc - 1) / hc;
  long long it = p.by_warp ? (long long)blockIdx.x * kRopeWarps + warp
                           : (long long)blockIdx.x;
  if (it >= (long long)p.groups * a.B * 2 * nh) return;
  const bool is_v = it & 1;
  it >>= 1;
  const int h0 = (int)(it % nh) * hc;
  it /= nh;
  const int b = (int)(it % a.B), gi = (int)(it / a.B);
  const int start = __ldg(p.start + b);
  const int rows = rows_of(p, b, start);
  const long long g0 = ((long long)(start >> p.c.lg) + gi) << p.c.lg;
  const int s0 = (int)max(g0 - start, 0ll);
  const int s1 = (int)min(g0 + p.c.group - start, (long long)rows);
  if (s0 >= s1) return;
  bool bad = false;
  const int page = q8_page(p.c, b, g0, bad);
  if (bad) {
    if (lane == 0) atomicOr(a.status, kStatusIndexRange);
    return;
  }
  const int n = s1 - s0, early = (int)max((long long)start - g0, 0ll);
  const int off = (int)(g0 % p.c.page_size);
  if (!is_v && half > 0) {
    const int nt = p.by_warp ? 32 : kRopeThreads;
    for (int i = p.by_warp ? lane : threadIdx.x; i < n * half; i += nt) {
      const int t = i / half;
      cs[i] = turn_of(a, (long long)start + s0 + t, fr[i - t * half]);
    }
    if (p.by_warp)
      __syncwarp();
    else
      __syncthreads();
  }
  const RopeRows &in = is_v ? a.v : a.k;
  const long long st = is_v ? p.c.v_t : p.c.k_t;
  const int nw = p.by_warp ? 1 : kRopeWarps, unit = p.by_warp ? 0 : warp;
  for (int h = h0; h < min(h0 + hc, a.k.heads); ++h) {
    const T *src = static_cast<const T *>(in.in) + b * in.sb + h * in.sh +
                   s0 * in.ss;
    uint8_t *at = (is_v ? p.c.v + page * p.c.v_p + h * p.c.v_h
                        : p.c.k + page * p.c.k_p + h * p.c.k_h) +
                  off * st;
    float *scale = (is_v ? p.c.vs : p.c.ks) + q8_scale_at(p.c, page, off, h);
    float *rd = red[(h - h0) & 1];
    if (is_v)
      store_group<LPR, RW, false>(p, in, nw, src, n, early, at, st, scale,
                                       e0, sub, unit, turn, cs, sw[1], buf, rd);
    else
      store_group<LPR, RW, true>(p, in, nw, src, n, early, at, st, scale,
                                      e0, sub, unit, turn, cs, sw[1], buf, rd);
  }
}

// What is the same for all rows of a thread: the weights of its 8 elements and
// of their partners, the latter with the rotation's sign; where its angles lie
// in a token's, or behind them (cosine 1, sine 0) outside the rotated part.
struct Fixed {
  float2 w[4], wp[4];
  int src_lane, at;
  bool rotated;
};

// x of 8 elements, normed and rotated: (x w c + x' w' s) rstd.
template <int LPR>
__device__ __forceinline__ void turned(const RopeArgs &a, const Fixed &f,
                                       const Chunk<__nv_bfloat16, true> &raw,
                                       const float2 *cs, const float2 *none,
                                       bool norm, float2 (&y)[4]) {
  Chunk<__nv_bfloat16, true> from;
  const uint32_t *x = reinterpret_cast<const uint32_t *>(raw.raw);
  uint32_t *o = reinterpret_cast<uint32_t *>(from.raw);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // neighbours swap places in their word, halves come from another lane;
    // (an infinity of an element that is its own partner stays out)
    const uint32_t v = a.interleaved
                           ? __byte_perm(x[i], x[i], 0x1032)
                           : __shfl_sync(0xffffffffu, x[i], f.src_lane);
    o[i] = f.rotated ? v : 0u;
  }
  float2 v[4], p[4];
  raw.get(v);
  from.get(p);
  const float4 *q =
      reinterpret_cast<const float4 *>(f.rotated ? cs + f.at : none);
  float sq = 0.f;
  if (norm) sq = row_sum<LPR>(squares(v));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 c, s;
    if (a.interleaved) {  // one angle for both
      const float2 t = reinterpret_cast<const float2 *>(q)[i];
      c = make_float2(t.x, t.x), s = make_float2(t.y, t.y);
    } else {
      const float4 t = q[i];
      c = make_float2(t.x, t.z), s = make_float2(t.y, t.w);
    }
    y[i] = __ffma2_rn(__fmul2_rn(v[i], f.w[i]), c,
                      __fmul2_rn(__fmul2_rn(p[i], f.wp[i]), s));
  }
  if (norm) {
    const float r = rsqrtf(sq * (1.f / a.D) + a.eps);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = __fmul2_rn(y[i], make_float2(r, r));
  }
}

// Rows in 16-byte pieces.  CTAs 0 .. kv - 1 take keys and values, the others
// queries as norm_rope_kernel() does.  Keys and values: an item is a group that
// a sequence's rows can reach, of the keys or the values, and one head (WARP: by
// a warp, where a group gets few new rows) or some (by a CTA; the angles of the
// group's tokens are in shared memory for all of them).  A thread holds 8
// elements of RW rows of a head as fp32 until the group's scale is known, and
// has the next head's rows on the way.
constexpr int kVecThreads = 256, kVecWarps = kVecThreads / 32;
constexpr int vec_ctas(int rw) { return rw <= 4 ? 3 : 2; }  // an SM

template <int LPR, int RW, bool WARP>
__global__ void __launch_bounds__(kVecThreads, vec_ctas(RW))
    append_q8_vec_kernel(const __grid_constant__ AppendQ8 p) {
  constexpr int RPW = 32 / LPR;
  using T = __nv_bfloat16;
  __shared__ unsigned long long fr[kRopeMaxD / 2];
  __shared__ __align__(16) float sw[2][kRopeMaxD];
  __shared__ float red[2][kVecWarps];
  __shared__ __align__(16) float2 none[8];  // of elements that do not turn
  extern __shared__ __align__(16) float2 angles[];
  const RopeArgs &a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / LPR, e0 = (lane % LPR) * 8;
  const int half = a.R / 2;
  auto frequencies = [&] {
    for (int i = threadIdx.x; i < half; i += kVecThreads) {
      double t = a.inv_freq[i] * 0.15915494309189535;  // 1 / (2 pi)
      t -= floor(t);
      fr[i] = __double2ull_rn(t * 18446744073709551616.0);
    }
  };

  if (blockIdx.x >= p.kv) {
    // ---------------- queries ----------------
    float *buf = nullptr;
    for (int i = threadIdx.x; i < kRopeMaxD; i += kVecThreads)
      sw[0][i] = a.q.w && i < a.D ? __ldg(a.q.w + i) : 0.f;
    frequencies();
    float2 *cs = angles + warp * p.angles;
    if (half == 0 && lane < 8) cs[lane] = make_float2(0.f, 0.f);
    __syncthreads();
    Turn<T, true> turn;
    turn.init(a, e0, lane, false);
    const unsigned items = (unsigned)a.S * a.B * a.chunks;
    const unsigned stride = (gridDim.x - p.kv) * kVecWarps;
    const int nq = a.q.heads;
    for (unsigned item = (blockIdx.x - p.kv) * kVecWarps + warp; item < items;
         item += stride) {
      const unsigned tk = item / (unsigned)a.chunks;
      const int s = (int)(tk / (unsigned)a.B), b = (int)(tk % (unsigned)a.B);
      const int h0 = (int)(item % (unsigned)a.chunks) * a.heads_per_item;
      const long long pos = (long long)__ldg(p.start + b) + s;
      __syncwarp();
      for (int i = lane; i < half; i += 32) cs[i] = turn_of(a, pos, fr[i]);
      __syncwarp();
      rope_heads<T, true, LPR, 0>(
          a, a.q, static_cast<const T *>(a.q.in) + s * a.q.ss + b * a.q.sb,
          static_cast<T *>(a.q.out) + tk * (long long)nq * a.D, a.D, h0,
          min(h0 + a.heads_per_item, nq), sub, e0, turn, cs, sw[0], buf);
    }
    return;
  }
  // ---------------- keys and values ----------------
  constexpr int nw = WARP ? 1 : kVecWarps;  // warps of an item
  const int unit = WARP ? 0 : warp;
  const int hc = WARP ? 1 : p.heads, nh = (a.k.heads + hc - 1) / hc;
  long long it = WARP ? (long long)blockIdx.x * kVecWarps + warp
                      : (long long)blockIdx.x;
  const bool some = it < (long long)p.groups * a.B * 2 * nh;
  const bool is_v = it & 1;
  it >>= 1;
  const int h0 = (int)(it % nh) * hc;
  it /= nh;
  const int b = some ? (int)(it % a.B) : 0, gi = some ? (int)(it / a.B) : 0;
  const int start = __ldg(p.start + b);
  const int rows = rows_of(p, b, start);
  const long long g0 = ((long long)(start >> p.c.lg) + gi) << p.c.lg;
  const int s0 = (int)max(g0 - start, 0ll);
  const int s1 = (int)min(g0 + p.c.group - start, (long long)rows);
  const int n = some ? s1 - s0 : 0;
  if (!WARP && n <= 0) return;
  const RopeRows &in = is_v ? a.v : a.k;
  const T *src0 = static_cast<const T *>(in.in) + b * in.sb + s0 * in.ss;
  Chunk<T, true> x[RW];
  auto fetch = [&](int h) {
#pragma unroll
    for (int u = 0; u < RW; ++u) {
      const int row = (u * nw + unit) * RPW + sub;
      if (u * nw * RPW < n)  // (the same for all)
        x[u].load(src0 + h * in.sh + row * in.ss, e0, row < n ? a.D : 0);
    }
  };
  if (n > 0) fetch(h0);
  bool bad = false;
  int page = -1;
  if (n > 0) {
    page = q8_page(p.c, b, g0, bad);
    if (bad && lane == 0) atomicOr(a.status, kStatusIndexRange);
  }
  if (!WARP && page < 0) return;
  const bool norm = a.k.w != nullptr;
  Fixed f;
  if (WARP || !is_v) {
    // (WARP: some of the CTA's items may be keys)
    frequencies();
    if (threadIdx.x < 8) none[threadIdx.x] = make_float2(1.f, 0.f);
    const int rel = e0 - a.r0;
    const bool first = a.interleaved || rel < half;
    f.rotated = rel >= 0 && rel < a.R;
    f.src_lane = lane;
    f.at = 0;
    if (f.rotated) {
      f.at = a.interleaved ? rel / 2 : first ? rel : rel - half;
      if (!a.interleaved) f.src_lane = first ? lane + a.R / 16 : lane - a.R / 16;
    }
    const int ep = a.interleaved || !f.rotated ? e0 : first ? e0 + half : e0 - half;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 w = make_float2(1.f, 1.f), o = w;
      if (norm && e0 < a.D) {
        w = make_float2(__ldg(a.k.w + e0 + 2 * i), __ldg(a.k.w + e0 + 2 * i + 1));
        o = make_float2(__ldg(a.k.w + ep + 2 * i), __ldg(a.k.w + ep + 2 * i + 1));
      }
      // (first: a cos - b sin; the other: a sin + b cos)
      f.w[i] = w;
      f.wp[i] = a.interleaved ? make_float2(-o.y, o.x)
                : first       ? make_float2(-o.x, -o.y)
                              : o;
    }
    __syncthreads();
  }
  if (WARP && page < 0) return;
  float2 *cs = angles + (WARP ? warp * p.angles : 0);
  if (!is_v && half > 0) {
    for (int i = WARP ? lane : threadIdx.x; i < n * half;
         i += WARP ? 32 : kVecThreads) {
      const int t = i / half;
      cs[i] = turn_of(a, (long long)start + s0 + t, fr[i - t * half]);
    }
    if (WARP)
      __syncwarp();
    else
      __syncthreads();
  }
  const int early = (int)max((long long)start - g0, 0ll);
  const int off = (int)(g0 % p.c.page_size);
  const long long st = is_v ? p.c.v_t : p.c.k_t;
  const int h1 = min(h0 + hc, a.k.heads);
  for (int h = h0; h < h1; ++h) {
    uint8_t *at = (is_v ? p.c.v + page * p.c.v_p + h * p.c.v_h
                        : p.c.k + page * p.c.k_p + h * p.c.k_h) +
                  off * st + e0;
    float *scale = (is_v ? p.c.vs : p.c.ks) + q8_scale_at(p.c, page, off, h);
    const float had = early > 0 ? *scale : 0.f;
    float2 y[RW][4];
    float top = 0.f;
#pragma unroll
    for (int u = 0; u < RW; ++u) {
      if (u * nw * RPW < n) {
        const int row = (u * nw + unit) * RPW + sub;
        if (is_v)
          x[u].get(y[u]);
        else
          turned<LPR>(a, f, x[u], cs + (row < n ? row : 0) * half, none, norm,
                      y[u]);
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          t = fmaxf(t, fmaxf(q8_mag(y[u][i].x), q8_mag(y[u][i].y)));
        // (padding of the last rows may hold what eps = 0 makes of zeros)
        if (row < n && e0 < a.D) top = fmaxf(top, t);
      }
    }
    if (h + 1 < h1) fetch(h + 1);
    // non-negative floats compare as integers
    top = __int_as_float(__reduce_max_sync(0xffffffffu, __float_as_int(top)));
    if constexpr (!WARP) {
      float *rd = red[(h - h0) & 1];
      if (lane == 0) rd[unit] = top;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kVecWarps; ++i) top = fmaxf(top, rd[i]);
    }
    __syncwarp();
    int e = q8_exp_for(top);
    if (early > 0) {
      const int e_old = q8_exp(had);
      if (e > e_old && e0 < a.D) {
        const float fc = q8_pow2(e_old - e);
        for (int t = unit * RPW + sub; t < early; t += nw * RPW) {
          uint2 *to = reinterpret_cast<uint2 *>(at + t * st);
          const uint2 c = *to;
          const float2 v0 = q8_float2(c.x & 0xffffu), v1 = q8_float2(c.x >> 16);
          const float2 v2 = q8_float2(c.y & 0xffffu), v3 = q8_float2(c.y >> 16);
          *to = make_uint2(
              q8_pack4(v0.x * fc, v0.y * fc, v1.x * fc, v1.y * fc),
              q8_pack4(v2.x * fc, v2.y * fc, v3.x * fc, v3.y * fc));
        }
      }
      e = max(e, e_old);
    }
    if (unit == 0 && lane == 0) *scale = q8_pow2(e);
    const float inv = q8_pow2(-e);
#pragma unroll
    for (int u = 0; u < RW; ++u) {
      const int row = (u * nw + unit) * RPW + sub;
      if (row < n && e0 < a.D)
        *reinterpret_cast<uint2 *>(at + (early + row) * st) = make_uint2(
            q8_pack4(y[u][0].x * inv, y[u][0].y * inv, y[u][1].x * inv,
                     y[u][1].y * inv),
            q8_pack4(y[u][2].x * inv, y[u][2].y * inv, y[u][3].x * inv,
                     y[u][3].y * inv));
    }
  }
}

// Heads of a CTA's item of keys or values: all share the angles, but fewer
// where that leaves SMs idle.  (One round of CTAs, and queries in the slots
// that it leaves: a ragged chunk of 8192 tokens 27 us, with three times the CTAs
// 29.)
int heads_of_item(long long groups, int heads, int num_sms) {
  int n = heads;
  while (n > 1 && groups * ((heads + n - 1) / n) < num_sms)
    n = (n + 1) / 2;
  return n;
}

// Queries: warps' items as launch_lpr() of norm_rope.cu cuts them; the CTAs.
long long query_ctas(RopeArgs &a, int rpw, int warps, long long cap,
                     int num_sms) {
  if (a.q.heads == 0) return 0;
  const long long toks = (long long)a.S * a.B;
  int per = (a.q.heads + rpw - 1) / rpw * rpw;
  while (per > rpw && toks * ((a.q.heads + per - 1) / per) < 32ll * num_sms)
    per = ((per / 2) + rpw - 1) / rpw * rpw;
  a.heads_per_item = per;
  a.chunks = (a.q.heads + per - 1) / per;
  const long long n = (toks * a.chunks + warps - 1) / warps;
  return n < cap ? n : cap;
}

template <int LPR, int RW, bool WARP>
int launch_vec(AppendQ8 &p, int num_sms, cudaStream_t st) {
  constexpr int RPW = 32 / LPR;
  RopeArgs &a = p.a;
  auto kern = append_q8_vec_kernel<LPR, RW, WARP>;
  // new rows that a group can get
  const int most = a.S < p.c.group ? a.S : p.c.group;
  // angles of the tokens of a group (a warp's, or a CTA's), and of a token of
  // queries for each warp
  const int half = a.R / 2 < 8 ? 8 : a.R / 2;
  p.angles = (WARP ? most : 1) * half;
  int angles = kVecWarps * p.angles;
  if (!WARP && most * half > angles) angles = most * half;
  const long long groups = 2ll * p.groups * a.B;
  p.heads = WARP ? 1 : heads_of_item(groups, a.k.heads, num_sms);
  long long kv = groups * ((a.k.heads + p.heads - 1) / p.heads);
  if (WARP) kv = (kv + kVecWarps - 1) / kVecWarps;
  if (kv >= (1ll << 30)) return DSA_ERR_UNSUPPORTED;
  p.kv = (unsigned)kv;
  // two rounds of CTAs: the first ones wait for keys and values to finish
  const long long q_ctas = query_ctas(a, RPW, kVecWarps,
                                      2ll * vec_ctas(RW) * num_sms, num_sms);
  // (D * group <= 16384 and R <= D: 64 KB at most)
  constexpr int kMost = 16384 / 2 * (int)sizeof(float2) + 8192;
  const int smem = angles * (int)sizeof(float2);
  if (smem > kMost) return DSA_ERR_UNSUPPORTED;
  if (allow_smem(kern, kMost) != cudaSuccess) return DSA_ERR_CUDA;
  kern<<<(unsigned)(kv + q_ctas), kVecThreads, smem, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

// RW: rows of a thread that a group takes.  A warp takes an item of its own
// where those are two passes of one: single tokens and drafts.
template <int LPR>
int launch_vec_rows(AppendQ8 &p, int num_sms, cudaStream_t st) {
  constexpr int RPW = 32 / LPR;
  const int most = p.a.S < p.c.group ? p.a.S : p.c.group;
  if (most <= RPW) return launch_vec<LPR, 1, true>(p, num_sms, st);
  if (most <= 2 * RPW) return launch_vec<LPR, 2, true>(p, num_sms, st);
  if (p.c.group <= 2 * kVecWarps * RPW)
    return launch_vec<LPR, 2, false>(p, num_sms, st);
  if constexpr (LPR > 8)  // (64 dimensions have 4 rows at most)
    if (p.c.group > 4 * kVecWarps * RPW)
      return launch_vec<LPR, 8, false>(p, num_sms, st);
  return launch_vec<LPR, 4, false>(p, num_sms, st);
}

// Rows without 16-byte pieces, RW of a thread.
template <int LPR, int RW>
int launch_any(AppendQ8 &p, int num_sms, cudaStream_t st) {
  RopeArgs &a = p.a;
  auto kern = append_q8_kernel<LPR, RW>;
  const int most = a.S < p.c.group ? a.S : p.c.group;
  p.by_warp = most <= 2;
  const int half = a.R / 2 < 8 ? 8 : a.R / 2;
  p.angles = (p.by_warp ? most : 1) * half;
  int angles = kRopeWarps * p.angles;
  if (!p.by_warp && most * half > angles) angles = most * half;
  const long long groups = 2ll * p.groups * a.B;
  p.heads = p.by_warp ? 1 : heads_of_item(groups, a.k.heads, num_sms);
  long long kv = groups * ((a.k.heads + p.heads - 1) / p.heads);
  if (p.by_warp) kv = (kv + kRopeWarps - 1) / kRopeWarps;
  if (kv >= (1ll << 30)) return DSA_ERR_UNSUPPORTED;
  p.kv = (unsigned)kv;
  const long long q_ctas =
      query_ctas(a, 32 / LPR, kRopeWarps, 3ll * num_sms, num_sms);
  constexpr int kMost = 16384 / 2 * (int)sizeof(float2) + 8192;
  const int smem = angles * (int)sizeof(float2);
  if (smem > kMost) return DSA_ERR_UNSUPPORTED;
  if (allow_smem(kern, kMost) != cudaSuccess) return DSA_ERR_CUDA;
  kern<<<(unsigned)(kv + q_ctas), kRopeThreads, smem, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

// A thread holds every row of a group that is its own: 16 at most, as D * group
// <= 16384.
template <int LPR>
int launch_any_rows(AppendQ8 &p, int num_sms, cudaStream_t st) {
  const int rows = p.c.group / (kRopeWarps * (32 / LPR));
  if (rows <= 8) return launch_any<LPR, 8>(p, num_sms, st);
  if constexpr (LPR > 8)  // (64 dimensions have 8 rows at most)
    if (rows <= 16) return launch_any<LPR, 16>(p, num_sms, st);
  return DSA_ERR_UNSUPPORTED;
}

int run_append(AppendQ8 &p, int num_sms, cudaStream_t st) {
  const RopeArgs &a = p.a;
  const bool vec = a.r0 % 8 == 0 && a.R % (a.interleaved ? 8 : 16) == 0 &&
                   vec_rows(a.q, 2, false) && vec_rows(a.k, 2, false) &&
                   vec_rows(a.v, 2, false);
  if (!vec) {
    if (a.D <= 64) return launch_any_rows<8>(p, num_sms, st);
    if (a.D <= 128) return launch_any_rows<16>(p, num_sms, st);
    return launch_any_rows<32>(p, num_sms, st);
  }
  if (a.D <= 64) return launch_vec_rows<8>(p, num_sms, st);
  if (a.D <= 128) return launch_vec_rows<16>(p, num_sms, st);
  return launch_vec_rows<32>(p, num_sms, st);
}

struct ReadQ8 {
  Q8Cache c;
  int T, B;
  const int32_t *first, *length;
  __nv_bfloat16 *k, *v;
  int *status;
};

// A warp takes kReadRows consecutive tokens of a sequence: their pages are
// looked up once, and a lane has the loads of all of them in flight, 16 values
// of one head each.
constexpr int kReadRows = 4, kReadThreads = 256;
__global__ void __launch_bounds__(kReadThreads, 4) read_q8_kernel(
    const __grid_constant__ ReadQ8 p) {
  const int lane = threadIdx.x & 31;
  const int ch = p.c.D / 16, pieces = p.c.Hk * ch;
  const unsigned tiles = (unsigned)((p.T + kReadRows - 1) / kReadRows);
  const unsigned items = tiles * p.B;
  const unsigned stride = gridDim.x * (kReadThreads / 32);
  for (unsigned it = blockIdx.x * (kReadThreads / 32) + (threadIdx.x >> 5);
       it < items; it += stride) {
    const int b = (int)(it / tiles), t0 = (int)(it % tiles) * kReadRows;
    // lane u: token t0 + u
    int page = -1, off = 0;
    {
      const int t = t0 + lane;
      const int n = p.length ? __ldg(p.length + b) : p.T;
      if (lane < kReadRows && t < min(n, p.T)) {
        const long long j = (p.first ? (long long)__ldg(p.first + b) : 0) + t;
        bool bad = false;
        page = q8_page(p.c, b, j, bad);
        if (bad) atomicOr(p.status, kStatusIndexRange);
        if (page >= 0) off = (int)((unsigned)j % (unsigned)p.c.page_size);
      }
    }
#pragma unroll 1
    for (int kv = 0; kv < 2; ++kv) {
      __nv_bfloat16 *out = kv ? p.v : p.k;
      if (!out) continue;
      const uint8_t *in = kv ? p.c.v : p.c.k;
      const float *scales = kv ? p.c.vs : p.c.ks;
      const long long sp = kv ? p.c.v_p : p.c.k_p, st = kv ? p.c.v_t : p.c.k_t;
      const long long sh = kv ? p.c.v_h : p.c.k_h;
#pragma unroll 1
      for (int c = lane; c - lane < pieces; c += 32) {
        const bool mine = c < pieces;  // (whole warps: they exchange pages)
        const int h = mine ? c / ch : 0, piece = c - h * ch;
        uint4 x[kReadRows];
        float s[kReadRows];
#pragma unroll
        for (int u = 0; u < kReadRows; ++u) {
          const int pg = __shfl_sync(0xffffffffu, page, u);
          const int of = __shfl_sync(0xffffffffu, off, u);
          x[u] = make_uint4(0u, 0u, 0u, 0u);
          s[u] = 0.f;
          if (pg >= 0 && mine) {
            x[u] = __ldg(reinterpret_cast<const uint4 *>(
                             in + pg * sp + of * st + h * sh) +
                         piece);
            s[u] = __ldg(scales + q8_scale_at(p.c, pg, of, h));
          }
        }
#pragma unroll
        for (int u = 0; u < kReadRows; ++u) {
          if (t0 + u >= p.T || !mine) break;
          const float f = q8_pow2(q8_exp(s[u]));
          const uint32_t q[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
          uint32_t w[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 lo = q8_float2(q[k] & 0xffffu);
            const float2 hi = q8_float2(q[k] >> 16);
            w[2 * k] = pack_bf16x2(lo.x * f, lo.y * f);
            w[2 * k + 1] = pack_bf16x2(hi.x * f, hi.y * f);
          }
          uint4 *to = reinterpret_cast<uint4 *>(
              out + ((((long long)(t0 + u) * p.B + b) * p.c.Hk + h) * ch +
                     piece) *
                        16);
          __stcs(to, make_uint4(w[0], w[1], w[2], w[3]));
          __stcs(to + 1, make_uint4(w[4], w[5], w[6], w[7]));
        }
      }
    }
  }
}

}  // namespace
}  // namespace dsa

extern "C" {

int dsa_paged_append_q8(
    const void *k, const int64_t *k_strides, const void *v,
    const int64_t *v_strides, const void *q, const int64_t *q_strides, int S,
    int B, int H, int Hk, int D, void *k_cache, void *v_cache,
    const int64_t *cache_strides, float *k_scale, float *v_scale, int group,
    int num_pages, int page_size, const int32_t *page_table, int max_pages,
    const int32_t *start, const int32_t *count, const float *wq,
    const float *wk, float eps, const double *inv_freq, int rot_start,
    int rot_dim, int interleaved, float rot_scale, void *out_q,
    void *workspace, size_t workspace_bytes, void *cuda_stream) {
  if (!k || !v || !k_cache || !v_cache || !k_scale || !v_scale || !start ||
      Hk <= 0)
    return DSA_ERR_INVALID_ARG;
  if (q && (!out_q || H <= 0)) return DSA_ERR_INVALID_ARG;
  dsa::AppendQ8 p{};
  dsa::RopeArgs &a = p.a;
  dsa::set_in(a.q, q, q_strides, S, B, H, D);
  dsa::set_in(a.k, k, k_strides, S, B, Hk, D);
  dsa::set_in(a.v, v, v_strides, S, B, Hk, D);
  a.q.out = out_q;
  a.q.w = wq;
  a.k.w = wk;
  a.S = S, a.B = B, a.D = D, a.r0 = rot_start, a.R = rot_dim;
  a.interleaved = interleaved != 0;
  a.eps = eps, a.mscale = rot_scale, a.inv_freq = inv_freq;
  int rc = dsa::check_rope(a, DSA_BF16);
  if (rc != DSA_OK) return rc;
  rc = dsa::set_q8_cache(p.c, k_cache, v_cache, cache_strides, k_scale,
                         v_scale, group, num_pages, page_size, page_table,
                         max_pages, Hk, D);
  if (rc != DSA_OK) return rc;
  if (D * group > 16384) return DSA_ERR_UNSUPPORTED;
  if (!dsa::aligned(start, 4) || !dsa::aligned(count, 4))
    return DSA_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < 256) return DSA_ERR_WORKSPACE;
  if (!dsa::aligned(workspace, 256)) return DSA_ERR_INVALID_ARG;
  a.status = static_cast<int *>(workspace);
  p.start = start, p.count = count;
  p.groups = (int)(((long long)S + group - 2) / group + 1);
  int num_sms = 0;
  rc = dsa::device_num_sms(&num_sms);
  if (rc != DSA_OK) return rc;
  return dsa::run_append(p, num_sms, static_cast<cudaStream_t>(cuda_stream));
}

int dsa_paged_read_q8(const void *k_cache, const void *v_cache,
                      const int64_t *cache_strides, const float *k_scale,
                      const float *v_scale, int group, int num_pages,
                      int page_size, const int32_t *page_table, int max_pages,
                      int T, int B, int Hk, int D, const int32_t *first,
                      const int32_t *length, void *out_k, void *out_v,
                      void *workspace, size_t workspace_bytes,
                      void *cuda_stream) {
  if (!k_cache || !v_cache || !k_scale || !v_scale || (!out_k && !out_v) ||
      T <= 0 || B <= 0)
    return DSA_ERR_INVALID_ARG;
  dsa::ReadQ8 p{};
  int rc = dsa::set_q8_cache(p.c, k_cache, v_cache, cache_strides, k_scale,
                             v_scale, group, num_pages, page_size, page_table,
                             max_pages, Hk, D);
  if (rc != DSA_OK) return rc;
  if (!dsa::aligned(first, 4) || !dsa::aligned(length, 4) ||
      !dsa::aligned(out_k, 16) || !dsa::aligned(out_v, 16))
    return DSA_ERR_INVALID_ARG;
  if ((long long)T * B >= (1ll << 31)) return DSA_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < 256) return DSA_ERR_WORKSPACE;
  if (!dsa::aligned(workspace, 256)) return DSA_ERR_INVALID_ARG;
  p.T = T, p.B = B, p.first = first, p.length = length;
  p.k = static_cast<__nv_bfloat16 *>(out_k);
  p.v = static_cast<__nv_bfloat16 *>(out_v);
  p.status = static_cast<int *>(workspace);
  int num_sms = 0;
  rc = dsa::device_num_sms(&num_sms);
  if (rc != DSA_OK) return rc;
  constexpr int kWarps = dsa::kReadThreads / 32;
  const long long items =
      (long long)((T + dsa::kReadRows - 1) / dsa::kReadRows) * B;
  const long long grid = (items + kWarps - 1) / kWarps;
  const long long most = 8ll * num_sms;
  dsa::read_q8_kernel<<<(unsigned)(grid < most ? grid : most),
                        dsa::kReadThreads, 0,
                        static_cast<cudaStream_t>(cuda_stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // extern "C"
