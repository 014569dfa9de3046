// Per-head RMS norm with the rotation of positions in the same pass (queries
// and keys in one launch), its backward, and the append of keys and values
// to a paged cache with the same arithmetic on the way.
//
// A row is one head of one token, x of D values:
//     n = x * rsqrt(mean(x^2) + eps) * w          (n = x without a weight)
// and inside [r0, r0 + R), for the pair (a, b) with index i,
//     (a, b) -> m (a cos t - b sin t, a sin t + b cos t),  t = pos * f_i,
// pairs being the neighbours (2i, 2i + 1) or the halves (i, i + R/2).  As
// every element e has one partner e', y_e = n_e c_e + n_e' s_e with
// coefficients that depend on (token, e) only: they are computed once and
// used for all heads that a warp takes of a token.
//
// The angle is held in turns as a 64-bit fixed-point fraction: f_i / (2 pi)
// is converted once (from 64-bit floating point), pos * that wraps modulo
// one turn exactly, and the top 32 bits go to sincospi.  A position of 2^30
// is as exact as position 1, and no table is read.
//
// Bounded by memory: each row is read once and written once, and the
// statistics stay in registers.  Lanes own 8 consecutive values (16 bytes in
// 16-bit types), so D = 128 puts two rows in a warp.  CTAs are persistent: the
// conversion of the frequencies (64-bit arithmetic, slow on this part) runs
// once a CTA into shared memory, sines and cosines once a token and warp (each
// lane R / 64 pairs, exchanged through shared memory), and a warp has the
// loads of kBatch row groups in flight.  Rows that cannot be read in 16-byte
// pieces (odd sizes, strides or pointers) take the same code with element
// loads and the partner exchanged through shared memory.
//
// Measured on one GB300 (copies 6776 GB/s): 32768 tokens of 72 heads of 128 in
// bf16, 1.2 GB: 205 us, 5.9 TB/s (a library copy of the same bytes 181 us, 6.7);
// without the rotation 187, without the norm 196.  It waits for loads: six
// CTAs of four warps hold what 80 registers a thread let them.  In fp32, with
// three CTAs an SM: 398 us, 6.1 TB/s (caches cold; bf16 and fp16 so 218 to 220).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "common.cuh"
#include "dsa_indexer.h"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeWarps = kRopeThreads / 32;
constexpr int kRopeMaxD = 256;
// CTAs an SM holds (the launch bounds); a grid has no more, so that all run
// at once and each takes its share of the rows.
constexpr int rope_ctas(int el, bool vec) { return el == 2 && vec ? 6 : 3; }
constexpr int kRopeBwdCtas = 4;
constexpr int kRopeMaxCtas = 6 * 160;

// One of the row sets (queries, keys or values) of a call.
struct RopeRows {
  const void *in;
  long long ss, sb, sh;  // element strides of in: s, b, head
  const void *gin;       // backward: the gradient of the output, dense
  void *out;             // dense [S, B, heads, D], or the paged cache
  long long ps, ts, hs;  // cache strides: page, token, head
  const float *w;        // nullptr: no norm
  int heads;
};

struct RopeArgs {
  RopeRows q, k, v;
  int S, B, D;
  int r0, R, interleaved;
  float eps, mscale;
  const int32_t *pos;      // [S, B] or nullptr (row s at position s)
  const double *inv_freq;  // [R / 2] radians a position
  // append: page table [B, max_pages] of pages [0, num_pages)
  const int32_t *table;
  int max_pages, page_size, num_pages;
  int *status;
  int heads_per_item, chunks;  // heads of one token that a warp takes
  float *partial;              // backward: [CTAs][2][D] weight gradients
};

template <typename T>
struct Cvt;
template <>
struct Cvt<__nv_bfloat16> {
  static __device__ float to(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __nv_bfloat16 from(float x) { return __float2bfloat16(x); }
};
template <>
struct Cvt<__half> {
  static __device__ float to(__half x) { return __half2float(x); }
  static __device__ __half from(float x) { return __float2half(x); }
};
template <>
struct Cvt<float> {
  static __device__ float to(float x) { return x; }
  static __device__ float from(float x) { return x; }
};

// Eight consecutive values of a row as fp32 (zeros past D).
template <typename T, bool VEC>
struct Chunk {
  alignas(16) T raw[8];
  __device__ __forceinline__ void load(const T *p, int e0, int D) {
    if constexpr (VEC) {
      if (e0 < D) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(raw) / 16; ++i)
          reinterpret_cast<uint4 *>(raw)[i] =
              __ldg(reinterpret_cast<const uint4 *>(p + e0) + i);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) raw[i] = Cvt<T>::from(0.f);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        raw[i] = e0 + i < D ? p[e0 + i] : Cvt<T>::from(0.f);
    }
  }
  __device__ __forceinline__ void get(float2 (&x)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        x[i] = make_float2(raw[2 * i], raw[2 * i + 1]);
      } else {
        const uint32_t w = reinterpret_cast<const uint32_t *>(raw)[i];
        if constexpr (std::is_same<T, __half>::value)
          x[i] = __half22float2(reinterpret_cast<const __half2 &>(w));
        else
          x[i] = make_float2(__uint_as_float(w << 16),
                             __uint_as_float(w & 0xffff0000u));
      }
    }
  }
  __device__ __forceinline__ void set(const float2 (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4)
        raw[2 * i] = x[i].x, raw[2 * i + 1] = x[i].y;
      else if constexpr (std::is_same<T, __half>::value)
        reinterpret_cast<__half2 *>(raw)[i] = __float22half2_rn(x[i]);
      else
        reinterpret_cast<uint32_t *>(raw)[i] = pack_bf16x2(x[i].x, x[i].y);
    }
  }
  __device__ __forceinline__ void store(T *p, int e0, int D) const {
    if constexpr (VEC) {
      if (e0 < D) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(raw) / 16; ++i)
          reinterpret_cast<uint4 *>(p + e0)[i] =
              reinterpret_cast<const uint4 *>(raw)[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e0 + i < D) p[e0 + i] = raw[i];
    }
  }
};

// Frequencies as turns a position, 64-bit fixed point.  Lanes outside the
// rotated part multiply the first eight coefficients of `cs` by zero; without a
// rotation nothing else writes them, and what is there may not be finite.
__device__ __forceinline__ void load_freqs(
    const RopeArgs &a, unsigned long long *fr,
    float2 (&cs)[kRopeWarps][kRopeMaxD / 2]) {
  if (a.R == 0 && threadIdx.x < kRopeWarps * 8)
    cs[threadIdx.x / 8][threadIdx.x % 8] = make_float2(0.f, 0.f);
  for (int i = threadIdx.x; i < a.R / 2; i += kRopeThreads) {
    double t = a.inv_freq[i] * 0.15915494309189535;  // 1 / (2 pi)
    t -= floor(t);
    fr[i] = __double2ull_rn(t * 18446744073709551616.0);
  }
}

// cos and sin (times m) of a token's angles into `cs`, by one warp.
__device__ __forceinline__ void token_turns(const RopeArgs &a, int pos,
                                            int lane,
                                            const unsigned long long *fr,
                                            float2 *cs) {
  __syncwarp();
  for (int i = lane; i < a.R / 2; i += 32) {
    const unsigned long long ph = (unsigned long long)(long long)pos * fr[i];
    // the top half as a signed fraction of half a turn
    const float x = (float)(int)(unsigned)(ph >> 32) * 4.656612873077393e-10f;
    float sn, co;
    sincospif(x, &sn, &co);
    cs[i] = make_float2(a.mscale * co, a.mscale * sn);
  }
  __syncwarp();
}

// The rotation's coefficients of a lane's 8 elements, with the weights where
// given: y_e = x_e c + x_partner s (times the row's rstd); s = 0 outside the
// rotated part.  There x_partner is left out where it may not be finite (an
// infinity stays one): `plain` says that the lane's elements all are.
// Arithmetic on pairs (two fp32 a register pair and instruction).
template <typename T, bool VEC>
struct Turn {
  float2 c[4], s[4];
  int src_lane;      // lane of the partners (halves layout, 16-byte pieces)
  unsigned rotated;  // a bit for each element with a partner

  int p0;            // VEC: first pair of the lane's chunk
  float sign;        // VEC, halves: of s

  static __device__ __forceinline__ int partner(const RopeArgs &a, int e) {
    const int rel = e - a.r0;
    if (rel < 0 || rel >= a.R) return e;
    if (a.interleaved) return a.r0 + (rel ^ 1);
    return rel < a.R / 2 ? e + a.R / 2 : e - a.R / 2;
  }
  // What stays the same from token to token; `back` turns the other way.
  __device__ __forceinline__ void init(const RopeArgs &a, int e0, int lane,
                                       bool back) {
    const int rel0 = e0 - a.r0;
    const bool first = a.interleaved || rel0 < a.R / 2;
    src_lane = lane;
    rotated = 0u;
    p0 = 0;
    sign = first != back ? -1.f : 1.f;
    if (VEC) {
      if (rel0 >= 0 && rel0 < a.R) {
        rotated = 0xffu;
        p0 = a.interleaved ? rel0 / 2 : first ? rel0 : rel0 - a.R / 2;
        if (!a.interleaved)
          src_lane = first ? lane + a.R / 16 : lane - a.R / 16;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (rel0 + i >= 0 && rel0 + i < a.R && e0 + i < a.D)
          rotated |= 1u << i;
    }
  }
  // The token's coefficients.  `w`: the weights in shared memory (zeros past
  // D), or nullptr.
  __device__ __forceinline__ void set(const RopeArgs &a, int e0, bool back,
                                      const float2 *cs, const float *w) {
    if constexpr (VEC) {
      const float4 *q = reinterpret_cast<const float4 *>(cs + p0);
      const float one = rotated ? 0.f : 1.f, turn = rotated ? 1.f : 0.f;
      if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // two pairs
          const float4 v = q[i];
          c[2 * i] = make_float2(fmaf(v.x, turn, one), fmaf(v.x, turn, one));
          c[2 * i + 1] = make_float2(fmaf(v.z, turn, one),
                                     fmaf(v.z, turn, one));
          s[2 * i] = make_float2(v.y * turn * sign, -v.y * turn * sign);
          s[2 * i + 1] = make_float2(v.w * turn * sign, -v.w * turn * sign);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 v = q[i];
          c[i] = make_float2(fmaf(v.x, turn, one), fmaf(v.z, turn, one));
          s[i] = make_float2(v.y * turn * sign, v.w * turn * sign);
        }
      }
      if (w) {
        // the partners' weights: the halves' other chunk, or the neighbours
        const int eo = a.interleaved || !rotated ? e0
                       : e0 - a.r0 < a.R / 2     ? e0 + a.R / 2
                                                 : e0 - a.R / 2;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4 m = *reinterpret_cast<const float4 *>(w + e0 + 4 * i);
          const float4 o = *reinterpret_cast<const float4 *>(w + eo + 4 * i);
          c[2 * i] = __fmul2_rn(c[2 * i], make_float2(m.x, m.y));
          c[2 * i + 1] = __fmul2_rn(c[2 * i + 1], make_float2(m.z, m.w));
          s[2 * i] = __fmul2_rn(s[2 * i], a.interleaved
                                              ? make_float2(o.y, o.x)
                                              : make_float2(o.x, o.y));
          s[2 * i + 1] = __fmul2_rn(s[2 * i + 1], a.interleaved
                                                      ? make_float2(o.w, o.z)
                                                      : make_float2(o.z, o.w));
        }
      }
    } else {
      float cc[8], ss[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int rel = e0 + i - a.r0;
        cc[i] = 1.f;
        ss[i] = 0.f;
        if (rotated >> i & 1u) {
          const int pi =
              a.interleaved ? rel >> 1 : rel < a.R / 2 ? rel : rel - a.R / 2;
          const bool first = a.interleaved ? (rel & 1) == 0 : rel < a.R / 2;
          const float2 v = cs[pi];
          cc[i] = v.x;
          ss[i] = first != back ? -v.y : v.y;
        }
        if (w && e0 + i < a.D) {
          cc[i] *= w[e0 + i];
          ss[i] *= w[partner(a, e0 + i)];
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[i] = make_float2(cc[2 * i], cc[2 * i + 1]);
        s[i] = make_float2(ss[2 * i], ss[2 * i + 1]);
      }
    }
  }
  // y = x turned.  `buf`: the row's LPR * 8 floats of shared memory.
  __device__ __forceinline__ void apply(const RopeArgs &a,
                                        const Chunk<T, VEC> &ch,
                                        const float2 (&x)[4], float2 (&y)[4],
                                        int e0, float *buf, bool plain) const {
    float2 o[4];
    if constexpr (VEC) {  // a chunk is turned whole or not at all
      if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = make_float2(x[i].y, x[i].x);
      } else {
        Chunk<T, VEC> from;
#pragma unroll
        for (int i = 0; i < (int)sizeof(ch.raw) / 4; ++i)
          reinterpret_cast<uint32_t *>(from.raw)[i] = __shfl_sync(
              0xffffffffu, reinterpret_cast<const uint32_t *>(ch.raw)[i],
              src_lane);
        from.get(o);
      }
    } else {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i)
        buf[e0 + 2 * i] = x[i].x, buf[e0 + 2 * i + 1] = x[i].y;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = e0 + 2 * i;  // past D: zero
        o[i].x = e < a.D ? buf[partner(a, e)] : 0.f;
        o[i].y = e + 1 < a.D ? buf[partner(a, e + 1)] : 0.f;
      }
    }
    if (!plain) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (!(rotated >> (2 * i) & 1u)) o[i].x = 0.f;
        if (!(rotated >> (2 * i + 1) & 1u)) o[i].y = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      y[i] = __ffma2_rn(x[i], c[i], __fmul2_rn(o[i], s[i]));
  }
};

// Sum of squares of a lane's elements.
__device__ __forceinline__ float squares(const float2 (&x)[4]) {
  float2 t = __fmul2_rn(x[0], x[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) t = __ffma2_rn(x[i], x[i], t);
  return t.x + t.y;
}

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = LPR / 2; o >= 1; o >>= 1)
    x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Both sets' weights into shared memory, zeros past D.
__device__ __forceinline__ void load_weights(const RopeArgs &a,
                                             float (&sw)[2][kRopeMaxD]) {
  for (int i = threadIdx.x; i < 2 * kRopeMaxD; i += kRopeThreads) {
    const float *w = i < kRopeMaxD ? a.q.w : a.k.w;
    const int e = i % kRopeMaxD;
    sw[i / kRopeMaxD][e] = w && e < a.D ? __ldg(w + e) : 0.f;
  }
}

// Row groups whose loads a warp has in flight.
constexpr int kBatch = 4;

// A warp's share of one token: heads [h0, h1) of the row set `r`.
// KIND 0: queries, 1: keys, 2: values (copied).  `dst0`: the token's first
// head in the output, heads `dh` elements apart; nullptr: not written.
template <typename T, bool VEC, int LPR, int KIND>
__device__ __forceinline__ void rope_heads(const RopeArgs &a,
                                           const RopeRows &r, const T *src0,
                                           T *dst0, long long dh, int h0,
                                           int h1, int sub, int e0,
                                           Turn<T, VEC> &turn,
                                           const float2 *cs, const float *w,
                                           float *buf) {
  constexpr int RPW = 32 / LPR;
  if (h0 >= h1) return;
  const bool norm = KIND < 2 && r.w != nullptr;
  Chunk<T, VEC> x[kBatch];
  auto fetch = [&](int hb) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int h = hb + u * RPW + sub;
      x[u].load(src0 + h * r.sh, e0, h < h1 ? a.D : 0);
    }
  };
  fetch(h0);  // on the way while the coefficients are made
  if (KIND < 2) turn.set(a, e0, false, cs, norm ? w : nullptr);
  const float over_d = 1.f / a.D;
  for (int hb = h0;;) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int h = hb + u * RPW + sub;
      if (hb + u * RPW >= h1) break;
      if constexpr (KIND < 2) {
        float2 n[4], y[4];
        x[u].get(n);
        const float sq = squares(n);
        turn.apply(a, x[u], n, y, e0, buf, sq < 3e38f);
        if (norm) {
          const float r2 = rsqrtf(row_sum<LPR>(sq) * over_d + a.eps);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            y[i] = __fmul2_rn(y[i], make_float2(r2, r2));
        }
        x[u].set(y);
      }
      if (h < h1 && dst0) x[u].store(dst0 + h * dh, e0, a.D);
    }
    hb += kBatch * RPW;
    if (hb >= h1) break;
    fetch(hb);
  }
}

// PAGED: k and v rows go to the cache; without it there is no v.
// Append, measured: 8192 tokens of 40 + 2 x 8 rows of 64: 33 us, 3.5 TB/s of
// 114 MB: a warp has two or three tokens, and for each a chain of the position,
// its page and five batches of rows.  One token of 64 sequences: 5 us.
template <typename T, bool VEC, int LPR, bool PAGED>
__global__ void __launch_bounds__(kRopeThreads, rope_ctas(sizeof(T), VEC))
    norm_rope_kernel(const RopeArgs a) {
  constexpr int RPW = 32 / LPR;
  __shared__ __align__(16) float xch[VEC ? 1 : kRopeWarps * RPW * LPR * 8];
  __shared__ unsigned long long fr[kRopeMaxD / 2];
  __shared__ __align__(16) float2 cs[kRopeWarps][kRopeMaxD / 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / LPR, e0 = (lane % LPR) * 8;
  float *buf = VEC ? xch : xch + (warp * RPW + sub) * LPR * 8;
  // below 2^31: only few tokens are cut into chunks
  const unsigned items = (unsigned)a.S * a.B * a.chunks;
  const int nq = a.q.heads, nk = a.k.heads, nv = a.v.heads;
  __shared__ __align__(16) float sw[2][kRopeMaxD];
  load_weights(a, sw);
  load_freqs(a, fr, cs);
  __syncthreads();
  Turn<T, VEC> turn;
  turn.init(a, e0, lane, false);
  const unsigned stride = gridDim.x * kRopeWarps;
  const unsigned item0 = blockIdx.x * kRopeWarps + warp;
  // (a position is asked for one item ahead)
  auto position = [&](unsigned item) {
    const unsigned tk = item / (unsigned)a.chunks;
    return item >= items ? 0
           : a.pos       ? __ldg(a.pos + tk)
                         : (int)(tk / (unsigned)a.B);
  };
  int next_pos = position(item0);
  for (unsigned item = item0; item < items; item += stride) {
    const unsigned tk = item / (unsigned)a.chunks;
    const long long tok = tk;
    const int s = (int)(tk / (unsigned)a.B), b = (int)(tk % (unsigned)a.B);
    const int h0 = (int)(item % (unsigned)a.chunks) * a.heads_per_item;
    const int h1 = h0 + a.heads_per_item;
    const int pos = next_pos;
    next_pos = position(item + stride);
    const int k0 = max(h0 - nq, 0), k1 = min(h1 - nq, nk);
    const int v0 = max(h0 - nq - nk, 0), v1 = min(h1 - nq - nk, nv);
    int page = -1;
    if constexpr (PAGED) {
      if (pos >= 0 && h1 > nq) {
        const int pg = pos / a.page_size;
        if (pg < a.max_pages)
          page = __ldg(a.table + (long long)b * a.max_pages + pg);
      }
    }
    token_turns(a, pos, lane, fr, cs[warp]);
    auto src = [&](const RopeRows &r) {
      return static_cast<const T *>(r.in) + s * r.ss + b * r.sb;
    };
    rope_heads<T, VEC, LPR, 0>(
        a, a.q, src(a.q), static_cast<T *>(a.q.out) + tok * nq * (long long)a.D,
        a.D, min(h0, nq), min(h1, nq), sub, e0, turn, cs[warp], sw[0], buf);
    if constexpr (PAGED) {
      if (pos < 0 || h1 <= nq) continue;
      if (page < 0 || page >= a.num_pages) {
        if (lane == 0) atomicOr(a.status, kStatusIndexRange);
        continue;
      }
      const long long off = pos % a.page_size;
      rope_heads<T, VEC, LPR, 1>(
          a, a.k, src(a.k),
          static_cast<T *>(a.k.out) + page * a.k.ps + off * a.k.ts, a.k.hs, k0,
          k1, sub, e0, turn, cs[warp], sw[1], buf);
      rope_heads<T, VEC, LPR, 2>(
          a, a.v, src(a.v),
          static_cast<T *>(a.v.out) + page * a.v.ps + off * a.v.ts, a.v.hs, v0,
          v1, sub, e0, turn, cs[warp], sw[1], buf);
    } else {
      rope_heads<T, VEC, LPR, 1>(
          a, a.k, src(a.k),
          static_cast<T *>(a.k.out) + tok * nk * (long long)a.D, a.D, k0, k1,
          sub, e0, turn, cs[warp], sw[1], buf);
    }
  }
}

// Backward.  With u = the output's gradient rotated back (times m), xh = x
// rstd:  dw += u xh;  g = u w;  dx = rstd (g - xh mean(g xh)); without a
// weight there is no norm either: dx = u.
// Measured: 8192 tokens of 40 heads of 128 in bf16, 252 MB: 60 us, 4.2 TB/s,
// and 8 more for the sum of the weights' parts.  Two inputs and the
// coefficients take 128 registers a thread, so 16 warps an SM have loads in
// flight instead of 24; each has the next two row groups on the way while it
// works on two (one batch of four after the other: 2.4 us more).  fp32 has
// registers for less and spills some 200 bytes a thread; at 32768 tokens of 72
// heads it runs at 5.5 TB/s all the same (661 us, caches cold) and bf16 at 4.9
// (369), so four CTAs an SM stay the rule for every type.
template <typename T, bool VEC, int LPR>
__device__ __forceinline__ void rope_heads_bwd(const RopeArgs &a,
                                               const RopeRows &r,
                                               const T *src0, long long at0,
                                               int h0, int h1, int sub,
                                               int e0, Turn<T, VEC> &turn,
                                               const float *sw, float *buf,
                                               float2 (&dw)[4]) {
  constexpr int RPW = 32 / LPR, U = 2;
  if (h0 >= h1) return;
  const bool norm = r.w != nullptr;
  const T *gin = static_cast<const T *>(r.gin) + at0;
  T *out = static_cast<T *>(r.out) + at0;
  float2 w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = *reinterpret_cast<const float2 *>(sw + e0 + 2 * i);
  const float over_d = 1.f / a.D;
  auto fetch = [&](Chunk<T, VEC> (&x)[U], Chunk<T, VEC> (&g)[U], int hb) {
#pragma unroll
    for (int v = 0; v < U; ++v) {
      const int h = hb + v * RPW + sub;
      g[v].load(gin + (long long)h * a.D, e0, h < h1 ? a.D : 0);
      x[v].load(src0 + h * r.sh, e0, norm && h < h1 ? a.D : 0);
    }
  };
  auto work = [&](Chunk<T, VEC> (&x)[U], Chunk<T, VEC> (&g)[U], int hb) {
#pragma unroll
    for (int v = 0; v < U; ++v) {
      const int h = hb + v * RPW + sub;
      if (hb + v * RPW >= h1) break;
      float2 u[4], y[4];
      g[v].get(y);
      turn.apply(a, g[v], y, u, e0, buf, squares(y) < 3e38f);
      if (norm) {
        float2 xh[4], gw[4];
        x[v].get(xh);
        float2 dot = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          gw[i] = __fmul2_rn(u[i], w[i]);
          dot = __ffma2_rn(gw[i], xh[i], dot);
        }
        // padding of a last group (h >= h1) is a row of zeros, whose root may
        // be infinite (eps = 0): it adds nothing to dw
        const float ms = row_sum<LPR>(squares(xh)) * over_d + a.eps;
        const float rstd = h < h1 ? rsqrtf(ms) : 0.f;
        // mean(g xh)
        const float back = row_sum<LPR>(dot.x + dot.y) * rstd * over_d;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          xh[i] = __fmul2_rn(xh[i], make_float2(rstd, rstd));
          dw[i] = __ffma2_rn(u[i], xh[i], dw[i]);
          u[i] = __fmul2_rn(
              make_float2(rstd, rstd),
              __ffma2_rn(xh[i], make_float2(-back, -back), gw[i]));
        }
      }
      g[v].set(u);
      if (h < h1) g[v].store(out + (long long)h * a.D, e0, a.D);
    }
  };
  Chunk<T, VEC> xa[U], ga[U], xb[U], gb[U];
  fetch(xa, ga, h0);
  for (int hb = h0; hb < h1; hb += 2 * U * RPW) {
    fetch(xb, gb, hb + U * RPW);
    work(xa, ga, hb);
    fetch(xa, ga, hb + 2 * U * RPW);
    work(xb, gb, hb + U * RPW);
  }
}

template <typename T, bool VEC, int LPR>
__global__ void __launch_bounds__(kRopeThreads, kRopeBwdCtas)
    norm_rope_bwd_kernel(const RopeArgs a) {
  constexpr int RPW = 32 / LPR;
  __shared__ __align__(16) float xch[kRopeWarps * RPW * LPR * 8];
  __shared__ unsigned long long fr[kRopeMaxD / 2];
  __shared__ __align__(16) float2 cs[kRopeWarps][kRopeMaxD / 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / LPR, e0 = (lane % LPR) * 8;
  float *buf = xch + (warp * RPW + sub) * LPR * 8;
  // below 2^31: only few tokens are cut into chunks
  const unsigned items = (unsigned)a.S * a.B * a.chunks;
  const int nq = a.q.heads, nk = a.k.heads;
  __shared__ __align__(16) float sw[2][kRopeMaxD];
  load_weights(a, sw);
  load_freqs(a, fr, cs);
  __syncthreads();
  float2 dw[2][4] = {};
  Turn<T, VEC> turn;
  turn.init(a, e0, lane, true);
  for (unsigned item = blockIdx.x * kRopeWarps + warp; item < items;
       item += gridDim.x * kRopeWarps) {
    const unsigned tk = item / (unsigned)a.chunks;
    const long long tok = tk;
    const int s = (int)(tk / (unsigned)a.B), b = (int)(tk % (unsigned)a.B);
    const int h0 = (int)(item % (unsigned)a.chunks) * a.heads_per_item;
    const int h1 = h0 + a.heads_per_item;
    token_turns(a, a.pos ? __ldg(a.pos + tok) : s, lane, fr, cs[warp]);
    turn.set(a, e0, true, cs[warp], nullptr);
    auto src = [&](const RopeRows &r) {
      return static_cast<const T *>(r.in) + s * r.ss + b * r.sb;
    };
    rope_heads_bwd<T, VEC, LPR>(a, a.q, src(a.q), tok * nq * (long long)a.D,
                                min(h0, nq), min(h1, nq), sub, e0, turn, sw[0],
                                buf, dw[0]);
    rope_heads_bwd<T, VEC, LPR>(a, a.k, src(a.k), tok * nk * (long long)a.D,
                                max(h0 - nq, 0), min(h1 - nq, nk), sub, e0,
                                turn, sw[1], buf, dw[1]);
  }
  // this CTA's weight gradients, summed over its rows in a fixed order
  for (int kind = 0; kind < 2; ++kind) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
      reinterpret_cast<float2 *>(xch)[((warp * RPW + sub) * LPR * 8 + e0) / 2 +
                                      i] = dw[kind][i];
    __syncthreads();
    for (int e = threadIdx.x; e < a.D; e += kRopeThreads) {
      float t = 0.f;
      for (int r = 0; r < kRopeWarps * RPW; ++r) t += xch[r * LPR * 8 + e];
      a.partial[((size_t)blockIdx.x * 2 + kind) * a.D + e] = t;
    }
  }
}

// Sums the CTAs' partial weight gradients: a CTA takes 32 columns, each warp
// every 32nd part.
__global__ void __launch_bounds__(1024)
    rope_dw_kernel(const float *partial, int ctas, int D, float *gwq,
                   float *gwk) {
  __shared__ float part[32][33];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + lane, kind = blockIdx.y;
  float *out = kind == 0 ? gwq : gwk;
  float t = 0.f;
  if (e < D) {
#pragma unroll 4
    for (int c = g; c < ctas; c += 32)
      t += partial[((size_t)c * 2 + kind) * D + e];
  }
  part[g][lane] = t;
  __syncthreads();
  if (g == 0 && e < D && out) {
    t = 0.f;
    for (int i = 0; i < 32; ++i) t += part[i][lane];
    out[e] = t;
  }
}

bool aligned(const void *p, unsigned n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

// 16-byte pieces are possible for this row set.
bool vec_rows(const RopeRows &r, int el, bool paged_out) {
  if (r.heads == 0) return true;
  const int m = 16 / el;
  bool ok = aligned(r.in, 16) && r.ss % m == 0 && r.sb % m == 0 &&
            r.sh % m == 0 && aligned(r.out, 16) && aligned(r.gin, 16);
  if (paged_out)
    ok = ok && r.ps % m == 0 && r.ts % m == 0 && r.hs % m == 0;
  return ok;
}

enum { kModeFwd, kModeAppend, kModeBwd };

template <typename T, bool VEC, int LPR>
cudaError_t launch_lpr(RopeArgs &a, int mode, int num_sms, int *ctas,
                       cudaStream_t st) {
  constexpr int RPW = 32 / LPR;
  const int heads = a.q.heads + a.k.heads + a.v.heads;
  const long long toks = (long long)a.S * a.B;
  // Heads per warp: all heads of a token share the coefficients, but a few
  // tokens have to be spread over the GPU: halve until there are 32 warps an
  // SM or one row group a warp is left.
  int per = (heads + RPW - 1) / RPW * RPW;
  while (per > RPW && toks * ((heads + per - 1) / per) < 32ll * num_sms)
    per = ((per / 2) + RPW - 1) / RPW * RPW;
  a.heads_per_item = per;
  a.chunks = (heads + per - 1) / per;
  const long long items = toks * a.chunks;
  const long long grid = (items + kRopeWarps - 1) / kRopeWarps;
  long long most = (long long)num_sms *
                   (mode == kModeBwd ? kRopeBwdCtas : rope_ctas(sizeof(T), VEC));
  if (most > kRopeMaxCtas) most = kRopeMaxCtas;
  *ctas = (int)(grid < most ? grid : most);
  if (mode == kModeBwd) {
    norm_rope_bwd_kernel<T, VEC, LPR><<<*ctas, kRopeThreads, 0, st>>>(a);
  } else if (mode == kModeAppend) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
      norm_rope_kernel<T, VEC, LPR, true>
          <<<*ctas, kRopeThreads, 0, st>>>(a);
  } else {
    norm_rope_kernel<T, VEC, LPR, false>
        <<<*ctas, kRopeThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_rope(RopeArgs &a, int mode, int num_sms, int *ctas,
                        cudaStream_t st) {
  const int el = (int)sizeof(T);
  const bool paged = mode == kModeAppend;
  const bool vec = a.D % 8 == 0 && a.r0 % 8 == 0 &&
                   a.R % (a.interleaved ? 8 : 16) == 0 &&
                   vec_rows(a.q, el, false) && vec_rows(a.k, el, paged) &&
                   vec_rows(a.v, el, paged);
  const int ch = (a.D + 7) / 8;
  if (vec) {
    if (ch <= 8) return launch_lpr<T, true, 8>(a, mode, num_sms, ctas, st);
    if (ch <= 16) return launch_lpr<T, true, 16>(a, mode, num_sms, ctas, st);
    return launch_lpr<T, true, 32>(a, mode, num_sms, ctas, st);
  }
  if (ch <= 8) return launch_lpr<T, false, 8>(a, mode, num_sms, ctas, st);
  return launch_lpr<T, false, 32>(a, mode, num_sms, ctas, st);
}

cudaError_t launch_rope_dtype(RopeArgs &a, int dtype, int mode, int num_sms,
                              int *ctas, cudaStream_t st) {
  switch (dtype) {
    case DSA_BF16:
      return launch_rope<__nv_bfloat16>(a, mode, num_sms, ctas, st);
    case DSA_FP16: return launch_rope<__half>(a, mode, num_sms, ctas, st);
    default: return launch_rope<float>(a, mode, num_sms, ctas, st);
  }
}

// Checks shared by the three entry points (no device access).
int check_rope(const RopeArgs &a, int dtype) {
  if (a.S <= 0 || a.B <= 0 || a.D <= 0 || a.q.heads < 0 || a.k.heads < 0 ||
      a.v.heads < 0 || a.q.heads + a.k.heads <= 0)
    return DSA_ERR_INVALID_ARG;
  if (a.R < 0 || a.r0 < 0 || a.R % 2 != 0 || a.R > a.D || a.r0 > a.D - a.R)
    return DSA_ERR_INVALID_ARG;
  if (a.R > 0 && !a.inv_freq) return DSA_ERR_INVALID_ARG;
  if (!(a.eps >= 0.f) || !(a.mscale > 0.f && a.mscale < 1e30f))
    return DSA_ERR_INVALID_ARG;
  if (dtype != DSA_BF16 && dtype != DSA_FP16 && dtype != DSA_FP32)
    return DSA_ERR_UNSUPPORTED;
  if (a.D > kRopeMaxD) return DSA_ERR_UNSUPPORTED;
  if ((long long)a.S * a.B >= (1ll << 31)) return DSA_ERR_UNSUPPORTED;
  if ((long long)a.q.heads + a.k.heads + a.v.heads > (1 << 16))
    return DSA_ERR_UNSUPPORTED;
  const unsigned el = dtype == DSA_FP32 ? 4 : 2;
  if (!aligned(a.q.in, el) || !aligned(a.k.in, el) || !aligned(a.v.in, el) ||
      !aligned(a.q.out, el) || !aligned(a.k.out, el) ||
      !aligned(a.v.out, el) || !aligned(a.q.gin, el) ||
      !aligned(a.k.gin, el) || !aligned(a.q.w, 4) || !aligned(a.k.w, 4) ||
      !aligned(a.pos, 4) || !aligned(a.inv_freq, 8))
    return DSA_ERR_INVALID_ARG;
  return DSA_OK;
}

// strides: 3 element strides (s, b, head), or nullptr for dense; that of a
// dimension of one element counts for nothing.
void set_in(RopeRows &r, const void *in, const int64_t *strides, int S, int B,
            int heads, int D) {
  r.in = in;
  r.heads = in ? heads : 0;
  r.ss = strides ? strides[0] : (long long)B * heads * D;
  r.sb = strides ? strides[1] : (long long)heads * D;
  r.sh = strides ? strides[2] : D;
  if (S == 1) r.ss = 0;
  if (B == 1) r.sb = 0;
  if (heads == 1) r.sh = 0;
}

}  // namespace
}  // namespace dsa

extern "C" {

int dsa_norm_rope_fwd(const void *q, const int64_t *q_strides, const void *k,
                      const int64_t *k_strides, int dtype, int S, int B,
                      int H, int Hk, int D, const float *wq, const float *wk,
                      float eps, const int32_t *positions,
                      const double *inv_freq, int rot_start, int rot_dim,
                      int interleaved, float rot_scale, void *out_q,
                      void *out_k, void *cuda_stream) {
  if (!q || !out_q || H <= 0) return DSA_ERR_INVALID_ARG;
  if (k && (!out_k || Hk <= 0)) return DSA_ERR_INVALID_ARG;
  dsa::RopeArgs a{};
  dsa::set_in(a.q, q, q_strides, S, B, H, D);
  dsa::set_in(a.k, k, k_strides, S, B, Hk, D);
  a.q.out = out_q;
  a.k.out = out_k;
  a.q.w = wq;
  a.k.w = wk;
  a.S = S, a.B = B, a.D = D, a.r0 = rot_start, a.R = rot_dim;
  a.interleaved = interleaved != 0;
  a.eps = eps, a.mscale = rot_scale, a.pos = positions, a.inv_freq = inv_freq;
  int rc = dsa::check_rope(a, dtype);
  if (rc != DSA_OK) return rc;
  int num_sms = 0, ctas = 0;
  rc = dsa::device_num_sms(&num_sms);
  if (rc != DSA_OK) return rc;
  return dsa::launch_rope_dtype(a, dtype, dsa::kModeFwd, num_sms, &ctas,
                                static_cast<cudaStream_t>(cuda_stream)) ==
                 cudaSuccess
             ? DSA_OK
             : DSA_ERR_CUDA;
}

size_t dsa_norm_rope_bwd_workspace_size(int D) {
  if (D <= 0 || D > dsa::kRopeMaxD) return 0;
  // (the first 256 bytes stay as they are: a workspace may be shared)
  return 256 + (size_t)dsa::kRopeMaxCtas * 2 * D * sizeof(float);
}

int dsa_norm_rope_bwd(const void *q, const int64_t *q_strides, const void *k,
                      const int64_t *k_strides, const void *grad_out_q,
                      const void *grad_out_k, int dtype, int S, int B, int H,
                      int Hk, int D, const float *wq, const float *wk,
                      float eps, const int32_t *positions,
                      const double *inv_freq, int rot_start, int rot_dim,
                      int interleaved, float rot_scale, void *grad_q,
                      void *grad_k, float *grad_wq, float *grad_wk,
                      void *workspace, size_t workspace_bytes,
                      void *cuda_stream) {
  if (!q || !grad_out_q || !grad_q || H <= 0) return DSA_ERR_INVALID_ARG;
  if (k && (!grad_out_k || !grad_k || Hk <= 0)) return DSA_ERR_INVALID_ARG;
  if ((wq && !grad_wq) || (k && wk && !grad_wk)) return DSA_ERR_INVALID_ARG;
  dsa::RopeArgs a{};
  dsa::set_in(a.q, q, q_strides, S, B, H, D);
  dsa::set_in(a.k, k, k_strides, S, B, Hk, D);
  a.q.gin = grad_out_q;
  a.k.gin = grad_out_k;
  a.q.out = grad_q;
  a.k.out = grad_k;
  a.q.w = wq;
  a.k.w = k ? wk : nullptr;
  a.S = S, a.B = B, a.D = D, a.r0 = rot_start, a.R = rot_dim;
  a.interleaved = interleaved != 0;
  a.eps = eps, a.mscale = rot_scale, a.pos = positions, a.inv_freq = inv_freq;
  int rc = dsa::check_rope(a, dtype);
  if (rc != DSA_OK) return rc;
  if (!dsa::aligned(grad_wq, 4) || !dsa::aligned(grad_wk, 4))
    return DSA_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < dsa_norm_rope_bwd_workspace_size(D))
    return DSA_ERR_WORKSPACE;
  if (!dsa::aligned(workspace, 256)) return DSA_ERR_INVALID_ARG;
  a.partial =
      reinterpret_cast<float *>(static_cast<char *>(workspace) + 256);
  int num_sms = 0, ctas = 0;
  rc = dsa::device_num_sms(&num_sms);
  if (rc != DSA_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (dsa::launch_rope_dtype(a, dtype, dsa::kModeBwd, num_sms, &ctas, st) !=
      cudaSuccess)
    return DSA_ERR_CUDA;
  if (a.q.w || a.k.w) {
    dsa::rope_dw_kernel<<<dim3((D + 31) / 32, 2), 1024, 0, st>>>(
        a.partial, ctas, D, a.q.w ? grad_wq : nullptr,
        a.k.w ? grad_wk : nullptr);
    if (cudaGetLastError() != cudaSuccess) return DSA_ERR_CUDA;
  }
  return DSA_OK;
}

int dsa_paged_append(const void *k, const int64_t *k_strides, const void *v,
                     const int64_t *v_strides, const void *q,
                     const int64_t *q_strides, int S, int B, int H, int Hk,
                     int D, void *k_cache, void *v_cache,
                     const int64_t *cache_strides, int num_pages,
                     int page_size, const int32_t *page_table, int max_pages,
                     const int32_t *positions, const float *wq,
                     const float *wk, float eps, const double *inv_freq,
                     int rot_start, int rot_dim, int interleaved,
                     float rot_scale, void *out_q, void *workspace,
                     size_t workspace_bytes, void *cuda_stream) {
  if (!k || !v || !k_cache || !v_cache || !page_table || !positions ||
      Hk <= 0)
    return DSA_ERR_INVALID_ARG;
  if (q && (!out_q || H <= 0)) return DSA_ERR_INVALID_ARG;
  if (num_pages <= 0 || page_size <= 0 || max_pages <= 0)
    return DSA_ERR_INVALID_ARG;
  dsa::RopeArgs a{};
  dsa::set_in(a.q, q, q_strides, S, B, H, D);
  dsa::set_in(a.k, k, k_strides, S, B, Hk, D);
  dsa::set_in(a.v, v, v_strides, S, B, Hk, D);
  a.q.out = out_q;
  a.k.out = k_cache;
  a.v.out = v_cache;
  for (int i = 0; i < 2; ++i) {
    dsa::RopeRows &r = i == 0 ? a.k : a.v;
    const int64_t *cs = cache_strides ? cache_strides + 3 * i : nullptr;
    r.ps = cs ? cs[0] : (long long)page_size * Hk * D;
    r.ts = cs ? cs[1] : (long long)Hk * D;
    r.hs = cs ? cs[2] : D;
    if (num_pages == 1) r.ps = 0;
    if (page_size == 1) r.ts = 0;
    if (Hk == 1) r.hs = 0;
  }
  a.q.w = wq;
  a.k.w = wk;
  a.S = S, a.B = B, a.D = D, a.r0 = rot_start, a.R = rot_dim;
  a.interleaved = interleaved != 0;
  a.eps = eps, a.mscale = rot_scale, a.pos = positions, a.inv_freq = inv_freq;
  a.table = page_table;
  a.max_pages = max_pages, a.page_size = page_size, a.num_pages = num_pages;
  int rc = dsa::check_rope(a, DSA_BF16);
  if (rc != DSA_OK) return rc;
  if (!dsa::aligned(page_table, 4)) return DSA_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < 256) return DSA_ERR_WORKSPACE;
  if (!dsa::aligned(workspace, 256)) return DSA_ERR_INVALID_ARG;
  a.status = static_cast<int *>(workspace);
  int num_sms = 0, ctas = 0;
  rc = dsa::device_num_sms(&num_sms);
  if (rc != DSA_OK) return rc;
  return dsa::launch_rope_dtype(a, DSA_BF16, dsa::kModeAppend, num_sms, &ctas,
                                static_cast<cudaStream_t>(cuda_stream)) ==
                 cudaSuccess
             ? DSA_OK
             : DSA_ERR_CUDA;
}

}  // extern "C"
