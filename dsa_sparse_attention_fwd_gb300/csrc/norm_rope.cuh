// Rows of queries and keys, their norm and the rotation of positions: what the
// kernels of norm_rope.cu and append_q8.cu share (the mathematics is written
// down in norm_rope.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "common.cuh"
#include "dsa_indexer.h"
#include "ptx.cuh"

namespace dsa {

constexpr int kRopeThreads = 128;
constexpr int kRopeWarps = kRopeThreads / 32;
constexpr int kRopeMaxD = 256;
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
__device__ __forceinline__ void token_turns(const RopeArgs &a, long long pos,
                                            int lane,
                                            const unsigned long long *fr,
                                            float2 *cs) {
  __syncwarp();
  for (int i = lane; i < a.R / 2; i += 32) {
    const unsigned long long ph = (unsigned long long)pos * fr[i];
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

inline bool aligned(const void *p, unsigned n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

// 16-byte pieces are possible for this row set.
inline bool vec_rows(const RopeRows &r, int el, bool paged_out) {
  if (r.heads == 0) return true;
  const int m = 16 / el;
  bool ok = aligned(r.in, 16) && r.ss % m == 0 && r.sb % m == 0 &&
            r.sh % m == 0 && aligned(r.out, 16) && aligned(r.gin, 16);
  if (paged_out)
    ok = ok && r.ps % m == 0 && r.ts % m == 0 && r.hs % m == 0;
  return ok;
}

// Checks shared by the entry points (no device access).
inline int check_rope(const RopeArgs &a, int dtype) {
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
inline void set_in(RopeRows &r, const void *in, const int64_t *strides, int S,
                   int B, int heads, int D) {
  r.in = in;
  r.heads = in ? heads : 0;
  r.ss = strides ? strides[0] : (long long)B * heads * D;
  r.sb = strides ? strides[1] : (long long)heads * D;
  r.sh = strides ? strides[2] : D;
  if (S == 1) r.ss = 0;
  if (B == 1) r.sb = 0;
  if (heads == 1) r.sh = 0;
}

}  // namespace dsa
