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
// 16-bit types), so D = 128 puts two rows in a warp.  Rows that cannot be
// read in 16-byte pieces (odd sizes, strides or pointers) take the same code
// with element loads and the partner exchanged through shared memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "dsa_indexer.h"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
constexpr int kRopeMaxD = 256;
constexpr int kRopeBwdMaxCtas = 1216;  // partial sums of the weight gradients

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
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = Cvt<T>::to(raw[i]);
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) raw[i] = Cvt<T>::from(x[i]);
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

// The rotation's coefficients of a lane's 8 elements at one token:
// y_e = n_e c + n_partner s.
template <bool VEC>
struct Turn {
  float c[8], s[8];
  int src_lane;  // lane of the partners (halves layout, 16-byte pieces)

  __device__ __forceinline__ void setup(const RopeArgs &a, int e0, int lane) {
    src_lane = lane;
    const int rel0 = e0 - a.r0;
    if (VEC && !a.interleaved && rel0 >= 0 && rel0 < a.R)
      src_lane = rel0 < a.R / 2 ? lane + a.R / 16 : lane - a.R / 16;
  }
  // Element e's pair index, or -1 outside the rotated part.
  static __device__ __forceinline__ int pair(const RopeArgs &a, int e) {
    const int rel = e - a.r0;
    if (rel < 0 || rel >= a.R) return -1;
    if (a.interleaved) return rel >> 1;
    return rel < a.R / 2 ? rel : rel - a.R / 2;
  }
  static __device__ __forceinline__ int partner(const RopeArgs &a, int e) {
    const int rel = e - a.r0;
    if (rel < 0 || rel >= a.R) return e;
    if (a.interleaved) return a.r0 + (rel ^ 1);
    return rel < a.R / 2 ? e + a.R / 2 : e - a.R / 2;
  }
  static __device__ __forceinline__ bool first(const RopeArgs &a, int e) {
    const int rel = e - a.r0;
    return a.interleaved ? (rel & 1) == 0 : rel < a.R / 2;
  }
  __device__ __forceinline__ void at(const RopeArgs &a, int e0, int pos,
                                     bool back) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int pi = pair(a, e0 + i);
      if (pi < 0) {
        c[i] = 1.f;
        s[i] = 0.f;
        continue;
      }
      if (VEC && a.interleaved && (i & 1)) {  // the neighbour's angle
        c[i] = c[i - 1];
        s[i] = -s[i - 1];
        continue;
      }
      double t = __ldg(a.inv_freq + pi) * 0.15915494309189535;  // 1 / (2 pi)
      t -= floor(t);
      const unsigned long long f = __double2ull_rn(t * 18446744073709551616.0);
      const unsigned long long ph = (unsigned long long)(long long)pos * f;
      const float x = (float)(int)(unsigned)(ph >> 32) * 4.656612873077393e-10f;
      float sn, cs;
      sincospif(x, &sn, &cs);
      c[i] = a.mscale * cs;
      sn = a.mscale * sn;
      s[i] = first(a, e0 + i) != back ? -sn : sn;
    }
  }
  // y = rotation of n.  `buf`: the row's LPR * 8 floats of shared memory.
  __device__ __forceinline__ void apply(const RopeArgs &a, const float (&n)[8],
                                        float (&y)[8], int e0,
                                        float *buf) const {
    if constexpr (VEC) {
      if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = fmaf(n[i], c[i], n[i ^ 1] * s[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float o = __shfl_sync(0xffffffffu, n[i], src_lane);
          y[i] = fmaf(n[i], c[i], o * s[i]);
        }
      }
    } else {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) buf[e0 + i] = n[i];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float o = e0 + i < a.D ? buf[partner(a, e0 + i)] : 0.f;
        y[i] = fmaf(n[i], c[i], o * s[i]);
      }
    }
  }
};

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = LPR / 2; o >= 1; o >>= 1)
    x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ void load_w(const float *w, int e0, int D,
                                       float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = e0 + i < D ? __ldg(w + e0 + i) : 0.f;
}

// PAGED: k and v rows go to the cache; without it there is no v.
template <typename T, bool VEC, int LPR, bool PAGED>
__global__ void __launch_bounds__(kRopeThreads)
    norm_rope_kernel(const RopeArgs a) {
  constexpr int RPW = 32 / LPR;
  __shared__ float xch[VEC ? 1 : kRopeWarps * RPW * LPR * 8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / LPR, e0 = (lane % LPR) * 8;
  float *buf = VEC ? xch : xch + (warp * RPW + sub) * LPR * 8;
  const long long item = (long long)blockIdx.x * kRopeWarps + warp;
  const long long tok = item / a.chunks;
  if (tok >= (long long)a.S * a.B) return;
  const int s = (int)(tok / a.B), b = (int)(tok % a.B);
  const int heads = a.q.heads + a.k.heads + a.v.heads;
  const int h0 = (int)(item % a.chunks) * a.heads_per_item;
  const int h1 = min(heads, h0 + a.heads_per_item);
  const int pos = a.pos ? __ldg(a.pos + tok) : s;
  long long slot_k = 0, slot_v = 0;
  bool keep = true;
  if constexpr (PAGED) {
    keep = pos >= 0;
    if (keep) {
      const int pg = pos / a.page_size;
      const int page =
          pg < a.max_pages ? __ldg(a.table + (long long)b * a.max_pages + pg)
                           : -1;
      if (page < 0 || page >= a.num_pages) {
        keep = false;
        if (lane == 0) atomicOr(a.status, kStatusIndexRange);
      } else {
        const long long off = pos - pg * a.page_size;
        slot_k = page * a.k.ps + off * a.k.ts;
        slot_v = page * a.v.ps + off * a.v.ts;
      }
    }
  }
  Turn<VEC> turn;
  turn.setup(a, e0, lane);
  turn.at(a, e0, pos, false);
  for (int h = h0; h < h1; h += RPW) {
    const int hh = h + sub;
    const bool live = hh < h1;
    const int kind = hh < a.q.heads ? 0 : hh < a.q.heads + a.k.heads ? 1 : 2;
    const RopeRows &r = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    const int hr = kind == 0   ? hh
                   : kind == 1 ? hh - a.q.heads
                               : hh - a.q.heads - a.k.heads;
    Chunk<T, VEC> x;
    const T *src =
        static_cast<const T *>(r.in) + s * r.ss + b * r.sb + hr * r.sh;
    x.load(src, e0, live ? a.D : 0);
    float n[8], y[8];
    x.get(n);
    float ms = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ms = fmaf(n[i], n[i], ms);
    ms = row_sum<LPR>(ms);
    if (r.w) {
      float w[8];
      load_w(r.w, e0, a.D, w);
      const float rstd = rsqrtf(ms / a.D + a.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) n[i] *= rstd * w[i];
    }
    turn.apply(a, n, y, e0, buf);
    if (kind < 2) x.set(y);
    T *dst;
    if (PAGED && kind > 0)
      dst = static_cast<T *>(r.out) + (kind == 1 ? slot_k : slot_v) +
            hr * r.hs;
    else
      dst = static_cast<T *>(r.out) +
            (tok * r.heads + hr) * (long long)a.D;
    if (live && (keep || kind == 0)) x.store(dst, e0, a.D);
  }
}

// Backward.  With u = the output's gradient rotated back (times m), xh = x
// rstd:  dw += u xh;  g = u w;  dx = rstd (g - xh mean(g xh)).
template <typename T, bool VEC, int LPR>
__global__ void __launch_bounds__(kRopeThreads)
    norm_rope_bwd_kernel(const RopeArgs a) {
  constexpr int RPW = 32 / LPR;
  __shared__ float xch[kRopeWarps * RPW * LPR * 8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / LPR, e0 = (lane % LPR) * 8;
  float *buf = xch + (warp * RPW + sub) * LPR * 8;
  const long long items = (long long)a.S * a.B * a.chunks;
  const int heads = a.q.heads + a.k.heads;
  float dw[2][8] = {};
  Turn<VEC> turn;
  turn.setup(a, e0, lane);
  for (long long item = (long long)blockIdx.x * kRopeWarps + warp;
       item < items; item += (long long)gridDim.x * kRopeWarps) {
    const long long tok = item / a.chunks;
    const int s = (int)(tok / a.B), b = (int)(tok % a.B);
    const int h0 = (int)(item % a.chunks) * a.heads_per_item;
    const int h1 = min(heads, h0 + a.heads_per_item);
    turn.at(a, e0, a.pos ? __ldg(a.pos + tok) : s, true);
    for (int h = h0; h < h1; h += RPW) {
      const int hh = h + sub;
      const bool live = hh < h1;
      const int kind = hh < a.q.heads ? 0 : 1;
      const RopeRows &r = kind == 0 ? a.q : a.k;
      const int hr = kind == 0 ? hh : hh - a.q.heads;
      Chunk<T, VEC> g;
      const long long at = (tok * r.heads + hr) * (long long)a.D;
      g.load(static_cast<const T *>(r.gin) + at, e0, live ? a.D : 0);
      float u[8], y[8];
      g.get(y);
      turn.apply(a, y, u, e0, buf);
      // without a weight there is no norm either: dx = u.  The sums run in
      // every lane, as neighbouring rows of a warp may be of both kinds.
      const bool norm = r.w != nullptr;
      Chunk<T, VEC> x;
      x.load(static_cast<const T *>(r.in) + s * r.ss + b * r.sb + hr * r.sh,
             e0, live && norm ? a.D : 0);
      float xh[8], w[8] = {};
      x.get(xh);
      if (norm) load_w(r.w, e0, a.D, w);
      float ms = 0.f, dot = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ms = fmaf(xh[i], xh[i], ms);
        dot = fmaf(u[i] * w[i], xh[i], dot);
      }
      ms = row_sum<LPR>(ms);
      dot = row_sum<LPR>(dot);
      if (norm) {
        const float rstd = rsqrtf(ms / a.D + a.eps);
        const float back = dot * rstd / a.D;  // mean(g xh)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          xh[i] *= rstd;
          const float d = u[i] * xh[i];
          dw[0][i] += kind == 0 ? d : 0.f;
          dw[1][i] += kind == 0 ? 0.f : d;
          u[i] = rstd * fmaf(-xh[i], back, u[i] * w[i]);
        }
      }
      g.set(u);
      if (live) g.store(static_cast<T *>(r.out) + at, e0, a.D);
    }
  }
  // this CTA's weight gradients, summed over its rows in a fixed order
  for (int kind = 0; kind < 2; ++kind) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i)
      xch[(warp * RPW + sub) * LPR * 8 + e0 + i] = dw[kind][i];
    __syncthreads();
    for (int e = threadIdx.x; e < a.D; e += kRopeThreads) {
      float t = 0.f;
      for (int r = 0; r < kRopeWarps * RPW; ++r) t += xch[r * LPR * 8 + e];
      a.partial[((size_t)blockIdx.x * 2 + kind) * a.D + e] = t;
    }
  }
}

// Sums the CTAs' partial weight gradients; one warp per 32 columns.
__global__ void rope_dw_kernel(const float *partial, int ctas, int D,
                               float *gwq, float *gwk) {
  __shared__ float part[8][32];
  const int e = blockIdx.x * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
  const int kind = blockIdx.y;
  float *out = kind == 0 ? gwq : gwk;
  float t = 0.f;
  if (e < D)
    for (int c = g; c < ctas; c += 8)
      t += partial[((size_t)c * 2 + kind) * D + e];
  part[g][threadIdx.x & 31] = t;
  __syncthreads();
  if (g == 0 && e < D && out) {
    for (int i = 1; i < 8; ++i) t += part[i][threadIdx.x & 31];
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
  // tokens have to be spread over the GPU: halve until there are 32 warps
  // an SM or one row set a warp is left.
  int per = (heads + RPW - 1) / RPW * RPW;
  while (per > RPW && toks * ((heads + per - 1) / per) < 32ll * num_sms)
    per = ((per / 2) + RPW - 1) / RPW * RPW;
  a.heads_per_item = per;
  a.chunks = (heads + per - 1) / per;
  const long long items = toks * a.chunks;
  const long long grid = (items + kRopeWarps - 1) / kRopeWarps;
  if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  if (mode == kModeBwd) {
    const long long most = 8ll * num_sms < kRopeBwdMaxCtas ? 8ll * num_sms
                                                           : kRopeBwdMaxCtas;
    *ctas = (int)(grid < most ? grid : most);
    norm_rope_bwd_kernel<T, VEC, LPR><<<*ctas, kRopeThreads, 0, st>>>(a);
  } else if (mode == kModeAppend) {
    norm_rope_kernel<T, VEC, LPR, true>
        <<<(int)grid, kRopeThreads, 0, st>>>(a);
  } else {
    norm_rope_kernel<T, VEC, LPR, false>
        <<<(int)grid, kRopeThreads, 0, st>>>(a);
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
    if (ch <= 4) return launch_lpr<T, true, 4>(a, mode, num_sms, ctas, st);
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

// strides: 3 element strides (s, b, head), or nullptr for dense.
void set_in(RopeRows &r, const void *in, const int64_t *strides, int B,
            int heads, int D) {
  r.in = in;
  r.heads = in ? heads : 0;
  r.ss = strides ? strides[0] : (long long)B * heads * D;
  r.sb = strides ? strides[1] : (long long)heads * D;
  r.sh = strides ? strides[2] : D;
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
  dsa::set_in(a.q, q, q_strides, B, H, D);
  dsa::set_in(a.k, k, k_strides, B, Hk, D);
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
  return (size_t)dsa::kRopeBwdMaxCtas * 2 * D * sizeof(float);
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
  dsa::set_in(a.q, q, q_strides, B, H, D);
  dsa::set_in(a.k, k, k_strides, B, Hk, D);
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
  a.partial = static_cast<float *>(workspace);
  int num_sms = 0, ctas = 0;
  rc = dsa::device_num_sms(&num_sms);
  if (rc != DSA_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (dsa::launch_rope_dtype(a, dtype, dsa::kModeBwd, num_sms, &ctas, st) !=
      cudaSuccess)
    return DSA_ERR_CUDA;
  if (a.q.w || a.k.w) {
    dsa::rope_dw_kernel<<<dim3((D + 31) / 32, 2), 256, 0, st>>>(
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
  dsa::set_in(a.q, q, q_strides, B, H, D);
  dsa::set_in(a.k, k, k_strides, B, Hk, D);
  dsa::set_in(a.v, v, v_strides, B, Hk, D);
  a.q.out = out_q;
  a.k.out = k_cache;
  a.v.out = v_cache;
  for (int i = 0; i < 2; ++i) {
    dsa::RopeRows &r = i == 0 ? a.k : a.v;
    const int64_t *cs = cache_strides ? cache_strides + 3 * i : nullptr;
    r.ps = cs ? cs[0] : (long long)page_size * Hk * D;
    r.ts = cs ? cs[1] : (long long)Hk * D;
    r.hs = cs ? cs[2] : D;
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
