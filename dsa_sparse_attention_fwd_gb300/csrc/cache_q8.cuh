// A paged cache held in 8 bits: e4m3 values [pages, page_size, Hk, D] and for
// each `group` of consecutive tokens and head a scale, a power of two, fp32
// [pages, page_size / group, Hk].  A value is its code times its scale.
//
// A power of two, because then only the exponent of a value changes when a
// group's scale grows with a new token: the codes that are there are rounded
// again without loss (but for subnormals of e4m3), and what a cache holds does
// not depend on how its tokens were cut into calls.  The scale costs no
// precision: e4m3 is a floating format, its relative step is the same at any
// scale.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "dsa_indexer.h"

namespace dsa {

// Exponents that a scale may have.  The range (values from 2^-49 to 448 2^40)
// is far wider than what a model's keys and values take, and products of scales
// and weights stay well inside fp32.
constexpr int kQ8MinExp = -40, kQ8MaxExp = 40;

struct Q8Cache {
  uint8_t *k, *v;
  long long k_p, k_t, k_h;  // element strides: page, token, head
  long long v_p, v_t, v_h;
  float *ks, *vs;           // scales, dense
  int group, lg;            // tokens of a scale, its logarithm
  int gpp;                  // scales of a page and head
  int Hk, D;
  int page_size, num_pages, max_pages;
  const int32_t *table;  // [B, max_pages]
};

// 2^e.
__device__ __forceinline__ float q8_pow2(int e) {
  return __int_as_float((e + 127) << 23);
}

// The exponent of a stored scale; whatever else the memory holds is taken as
// the power of two at or below it, within the range.
__device__ __forceinline__ int q8_exp(float scale) {
  const int e = (__float_as_int(scale) >> 23 & 0xff) - 127;
  return min(max(e, kQ8MinExp), kQ8MaxExp);
}

// The exponent of the smallest power of two s with top <= 448 s, top >= 0
// finite; 448 = 1.75 * 2^8.  (Below 2^-126 the field says -127: clamped.)
__device__ __forceinline__ int q8_exp_for(float top) {
  const int u = __float_as_int(top);
  const int e = (u >> 23) - 127 - 8 + ((u & 0x7fffff) > 0x600000 ? 1 : 0);
  return min(max(e, kQ8MinExp), kQ8MaxExp);
}

// |x| as it counts for a scale: an infinity or a NaN does not.
__device__ __forceinline__ float q8_mag(float x) {
  const float a = fabsf(x);
  return a < __int_as_float(0x7f800000) ? a : 0.f;
}

// Two fp32 to e4m3, round to nearest even, saturating (a NaN stays one);
// `lo` in the low byte.
__device__ __forceinline__ uint32_t q8_pack2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t q8_pack4(float a, float b, float c,
                                             float d) {
  return q8_pack2(a, b) | q8_pack2(c, d) << 16;
}

// Two e4m3 (the low 16 bits) as fp16, exactly.
__device__ __forceinline__ uint32_t q8_half2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}
// Four e4m3 as two pairs of fp16.
__device__ __forceinline__ void q8_half4(uint32_t w, uint32_t &lo,
                                         uint32_t &hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ float2 q8_float2(uint32_t w) {
  const uint32_t h = q8_half2(w);
  float2 r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(h));
  return r;
}

// Page of token j of sequence b, or -1 (`bad`) where the table names none.
__device__ __forceinline__ int q8_page(const Q8Cache &c, int b, long long j,
                                       bool &bad) {
  const long long pg = j / c.page_size;
  if (j >= 0 && pg < c.max_pages) {
    const int page = __ldg(c.table + (long long)b * c.max_pages + pg);
    if (page >= 0 && page < c.num_pages) return page;
  }
  bad = true;
  return -1;
}

// Scale of the group that begins at or holds token `off` of a page.
__device__ __forceinline__ long long q8_scale_at(const Q8Cache &c, int page,
                                                 int off, int h) {
  return ((long long)page * c.gpp + (off >> c.lg)) * c.Hk + h;
}

// Checks of a cache's arguments (no device access); fills in the struct.
// Tokens of one cache may not share their memory where it is written.
inline int set_q8_cache(Q8Cache &c, const void *k, const void *v,
                        const int64_t *strides, const float *ks,
                        const float *vs, int group, int num_pages,
                        int page_size, const int32_t *table, int max_pages,
                        int Hk, int D) {
  auto al = [](const void *p, unsigned n) {
    return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
  };
  if (!table || num_pages <= 0 || page_size <= 0 || max_pages <= 0 ||
      Hk <= 0 || D <= 0 || group <= 0)
    return DSA_ERR_INVALID_ARG;
  if (group != 16 && group != 32 && group != 64 && group != 128)
    return DSA_ERR_UNSUPPORTED;
  if (page_size % group != 0 || D % 16 != 0 || D > 256 ||
      (long long)max_pages * page_size >= (1ll << 31))
    return DSA_ERR_UNSUPPORTED;
  if (!al(k, 16) || !al(v, 16) || !al(ks, 4) || !al(vs, 4) || !al(table, 4))
    return DSA_ERR_INVALID_ARG;
  c.k = static_cast<uint8_t *>(const_cast<void *>(k));
  c.v = static_cast<uint8_t *>(const_cast<void *>(v));
  c.ks = const_cast<float *>(ks);
  c.vs = const_cast<float *>(vs);
  c.group = group;
  c.lg = group == 16 ? 4 : group == 32 ? 5 : group == 64 ? 6 : 7;
  c.gpp = page_size / group;
  c.Hk = Hk, c.D = D;
  c.page_size = page_size, c.num_pages = num_pages, c.max_pages = max_pages;
  c.table = table;
  const long long dense[3] = {(long long)page_size * Hk * D, (long long)Hk * D,
                              D};
  long long *to[6] = {&c.k_p, &c.k_t, &c.k_h, &c.v_p, &c.v_t, &c.v_h};
  for (int i = 0; i < 6; ++i) {
    const long long s = strides ? strides[i] : dense[i % 3];
    if (s < 0 || s >= (1ll << 40)) return DSA_ERR_INVALID_ARG;
    // a dimension of one element may have any stride
    const bool one = i % 3 == 0 ? num_pages == 1 : i % 3 == 1 ? page_size == 1
                                                              : Hk == 1;
    *to[i] = one ? 0 : s;
    if (!one && (s == 0 || s % 16 != 0)) return DSA_ERR_INVALID_ARG;
  }
  return DSA_OK;
}

}  // namespace dsa
