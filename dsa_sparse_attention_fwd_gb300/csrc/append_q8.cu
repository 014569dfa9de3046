// Append to a paged cache held in 8 bits (cache_q8.cuh), the keys normed and
// rotated on the way (norm_rope.cuh), the queries too; and the read back.
//
// Sequence b appends its first n = count[b] rows at positions p = start[b] ..
// start[b] + n - 1.  For each group of the cache that they reach and each head,
//     s = 2^e, the smallest with max |x| <= 448 s over the group's new rows x;
// where the group holds earlier tokens (it begins before start[b]), s is not
// smaller than the scale s0 that it has, and their codes c become
// round(c s0 / s) where it is larger.  New codes are round(x / s).
#include "cache_q8.cuh"
#include "norm_rope.cuh"

namespace dsa {
namespace {

struct AppendQ8 {
  RopeArgs a;  // a.k, a.v: inputs only
  Q8Cache c;
  const int32_t *start, *count;  // [B]; count nullptr: all S rows
  int groups;                    // groups that a sequence's rows can reach
};

// The rows of a sequence that are appended: [0, n).
__device__ __forceinline__ int rows_of(const AppendQ8 &p, int b, int start) {
  const int n = p.count ? __ldg(p.count + b) : p.a.S;
  return start < 0 ? 0 : min(max(n, 0), p.a.S);
}

// A row's values, normed and rotated, into y[0 .. D) of shared memory; one
// warp.
__device__ __forceinline__ void turned_row(const RopeArgs &a, const RopeRows &r,
                                           const __nv_bfloat16 *x, bool turn,
                                           long long pos, float *n, float *y,
                                           int lane) {
  float sq = 0.f;
  for (int e = lane; e < a.D; e += 32) {
    n[e] = __bfloat162float(x[e]);
    sq = fmaf(n[e], n[e], sq);
  }
  if (turn && r.w) {
    for (int o = 16; o; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    const float rstd = rsqrtf(sq / a.D + a.eps);
    for (int e = lane; e < a.D; e += 32) n[e] = n[e] * rstd * __ldg(r.w + e);
  }
  __syncwarp();
  for (int e = lane; e < a.D; e += 32) {
    const int rel = e - a.r0;
    float v = n[e];
    if (turn && rel >= 0 && rel < a.R) {
      const bool first = a.interleaved ? (rel & 1) == 0 : rel < a.R / 2;
      const int i = a.interleaved ? rel >> 1 : rel % (a.R / 2);
      const int o = a.r0 + (a.interleaved ? rel ^ 1
                            : first       ? rel + a.R / 2
                                          : rel - a.R / 2);
      double t = a.inv_freq[i] * 0.15915494309189535;
      t -= floor(t);
      const unsigned long long ph =
          (unsigned long long)pos * __double2ull_rn(t * 18446744073709551616.0);
      float sn, co;
      sincospif((float)(int)(unsigned)(ph >> 32) * 4.656612873077393e-10f, &sn,
                &co);
      v = a.mscale * (first ? v * co - n[o] * sn : n[o] * sn + v * co);
    }
    y[e] = v;
  }
  __syncwarp();
}

// One warp an item: a query row, or a (group, head) of keys or values.
__global__ void __launch_bounds__(128) append_q8_kernel(const AppendQ8 p) {
  __shared__ float sn[4][256], sy[4][256];
  const RopeArgs &a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float *n = sn[warp], *y = sy[warp];
  const long long qrows = (long long)a.S * a.B * a.q.heads;
  const long long kv = (long long)p.groups * a.B * a.k.heads * 2;
  for (long long it = (long long)blockIdx.x * 4 + warp; it < qrows + kv;
       it += (long long)gridDim.x * 4) {
    if (it < qrows) {
      const int h = (int)(it % a.q.heads);
      const long long tok = it / a.q.heads;
      const int s = (int)(tok / a.B), b = (int)(tok % a.B);
      const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(a.q.in) +
                               s * a.q.ss + b * a.q.sb + h * a.q.sh;
      turned_row(a, a.q, x, true, (long long)__ldg(p.start + b) + s, n, y,
                 lane);
      __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.q.out) + it * a.D;
      for (int e = lane; e < a.D; e += 32) out[e] = __float2bfloat16(y[e]);
      __syncwarp();
      continue;
    }
    long long r = it - qrows;
    const bool is_v = r & 1;
    r >>= 1;
    const int h = (int)(r % a.k.heads);
    r /= a.k.heads;
    const int b = (int)(r % a.B), gi = (int)(r / a.B);
    const int start = __ldg(p.start + b);
    const int rows = rows_of(p, b, start);
    const long long g0 = ((long long)(start >> p.c.lg) + gi) << p.c.lg;
    const int s0 = (int)max(g0 - start, 0ll);
    const int s1 = (int)min(g0 + p.c.group - start, (long long)rows);
    if (s0 >= s1) continue;
    bool bad = false;
    const int page = q8_page(p.c, b, g0, bad);
    if (bad) {
      if (lane == 0) atomicOr(a.status, kStatusIndexRange);
      continue;
    }
    const int off = (int)(g0 % p.c.page_size);
    const RopeRows &in = is_v ? a.v : a.k;
    const __nv_bfloat16 *src =
        static_cast<const __nv_bfloat16 *>(in.in) + b * in.sb + h * in.sh;
    uint8_t *dst = (is_v ? p.c.v + page * p.c.v_p + h * p.c.v_h
                         : p.c.k + page * p.c.k_p + h * p.c.k_h);
    const long long st = is_v ? p.c.v_t : p.c.k_t;
    float *scale = (is_v ? p.c.vs : p.c.ks) + q8_scale_at(p.c, page, off, h);
    float top = 0.f;
    for (int s = s0; s < s1; ++s) {
      turned_row(a, in, src + s * in.ss, !is_v, (long long)start + s, n, y,
                 lane);
      for (int e = lane; e < a.D; e += 32) top = fmaxf(top, q8_mag(y[e]));
      __syncwarp();
    }
    for (int o = 16; o; o >>= 1)
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    int e = q8_exp_for(top);
    const int early = (int)max((long long)start - g0, 0ll);
    if (early > 0) {
      const int e0 = q8_exp(*scale);
      if (e > e0) {
        const float f = q8_pow2(e0 - e);
        for (int t = 0; t < early; ++t)
          for (int d = lane * 2; d < a.D; d += 64) {
            uint16_t *at =
                reinterpret_cast<uint16_t *>(dst + (off + t) * st + d);
            const float2 v = q8_float2(*at);
            *at = (uint16_t)q8_pack2(v.x * f, v.y * f);
          }
      }
      e = max(e, e0);
    }
    __syncwarp();
    if (lane == 0) *scale = q8_pow2(e);
    const float inv = q8_pow2(-e);
    for (int s = s0; s < s1; ++s) {
      turned_row(a, in, src + s * in.ss, !is_v, (long long)start + s, n, y,
                 lane);
      uint8_t *row = dst + (off + (start + s - g0)) * st;
      for (int d = lane * 2; d < a.D; d += 64)
        *reinterpret_cast<uint16_t *>(row + d) =
            (uint16_t)q8_pack2(y[d] * inv, y[d + 1] * inv);
      __syncwarp();
    }
  }
}

struct ReadQ8 {
  Q8Cache c;
  int T, B;
  const int32_t *first, *length;
  __nv_bfloat16 *k, *v;
  int *status;
};

// A thread takes 16 values of a row.
__global__ void __launch_bounds__(256) read_q8_kernel(const ReadQ8 p) {
  const int ch = p.c.D / 16;
  const long long per = (long long)p.T * p.B * p.c.Hk * ch;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
       i < 2 * per; i += (long long)gridDim.x * blockDim.x) {
    const bool is_v = i >= per;
    __nv_bfloat16 *out = is_v ? p.v : p.k;
    if (!out) continue;
    const long long at = is_v ? i - per : i;
    const int c = (int)(at % ch);
    const int h = (int)(at / ch % p.c.Hk);
    const long long row = at / ch / p.c.Hk;
    const int b = (int)(row % p.B), t = (int)(row / p.B);
    uint32_t w[8] = {};
    const int n = p.length ? __ldg(p.length + b) : p.T;
    if (t < n) {
      const long long j = (p.first ? (long long)__ldg(p.first + b) : 0) + t;
      bool bad = false;
      const int page = q8_page(p.c, b, j, bad);
      if (bad) {
        atomicOr(p.status, kStatusIndexRange);
      } else {
        const int off = (int)(j % p.c.page_size);
        const uint8_t *src =
            is_v ? p.c.v + page * p.c.v_p + off * p.c.v_t + h * p.c.v_h
                 : p.c.k + page * p.c.k_p + off * p.c.k_t + h * p.c.k_h;
        const float s = q8_pow2(
            q8_exp(__ldg((is_v ? p.c.vs : p.c.ks) +
                         q8_scale_at(p.c, page, off, h))));
        const uint4 x = __ldg(reinterpret_cast<const uint4 *>(src) + c);
        const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 lo = q8_float2(u[k] & 0xffffu);
          const float2 hi = q8_float2(u[k] >> 16);
          w[2 * k] = pack_bf16x2(lo.x * s, lo.y * s);
          w[2 * k + 1] = pack_bf16x2(hi.x * s, hi.y * s);
        }
      }
    }
    uint4 *to = reinterpret_cast<uint4 *>(out + at * 16);
    to[0] = make_uint4(w[0], w[1], w[2], w[3]);
    to[1] = make_uint4(w[4], w[5], w[6], w[7]);
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
  const long long items =
      (long long)S * B * a.q.heads + 2ll * p.groups * B * Hk;
  const long long grid = (items + 3) / 4;
  const long long most = 16ll * num_sms;
  dsa::append_q8_kernel<<<(unsigned)(grid < most ? grid : most), 128, 0,
                          static_cast<cudaStream_t>(cuda_stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
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
  const long long grid = ((long long)T * B * Hk * (D / 16) * 2 + 255) / 256;
  const long long most = 8ll * num_sms;
  dsa::read_q8_kernel<<<(unsigned)(grid < most ? grid : most), 256, 0,
                        static_cast<cudaStream_t>(cuda_stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // extern "C"
