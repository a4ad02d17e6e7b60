// Row kernels between a projection and its attention: per-head RMSNorm of queries and keys
// with the position rotation in the same pass, and appends of keys and values to the caches
// (contiguous or paged) in bf16 or in 8 bits.
//
//   norm      x * g / sqrt(mean(x^2) + eps) over the hd values of one head, fp32
//   rotation  for d < hd/2 by the angle a = p * base^(-2d/hd) at position p:
//             y[d] = x[d] cos a - x[d+hd/2] sin a,  y[d+hd/2] = x[d+hd/2] cos a + x[d] sin a
//
// The angle is kept in turns as a 64-bit fixed-point fraction: the host gives
// base^(-2d/hd) / (2 pi) * 2^64, and the low 64 bits of its product with the position are the
// angle modulo one turn, so far positions lose nothing (a float product is off by 2^-24 of
// the whole angle: 0.008 rad at position 131072).
#include <algorithm>
#include <cfloat>

#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace df {

namespace {

__device__ __forceinline__ void turn_sincos(long long pos, unsigned long long turn, float *sn, float *cs) {
  // the upper 32 of the fraction's 64 bits, as a signed number of 2^-32 turns in [-1/2, 1/2)
  const int t = static_cast<int>((static_cast<unsigned long long>(pos) * turn) >> 32);
  __sincosf(static_cast<float>(t) * 1.4629180792671596e-9f, sn, cs);  // 2 pi / 2^32
}

__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(w[e] << 16);
    x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// New rows of sequence i (n_rows clipped to [0, R]; every row without n_rows).
__device__ __forceinline__ int new_rows(const int *n_rows, int i, int R) {
  return n_rows ? max(0, min(n_rows[i], R)) : R;
}

// Reported once per sequence: a row count outside [0, R], or rows outside [0, Cmax).
__device__ __forceinline__ void report_lengths(const KvRowsParams &p, int i) {
  const int n = p.n_rows ? p.n_rows[i] : p.R;
  const int c = p.ctx_len[i];
  if (n < 0 || n > p.R || c < 0 || static_cast<long long>(c) + max(n, 0) > p.Cmax)
    flag_status(p.status, kStatusCheck);
}

}  // namespace

// One warp takes one row and `iters` groups of heads (32 / TPH heads each); a head is TPH = hd/16
// threads, each with 8 values of the lower half and the 8 they rotate with. The angles of
// a lane are the same for every head of the row: they are computed once. APPEND writes the
// first tensor's rows (keys) and the second's (values) into the caches.
template <int HD, bool APPEND>
__global__ void __launch_bounds__(256) kv_rows_kernel(const __grid_constant__ KvRowsParams p) {
  constexpr int TPH = HD / 16;
  constexpr int HPW = 32 / TPH;
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31;
  const long long w = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const long long row = w / p.warps_per_row;
  const int part = static_cast<int>(w % p.warps_per_row);
  if (row >= static_cast<long long>(p.nb) * p.R) return;
  const int i = static_cast<int>(row / p.R);
  const int j = static_cast<int>(row % p.R);
  const long long pos = static_cast<long long>(p.ctx_len[i]) + j;
  long long crow = 0;  // APPEND: cache row of head 0, and the rows from one head to the next
  long long chead = 0;
  if (APPEND) {
    if (j == 0 && part == 0 && lane == 0) report_lengths(p, i);
    if (j >= new_rows(p.n_rows, i, p.R) || pos < 0 || pos >= p.Cmax) return;
    if (p.page_table) {
      const int pg = p.page_table[static_cast<long long>(i) * p.pages_per_seq + pos / kPageRows];
      if (pg < 0 || pg >= p.num_pages) {
        if (lane == 0) flag_status(p.status, kStatusCheck);
        return;
      }
      crow = static_cast<long long>(pg) * p.heads[0] * kPageRows + pos % kPageRows;
      chead = kPageRows;
    } else {
      crow = static_cast<long long>(i) * p.heads[0] * p.Cmax + pos;
      chead = p.Cmax;
    }
  }
  const int d0 = (lane % TPH) * 8;
  float sn[8], cs[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    sn[e] = 0.f;
    cs[e] = 1.f;
    if (p.rotate) turn_sincos(pos, p.turn[d0 + e], &sn[e], &cs[e]);
  }
  const int total = p.heads[0] + p.heads[1];
  const int h0 = part * p.iters * HPW + lane / TPH;
#pragma unroll 4
  for (int it = 0; it < p.iters; ++it) {
    const int hh = h0 + it * HPW;
    const bool live = hh < total;
    const int t = live && hh >= p.heads[0] ? 1 : 0;
    const int head = t ? hh - p.heads[0] : hh;
    const uint16_t *src = p.src[t] + row * p.ld[t] + static_cast<long long>(head) * HD + d0;
    uint4 ua = make_uint4(0, 0, 0, 0), ub = ua;
    if (live) {
      ua = *reinterpret_cast<const uint4 *>(src);
      ub = *reinterpret_cast<const uint4 *>(src + HD / 2);
    }
    const bool plain = APPEND && t == 1;  // values go as they are
    if (__any_sync(0xffffffffu, !plain)) {
      float a[8], b[8];
      unpack8(ua, a);
      unpack8(ub, b);
      if (p.g[0] || p.g[1]) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += a[e] * a[e] + b[e] * b[e];
#pragma unroll
        for (int o = TPH / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const uint16_t *g = p.g[t];
        if (g && !plain) {
          const float inv = rsqrtf(ss * (1.f / HD) + p.eps);
          float ga[8], gb[8];
          unpack8(__ldg(reinterpret_cast<const uint4 *>(g + d0)), ga);
          unpack8(__ldg(reinterpret_cast<const uint4 *>(g + d0 + HD / 2)), gb);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            a[e] *= inv * ga[e];
            b[e] *= inv * gb[e];
          }
        }
      }
      if (!plain) {
        float ra[8], rb[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ra[e] = a[e] * cs[e] - b[e] * sn[e];
          rb[e] = b[e] * cs[e] + a[e] * sn[e];
        }
        ua = pack8(ra);
        ub = pack8(rb);
      }
    }
    if (!live) continue;
    uint16_t *dst;
    if (APPEND)
      dst = p.dst[t] + (crow + head * chead) * HD + d0;
    else
      dst = p.dst[t] + (row * p.heads[t] + head) * HD + d0;
    *reinterpret_cast<uint4 *>(dst) = ua;
    *reinterpret_cast<uint4 *>(dst + HD / 2) = ub;
  }
}

// Append in 8 bits: one CTA per (64-row block of a sequence, kv head, keys or values), four
// threads per row, each with HD/8 values of either half. The block's scale is the power of two
// that takes its largest new value to at most 448 (e4m3's largest), and not less than the
// scale of the rows that stay; those are rounded again only when the scale grows. A power of
// two loses nothing against amax / 448: e4m3 is a floating format, and rescaling rows by a
// power of two is exact but for values that become subnormal.
constexpr int kScaleExpMin = -100, kScaleExpMax = 119;

template <int HD>
__global__ void __launch_bounds__(256) kv_append8_kernel(const __grid_constant__ KvRowsParams p) {
  constexpr int E = HD / 8;  // values of one half per thread
  griddep_wait();
  griddep_launch();
  __shared__ float red[8];
  const int i = blockIdx.z;
  const int head = blockIdx.y >> 1, t = blockIdx.y & 1;
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) report_lengths(p, i);
  const int n = new_rows(p.n_rows, i, p.R);
  const int c0 = p.ctx_len[i];
  if (c0 < 0 || n == 0) return;
  const int hi = static_cast<int>(min(static_cast<long long>(c0) + n, static_cast<long long>(p.Cmax)));
  const int blk = c0 / kPageRows + blockIdx.x;
  if (blk * kPageRows >= hi) return;
  long long block;  // index of this (block, head) in the cache, in blocks of 64 rows
  if (p.page_table) {
    const int pg = p.page_table[static_cast<long long>(i) * p.pages_per_seq + blk];
    if (pg < 0 || pg >= p.num_pages) {
      if (threadIdx.x == 0) flag_status(p.status, kStatusCheck);
      return;
    }
    block = static_cast<long long>(pg) * p.heads[0] + head;
  } else {
    block = (static_cast<long long>(i) * p.heads[0] + head) * (p.Cmax / kPageRows) + blk;
  }
  const int r = threadIdx.x >> 2, part = threadIdx.x & 3;
  const int pos = blk * kPageRows + r;
  const bool fresh = pos >= c0 && pos < hi;
  const bool keeps = blk * kPageRows < c0;  // rows of earlier calls lie in this block
  const int d0 = part * E;
  float *scale_at = p.scale[t] + block;
  const float s_old = keeps ? *scale_at : 0.f;
  float a[E], b[E];
#pragma unroll
  for (int e = 0; e < E; ++e) a[e] = b[e] = 0.f;
  if (fresh) {
    const long long row = static_cast<long long>(i) * p.R + (pos - c0);
    const uint16_t *src = p.src[t] + row * p.ld[t] + static_cast<long long>(head) * HD + d0;
#pragma unroll
    for (int q = 0; q < E / 8; ++q) {
      float x[8];
      unpack8(*reinterpret_cast<const uint4 *>(src + 8 * q), x);
#pragma unroll
      for (int e = 0; e < 8; ++e) a[8 * q + e] = x[e];
      unpack8(*reinterpret_cast<const uint4 *>(src + HD / 2 + 8 * q), x);
#pragma unroll
      for (int e = 0; e < 8; ++e) b[8 * q + e] = x[e];
    }
  }
  if (t == 0) {
    if (p.g[0]) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) ss += a[e] * a[e] + b[e] * b[e];
      ss += __shfl_xor_sync(0xffffffffu, ss, 1);
      ss += __shfl_xor_sync(0xffffffffu, ss, 2);
      const float inv = rsqrtf(ss * (1.f / HD) + p.eps);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        a[e] *= inv * __uint_as_float(static_cast<uint32_t>(p.g[0][d0 + e]) << 16);
        b[e] *= inv * __uint_as_float(static_cast<uint32_t>(p.g[0][d0 + HD / 2 + e]) << 16);
      }
    }
    if (p.rotate) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        float sn, cs;
        turn_sincos(pos, p.turn[d0 + e], &sn, &cs);
        const float x = a[e], y = b[e];
        a[e] = x * cs - y * sn;
        b[e] = y * cs + x * sn;
      }
    }
  }
  // largest finite new value of the block (rows that are not new hold zeros)
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float x = fabsf(a[e]), y = fabsf(b[e]);
    m = fmaxf(m, fmaxf(x <= FLT_MAX ? x : 0.f, y <= FLT_MAX ? y : 0.f));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  m = red[0];
#pragma unroll
  for (int q = 1; q < 8; ++q) m = fmaxf(m, red[q]);
  // smallest e with m <= 448 * 2^e = 1.75 * 2^(e + 8)
  const uint32_t mb = __float_as_uint(m);
  int ex = static_cast<int>(mb >> 23) - 127 - 8 + ((mb & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  ex = max(kScaleExpMin, min(ex, kScaleExpMax));
  const float s = fmaxf(__uint_as_float(static_cast<uint32_t>(ex + 127) << 23), s_old);
  uint8_t *dst = p.dst8[t] + block * (kPageRows * HD) + r * HD + d0;
  if (fresh) {
    const float inv = 1.f / s;
    uint32_t qa[E / 4], qb[E / 4];
#pragma unroll
    for (int q = 0; q < E / 4; ++q) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a[4 * q] * inv, a[4 * q + 1] * inv),
                                                   __NV_SATFINITE, __NV_E4M3);
      const uint32_t up = __nv_cvt_float2_to_fp8x2(make_float2(a[4 * q + 2] * inv, a[4 * q + 3] * inv),
                                                   __NV_SATFINITE, __NV_E4M3);
      qa[q] = lo | (up << 16);
      const uint32_t lo2 = __nv_cvt_float2_to_fp8x2(make_float2(b[4 * q] * inv, b[4 * q + 1] * inv),
                                                    __NV_SATFINITE, __NV_E4M3);
      const uint32_t up2 = __nv_cvt_float2_to_fp8x2(make_float2(b[4 * q + 2] * inv, b[4 * q + 3] * inv),
                                                    __NV_SATFINITE, __NV_E4M3);
      qb[q] = lo2 | (up2 << 16);
    }
    if constexpr (E == 16) {
      *reinterpret_cast<uint4 *>(dst) = make_uint4(qa[0], qa[1], qa[2], qa[3]);
      *reinterpret_cast<uint4 *>(dst + HD / 2) = make_uint4(qb[0], qb[1], qb[2], qb[3]);
    } else {
      *reinterpret_cast<uint2 *>(dst) = make_uint2(qa[0], qa[1]);
      *reinterpret_cast<uint2 *>(dst + HD / 2) = make_uint2(qb[0], qb[1]);
    }
  } else if (keeps && pos < c0 && s > s_old) {
    const float ratio = s_old / s;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t *at = reinterpret_cast<uint32_t *>(dst + half * (HD / 2));
#pragma unroll
      for (int q = 0; q < E / 4; ++q) {
        const uint32_t v = at[q];
        uint32_t out = 0;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
              static_cast<__nv_fp8x2_storage_t>((v >> (16 * x)) & 0xFFFFu), __NV_E4M3);
          const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&hr));
          out |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(f.x * ratio, f.y * ratio),
                                                                __NV_SATFINITE, __NV_E4M3))
                 << (16 * x);
        }
        at[q] = out;
      }
    }
  }
  if (threadIdx.x == 0 && !(keeps && s == s_old)) *scale_at = s;
}

static cudaError_t launch_rows(KvRowsParams &p, bool append, int num_sms, cudaStream_t s) {
  const int hpw = 32 / (p.hd / 16);
  const int groups = (p.heads[0] + p.heads[1] + hpw - 1) / hpw;  // head groups of a row
  const long long rows = static_cast<long long>(p.nb) * p.R;
  // few rows: a warp for every head group (latency); many: up to 8 groups per warp, so the
  // angles are computed once for them and their loads are in flight together
  const long long target = static_cast<long long>(num_sms) * 32;
  int iters = static_cast<int>(std::min<long long>(std::min(groups, 8), std::max<long long>(1, rows * groups / target)));
  p.warps_per_row = (groups + iters - 1) / iters;
  p.iters = (groups + p.warps_per_row - 1) / p.warps_per_row;
  const long long ctas = (rows * p.warps_per_row + 7) / 8;
  if (ctas > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(ctas));
  if (p.hd == 128)
    return append ? launch_pdl(kv_rows_kernel<128, true>, grid, dim3(256), 0, s, p)
                  : launch_pdl(kv_rows_kernel<128, false>, grid, dim3(256), 0, s, p);
  return append ? launch_pdl(kv_rows_kernel<64, true>, grid, dim3(256), 0, s, p)
                : launch_pdl(kv_rows_kernel<64, false>, grid, dim3(256), 0, s, p);
}

cudaError_t launch_qk_norm_rope(KvRowsParams &p, int num_sms, cudaStream_t s) {
  return launch_rows(p, false, num_sms, s);
}

cudaError_t launch_kv_append(KvRowsParams &p, int num_sms, cudaStream_t s) {
  return launch_rows(p, true, num_sms, s);
}

cudaError_t launch_kv_append8(const KvRowsParams &p, cudaStream_t s) {
  // blocks of 64 rows that R rows can touch
  const dim3 grid((p.R + 62) / kPageRows + 1, 2 * p.heads[0], p.nb);
  return p.hd == 128 ? launch_pdl(kv_append8_kernel<128>, grid, dim3(256), 0, s, p)
                     : launch_pdl(kv_append8_kernel<64>, grid, dim3(256), 0, s, p);
}

}  // namespace df
