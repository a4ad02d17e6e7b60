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
// angle modulo one turn, so far positions lose little: the host's 64-bit floats are off by 2^-53 of the whole
// angle, 2^-30 rad at position 2^23 and 2^-22 at 2^31 (a float product by 2^-24: 0.008 rad at position 131072).
#include <algorithm>
#include <cfloat>

#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace df {

namespace {

// Sine and cosine of pos * turn 2^-64 turns: the nearest quarter turn comes off in fixed point, exactly, and
// Taylor's polynomials give the rest of at most pi/4 (left out: x^11/11! < 2^-28 and x^12/12! < 2^-33). The
// angle is the sum x + xl, and each polynomial adds its first term last, so both results are little
// more than their last rounding off. In the 8-bit caches a value rounded the other way is off by a whole
// step: the fast sine's 2^-21 showed there.
__device__ __forceinline__ void turn_sincos(long long pos, unsigned long long turn, float *sn, float *cs) {
  constexpr double kStep = 1.4629180792671596e-9;  // 2 pi / 2^32
  constexpr float kHi = static_cast<float>(kStep), kLo = static_cast<float>(kStep - kHi);
  const uint32_t t = static_cast<uint32_t>((static_cast<unsigned long long>(pos) * turn + 0x80000000u) >> 32);
  const uint32_t quarter = (t + 0x20000000u) >> 30;
  const int rest = static_cast<int>(t - (quarter << 30));  // 2^-32 turns
  const float f = static_cast<float>(rest);
  const float x = f * kHi;
  const float xl = fmaf(f, kHi, -x) + fmaf(f, kLo, static_cast<float>(rest - static_cast<int>(f)) * kHi);
  const float y = x * x;
  const float ps = fmaf(y, fmaf(y, fmaf(y, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6);
  const float pc =
      fmaf(y, fmaf(y, fmaf(y, fmaf(y, -1.f / 3628800, 1.f / 40320), -1.f / 720), 1.f / 24), -0.5f);
  const float s = x + fmaf(xl, fmaf(-0.5f, y, 1.f), x * y * ps);
  const float c = 1.f + fmaf(-xl, x, y * pc);
  const bool odd = quarter & 1;
  const uint32_t us = __float_as_uint(odd ? c : s), uc = __float_as_uint(odd ? s : c);
  *sn = __uint_as_float(us ^ ((quarter & 2) << 30));
  *cs = __uint_as_float(uc ^ (((quarter + 1) & 2) << 30));
}

// Two bf16 values as floats.
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// W consecutive 32-bit words, CW (1, 2 or 4) loaded at once.
template <int W, int CW>
__device__ __forceinline__ void load_runs(const void *from, uint32_t (&w)[W]) {
#pragma unroll
  for (int q = 0; q < W; q += CW) {
    const uint32_t *at = static_cast<const uint32_t *>(from) + q;
    if constexpr (CW == 1) {
      w[q] = *at;
    } else if constexpr (CW == 2) {
      const uint2 u = *reinterpret_cast<const uint2 *>(at);
      w[q] = u.x, w[q + 1] = u.y;
    } else {
      const uint4 u = *reinterpret_cast<const uint4 *>(at);
      w[q] = u.x, w[q + 1] = u.y, w[q + 2] = u.z, w[q + 3] = u.w;
    }
  }
}

// Two floats to two e4m3 bytes.
__device__ __forceinline__ uint32_t e4m3x2(float2 v) {
  return __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
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

// A CTA has four warps: `cta_rows` (1, 2 or 4) rows with 4 / cta_rows warps each, and a warp `iters` groups
// of heads (32 / TPH heads each). A head is TPH = hd/16 threads, each with 8 values of the lower half and
// the 8 they rotate with. The CTA computes its rows' angles once; gains and angles meet in four
// factors per pair of values, the same for every head of a tensor, so that a value costs two
// products of packed floats and the row's 1 / norm. APPEND writes the first tensor's rows (keys) and the
// second's (values) into the caches.
// Memory bounds it: 8191 rows of 40 heads take 29.7 us, 168 MB at 5.7 TB/s, and 2 x 8189 rows appended to
// 8 + 8 heads 24.1 us, 134 MB at 5.6 TB/s, both with the same buffers again and again, of which the L2 keeps
// a part; with others each time 31.1 and 26.2. Groups go in batches of four, all loads before the first
// store: two at a time took 32.5 us, and each group's loads right after its predecessor's stores 35.8.
// Registers for five CTAs a SM (the append spills 12 bytes there); six spill more (41.7 us). Single tokens are a
// launch and four dependent loads: 2.4 us.
constexpr int kRowBatch = 4;  // groups whose loads are in flight together

template <int HD, bool APPEND>
__global__ void __launch_bounds__(128, 5) kv_rows_kernel(const __grid_constant__ KvRowsParams p) {
  constexpr int TPH = HD / 16;
  constexpr int HPW = 32 / TPH;
  __shared__ __align__(16) float angles[4][2][HD / 2];  // of the CTA's rows: cosines, sines
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per_row = 4 / p.cta_rows;  // warps
  const uint32_t rows = static_cast<uint32_t>(p.nb) * p.R;
  const uint32_t row0 = blockIdx.x * p.cta_rows;
  const uint32_t row = row0 + warp / per_row;
  const int part = blockIdx.y * per_row + warp % per_row;
  const int total = p.heads[0] + p.heads[1];
  const int d0 = (lane % TPH) * 8;
  const int h0 = part * p.iters * HPW + lane / TPH;
  bool live = row < rows && part * p.iters * HPW < total;
  const int i = live ? row / p.R : 0;
  const int j = row - i * p.R;
  long long crow = 0, chead = 0;  // APPEND: cache row of head 0, and the rows from one head to the next
  if (APPEND && live) {
    const long long pos = static_cast<long long>(p.ctx_len[i]) + j;
    if (j == 0 && part == 0 && lane == 0) report_lengths(p, i);
    live = j < new_rows(p.n_rows, i, p.R) && pos >= 0 && pos < p.Cmax;
    if (live && p.page_table) {
      const int pg = p.page_table[static_cast<long long>(i) * p.pages_per_seq + pos / kPageRows];
      crow = static_cast<long long>(pg) * p.heads[0] * kPageRows + pos % kPageRows;
      chead = kPageRows;
      if (pg < 0 || pg >= p.num_pages) {
        if (lane == 0) flag_status(p.status, kStatusCheck);
        live = false;
      }
    } else {
      crow = static_cast<long long>(i) * p.heads[0] * p.Cmax + pos;
      chead = p.Cmax;
    }
  }
  uint4 ua[kRowBatch], ub[kRowBatch];
  auto load = [&](int it0) {
#pragma unroll
    for (int k = 0; k < kRowBatch; ++k) {
      const int hh = h0 + (it0 + k) * HPW;
      ua[k] = ub[k] = make_uint4(0, 0, 0, 0);
      if (live && it0 + k < p.iters && hh < total) {
        const int t = hh >= p.heads[0] ? 1 : 0;
        const uint16_t *src = p.src[t] + row * p.ld[t] + static_cast<long long>(t ? hh - p.heads[0] : hh) * HD + d0;
        ua[k] = *reinterpret_cast<const uint4 *>(src);
        ub[k] = *reinterpret_cast<const uint4 *>(src + HD / 2);
      }
    }
  };
  load(0);
  for (int e = threadIdx.x; e < p.cta_rows * (HD / 2); e += 128) {
    const uint32_t r = row0 + e / (HD / 2);
    const int d = e % (HD / 2);
    float sn = 0.f, cs = 1.f;
    if (p.rotate && r < rows) {
      const uint32_t s = r / p.R;
      turn_sincos(static_cast<long long>(p.ctx_len[s]) + (r - s * p.R), p.turn[d], &sn, &cs);
    }
    angles[e / (HD / 2)][0][d] = cs;
    angles[e / (HD / 2)][1][d] = sn;
  }
  __syncthreads();
  if (!live) return;
  int cur = -1;                            // tensor whose factors the lane holds
  float2 fa[4], fb[4], fc[4], fd[4];       // a' = a fa + b fb,  b' = b fc + a fd
#pragma unroll 1
  for (int it0 = 0; it0 < p.iters; it0 += kRowBatch) {
    if (it0 > 0) load(it0);
#pragma unroll
    for (int k = 0; k < kRowBatch; ++k) {
      const int hh = h0 + (it0 + k) * HPW;
      const bool have = it0 + k < p.iters && hh < total;
      const int t = have && hh >= p.heads[0] ? 1 : 0;
      // values go as they are, and so do keys that are rotated and normed already
      const bool plain = !have || (APPEND && (t == 1 || !(p.rotate || p.g[0])));
      if (__any_sync(0xffffffffu, !plain)) {
        if (!plain && t != cur) {
          cur = t;
          const float *at = angles[warp / per_row][0] + d0;
          uint32_t ga[4] = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u}, gb[4];  // ones
          if (p.g[t]) load_runs<4, 4>(p.g[t] + d0, ga);
#pragma unroll
          for (int e = 0; e < 4; ++e) gb[e] = ga[e];
          if (p.g[t]) load_runs<4, 4>(p.g[t] + d0 + HD / 2, gb);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 cs = reinterpret_cast<const float2 *>(at)[e];
            const float2 sn = reinterpret_cast<const float2 *>(at + HD / 2)[e];
            const float2 a = unpack2(ga[e]), b = unpack2(gb[e]);
            fa[e] = mul2(a, cs);
            fb[e] = mul2(b, make_float2(-sn.x, -sn.y));
            fc[e] = mul2(b, cs);
            fd[e] = mul2(a, sn);
          }
        }
        const uint32_t wa[4] = {ua[k].x, ua[k].y, ua[k].z, ua[k].w}, wb[4] = {ub[k].x, ub[k].y, ub[k].z, ub[k].w};
        float2 a[4], b[4], ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          a[e] = unpack2(wa[e]);
          b[e] = unpack2(wb[e]);
          ss = fma2(a[e], a[e], fma2(b[e], b[e], ss));
        }
        float inv = 1.f;
        if (p.g[0] || p.g[1]) {
          float sum = ss.x + ss.y;
#pragma unroll
          for (int o = TPH / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          if (p.g[t]) inv = rsqrtf(sum * (1.f / HD) + p.eps);
        }
        if (!plain) {
          const float2 inv2 = make_float2(inv, inv);
          uint32_t ra[4], rb[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 x = mul2(a[e], inv2), y = mul2(b[e], inv2);
            float2 u = mul2(x, fa[e]), v = mul2(y, fc[e]);
            if (!APPEND || p.rotate) {  // else no product with a sine of zero: infinities would make NaN of it
              u = fma2(y, fb[e], u);
              v = fma2(x, fd[e], v);
            }
            ra[e] = pack_bf16x2(u.x, u.y);
            rb[e] = pack_bf16x2(v.x, v.y);
          }
          ua[k] = make_uint4(ra[0], ra[1], ra[2], ra[3]);
          ub[k] = make_uint4(rb[0], rb[1], rb[2], rb[3]);
        }
      }
      if (have) {
        const int head = t ? hh - p.heads[0] : hh;
        uint16_t *dst = APPEND ? p.dst[t] + (crow + head * chead) * HD + d0
                               : p.dst[t] + (static_cast<long long>(row) * p.heads[t] + head) * HD + d0;
        *reinterpret_cast<uint4 *>(dst) = ua[k];
        *reinterpret_cast<uint4 *>(dst + HD / 2) = ub[k];
      }
    }
  }
}

// Append in 8 bits: SLOTS * TPR threads per (64-row block of a sequence, keys or values), which go through
// `iters` kv heads; TPR threads per new row, each with HD / 2 / TPR values of either half, whose angles and
// gains serve every head. The block's scale is the power of two that takes its largest new value to at
// most 448 (e4m3's largest), and not less than the scale of the rows that stay; those are rounded
// again only when the scale grows. A power of two loses nothing against amax / 448: e4m3 is a
// floating format, and rescaling rows by a power of two is exact but for values that become
// subnormal. It also joins 1 / norm exactly, so a value costs one product for both.
// The values before their rounding to e4m3 are fp32's, off by 5e-8 on average, so one key in 1.6 million
// lies so near the middle of a step that it goes to the other side than in exact arithmetic (with the
// norm, the gain and the rotation each rounded on its own, one in 1.1 million).
// Two prompts of up to 8189 rows (67 MB) take 17.4 us, 3.9 TB/s, and 13.8 where they lie in the L2 from the call
// before: a step from head to head is a chain of norm, maximum over the block and scale, which the four warps
// a scheduler has room for hide in part. From the L2 it was 15.6 with the angles in registers, which leaves room for
// no more warps, and 15 to 16.7 with the heads' values asked for two to four steps ahead through shared memory.
constexpr int kScaleExpMin = -100, kScaleExpMax = 119;

template <int HD, int SLOTS, int TPR>
__global__ void __launch_bounds__(SLOTS *TPR < 128 ? 128 : SLOTS * TPR, SLOTS * TPR > 128 ? 2 : 4)
    kv_append8_kernel(const __grid_constant__ KvRowsParams p) {
  constexpr int GT = SLOTS * TPR;           // threads that share a block: a warp, or the CTA
  constexpr int GROUPS = GT < 128 ? 128 / GT : 1;
  constexpr int E = HD / 2 / TPR, W = E / 2;  // values of one half per thread, and words
  constexpr int CW = W < 4 ? W : 4;           // words loaded at once
  static_assert(GT == 32 || GT >= 128, "a warp or a CTA");
  griddep_wait();
  griddep_launch();
  __shared__ float red[2][GT / 32];
  const int i = blockIdx.y;
  const int tid = threadIdx.x % GT;
  // keys first: their groups have the most to do
  const int group = blockIdx.z * GROUPS + threadIdx.x / GT, keys = (p.heads[0] + p.iters - 1) / p.iters;
  const int t = group >= keys ? 1 : 0, per = t ? p.iters_v : p.iters;
  const int h0 = (group - t * keys) * per, h1 = min(h0 + per, p.heads[0]);
  if (blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0) report_lengths(p, i);
  const int n = new_rows(p.n_rows, i, p.R);
  const int c0 = p.ctx_len[i];
  if (c0 < 0 || n == 0 || h0 >= h1) return;
  const int hi = static_cast<int>(min(static_cast<long long>(c0) + n, static_cast<long long>(p.Cmax)));
  const int blk = c0 / kPageRows + blockIdx.x;
  if (blk > (hi - 1) / kPageRows) return;  // in blocks: a length near 2^31 times 64 would not fit
  const int row0 = blk * kPageRows;
  long long block, bhead;  // (block, head 0) in the cache, in blocks of 64 rows, and the step to the next head
  if (p.page_table) {
    const int pg = p.page_table[static_cast<long long>(i) * p.pages_per_seq + blk];
    if (pg < 0 || pg >= p.num_pages) {
      if (tid == 0) flag_status(p.status, kStatusCheck);
      return;
    }
    block = static_cast<long long>(pg) * p.heads[0];
    bhead = 1;
  } else {
    bhead = p.Cmax / kPageRows;
    block = static_cast<long long>(i) * p.heads[0] * bhead + blk;
  }
  const int part = tid % TPR, slot = tid / TPR;
  const int kept = max(c0 - row0, 0);       // rows of earlier calls in this block
  const int pos = row0 + kept + slot;
  const bool fresh = pos < min(hi, row0 + kPageRows);
  const int d0 = part * E;
  const uint16_t *src = p.src[t] + (static_cast<long long>(i) * p.R + (pos - c0)) * p.ld[t] + d0;
  const int lane = threadIdx.x & 31;
  float scales = 0.f;                       // lane l: scale of head h0 + l's kept rows
  if (kept > 0 && h0 + lane < h1) scales = p.scale[t][block + (h0 + lane) * bhead];
  uint32_t na[W], nb[W];                    // the next head's values
  auto load = [&](int head) {
#pragma unroll
    for (int e = 0; e < W; ++e) na[e] = nb[e] = 0u;
    if (fresh && head < h1) {
      load_runs<W, CW>(src + static_cast<long long>(head) * HD, na);
      load_runs<W, CW>(src + static_cast<long long>(head) * HD + HD / 2, nb);
    }
  };
  load(h0);
  const bool norm = t == 0 && p.g[0], rotate = t == 0 && p.rotate;
  constexpr bool TAB = GT > 128;            // a thread's own angles in shared memory, to spare it the registers
  __shared__ float4 tab[TAB ? W : 1][TAB ? GT : 1];
  float2 cs[W], sn[W];
  uint32_t ga[W], gb[W];
  if (rotate) {
#pragma unroll
    for (int e = 0; e < W; ++e) {
      turn_sincos(pos, p.turn[d0 + 2 * e], &sn[e].x, &cs[e].x);
      turn_sincos(pos, p.turn[d0 + 2 * e + 1], &sn[e].y, &cs[e].y);
      if constexpr (TAB) tab[e][tid] = make_float4(cs[e].x, cs[e].y, sn[e].x, sn[e].y);
    }
  }
  if (norm) {
    load_runs<W, CW>(p.g[0] + d0, ga);
    load_runs<W, CW>(p.g[0] + d0 + HD / 2, gb);
  }
#pragma unroll 1
  for (int head = h0; head < h1; ++head) {
    float2 a[W], b[W];
#pragma unroll
    for (int e = 0; e < W; ++e) {
      a[e] = unpack2(na[e]);
      b[e] = unpack2(nb[e]);
    }
    const float s_old = __shfl_sync(0xffffffffu, scales, head - h0);
    load(head + 1);
    float inv = 1.f;                        // of the row, joined to its values below
    if (norm) {
      float2 sa = make_float2(0.f, 0.f), sb = sa;
#pragma unroll
      for (int e = 0; e < W; ++e) {
        sa = fma2(a[e], a[e], sa);
        sb = fma2(b[e], b[e], sb);
      }
      float ss = (sa.x + sa.y) + (sb.x + sb.y);
#pragma unroll
      for (int o = 1; o < TPR; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      inv = __frsqrt_rn(ss * (1.f / HD) + p.eps);  // rsqrtf may be two steps off: e4m3 roundings would show it
#pragma unroll
      for (int e = 0; e < W; ++e) {
        a[e] = mul2(a[e], unpack2(ga[e]));
        b[e] = mul2(b[e], unpack2(gb[e]));
      }
    }
    if (rotate) {
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const float2 x = a[e], y = b[e];
        if constexpr (TAB) {
          const float4 f = tab[e][tid];
          cs[e] = make_float2(f.x, f.y);
          sn[e] = make_float2(f.z, f.w);
        }
        a[e] = fma2(y, make_float2(-sn[e].x, -sn[e].y), mul2(x, cs[e]));
        b[e] = fma2(x, sn[e], mul2(y, cs[e]));
      }
    }
    // largest finite new value of the block (slots without a row hold zeros); a NaN is no maximum
    float m = 0.f, mb = 0.f;
#pragma unroll
    for (int e = 0; e < W; ++e) {
      m = max3(m, fabsf(a[e].x), fabsf(a[e].y));
      mb = max3(mb, fabsf(b[e].x), fabsf(b[e].y));
    }
    m = fmaxf(m, mb);
    if (m > FLT_MAX) {
      m = 0.f;
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const float v[4] = {fabsf(a[e].x), fabsf(a[e].y), fabsf(b[e].x), fabsf(b[e].y)};
#pragma unroll
        for (int x = 0; x < 4; ++x) m = fmaxf(m, v[x] <= FLT_MAX ? v[x] : 0.f);
      }
    }
    m *= inv;                               // rounding keeps the order: the largest of the products
    m = m <= FLT_MAX ? m : 0.f;
    m = warp_max(m);
    if constexpr (GT > 32) {
      float *to = red[(head - h0) & 1];     // two, so that one barrier a head is enough
      if ((tid & 31) == 0) to[tid >> 5] = m;
      __syncthreads();
      m = warp_max(to[tid % (GT / 32)]);
    }
    // smallest e with m <= 448 * 2^e = 1.75 * 2^(e + 8)
    const uint32_t bits = __float_as_uint(m);
    int ex = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    ex = max(kScaleExpMin, min(ex, kScaleExpMax));
    const float s = fmaxf(__uint_as_float(static_cast<uint32_t>(ex + 127) << 23), s_old);
    const long long bi = block + head * bhead;
    uint8_t *dst = p.dst8[t] + bi * (kPageRows * HD) + d0;
    if (fresh) {
      // a scale that this call has not made need not be a power of two
      const uint32_t sb = __float_as_uint(s);
      const float f = inv * ((sb & 0x7FFFFFu) == 0 && sb < 0x7E800000u ? __uint_as_float(0x7F000000u - sb) : 1.f / s);
      const float2 f2 = make_float2(f, f);
      uint8_t *to = dst + (pos - row0) * HD;
      if constexpr (W == 1) {
        *reinterpret_cast<uint16_t *>(to) = static_cast<uint16_t>(e4m3x2(mul2(a[0], f2)));
        *reinterpret_cast<uint16_t *>(to + HD / 2) = static_cast<uint16_t>(e4m3x2(mul2(b[0], f2)));
      } else {
        uint32_t qa[W / 2], qb[W / 2];
#pragma unroll
        for (int q = 0; q < W / 2; ++q) {
          qa[q] = e4m3x2(mul2(a[2 * q], f2)) | (e4m3x2(mul2(a[2 * q + 1], f2)) << 16);
          qb[q] = e4m3x2(mul2(b[2 * q], f2)) | (e4m3x2(mul2(b[2 * q + 1], f2)) << 16);
        }
        if constexpr (W == 2) {
          *reinterpret_cast<uint32_t *>(to) = qa[0];
          *reinterpret_cast<uint32_t *>(to + HD / 2) = qb[0];
        } else if constexpr (W == 4) {
          *reinterpret_cast<uint2 *>(to) = make_uint2(qa[0], qa[1]);
          *reinterpret_cast<uint2 *>(to + HD / 2) = make_uint2(qb[0], qb[1]);
        } else {
          *reinterpret_cast<uint4 *>(to) = make_uint4(qa[0], qa[1], qa[2], qa[3]);
          *reinterpret_cast<uint4 *>(to + HD / 2) = make_uint4(qb[0], qb[1], qb[2], qb[3]);
        }
      }
    }
    if (kept > 0 && s > s_old) {
      const float ratio = s_old / s;
#pragma unroll 1
      for (int r = slot; r < kept; r += SLOTS)
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          uint16_t *at = reinterpret_cast<uint16_t *>(dst + r * HD + half * (HD / 2));
#pragma unroll
          for (int q = 0; q < W; ++q) {
            const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(at[q]), __NV_E4M3);
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&hr));
            at[q] = static_cast<uint16_t>(e4m3x2(make_float2(f.x * ratio, f.y * ratio)));
          }
        }
    }
    if (tid == 0 && !(kept > 0 && s == s_old)) p.scale[t][bi] = s;
  }
}

static cudaError_t launch_rows(KvRowsParams &p, bool append, int num_sms, cudaStream_t s) {
  const int hpw = 32 / (p.hd / 16);
  const int groups = (p.heads[0] + p.heads[1] + hpw - 1) / hpw;  // head groups of a row
  const long long rows = static_cast<long long>(p.nb) * p.R;
  // few rows: a warp for every head group (latency); many: the whole row in one warp, so that the factors
  // are computed once for it (8191 rows of 40 heads: 29.9 us; with two groups a warp 61). Between them about
  // 10 warps a SM and whole CTAs of warps, which all fit at once: 512 rows of 40 heads 4.3 us, at 16 a SM
  // and with idle warps 5.4; 1024 appended rows 4.7 and 6.4; at 6 a SM 4.7 and 4.7.
  const long long target = static_cast<long long>(num_sms) * 10;
  const int iters = static_cast<int>(std::min<long long>(groups, std::max<long long>(1, rows * groups / target)));
  const int parts = (groups + iters - 1) / iters;
  p.cta_rows = parts == 1 ? 4 : parts == 2 ? 2 : 1;
  const int per_row = 4 / p.cta_rows;
  const int y = iters == 1 ? (parts + per_row - 1) / per_row : std::max(1, parts / per_row);
  p.iters = (groups + y * per_row - 1) / (y * per_row);
  const dim3 grid(static_cast<unsigned>((rows + p.cta_rows - 1) / p.cta_rows), y);
  if (p.hd == 128)
    return append ? launch_pdl(kv_rows_kernel<128, true>, grid, dim3(128), 0, s, p)
                  : launch_pdl(kv_rows_kernel<128, false>, grid, dim3(128), 0, s, p);
  return append ? launch_pdl(kv_rows_kernel<64, true>, grid, dim3(128), 0, s, p)
                : launch_pdl(kv_rows_kernel<64, false>, grid, dim3(128), 0, s, p);
}

cudaError_t launch_qk_norm_rope(KvRowsParams &p, int num_sms, cudaStream_t s) {
  return launch_rows(p, false, num_sms, s);
}

cudaError_t launch_kv_append(KvRowsParams &p, int num_sms, cudaStream_t s) {
  return launch_rows(p, true, num_sms, s);
}

template <int HD, int SLOTS, int TPR>
static cudaError_t launch_slots(KvRowsParams &p, int num_sms, cudaStream_t s) {
  constexpr int GT = SLOTS * TPR;
  constexpr int GROUPS = GT < 128 ? 128 / GT : 1;
  const int blocks = (p.R + kPageRows - 2) / kPageRows + 1;  // of 64 rows that R rows can touch
  p.iters = 1;
  if (GT > 32) {  // heads one after the other while that leaves enough CTAs (64 x 8 rows: 4.7 us at 6 a SM, 5.2 at 3)
    p.iters = std::min(p.heads[0], 32);
    auto ctas = [&] { return static_cast<long long>(blocks) * p.nb * 2 * ((p.heads[0] + p.iters - 1) / p.iters); };
    while (p.iters > 1 && ctas() < (GT > 128 ? 3LL : 6LL) * num_sms) p.iters = (p.iters + 1) / 2;
  }
  // values have no angles to share: groups of half as many, which fill in behind the keys (two prompts of
  // 8189 rows: 14.2 us, with groups as large as the keys' 15.5, of a quarter 14.6)
  p.iters_v = (p.iters + 1) / 2;
  const int groups = (p.heads[0] + p.iters - 1) / p.iters + (p.heads[0] + p.iters_v - 1) / p.iters_v;
  return launch_pdl(kv_append8_kernel<HD, SLOTS, TPR>, dim3(blocks, p.nb, (groups + GROUPS - 1) / GROUPS),
                    dim3(GT < 128 ? 128 : GT), 0, s, p);
}

template <int HD>
static cudaError_t launch_append8(KvRowsParams &p, int num_sms, cudaStream_t s) {
  // As many row slots as R needs, of 2, 16 or 64: 64 sequences with one row each take 2.9 us with 2 slots, 4.5
  // with 16 and 8.0 with 64; with 8 rows each 4.7 with 16 slots, 7.7 with 64.
  return p.R <= 2    ? launch_slots<HD, 2, 16>(p, num_sms, s)
         : p.R <= 16 ? launch_slots<HD, 16, 8>(p, num_sms, s)
                     : launch_slots<HD, 64, 4>(p, num_sms, s);
}

cudaError_t launch_kv_append8(KvRowsParams &p, int num_sms, cudaStream_t s) {
  return p.hd == 128 ? launch_append8<128>(p, num_sms, s) : launch_append8<64>(p, num_sms, s);
}

}  // namespace df
