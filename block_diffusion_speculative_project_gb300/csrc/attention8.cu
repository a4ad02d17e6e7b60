// Attention of m query rows per sequence over a cache held in 8 bits: e4m3 keys and values with
// one scale for each block of 64 rows and kv head.
//   o = softmax(q K^T / sqrt(hd)) V over the rows [0, ctx + n) of the sequence's kv head, with
//   `causal` only over [0, ctx + j + 1) for the query of row j; rows j >= n are not computed.
//
// A block of 64 rows is the unit of work: its scale is one number, so K's goes into the scores'
// factor and V's into the probabilities. The units of all (sequence, kv head) pairs, in that
// order, are cut into `grid` contiguous ranges of equal size, one per CTA; a CTA's run of units
// of one pair is a segment. A segment that covers its pair writes the output, any other an
// unnormalised partial (o, running maximum, running sum) to slot pair + cta, which the merge
// kernel joins in CTA order.
#include <cfloat>
#include <cmath>

#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace df {

namespace {

constexpr int kUnit = kPageRows;   // keys per unit: rows that share a scale, rows of a page
constexpr float kNoMax = -1e30f;   // running maximum (log2 units) before the first key

// Rows of sequence i that the call computes, its context rows (clamped to the caller's bound
// and the cache) and its units.
struct Seq8 {
  int n, ctx, units;
};
__device__ __forceinline__ Seq8 seq8(const Attn8Params &p, int i) {
  Seq8 s;
  s.n = p.n_rows ? max(0, min(p.n_rows[i], p.m)) : p.m;
  s.ctx = max(0, min(p.ctx_len[i], min(p.max_ctx, p.Cmax - s.n)));
  s.units = s.n > 0 ? (s.ctx + s.n + kUnit - 1) / kUnit : 0;
  return s;
}

// Unit u of the pair (sequence i, kv head g) as a block index of the cache.
__device__ __forceinline__ long long block_of(const Attn8Params &p, int i, int g, int u) {
  if (p.page_table == nullptr) return (static_cast<long long>(i) * p.Hkv + g) * (p.Cmax / kUnit) + u;
  int pg = p.page_table[static_cast<long long>(i) * p.pages_per_seq + u];
  if (pg < 0 || pg >= p.num_pages) {
    flag_status(p.status, kStatusCheck);
    pg = 0;
  }
  return static_cast<long long>(pg) * p.Hkv + g;
}

__device__ __forceinline__ long long cta_start(long long T, int G, int c) {
  return static_cast<long long>(c) * T / G;
}
__device__ __forceinline__ int cta_of(long long T, int G, long long u) {
  return static_cast<int>(((u + 1) * G + T - 1) / T - 1);
}

// Where a CTA's range begins: pair i * Hkv + g, unit inside it, number of units.
struct Range8 {
  int pair, unit;
  long long count;
};
// Warp-collective.
__device__ Range8 find_range(const Attn8Params &p, int cta, int lane) {
  long long T = 0;
  for (int i = lane; i < p.nb; i += 32) T += seq8(p, i).units;
#pragma unroll
  for (int o = 16; o; o >>= 1) T += __shfl_xor_sync(0xffffffffu, T, o);
  T *= p.Hkv;
  const int Ge = T < p.grid ? static_cast<int>(T) : p.grid;
  Range8 r = {0, 0, 0};
  if (cta >= Ge) return r;
  const long long u0 = cta_start(T, Ge, cta);
  r.count = cta_start(T, Ge, cta + 1) - u0;
  long long base = 0;
  for (int b = 0; b < p.nb; b += 32) {
    const int i = b + lane;
    const int U = i < p.nb ? seq8(p, i).units : 0;
    long long v = static_cast<long long>(p.Hkv) * U;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, base + v > u0);
    if (hit) {
      const int l = __ffs(hit) - 1;
      const int Ul = __shfl_sync(0xffffffffu, U, l);
      const long long off = u0 - (base + __shfl_sync(0xffffffffu, v, l) - static_cast<long long>(p.Hkv) * Ul);
      r.pair = (b + l) * p.Hkv + static_cast<int>(off / Ul);
      r.unit = static_cast<int>(off % Ul);
      return r;
    }
    base += __shfl_sync(0xffffffffu, v, 31);
  }
  r.count = 0;
  return r;
}

}  // namespace

constexpr int kA8Threads = 256;

__device__ __forceinline__ float e4m3_to_f32(uint8_t b) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(b, __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half *>(&h));
}

template <int HD>
__global__ void __launch_bounds__(kA8Threads) attn8_kernel(const __grid_constant__ Attn8Params p) {
  extern __shared__ float sm[];
  griddep_wait();
  griddep_launch();
  const int G = p.Hq / p.Hkv, R = G * p.m;
  float *sQ = sm;                         // [R][HD]
  float *sK = sQ + R * HD;                // [64][HD + 1]
  float *sV = sK + kUnit * (HD + 1);      // [64][HD]
  float *sP = sV + kUnit * HD;            // [R][64]
  float *sM = sP + R * kUnit;             // [R] maximum, [R] sum, [R] rescale
  __shared__ Range8 range;
  const int t = threadIdx.x;
  if (t < 32) {
    const Range8 r = find_range(p, blockIdx.x, t);
    if (t == 0) range = r;
    if (blockIdx.x == 0)
      for (int i = t; i < p.nb; i += 32) {
        const int n = p.n_rows ? p.n_rows[i] : p.m, c = p.ctx_len[i];
        if (n < 0 || n > p.m || c < 0 || c > p.max_ctx || static_cast<long long>(c) + max(n, 0) > p.Cmax)
          flag_status(p.status, kStatusCheck);
      }
  }
  __syncthreads();
  long long left = range.count;
  int pair = range.pair, unit = range.unit;
  const float sl2 = rsqrtf(static_cast<float>(HD)) * 1.4426950408889634f;
  constexpr int CPT = 16;                 // output columns per thread of a row
  constexpr int TPR = HD / CPT;
  while (left > 0) {
    const int i = pair / p.Hkv, g = pair % p.Hkv;
    const Seq8 s = seq8(p, i);
    if (s.units == 0) {
      ++pair;
      continue;
    }
    const int unit0 = unit;
    const int last = static_cast<int>(min(static_cast<long long>(s.units), unit + left));
    for (int e = t; e < R * HD; e += kA8Threads) {
      const int r = e / HD, d = e % HD, j = r / G, h = g * G + r % G;
      sQ[e] = __uint_as_float(static_cast<uint32_t>(p.q[((static_cast<size_t>(i) * p.m + j) * p.Hq + h) * HD + d]) << 16);
    }
    for (int r = t; r < R; r += kA8Threads) {
      sM[r] = kNoMax;
      sM[R + r] = 0.f;
    }
    float acc[4][CPT];
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int c = 0; c < CPT; ++c) acc[a][c] = 0.f;
    for (; unit < last; ++unit, --left) {
      const long long blk = block_of(p, i, g, unit);
      const float sk = p.ks[blk], sv = p.vs[blk];
      const int keys = s.ctx + s.n - unit * kUnit;
      __syncthreads();
      for (int e = t; e < kUnit * HD; e += kA8Threads) {
        const int k = e / HD, d = e % HD;
        sK[k * (HD + 1) + d] = k < keys ? e4m3_to_f32(p.k8[blk * (kUnit * HD) + e]) * sk : 0.f;
        sV[e] = k < keys ? e4m3_to_f32(p.v8[blk * (kUnit * HD) + e]) * sv : 0.f;
      }
      __syncthreads();
      for (int e = t; e < R * kUnit; e += kA8Threads) {
        const int r = e / kUnit, k = e % kUnit;
        float x = 0.f;
        for (int d = 0; d < HD; ++d) x = fmaf(sQ[r * HD + d], sK[k * (HD + 1) + d], x);
        const int lim = p.causal ? s.ctx + r / G + 1 : s.ctx + s.n;
        sP[e] = unit * kUnit + k < lim ? x * sl2 : -INFINITY;
      }
      __syncthreads();
      for (int r = t >> 5; r < R; r += kA8Threads / 32) {
        const int l = t & 31;
        const float x0 = sP[r * kUnit + l], x1 = sP[r * kUnit + l + 32];
        float mx = fmaxf(x0, x1);
        for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float m0 = sM[r], m1 = fmaxf(m0, mx);
        const float e0 = exp2f(x0 - m1), e1 = exp2f(x1 - m1);
        float sum = e0 + e1;
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        sP[r * kUnit + l] = e0;
        sP[r * kUnit + l + 32] = e1;
        __syncwarp();
        if (l == 0) {
          const float al = exp2f(m0 - m1);
          sM[r] = m1;
          sM[R + r] = sM[R + r] * al + sum;
          sM[2 * R + r] = al;
        }
      }
      __syncthreads();
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const int slot = t + a * kA8Threads;
        const int r = slot / TPR, d0 = (slot % TPR) * CPT;
        if (r >= R) continue;
        const float al = sM[2 * R + r];
#pragma unroll
        for (int c = 0; c < CPT; ++c) acc[a][c] *= al;
        for (int k = 0; k < kUnit; ++k) {
          const float w = sP[r * kUnit + k];
#pragma unroll
          for (int c = 0; c < CPT; ++c) acc[a][c] = fmaf(w, sV[k * HD + d0 + c], acc[a][c]);
        }
      }
    }
    const bool whole = unit0 == 0 && unit == s.units;
    const long long slot0 = static_cast<long long>(pair) + blockIdx.x;
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int slot = t + a * kA8Threads;
      const int r = slot / TPR, d0 = (slot % TPR) * CPT;
      if (r >= R || r / G >= s.n) continue;
      if (whole) {
        const float inv = 1.f / sM[R + r];
        uint16_t *dst = p.o + ((static_cast<size_t>(i) * p.m + r / G) * p.Hq + g * G + r % G) * HD + d0;
#pragma unroll
        for (int c = 0; c < CPT; c += 2)
          *reinterpret_cast<uint32_t *>(dst + c) = pack_bf16x2(acc[a][c] * inv, acc[a][c + 1] * inv);
      } else {
        float *dst = p.part_o + (slot0 * R + r) * HD + d0;
#pragma unroll
        for (int c = 0; c < CPT; ++c) dst[c] = acc[a][c];
        if (d0 == 0) {
          p.part_ml[(slot0 * R + r) * 2] = sM[r];
          p.part_ml[(slot0 * R + r) * 2 + 1] = sM[R + r];
        }
      }
    }
    __syncthreads();
    if (unit == s.units) {
      ++pair;
      unit = 0;
    }
  }
}

// Joins the partials of every pair whose units several CTAs took, in CTA order. One warp per
// query row, HD/32 consecutive values per lane.
constexpr int kMerge8Warps = 8;

template <int HD>
__global__ void __launch_bounds__(kMerge8Warps * 32) attn8_merge_kernel(const __grid_constant__ Attn8Params p) {
  constexpr int E = HD / 32;
  griddep_wait();
  griddep_launch();
  const int pair = blockIdx.x;
  const int i = pair / p.Hkv, g = pair % p.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv;
  const int R = G * p.m;
  const int r = blockIdx.y * kMerge8Warps + warp;
  const Seq8 s = seq8(p, i);
  if (r >= R || r / G >= s.n) return;
  long long T = 0, before = 0;
  for (int q = lane; q < p.nb; q += 32) {
    const int u = seq8(p, q).units;
    T += u;
    before += q < i ? u : 0;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    T += __shfl_xor_sync(0xffffffffu, T, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  T *= p.Hkv;
  const int Ge = T < p.grid ? static_cast<int>(T) : p.grid;
  const long long A = before * p.Hkv + static_cast<long long>(g) * s.units;
  const int c0 = cta_of(T, Ge, A), c1 = cta_of(T, Ge, A + s.units - 1);
  if (c0 == c1) return;  // written whole by the attention kernel
  float M = kNoMax, L = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int c = c0; c <= c1; ++c) {
    const size_t row = static_cast<size_t>(pair + c) * R + r;
    const float2 ml = *reinterpret_cast<const float2 *>(p.part_ml + row * 2);
    float v[E];
    const float *src = p.part_o + row * HD + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 x = *reinterpret_cast<const float2 *>(src + e);
      v[e] = x.x;
      v[e + 1] = x.y;
    }
    const float Mn = fmaxf(M, ml.x);
    const float a_old = exp2f(M - Mn), a_new = exp2f(ml.x - Mn);
    L = L * a_old + ml.y * a_new;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * a_old + v[e] * a_new;
    M = Mn;
  }
  const float inv = 1.0f / L;
  uint16_t *dst = p.o + ((static_cast<size_t>(i) * p.m + r / G) * p.Hq + g * G + r % G) * HD + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t *>(dst + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
}

template <int HD>
static cudaError_t launch_attn8(const Attn8Params &p, cudaStream_t s) {
  const int R = (p.Hq / p.Hkv) * p.m;
  const size_t smem = sizeof(float) * (static_cast<size_t>(R) * HD + kUnit * (HD + 1) + kUnit * HD + R * kUnit + 3 * R);
  static const cudaError_t configured =
      cudaFuncSetAttribute(attn8_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
  if (configured != cudaSuccess) return configured;
  cudaError_t e = launch_pdl(attn8_kernel<HD>, dim3(p.grid), dim3(kA8Threads), smem, s, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn8_merge_kernel<HD>, dim3(p.nb * p.Hkv, (R + kMerge8Warps - 1) / kMerge8Warps),
                    dim3(kMerge8Warps * 32), 0, s, p);
}

cudaError_t launch_attention8(const Attn8Params &p, cudaStream_t s) {
  if (p.Hq % p.Hkv != 0 || (p.Hq / p.Hkv) * p.m > 128) return cudaErrorInvalidValue;
  return p.hd == 128 ? launch_attn8<128>(p, s) : launch_attn8<64>(p, s);
}

}  // namespace df
