// What the kernels of the 8-bit attention (attention8.cu, attention8_wide.cu) share: the split of the
// work over CTAs and small device functions.
#pragma once

#include <cfloat>
#include <cmath>

#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace df {


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

// A weight of T is split over G CTAs: the first T % G take one more than the others (the units are
// below 2^25, as a handle's caches hold fewer than 2^31 rows, and T is at most 1 + pair_cost times that).
// The CTA that weight u lies in:
__device__ __forceinline__ int cta_of(int T, int G, int u) {
  const int q = T / G, big = (T % G) * (q + 1);
  return u < big ? u / (q + 1) : T % G + (u - big) / q;
}

// What the split counts for a pair: its units and p.pair_cost more before them, the time that a CTA
// takes to begin a pair and to write its rows, in units.
__device__ __forceinline__ int weight8(const Attn8Params &p, int units) { return units > 0 ? units + p.pair_cost : 0; }

// Weights of the sequences before i (`before`) and of all of them, times Hkv. Warp-collective.
__device__ __forceinline__ int total_weight(const Attn8Params &p, int i, int lane, int *before) {
  int t = 0, b = 0;
#pragma unroll 1
  for (int s = lane; s < p.nb; s += 32) {
    const int u = weight8(p, seq8(p, s).units);
    t += u;
    b += s < i ? u : 0;
  }
  *before = __reduce_add_sync(0xffffffffu, b) * p.Hkv;
  return __reduce_add_sync(0xffffffffu, t) * p.Hkv;
}

// x / d for quotients below 2^21: the float estimate is at most one off.
__device__ __forceinline__ int div_near(int x, int d) {
  int q = static_cast<int>(__fdividef(static_cast<float>(x), static_cast<float>(d)));
  const int r = x - q * d;
  q += r < 0 ? -1 : r >= d ? 1 : 0;
  return q;
}

// A CTA's range: sequence, kv head and unit where it begins, its number of units (0 for a range inside one
// pair's cost), and that sequence's rows, context and units.
struct Range8 {
  int i, g, unit, count, n, ctx, units;
};
// Warp-collective.
static __device__ void find_range(const Attn8Params &p, int cta, int lane, Range8 *out) {
  const Seq8 s0 = lane < p.nb ? seq8(p, lane) : Seq8{0, 0, 0};
  int t = weight8(p, s0.units);
#pragma unroll 1
  for (int s = lane + 32; s < p.nb; s += 32) t += weight8(p, seq8(p, s).units);
  const int T = __reduce_add_sync(0xffffffffu, t) * p.Hkv;
  const int Ge = min(T, p.grid);
  Range8 at = {};
  if (cta < Ge) {
    const int each = div_near(T, Ge), more = T - each * Ge;
    const int w0 = cta * each + min(cta, more), w1 = w0 + each + (cta < more ? 1 : 0);
    int base = 0, pairs = 0;               // weight and pairs with units before this chunk of sequences
    int first = 0, last = 0;               // units of all pairs before the range's ends
    bool ended = false;
#pragma unroll 1
    for (int b = 0; b < p.nb && !ended; b += 32) {
      const Seq8 s = b == 0 ? s0 : b + lane < p.nb ? seq8(p, b + lane) : Seq8{0, 0, 0};
      const int W = weight8(p, s.units);
      int v = p.Hkv * W;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
      }
      const unsigned some = __ballot_sync(0xffffffffu, s.units > 0);
      const int start = base + v - p.Hkv * W;  // of the lane's sequence
      const int units = start - p.pair_cost * (pairs + p.Hkv * __popc(some & ((1u << lane) - 1)));
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int x = (k == 0 ? w0 : w1) - start;
        const unsigned hit = __ballot_sync(0xffffffffu, x >= 0 && x < p.Hkv * W);
        if (hit) {
          const int g = div_near(x, max(W, 1)), in = max(x - g * W - p.pair_cost, 0);  // the lane that was hit counts
          const int l = __ffs(hit) - 1;
          const int before = __shfl_sync(0xffffffffu, units + g * s.units + in, l);
          if (k == 0) {
            at = {b + l, __shfl_sync(0xffffffffu, g, l), __shfl_sync(0xffffffffu, in, l), 0,
                  __shfl_sync(0xffffffffu, s.n, l), __shfl_sync(0xffffffffu, s.ctx, l),
                  __shfl_sync(0xffffffffu, s.units, l)};
            first = before;
          } else {
            last = before;
            ended = true;
          }
        }
      }
      base += __shfl_sync(0xffffffffu, v, 31);
      pairs += p.Hkv * __popc(some);
    }
    if (!ended) last = T - p.pair_cost * pairs;  // the last range: w1 = T
    at.count = last - first;
  }
  if (lane == 0) *out = at;
}

// Asks for the parameters that the split reads, so that they come while the launch before this one
// ends and not one miss after the other behind it.
__device__ __forceinline__ void touch8(const Attn8Params &p) {
  asm volatile("" ::"r"(p.nb), "r"(p.m), "r"(p.Hq), "r"(p.Cmax), "r"(p.grid), "l"(p.n_rows), "l"(p.page_table));
}

constexpr int kSeqCache = 128;     // sequences whose lengths a CTA keeps in shared memory
constexpr int kDrainSpin = 1 << 22;

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A block's scales as the softmax uses them: K's, log2 of V's, the factor that takes P to its share of the sum, and
// what the block is. P = 2^(x + log2 V - reference + base) weighs a key's values, so the reference follows what
// counts in the output; the sum takes 2^(x - reference + base - kSumExp), without V's scale. Where that scale is low, P
// can be zero though the sum counts the key: there (kLowScale, kZeroScale) the sum's terms are exponentials of their
// own and the factor is zero. Sums move in two halves, since 2^-d may be zero where a sum times 2^-d is not.
// With V scales of 2^-100 .. 2^80 all of it stays within fp32: low is below 2^-20, and beside a scale of 2^80 one of
// 2^-20 has P zero only for keys 2^34 below the reference's. Scales below 2^-100 count as that; zero does
// too, so that it moves no reference, but its P is zero (so a NaN byte gives NaN, as NaN times zero).
constexpr float kSumExp = 20.f, kSumScale = 1.f / (1 << 20);
constexpr float kLowScale = 1.f, kZeroScale = 2.f;
__device__ __forceinline__ float4 scale_terms(float ks, float vs) {
  const bool low = vs < 1.f / (1 << 20);
  return make_float4(ks, fmaxf(log2f(vs), -100.f), low ? 0.f : kSumScale / vs,
                     vs == 0.f ? kZeroScale : low ? kLowScale : 0.f);
}
// 2^d times a sum, for d <= 0.
__device__ __forceinline__ float moved_sum(float sum, float d) {
  const float h = ex2f(0.5f * d);
  return sum * h * h;
}

// A NaN among values that only some query rows see would reach the others as well, as 0 * NaN in the product
// of P and V. So it is taken out of the operand, and `first[column]` keeps the first row that sees one; that
// row and those behind it get the NaN with their output. Returns the word without its NaN bytes, which
// belong to the columns from col on and are seen from row `row` on.
constexpr int kNoNan = 1 << 30;
__device__ __forceinline__ uint32_t take_nan(uint32_t w, int *first, int col, int row) {
  const uint32_t nan = ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
  if (nan == 0) [[likely]] return w;
#pragma unroll
  for (int b = 0; b < 4; ++b)
    if (nan >> (8 * b + 7) & 1) atomicMin(first + col + b, row);
  return w & ~((nan >> 7) * 0xFFu);
}

// One of the warp's threads, the same one every time; the branch on it leaves the code around it
// warp-uniform.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
  return ok != 0;
}

// A unit inside a CTA's range: sequence i, kv head g, unit of `units`.
struct Pos8 {
  int i, g, unit, units, n, ctx;
};
static __device__ __noinline__ int2 seq_far(const Attn8Params &p, int i) {
  const Seq8 s = seq8(p, i);
  return make_int2(s.n, s.ctx);
}
__device__ __forceinline__ void pos_seq(Pos8 &w, const Attn8Params &p, const int2 *sseq) {
#pragma unroll 1
  for (;; ++w.i) {  // a sequence without rows has no units (one with rows follows)
    const int2 s = w.i < kSeqCache ? sseq[w.i] : seq_far(p, w.i);
    w.n = s.x;
    w.ctx = s.y;
    w.units = w.n > 0 ? (w.ctx + w.n + kUnit - 1) / kUnit : 0;
    if (w.units > 0) return;
  }
}
// To the pair (sequence, kv head) after this one.
__device__ __forceinline__ void pos_next_pair(Pos8 &w, const Attn8Params &p, const int2 *sseq) {
  w.unit = 0;
  if (++w.g == p.Hkv) {
    w.g = 0;
    ++w.i;
    pos_seq(w, p, sseq);
  }
}

}  // namespace df
