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
__device__ __forceinline__ int cta_start(int T, int G, int c) { return c * (T / G) + min(c, T % G); }
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

// Where a CTA's range begins (pair i * Hkv + g, unit inside it) and its number of units, which is 0
// for a range inside one pair's cost. Warp-collective.
static __device__ void find_range(const Attn8Params &p, int cta, int lane, int *out) {
  int base;
  const int T = total_weight(p, 0, lane, &base);
  const int Ge = min(T, p.grid);
  int pair = 0, unit = 0, first = 0, last = 0;  // units of all pairs before the range's ends
  if (cta < Ge) {
    const int w0 = cta_start(T, Ge, cta), w1 = cta_start(T, Ge, cta + 1);
    int pairs = 0;  // with units, before this chunk of sequences
    bool ended = false;
#pragma unroll 1
    for (int b = 0; b < p.nb && !ended; b += 32) {
      const int U = b + lane < p.nb ? seq8(p, b + lane).units : 0;
      const int W = weight8(p, U);
      int v = p.Hkv * W;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
      }
      const unsigned some = __ballot_sync(0xffffffffu, U > 0);
      const int start = base + v - p.Hkv * W;  // of the lane's sequence
      const int units = start - p.pair_cost * (pairs + p.Hkv * __popc(some & ((1u << lane) - 1)));
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int w = k == 0 ? w0 : w1;
        const unsigned hit = __ballot_sync(0xffffffffu, start <= w && w < base + v);
        if (hit) {
          const int off = (w - start) / max(W, 1), in = max((w - start) % max(W, 1) - p.pair_cost, 0);
          const int l = __ffs(hit) - 1;
          const int at = __shfl_sync(0xffffffffu, units + off * U + in, l);
          if (k == 0) {
            pair = (b + l) * p.Hkv + __shfl_sync(0xffffffffu, off, l);
            unit = __shfl_sync(0xffffffffu, in, l);
            first = at;
          } else {
            last = at;
            ended = true;
          }
        }
      }
      base += __shfl_sync(0xffffffffu, v, 31);
      pairs += p.Hkv * __popc(some);
    }
    if (!ended) last = T - p.pair_cost * pairs;  // the last range: w1 = T
  }
  if (lane == 0) {
    out[0] = pair;
    out[1] = unit;
    out[2] = last - first;
  }
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
