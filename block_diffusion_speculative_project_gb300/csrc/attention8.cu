// Attention of m query rows per sequence over a cache held in 8 bits (tcgen05): e4m3 keys and values with
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
#include <mutex>

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

// ---------------------------------------------------------------- tensor-core kernel

// RHO copies of the query rows fill the 128 lanes of the MMA (rows padded to 128 / RHO): the lanes
// of copy c take only the c-th part of a unit's keys, the other parts' probabilities being zero
// in the P operand, so that every SM quarter's warps share the exponentials of few rows.
template <int HD>
struct A8Cfg {
  static constexpr int ATOMS = HD / 64;              // 128-byte swizzle atoms across hd (f16)
  static constexpr int UNIT8 = kUnit * HD;           // bytes of a unit's keys (or values) in the cache
  static constexpr int NS = HD == 128 ? 8 : 16;      // ring of units in 8 bits
  static constexpr int ATOM16 = kUnit * 128;
  static constexpr int TILE16 = ATOMS * ATOM16;      // a unit's keys (or values) in f16
  static constexpr int OFF_V16 = 2 * TILE16;
  static constexpr int OFF_8 = 4 * TILE16;
  static constexpr int OFF_STG = OFF_8 + NS * 2 * UNIT8;  // O of the copies c > 0, 16 columns at a time
  static constexpr int STG = 3 * 32 * 17 * 4;             // (RHO - 1) * (128 / RHO) rows of 17 floats
  static constexpr int OFF_ML = OFF_STG + STG;            // [2 halves][128 lanes] (maximum, sum)
  static constexpr int OFF_BAR = OFF_ML + 2 * 128 * 8;
  static constexpr int OFF_SEQ = OFF_BAR + 512;           // [kSeqCache] (rows, context)
  static constexpr size_t SMEM = 1024 + OFF_SEQ + 128 * 8;
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t S_COL = 0;                // S of unit j in buffer j % 2: 64 columns each
  static constexpr uint32_t O_COL = 128;              // O_0, O_1: hd columns each
  static constexpr uint32_t Q_COL = 128 + 2 * HD;     // f16 queries: hd / 2 columns
  static constexpr uint32_t P_COL = Q_COL + HD / 2;   // P of unit j in buffer j % 2: 32 columns each
  static_assert(P_COL + 64 <= TMEM_COLS, "tensor memory");
};
constexpr int kSeqCache = 128;
constexpr int kDrainSpin = 1 << 22;
// P is 2^(x - m_run + kPBase), m_run the maximum at the last rescale: O is rescaled only when the
// maximum has grown by more than 2^kRescale, so P stays at most 2^15 in f16, and what is 2^-21 of
// the largest still has all 11 bits (2^-31 one bit).
constexpr float kPBase = 7.f, kRescale = 8.f;

// Warps: softmax half h = 0, 1 (units j % 2 == h) in 4h .. 4h + 3 (warp w reads TMEM lanes of
// quarter w % 4), producer, S issuer, PV issuer, then the converters (two for K, two for V).
constexpr int kWProd = 8, kWS = 9, kWPV = 10, kWConv = 11, kNumConv = 4;
constexpr int kA8Threads = (kWConv + kNumConv) * 32;

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct Walk8 {
  int pair, unit, n, ctx, units, left, seg, seg_unit0;
};
__device__ __forceinline__ void walk_pair(Walk8 &w, const Attn8Params &p, const int2 *sseq) {
  for (;;) {
    const int i = w.pair / p.Hkv;
    if (i < kSeqCache) {
      w.n = sseq[i].x;
      w.ctx = sseq[i].y;
      w.units = w.n > 0 ? (w.ctx + w.n + kUnit - 1) / kUnit : 0;
    } else {
      const Seq8 s = seq8(p, i);
      w.n = s.n;
      w.ctx = s.ctx;
      w.units = s.units;
    }
    if (w.units > 0) return;
    w.pair = (i + 1) * p.Hkv;  // a sequence without rows (left > 0: one with rows follows)
  }
}
__device__ __forceinline__ bool walk_first(const Walk8 &w) { return w.unit == w.seg_unit0; }
__device__ __forceinline__ bool walk_last(const Walk8 &w) { return w.left == 1 || w.unit == w.units - 1; }
__device__ __forceinline__ void walk_next(Walk8 &w, const Attn8Params &p, const int2 *sseq) {
  --w.left;
  if (++w.unit == w.units) {
    ++w.pair;
    w.unit = 0;
    w.seg_unit0 = 0;
    ++w.seg;
    if (w.left > 0) walk_pair(w, p, sseq);
  }
}
// One past the last unit of the current segment.
__device__ __forceinline__ int walk_end(const Walk8 &w) { return min(w.units, w.unit + w.left); }

template <int KW>
__device__ __forceinline__ void load_s(uint32_t taddr, float (&v)[KW]) {
  if constexpr (KW == 64)
    tmem_ld64(taddr, v);
  else if constexpr (KW == 32)
    tmem_ld32(taddr, v);
  else
    tmem_ld16(taddr, v);
}
template <int KW>
__device__ __forceinline__ void store_p(uint32_t taddr, const uint32_t *v) {
  if constexpr (KW == 64)
    tmem_st32_raw(taddr, v);
  else if constexpr (KW == 32)
    tmem_st16_raw(taddr, v);
  else
    tmem_st8_raw(taddr, v);
}

// 16 e4m3 values to 32 bytes of f16 (exact).
__device__ __forceinline__ void widen16(const uint4 &u, uint32_t (&h)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[e] & 0xFFFFu), __NV_E4M3);
    const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[e] >> 16), __NV_E4M3);
    h[2 * e] = static_cast<uint32_t>(lo.x) | (static_cast<uint32_t>(lo.y) << 16);
    h[2 * e + 1] = static_cast<uint32_t>(hi.x) | (static_cast<uint32_t>(hi.y) << 16);
  }
}

template <int HD, int RHO>
__global__ void __launch_bounds__(kA8Threads, 1) attn8_kernel(const __grid_constant__ Attn8Params p) {
  using C = A8Cfg<HD>;
  constexpr int KW = kUnit / RHO;      // keys of a unit per copy
  constexpr int ROWS = 128 / RHO;      // padded query rows
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint8_t *sK16 = smem, *sV16 = smem + C::OFF_V16, *s8 = smem + C::OFF_8;
  float *stage = reinterpret_cast<float *>(smem + C::OFF_STG);
  float2 *ml = reinterpret_cast<float2 *>(smem + C::OFF_ML);
  uint64_t *kv8_full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
  uint64_t *kv8_empty = kv8_full + C::NS;
  uint64_t *k16_full = kv8_empty + C::NS;   // [2] unit j in buffer j % 2
  uint64_t *v16_full = k16_full + 2;        // [2]
  uint64_t *s_full = v16_full + 2;          // [2] S(j) complete: also K16 buffer j % 2 read
  uint64_t *s_empty = s_full + 2;           // [2]
  uint64_t *p_full = s_empty + 2;           // [2]
  uint64_t *p_empty = p_full + 2;           // [2] PV(j) complete: P and V16 buffers j % 2 read
  uint64_t *q_full = p_empty + 2;
  uint64_t *q_empty = q_full + 1;
  uint64_t *o_free = q_empty + 1;           // both O and ml read at a segment's end
  uint64_t *ml_ready = o_free + 1;
  uint64_t *half0 = ml_ready + 1;           // the four warps of half 0 among themselves
  uint64_t *mma_done = half0 + 1;           // [2]
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_done + 2);
  int *sched = reinterpret_cast<int *>(tmem_slot + 1);
  static_assert((2 * 16 + 12 + 7) * 8 + 16 <= 512, "barrier region overflows");
  int2 *sseq = reinterpret_cast<int2 *>(smem + C::OFF_SEQ);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv;
  const int R = G * p.m;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(&kv8_full[s], 1);
      mbar_init(&kv8_empty[s], kNumConv);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&k16_full[b], kNumConv / 2);
      mbar_init(&v16_full[b], kNumConv / 2);
      mbar_init(&s_full[b], 1);
      mbar_init(&s_empty[b], 4);
      mbar_init(&p_full[b], 4);
      mbar_init(&p_empty[b], 1);
      mbar_init(&mma_done[b], 1);
    }
    mbar_init(q_full, 4);
    mbar_init(q_empty, 1);
    mbar_init(o_free, 4);
    mbar_init(ml_ready, 4);
    mbar_init(half0, 4);
    fence_mbar_init();
  }
  if (warp == kWS) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch();
  if (warp == kWProd) {
    const Range8 r = find_range(p, blockIdx.x, lane);
    if (lane == 0) {
      sched[0] = r.pair;
      sched[1] = r.unit;
      sched[2] = static_cast<int>(r.count);
    }
  } else if (warp == kWConv) {
    for (int i = lane; i < p.nb && i < kSeqCache; i += 32) {
      const Seq8 s = seq8(p, i);
      sseq[i] = make_int2(s.n, s.ctx);
    }
  } else if (warp == kWPV && blockIdx.x == 0) {
    for (int i = lane; i < p.nb; i += 32) {
      const int n = p.n_rows ? p.n_rows[i] : p.m, c = p.ctx_len[i];
      if (n < 0 || n > p.m || c < 0 || c > p.max_ctx || static_cast<long long>(c) + max(n, 0) > p.Cmax)
        flag_status(p.status, kStatusCheck);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int nunits = sched[2];
  Walk8 w;
  w.pair = sched[0];
  w.unit = sched[1];
  w.left = nunits;
  w.seg = 0;
  w.seg_unit0 = w.unit;
  w.n = w.ctx = w.units = 0;
  if (nunits > 0) walk_pair(w, p, sseq);

  if (nunits == 0) {
    // nothing to do
  } else if (warp == kWProd) {
    // ---------------- producer: a unit's keys and values are contiguous 64 * hd bytes each. The
    // warp reads the block indices of 32 units at once, lane 0 issues the copies.
    const uint64_t pol = policy_evict_first();
    bool ok = !p.stall;
    int j = 0, issued = 0, blk = 0;
    for (; j < nunits && ok; ++j) {
      const int k = (w.unit - w.seg_unit0) & 31;
      const int i = w.pair / p.Hkv, g = w.pair % p.Hkv;
      if (k == 0) blk = static_cast<int>(block_of(p, i, g, min(w.unit + lane, walk_end(w) - 1)));
      const long long b = __shfl_sync(0xffffffffu, blk, k);
      const int st = j % C::NS;
      if (lane == 0) {
        ok = j < C::NS || mbar_wait(&kv8_empty[st], ((j / C::NS) - 1) & 1, p.max_spin);
        if (ok) {
          uint8_t *dst = s8 + st * 2 * C::UNIT8;
          mbar_arrive_expect_tx(&kv8_full[st], 2 * C::UNIT8);
          bulk_load(dst, p.k8 + b * C::UNIT8, C::UNIT8, &kv8_full[st], pol);
          bulk_load(dst + C::UNIT8, p.v8 + b * C::UNIT8, C::UNIT8, &kv8_full[st], pol);
          ++issued;
        }
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      walk_next(w, p, sseq);
    }
    if (lane == 0) {
      if (!ok && !p.stall) flag_status(p.status, kStatusTimeout);
      // every issued copy must land before the CTA may exit (bounded)
      for (int k = max(0, issued - C::NS); k < issued; ++k)
        mbar_wait(&kv8_full[k % C::NS], (k / C::NS) & 1, kDrainSpin);
    }
  } else if (warp == kWS) {
    if (lane == 0) {
      // ---------------- S issuer: S(j) = Q K(j)^T, queries from tensor memory
      constexpr uint32_t id_s = idesc_f16_f32(128, kUnit);
      const uint64_t kd0 = sw128_kmajor_desc(smem_u32(sK16));
      bool ok = true;
      for (int j = 0; j < nunits; ++j) {
        const int b = j & 1;
        if (walk_first(w)) ok = mbar_wait(q_full, w.seg & 1, p.max_spin);
        ok = ok && mbar_wait(&k16_full[b], (j >> 1) & 1, p.max_spin);
        ok = ok && (j < 2 || mbar_wait(&s_empty[b], ((j >> 1) - 1) & 1, p.max_spin));
        if (!ok) break;
        tc_fence_after();
        const uint64_t kd = kd0 + static_cast<uint64_t>((b * C::TILE16) >> 4);
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
          tc_mma_bf16_tmem_a(tmem + C::S_COL + b * kUnit, tmem + C::Q_COL + kk * 8,
                             kd + static_cast<uint64_t>(((kk >> 2) * C::ATOM16 + (kk & 3) * 32) >> 4), id_s,
                             kk > 0 ? 1u : 0u);
        tc_commit(&s_full[b]);
        if (walk_last(w)) tc_commit(q_empty);
        walk_next(w, p, sseq);
      }
      if (!ok) flag_status(p.status, kStatusTimeout);
      // every issued MMA must complete before TMEM is freed (bounded)
      tc_commit(&mma_done[0]);
      mbar_wait(&mma_done[0], 0, kDrainSpin);
    }
  } else if (warp == kWPV) {
    if (lane == 0) {
      // ---------------- PV issuer: O_{j%2} += P(j) V(j); the first unit of each half in a segment
      // starts the accumulator, after both O of the previous segment were read
      constexpr uint32_t id_pv = idesc_f16_f32(128, HD) | kIdescBMajorMN;
      const uint64_t vd0 = sw128_mnmajor_desc(smem_u32(sV16), C::ATOM16);
      bool ok = true;
      int jf = 0;
      for (int j = 0; j < nunits; ++j) {
        const int b = j & 1;
        if (walk_first(w)) jf = j;
        const bool start = j < jf + 2;
        ok = mbar_wait(&v16_full[b], (j >> 1) & 1, p.max_spin);
        ok = ok && mbar_wait(&p_full[b], (j >> 1) & 1, p.max_spin);
        if (start && w.seg > 0) ok = ok && mbar_wait(o_free, (w.seg - 1) & 1, p.max_spin);
        if (!ok) break;
        tc_fence_after();
        const uint64_t vd = vd0 + static_cast<uint64_t>((b * C::TILE16) >> 4);
#pragma unroll
        for (int kk = 0; kk < kUnit / 16; ++kk)
          tc_mma_bf16_tmem_a(tmem + C::O_COL + b * HD, tmem + C::P_COL + b * 32 + kk * 8,
                             vd + static_cast<uint64_t>((kk * 16 * 128) >> 4), id_pv,
                             (!start || kk > 0) ? 1u : 0u);
        tc_commit(&p_empty[b]);
        walk_next(w, p, sseq);
      }
      if (!ok) flag_status(p.status, kStatusTimeout);
      tc_commit(&mma_done[1]);
      mbar_wait(&mma_done[1], 0, kDrainSpin);
    }
  } else if (warp >= kWConv) {
    // ---------------- converters: e4m3 tiles to f16 tiles in the layout of a 128-byte-swizzled
    // copy (rows of 64 values, 16-byte chunk c of row r at c ^ (r & 7)); warps 0, 1 keys, 2, 3 values
    const int cw = warp - kWConv;
    const bool is_v = cw >= 2;
    uint64_t *full16 = is_v ? v16_full : k16_full;
    uint64_t *empty16 = is_v ? p_empty : s_full;   // the MMAs that read the buffer have completed
    uint8_t *out = is_v ? sV16 : sK16;
    constexpr int CPR = HD / 16;                   // 16-byte chunks of a row in 8 bits
    constexpr int PER = kUnit * CPR / 64;          // chunks per thread (two warps)
    const int t = (cw & 1) * 32 + lane;
    bool ok = true;
    for (int j = 0; j < nunits; ++j) {
      const int st = j % C::NS, b = j & 1;
      const int keys = w.ctx + w.n - w.unit * kUnit;  // rows of the unit that hold keys
      ok = mbar_wait(&kv8_full[st], (j / C::NS) & 1, p.max_spin);
      ok = ok && (j < 2 || mbar_wait(&empty16[b], ((j >> 1) - 1) & 1, p.max_spin));
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint8_t *src = s8 + st * 2 * C::UNIT8 + (is_v ? C::UNIT8 : 0);
      uint8_t *dst = out + b * C::TILE16;
#pragma unroll 4
      for (int e = 0; e < PER; ++e) {
        const int c = t + e * 64;
        const int r = c / CPR, cc = c % CPR;
        uint4 u = *reinterpret_cast<const uint4 *>(src + c * 16);
        // V rows beyond the last key may hold anything (even NaN); P is 0 there
        if (is_v && r >= keys) u = make_uint4(0, 0, 0, 0);
        uint32_t h[8];
        widen16(u, h);
        uint8_t *row = dst + (cc >> 2) * C::ATOM16 + r * 128;
        const int c0 = (cc & 3) * 2;
        // lanes of the second atom store their halves in the other order: no bank conflicts
        const int first = (cc >> 2) & 1;
        const uint4 a = first ? make_uint4(h[4], h[5], h[6], h[7]) : make_uint4(h[0], h[1], h[2], h[3]);
        const uint4 d = first ? make_uint4(h[0], h[1], h[2], h[3]) : make_uint4(h[4], h[5], h[6], h[7]);
        *reinterpret_cast<uint4 *>(row + (((c0 + first) ^ (r & 7)) << 4)) = a;
        *reinterpret_cast<uint4 *>(row + (((c0 + 1 - first) ^ (r & 7)) << 4)) = d;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&full16[b]);
        mbar_arrive(&kv8_empty[st]);
      }
      walk_next(w, p, sseq);
    }
    if (!ok && lane == 0) flag_status(p.status, kStatusTimeout);
  } else {
    // ---------------- softmax: thread = TMEM lane; lane l holds query row l % ROWS, copy l / ROWS
    const int half = warp >> 2, q = warp & 3;
    const int tl = q * 32 + lane;
    const int r = tl % ROWS, copy = tl / ROWS;
    const int k0 = copy * KW;
    const bool real = r < R;
    const uint32_t trow = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const int jq = r / G, hq = r % G;   // row r: query row jq of query head g * G + hq
    const float sl2 = rsqrtf(static_cast<float>(HD)) * 1.4426950408889634f;
    if (RHO > 1) {  // the other copies' parts of the P rows stay zero
      const uint32_t z[32] = {};
      tmem_st32_raw(trow + C::P_COL + half * 32, z);
      tmem_wait_st();
    }
    // Barrier of half 0's warps, bounded like every other wait.
    uint32_t half0_phase = 0;
    auto half0_sync = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(half0);
      const bool done = mbar_wait(half0, half0_phase, p.max_spin);
      half0_phase ^= 1;
      return __all_sync(0xffffffffu, done) != 0;
    };
    bool ok = true;
    float m_run = kNoMax, l_run = 0.f, qfac = 0.f;
    float ks_c = 0.f, lv_c = 0.f, iv_c = 0.f;   // scales of 32 units (this lane's): K, log2 of V, 1 / V
    float ks_n = 0.f, vs_n = 0.f;               // the next 32
    int jf = 0;
    for (int j = 0; j < nunits; ++j) {
      const int i = w.pair / p.Hkv, g = w.pair % p.Hkv;
      const int ku = w.unit - w.seg_unit0;
      if ((ku & 31) == 0) {
        const int end = walk_end(w) - 1;
        if (ku == 0) {
          const long long b = block_of(p, i, g, min(w.unit + lane, end));
          ks_n = p.ks[b];
          vs_n = p.vs[b];
        }
        ks_c = ks_n;
        lv_c = vs_n == 0.f ? 0.f : log2f(vs_n);
        iv_c = vs_n == 0.f ? 0.f : 1.f / vs_n;   // 0 marks a block of zeros
        if (w.unit + 32 <= end) {
          const long long b = block_of(p, i, g, min(w.unit + 32 + lane, end));
          ks_n = p.ks[b];
          vs_n = p.vs[b];
        }
      }
      if (walk_first(w)) {
        jf = j;
        m_run = kNoMax;
        l_run = 0.f;
        // this thread's query row, scaled by a power of two so that its largest value lies in
        // [2^14, 2^15): exact in f16 down to 2^-31 of it
        const uint4 *src = reinterpret_cast<const uint4 *>(
            p.q + ((static_cast<size_t>(i) * p.m + jq) * p.Hq + g * G + hq) * HD);
        const bool have = real && jq < w.n;
        float am = 0.f;
#pragma unroll 8
        for (int e = 0; e < HD / 8; ++e) {
          const uint4 u = have ? src[e] : make_uint4(0, 0, 0, 0);
          const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int f = 0; f < 4; ++f)
            am = fmaxf(am, fmaxf(fabsf(__uint_as_float(x[f] << 16)), fabsf(__uint_as_float(x[f] & 0xFFFF0000u))));
        }
        int ex = static_cast<int>(__float_as_uint(am) >> 23) - 127;   // -127: zero or subnormal, 128: infinite
        ex = ex == 128 ? 14 : max(ex, -100);
        const float mul = __uint_as_float(static_cast<uint32_t>(14 - ex + 127) << 23);
        qfac = sl2 * __uint_as_float(static_cast<uint32_t>(ex - 14 + 127) << 23);
        if (half == 0) {
          ok = w.seg == 0 || mbar_wait(q_empty, (w.seg - 1) & 1, p.max_spin);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int part = 0; part < HD / 32; ++part) {
            uint32_t h[16];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint4 u = have ? src[part * 4 + e] : make_uint4(0, 0, 0, 0);
              const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
              for (int f = 0; f < 4; ++f) {
                const __half2 y = __floats2half2_rn(__uint_as_float(x[f] << 16) * mul,
                                                    __uint_as_float(x[f] & 0xFFFF0000u) * mul);
                h[4 * e + f] = *reinterpret_cast<const uint32_t *>(&y);
              }
            }
            tmem_st16_raw(trow + C::Q_COL + part * 16, h);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(q_full);
        }
      }
      if ((j & 1) == half) {
        const bool first = j < jf + 2;  // first unit of this half in the segment
        const float ks = __shfl_sync(0xffffffffu, ks_c, ku & 31);
        const float lv = __shfl_sync(0xffffffffu, lv_c, ku & 31);
        const float iv = __shfl_sync(0xffffffffu, iv_c, ku & 31);
        const int lim = p.causal ? min(w.ctx + jq + 1, w.ctx + w.n) : w.ctx + w.n;
        const int nv = lim - w.unit * kUnit - k0;  // keys this thread sees of its part
        ok = mbar_wait(&s_full[half], (j >> 1) & 1, p.max_spin);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        float sv[KW];
        load_s<KW>(trow + C::S_COL + half * kUnit + k0, sv);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_empty[half]);

        if (__any_sync(0xffffffffu, nv < KW)) {
#pragma unroll
          for (int c = 0; c < KW; ++c) sv[c] = c < nv ? sv[c] : -INFINITY;
        }
        const float c1 = fmaxf(qfac * ks, 1e-37f);
        float mx[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
        for (int c = 4; c < KW; ++c) mx[c & 3] = fmaxf(mx[c & 3], sv[c]);
        const float m_new = fmaf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), c1, lv);
        const bool need = m_new - m_run > kRescale;
        float alpha = 1.f;
        if (need) {
          alpha = ex2f(m_run - m_new);
          m_run = m_new;
          l_run *= alpha;
        }
        // P buffer and O_half: free once PV of this half's previous unit has completed
        if (j >= 2) {
          ok = mbar_wait(&p_empty[half], ((j >> 1) - 1) & 1, p.max_spin);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          tc_fence_after();
        }
        if (!first && __any_sync(0xffffffffu, need && real)) {
#pragma unroll 1
          for (int cc = 0; cc < HD / 16; ++cc) {
            float ov[16];
            tmem_ld16(trow + C::O_COL + half * HD + cc * 16, ov);
            uint32_t x[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) x[c] = __float_as_uint(ov[c] * alpha);
            tmem_st16_raw(trow + C::O_COL + half * HD + cc * 16, x);
          }
        }
        const float c2 = lv - m_run + kPBase;
        uint32_t pk[KW / 2];
        float ls[2] = {0.f, 0.f};
#pragma unroll
        for (int c = 0; c < KW; c += 2) {
          const float p0 = ex2f(fmaf(sv[c], c1, c2));
          const float p1 = ex2f(fmaf(sv[c + 1], c1, c2));
          ls[0] += p0;
          ls[1] += p1;
          const __half2 y = __floats2half2_rn(p0, p1);
          pk[c / 2] = *reinterpret_cast<const uint32_t *>(&y);
        }
        l_run = fmaf(ls[0] + ls[1], iv == 0.f ? 1.f : iv, l_run);
        if (iv == 0.f) {
#pragma unroll
          for (int c = 0; c < KW / 2; ++c) pk[c] = 0u;
        }
        store_p<KW>(trow + C::P_COL + half * 32 + k0 / 2, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[half]);
      }

      if (walk_last(w)) {
        // segment [jf, j]: the last unit of each half in it, or -1
        const int seg = w.seg;
        const int last0 = (j & 1) == 0 ? j : (j - 1 >= jf ? j - 1 : -1);
        const int last1 = (j & 1) == 1 ? j : (j - 1 >= jf ? j - 1 : -1);
        const int mine = half ? last1 : last0;
        ok = mine < 0 || mbar_wait(&p_empty[half], (mine >> 1) & 1, p.max_spin);
        // the (maximum, sum) slots are free once the previous segment's were read
        if (half == 1) ok = ok && (seg == 0 || mbar_wait(o_free, (seg - 1) & 1, p.max_spin));
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        const float2 own = mine >= 0 ? make_float2(m_run, l_run) : make_float2(kNoMax, 0.f);
        ml[half * 128 + tl] = own;
        if (half == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(ml_ready);
        } else {
          ok = mbar_wait(ml_ready, seg & 1, p.max_spin) && ok;
          if (!__all_sync(0xffffffffu, ok) || !half0_sync()) {
            ok = false;
            break;
          }
          tc_fence_after();
          float M = kNoMax;
#pragma unroll
          for (int c = 0; c < RHO; ++c)
            M = fmaxf(M, fmaxf(ml[c * ROWS + r].x, ml[128 + c * ROWS + r].x));
          float L = 0.f;
#pragma unroll
          for (int c = 0; c < RHO; ++c) {
            const float2 x = ml[c * ROWS + r], y = ml[128 + c * ROWS + r];
            L += x.y * ex2f(x.x - M) + y.y * ex2f(y.x - M);
          }
          const bool has0 = last0 >= 0, has1 = last1 >= 0;
          const float a0 = ex2f(own.x - M), a1 = ex2f(ml[128 + tl].x - M);
          const bool whole = w.seg_unit0 == 0 && w.unit == w.units - 1;
          const size_t row = (static_cast<size_t>(w.pair) + blockIdx.x) * R + r;
          const float inv = 1.0f / L;
          const bool put = real && jq < w.n;
#pragma unroll 1
          for (int cc = 0; cc < HD / 16 && ok; ++cc) {
            float ov[16], o1[16];
            if (has0) tmem_ld16(trow + C::O_COL + cc * 16, ov);
            if (has1) tmem_ld16(trow + C::O_COL + HD + cc * 16, o1);
#pragma unroll
            for (int c = 0; c < 16; ++c) ov[c] = (has0 ? ov[c] * a0 : 0.f) + (has1 ? o1[c] * a1 : 0.f);
            if (RHO > 1) {
              if (copy > 0) {
                float *to = stage + ((copy - 1) * ROWS + r) * 17;
#pragma unroll
                for (int c = 0; c < 16; ++c) to[c] = ov[c];
              }
              ok = half0_sync();
              if (copy == 0) {
#pragma unroll
                for (int x = 0; x < RHO - 1; ++x) {
                  const float *from = stage + (x * ROWS + r) * 17;
#pragma unroll
                  for (int c = 0; c < 16; ++c) ov[c] += from[c];
                }
              }
              ok = ok && half0_sync();
            }
            if (copy == 0 && put && whole) {
              uint16_t *dst = p.o + ((static_cast<size_t>(i) * p.m + jq) * p.Hq + g * G + hq) * HD + cc * 16;
#pragma unroll
              for (int v = 0; v < 2; ++v)
                reinterpret_cast<uint4 *>(dst)[v] =
                    make_uint4(pack_bf16x2(ov[8 * v] * inv, ov[8 * v + 1] * inv),
                               pack_bf16x2(ov[8 * v + 2] * inv, ov[8 * v + 3] * inv),
                               pack_bf16x2(ov[8 * v + 4] * inv, ov[8 * v + 5] * inv),
                               pack_bf16x2(ov[8 * v + 6] * inv, ov[8 * v + 7] * inv));
            } else if (copy == 0 && put) {
              float *dst = p.part_o + row * HD + cc * 16;
#pragma unroll
              for (int v = 0; v < 4; ++v)
                reinterpret_cast<float4 *>(dst)[v] =
                    make_float4(ov[4 * v], ov[4 * v + 1], ov[4 * v + 2], ov[4 * v + 3]);
            }
            __syncwarp();
          }
          if (!ok) break;
          if (put && copy == 0 && !whole)
            *reinterpret_cast<float2 *>(p.part_ml + row * 2) = make_float2(M, L);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(o_free);
        }
      }
      walk_next(w, p, sseq);
    }
    if (!ok && lane == 0) flag_status(p.status, kStatusTimeout);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWS) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
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

// The dynamic shared memory limit is a property of the kernel on one device.
template <int HD, int RHO>
static cudaError_t configure_attn8() {
  static std::mutex mutex;
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mutex);
  if (dev < 64 && done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(attn8_kernel<HD, RHO>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(A8Cfg<HD>::SMEM));
  if (e == cudaSuccess && dev < 64) done[dev] = true;
  return e;
}

template <int HD, int RHO>
static cudaError_t launch_attn8(const Attn8Params &p, cudaStream_t s) {
  const int R = (p.Hq / p.Hkv) * p.m;
  cudaError_t e = configure_attn8<HD, RHO>();
  if (e != cudaSuccess) return e;
  e = launch_pdl(attn8_kernel<HD, RHO>, dim3(p.grid), dim3(kA8Threads), A8Cfg<HD>::SMEM, s, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn8_merge_kernel<HD>, dim3(p.nb * p.Hkv, (R + kMerge8Warps - 1) / kMerge8Warps),
                    dim3(kMerge8Warps * 32), 0, s, p);
}

cudaError_t launch_attention8(const Attn8Params &p, cudaStream_t s) {
  const int R = (p.Hq / p.Hkv) * p.m;
  if (p.Hq % p.Hkv != 0 || R > 128) return cudaErrorInvalidValue;
  // copies of the query rows that fill the MMA's 128
  if (p.hd == 128)
    return R > 64 ? launch_attn8<128, 1>(p, s) : R > 32 ? launch_attn8<128, 2>(p, s) : launch_attn8<128, 4>(p, s);
  return R > 64 ? launch_attn8<64, 1>(p, s) : R > 32 ? launch_attn8<64, 2>(p, s) : launch_attn8<64, 4>(p, s);
}

}  // namespace df
