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

// The T units are split over G CTAs: the first T % G take one more than the others (T is below
// 2^25: a handle's caches hold fewer than 2^31 rows).
__device__ __forceinline__ int cta_start(int T, int G, int c) { return c * (T / G) + min(c, T % G); }
__device__ __forceinline__ int cta_of(int T, int G, int u) {
  const int q = T / G, big = (T % G) * (q + 1);
  return u < big ? u / (q + 1) : T % G + (u - big) / q;
}

// Units of the sequences before i (`before`) and of all of them, times Hkv. Warp-collective.
__device__ __forceinline__ int total_units(const Attn8Params &p, int i, int lane, int *before) {
  int t = 0, b = 0;
#pragma unroll 1
  for (int s = lane; s < p.nb; s += 32) {
    const int u = seq8(p, s).units;
    t += u;
    b += s < i ? u : 0;
  }
  *before = __reduce_add_sync(0xffffffffu, b) * p.Hkv;
  return __reduce_add_sync(0xffffffffu, t) * p.Hkv;
}

// Where a CTA's range begins (pair i * Hkv + g, unit inside it) and its number of units.
// Warp-collective.
__device__ void find_range(const Attn8Params &p, int cta, int lane, int *out) {
  int base;
  const int T = total_units(p, 0, lane, &base);
  const int Ge = min(T, p.grid);
  int count = 0, pair = 0, unit = 0;
  if (cta < Ge) {
    const int u0 = cta_start(T, Ge, cta);
    count = cta_start(T, Ge, cta + 1) - u0;
#pragma unroll 1
    for (int b = 0; b < p.nb; b += 32) {
      const int U = b + lane < p.nb ? seq8(p, b + lane).units : 0;
      int v = p.Hkv * U;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, base + v > u0);
      if (hit) {
        const int l = __ffs(hit) - 1;
        const int Ul = __shfl_sync(0xffffffffu, U, l);
        const int off = u0 - (base + __shfl_sync(0xffffffffu, v, l) - p.Hkv * Ul);
        pair = (b + l) * p.Hkv + off / Ul;
        unit = off % Ul;
        break;
      }
      base += __shfl_sync(0xffffffffu, v, 31);
    }
  }
  if (lane == 0) {
    out[0] = pair;
    out[1] = unit;
    out[2] = count;
  }
}

}  // namespace

// ---------------------------------------------------------------- tensor-core kernel

// RHO copies of the query rows fill the 128 lanes of the MMA (rows padded to 128 / RHO); each copy
// takes units of its own, so that a softmax thread works on all 64 keys of a unit and every SM
// quarter's warps share the work of few rows. PV leaves the other copies' lanes of O as they are.
//   RHO = 4   groups 0 .. 3 of one warp: the lanes of copy g; a pair of units (see below) goes to
//             the groups 0, 1 or 2, 3 in turn
//   RHO = 2   groups 0, 1 of two warps
//   RHO = 1   groups 0, 1 of four warps, with an O each (there is no second copy), for which one
//             pair of S and of P buffers has to do
template <int HD, int RHO>
struct A8Cfg {
  static constexpr int ROWS = 128 / RHO;             // padded query rows
  static constexpr int NG = RHO == 4 ? 4 : 2;        // softmax groups
  static constexpr int NO = RHO == 1 ? 2 : 1;        // O accumulators
  static constexpr int WPG = RHO == 4 ? 1 : RHO == 2 ? 2 : 4;  // warps of a group
  static constexpr int DEEP = RHO == 1 ? 1 : 2;      // buffers of a pair's S and P
  static constexpr int ATOMS = HD / 64;              // 128-byte swizzle atoms across hd (f16)
  static constexpr int UNIT8 = kUnit * HD;           // bytes of a unit's keys (or values) in the cache
  static constexpr int PAIR8 = 2 * UNIT8;
  // ring of pairs of units in 8 bits, keys then values, as much as shared memory holds
  static constexpr int NS = (RHO == 1 ? 3 : 4) * (128 / HD);
  static constexpr int ATOM16 = kUnit * 128;
  static constexpr int TILE16 = ATOMS * ATOM16;      // a unit's values in f16
  static constexpr int QPITCH = HD * 2 + 16;         // bytes of a query row (bf16): rows apart by 16 bytes mod 128
  static constexpr int STAGE = RHO == 1 ? 0 : 128 * 16;  // floats of the exchange of O between copies
  static constexpr int OFF_8 = 4 * TILE16;           // two pairs of units' V in f16, then the ring
  static constexpr int OFF_Q = OFF_8 + NS * 2 * PAIR8;
  static constexpr int OFF_STG = OFF_Q + ROWS * QPITCH;
  static constexpr int OFF_ML = OFF_STG + STAGE * 4;      // [NO][128 lanes] (maximum, sum)
  static constexpr int OFF_SC = OFF_ML + NO * 128 * 8;    // [2 chunks][32 units] scales
  static constexpr int OFF_BAR = OFF_SC + 64 * 16;
  static constexpr int OFF_SEQ = OFF_BAR + 512;           // [kSeqCache] (rows, context)
  static constexpr size_t SMEM = 1024 + OFF_SEQ + 128 * 8;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t S_COL = 0;                     // S of pair pj in buffer pj % DEEP: 64 columns a unit
  static constexpr uint32_t O_COL = DEEP * 128;            // O: hd columns each
  static constexpr uint32_t Q_COL = O_COL + NO * HD;       // queries, two e4m3 terms: hd / 4 columns each
  static constexpr uint32_t P_COL = Q_COL + HD / 2;        // P: 32 columns a unit; a buffer pj % 2 for the
                                                           // pair (its units lie in different lanes), or,
                                                           // RHO = 1, one for either unit
  static_assert(P_COL + 64 <= TMEM_COLS, "tensor memory");
  // Warps: producer, S issuer, PV issuer, one that only helps at the start, softmax (warp w reads
  // TMEM lanes of quarter w % 4), then the converters of V.
  static constexpr int W_CONV = 4 + 4 * NO;
  static constexpr int THREADS = (W_CONV + 4) * 32;
};
constexpr int kSeqCache = 128;
constexpr int kDrainSpin = 1 << 22;
// P is 2^(x - m_run + kPBase), m_run the maximum at the last rescale: O is rescaled only when the
// maximum has grown by more than 2^kRescale, so P stays at most 2^15 in f16, and what is 2^-21 of
// the largest still has all 11 bits (2^-31 one bit).
constexpr float kPBase = 7.f, kRescale = 8.f;

// A segment's units are taken in pairs: one S product of 128 keys, then a softmax for each unit by a
// group of its own, then both PV. What bounds the kernel are the steps from one role to the next
// (with every copy, product and exponential left out it still took 0.7 of its time, when each
// warp went through every unit), so they are paid for two units at once, and a softmax warp goes
// through every second or fourth unit only. Half a pair at the end of a segment of an odd number of
// units is signalled by its group without work.
constexpr int kWProd = 0, kWS = 1, kWPV = 2, kWAid = 3, kWSoft = 4, kNumConv = 4;

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A unit inside a CTA's range: sequence i, kv head g, unit of `units`.
struct Pos8 {
  int i, g, unit, units, n, ctx;
};
__device__ __noinline__ int2 seq_far(const Attn8Params &p, int i) {
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
// To the pair after this one.
__device__ __forceinline__ void pos_next_pair(Pos8 &w, const Attn8Params &p, const int2 *sseq) {
  w.unit = 0;
  if (++w.g == p.Hkv) {
    w.g = 0;
    ++w.i;
    pos_seq(w, p, sseq);
  }
}

// 8 e4m3 values to f16 (exact).
__device__ __forceinline__ uint4 widen8(uint2 u) {
  uint4 h;
  asm("{\n\t.reg .b16 a, b, c, d;\n\t"
      "mov.b32 {a, b}, %4;\n\t"
      "mov.b32 {c, d}, %5;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t"
      "cvt.rn.f16x2.e4m3x2 %2, c;\n\t"
      "cvt.rn.f16x2.e4m3x2 %3, d;\n\t}"
      : "=r"(h.x), "=r"(h.y), "=r"(h.z), "=r"(h.w)
      : "r"(u.x), "r"(u.y));
  return h;
}

// One of the warp's threads, the same one every time; the branch on it leaves the code around it
// warp-uniform.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
  return ok != 0;
}

template <int HD, int RHO>
__global__ void __launch_bounds__(A8Cfg<HD, RHO>::THREADS, 1) attn8_kernel(const __grid_constant__ Attn8Params p) {
  using C = A8Cfg<HD, RHO>;
  constexpr int ROWS = C::ROWS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint8_t *sV16 = smem, *s8 = smem + C::OFF_8, *sQ = smem + C::OFF_Q;
  float2 *ml = reinterpret_cast<float2 *>(smem + C::OFF_ML);
  float4 *sscale = reinterpret_cast<float4 *>(smem + C::OFF_SC);
  uint64_t *kv8_full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
  uint64_t *kv8_empty = kv8_full + C::NS;
  uint64_t *v16_full = kv8_empty + C::NS;   // [2] V of pair pj in f16, buffer pj % 2
  uint64_t *p_full = v16_full + 2;          // [2] P of pair pj
  uint64_t *pv_done = p_full + 2;           // [2] PV of pair pj complete: P and V16 have been read
  uint64_t *s_full = pv_done + 2;           // [2] S of pair pj complete, buffer pj % DEEP
  uint64_t *s_empty = s_full + 2;           // [2] and read by both groups
  uint64_t *sc_full = s_empty + 2;          // [2] scales of 32 units, chunk c in buffer c % 2
  uint64_t *sc_empty = sc_full + 2;         // [2]
  uint64_t *half_bar = sc_empty + 2;        // [2] four softmax warps among themselves
  uint64_t *mma_done = half_bar + 2;        // [2]
  uint64_t *q8_full = mma_done + 2;         // a segment's query rows have landed
  uint64_t *q8_empty = q8_full + 1;
  uint64_t *q_full = q8_empty + 1;          // and are in tensor memory
  uint64_t *q_empty = q_full + 1;
  uint64_t *seg_bar = q_empty + 1;          // every softmax warp: (maximum, sum) of a segment written
  uint64_t *o_free = seg_bar + 1;           // O and ml read
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(o_free + 1);
  int *sched = reinterpret_cast<int *>(tmem_slot + 1);
  static_assert((2 * C::NS + 18 + 6) * 8 + 16 <= 512, "barrier region overflows");
  int2 *sseq = reinterpret_cast<int2 *>(smem + C::OFF_SEQ);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv;
  const int R = G * p.m;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(&kv8_full[s], 1);
      mbar_init(&kv8_empty[s], kNumConv + 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&v16_full[b], kNumConv);
      mbar_init(&p_full[b], 2 * C::WPG);
      mbar_init(&pv_done[b], 1);
      mbar_init(&s_full[b], 1);
      mbar_init(&s_empty[b], 2 * C::WPG);
      mbar_init(&sc_full[b], 1);
      mbar_init(&sc_empty[b], 4 * C::NO);
      mbar_init(&half_bar[b], 4);
      mbar_init(&mma_done[b], 1);
    }
    mbar_init(q8_full, 1);
    mbar_init(q8_empty, 4 * C::NO);
    mbar_init(q_full, 4);
    mbar_init(q_empty, 1);
    mbar_init(seg_bar, 4 * C::NO);
    mbar_init(o_free, 4 * C::NO);
    fence_mbar_init();
  }
  if (warp == kWS) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch();
  if (warp == kWProd) {
    find_range(p, blockIdx.x, lane, sched);
  } else if (warp == kWAid) {
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
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const int nunits = __shfl_sync(0xffffffffu, sched[2], 0);
  Pos8 w;
  w.i = sched[0] / p.Hkv;
  w.g = sched[0] % p.Hkv;
  w.unit = sched[1];
  if (nunits > 0) pos_seq(w, p, sseq);

  // Every role goes through the CTA's segments: `cnt` units from unit j0 of the CTA on, in pairs pj
  // of units u, u + 1 of the segment. A wait that runs out ends the role (ok = false).
  if (nunits == 0) {
    // nothing to do
  } else if (warp == kWProd) {
    // ---------------- producer: a unit's keys and values are contiguous 64 * hd bytes each (the keys
    // arrive swizzled, as the tensor cores read them), a query row hd bf16. Lane l looks up the block of unit 32 c + l of the CTA's range two chunks c
    // ahead and its scales one chunk ahead, so the copies wait for neither.
    const uint64_t pol = policy_evict_first();
    bool ok = !p.stall;
    int pairs = 0, segs = 0;
    Pos8 a = w;
    int x = lane;
    a.unit += lane;
    auto look_up = [&]() {
      if (x >= nunits) return 0;
      while (a.unit >= a.units) {
        const int over = a.unit - a.units;
        pos_next_pair(a, p, sseq);
        a.unit = over;
      }
      const int b = static_cast<int>(block_of(p, a.i, a.g, a.unit));
      a.unit += 32;
      return b;
    };
    int blk = look_up();
    x += 32;
    int blk1 = look_up();
    float ks = lane < nunits ? p.ks[blk] : 0.f, vs = lane < nunits ? p.vs[blk] : 0.f;
    int cnt_left = 0, slot = 0, st = 0, ph = 0;
    bool published = false;
#pragma unroll 1
    for (int j = 0; j < nunits && ok; ++j) {
      const int k = j & 31, c = j >> 5;
      if (cnt_left == 0) {  // a segment begins: its query rows
        if (j > 0) pos_next_pair(w, p, sseq);
        cnt_left = min(w.units - w.unit, nunits - j);
        ok = segs == 0 || mbar_wait_warp(q8_empty, (segs - 1) & 1, p.max_spin);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(q8_full, w.n * G * HD * 2);
        __syncwarp();
#pragma unroll 1
        for (int r = lane; r < w.n * G; r += 32)
          bulk_load(sQ + r * C::QPITCH,
                    p.q + ((static_cast<size_t>(w.i) * p.m + r / G) * p.Hq + w.g * G + r % G) * HD, HD * 2, q8_full,
                    pol);
        ++segs;
        slot = 0;
      }
      --cnt_left;
      const long long b = __shfl_sync(0xffffffffu, blk, k);
      if (slot == 0) ok = pairs < C::NS || mbar_wait_warp(&kv8_empty[st], ph ^ 1, p.max_spin);
      if (!ok) break;
      if (elect_one()) {
        uint8_t *dst = s8 + st * 2 * C::PAIR8;
        if (slot == 0) mbar_arrive_expect_tx(&kv8_full[st], (cnt_left > 0 ? 2 : 1) * C::PAIR8);
        tma_load_2d(dst + slot * C::UNIT8, &p.tmK, &kv8_full[st], 0, static_cast<int>(b) * kUnit, pol);
        bulk_load(dst + C::PAIR8 + slot * C::UNIT8, p.v8 + b * C::UNIT8, C::UNIT8, &kv8_full[st], pol);
      }
      __syncwarp();
      if (slot == 0) ++pairs;
      if (slot == 1 || cnt_left == 0) {  // the pair is complete
        slot = 0;
        if (++st == C::NS) {
          st = 0;
          ph ^= 1;
        }
      } else {
        slot = 1;
      }
      // The chunk's scales, after its first copies are under way, and before any wait for a unit
      // of the chunk: a copy waits for the pair NS >= 3 before its own, the next segment's queries
      // for the units of the segment before last.
      published = published && k != 0;
      if (!published && (k == 2 || j == nunits - 1 || cnt_left == 0)) {
        published = true;
        ok = c < 2 || mbar_wait_warp(&sc_empty[c & 1], ((c >> 1) - 1) & 1, p.max_spin);
        if (!ok) break;
        const bool zero = vs == 0.f;  // a block of zeros: P must not see the scale
        sscale[(c & 1) * 32 + lane] = make_float4(ks, zero ? 0.f : log2f(vs), zero ? 1.f : 1.f / vs, zero ? 0.f : 1.f);
        __syncwarp();
        mbar_arrive_if(&sc_full[c & 1], lane == 0);
      }
      if (k == 31) {
        blk = blk1;
        x += 32;
        const bool more = x - 32 < nunits;
        ks = more ? p.ks[blk] : 0.f;
        vs = more ? p.vs[blk] : 0.f;
        blk1 = look_up();
      }
    }
    if (!ok && !p.stall && lane == 0) flag_status(p.status, kStatusTimeout);
    // every issued copy must land before the CTA may exit (bounded)
#pragma unroll 1
    for (int x = max(0, pairs - C::NS); x < pairs; ++x)
      mbar_wait_warp(&kv8_full[x % C::NS], (x / C::NS) & 1, kDrainSpin);
    if (segs > 0) mbar_wait_warp(q8_full, (segs - 1) & 1, kDrainSpin);
  } else if (warp == kWS) {
    // ---------------- S issuer: S(j) = Q K(j)^T straight from the 8-bit keys, the queries' two e4m3
    // terms one after the other from tensor memory
    constexpr uint32_t id_s = idesc_f32_format0(128, kUnit);
    const uint64_t kd0 = HD == 128 ? sw128_kmajor_desc(smem_u32(s8)) : sw64_kmajor_desc(smem_u32(s8));
    constexpr uint32_t id_s2 = idesc_f32_format0(128, 2 * kUnit);
    int st = 0, ph = 0, pj = 0;
    bool ok = true;
#pragma unroll 1
    for (int j0 = 0, seg = 0; j0 < nunits && ok; ++seg) {
      const int cnt = min(w.units - w.unit, nunits - j0);
      ok = mbar_wait_warp(q_full, seg & 1, p.max_spin);
#pragma unroll 1
      for (int u = 0; u < cnt && ok; u += 2, ++pj) {
        ok = mbar_wait_warp(&kv8_full[st], ph, p.max_spin);
        const int b = pj % C::DEEP;
        ok = ok && (pj < C::DEEP || mbar_wait_warp(&s_empty[b], (pj / C::DEEP - 1) & 1, p.max_spin));
        if (!ok) break;
        tc_fence_after();
        const uint64_t kd = kd0 + static_cast<uint64_t>((st * 2 * C::PAIR8) >> 4);
        const uint32_t id = u + 1 < cnt ? id_s2 : id_s;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 2 * HD / 32; ++kk)
            tc_mma_e4m3_tmem_a(tmem + C::S_COL + b * 128, tmem + C::Q_COL + kk * 8,
                               kd + static_cast<uint64_t>((kk % (HD / 32)) * 32 >> 4), id, kk > 0 ? 1u : 0u);
          tc_commit(&s_full[b]);
          if (u + 2 >= cnt) tc_commit(q_empty);
        }
        __syncwarp();
        if (++st == C::NS) {
          st = 0;
          ph ^= 1;
        }
      }
      j0 += cnt;
      if (j0 < nunits) pos_next_pair(w, p, sseq);
    }
    if (!ok && lane == 0) flag_status(p.status, kStatusTimeout);
    // every issued MMA must complete before TMEM is freed (bounded)
    if (elect_one()) tc_commit(&mma_done[0]);
    __syncwarp();
    mbar_wait_warp(&mma_done[0], 0, kDrainSpin);
  } else if (warp == kWPV) {
    // ---------------- PV issuer: O += P V for both units of a pair; a segment's first unit of each
    // group starts the accumulator, after the previous segment's O was read
    constexpr uint32_t id_pv = idesc_f32_format0(128, HD) | kIdescBMajorMN;
    const uint64_t vd0 = sw128_mnmajor_desc(smem_u32(sV16), C::ATOM16);
    bool ok = true;
    int pj = 0;
#pragma unroll 1
    for (int j0 = 0, seg = 0; j0 < nunits && ok; ++seg) {
      const int cnt = min(w.units - w.unit, nunits - j0);
      if (seg > 0) ok = mbar_wait_warp(o_free, (seg - 1) & 1, p.max_spin);
#pragma unroll 1
      for (int u = 0; u < cnt && ok; u += 2, ++pj) {
        const int b = pj & 1;
        ok = mbar_wait_warp(&v16_full[b], (pj >> 1) & 1, p.max_spin);
        ok = ok && mbar_wait_warp(&p_full[b], (pj >> 1) & 1, p.max_spin);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t add = u >= C::NG ? 1u : 0u;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (u + x >= cnt) break;
            const uint64_t vd = vd0 + static_cast<uint64_t>(((b * 2 + x) * C::TILE16) >> 4);
            const int g = RHO == 4 ? 2 * b + x : x;  // the unit's group
            uint32_t off[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) off[y] = RHO == 1 || y * 32 / ROWS == g ? 0u : 0xFFFFFFFFu;
#pragma unroll
            for (int kk = 0; kk < kUnit / 16; ++kk) {
              const uint64_t d = vd + static_cast<uint64_t>((kk * 16 * 128) >> 4);
              if (RHO == 1)
                tc_mma_bf16_tmem_a(tmem + C::O_COL + x * HD, tmem + C::P_COL + x * 32 + kk * 8, d, id_pv,
                                   kk > 0 ? 1u : add);
              else
                tc_mma_bf16_tmem_a_lanes(tmem + C::O_COL, tmem + C::P_COL + b * 32 + kk * 8, d, id_pv, off,
                                         kk > 0 ? 1u : add);
            }
          }
          tc_commit(&pv_done[b]);
        }
        __syncwarp();
      }
      j0 += cnt;
      if (j0 < nunits) pos_next_pair(w, p, sseq);
    }
    if (!ok && lane == 0) flag_status(p.status, kStatusTimeout);
    if (elect_one()) tc_commit(&mma_done[1]);
    __syncwarp();
    mbar_wait_warp(&mma_done[1], 0, kDrainSpin);
  } else if (warp >= C::W_CONV) {
    // ---------------- converters: V from e4m3 to f16, in the layout of a 128-byte-swizzled copy (rows
    // of 64 values, 16-byte chunk c of row r at c ^ (r & 7))
    constexpr int CPR = HD / 8;                        // 8-value chunks of a row: 8 bytes to 16
    constexpr int RPI = kNumConv * 32 / CPR;           // rows per iteration: 8 or 16
    constexpr int PER = kUnit / RPI;                   // chunks per thread
    static_assert(RPI % 8 == 0, "a thread's chunks all lie at the same place of their rows");
    const int t = (warp - C::W_CONV) * 32 + lane;
    const int cc = t % CPR, r0 = t / CPR;
    uint8_t *out = sV16 + (cc >> 3) * C::ATOM16 + r0 * 128 + (((cc & 7) ^ (r0 & 7)) << 4);
    const uint8_t *src0 = s8 + C::PAIR8 + t * 8;
    bool ok = true;
    int st = 0, ph = 0, pj = 0;
#pragma unroll 1
    for (int j0 = 0; j0 < nunits && ok;) {
      const int cnt = min(w.units - w.unit, nunits - j0);
      int keys = w.ctx + w.n - w.unit * kUnit;     // rows of the unit that hold keys
#pragma unroll 1
      for (int x = 0; x < cnt; ++x, keys -= kUnit) {
        const int b = pj & 1, slot = x & 1;
        if (slot == 0) {
          ok = mbar_wait_warp(&kv8_full[st], ph, p.max_spin);
          ok = ok && (pj < 2 || mbar_wait_warp(&pv_done[b], ((pj >> 1) - 1) & 1, p.max_spin));
          if (!ok) break;
        }
        const uint8_t *src = src0 + st * 2 * C::PAIR8 + slot * C::UNIT8;
        uint8_t *dst = out + (b * 2 + slot) * C::TILE16;
        if (keys < kUnit) {
          // rows beyond the last key may hold anything (even NaN); P is 0 there
#pragma unroll 2
          for (int e = 0; e < PER; ++e) {
            uint4 h = make_uint4(0, 0, 0, 0);
            if (r0 + e * RPI < keys) h = widen8(*reinterpret_cast<const uint2 *>(src + e * RPI * HD));
            *reinterpret_cast<uint4 *>(dst + e * RPI * 128) = h;
          }
        } else {
          uint2 u[PER];
#pragma unroll
          for (int e = 0; e < PER; ++e) u[e] = *reinterpret_cast<const uint2 *>(src + e * RPI * HD);
#pragma unroll
          for (int e = 0; e < PER; ++e) *reinterpret_cast<uint4 *>(dst + e * RPI * 128) = widen8(u[e]);
        }
        if (slot == 1 || x == cnt - 1) {  // the pair is complete
          fence_proxy_async_smem();
          __syncwarp();
          mbar_arrive_if(&v16_full[b], lane == 0);
          mbar_arrive_if(&kv8_empty[st], lane == 0);
          ++pj;
          if (++st == C::NS) {
            st = 0;
            ph ^= 1;
          }
        }
      }
      j0 += cnt;
      if (j0 < nunits) pos_next_pair(w, p, sseq);
    }
    if (!ok && lane == 0) flag_status(p.status, kStatusTimeout);
  } else if (warp >= kWSoft) {
    // ---------------- softmax: thread = TMEM lane; lane l holds query row l % ROWS, copy l / ROWS
    const int half = (warp - kWSoft) >> 2;   // RHO = 1: the group, and its O
    const int tl = (warp & 3) * 32 + lane;
    const int r = tl % ROWS, copy = tl / ROWS;
    const int grp = RHO == 1 ? half : copy, slot = grp & 1;
    const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t o_mine = trow + C::O_COL + (RHO == 1 ? half * HD : 0);
    const int jq = r / G;               // row r: query row jq of query head g * G + r % G
    const float sl2 = rsqrtf(static_cast<float>(HD)) * 1.4426950408889634f;
    uint32_t half_phase = 0;
    // Barrier of four warps, bounded like every other wait.
    auto half_sync = [&]() {
      __syncwarp();
      mbar_arrive_if(&half_bar[half], lane == 0);
      const bool done = mbar_wait_warp(&half_bar[half], half_phase, p.max_spin);
      half_phase ^= 1;
      return done;
    };
    // The query row of segment `seg` (n rows a sequence), scaled by a power of two so that its
    // largest value lies in [2^7, 2^8), to tensor memory as the sum of two e4m3 terms: 4 bits each
    // hold bf16's 8, exactly down to 2^-10 of the largest value, below that to 2^-18 of it.
    // Returns the factor that takes S to log2 units, 1/sqrt(hd) included; < 0 on a wait run out.
    auto load_q = [&](int seg, int n) {
      bool ok = mbar_wait_warp(q8_full, seg & 1, p.max_spin);
      if (half == 0 && seg > 0) ok = ok && mbar_wait_warp(q_empty, (seg - 1) & 1, p.max_spin);
      if (!ok) return -1.f;
      const uint4 *src = reinterpret_cast<const uint4 *>(sQ + r * C::QPITCH);
      const bool have = r < n * G;
      float am = 0.f;
#pragma unroll 4
      for (int e = 0; e < HD / 8; ++e) {
        const uint4 u = have ? src[e] : make_uint4(0, 0, 0, 0);
        const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int f = 0; f < 4; ++f)
          am = fmaxf(am, fmaxf(fabsf(__uint_as_float(x[f] << 16)), fabsf(__uint_as_float(x[f] & 0xFFFF0000u))));
      }
      int ex = static_cast<int>(__float_as_uint(am) >> 23) - 127;   // -127: zero or subnormal, 128: infinite
      const bool inf = ex == 128;          // the row's outputs are NaN
      ex = max(min(ex, 127), -100);
      if (half == 0) {
        const float mul = inf ? __int_as_float(0x7FC00000) : __uint_as_float(static_cast<uint32_t>(7 - ex + 127) << 23);
        tc_fence_after();
#pragma unroll 1
        for (int part = 0; part < HD / 32; ++part) {
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint4 u = have ? src[part * 4 + e] : make_uint4(0, 0, 0, 0);
            const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int f = 0; f < 4; ++f) {
              const float2 y = make_float2(__uint_as_float(x[f] << 16) * mul, __uint_as_float(x[f] & 0xFFFF0000u) * mul);
              const __nv_fp8x2_storage_t a = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
              const __half2_raw ar = __nv_cvt_fp8x2_to_halfraw2(a, __NV_E4M3);
              const float2 af = __half22float2(*reinterpret_cast<const __half2 *>(&ar));
              const __nv_fp8x2_storage_t b =
                  __nv_cvt_float2_to_fp8x2(make_float2(y.x - af.x, y.y - af.y), __NV_SATFINITE, __NV_E4M3);
              const int d = 2 * e + f / 2;
              hi[d] = f % 2 ? hi[d] | (static_cast<uint32_t>(a) << 16) : a;
              lo[d] = f % 2 ? lo[d] | (static_cast<uint32_t>(b) << 16) : b;
            }
          }
          tmem_st8_raw(trow + C::Q_COL + part * 8, hi);
          tmem_st8_raw(trow + C::Q_COL + HD / 4 + part * 8, lo);
        }
        tmem_wait_st();
        tc_fence_before();
      }
      __syncwarp();
      mbar_arrive_if(q_full, lane == 0 && half == 0);
      mbar_arrive_if(q8_empty, lane == 0);
      return sl2 * __uint_as_float(static_cast<uint32_t>(ex - 7 + 127) << 23);
    };
    float qfac = 0.f;
    bool ok = true;
    int chunk = -1;                      // chunk of 32 units whose scales this warp may read
    int pj = 0, st = 0;                  // pair of units, and its stage of the ring
    // Segment by segment: its units, then the queries of the next one (whose S can start), then the
    // output of this one. The round before the first segment has the queries alone.
#pragma unroll 1
    for (int j0 = 0, seg = -1;; ++seg) {
      const int cnt = seg < 0 ? 0 : min(w.units - w.unit, nunits - j0);
      const int lim = p.causal ? min(w.ctx + jq + 1, w.ctx + w.n) : w.ctx + w.n;
      // keys from the segment's first unit on that every row sees
      const int all = (p.causal ? w.ctx + 1 : w.ctx + w.n) - w.unit * kUnit;
      float m_run = kNoMax, l_run = 0.f;
#pragma unroll 1
      for (int u = slot; u < ((cnt + 1) & ~1) + slot; u += 2, ++pj) {
        const int j = min(j0 + u, j0 + cnt - 1);
        if (chunk < (j >> 5)) {          // the next chunk: give the one before back
          __syncwarp();
          if (chunk >= 0) mbar_arrive_if(&sc_empty[chunk & 1], lane == 0);
          ++chunk;
          ok = mbar_wait_warp(&sc_full[chunk & 1], (chunk >> 1) & 1, p.max_spin);
          if (!ok) break;
        }
        const int st_now = st;
        st = st + 1 == C::NS ? 0 : st + 1;
        if (RHO == 4 && (pj & 1) != (grp >> 1)) continue;  // the other two groups' pair
        const float4 sc = sscale[(chunk & 1) * 32 + (j & 31)];  // K scale, log2 V, 1 / V, 0 for zeros
        const int sb = pj % C::DEEP, pb = pj & 1;
        ok = mbar_wait_warp(&s_full[sb], (pj / C::DEEP) & 1, p.max_spin);
        if (!ok) break;
        tc_fence_after();
        float sv[kUnit];
        tmem_ld64(trow + C::S_COL + sb * 128 + slot * kUnit, sv);
        tc_fence_before();
        __syncwarp();
        mbar_arrive_if(&s_empty[sb], lane == 0);
        mbar_arrive_if(&kv8_empty[st_now], slot == 0 && r == 0);  // S complete: the keys have been read
        // this group's P buffer is free once the PV that read it has completed
        const int pp = RHO == 1 ? pj - 1 : pj - 2;
        bool freed = pp < 0;
        if (u >= cnt) {                  // half a pair
          ok = freed || mbar_wait_warp(&pv_done[pp & 1], (pp >> 1) & 1, p.max_spin);
          if (!ok) break;
          mbar_arrive_if(&p_full[pb], lane == 0);
          continue;
        }
        if (all - kUnit * u < kUnit) {   // some row does not see the whole unit
          const int nv = lim - (w.unit + u) * kUnit;  // keys this row sees
#pragma unroll
          for (int c = 0; c < kUnit; ++c) sv[c] = c < nv ? sv[c] : -INFINITY;
        }
        const float c1 = fmaxf(qfac * sc.x, 1e-37f);
        float mx[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
        for (int c = 4; c + 8 <= kUnit; c += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], sv[c + 2 * e], sv[c + 2 * e + 1]);
        mx[3] = max3(max3(mx[3], sv[kUnit - 4], sv[kUnit - 3]), sv[kUnit - 2], sv[kUnit - 1]);
        const float m_new = fmaf(fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]), c1, sc.y);
        const bool need = m_new - m_run > kRescale;
        float alpha = 1.f;
        if (need) {
          alpha = ex2f(m_run - m_new);
          m_run = m_new;
          l_run *= alpha;
        }
        if (u >= C::NG && __any_sync(0xffffffffu, need && r < R)) {
          // O *= alpha, once this group's last PV has completed: the pair NG / 2 before
          const int pl = pj - C::NG / 2;
          ok = mbar_wait_warp(&pv_done[pl & 1], (pl >> 1) & 1, p.max_spin);
          if (!ok) break;
          tc_fence_after();
          freed = pl >= pp;
#pragma unroll 1
          for (int cc = 0; cc < HD / 16; ++cc) {
            float ov[16];
            tmem_ld16(o_mine + cc * 16, ov);
            uint32_t x[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) x[c] = __float_as_uint(ov[c] * alpha);
            tmem_st16_raw(o_mine + cc * 16, x);
          }
        }
        const float c2 = sc.y - m_run + kPBase;
        uint32_t pk[kUnit / 2];
        float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < kUnit; c += 2) {
          const float2 x = fma2(make_float2(sv[c], sv[c + 1]), make_float2(c1, c1), make_float2(c2, c2));
          const float2 e = make_float2(ex2f(x.x), ex2f(x.y));
          ls[(c >> 1) & 1] = add2(ls[(c >> 1) & 1], e);
          const __half2 y = __floats2half2_rn(e.x, e.y);
          pk[c / 2] = *reinterpret_cast<const uint32_t *>(&y);
        }
        const float2 lt = add2(ls[0], ls[1]);
        l_run = fmaf(lt.x + lt.y, sc.z, l_run);
        if (sc.w == 0.f) {
#pragma unroll
          for (int c = 0; c < kUnit / 2; ++c) pk[c] = 0u;
        }
        if (!freed) {
          ok = mbar_wait_warp(&pv_done[pp & 1], (pp >> 1) & 1, p.max_spin);
          if (!ok) break;
          tc_fence_after();
        }
        tmem_st32_raw(trow + C::P_COL + (RHO == 1 ? slot : pb) * 32, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        mbar_arrive_if(&p_full[pb], lane == 0);
      }
      if (!ok) break;
      const int i = w.i, g = w.g, n = w.n;
      const bool whole = w.unit == 0 && cnt == w.units;
      j0 += cnt;
      const bool more = j0 < nunits;
      if (more) {
        if (seg >= 0) pos_next_pair(w, p, sseq);
        qfac = load_q(seg + 1, w.n);
        ok = qfac >= 0.f;
      }
      if (seg < 0 && ok) continue;
      // every PV of the segment has completed
      ok = ok && mbar_wait_warp(&pv_done[(pj - 1) & 1], ((pj - 1) >> 1) & 1, p.max_spin);
      // the (maximum, sum) slots are free once the previous segment's were read
      ok = ok && (seg == 0 || mbar_wait_warp(o_free, (seg - 1) & 1, p.max_spin));
      if (!ok) break;
      ml[half * 128 + tl] = make_float2(m_run, l_run);
      tc_fence_before();
      __syncwarp();
      mbar_arrive_if(seg_bar, lane == 0);
      ok = mbar_wait_warp(seg_bar, seg & 1, p.max_spin);
      if (!ok) break;
      tc_fence_after();
      // the sets that make up a row: a copy's lanes, or RHO = 1 the two O of its lane
      float M = kNoMax, L = 0.f;
#pragma unroll
      for (int c = 0; c < C::NG; ++c) M = fmaxf(M, ml[c * ROWS + r].x);
#pragma unroll
      for (int c = 0; c < C::NG; ++c) L += ml[c * ROWS + r].y * ex2f(ml[c * ROWS + r].x - M);
      const size_t row0 = (static_cast<size_t>(i * p.Hkv + g) + blockIdx.x) * R;   // partial rows
      const float inv = whole ? 1.0f / L : 1.0f;
      const int live = n * G;            // rows that are computed
      if (half == 0 && copy == 0 && r < live && !whole)
        *reinterpret_cast<float2 *>(p.part_ml + (row0 + r) * 2) = make_float2(M, L);
      uint16_t *o = p.o + (static_cast<size_t>(i) * p.m * p.Hq + g * G) * HD;
      if constexpr (RHO == 1) {
        // each group takes half of the columns of both O
        const bool has1 = cnt > 1;
        const float a0 = ex2f(ml[tl].x - M) * inv, a1 = ex2f(ml[128 + tl].x - M) * inv;
#pragma unroll 1
        for (int c0 = half * (HD / 2); c0 < (half + 1) * (HD / 2); c0 += 16) {
          float ov[16], o1[16];
          tmem_ld16(trow + C::O_COL + c0, ov);
          tmem_ld16(trow + C::O_COL + HD + c0, o1);
#pragma unroll
          for (int c = 0; c < 16; ++c) ov[c] = ov[c] * a0 + (has1 ? o1[c] * a1 : 0.f);
          if (r < live) {
            if (whole) {
              uint16_t *dst = o + (static_cast<size_t>(jq) * p.Hq + r % G) * HD + c0;
#pragma unroll
              for (int v = 0; v < 2; ++v)
                reinterpret_cast<uint4 *>(dst)[v] =
                    make_uint4(pack_bf16x2(ov[8 * v], ov[8 * v + 1]), pack_bf16x2(ov[8 * v + 2], ov[8 * v + 3]),
                               pack_bf16x2(ov[8 * v + 4], ov[8 * v + 5]), pack_bf16x2(ov[8 * v + 6], ov[8 * v + 7]));
            } else {
              float *dst = p.part_o + (row0 + r) * HD + c0;
#pragma unroll
              for (int v = 0; v < 4; ++v)
                reinterpret_cast<float4 *>(dst)[v] =
                    make_float4(ov[4 * v], ov[4 * v + 1], ov[4 * v + 2], ov[4 * v + 3]);
            }
          }
          __syncwarp();
        }
      } else {
        // A chunk of cw columns of every copy goes through shared memory, and the threads add the
        // copies up. A copy that had no unit of the segment holds what it held before.
        const float a = ex2f(m_run - M) * inv;
        const bool has = m_run != kNoMax || l_run != 0.f;
        float *stage = reinterpret_cast<float *>(smem + C::OFF_STG);
        int cw = HD;                     // columns per chunk: RHO * live rows of cw fit the buffer
        while (RHO * live * cw > C::STAGE) cw >>= 1;
#pragma unroll 1
        for (int c0 = 0; c0 < HD && ok; c0 += cw) {
#pragma unroll 1
          for (int cc = 0; cc < cw; cc += 16) {
            float ov[16];
            tmem_ld16(o_mine + c0 + cc, ov);
            if (r < live) {
              float *to = stage + (copy * live + r) * cw;
#pragma unroll
              for (int c = 0; c < 16; ++c)   // columns turned by the row: no bank conflicts
                to[(cc + c + r) & (cw - 1)] = has ? ov[c] * a : 0.f;
            }
            __syncwarp();
          }
          ok = half_sync();
#pragma unroll 1
          for (int e = tl; e < live * cw / 2 && ok; e += 128) {
            const int rr = e / (cw / 2), c = (e % (cw / 2)) * 2;
            float v0 = 0.f, v1 = 0.f;
#pragma unroll
            for (int y = 0; y < RHO; ++y) {
              const float *from = stage + (y * live + rr) * cw;
              v0 += from[(c + rr) & (cw - 1)];
              v1 += from[(c + 1 + rr) & (cw - 1)];
            }
            if (whole)
              *reinterpret_cast<uint32_t *>(o + (static_cast<size_t>(rr / G) * p.Hq + rr % G) * HD + c0 + c) =
                  pack_bf16x2(v0, v1);
            else
              *reinterpret_cast<float2 *>(p.part_o + (row0 + rr) * HD + c0 + c) = make_float2(v0, v1);
          }
          ok = ok && half_sync();
        }
        if (!ok) break;
      }
      tc_fence_before();
      __syncwarp();
      mbar_arrive_if(o_free, lane == 0);
      if (!more) break;
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
  // The schedule reads only the lengths, written before the attention kernel let this one start.
  // This grid's end must imply the attention's: CTA (0, 0) always waits for it; others with
  // nothing to join leave at once.
  const int pair = blockIdx.x;
  const int i = pair / p.Hkv, g = pair % p.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv;
  const int R = G * p.m;
  const int r = blockIdx.y * kMerge8Warps + warp;
  const Seq8 s = seq8(p, i);
  int before, c0 = 0, c1 = 0;
  const int T = total_units(p, i, lane, &before);
  const bool live = r < R && r / G < s.n;
  if (live) {
    const int Ge = min(T, p.grid);
    const int A = before + g * s.units;
    c0 = cta_of(T, Ge, A);
    c1 = cta_of(T, Ge, A + s.units - 1);
  }
  const bool join = live && c0 != c1;  // else written whole by the attention kernel
  if (join || (blockIdx.x == 0 && blockIdx.y == 0)) griddep_wait();
  griddep_launch();
  if (!join) return;
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
                           static_cast<int>(A8Cfg<HD, RHO>::SMEM));
  if (e == cudaSuccess && dev < 64) done[dev] = true;
  return e;
}

template <int HD, int RHO>
static cudaError_t launch_attn8(const Attn8Params &p, cudaStream_t s) {
  const int R = (p.Hq / p.Hkv) * p.m;
  cudaError_t e = configure_attn8<HD, RHO>();
  if (e != cudaSuccess) return e;
  e = launch_pdl(attn8_kernel<HD, RHO>, dim3(p.grid), dim3(A8Cfg<HD, RHO>::THREADS), A8Cfg<HD, RHO>::SMEM, s, p);
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
