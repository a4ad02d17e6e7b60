// Attention of m query rows per sequence over a cache held in 8 bits (tcgen05): e4m3 keys and values with
// one scale for each block of 64 rows and kv head.
//   o = softmax(q K^T / sqrt(hd)) V over the rows [0, ctx + n) of the sequence's kv head, with
//   `causal` only over [0, ctx + j + 1) for the query of row j; rows j >= n are not computed.
//
// A block of 64 rows is the unit of work: its scale is one number, so K's goes into the scores'
// factor and V's into the probabilities. The units of all (sequence, kv head) pairs, in that
// order, are cut into `grid` contiguous ranges of equal weight, one per CTA (a pair weighs its
// units and a constant more); a CTA's run of units of one pair is a segment. A segment that covers
// its pair writes the output, any other an unnormalised partial (o, running maximum, running sum) to
// slot pair + cta, which the merge kernel joins in a fixed order.
#include <mutex>

#include "attention8.cuh"

namespace df {

// ---------------------------------------------------------------- tensor-core kernel

// Both products read the cache's bytes as they are, with the keys and the head's columns as the 128
// rows of the MMA and the query rows (kRP of them, padded) as its columns:
//   S^T [128 keys][kRP]  = K [keys x hd, e4m3] Q^T, each query row as the sum of an e4m3 and two e5m2 terms
//   O^T [hd][3 kRP]     += V^T [hd x keys, e4m3] P^T, each probability as the sum of three e5m2 terms
// so nothing is widened, and a softmax thread (a TMEM lane) is one key, whose scale is a number of the
// thread. P's terms are columns of one pass over V; Q's are three passes over K, which the tensor cores
// have the time for and which spare the softmax the columns of the others.
// Queries: what the first term leaves of bf16's 8 bits is at most 8 of their last steps, which e5m2's 3 bits
// hold exactly, and its smallest step, 2^-16, lies far enough below: a query's values are exact from 2^-16 of the
// largest of its block of rows on, and what is smaller is off by at most 2^-24 of that (put_q). Two e4m3 terms were
// exact from 2^-9 on only, off by 2^-17 below, which shows where a channel of the queries stands out.
// Probabilities: three e5m2 terms keep 9 bits over f16's range. The terms' products lie in columns of their
// own, so the second and third carry powers of two (2^kSplit2, 2^kSplit3) that put what is left of small
// probabilities where e5m2 has its bits; the output takes them back. What is lost is at most 2^-24 + 2^-25 (f16)
// where the largest is 2^kPBase: 2^-31 of it. (All terms alike lost 2^-24 of the largest for every key, which is
// 40% of a key 2^23 below a sink.)
//
// Units are taken in pairs (128 keys); a segment of an odd number of units ends with one alone.
//
// What bounds it: HBM for long caches. 64 single tokens over 1024 .. 8191 keys (602 MB) take 98 us, 6.1
// TB/s (with 4 rows each, 16 a kv head, 102); under ncu (16 x 16,385 keys) 6.0 TB/s with the tensor pipe busy for
// 13% and 39% of the issue slots used. A segment costs about 4000 cycles besides its pairs (queries, the first
// reference, sums, output). One token over 2047 rows takes 8.7 us, of which reading the lengths and finding
// the range are 1, the queries 0.8, two units 1.3, the merge 2.5. With hd 64 the same tokens take 94 us: half the
// bytes, but as many pairs, and a pair's chain takes as long.
constexpr int kRP = kAttn8FewRows;  // query rows of a kv head, padded

template <int HD>
struct A8Cfg {
  // Query rows of a softmax thread: two groups of four warps halve the chain from S to P (64 single tokens
  // 103.5 us with one group, 99.6 with two).
  static constexpr int ROWS = 8;
  static constexpr int NRG = kRP / ROWS;              // groups of four softmax warps
  static constexpr int NSW = 4 * NRG;
  static constexpr int SB = 2, OB = 2;               // buffers of S, and of O
  static constexpr int UNIT8 = kUnit * HD;           // bytes of a unit's keys (or values)
  static constexpr int PAIR8 = 2 * UNIT8;
  // rings of pairs, one of keys and one of values, as much as shared memory holds
  static constexpr int NS = 5 * (128 / HD);
  static constexpr int P_BYTES = 128 * 128;          // P^T: 128 keys, rows of 128 bytes of which 3 kRP hold terms
  static constexpr int OFF_V8 = NS * PAIR8;
  static constexpr int OFF_P = 2 * NS * PAIR8;       // two buffers
  static constexpr int OFF_Q = OFF_P + 2 * P_BYTES;  // 3 kRP rows of hd bytes
  static constexpr int OFF_REF = OFF_Q + 3 * kRP * HD;     // [kRP] -reference of a row
  static constexpr int OFF_FAC = OFF_REF + kRP * 4;        // [kRP] factor of a row, [kRP / 16] of a block of rows
  static constexpr int OFF_LIM = OFF_FAC + kRP * 4 + 64;        // [kRP] keys that a row sees
  static constexpr int OFF_RED = OFF_LIM + kRP * 4;        // [4][kRP] a quarter's maxima, sums
  static constexpr int OFF_ROW = OFF_RED + 4 * kRP * 4;    // [kRP] a number for every row
  static constexpr int OFF_SC = OFF_ROW + kRP * 4;         // [2 chunks][32 units] scales
  static constexpr int OFF_BAR = OFF_SC + 64 * 16;
  static constexpr int OFF_SEQ = OFF_BAR + 512;           // [kSeqCache] (rows, context)
  static constexpr int OFF_NAN = OFF_SEQ + 128 * 8;       // [hd] first row that sees a NaN in the column
  static constexpr size_t SMEM = 1024 + OFF_NAN + HD * 4;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert(OFF_P % 1024 == 0 && OFF_Q % 1024 == 0 && OFF_REF % 16 == 0 && OFF_LIM % 16 == 0 &&
                    OFF_RED % 16 == 0 && OFF_SC % 16 == 0 && OFF_BAR % 16 == 0 && OFF_SEQ % 16 == 0,
                "alignment: 1024 bytes for swizzled tiles, 16 for what is read as vectors");
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr int OCOLS = 3 * kRP;
  static constexpr uint32_t S_COL = 0;               // S^T of pair pj in buffer pj % SB: kRP columns
  static constexpr uint32_t O_COL = SB * kRP;     // O^T of segment seg in buffer seg % OB
  static_assert(O_COL + OB * OCOLS <= TMEM_COLS, "tensor memory");
  static constexpr int THREADS = (4 + NSW) * 32;
};
// P is 2^(x - reference + kPBase) for x in log2 units; the reference moves (and O with it) only when a
// key exceeds it by more than kRescale: P stays at most 2^15, which e5m2 and f16 hold.
constexpr float kPBase = 8.f, kRescale = 7.f;
// The second term of p < 2^15 is below 2^12, the third at most 2^8: with these factors both stay at most 2^15.
constexpr int kSplit2 = 3, kSplit3 = 7;

// Warps: producer of values and scales, S issuer, PV issuer, producer of keys, softmax (warp w reads
// TMEM lanes of quarter w % 4; rows of group (w - 4) / 4).
constexpr int kWValues = 0, kWS = 1, kWPV = 2, kWKeys = 3, kWSoft = 4;

// The blocks of a CTA's units in order, for a producer warp: lane l looks up unit 32 c + l of chunk
// c, a chunk ahead.
struct Blocks8 {
  Pos8 a;
  int x, now, next;
  __device__ __forceinline__ void init(const Pos8 &w, int lane) {
    a = w;
    a.unit += lane;
    x = lane;
  }
  __device__ __forceinline__ int look_up(const Attn8Params &p, const int2 *sseq, int nunits) {
    int b = 0;
    if (x < nunits) {
#pragma unroll 1
      while (a.unit >= a.units) {
        const int over = a.unit - a.units;
        pos_next_pair(a, p, sseq);
        a.unit = over;
      }
      b = static_cast<int>(block_of(p, a.i, a.g, a.unit));
    }
    a.unit += 32;
    x += 32;
    return b;
  }
  // now, next: the blocks of the first two chunks, then of the following ones
  __device__ __forceinline__ void start(const Attn8Params &p, const int2 *sseq, int nunits) {
    now = look_up(p, sseq, nunits);
    next = look_up(p, sseq, nunits);
  }
  __device__ __forceinline__ void step(const Attn8Params &p, const int2 *sseq, int nunits) {
    now = next;
    next = look_up(p, sseq, nunits);
  }
};

// Sums v[0 .. N) over the warp's lanes; lane l gets the sum of element l % N (N <= 32), in a fixed order.
template <int N>
__device__ __forceinline__ float lane_sums(float (&v)[N], int lane) {
  int o = 16;
#pragma unroll
  for (int n = N / 2; n >= 1; n >>= 1) {
    o = n;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const bool up = lane & o;
      const float send = up ? v[i] : v[i + n];
      v[i] = (up ? v[i + n] : v[i]) + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  float s = v[0];
#pragma unroll
  for (int x = N; x < 32; x <<= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
  return s;
}

// Four probabilities (two f16 pairs, non-negative) as three e5m2 terms each, four to a word, the second times
// 2^kSplit2 and the third times 2^kSplit3. e5m2 is f16's upper byte: the first term cuts, the others
// round (half a step is 0x80, which carries into the byte; the sums, differences and products with powers of two
// are exact), so what is left is at most 2^-10 of the value.
__device__ __forceinline__ void split4(uint32_t p01, uint32_t p23, uint32_t &a, uint32_t &b, uint32_t &c) {
  constexpr uint32_t kUpper = 0xFF00FF00u, kHalf = 0x00800080u;
  auto rest = [](uint32_t x, uint32_t y, float times) {
    const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&x), *reinterpret_cast<const __half2 *>(&y));
    const __half2 t = __hmul2(d, __float2half2_rn(times));
    return *reinterpret_cast<const uint32_t *>(&t);
  };
  constexpr float k2 = 1 << kSplit2, k3 = 1 << (kSplit3 - kSplit2);
  a = __byte_perm(p01, p23, 0x7531);
  const uint32_t r01 = rest(p01, p01 & kUpper, k2), r23 = rest(p23, p23 & kUpper, k2);
  const uint32_t b01 = r01 + kHalf, b23 = r23 + kHalf;
  b = __byte_perm(b01, b23, 0x7531);
  const uint32_t c01 = rest(r01, b01 & kUpper, k3) + kHalf, c23 = rest(r23, b23 & kUpper, k3) + kHalf;
  c = __byte_perm(c01, c23, 0x7531);
}

template <int HD>
__global__ void __launch_bounds__(A8Cfg<HD>::THREADS, 1) attn8_kernel(const __grid_constant__ Attn8Params p) {
  using C = A8Cfg<HD>;
  constexpr int ROWS = C::ROWS, NSW = C::NSW, T = NSW * 32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint8_t *sK8 = smem, *sV8 = smem + C::OFF_V8, *sP = smem + C::OFF_P, *sQ = smem + C::OFF_Q;
  float *nref = reinterpret_cast<float *>(smem + C::OFF_REF);
  float *sfac = reinterpret_cast<float *>(smem + C::OFF_FAC);
  int *slim = reinterpret_cast<int *>(smem + C::OFF_LIM);
  float *red = reinterpret_cast<float *>(smem + C::OFF_RED);
  float *srow = reinterpret_cast<float *>(smem + C::OFF_ROW);
  float4 *sscale = reinterpret_cast<float4 *>(smem + C::OFF_SC);
  uint64_t *k8_full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);  // [NS] keys of a pair have landed
  uint64_t *k8_empty = k8_full + C::NS;
  uint64_t *v8_full = k8_empty + C::NS;
  uint64_t *v8_empty = v8_full + C::NS;
  uint64_t *s_full = v8_empty + C::NS;      // [2] S^T of pair pj complete (in buffer pj % SB)
  uint64_t *s_empty = s_full + 2;           // [2] and read
  uint64_t *p_full = s_empty + 2;           // [2] P^T of pair pj written
  uint64_t *pv_done = p_full + 2;           // [2] O^T += of pair pj complete
  uint64_t *sc_full = pv_done + 2;          // [2] scales of 32 units, chunk c in buffer c % 2
  uint64_t *sc_empty = sc_full + 2;         // [2]
  uint64_t *o_free = sc_empty + 2;          // [2] O^T of segment seg read (buffer seg % OB)
  uint64_t *mma_done = o_free + 2;          // [2]
  uint64_t *q_full = mma_done + 2;          // a segment's query terms are in shared memory
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(q_full + 1);
  Range8 *sched = reinterpret_cast<Range8 *>(tmem_slot + 1);
  static_assert((4 * C::NS + 17) * 8 + 4 + sizeof(Range8) <= 512, "barrier region overflows");
  int2 *sseq = reinterpret_cast<int2 *>(smem + C::OFF_SEQ);
  int *first_nan = reinterpret_cast<int *>(smem + C::OFF_NAN);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv;
  const int R = G * p.m;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(&k8_full[s], 1);
      mbar_init(&k8_empty[s], 1);
      mbar_init(&v8_full[s], 1);
      mbar_init(&v8_empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&s_empty[b], NSW);
      mbar_init(&p_full[b], NSW);
      mbar_init(&pv_done[b], 1);
      mbar_init(&sc_full[b], 1);
      mbar_init(&sc_empty[b], NSW);
      mbar_init(&o_free[b], NSW);
      mbar_init(&mma_done[b], 1);
    }
    mbar_init(q_full, NSW);
    fence_mbar_init();
  }
  if (warp == kWKeys && lane == 0) {
    tma_prefetch_desc(&p.tmK);
    tma_prefetch_desc(&p.tmV);
  }
  if (warp == kWS) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  touch8(p);
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch();
  if (warp == kWValues) {
    find_range(p, blockIdx.x, lane, sched);
  } else if (warp == kWKeys) {
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
  const int nunits = __shfl_sync(0xffffffffu, sched->count, 0);
  Pos8 w = {sched->i, sched->g, sched->unit, sched->units, sched->n, sched->ctx};

  // Every role goes through the CTA's segments: `cnt` units from unit j0 of the CTA on, in pairs pj
  // of units u, u + 1 of the segment. A wait that runs out ends the role (ok = false).
  if (nunits == 0) {
    // nothing to do
  } else if (warp == kWKeys || warp == kWValues) {
    // ---------------- producers of keys and of values: a unit's are 64 rows of hd bytes, which arrive
    // swizzled as the tensor cores read them. The warp of the values also writes the scales of 32
    // units at a time.
    const bool keys = warp == kWKeys;
    const CUtensorMap *map = keys ? &p.tmK : &p.tmV;
    uint8_t *ring = keys ? sK8 : sV8;
    uint64_t *full = keys ? k8_full : v8_full, *empty = keys ? k8_empty : v8_empty;
    const uint64_t pol = policy_evict_first();
    bool ok = !p.stall;
    Blocks8 bl;
    bl.init(w, lane);
    bl.start(p, sseq, nunits);
    float ks = 0.f, vs = 0.f;
    if (!keys && lane < nunits) {
      ks = p.ks[bl.now];
      vs = p.vs[bl.now];
    }
    int pj = 0, st = 0, ph = 1;
    int chunk = keys ? 1 << 30 : 0;      // chunk whose scales are to be written next
#pragma unroll 1
    for (int j0 = 0; j0 < nunits && ok;) {
      const int cnt = min(w.units - w.unit, nunits - j0);
#pragma unroll 1
      for (int u = 0; u < cnt; u += 2, ++pj) {
        const int j = j0 + u, k = j & 31;
        const bool two = u + 1 < cnt;
        const int b0 = __shfl_sync(0xffffffffu, bl.now, k);
        const int bn = __shfl_sync(0xffffffffu, bl.next, 0);
        const int b1 = k == 31 ? bn : __shfl_sync(0xffffffffu, bl.now, (k + 1) & 31);
        ok = pj < C::NS || mbar_wait_warp(&empty[st], ph, p.max_spin);
        if (!ok) break;
        if (elect_one()) {
          uint8_t *dst = ring + st * C::PAIR8;
          mbar_arrive_expect_tx(&full[st], (two ? 2 : 1) * C::UNIT8);
          tma_load_2d(dst, map, &full[st], 0, b0 * kUnit, pol);
          if (two) tma_load_2d(dst + C::UNIT8, map, &full[st], 0, b1 * kUnit, pol);
        }
        __syncwarp();
        if (++st == C::NS) {
          st = 0;
          ph ^= 1;
        }
        // The scales of a chunk, once a first pair of it is under way (of the first chunk: two pairs,
        // whose copies wait for nothing), and before any wait for a unit that needs them; first the
        // chunk of unit j, then that of unit j + 1 where the next chunk begins with it.
#pragma unroll 1
        for (int x = 0; x < 2; ++x) {
          const bool due = x == 0 ? chunk == (j >> 5) && (chunk > 0 || pj == 1 || u + 2 >= cnt || k >= 30)
                                  : k == 31 && two && chunk == (j >> 5) + 1;
          if (due) {
            const int b = chunk & 1;
            ok = chunk < 2 || mbar_wait_warp(&sc_empty[b], ((chunk >> 1) - 1) & 1, p.max_spin);
            if (!ok) break;
            sscale[b * 32 + lane] = scale_terms(ks, vs);
            __syncwarp();
            mbar_arrive_if(&sc_full[b], lane == 0);
            ++chunk;
            const bool more = chunk * 32 + lane < nunits;
            ks = more ? p.ks[bl.next] : 0.f;
            vs = more ? p.vs[bl.next] : 0.f;
          }
          if (x == 0 && (k == 31 || (k == 30 && two))) bl.step(p, sseq, nunits);  // the chunk ends here
        }
        if (!ok) break;
      }
      j0 += cnt;
      if (ok && j0 < nunits) pos_next_pair(w, p, sseq);
    }
    if (!ok && !p.stall && lane == 0) flag_status(p.status, kStatusTimeout);
    // every issued copy must land before the CTA may exit (bounded)
#pragma unroll 1
    for (int x = max(0, pj - C::NS); x < pj; ++x) mbar_wait_warp(&full[x % C::NS], (x / C::NS) & 1, kDrainSpin);
  } else if (warp == kWS) {
    // ---------------- S issuer: S^T = K Q^T, the queries' three terms one after the other
    constexpr uint32_t id = idesc_8bit_f32(128, kRP);
    constexpr int STEPS = HD / 32;       // MMAs of a term
    const uint64_t kd0 = HD == 128 ? sw128_kmajor_desc(smem_u32(sK8)) : sw64_kmajor_desc(smem_u32(sK8));
    const uint64_t qd = HD == 128 ? sw128_kmajor_desc(smem_u32(sQ)) : sw64_kmajor_desc(smem_u32(sQ));
    int st = 0, ph = 0, pj = 0;
    bool ok = true;
#pragma unroll 1
    for (int j0 = 0, seg = 0; j0 < nunits && ok; ++seg) {
      const int cnt = min(w.units - w.unit, nunits - j0);
      ok = mbar_wait_warp(q_full, seg & 1, p.max_spin);
#pragma unroll 1
      for (int u = 0; u < cnt && ok; u += 2, ++pj) {
        const int pe = pj - C::SB;
        ok = mbar_wait_warp(&k8_full[st], ph, p.max_spin) &&
             (pe < 0 || mbar_wait_warp(&s_empty[pe & 1], (pe >> 1) & 1, p.max_spin));
        if (!ok) break;
        tc_fence_after();
        const uint64_t kd = kd0 + static_cast<uint64_t>((st * C::PAIR8) >> 4);
        const uint32_t d = tmem + C::S_COL + (pj % C::SB) * kRP;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 3 * STEPS; ++kk)
            tc_mma_8bit(d, kd + kk % STEPS * 2, qd + kk % STEPS * 2 + kk / STEPS * (kRP * HD >> 4),
                        kk < STEPS ? id : id | kIdescBE5M2, kk > 0 ? 1u : 0u);
          tc_commit(&s_full[pj & 1]);
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
    // ---------------- PV issuer: O^T += V^T P^T; a segment's first pair starts the accumulator, after
    // its buffer's previous segment was read
    constexpr uint32_t id = idesc_8bit_f32(128, C::OCOLS) | kIdescBE5M2 | kIdescAMajorMN | kIdescBMajorMN;
    // hd = 64: the second half of the MMA's rows reads the next unit's values and is not used
    const uint64_t vd0 = HD == 128 ? sw128_mnmajor_desc(smem_u32(sV8), C::UNIT8)
                                   : sw64_mnmajor_desc(smem_u32(sV8), C::UNIT8);
    const uint64_t pd0 = sw128_mnmajor_desc(smem_u32(sP), C::P_BYTES);
    int st = 0, ph = 0, pj = 0;
    bool ok = true;
#pragma unroll 1
    for (int j0 = 0, seg = 0; j0 < nunits && ok; ++seg) {
      const int cnt = min(w.units - w.unit, nunits - j0);
      const int se = seg - C::OB;
      ok = se < 0 || mbar_wait_warp(&o_free[se % C::OB], (se / C::OB) & 1, p.max_spin);
      const uint32_t d = tmem + C::O_COL + (seg % C::OB) * C::OCOLS;
#pragma unroll 1
      for (int u = 0; u < cnt && ok; u += 2, ++pj) {
        const int b = pj & 1;
        ok = mbar_wait_warp(&v8_full[st], ph, p.max_spin) && mbar_wait_warp(&p_full[b], (pj >> 1) & 1, p.max_spin);
        if (!ok) break;
        tc_fence_after();
        const uint64_t vd = vd0 + static_cast<uint64_t>((st * C::PAIR8) >> 4);
        const uint64_t pd = pd0 + static_cast<uint64_t>((b * C::P_BYTES) >> 4);
        const uint32_t add = u > 0 ? 1u : 0u;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            if (kk >= 2 && u + 1 >= cnt) break;   // one unit alone
            tc_mma_8bit(d, vd + static_cast<uint64_t>((kk * 32 * HD) >> 4),
                        pd + static_cast<uint64_t>((kk * 32 * 128) >> 4), id, kk > 0 ? 1u : add);
          }
          tc_commit(&pv_done[b]);
          tc_commit(&v8_empty[st]);
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
    if (elect_one()) tc_commit(&mma_done[1]);
    __syncwarp();
    mbar_wait_warp(&mma_done[1], 0, kDrainSpin);
  } else {
    // ---------------- softmax: a thread is key `key` of the pair, for the rows [r0, r0 + ROWS). Every
    // softmax warp goes through the same barriers, also when a wait has run out: `fail` is told
    // to all of them at the next one, and they leave together.
    const int tid = threadIdx.x - kWSoft * 32;
    const int quarter = warp & 3, rg = tid >> 7, r0 = rg * ROWS;
    const int key = quarter * 32 + lane, slot = key >> 6;
    const uint32_t trow = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const float sl2 = rsqrtf(static_cast<float>(HD)) * 1.4426950408889634f;
    constexpr float kTop = kPBase + kRescale;
    bool fail = false, gone = false;

    // The query rows of a segment, read a segment ahead.
    constexpr int TPQ = T / kRP, QW = HD / TPQ / 2;  // threads a row, words of a thread (4 or 2)
    static_assert(ROWS == 8 && TPQ == 16, "widths of the accesses below");
    const int qrow = tid / TPQ, qpart = tid % TPQ;
    uint32_t qr[QW];
    auto fetch_q = [&](const Pos8 &a) {
      const int j = qrow / G;
      const uint16_t *src =
          p.q + ((static_cast<size_t>(a.i) * p.m + j) * p.Hq + a.g * G + qrow % G) * HD + qpart * 2 * QW;
      const bool have = j < a.n;
      if constexpr (QW == 2) {
        const uint2 u = have ? *reinterpret_cast<const uint2 *>(src) : make_uint2(0, 0);
        qr[0] = u.x, qr[1] = u.y;
      } else {
        const uint4 u = have ? *reinterpret_cast<const uint4 *>(src) : make_uint4(0, 0, 0, 0);
        qr[0] = u.x, qr[1] = u.y, qr[2] = u.z, qr[3] = u.w;
      }
    };
    // The rows are scaled by a power of two so that the largest value of a block of 16 rows lies in
    // [2^7, 2^8), and stored as an e4m3 term and two e5m2 terms of what is left. A block whose rows'
    // largest values differ by more than 2^3 scales every row on its own (the block's factor is then -1).
    // Two barriers.
    auto put_q = [&](const Pos8 &a) {
      int *sexp = reinterpret_cast<int *>(red);
      float am = 0.f;
#pragma unroll
      for (int y = 0; y < QW; ++y)
        am = max3(am, fabsf(__uint_as_float(qr[y] << 16)), fabsf(__uint_as_float(qr[y] & 0xFFFF0000u)));
#pragma unroll
      for (int o = 1; o < TPQ; o <<= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
      // -127: zero or subnormal, 128: infinite
      if (qpart == 0) sexp[qrow] = static_cast<int>(__float_as_uint(am) >> 23) - 127;
      named_bar_sync(1, T);
      int top = -100, low = 200;
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        const int4 v = *reinterpret_cast<const int4 *>(sexp + (qrow & ~15) + e);
        top = max(max(top, max(v.x, v.y)), max(v.z, v.w));
        low = min(min(low, min(v.x == -127 ? 200 : v.x, v.y == -127 ? 200 : v.y)),
                  min(v.z == -127 ? 200 : v.z, v.w == -127 ? 200 : v.w));
      }
      const bool apart = top == 128 || top - low > 3;
      const int exs = apart ? max(sexp[qrow], -100) : top;
      if (qpart == 0 && (qrow & 15) == 0)
        sfac[kRP + (qrow >> 4)] = apart ? -1.f : sl2 * __uint_as_float(static_cast<uint32_t>(top + 120) << 23);
      const bool inf = exs == 128;                              // the row's outputs are NaN
      const int ex = min(exs, 127);
      const float mul = inf ? __int_as_float(0x7FC00000) : __uint_as_float(static_cast<uint32_t>(134 - ex) << 23);
      uint32_t term[3][QW / 2];
#pragma unroll
      for (int y = 0; y < QW; ++y) {
        float2 q = make_float2(__uint_as_float(qr[y] << 16) * mul, __uint_as_float(qr[y] & 0xFFFF0000u) * mul);
#pragma unroll
        for (int t = 0; t < 3; ++t) {
          const __nv_fp8_interpretation_t kind = t == 0 ? __NV_E4M3 : __NV_E5M2;
          const __nv_fp8x2_storage_t h = __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, kind);
          const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(h, kind);
          const float2 hf = __half22float2(*reinterpret_cast<const __half2 *>(&hr));
          q = make_float2(q.x - hf.x, q.y - hf.y);  // exact
          term[t][y / 2] = y % 2 ? term[t][y / 2] | (static_cast<uint32_t>(h) << 16) : h;
        }
      }
      // rows t kRP + r of the operand, 16-byte chunks swizzled as a copy would
      constexpr int BYTES = 2 * QW;                             // of a thread
      const int chunk = qpart * BYTES >> 4, xor8 = HD == 128 ? qrow & 7 : (qrow >> 1) & 3;
      uint8_t *dst = sQ + qrow * HD + ((chunk ^ xor8) << 4) + (qpart * BYTES & 15);
#pragma unroll
      for (int t = 0; t < 3; ++t) {
        if constexpr (BYTES == 8)
          *reinterpret_cast<uint2 *>(dst + t * (kRP * HD)) = make_uint2(term[t][0], term[t][1]);
        else
          *reinterpret_cast<uint32_t *>(dst + t * (kRP * HD)) = term[t][0];
      }
      if (qpart == 0) {
        // the factor takes S to log2 units, 1/sqrt(hd) included; rows that are not there get P = 0
        const int j = qrow / G;
        const bool live = j < a.n;
        sfac[qrow] = live ? sl2 * __uint_as_float(static_cast<uint32_t>(ex + 120) << 23) : 0.f;
        nref[qrow] = live ? 0.f : -1e30f;
        slim[qrow] = p.causal ? min(a.ctx + j + 1, a.ctx + a.n) : a.ctx + a.n;
      }
      fence_proxy_async_smem();
      __syncwarp();
      mbar_arrive_if(q_full, lane == 0);
      named_bar_sync(1, T);
    };

    fetch_q(w);
    put_q(w);
    int pj = 0, st = 0, chunk = -1, freed = 0;  // chunk: scales that may be read; freed: given back
    float lsum[ROWS];
    float own[ROWS];       // -references of this thread's rows
    float fac;                           // factor of their block of 16
    auto keep_rows = [&]() {
#pragma unroll
      for (int c = 0; c < ROWS; c += 4)
        *reinterpret_cast<float4 *>(own + c) = *reinterpret_cast<const float4 *>(nref + r0 + c);
      fac = sfac[kRP + r0 / 16];
    };
    keep_rows();
#pragma unroll 1
    for (int j0 = 0, seg = 0; j0 < nunits; ++seg) {
      const int cnt = min(w.units - w.unit, nunits - j0);
      const bool whole = w.unit == 0 && cnt == w.units;
      Pos8 wn = w;                       // the next segment, whose queries are fetched now
      const bool more = j0 + cnt < nunits;
      if (more) {
        pos_next_pair(wn, p, sseq);
        fetch_q(wn);
      }
      const int every = p.causal ? w.ctx + 1 : w.ctx + w.n;  // keys that every row sees
      const int last_key = w.ctx + w.n;
      const uint32_t o_at = trow + C::O_COL + (seg % C::OB) * C::OCOLS;
#pragma unroll 1
      for (int u = 0; u < cnt; u += 2, ++pj) {
        const int j = j0 + u, base = (w.unit + u) * kUnit;
        const bool two = u + 1 < cnt;
        const int jl = j + (two ? 1 : 0);
        if (chunk < (jl >> 5)) [[unlikely]] {  // (a unit that begins a chunk, or the pair after it)
          fail |= !mbar_wait_warp(&sc_full[(chunk + 1) & 1], ((chunk + 1) >> 1) & 1, p.max_spin);
          ++chunk;
        }
        if (freed < (j >> 5)) [[unlikely]] {  // a chunk is behind this pair
          __syncwarp();
          mbar_arrive_if(&sc_empty[freed & 1], lane == 0);
          ++freed;
        }
        const int js = two ? j + slot : j;
        const float4 sc = sscale[((js >> 5) & 1) * 32 + (js & 31)];  // scale_terms
        // S^T, and that P^T's buffer was read by the pair before last (before the first two: at once)
        fail |= !mbar_wait_warp2(&s_full[pj & 1], (pj >> 1) & 1, &pv_done[pj & 1], ((pj >> 1) - 1) & 1, p.max_spin);
        tc_fence_after();
        // y = log2 of P: score in log2 units + log2 V scale - reference + kPBase
        float y[ROWS];
        float top = -INFINITY;
        const uint32_t s_at = trow + C::S_COL + (pj % C::SB) * kRP + r0;
        const float2 c2 = make_float2(sc.y + kPBase, sc.y + kPBase);
        float h[ROWS];
        tmem_ld8(s_at, h);
        if (fac < 0.f) [[unlikely]] {    // the rows' factors are apart
#pragma unroll
          for (int e = 0; e < ROWS; ++e) h[e] *= sfac[r0 + e];
        }
        const float f = fac < 0.f ? sc.x : fac * sc.x;
        const float2 f2 = make_float2(f, f);
#pragma unroll
        for (int e = 0; e < ROWS; e += 2) {
          const float2 v = fma2(make_float2(h[e], h[e + 1]), f2, add2(make_float2(own[e], own[e + 1]), c2));
          y[e] = v.x;
          y[e + 1] = v.y;
        }
        tc_fence_before();
        __syncwarp();
        mbar_arrive_if(&s_empty[pj & 1], lane == 0);
        mbar_arrive_if(&k8_empty[st], tid == 0);  // S complete: the keys have been read
        const bool there = base + key < last_key && (two || slot == 0);
        if (base + 2 * kUnit > every || !two) [[unlikely]] {  // some row does not see the whole pair
#pragma unroll
          for (int c = 0; c < ROWS; ++c) y[c] = there && base + key < slim[r0 + c] ? y[c] : -INFINITY;
        }
#pragma unroll
        for (int c = 0; c < ROWS; c += 2) top = max3(top, y[c], y[c + 1]);
        // rows of V beyond the last key may hold anything
        const bool bad = rg == 0 && (two || slot == 0) && !there;
        const bool some = rg == 0 && there && base + key >= every;  // seen by some rows: no NaN may stay
        if (named_bar_or(1, T, u == 0 || top > kTop || bad || some || sc.w != 0.f || fail)) [[unlikely]] {
          // ---- now and then: the segment's first pair, a reference that has to move, values to clear, low scales
          if (u == 0 && tid < HD) first_nan[tid] = kNoNan;
          if (named_bar_or(1, T, fail)) {
            gone = true;
            break;
          }
          if (rg == 0 && __any_sync(0xffffffffu, bad || some)) {
            fail |= !mbar_wait_warp(&v8_full[st], (pj / C::NS) & 1, p.max_spin);
            uint4 *row = reinterpret_cast<uint4 *>(sV8 + st * C::PAIR8 + key * HD);
            if (bad) {
#pragma unroll
              for (int e = 0; e < HD / 16; ++e) row[e] = make_uint4(0, 0, 0, 0);
            } else if (some) {
#pragma unroll 1
              for (int e = 0; e < HD / 16; ++e) {   // 16-byte chunks as a copy swizzles them
                const int col = 16 * (e ^ (HD == 128 ? key & 7 : (key >> 1) & 3)), from = base + key - w.ctx;
                uint4 v = row[e];
                v.x = take_nan(v.x, first_nan, col, from);
                v.y = take_nan(v.y, first_nan, col + 4, from);
                v.z = take_nan(v.z, first_nan, col + 8, from);
                v.w = take_nan(v.w, first_nan, col + 12, from);
                row[e] = v;
              }
            }
          }
          float mine = 0.f;
#pragma unroll
          for (int c = 0; c < ROWS; ++c) {
            const float m = warp_max(y[c]);
            mine = lane == c ? m : mine;
          }
          if (lane < ROWS) red[quarter * kRP + r0 + lane] = mine;
          named_bar_sync(1, T);
          float d = 0.f;                 // the row's reference moves by d
          if (tid < kRP) {
            const float m = fmaxf(fmaxf(red[tid], red[kRP + tid]), fmaxf(red[2 * kRP + tid], red[3 * kRP + tid]));
            if (tid < w.n * G && (u == 0 ? m > -INFINITY : m > kTop)) d = m - kPBase;
            srow[tid] = d;
            nref[tid] -= d;
          }
          const bool moved = named_bar_or(1, T, d != 0.f);
          if (moved) {
            keep_rows();
            float sh[ROWS];              // d, then 2^-d
            bool any = false;            // of this group's rows
#pragma unroll
            for (int c = 0; c < ROWS; ++c) {
              sh[c] = srow[r0 + c];
              any |= sh[c] != 0.f;
              y[c] -= sh[c];
            }
            if (u > 0 && any) {
#pragma unroll
              for (int c = 0; c < ROWS; ++c) {
                const float half = ex2f(-0.5f * sh[c]);  // in two halves: scale_terms
                lsum[c] = lsum[c] * half * half;
                sh[c] = half * half;
              }
              // O^T *= 2^-d, once every product before has been added
              fail |= !mbar_wait_warp(&pv_done[(pj - 1) & 1], ((pj - 1) >> 1) & 1, p.max_spin);
              tc_fence_after();
              float ov[3][ROWS];
#pragma unroll
              for (int t = 0; t < 3; ++t) tmem_ld8(o_at + t * kRP + r0, ov[t]);
#pragma unroll
              for (int t = 0; t < 3; ++t) {
                uint32_t x[ROWS];
#pragma unroll
                for (int e = 0; e < ROWS; ++e) x[e] = __float_as_uint(ov[t][e] * sh[e]);
                tmem_st8_raw(o_at + t * kRP + r0, x);
              }
              tmem_wait_st();
            }
          }
          if (u == 0) {
#pragma unroll
            for (int c = 0; c < ROWS; ++c) lsum[c] = 0.f;
          }
          if (sc.w != 0.f) {             // the key's share of the sums on its own
#pragma unroll
            for (int c = 0; c < ROWS; ++c) {
              lsum[c] += ex2f(y[c] - (sc.y + kSumExp));
              if (sc.w == kZeroScale) y[c] -= INFINITY;
            }
          }
        }
        uint8_t *prow = sP + (pj & 1) * C::P_BYTES + key * 128;
        const float2 iv = make_float2(sc.z, sc.z);
        uint32_t ta[ROWS / 4], tb[ROWS / 4], tc[ROWS / 4];
#pragma unroll
        for (int e = 0; e < ROWS; e += 4) {
          const float2 p0 = make_float2(ex2f(y[e]), ex2f(y[e + 1]));
          const float2 p1 = make_float2(ex2f(y[e + 2]), ex2f(y[e + 3]));
          const float2 l0 = fma2(p0, iv, make_float2(lsum[e], lsum[e + 1]));
          const float2 l1 = fma2(p1, iv, make_float2(lsum[e + 2], lsum[e + 3]));
          lsum[e] = l0.x;
          lsum[e + 1] = l0.y;
          lsum[e + 2] = l1.x;
          lsum[e + 3] = l1.y;
          const __half2 a = __floats2half2_rn(p0.x, p0.y), b = __floats2half2_rn(p1.x, p1.y);
          split4(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b), ta[e / 4],
                 tb[e / 4], tc[e / 4]);
        }
        // column t * kRP + row of the key's row, 16-byte chunks swizzled
        auto put = [&](int col, const uint32_t (&v)[ROWS / 4]) {
          *reinterpret_cast<uint2 *>(prow + (((col >> 4) ^ (key & 7)) << 4) + (col & 15)) = make_uint2(v[0], v[1]);
        };
        put(r0, ta);
        put(kRP + r0, tb);
        put(2 * kRP + r0, tc);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        mbar_arrive_if(&p_full[pj & 1], lane == 0);
        st = st + 1 == C::NS ? 0 : st + 1;
      }
      if (gone) break;
      // ---- segment end: sums, then the next segment's queries (its S can start), then the output
      j0 += cnt;
      const int live = w.n * G;
      const size_t row0 = (static_cast<size_t>(w.i * p.Hkv + w.g) + blockIdx.x) * R;  // partial rows
      const float sum = lane_sums<ROWS>(lsum, lane);
      if (lane < ROWS) red[quarter * kRP + r0 + lane] = sum;
      named_bar_sync(1, T);
      if (tid < kRP) {
        const float L = (red[tid] + red[kRP + tid]) + (red[2 * kRP + tid] + red[3 * kRP + tid]);
        srow[tid] = whole ? kSumScale / L : 1.0f;
        if (!whole && tid < live)
          *reinterpret_cast<float2 *>(p.part_ml + (row0 + tid) * 2) =
              make_float2(L == 0.f ? kNoMax : -nref[tid], L);
      }
      named_bar_sync(1, T);
      uint16_t *o = p.o + (static_cast<size_t>(w.i) * p.m * p.Hq + w.g * G) * HD + key;
      if (more) {
        w = wn;
        put_q(w);
      }
      fail |= !mbar_wait_warp(&pv_done[(pj - 1) & 1], ((pj - 1) >> 1) & 1, p.max_spin);
      tc_fence_after();
      // lane = column `key` of the head; a row is written by a warp's lanes together
      if (r0 < live) {
        float ov[ROWS];
        tmem_ld8(o_at + r0, ov);
#pragma unroll 1
        for (int t = 1; t < 3; ++t) {
          float x[ROWS];
          tmem_ld8(o_at + t * kRP + r0, x);
          const float f = t == 1 ? 1.f / (1 << kSplit2) : 1.f / (1 << kSplit3);
#pragma unroll
          for (int e = 0; e < ROWS; ++e) ov[e] = fmaf(x[e], f, ov[e]);
        }
        int jr = r0 / G, hr = r0 % G;
#pragma unroll
        for (int e = 0; e < ROWS; ++e) {
          if (r0 + e >= live) break;
          if (HD == 128 || key < HD) {
            const float v = jr < first_nan[key] ? ov[e] * srow[r0 + e] : __int_as_float(0x7FC00000);
            if (whole)
              o[(static_cast<size_t>(jr) * p.Hq + hr) * HD] = static_cast<uint16_t>(pack_bf16x2(v, v));
            else
              p.part_o[(row0 + r0 + e) * HD + key] = v;
          }
          if (++hr == G) {
            hr = 0;
            ++jr;
          }
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      mbar_arrive_if(&o_free[seg % C::OB], lane == 0);
      keep_rows();
    }
    if ((fail || gone) && lane == 0) flag_status(p.status, kStatusTimeout);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWS) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// Joins the partials of every pair whose units several CTAs took, in a fixed order. SPLIT warps per
// query row, HD/32 consecutive values per lane; the maxima and sums come first, a lane per part, so
// that the partial outputs load without waiting for one another. SPLIT is 8 where a pair has 8 parts
// or more (128 rows of 19 parts: 12.5 -> 9.0 us with the attention of 32 units a pair before it; 512
// rows of 19 parts 115 -> 107 us with the attention of 4096) and 1 with fewer, where most of the 8
// warps had nothing (4096 rows of 3 parts: 34 us with 1, 44 with 8, the attention included).
constexpr int kMerge8Warps = 8;

template <int HD, int SPLIT>
__global__ void __launch_bounds__(kMerge8Warps * 32) attn8_merge_kernel(const __grid_constant__ Attn8Params p) {
  constexpr int E = HD / 32;
  constexpr int ROWS = kMerge8Warps / SPLIT;
  __shared__ __align__(16) float sum[SPLIT > 1 ? SPLIT - 1 : 1][HD];
  touch8(p);
  // The schedule reads only the lengths, written before the attention kernel let this one start.
  // This grid's end must imply the attention's: CTA (0, 0) always waits for it; others with
  // nothing to join leave at once.
  const int pair = blockIdx.x;
  const int i = pair / p.Hkv, g = pair % p.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv;
  const int R = G * p.m;
  const int r = blockIdx.y * ROWS + warp / SPLIT;
  const Seq8 s = seq8(p, i);
  int before, c0 = 0, c1 = 0;
  const int T = total_weight(p, i, lane, &before);
  const bool live = r < R && r / G < s.n;
  if (live) {
    const int Ge = min(T, p.grid);
    const int A = before + g * (s.units + p.pair_cost) + p.pair_cost;
    c0 = cta_of(T, Ge, A);
    c1 = cta_of(T, Ge, A + s.units - 1);
  }
  const bool join = live && c0 != c1;  // else written whole by the attention kernel
  if (join || (blockIdx.x == 0 && blockIdx.y == 0)) griddep_wait();
  griddep_launch();
  if (!join) return;  // with SPLIT > 1 a CTA has one row, and leaves as one
  const size_t row0 = (static_cast<size_t>(pair) + c0) * R + r;  // parts are R rows apart
  const int parts = c1 - c0 + 1;
  const float *src = p.part_o + row0 * HD + lane * E;
  float v[4][E], w[4];
  auto load = [&](int b) {  // parts b, b + SPLIT, .. of this warp
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = b + k * SPLIT;
      w[k] = kNoMax;
#pragma unroll
      for (int e = 0; e < E; ++e) v[k][e] = 0.f;
      if (c < parts) {
        const size_t at = static_cast<size_t>(c) * R;
        w[k] = p.part_ml[(row0 + at) * 2];
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 x = *reinterpret_cast<const float2 *>(src + at * HD + e);
          v[k][e] = x.x;
          v[k][e + 1] = x.y;
        }
      }
    }
  };
  load(warp % SPLIT);
  float M = kNoMax, L = 0.f;
#pragma unroll 1
  for (int b = 0; b < parts; b += 32) {
    const int c = b + lane;
    float2 ml = make_float2(kNoMax, 0.f);
    if (c < parts) ml = *reinterpret_cast<const float2 *>(p.part_ml + (row0 + static_cast<size_t>(c) * R) * 2);
    const float Mn = fmaxf(M, warp_max(ml.x));
    float l = moved_sum(ml.y, ml.x - Mn);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    L = moved_sum(L, M - Mn) + l;
    M = Mn;
  }
  const float inv = kSumScale / L;
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 1
  for (int b = warp % SPLIT; b < parts; b += 4 * SPLIT) {
    if (b >= 4 * SPLIT) load(b);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float f = exp2f(w[k] - M);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += v[k][e] * f;
    }
  }
  if constexpr (SPLIT > 1) {
    const int sub = warp % SPLIT;
    if (sub > 0) {
#pragma unroll
      for (int e = 0; e < E; ++e) sum[sub - 1][lane * E + e] = acc[e];
    }
    __syncthreads();
    if (sub > 0) return;
#pragma unroll
    for (int k = 0; k < SPLIT - 1; ++k)
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += sum[k][lane * E + e];
  }
  uint16_t *dst = p.o + ((static_cast<size_t>(i) * p.m + r / G) * p.Hq + g * G + r % G) * HD + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t *>(dst + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
}

// The dynamic shared memory limit is a property of the kernel on one device.
template <int HD>
static cudaError_t configure_attn8() {
  static std::mutex mutex;
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mutex);
  if (dev < 64 && done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(attn8_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(A8Cfg<HD>::SMEM));
  if (e == cudaSuccess && dev < 64) done[dev] = true;
  return e;
}

template <int HD>
static cudaError_t launch_attn8(const Attn8Params &p, cudaStream_t s) {
  cudaError_t e = configure_attn8<HD>();
  if (e != cudaSuccess) return e;
  return launch_pdl(attn8_kernel<HD>, dim3(p.grid), dim3(A8Cfg<HD>::THREADS), A8Cfg<HD>::SMEM, s, p);
}

template <int HD, int SPLIT>
static cudaError_t launch_merge(const Attn8Params &p, int R, cudaStream_t s) {
  constexpr int ROWS = kMerge8Warps / SPLIT;
  return launch_pdl(attn8_merge_kernel<HD, SPLIT>, dim3(p.nb * p.Hkv, (R + ROWS - 1) / ROWS), dim3(kMerge8Warps * 32), 0,
                    s, p);
}

// What a pair costs besides its units, in units: the pipeline's start and end, the output rows. Even
// ranges of units alone left the CTAs of many short pairs behind the others (64 sequences of 1024 ..
// 8191 keys, 8 kv heads, single tokens: 120 us at 0, 106 at 6, 104 at 8, 105 at 10; with 32 query rows
// 122.3 at 8, 123.0 at 12).
constexpr int kPairCost = 8;

template <int HD>
static cudaError_t launch_rows(const Attn8Params &in, cudaStream_t s) {
  Attn8Params p = in;
  p.pair_cost = kPairCost;
  const int R = (p.Hq / p.Hkv) * p.m;
  // both forms' times: attention8_wide.cu
  cudaError_t e = R <= kRP ? launch_attn8<HD>(p, s) : launch_attention8_wide(p, R, s);
  if (e != cudaSuccess) return e;
  return p.nb * p.Hkv * kMerge8Warps <= p.grid ? launch_merge<HD, kMerge8Warps>(p, R, s) : launch_merge<HD, 1>(p, R, s);
}

cudaError_t launch_attention8(const Attn8Params &p, cudaStream_t s) {
  if (p.Hq % p.Hkv != 0 || (p.Hq / p.Hkv) * p.m > 128) return cudaErrorInvalidValue;
  return p.hd == 128 ? launch_rows<128>(p, s) : launch_rows<64>(p, s);
}

}  // namespace df
