// The 8-bit attention for more than 16 query rows of a kv head (attention8.cu has the formula, the
// split over CTAs and the form for fewer rows): the query rows are the 128 rows of the MMA,
//   S [rows][128 keys] = Q K^T     Q an e4m3 and an e5m2 term in tensor memory, K the cache's bytes
//   O [rows][hd]      += P V       P f16 in tensor memory, V widened to f16 in shared memory
// so that a softmax thread is a query row. Widening V costs the same for any number of rows; splitting
// probabilities into 8-bit terms, as the form for few rows does, grows with them: 64 sequences of 1024
// .. 8191 keys take 102 us there and 124 here with 16 rows (hd 64: 100 and 104); with 32 rows, when the form for few
// rows still took them, it was 127 there and 122 here (hd 64: 123 and 107).
// What bounds it: the chain from role to role, beside shared memory's bandwidth (72 KB written and read for
// a unit, 560 cycles of about 720): the same 64 sequences with up to 32 rows (607 MB) take 123 us, 4.9 TB/s, with 64
// rows 139, with 96 160 and with 128 170 (hd 64: 147); one context of 262,155 keys takes 111 with 64 rows, 4.8 TB/s,
// and 128 with 128, for seconds on end, when the power limit holds the clock at 1.70 GHz. Under ncu (8 x 16,400 keys)
// DRAM is busy for 55%, the tensor pipe for 53%, and 42% of the issue slots are used with 64 rows; 47%, 43% and 45%
// with 128. When it took 107 us, it took as long without the conversion instructions, 114 with 8 converter warps,
// which leaves the softmax fewer registers, and 125 with the conversion in integer arithmetic.
#include <mutex>

#include "attention8.cuh"

namespace df {

namespace {
// RHO copies of the query rows fill the 128 lanes of the MMA (rows padded to 128 / RHO): the lanes
// of copy c take only the c-th part of a unit's keys, the other parts' probabilities being zero
// in the P operand, so that every SM quarter's warps share the exponentials of few rows.
template <int HD, int RHO>
struct WideCfg {
  static constexpr int KW = kUnit / RHO;             // keys of a unit per copy
  static constexpr int ROWS = 128 / RHO;             // padded query rows
  static constexpr int ATOMS = HD / 64;              // 128-byte swizzle atoms across hd (f16)
  static constexpr int UNIT8 = kUnit * HD;           // bytes of a unit's keys (or values) in the cache
  static constexpr int PAIR8 = 2 * UNIT8;
  // ring of pairs of units in 8 bits, keys then values, as much as shared memory holds
  static constexpr int NS = 3 * (128 / HD);
  static constexpr int ATOM16 = kUnit * 128;
  static constexpr int TILE16 = ATOMS * ATOM16;      // a unit's values in f16
  static constexpr int QPITCH = HD * 2 + 16;         // bytes of a query row (bf16): rows apart by 16 bytes mod 128
  static constexpr int STAGE = RHO == 1 ? 0 : 128 * HD / 4;  // floats of a half's exchange of O between copies
  static_assert(RHO <= 2, "copies exchange halves");
  static constexpr int OFF_8 = 4 * TILE16;            // values in f16: a pair's two units, two pairs
  static constexpr int OFF_Q = OFF_8 + NS * 2 * PAIR8;
  static constexpr int OFF_STG = OFF_Q + ROWS * QPITCH;
  static constexpr int OFF_ML = OFF_STG + 2 * STAGE * 4;  // [2 halves][128 lanes] (maximum, sum)
  static constexpr int OFF_SC = OFF_ML + 2 * 128 * 8;     // [2 chunks][32 units] scales
  static constexpr int OFF_BAR = OFF_SC + 64 * 16;
  static constexpr int OFF_SEQ = OFF_BAR + 512;           // [kSeqCache] (rows, context)
  static constexpr int OFF_NAN = OFF_SEQ + 128 * 8;       // [4 segments][hd] first row that sees a NaN in the column
  static constexpr size_t SMEM = 1024 + OFF_NAN + 4 * HD * 4;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t S_COL = 0;                // S of a pair of units: 64 columns each
  static constexpr uint32_t O_COL = 128;              // O_0, O_1: hd columns each
  static constexpr uint32_t Q_COL = 128 + 2 * HD;     // queries, two terms of 8 bits: hd / 4 columns each
  static constexpr uint32_t P_COL = Q_COL + HD / 2;   // P of a pair's units: 32 columns each
  static_assert(P_COL + 64 <= TMEM_COLS, "tensor memory");
};
// P is 2^(x - m_run + kPBase), m_run the maximum at the last rescale: O is rescaled only when the
// maximum has grown by more than 2^kRescale, so P stays at most 2^15 in f16, and half a step of f16's smallest
// values is 2^-32 of the largest probability. A maximum that may grow by 2^13 costs less (64 verified blocks 122.9 us
// from a graph, 125.3 with 2^8), but with the largest at 2^2 it rounds keys 2^23 below a sink by up to a tenth.
constexpr float kPBase = 7.f, kRescale = 8.f;

// A segment's units are taken in pairs: one S product of 128 keys, then softmax, PV and O for each
// unit of the pair on its own, so that the steps from one role to the next are paid for two units at
// once. Half a pair at the end of a segment of an odd number of units is signalled by every role
// without work.
// Warps: producer, S issuer, PV issuer, loader of queries, softmax half h = 0, 1 (a
// pair's first or second unit) in 4 + 4h .. 7 + 4h (warp w reads TMEM lanes of quarter w % 4), then
// the converters of V.
constexpr int kWProd = 0, kWS = 1, kWPV = 2, kWQ = 3, kWSoft = 4, kWConv = 12, kNumConv = 4;
constexpr int kWideThreads = (kWConv + kNumConv) * 32;

template <int KW>
__device__ __forceinline__ void load_s(uint32_t taddr, float (&v)[KW]) {
  if constexpr (KW == 64)
    tmem_ld64(taddr, v);
  else
    tmem_ld32(taddr, v);
}
template <int KW>
__device__ __forceinline__ void store_p(uint32_t taddr, const uint32_t *v) {
  if constexpr (KW == 64)
    tmem_st32_raw(taddr, v);
  else
    tmem_st16_raw(taddr, v);
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

template <int HD, int RHO>
__global__ void __launch_bounds__(kWideThreads, 1) attn8_wide_kernel(const __grid_constant__ Attn8Params p) {
  using C = WideCfg<HD, RHO>;
  constexpr int KW = C::KW, ROWS = C::ROWS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint8_t *sV16 = smem, *s8 = smem + C::OFF_8, *sQ = smem + C::OFF_Q;
  float2 *ml = reinterpret_cast<float2 *>(smem + C::OFF_ML);
  float4 *sscale = reinterpret_cast<float4 *>(smem + C::OFF_SC);
  uint64_t *kv8_full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
  uint64_t *kv8_empty = kv8_full + C::NS;
  uint64_t *v16_full = kv8_empty + C::NS;   // [2] values of pair pj in f16, in buffers pj % 2 * 2 + (0, 1)
  uint64_t *v16_empty = v16_full + 2;       // [2] and read
  uint64_t *p_full = v16_empty + 2;         // [2] a pair's first and second unit
  uint64_t *p_empty = p_full + 2;           // [2] PV complete: the P buffer has been read
  uint64_t *sc_full = p_empty + 2;          // [2] scales of 32 units, chunk c in buffer c % 2
  uint64_t *sc_empty = sc_full + 2;         // [2]
  uint64_t *half_bar = sc_empty + 2;        // [2] the four warps of a half among themselves
  uint64_t *mma_done = half_bar + 2;        // [2]
  uint64_t *s_full = mma_done + 2;          // S of a pair complete
  uint64_t *s_empty = s_full + 1;           // and read by both halves
  uint64_t *q8_full = s_empty + 1;          // a segment's query rows have landed
  uint64_t *q8_empty = q8_full + 1;
  uint64_t *q_full = q8_empty + 1;          // and are in tensor memory
  uint64_t *q_empty = q_full + 1;
  uint64_t *seg_bar = q_empty + 1;          // both halves: (maximum, sum) of a segment written
  uint64_t *o_free = seg_bar + 1;           // both O and ml read
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(o_free + 1);
  Range8 *sched = reinterpret_cast<Range8 *>(tmem_slot + 1);
  static_assert((2 * C::NS + 16 + 8) * 8 + 4 + sizeof(Range8) <= 512, "barrier region overflows");
  int2 *sseq = reinterpret_cast<int2 *>(smem + C::OFF_SEQ);
  // Segment seg uses the part seg % 4. The softmax clears it behind seg_bar of seg + 1, past every read, and
  // before it frees that segment's O; a converter gets to seg + 4 only after a PV of seg + 2, which waits
  // for that.
  int *first_nan = reinterpret_cast<int *>(smem + C::OFF_NAN);

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
      mbar_init(&v16_empty[b], 1);
      mbar_init(&p_full[b], 4);
      mbar_init(&p_empty[b], 1);
      mbar_init(&sc_full[b], 1);
      mbar_init(&sc_empty[b], 8);
      mbar_init(&half_bar[b], 4);
      mbar_init(&mma_done[b], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(s_empty, 8);
    mbar_init(q8_full, 32);
    mbar_init(q8_empty, 8);
    mbar_init(q_full, 8);
    mbar_init(q_empty, 1);
    mbar_init(seg_bar, 8);
    mbar_init(o_free, 8);
    fence_mbar_init();
  }
  for (int x = threadIdx.x; x < 4 * HD; x += kWideThreads) first_nan[x] = kNoNan;
  if (warp == kWS) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  touch8(p);
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch();
  if (warp == kWProd) {
    find_range(p, blockIdx.x, lane, sched);
  } else if (warp == kWQ) {
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
  } else if (warp == kWProd) {
    // ---------------- producer: a unit's keys and values are contiguous 64 * hd bytes each (the keys
    // arrive swizzled, as the tensor cores read them). Lane l looks up the block of unit 32 c + l of the
    // CTA's range two chunks c ahead and its scales one chunk ahead, so the copies wait for neither.
    const uint64_t pol = policy_evict_first();
    bool ok = !p.stall;
    int pairs = 0;
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
      if (cnt_left == 0) {  // a segment begins
        if (j > 0) pos_next_pair(w, p, sseq);
        cnt_left = min(w.units - w.unit, nunits - j);
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
      // of the chunk: a copy waits for the pair NS >= 3 before its own.
      published = published && k != 0;
      if (!published && (k == 3 || j == nunits - 1 || cnt_left == 0)) {
        published = true;
        ok = c < 2 || mbar_wait_warp(&sc_empty[c & 1], ((c >> 1) - 1) & 1, p.max_spin);
        if (!ok) break;
        sscale[(c & 1) * 32 + lane] = scale_terms(ks, vs);
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
  } else if (warp == kWQ) {
    // ---------------- query rows of every segment, a segment ahead: 16 bytes a lane (a bulk copy for each
    // row took 2.4 us for 64, one after the other)
    bool ok = !p.stall;
#pragma unroll 1
    for (int j0 = 0, seg = 0; j0 < nunits && ok; ++seg) {
      ok = seg == 0 || mbar_wait_warp(q8_empty, (seg - 1) & 1, p.max_spin);
      if (!ok) break;
      constexpr int CPR = HD / 8;        // 16-byte chunks of a row
      const uint16_t *src = p.q + (static_cast<size_t>(w.i) * p.m * p.Hq + w.g * G) * HD + lane % CPR * 8;
      int r = lane / CPR, j = r / G, h = r % G;
#pragma unroll 1
      for (; r < w.n * G; r += 32 / CPR) {
        cp_async16(smem_u32(sQ + r * C::QPITCH + lane % CPR * 16), src + (static_cast<size_t>(j) * p.Hq + h) * HD);
        for (h += 32 / CPR; h >= G; h -= G) ++j;
      }
      cp_async_arrive(q8_full);
      j0 += min(w.units - w.unit, nunits - j0);
      if (j0 < nunits) pos_next_pair(w, p, sseq);
    }
    if (!ok && !p.stall && lane == 0) flag_status(p.status, kStatusTimeout);
    cp_async_wait_all();
  } else if (warp == kWS) {
    // ---------------- S issuer: S(j) = Q K(j)^T straight from the 8-bit keys, the queries' two
    // terms one after the other from tensor memory
    constexpr uint32_t id_s = idesc_8bit_f32(128, kUnit);
    const uint64_t kd0 = HD == 128 ? sw128_kmajor_desc(smem_u32(s8)) : sw64_kmajor_desc(smem_u32(s8));
    constexpr uint32_t id_s2 = idesc_8bit_f32(128, 2 * kUnit);
    int st = 0, ph = 0, pj = 0;
    bool ok = true;
#pragma unroll 1
    for (int j0 = 0, seg = 0; j0 < nunits && ok; ++seg) {
      const int cnt = min(w.units - w.unit, nunits - j0);
      ok = mbar_wait_warp(q_full, seg & 1, p.max_spin);
#pragma unroll 1
      for (int u = 0; u < cnt && ok; u += 2, ++pj) {
        ok = mbar_wait_warp(&kv8_full[st], ph, p.max_spin);
        ok = ok && (pj == 0 || mbar_wait_warp(s_empty, (pj - 1) & 1, p.max_spin));
        if (!ok) break;
        tc_fence_after();
        const uint64_t kd = kd0 + static_cast<uint64_t>((st * 2 * C::PAIR8) >> 4);
        const uint32_t id = u + 1 < cnt ? id_s2 : id_s;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 2 * HD / 32; ++kk)
            tc_mma_8bit_tmem_a(tmem + C::S_COL, tmem + C::Q_COL + kk * 8,
                               kd + static_cast<uint64_t>((kk % (HD / 32)) * 32 >> 4),
                               kk < HD / 32 ? id : id | kIdescAE5M2, kk > 0 ? 1u : 0u);
          tc_commit(s_full);
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
    // ---------------- PV issuer: O_b += P V for a pair's unit b; a segment's first pair starts the
    // accumulators, after both O of the previous segment were read
    constexpr uint32_t id_pv = idesc_f16_f32(128, HD) | kIdescBMajorMN;
    const uint64_t vd0 = sw128_mnmajor_desc(smem_u32(sV16), C::ATOM16);
    bool ok = true;
    int pj = 0;
#pragma unroll 1
    for (int j0 = 0, seg = 0; j0 < nunits && ok; ++seg) {
      const int cnt = min(w.units - w.unit, nunits - j0);
      if (seg > 0) ok = mbar_wait_warp(o_free, (seg - 1) & 1, p.max_spin);
#pragma unroll 1
      for (int x = 0; x < ((cnt + 1) & ~1) && ok; ++x) {
        const int b = x & 1;
        const int vb = (pj & 1) * 2 + b;
        ok = mbar_wait_warp2(&v16_full[pj & 1], (pj >> 1) & 1, &p_full[b], pj & 1, p.max_spin);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          if (x < cnt) {
            const uint64_t vd = vd0 + static_cast<uint64_t>((vb * C::TILE16) >> 4);
#pragma unroll
            for (int kk = 0; kk < kUnit / 16; ++kk)
              tc_mma_bf16_tmem_a(tmem + C::O_COL + b * HD, tmem + C::P_COL + b * 32 + kk * 8,
                                 vd + static_cast<uint64_t>((kk * 16 * 128) >> 4), id_pv, (x > 1 || kk > 0) ? 1u : 0u);
          }
          tc_commit(&p_empty[b]);
          if (b == 1) tc_commit(&v16_empty[pj & 1]);
        }
        __syncwarp();
        pj += b;
      }
      j0 += cnt;
      if (j0 < nunits) pos_next_pair(w, p, sseq);
    }
    if (!ok && lane == 0) flag_status(p.status, kStatusTimeout);
    if (elect_one()) tc_commit(&mma_done[1]);
    __syncwarp();
    mbar_wait_warp(&mma_done[1], 0, kDrainSpin);
  } else if (warp >= kWConv) {
    // ---------------- converters: V from e4m3 to f16, in the layout of a 128-byte-swizzled copy (rows
    // of 64 values, 16-byte chunk c of row r at c ^ (r & 7))
    constexpr int CPR = HD / 8;                        // 8-value chunks of a row: 8 bytes to 16
    constexpr int RPI = kNumConv * 32 / CPR;           // rows per iteration: 8 or 16
    constexpr int PER = kUnit / RPI;                   // chunks per thread
    static_assert(RPI % 8 == 0, "a thread's chunks all lie at the same place of their rows");
    const int t = (warp - kWConv) * 32 + lane;
    const int cc = t % CPR, r0 = t / CPR;
    uint8_t *out = sV16 + (cc >> 3) * C::ATOM16 + r0 * 128 + (((cc & 7) ^ (r0 & 7)) << 4);
    const uint8_t *src0 = s8 + C::PAIR8 + t * 8;
    bool ok = true;
    int st = 0, ph = 0, pj = 0;
#pragma unroll 1
    for (int j0 = 0, seg = 0; j0 < nunits && ok; ++seg) {
      const int cnt = min(w.units - w.unit, nunits - j0);
      int keys = w.ctx + w.n - w.unit * kUnit;     // rows of the unit that hold keys
      const int some = p.causal ? w.n - 1 : 0;     // the last of them are seen by some query rows only
#pragma unroll 1
      for (int u = 0; u < cnt; u += 2, ++pj, keys -= 2 * kUnit) {
        // the pair's bytes, and its f16 buffers read by the pair before last (before the first two: at once)
        ok = mbar_wait_warp2(&kv8_full[st], ph, &v16_empty[pj & 1], ((pj >> 1) - 1) & 1, p.max_spin);
        if (!ok) break;
        const uint8_t *src = src0 + st * 2 * C::PAIR8;
        uint8_t *dst = out + (pj & 1) * 2 * C::TILE16;
        if (keys - some < 2 * kUnit || u + 1 >= cnt) [[unlikely]] {
          // one unit alone; rows that some queries see; rows beyond the last key, which may hold anything
          // (even NaN): P is 0 there
#pragma unroll 1
          for (int b = 0; b < 2 && u + b < cnt; ++b) {
#pragma unroll 2
            for (int e = 0; e < PER; ++e) {
              uint4 h = make_uint4(0, 0, 0, 0);
              const int row = b * kUnit + r0 + e * RPI;
              if (row < keys) {
                uint2 v = *reinterpret_cast<const uint2 *>(src + b * C::UNIT8 + e * RPI * HD);
                if (row >= keys - some) {
                  int *first = first_nan + (seg & 3) * HD;
                  v.x = take_nan(v.x, first, cc * 8, row - keys + w.n);
                  v.y = take_nan(v.y, first, cc * 8 + 4, row - keys + w.n);
                }
                h = widen8(v);
              }
              *reinterpret_cast<uint4 *>(dst + b * C::TILE16 + e * RPI * 128) = h;
            }
          }
        } else {
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            uint2 v[PER];
#pragma unroll
            for (int e = 0; e < PER; ++e)
              v[e] = *reinterpret_cast<const uint2 *>(src + b * C::UNIT8 + e * RPI * HD);
#pragma unroll
            for (int e = 0; e < PER; ++e)
              *reinterpret_cast<uint4 *>(dst + b * C::TILE16 + e * RPI * 128) = widen8(v[e]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        mbar_arrive_if(&v16_full[pj & 1], lane == 0);
        mbar_arrive_if(&kv8_empty[st], lane == 0);
        if (++st == C::NS) {
          st = 0;
          ph ^= 1;
        }
      }
      j0 += cnt;
      if (j0 < nunits) pos_next_pair(w, p, sseq);
    }
    if (!ok && lane == 0) flag_status(p.status, kStatusTimeout);
  } else if (warp >= kWSoft) {
    // ---------------- softmax: thread = TMEM lane; lane l holds query row l % ROWS, copy l / ROWS
    const int half = (warp - kWSoft) >> 2, q = warp & 3;
    const int tl = q * 32 + lane;
    const int r = tl % ROWS, copy = tl / ROWS;
    const int k0 = copy * KW;
    const uint32_t trow = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const int jq = r / G;               // row r: query row jq of query head g * G + r % G
    const float sl2 = rsqrtf(static_cast<float>(HD)) * 1.4426950408889634f;
    uint32_t half_phase = 0;
    // Barrier of a half's warps, bounded like every other wait.
    auto half_sync = [&]() {
      __syncwarp();
      mbar_arrive_if(&half_bar[half], lane == 0);
      const bool done = mbar_wait_warp(&half_bar[half], half_phase, p.max_spin);
      half_phase ^= 1;
      return done;
    };
    if (RHO > 1) {  // the other copies' parts of the P rows stay zero
      const uint32_t z[16] = {};
      tmem_st16_raw(trow + C::P_COL + half * 32, z);
      tmem_st16_raw(trow + C::P_COL + half * 32 + 16, z);
      tmem_wait_st();
    }
    // The query row of segment `seg` (n rows a sequence), scaled by a power of two so that its
    // largest value lies in [2^7, 2^8), to tensor memory as the sum of an e4m3 term and an e5m2 term of what is left
    // (at most 8 steps of bf16's last bit, which 3 bits hold): exact from 2^-13 of the largest value on, and
    // off by at most 2^-21 of it below. (Two e4m3 terms: from 2^-9 on, 2^-17 below.)
    // Returns the factor that takes S to log2 units, 1/sqrt(hd) included; < 0 on a wait run out.
    auto load_q = [&](int seg, int n) {
      bool ok = mbar_wait_warp(q8_full, seg & 1, p.max_spin);
      if (seg > 0) ok = ok && mbar_wait_warp(q_empty, (seg - 1) & 1, p.max_spin);
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
      const float mul = inf ? __int_as_float(0x7FC00000) : __uint_as_float(static_cast<uint32_t>(7 - ex + 127) << 23);
      tc_fence_after();
#pragma unroll 1
      for (int part = half * (HD / 64); part < (half + 1) * (HD / 64); ++part) {  // a half of the columns
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
                __nv_cvt_float2_to_fp8x2(make_float2(y.x - af.x, y.y - af.y), __NV_SATFINITE, __NV_E5M2);
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
      __syncwarp();
      mbar_arrive_if(q_full, lane == 0);
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
      for (int u = half; u < ((cnt + 1) & ~1) + half; u += 2, ++pj) {
        const int j = min(j0 + u, j0 + cnt - 1);
        if (chunk < (j >> 5)) [[unlikely]] {  // the next chunk: give the one before back
          __syncwarp();
          if (chunk >= 0) mbar_arrive_if(&sc_empty[chunk & 1], lane == 0);
          ++chunk;
          ok = mbar_wait_warp(&sc_full[chunk & 1], (chunk >> 1) & 1, p.max_spin);
        }
        const float4 sc = sscale[(chunk & 1) * 32 + (j & 31)];  // scale_terms
        ok = ok && mbar_wait_warp(s_full, pj & 1, p.max_spin);
        if (!ok) break;
        tc_fence_after();
        float sv[KW];
        load_s<KW>(trow + C::S_COL + half * kUnit + k0, sv);
        tc_fence_before();
        __syncwarp();
        mbar_arrive_if(s_empty, lane == 0);
        mbar_arrive_if(&kv8_empty[st], lane == 0 && warp == kWSoft);  // S complete: the keys have been read
        st = st + 1 == C::NS ? 0 : st + 1;
        // the P buffer and O_half are free once PV of this half's previous unit has completed
        bool freed = pj == 0;
        if (u >= cnt) [[unlikely]] {     // half a pair
          ok = freed || mbar_wait_warp(&p_empty[half], (pj - 1) & 1, p.max_spin);
          if (!ok) break;
          mbar_arrive_if(&p_full[half], lane == 0);
          continue;
        }
        if (all - kUnit * u < kUnit) [[unlikely]] {  // some row does not see the whole unit
          const int nv = lim - (w.unit + u) * kUnit - k0;  // keys this thread sees of its part
#pragma unroll
          for (int c = 0; c < KW; ++c) sv[c] = c < nv ? sv[c] : -INFINITY;
        }
        const float c1 = fmaxf(qfac * sc.x, 1e-37f);
        float mx[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
        for (int c = 4; c + 8 <= KW; c += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], sv[c + 2 * e], sv[c + 2 * e + 1]);
        mx[3] = max3(max3(mx[3], sv[KW - 4], sv[KW - 3]), sv[KW - 2], sv[KW - 1]);
        const float m_new = fmaf(fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]), c1, sc.y);
        const bool need = m_new - m_run > kRescale;
        float alpha = 1.f;
        if (need) {
          const float h = ex2f(0.5f * (m_run - m_new));  // in two halves: scale_terms
          alpha = h * h;
          l_run = l_run * h * h;
          m_run = m_new;
        }
        if (u >= 2 && __any_sync(0xffffffffu, need && r < R)) [[unlikely]] {
          ok = mbar_wait_warp(&p_empty[half], (pj - 1) & 1, p.max_spin);
          if (!ok) break;
          tc_fence_after();
          freed = true;
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
        float c2 = sc.y - m_run + kPBase;
        if (sc.w != 0.f) [[unlikely]] {
          const float cs = c2 - (sc.y + kSumExp);
          float s = 0.f;
#pragma unroll
          for (int c = 0; c < KW; ++c) s += ex2f(fmaf(sv[c], c1, cs));
          l_run += s;
          if (sc.w == kZeroScale) c2 = -INFINITY;
        }
        uint32_t pk[KW / 2];
        float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < KW; c += 2) {
          const float2 x = fma2(make_float2(sv[c], sv[c + 1]), make_float2(c1, c1), make_float2(c2, c2));
          const float2 e = make_float2(ex2f(x.x), ex2f(x.y));
          ls[(c >> 1) & 1] = add2(ls[(c >> 1) & 1], e);
          const __half2 y = __floats2half2_rn(e.x, e.y);
          pk[c / 2] = *reinterpret_cast<const uint32_t *>(&y);
        }
        const float2 lt = add2(ls[0], ls[1]);
        l_run = fmaf(lt.x + lt.y, sc.z, l_run);
        if (!freed) {
          ok = mbar_wait_warp(&p_empty[half], (pj - 1) & 1, p.max_spin);
          if (!ok) break;
          tc_fence_after();
        }
        store_p<KW>(trow + C::P_COL + half * 32 + k0 / 2, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        mbar_arrive_if(&p_full[half], lane == 0);
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
      ok = ok && mbar_wait_warp(&p_empty[half], (pj - 1) & 1, p.max_spin);
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
      float M = kNoMax, L = 0.f;
#pragma unroll
      for (int c = 0; c < 2 * RHO; ++c) M = fmaxf(M, ml[c * ROWS + r].x);
#pragma unroll
      for (int c = 0; c < 2 * RHO; ++c) L += moved_sum(ml[c * ROWS + r].y, ml[c * ROWS + r].x - M);
      const size_t row0 = (static_cast<size_t>(i * p.Hkv + g) + blockIdx.x) * R;   // partial rows
      const float inv = whole ? kSumScale / L : 1.0f;
      const bool has1 = cnt > 1;
      const float a0 = ex2f(ml[tl].x - M) * inv, a1 = has1 ? ex2f(ml[128 + tl].x - M) * inv : 0.f;
      const int live = n * G;            // rows that are computed
      if (half == 0 && copy == 0 && r < live && !whole)
        *reinterpret_cast<float2 *>(p.part_ml + (row0 + r) * 2) = make_float2(M, L);
      // Each half takes its half of the columns of O_0 and O_1. With two copies, a copy's threads
      // write half of those, and hand their part of the others over through shared memory, which
      // the next segment writes only after its seg_bar, past every read here.
      uint16_t *o = p.o + ((static_cast<size_t>(i) * p.m + jq) * p.Hq + g * G + r % G) * HD;
      float *po = p.part_o + (row0 + r) * HD;
      int *first = first_nan + (seg & 3) * HD;
      if (seg > 0 && half * 128 + tl < HD) first_nan[((seg - 1) & 3) * HD + half * 128 + tl] = kNoNan;
      auto put = [&](uint32_t col, float (&v)[16]) {
        if (p.causal) {
#pragma unroll
          for (int c = 0; c < 16; ++c) v[c] = jq < first[col + c] ? v[c] : __int_as_float(0x7FC00000);
        }
        if (r < live && whole) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
            reinterpret_cast<uint4 *>(o + col)[e] =
                make_uint4(pack_bf16x2(v[8 * e], v[8 * e + 1]), pack_bf16x2(v[8 * e + 2], v[8 * e + 3]),
                           pack_bf16x2(v[8 * e + 4], v[8 * e + 5]), pack_bf16x2(v[8 * e + 6], v[8 * e + 7]));
        } else if (r < live) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            reinterpret_cast<float4 *>(po + col)[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        }
        __syncwarp();
      };
      if constexpr (RHO == 1) {
#pragma unroll 1
        for (uint32_t col = half * (HD / 2); col < (half + 1) * (HD / 2); col += 16) {
          float v[16], o1[16];
          tmem_ld16_two(trow + C::O_COL + col, v, trow + C::O_COL + HD + col, o1);
#pragma unroll
          for (int c = 0; c < 16; ++c) v[c] = v[c] * a0 + (has1 ? o1[c] * a1 : 0.f);
          put(col, v);
        }
      } else {
        float *stage = reinterpret_cast<float *>(smem + C::OFF_STG) + half * C::STAGE;
        auto columns = [&](uint32_t col, float (&v)[16]) {  // of this copy, both units' O
          float o1[16];
          tmem_ld16_two(trow + C::O_COL + col, v, trow + C::O_COL + HD + col, o1);
#pragma unroll
          for (int c = 0; c < 16; ++c) v[c] = v[c] * a0 + (has1 ? o1[c] * a1 : 0.f);
        };
#pragma unroll 1
        for (int cc = 0; cc < HD / 4; cc += 16) {
          float v[16];
          columns(half * (HD / 2) + (1 - copy) * (HD / 4) + cc, v);
#pragma unroll
          for (int c = 0; c < 16; ++c) stage[((1 - copy) * (HD / 4) + cc + c) * ROWS + r] = v[c];
        }
        ok = half_sync();
        if (!ok) break;
#pragma unroll 1
        for (int cc = 0; cc < HD / 4; cc += 16) {
          const uint32_t col = half * (HD / 2) + copy * (HD / 4) + cc;
          float v[16];
          columns(col, v);
#pragma unroll
          for (int c = 0; c < 16; ++c) v[c] += stage[(copy * (HD / 4) + cc + c) * ROWS + r];
          put(col, v);
        }
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


template <int HD, int RHO>
cudaError_t launch_wide_form(const Attn8Params &p, cudaStream_t s) {
  static std::mutex mutex;
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lock(mutex);
    if (dev >= 64 || !done[dev]) {
      e = cudaFuncSetAttribute(attn8_wide_kernel<HD, RHO>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(WideCfg<HD, RHO>::SMEM));
      if (e != cudaSuccess) return e;
      if (dev < 64) done[dev] = true;
    }
  }
  return launch_pdl(attn8_wide_kernel<HD, RHO>, dim3(p.grid), dim3(kWideThreads), WideCfg<HD, RHO>::SMEM, s, p);
}

}  // namespace

cudaError_t launch_attention8_wide(const Attn8Params &p, int R, cudaStream_t s) {
  // copies of the query rows that fill the MMA's 128
  if (p.hd == 128) return R > 64 ? launch_wide_form<128, 1>(p, s) : launch_wide_form<128, 2>(p, s);
  return R > 64 ? launch_wide_form<64, 1>(p, s) : launch_wide_form<64, 2>(p, s);
}

}  // namespace df
