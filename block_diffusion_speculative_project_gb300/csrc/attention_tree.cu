// Attention of a tree of drafted tokens over the bf16 caches, with a sliding window and first rows
// ("sinks") that stay visible, on the tcgen05 tensor cores. For node j of sequence i (position
// ctx + depth(j)) and query head h of kv head g = h / (Hq/Hkv):
//   o = softmax(q K^T / sqrt(hd)) V over
//     the context rows p < ctx with  no window,  or p > ctx + depth(j) - window,  or p < sinks
//     the rows ctx + a of the nodes a from j up to the root, by the same rule at ctx + depth(a)
// (KV injection and the attention equations of "DFlash 投机解码：块扩散草稿与 KV 注入", 二; the pages verify
// one path, a tree holds several). A chain of nodes is causal attention, one node the decode step.
//
// Bound: the visible K and V rows, read once; at 256 query rows a kv head as much tensor time. So
// query rows R = (Hq/Hkv) * m of a kv head are the rows of M = 128 MMAs, in one of two forms:
//   one tile (R <= 128)   two halves of softmax warps take units of 64 keys in turn, each with its own
//                         running maximum, sum and O, joined at the end of a segment
//   two tiles (R > 128)   both halves work on every unit, each for its own tile of up to 128 rows: K and
//                         V are read once for 256 rows. More rows take further groups of two tiles.
// A (sequence, kv head, group) is a pair; the visible units of all pairs are cut into equal ranges, one
// per CTA (one CTA per SM). The run of one pair inside a range is a segment: it writes the output, or if
// the pair goes on in another CTA an unnormalised partial (only a range's first and last segment can
// be one: two slots a CTA), which attn_tree_merge_kernel joins in CTA order. With a window a pair's units
// are those of the sinks, then those from the root's first visible row on.
//
// Masks: a unit that every row sees whole takes none. The others (the window's edge, the end of the
// sinks, the tree's own rows) get a 64-bit mask a row from its node's line of ancestors. Values in
// rows that a query row does not see may be NaN or infinite: in masked units a warp of its own (the
// cleaner) zeroes such values before the product sees them and notes their keys, and the rows that see
// such a key get a NaN probability for it.
//
// One CTA: TMA producer (Q tiles of the segment; K and V of a unit per stage), S issuer (S = Q K^T into
// buffer step % 2), PV issuer (O_half += P V, P from tensor memory, buffer step % 4), the cleaner, and
// the softmax warps: a thread owns a query row (its TMEM lane), keeps its maximum and sum in fp32,
// rounds P to bf16 (2^-9 of each probability, as the values have) and rescales O only when the row's
// maximum grew by more than 2^8, so most units need no round trip of O.
#include <cfloat>

#include "common.cuh"
#include "kernels.h"

namespace df {

namespace {

constexpr int kKeys = 64;      // keys of a unit: one page
constexpr int kTileRows = 128; // M of the MMAs
constexpr int kDrainSpin = 1 << 22;
constexpr float kGrowLog2 = 8.0f;

// NQ: TMEM lane quarters with real query rows. Warp w reads the lanes of quarter w % 4, so half 0 is
// warps [0, NQ), half 1 warps [4, 4 + NQ), and the other roles take what is left.
template <int NQ>
struct Roles {
  static constexpr int PRODUCER = NQ == 4 ? 8 : NQ;
  static constexpr int S = PRODUCER + 1;
  static constexpr int PV = NQ == 4 ? 10 : NQ == 2 ? 6 : 3;
  static constexpr int CLEAN = NQ == 4 ? 11 : NQ == 2 ? 7 : 5;
  static constexpr int THREADS = NQ == 4 ? 384 : NQ == 2 ? 256 : 192;
  static constexpr int HALF = NQ * 32;
};

template <int HD, bool TWO>
struct Cfg {
  static constexpr int ATOMS = HD / 64;            // 128-byte swizzle atoms across hd
  static constexpr int ATOM_Q = kTileRows * 128;
  static constexpr int TILES = TWO ? 2 : 1;
  static constexpr int Q_TILE = ATOMS * ATOM_Q;
  static constexpr int ATOM_KV = kKeys * 128;
  static constexpr int KV_TILE = ATOMS * ATOM_KV;
  static constexpr int STAGE = 2 * KV_TILE;        // K, then V
  static constexpr int STAGES = HD == 64 ? 8 : TWO ? 5 : 6;
  static constexpr int OFF_KV = TILES * Q_TILE;
  static constexpr int OFF_BAR = OFF_KV + STAGES * STAGE;
  static constexpr int OFF_SEQ = OFF_BAR + 512;
  static constexpr int OFF_ML = OFF_SEQ + 512;
  static constexpr size_t SMEM = 1024 + OFF_ML + kTileRows * 8;
  static constexpr uint32_t S_COL = 0;             // two S buffers of 64 columns
  static constexpr uint32_t O_COL = 128;           // O of the two halves
  static constexpr uint32_t P_COL = 128 + 2 * HD;  // four P buffers of 32 columns
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What sequence i attends to: its lengths, and its visible units as A of the sinks and those from W0 on.
struct Span {
  int ctx, n, U, A, W0;
};
__device__ __forceinline__ int clamp_nodes(const AttnTreeParams &p, int i) {
  return p.n_rows ? max(0, min(p.n_rows[i], p.m)) : p.m;
}
__device__ __forceinline__ int clamp_ctx(const AttnTreeParams &p, int i, int n) {
  return max(0, min(p.ctx_len[i], min(p.max_ctx, p.Cmax - n)));
}
__device__ __forceinline__ Span make_span(const AttnTreeParams &p, int ctx, int n) {
  Span s;
  s.ctx = ctx;
  s.n = n;
  s.A = s.W0 = 0;
  const int L = ctx + n;
  if (p.window > 0 && ctx + 1 > p.window) {
    s.W0 = (ctx + 1 - p.window) / kKeys;
    s.A = min((min(p.sinks, L) + kKeys - 1) / kKeys, s.W0);
  }
  s.U = n > 0 ? s.A + (L + kKeys - 1) / kKeys - s.W0 : 0;
  return s;
}
__device__ __forceinline__ int units_of(const AttnTreeParams &p, int i) {
  const int n = clamp_nodes(p, i);
  return make_span(p, clamp_ctx(p, i, n), n).U;
}
__device__ __forceinline__ int unit_base(const Span &s, int u) { return (u < s.A ? u : u - s.A + s.W0) * kKeys; }
// Whether every row sees all of the unit's keys.
__device__ __forceinline__ bool unit_plain(const AttnTreeParams &p, const Span &s, int base) {
  return base + kKeys <= s.ctx &&
         (p.window <= 0 || base >= s.ctx + s.n - p.window || base + kKeys <= p.sinks);
}

// First unit of CTA c's range, T units over G CTAs; and the CTA that has unit u.
__device__ __forceinline__ long long range_start(long long T, int G, int c) { return (long long)c * T / G; }
__device__ __forceinline__ int range_of(long long T, int G, long long u) {
  return static_cast<int>(((u + 1) * G + T - 1) / T - 1);
}

// Warp-collective: units of all pairs.
__device__ long long all_units(const AttnTreeParams &p, int lane) {
  long long s = 0;
  for (int i = lane; i < p.nb; i += 32) s += units_of(p, i);
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s * (p.Hkv * p.groups);
}

// Warp-collective: the sequence that has unit u0 of all, and the units before it; -1: none.
__device__ int find_sequence(const AttnTreeParams &p, long long u0, int lane, long long *before) {
  const int per = p.Hkv * p.groups;
  long long base = 0;
  for (int b = 0; b < p.nb; b += 32) {
    const int i = b + lane;
    const long long own = i < p.nb ? (long long)per * units_of(p, i) : 0;
    long long v = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, i < p.nb && base + v > u0);
    if (hit) {
      const int l = __ffs(hit) - 1;
      *before = base + __shfl_sync(0xffffffffu, v - own, l);
      return b + l;
    }
    base += __shfl_sync(0xffffffffu, v, 31);
  }
  return -1;
}

constexpr int kSeqCache = 64;  // sequences whose lengths a CTA keeps in shared memory

struct Walk {
  int pair, unit, seg, seg_unit0, left;
  int stage;   // units before this one
  Span s;
};
__device__ __forceinline__ Span walk_span(const AttnTreeParams &p, const int2 *seqs, int i) {
  int2 v;
  if (i < kSeqCache) {
    v = seqs[i];
  } else {
    v.y = clamp_nodes(p, i);
    v.x = clamp_ctx(p, i, v.y);
  }
  return make_span(p, v.x, v.y);
}
__device__ __forceinline__ bool walk_first(const Walk &w) { return w.unit == w.seg_unit0; }
__device__ __forceinline__ bool walk_last(const Walk &w) { return w.left == 1 || w.unit == w.s.U - 1; }
__device__ __forceinline__ void walk_next(Walk &w, const AttnTreeParams &p, const int2 *seqs) {
  ++w.stage;
  --w.left;
  if (++w.unit == w.s.U) {
    ++w.pair;
    w.unit = 0;
    w.seg_unit0 = 0;
    ++w.seg;
    if (w.left > 0) {
      const int per = p.Hkv * p.groups;
      int i = w.pair / per;
      if (w.pair % per == 0) {
        w.s = walk_span(p, seqs, i);
        while (w.s.U == 0 && i + 1 < p.nb) {  // sequences without rows have no units
          w.s = walk_span(p, seqs, ++i);
          w.pair += per;
        }
      }
    }
  }
}

// Bits [0, k).
__device__ __forceinline__ unsigned long long low_bits(int k) {
  return k >= 64 ? ~0ull : k <= 0 ? 0ull : (1ull << k) - 1;
}

// The nodes that node j sees, itself among them, and its depth.
__device__ __forceinline__ unsigned long long line_of(const AttnTreeParams &p, const Span &s, int i, int j, int *depth) {
  unsigned long long seen = 0;
  if (p.parent == nullptr) {
    *depth = j;
    seen = low_bits(j + 1);
    if (p.window > 0) seen &= ~low_bits(j + 1 - p.window) | low_bits(p.sinks - s.ctx);
    return seen;
  }
  const int *parent = p.parent + (long long)i * p.m;
  int d = 0;
  bool bad = false;
  for (int a = j;; ++d) {  // parents lie below their nodes
    if (p.window <= 0 || d < p.window) seen |= 1ull << a;
    const int up = parent[a];
    if (a == 0 || up < 0 || up >= a) {
      bad = a == 0 ? up != -1 : true;
      break;
    }
    a = up;
  }
  *depth = d;
  if (p.window > 0 && p.sinks > s.ctx) {  // nodes among the first rows
    int a = j;
    for (int e = d;; --e) {
      if (s.ctx + e < p.sinks) seen |= 1ull << a;
      if (e == 0) break;
      a = parent[a];
    }
  }
  if (bad) flag_status(p.status, kStatusCheck);
  return seen;
}

template <int HD, int NQ, bool TWO>
__global__ void __launch_bounds__(Roles<NQ>::THREADS, 1) attn_tree_kernel(const __grid_constant__ AttnTreeParams p) {
  using C = Cfg<HD, TWO>;
  using Ro = Roles<NQ>;
  constexpr int ST = C::STAGES;
  constexpr int HT = Ro::HALF;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint8_t *sQ = smem;
  uint8_t *sKV = smem + C::OFF_KV;
  uint64_t *kv_full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
  uint64_t *kv_empty = kv_full + ST;    // the last product of the stage, and the cleaner
  uint64_t *clean = kv_empty + ST;      // masked units: values zeroed, their keys noted
  uint64_t *s_full = clean + ST;        // [2]
  uint64_t *s_empty = s_full + 2;       // [2]
  uint64_t *p_full = s_empty + 2;       // [4]: P of step j in buffer j % 4
  uint64_t *p_empty = p_full + 4;       // [4]: its product done
  uint64_t *q_full = p_empty + 4;
  uint64_t *q_empty = q_full + 1;
  uint64_t *o_free = q_empty + 1;       // [2]: O read at a segment's end (one tile: both by half 0)
  uint64_t *ml_ready = o_free + 2;      // one tile: half 1's maximum and sum written
  uint64_t *mma_done = ml_ready + 1;    // [2]
  uint64_t *poison = mma_done + 2;      // [ST] keys of the stage whose values were not finite
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(poison + ST);
  int *sched = reinterpret_cast<int *>(tmem_slot + 1);  // pair, unit, count
  int2 *seqs = reinterpret_cast<int2 *>(smem + C::OFF_SEQ);
  float2 *ml1 = reinterpret_cast<float2 *>(smem + C::OFF_ML);
  static_assert((4 * ST + 2 + 2 + 4 + 4 + 2 + 2 + 1 + 2) * 8 + 16 <= 512, "barrier region");
  static_assert(kSeqCache * 8 <= 512, "lengths");

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv;
  const int R = p.npt * G;  // rows of a full tile

  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 2);
      mbar_init(&clean[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&s_empty[b], HT);
      mbar_init(&o_free[b], HT);
      mbar_init(&mma_done[b], 1);
    }
    for (int b = 0; b < 4; ++b) {
      mbar_init(&p_full[b], HT);
      mbar_init(&p_empty[b], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(ml_ready, HT);
    fence_mbar_init();
  }
  if (warp == Ro::PRODUCER && lane == 0) {
    tma_prefetch_desc(&p.tmQ);
    tma_prefetch_desc(&p.tmK);
    tma_prefetch_desc(&p.tmV);
  }
  if (warp == Ro::S) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (warp < NQ) {
    // rows that no copy fills stay zero
    for (int a = 0; a < C::TILES * C::ATOMS; ++a)
      for (int e = R * 8 + static_cast<int>(threadIdx.x); e < kTileRows * 8; e += HT)
        *reinterpret_cast<uint4 *>(sQ + a * C::ATOM_Q + e * 16) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  griddep_wait();  // the lengths may come from the launch before
  if (threadIdx.x == 0) griddep_launch();
  if (warp == Ro::PRODUCER) {
    for (int i = lane; i < p.nb && i < kSeqCache; i += 32) {
      const int n = clamp_nodes(p, i);
      seqs[i] = make_int2(clamp_ctx(p, i, n), n);
    }
    const long long T = all_units(p, lane);
    const int Ge = T < p.grid ? static_cast<int>(T) : p.grid;
    int count = 0, pair0 = 0, unit0 = 0;
    if (static_cast<int>(blockIdx.x) < Ge) {
      const long long u0 = range_start(T, Ge, blockIdx.x);
      count = static_cast<int>(range_start(T, Ge, blockIdx.x + 1) - u0);
      long long before = 0;
      const int i = find_sequence(p, u0, lane, &before);
      if (i < 0) {
        count = 0;
      } else {
        const int U = units_of(p, i);
        const int off = static_cast<int>(u0 - before);
        pair0 = i * p.Hkv * p.groups + off / U;
        unit0 = off % U;
      }
    }
    if (lane == 0) {
      sched[0] = pair0;
      sched[1] = unit0;
      sched[2] = count;
    }
  }
  if (warp == Ro::CLEAN && blockIdx.x == 0) {
    bool bad = false;  // lengths out of range, reported once a launch
    for (int i = lane; i < p.nb; i += 32) {
      const int n = p.n_rows ? p.n_rows[i] : p.m, c = p.ctx_len[i];
      bad |= n < 0 || n > p.m || c < 0 || c > p.max_ctx || c > p.Cmax - clamp_nodes(p, i);
    }
    if (bad) flag_status(p.status, kStatusCheck);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int nunits = sched[2];
  const int per = p.Hkv * p.groups;
  Walk w;
  w.pair = sched[0];
  w.unit = w.seg_unit0 = sched[1];
  w.seg = 0;
  w.left = nunits;
  w.stage = 0;
  if (nunits > 0) w.s = walk_span(p, seqs, w.pair / per);

  if (warp == Ro::PRODUCER) {
    if (lane == 0 && nunits > 0 && !p.stall) {
      // K and V of one pair are read by its groups of tiles one after another
      const uint64_t pol_kv = p.groups > 1 ? policy_evict_last() : policy_evict_first();
      const uint64_t pol_q = policy_evict_last();
      bool ok = true;
      int q_loads = 0, loads = 0;
      for (; w.left > 0; walk_next(w, p, seqs)) {
        const int i = w.pair / per, g = w.pair % per / p.groups, grp = w.pair % p.groups;
        const int base = unit_base(w.s, w.unit);
        int row;
        if (p.page_table == nullptr) {
          row = p.layer_row0 + (i * p.Hkv + g) * p.Cmax + base;
        } else {
          int pg = p.page_table[(long long)i * p.pages_per_seq + base / kKeys];
          if (pg < 0 || pg >= p.num_pages) {
            flag_status(p.status, kStatusCheck);
            pg = 0;
          }
          row = p.layer_row0 + (pg * p.Hkv + g) * kPageRows;
        }
        if (walk_first(w)) {
          if (w.seg > 0 && !mbar_wait(q_empty, (w.seg - 1) & 1, p.max_spin)) {
            ok = false;
            break;
          }
          const int node0 = grp * C::TILES * p.npt;
          const int tiles = TWO && node0 + p.npt < p.m ? 2 : 1;  // a last group may have one tile
          mbar_arrive_expect_tx(q_full, static_cast<uint32_t>(tiles * C::ATOMS * R * 128));
          for (int h = 0; h < tiles; ++h)
#pragma unroll
            for (int a = 0; a < C::ATOMS; ++a)
              tma_load_3d(sQ + h * C::Q_TILE + a * C::ATOM_Q, &p.tmQ, q_full, a * 64, g * G,
                          i * p.m + node0 + h * p.npt, pol_q);
          ++q_loads;
        }
        const int st = w.stage % ST;
        if (w.stage >= ST && !mbar_wait(&kv_empty[st], ((w.stage / ST) & 1) ^ 1, p.max_spin)) {
          ok = false;
          break;
        }
        uint8_t *kt = sKV + st * C::STAGE;
        mbar_arrive_expect_tx(&kv_full[st], C::STAGE);
        tma_load_3d(kt, &p.tmK, &kv_full[st], 0, row, 0, pol_kv);
        tma_load_3d(kt + C::KV_TILE, &p.tmV, &kv_full[st], 0, row, 0, pol_kv);
        loads = w.stage + 1;
      }
      if (!ok) flag_status(p.status, kStatusTimeout);
      for (int k = max(0, loads - ST); k < loads; ++k)  // every copy lands before the CTA ends
        mbar_wait(&kv_full[k % ST], (k / ST) & 1, kDrainSpin);
      if (q_loads > 0) mbar_wait(q_full, (q_loads - 1) & 1, kDrainSpin);
    }
  } else if (warp == Ro::S) {
    if (lane == 0 && nunits > 0) {
      constexpr uint32_t id_s = idesc_bf16_f32(kTileRows, kKeys);
      const uint64_t q_desc0 = sw128_kmajor_desc(smem_u32(sQ));
      const uint64_t k_desc0 = sw128_kmajor_desc(smem_u32(sKV));
      bool ok = true;
      int step = 0;
      for (; w.left > 0 && ok; walk_next(w, p, seqs)) {
        const int st = w.stage % ST;
        if (walk_first(w) && !mbar_wait(q_full, w.seg & 1, p.max_spin)) ok = false;
        if (ok && !mbar_wait(&kv_full[st], (w.stage / ST) & 1, p.max_spin)) ok = false;
#pragma unroll
        for (int h = 0; h < C::TILES; ++h) {
          const int sb = step & 1;
          if (ok && step >= 2 && !mbar_wait(&s_empty[sb], ((step >> 1) - 1) & 1, p.max_spin)) ok = false;
          if (!ok) break;
          tc_fence_after();
          const uint64_t qd = q_desc0 + static_cast<uint64_t>((h * C::Q_TILE) >> 4);
          const uint64_t kd = k_desc0 + static_cast<uint64_t>((st * C::STAGE) >> 4);
          const uint32_t d_s = tmem_base + C::S_COL + sb * kKeys;
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk)
            tc_mma_bf16(d_s, qd + static_cast<uint64_t>(((kk >> 2) * C::ATOM_Q + (kk & 3) * 32) >> 4),
                        kd + static_cast<uint64_t>(((kk >> 2) * C::ATOM_KV + (kk & 3) * 32) >> 4), id_s,
                        kk > 0 ? 1u : 0u);
          tc_commit(&s_full[sb]);
          ++step;
        }
        if (ok && walk_last(w)) tc_commit(q_empty);
      }
      if (!ok) flag_status(p.status, kStatusTimeout);
      tc_commit(&mma_done[0]);  // every product completes before tensor memory is freed
      mbar_wait(&mma_done[0], 0, kDrainSpin);
    }
  } else if (warp == Ro::PV) {
    if (lane == 0 && nunits > 0) {
      constexpr uint32_t id_pv = idesc_bf16_f32(kTileRows, HD) | kIdescBMajorMN;
      const uint64_t v_desc0 = sw128_mnmajor_desc(smem_u32(sKV + C::KV_TILE), C::ATOM_KV);
      bool ok = true;
      int step = 0, first = 0;
      for (; w.left > 0 && ok; walk_next(w, p, seqs)) {
        const int st = w.stage % ST;
        if (walk_first(w)) first = step;
#pragma unroll
        for (int h = 0; h < C::TILES; ++h) {
          const int half = step & 1, pb = step & 3;
          const bool start = step < first + 2;  // the half's first unit of the segment
          if (!mbar_wait(&p_full[pb], (step >> 2) & 1, p.max_spin)) ok = false;
          if (ok && start && w.seg > 0 && !mbar_wait(&o_free[TWO ? half : 0], (w.seg - 1) & 1, p.max_spin)) ok = false;
          if (!ok) break;
          tc_fence_after();
          const uint64_t vd = v_desc0 + static_cast<uint64_t>((st * C::STAGE) >> 4);
          const uint32_t d_o = tmem_base + C::O_COL + half * HD;
          const uint32_t a_p = tmem_base + C::P_COL + pb * 32;
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            tc_mma_bf16_tmem_a(d_o, a_p + kk * 8, vd + static_cast<uint64_t>((kk * 16 * 128) >> 4), id_pv,
                               (!start || kk > 0) ? 1u : 0u);
          tc_commit(&p_empty[pb]);
          ++step;
        }
        if (ok) tc_commit(&kv_empty[st]);
      }
      if (!ok) flag_status(p.status, kStatusTimeout);
      tc_commit(&mma_done[1]);
      mbar_wait(&mma_done[1], 0, kDrainSpin);
    }
  } else if (warp == Ro::CLEAN) {
    // follows every stage, in order, so that it never takes one phase of a barrier for another
    bool ok = true;
    for (; w.left > 0; walk_next(w, p, seqs)) {
      const int st = w.stage % ST;
      ok = mbar_wait_warp(&kv_full[st], (w.stage / ST) & 1, p.max_spin);
      if (!ok) break;
      const int base = unit_base(w.s, w.unit);
      if (!unit_plain(p, w.s, base)) {
        const int nv = w.s.ctx + w.s.n - base;  // keys of the unit that exist
        uint8_t *vt = sKV + st * C::STAGE + C::KV_TILE;
        unsigned long long found = 0;
#pragma unroll 4
        for (int e = lane; e < C::KV_TILE / 16; e += 32) {
          const int key = (e >> 3) % kKeys;  // 16-byte pieces, eight of a row and atom
          uint4 *at = reinterpret_cast<uint4 *>(vt + e * 16);
          if (key >= nv) {
            *at = make_uint4(0, 0, 0, 0);
            continue;
          }
          uint4 x = *at;
          uint32_t *word = &x.x;
          bool odd = false;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const bool lo = (word[q] & 0x7F80u) == 0x7F80u, hi = (word[q] & 0x7F800000u) == 0x7F800000u;
            word[q] &= (lo ? 0xFFFF0000u : 0xFFFFFFFFu) & (hi ? 0x0000FFFFu : 0xFFFFFFFFu);
            odd |= lo | hi;
          }
          if (odd) {
            *at = x;
            found |= 1ull << key;
          }
        }
        fence_proxy_async_smem();
        const uint32_t f0 = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(found));
        const uint32_t f1 = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(found >> 32));
        if (lane == 0) {
          poison[st] = static_cast<unsigned long long>(f1) << 32 | f0;
          mbar_arrive(&clean[st]);
        }
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(&kv_empty[st]);
    }
    if (!ok && lane == 0) flag_status(p.status, kStatusTimeout);
  } else if ((warp & 3) < NQ) {
    // ---------------- softmax
    const int half = warp >> 2;
    const int q = warp & 3;
    const int r = q * 32 + lane;
    const int jr = r / G, hq = r - jr * G;  // node of the tile and head of its group
    const uint32_t trow = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    const uint32_t o_mine = trow + C::O_COL + half * HD;
    const float sl2 = rsqrtf(static_cast<float>(HD)) * 1.4426950408889634f;
    float m_run = -FLT_MAX, l_run = 0.f;
    unsigned long long line = 0;  // nodes this row sees
    int lo = 0;                   // its first context row behind the sinks
    bool have_line = false, real = false, warp_real = false;
    uint32_t clean_phase = 0;
    bool ok = true;
    int step = 0, first = 0, node = 0;
    for (; w.left > 0 && ok; walk_next(w, p, seqs), step += C::TILES) {
      const int st = w.stage % ST;
      if (walk_first(w)) {
        first = step;
        m_run = -FLT_MAX;
        l_run = 0.f;
        have_line = false;
        const int grp = w.pair % p.groups;
        const int node0 = (grp * C::TILES + (TWO ? half : 0)) * p.npt;
        node = node0 + jr;
        real = r < R && node < w.s.n;
        warp_real = __any_sync(0xffffffffu, real);
      }
      const int base = unit_base(w.s, w.unit);
      const bool masked = !unit_plain(p, w.s, base);
      const uint32_t cph = clean_phase >> st & 1;
      if (masked) clean_phase ^= 1u << st;
      const int mine = TWO ? step + half : step;  // this half's step of the unit
      if (TWO || (step & 1) == half) {
        const bool start = mine < first + 2;
        const int pb = mine & 3;
        ok = mbar_wait_warp(&s_full[half], (mine >> 1) & 1, p.max_spin);
        if (!ok) break;
        tc_fence_after();
        float sv[kKeys];
        if (warp_real) tmem_ld64(trow + C::S_COL + half * kKeys, sv);
        tc_fence_before();
        mbar_arrive(&s_empty[half]);

        unsigned long long bad = 0;
        if (masked) {
          if (!have_line) {
            int depth = 0;
            line = real ? line_of(p, w.s, w.pair / per, node, &depth) : 0;
            lo = p.window > 0 ? w.s.ctx + depth - p.window + 1 : 0;
            have_line = true;
          }
          unsigned long long keep = low_bits(w.s.ctx - base);
          if (p.window > 0) keep &= ~low_bits(lo - base) | low_bits(p.sinks - base);
          const int sh = base - w.s.ctx;  // key k of the unit is node k + sh
          keep |= sh >= 64 || sh <= -64 ? 0ull : sh >= 0 ? line >> sh : line << -sh;
#pragma unroll
          for (int c = 0; c < kKeys; ++c) sv[c] = keep >> c & 1 ? sv[c] : -INFINITY;
          ok = mbar_wait_warp(&clean[st], cph, p.max_spin);
          if (!ok) break;
          bad = poison[st] & keep;
        }
        bool need = false;
        float alpha = 1.f;
        if (warp_real) {
          float m8[8];
#pragma unroll
          for (int a = 0; a < 8; ++a) m8[a] = max3(sv[a], sv[a + 8], sv[a + 16]);
#pragma unroll
          for (int a = 0; a < 8; ++a) m8[a] = max3(m8[a], sv[a + 24], sv[a + 32]);
#pragma unroll
          for (int a = 0; a < 8; ++a) m8[a] = max3(m8[a], sv[a + 40], sv[a + 48]);
#pragma unroll
          for (int a = 0; a < 8; ++a) m8[a] = fmaxf(m8[a], sv[a + 56]);
          const float mx = max3(max3(m8[0], m8[1], m8[2]), max3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
          need = real && (mx - m_run) * sl2 > kGrowLog2;
          if (need) {
            alpha = ex2((m_run - mx) * sl2);
            m_run = mx;
            l_run *= alpha;
          }
          if (bad) {
#pragma unroll
            for (int c = 0; c < kKeys; ++c) sv[c] = bad >> c & 1 ? __int_as_float(0x7fffffff) : sv[c];
          }
        }
        if (!start && __any_sync(0xffffffffu, need)) {
          // O *= alpha once the half's product before is done
          ok = mbar_wait_warp(&p_empty[(mine - 2) & 3], ((mine - 2) >> 2) & 1, p.max_spin);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int cc = 0; cc < HD / 32; ++cc) {
            float ov[32];
            tmem_ld32(o_mine + cc * 32, ov);
#pragma unroll
            for (int c = 0; c < 32; ++c) ov[c] *= alpha;
            tmem_st32(o_mine + cc * 32, ov);
          }
        }
        ok = mine < 4 || mbar_wait_warp(&p_empty[pb], ((mine >> 2) - 1) & 1, p.max_spin);
        if (!ok) break;
        if (warp_real) {
          uint32_t pk[kKeys / 2];
          float ls[4] = {0.f, 0.f, 0.f, 0.f};
          const float mb = m_run * sl2;
#pragma unroll
          for (int c = 0; c < kKeys; c += 2) {
            const float p0 = ex2(fmaf(sv[c], sl2, -mb));
            const float p1 = ex2(fmaf(sv[c + 1], sl2, -mb));
            ls[(c >> 1) & 3] += p0 + p1;
            pk[c >> 1] = real ? pack_bf16x2(p0, p1) : 0u;
          }
          l_run += (ls[0] + ls[1]) + (ls[2] + ls[3]);
          tmem_st32_raw(trow + C::P_COL + pb * 32, pk);
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(&p_full[pb]);
      }
      if (!walk_last(w)) continue;

      // ---------------- a segment's end
      const int seg = w.seg;
      const bool whole = w.seg_unit0 == 0 && w.unit == w.s.U - 1;
      const int i = w.pair / per, g = w.pair % per / p.groups;
      const int slot = 2 * static_cast<int>(blockIdx.x) + (seg > 0);
      float M, L, a0 = 1.f, a1 = 0.f;
      bool has0 = true, has1 = false;
      if (TWO) {
        ok = mbar_wait_warp(&p_empty[mine & 3], (mine >> 2) & 1, p.max_spin);
        if (!ok) break;
        tc_fence_after();
        M = m_run;
        L = l_run;
      } else {
        // the halves' last steps of the segment, -1: none
        const int e0 = (step & 1) == 0 ? step : step - 1, e1 = (step & 1) ? step : step - 1;
        const int last0 = e0 >= first ? e0 : -1, last1 = e1 >= first ? e1 : -1;
        if (half == 1) {
          ok = seg == 0 || mbar_wait_warp(&o_free[0], (seg - 1) & 1, p.max_spin);  // half 0 read the one before
          if (ok && last1 >= 0) ok = mbar_wait_warp(&p_empty[last1 & 3], (last1 >> 2) & 1, p.max_spin);
          if (!ok) break;
          ml1[r] = last1 >= 0 ? make_float2(m_run, l_run) : make_float2(-FLT_MAX, 0.f);
          tc_fence_before();
          mbar_arrive(ml_ready);
          continue;
        }
        ok = last0 < 0 || mbar_wait_warp(&p_empty[last0 & 3], (last0 >> 2) & 1, p.max_spin);
        if (ok) ok = mbar_wait_warp(ml_ready, seg & 1, p.max_spin);
        if (!ok) break;
        tc_fence_after();
        const float2 o1 = ml1[r];
        has0 = last0 >= 0;
        has1 = last1 >= 0;
        const float m0 = has0 ? m_run : -FLT_MAX;
        M = fmaxf(m0, o1.x);
        a0 = has0 ? ex2((m0 - M) * sl2) : 0.f;
        a1 = has1 ? ex2((o1.x - M) * sl2) : 0.f;
        L = (has0 ? l_run * a0 : 0.f) + (has1 ? o1.y * a1 : 0.f);
      }
      if (warp_real) {
        const float inv = 1.0f / L;
        const int prow = slot * p.part_rows + (TWO ? half * kTileRows : 0) + r;
#pragma unroll 1
        for (int cc = 0; cc < HD / 32; ++cc) {
          float ov[32];
          if (TWO) {
            tmem_ld32(o_mine + cc * 32, ov);
          } else {
            float o1v[32];
            if (has0) tmem_ld32(trow + C::O_COL + cc * 32, ov);
            if (has1) tmem_ld32(trow + C::O_COL + HD + cc * 32, o1v);
#pragma unroll
            for (int c = 0; c < 32; ++c) ov[c] = (has0 ? ov[c] * a0 : 0.f) + (has1 ? o1v[c] * a1 : 0.f);
          }
          if (!real) continue;
          if (whole) {
            uint16_t *dst = p.o + (((long long)i * p.m + node) * p.Hq + g * G + hq) * HD + cc * 32;
#pragma unroll
            for (int v = 0; v < 4; ++v)
              reinterpret_cast<uint4 *>(dst)[v] =
                  make_uint4(pack_bf16x2(ov[8 * v] * inv, ov[8 * v + 1] * inv),
                             pack_bf16x2(ov[8 * v + 2] * inv, ov[8 * v + 3] * inv),
                             pack_bf16x2(ov[8 * v + 4] * inv, ov[8 * v + 5] * inv),
                             pack_bf16x2(ov[8 * v + 6] * inv, ov[8 * v + 7] * inv));
          } else {
            float *dst = p.part_o + (long long)prow * HD + cc * 32;
#pragma unroll
            for (int v = 0; v < 8; ++v)
              reinterpret_cast<float4 *>(dst)[v] = make_float4(ov[4 * v], ov[4 * v + 1], ov[4 * v + 2], ov[4 * v + 3]);
          }
        }
        if (real && !whole) *reinterpret_cast<float2 *>(p.part_ml + (long long)prow * 2) = make_float2(M, L);
      }
      tc_fence_before();
      mbar_arrive(&o_free[TWO ? half : 0]);
    }
    if (!ok) flag_status(p.status, kStatusTimeout);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == Ro::S) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// Joins the partials of a pair that several CTAs share, in CTA order. CTA x of this grid stands for the
// boundary at the start of range x + 1, and joins the pair that is cut there for the first time; one warp
// a row, hd/32 values a lane.
constexpr int kMergeWarps = 8;

template <int HD>
__global__ void __launch_bounds__(kMergeWarps * 32) attn_tree_merge_kernel(const __grid_constant__ AttnTreeParams p) {
  constexpr int E = HD / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv, R = p.npt * G, per = p.Hkv * p.groups;
  const int r = blockIdx.y * kMergeWarps + warp;  // row of the slot
  // This grid's end has to imply the attention's: CTA (0, 0) always waits for it. The lengths are older than
  // the attention, which lets this launch begin only once it waited itself.
  const bool anchor = blockIdx.x == 0 && blockIdx.y == 0;
  const long long T = all_units(p, lane);
  const int Ge = T < p.grid ? static_cast<int>(T) : p.grid;
  const int c0 = blockIdx.x;
  int i = -1, c1 = 0, pair = 0, first_slot = 0;
  if (c0 + 1 < Ge) {
    const long long u = range_start(T, Ge, c0 + 1);
    long long before = 0;
    i = find_sequence(p, u, lane, &before);
    if (i >= 0) {
      const int U = units_of(p, i);
      const int k = static_cast<int>((u - before) / U);
      const long long start = before + (long long)k * U;
      pair = i * per + k;
      // cut here, and not in an earlier range
      if (start == u || range_of(T, Ge, start) != c0) i = -1;
      c1 = range_of(T, Ge, start + U - 1);
      first_slot = 2 * c0 + (range_start(T, Ge, c0) != start);
    }
  }
  int node = 0, hq = 0;
  if (i >= 0) {
    const int tile = r / kTileRows, rt = r % kTileRows;
    const int tiles = p.part_rows > kTileRows ? 2 : 1;
    const int jr = rt / G;
    hq = rt - jr * G;
    node = (pair % p.groups * tiles + tile) * p.npt + jr;
    if (rt >= R || node >= clamp_nodes(p, i)) i = -1;
  }
  if (i < 0) {
    if (anchor) griddep_wait();
    return;
  }
  griddep_wait();
  griddep_launch();
  const float sl2 = rsqrtf(static_cast<float>(HD)) * 1.4426950408889634f;
  float M = -FLT_MAX, L = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int c = c0; c <= c1; ++c) {
    const long long row = (long long)(c == c0 ? first_slot : 2 * c) * p.part_rows + r;
    const float2 ml = *reinterpret_cast<const float2 *>(p.part_ml + row * 2);
    float v[E];
    const float *src = p.part_o + row * HD + lane * E;
    if constexpr (E == 4) {
      const float4 x = *reinterpret_cast<const float4 *>(src);
      v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
      const float2 x = *reinterpret_cast<const float2 *>(src);
      v[0] = x.x, v[1] = x.y;
    }
    const float Mn = fmaxf(M, ml.x);
    const float a_old = exp2f((M - Mn) * sl2), a_new = exp2f((ml.x - Mn) * sl2);
    L = L * a_old + ml.y * a_new;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * a_old + v[e] * a_new;
    M = Mn;
  }
  const float inv = 1.0f / L;
  const int g = pair % per / p.groups;
  uint16_t *dst = p.o + (((long long)i * p.m + node) * p.Hq + g * G + hq) * HD + lane * E;
  if constexpr (E == 4)
    *reinterpret_cast<uint2 *>(dst) =
        make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t *>(dst) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
}

template <int HD, int NQ, bool TWO>
cudaError_t launch(const AttnTreeParams &p, cudaStream_t s) {
  using C = Cfg<HD, TWO>;
  static const cudaError_t configured = cudaFuncSetAttribute(
      attn_tree_kernel<HD, NQ, TWO>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
  if (configured != cudaSuccess) return configured;
  cudaError_t e = launch_pdl(attn_tree_kernel<HD, NQ, TWO>, dim3(p.grid), dim3(Roles<NQ>::THREADS), C::SMEM, s, p);
  if (e != cudaSuccess) return e;
  const int rows = TWO ? 2 * kTileRows : p.npt * (p.Hq / p.Hkv);
  return launch_pdl(attn_tree_merge_kernel<HD>, dim3(p.grid, (rows + kMergeWarps - 1) / kMergeWarps),
                    dim3(kMergeWarps * 32), 0, s, p);
}

template <int HD>
cudaError_t launch_form(const AttnTreeParams &p, cudaStream_t s) {
  const int R = p.npt * (p.Hq / p.Hkv);
  if (p.part_rows > kTileRows) return launch<HD, 4, true>(p, s);
  if (R > 64) return launch<HD, 4, false>(p, s);
  return R > 32 ? launch<HD, 2, false>(p, s) : launch<HD, 1, false>(p, s);
}

}  // namespace

// Nodes per tile and groups of tiles for m nodes of G query heads: one tile where all rows fit, else
// pairs of tiles of about the same size.
void attention_tree_plan(int m, int G, int *npt, int *groups, int *part_rows) {
  const int most = kTileRows / G;  // nodes of a tile
  if (m <= most) {
    *npt = m;
    *groups = 1;
    *part_rows = kTileRows;
    return;
  }
  *groups = (m + 2 * most - 1) / (2 * most);
  *npt = (m + 2 * *groups - 1) / (2 * *groups);
  *part_rows = 2 * kTileRows;
}

cudaError_t launch_attention_tree(const AttnTreeParams &p, cudaStream_t s) {
  switch (p.hd) {
    case 64: return launch_form<64>(p, s);
    case 128: return launch_form<128>(p, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace df
