// Attention of a tree of drafted tokens over the bf16 caches, with a sliding window and first rows
// ("sinks") that stay visible, on the tcgen05 tensor cores. For node j of sequence i (position
// ctx + depth(j)) and query head h of kv head g = h / (Hq/Hkv):
//   o = softmax(q K^T / sqrt(hd)) V over
//     the context rows p < ctx with  no window,  or p > ctx + depth(j) - window,  or p < sinks
//     the rows ctx + a of the nodes a from j up to the root, by the same rule at ctx + depth(a)
// (KV injection and the attention equations of "DFlash 投机解码：块扩散草稿与 KV 注入", 二; the pages verify
// one path, a tree holds several). A chain of nodes is causal attention, one node the decode step.
//
// Bound: the visible K and V rows, read once. Query rows R = (Hq/Hkv) * m of a kv head are the rows of M = 128 MMAs,
// in one of two forms:
//   one tile (R <= 128)   two halves of softmax warps take units of 64 keys in turn, each with its own
//                         running maximum, sum and O, joined at the end of a segment. 64 sequences of 1024 to 8191
//                         rows, 32 heads over 8: one token 178 us and 6.8 TB/s, trees of 16 nodes 192 us and 6.4 TB/s.
//   two tiles (R > 128)   both halves work on every unit, each for its own tile of up to 128 rows: K and
//                         V are read once for 256 rows. More rows take further groups of two tiles. Bound by the
//                         chain of a unit, S, softmax, product, and what the products of both tiles take from
//                         shared memory: 262147 rows under 64 nodes 194 us in short graph runs, 1.42 PFLOP/s and
//                         5.5 TB/s; called for seconds on end, at the power limit, 226 us, 1.21 PFLOP/s and 4.7 TB/s;
//                         with each tile's rows in a CTA of its own, K and V read twice, 314 us.
// A (sequence, kv head, group) is a pair; the visible units of all pairs are cut into equal ranges, one
// per CTA (one CTA per SM; two one-tile CTAs an SM, each with half the stages: 206 us for the trees above).
// The run of one pair inside a range is a segment: it writes the output, or if the pair goes on in another
// CTA an unnormalised partial (only a range's first and last segment can be one: two slots a CTA), which
// attn_tree_merge_kernel joins in CTA order. With a window a pair's units are those of the sinks, then those
// from the root's first visible row on.
//
// Masks: a unit that every row sees whole takes none. The others (the window's edge, the end of the
// sinks, the tree's own rows) get a 64-bit mask a row from its node's line of ancestors. Values in
// rows that a query row does not see may be NaN or infinite: in masked units a warp of its own (the
// cleaner) zeroes such values before the product sees them and notes their keys, and the rows that see
// such a key get a NaN probability for it.
//
// One CTA: TMA producer (K and V of a unit per stage, Q tiles of the segments), S issuer (S = Q K^T into buffer
// step % 2, Q from tensor memory as far as it fits), PV issuer (O_half += P V, P from tensor memory), the cleaner, and
// the softmax warps: a thread owns a query row (its TMEM lane), keeps its maximum and sum in fp32, rounds P to bf16
// (by up to 2^-8 of each probability, the type of the values that it multiplies) and rescales O only when the row's
// maximum grew by more than 2^8, so most units need no round trip of O.
//
// Figures above are of the kernel as it is, from graphs of some thirty calls where nothing else is said; pairs of
// figures beside the code compare a step with what stood before it, as things were then.
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
};

template <int HD, int NQ, bool TWO>
struct Cfg {
  static constexpr int ATOMS = HD / 64;            // 128-byte swizzle atoms across hd
  static constexpr int ATOM_Q = (TWO ? kTileRows : NQ * 32) * 128;
  static constexpr int TILES = TWO ? 2 : 1;
  static constexpr int Q_TILE = ATOMS * ATOM_Q;
  static constexpr int ATOM_KV = kKeys * 128;
  static constexpr int KV_TILE = ATOMS * ATOM_KV;
  static constexpr int STAGE = 2 * KV_TILE;        // K, then V
  // K and V on the way, 160 to 192 KB. 64 single tokens of 128 channels: 178 us, with 160 KB 184, with K and V in
  // places of their own (K's free sooner) 182; of 64 channels 100.5 us with 12 stages, with 8 102.6.
  static constexpr int STAGES = HD == 64 ? (TWO ? 10 : 12) : TWO ? 5 : 6;
  static constexpr int BARS = HD == 64 ? 1024 : 512;  // bytes for the barriers
  static constexpr int OFF_KV = TILES * Q_TILE;
  static constexpr int OFF_BAR = OFF_KV + STAGES * STAGE;
  static constexpr int OFF_SEQ = OFF_BAR + BARS;
  static constexpr int OFF_ML = OFF_SEQ + 512;
  static constexpr size_t SMEM = OFF_ML + 2 * kTileRows * 8;
  static constexpr uint32_t S_COL = 0;             // two S buffers of 64 columns
  static constexpr uint32_t O_COL = 128;           // O of the two halves
  static constexpr uint32_t P_COL = 128 + 2 * HD;  // P of the two halves, 32 columns each
  static constexpr uint32_t Q_COL = P_COL + 64;    // the first QT tiles of Q: hd / 2 columns each
  static constexpr int QT = TWO && HD == 64 ? 2 : 1;
  static_assert(Q_COL + QT * HD / 2 <= 512, "tensor memory");
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
__device__ __forceinline__ int unit_base(const Span &s, int u) { return (u < s.A ? u : u - s.A + s.W0) * kKeys; }
// The units all of whose keys every row sees, as far as their places tell: whole ones of the sinks, and from the last
// window's edge to the tree's own rows.
struct Plain {
  int sinks, from, to;
};
__device__ __forceinline__ Plain plain_units(const AttnTreeParams &p, const Span &s) {
  Plain u = {0, 0, s.A + s.ctx / kKeys - s.W0};
  if (p.window > 0) {
    u.sinks = min(s.A, min(p.sinks, s.ctx) / kKeys);
    u.from = s.A + max(0, (max(0, s.ctx + s.n - p.window) + kKeys - 1) / kKeys - s.W0);
  }
  return u;
}
__device__ __forceinline__ bool unit_plain(const Plain &s, int u) { return u < s.sinks || (u >= s.from && u < s.to); }

constexpr int kCostFrom = 16;  // units of a CTA from which a pair's cost counts
constexpr int kSeqCache = 64;  // sequences whose lengths a CTA keeps in shared memory

__device__ __forceinline__ Span span_of(const AttnTreeParams &p, const int2 *seqs, int i) {
  int2 v;
  if (i < kSeqCache) {
    v = seqs[i];
  } else {
    v.y = clamp_nodes(p, i);
    v.x = clamp_ctx(p, i, v.y);
  }
  return make_span(p, v.x, v.y);
}

// All units of a call over its CTAs: CTA c has q or (the first r CTAs) q + 1 of them in a row. Where a CTA has
// some, a pair counts as `cost` units more, which come first: what a segment takes besides its units. Their
// number stays below 2^31: pairs of fewer than 2^31 cache rows, in up to 16 groups.
struct Split {
  int T, ctas, q, r, cost;
};
__device__ __forceinline__ int range_start(const Split &s, int c) { return c * s.q + min(c, s.r); }
__device__ __forceinline__ int range_of(const Split &s, int u) {  // the CTA that has unit u
  const int first = s.r * (s.q + 1);
  return u < first ? u / (s.q + 1) : s.r + (u - first) / s.q;
}

// Where one of these is: sequence i (-1: nowhere), kv head g, group grp, place `at` in a pair of U units.
struct Place {
  int i, g, grp, at, U;
};

// Warp-collective: the lengths of the first sequences to `seqs`, and the split.
__device__ __forceinline__ Split make_split(const AttnTreeParams &p, int2 *seqs, int lane) {
  int sum = 0, some = 0;
  for (int i = lane; i < p.nb; i += 32) {
    const int n = clamp_nodes(p, i), ctx = clamp_ctx(p, i, n);
    if (i < kSeqCache) seqs[i] = make_int2(ctx, n);
    sum += make_span(p, ctx, n).U;
    some += n > 0;
  }
  __syncwarp();
  const int per = p.Hkv * p.groups;
  Split s;
  s.T = __reduce_add_sync(0xffffffffu, sum) * per;
  s.cost = s.T >= kCostFrom * p.grid ? p.pair_cost : 0;
  s.T += __reduce_add_sync(0xffffffffu, some) * per * s.cost;
  s.ctas = max(1, min(s.T, p.grid));
  s.q = s.T / s.ctas;
  s.r = s.T - s.q * s.ctas;
  return s;
}

// Warp-collective: the place of u, 0 <= u < T.
__device__ __forceinline__ Place find_unit(const AttnTreeParams &p, const int2 *seqs, const Split &s, int u,
                                           int lane) {
  const int per = p.Hkv * p.groups;
  Place f = {-1, 0, 0, 0, 1};
  int base = 0;
  for (int b = 0; b < p.nb; b += 32) {
    const int i = b + lane;
    const int U = i < p.nb ? span_of(p, seqs, i).U : 0;
    const int all = U > 0 ? U + s.cost : 0;
    int v = all * per;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, i < p.nb && base + v > u);
    if (hit) {
      const int l = __ffs(hit) - 1;
      f.i = b + l;
      f.U = __shfl_sync(0xffffffffu, U, l);
      const int V = f.U + s.cost;
      const int off = u - base - (__shfl_sync(0xffffffffu, v, l) - V * per);
      const int k = off / V;
      f.at = off - k * V;
      f.g = k / p.groups;
      f.grp = k - f.g * p.groups;
      return f;
    }
    base += __shfl_sync(0xffffffffu, v, 31);
  }
  return f;
}

// A run of one pair's units [u0, u1) in this CTA's range: sequence i, kv head g, group grp of tiles. All
// roles go through the same segments; `left` of the range are not before its pair's, 0 behind the last one; the
// pair begins at `pos` of all units.
struct Seg {
  int i, g, grp, u0, u1, index, left, cost, pos;
  Span s;
};
__device__ __forceinline__ void seg_units(Seg &e, int at) {
  e.u0 = max(0, at - e.cost);
  e.u1 = min(e.s.U, at + e.left - e.cost);
  if (e.u1 <= e.u0) e.left = 0;  // the range ends before the pair's first unit
}
__device__ __forceinline__ bool seg_more(const Seg &e) {  // a segment follows
  return e.left - (e.s.U - e.u0 + e.cost) > e.cost;
}
// sched: sequence, kv head, group, place in the pair, length of the range; first unit, and the split's q, r and cost
__device__ __forceinline__ Seg seg_begin(const AttnTreeParams &p, const int2 *seqs, const int *sched) {
  Seg e;
  e.i = sched[0];
  e.g = sched[1];
  e.grp = sched[2];
  e.left = sched[4];
  e.cost = sched[8];
  e.index = 0;
  e.pos = sched[5] - sched[3];
  if (e.left > 0) {
    e.s = span_of(p, seqs, e.i);
    const int at = sched[3];
    seg_units(e, at);
    if (e.left > 0) e.left += min(at, e.cost);  // as if the range had begun with the pair's cost
  }
  return e;
}
__device__ __forceinline__ void seg_next(Seg &e, const AttnTreeParams &p, const int2 *seqs) {
  e.left -= e.s.U - e.u0 + e.cost;
  if (e.left <= 0) return;
  ++e.index;
  e.pos += e.s.U + e.cost;
  if (++e.grp == p.groups) {
    e.grp = 0;
    if (++e.g == p.Hkv) {
      e.g = 0;
      do {  // sequences without rows have no units
        e.s = span_of(p, seqs, ++e.i);
      } while (e.s.U == 0 && e.i + 1 < p.nb);
    }
  }
  seg_units(e, 0);
}

// A ring's next stage: its place, and the parity of its barriers.
template <int ST>
__device__ __forceinline__ void ring_next(int &st, uint32_t &ph) {
  if (++st == ST) {
    st = 0;
    ph ^= 1;
  }
}
// One arrival of a converged warp, behind what all of its lanes did.
__device__ __forceinline__ void warp_arrive(uint64_t *bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// One lane of a converged warp, always the same. The operands of the products that it issues stay in uniform registers:
// two tiles' 24 products of a unit go out in 1150 cycles, from a thread of its own in 1410 (262147 rows under 64 nodes,
// short graph runs: 217 us, so 191).
__device__ __forceinline__ bool elect_one() {
  uint32_t mine;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(mine));
  return mine != 0;
}

// Bits [0, k).
__device__ __forceinline__ unsigned long long low_bits(int k) {
  return k >= 64 ? ~0ull : k <= 0 ? 0ull : (1ull << k) - 1;
}

// Warp-collective: the nodes that this lane's node j sees, itself among them, and its depth (j < 0: none). up0 and
// up1 of lane k are the parents of nodes k and k + 32.
__device__ __forceinline__ unsigned long long line_of(const AttnTreeParams &p, const Span &s, int j, int up0, int up1,
                                                      int lane, int *depth) {
  if (p.parent == nullptr) {
    *depth = max(j, 0);
    unsigned long long seen = low_bits(j + 1);
    if (p.window > 0) seen &= ~low_bits(j + 1 - p.window) | low_bits(p.sinks - s.ctx);
    return seen;
  }
  if (p.window <= 0 || p.window >= kTreeMax) {  // all of them: a line grows by its end's line, in log2 of the depth
    const int k1 = lane + 32;
    const bool top0 = up0 < 0 || up0 >= lane, top1 = up1 < 0 || up1 >= k1;
    const bool bad = (lane < s.n && top0 && (lane != 0 || up0 != -1)) || (k1 < s.n && top1);
    if (bad) flag_status(p.status, kStatusCheck);
    int end0 = top0 ? lane : up0, end1 = top1 ? k1 : up1;
    uint32_t line0 = 1u << lane, low1 = 0, high1 = 1u << lane;  // nodes below 32 have their line there
    bool grew;
    do {
      const uint32_t to0 = __shfl_sync(0xffffffffu, line0, end0), next0 = __shfl_sync(0xffffffffu, end0, end0);
      grew = next0 != static_cast<uint32_t>(end0);
      if (p.m > 32) {
        const int at = end1 & 31;
        const uint32_t a = __shfl_sync(0xffffffffu, line0, at), b = __shfl_sync(0xffffffffu, low1, at);
        const uint32_t c = __shfl_sync(0xffffffffu, high1, at);
        const int x = __shfl_sync(0xffffffffu, end0, at), y = __shfl_sync(0xffffffffu, end1, at);
        const int next1 = end1 < 32 ? x : y;
        low1 |= end1 < 32 ? a : b;
        high1 |= end1 < 32 ? 0u : c;
        grew |= next1 != end1;
        end1 = next1;
      }
      line0 |= to0;
      end0 = next0;
    } while (__any_sync(0xffffffffu, grew));
    const int at = max(j, 0) & 31;
    const uint32_t a = __shfl_sync(0xffffffffu, line0, at), b = __shfl_sync(0xffffffffu, low1, at);
    const uint32_t c = __shfl_sync(0xffffffffu, high1, at);
    const unsigned long long seen = j < 32 ? a : static_cast<unsigned long long>(c) << 32 | b;
    *depth = __popcll(seen) - 1;
    return j < 0 ? 0ull : seen;
  }
  unsigned long long seen = 0;  // a window of fewer positions than a tree may have
  int a = max(j, 0), d = 0;
  bool on = j >= 0, bad = false;
  while (__any_sync(0xffffffffu, on)) {  // parents lie below their nodes
    if (on && d < p.window) seen |= 1ull << a;
    const int x = __shfl_sync(0xffffffffu, up0, a & 31), y = __shfl_sync(0xffffffffu, up1, a & 31);
    const int up = a < 32 ? x : y;
    const bool top = a == 0 || up < 0 || up >= a;
    bad |= on && top && (a != 0 || up != -1);
    on &= !top;
    if (on) {
      a = up;
      ++d;
    }
  }
  *depth = d;
  if (p.sinks > s.ctx) {  // nodes among the first rows
    a = max(j, 0);
    int e = d;
    on = j >= 0;
    while (__any_sync(0xffffffffu, on)) {
      if (on && s.ctx + e < p.sinks) seen |= 1ull << a;
      const int x = __shfl_sync(0xffffffffu, up0, a & 31), y = __shfl_sync(0xffffffffu, up1, a & 31);
      on &= e-- > 0;
      if (on) a = a < 32 ? x : y;
    }
  }
  if (bad) flag_status(p.status, kStatusCheck);
  return seen;
}

// The larger magnitude of each of two bf16 values, NaN if one is.
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Warp-collective: zeroes a unit's values (ATOMS pieces of 64 rows of 128 bytes side by side) that are not finite, and
// its rows from nv on; returns the keys that had such values. One look at the magnitudes first: they hardly ever have.
template <int ATOMS>
__device__ __forceinline__ unsigned long long clean_values(uint8_t *v, int nv, int lane) {
  constexpr int PIECE = kKeys * 128;
  if (nv < kKeys) {
#pragma unroll
    for (int a = 0; a < ATOMS; ++a)
      for (int k = max(nv, 0) * 8 + lane; k < kKeys * 8; k += 32)
        *reinterpret_cast<uint4 *>(v + a * PIECE + k * 16) = make_uint4(0, 0, 0, 0);
    __syncwarp();
  }
  uint4 top = make_uint4(0, 0, 0, 0);
#pragma unroll 16
  for (int k = 0; k < 16 * ATOMS; ++k) {
    const uint4 x = *reinterpret_cast<const uint4 *>(v + (k * 32 + lane) * 16);
    top.x = max_abs2(top.x, x.x), top.y = max_abs2(top.y, x.y);
    top.z = max_abs2(top.z, x.z), top.w = max_abs2(top.w, x.w);
  }
  const uint32_t m = max_abs2(max_abs2(top.x, top.y), max_abs2(top.z, top.w));
  bool wrote = nv < kKeys;
  unsigned long long found = 0;
  if (__any_sync(0xffffffffu, (m & 0x7F80u) == 0x7F80u || (m & 0x7F800000u) == 0x7F800000u)) {
    uint32_t found0 = 0, found1 = 0;
    // 16-byte pieces, eight of a row: a lane's are those of row lane / 8 and every fourth from it
    for (int k = 0; k < 16 * ATOMS; ++k) {
      const int key = (4 * k + (lane >> 3)) % kKeys;
      uint4 *at = reinterpret_cast<uint4 *>(v + (k * 32 + lane) * 16);
      const uint4 x = *at;
      uint32_t word[4] = {x.x, x.y, x.z, x.w};
      uint32_t odd = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t lo = (word[q] & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u;
        const uint32_t hi = (word[q] & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u;
        word[q] &= ~(lo | hi);
        odd |= lo | hi;
      }
      if (odd) {
        *at = make_uint4(word[0], word[1], word[2], word[3]);
        (key < 32 ? found0 : found1) |= 1u << (key & 31);
      }
    }
    found = static_cast<unsigned long long>(__reduce_or_sync(0xffffffffu, found1)) << 32 |
            __reduce_or_sync(0xffffffffu, found0);
    wrote = true;
  }
  if (wrote) fence_proxy_async_smem();  // for the products
  return found;
}

template <int HD, int NQ, bool TWO>
__global__ void __launch_bounds__(Roles<NQ>::THREADS, 1) attn_tree_kernel(const __grid_constant__ AttnTreeParams p) {
  using C = Cfg<HD, NQ, TWO>;
  using Ro = Roles<NQ>;
  constexpr int ST = C::STAGES;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *sQ = smem;
  uint8_t *sKV = smem + C::OFF_KV;
  uint64_t *kv_full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
  uint64_t *kv_empty = kv_full + ST;    // the last product of the stage, and the cleaner
  uint64_t *clean = kv_empty + ST;      // looked through by the cleaner
  uint64_t *s_full = clean + ST;        // [2]
  uint64_t *s_empty = s_full + 2;       // [2]
  uint64_t *p_full = s_empty + 2;       // [2]
  uint64_t *p_empty = p_full + 2;       // [2]: the product done
  uint64_t *q_full = p_empty + 2;       // Q landed in shared memory
  uint64_t *q_ready = q_full + 1;       // the first tile copied to tensor memory
  uint64_t *q_free = q_ready + 1;       // every S of the segment done
  uint64_t *o_free = q_free + 1;        // [2]: O read at a segment's end (one tile: both, as [0])
  uint64_t *ml_ready = o_free + 2;      // [2], one tile: the half's maximum and sum written, its O done
  uint64_t *mma_done = ml_ready + 2;    // [2]
  uint64_t *poison = mma_done + 2;      // [ST] keys of the stage whose values were not finite
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(poison + ST);
  int *sched = reinterpret_cast<int *>(tmem_slot + 1);  // [9]
  int2 *seqs = reinterpret_cast<int2 *>(smem + C::OFF_SEQ);
  float2 *ml = reinterpret_cast<float2 *>(smem + C::OFF_ML);  // [2][128] a half's maximum and sum
  static_assert((4 * ST + 2 + 2 + 2 + 2 + 3 + 2 + 2 + 2) * 8 + 40 <= C::BARS, "barrier region");
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
      mbar_init(&s_empty[b], NQ);
      mbar_init(&o_free[b], TWO ? NQ : 2 * NQ);
      mbar_init(&ml_ready[b], NQ);
      mbar_init(&mma_done[b], 1);
      mbar_init(&p_full[b], NQ);
      mbar_init(&p_empty[b], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_ready, NQ * C::QT);
    mbar_init(q_free, 1);
    fence_mbar_init();
    if (smem_u32(smem) & 1023) flag_status(p.status, kStatusTimeout);  // never: the swizzled tiles' alignment
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
  griddep_wait();  // the lengths may come from the launch before
  if (threadIdx.x == 0) griddep_launch();
  if (warp == Ro::PRODUCER) {
    const Split sp = make_split(p, seqs, lane);
    Place at = {-1, 0, 0, 0, 1};
    int count = 0;
    const int u0 = range_start(sp, blockIdx.x);
    if (static_cast<int>(blockIdx.x) < sp.ctas && sp.T > 0) {
      at = find_unit(p, seqs, sp, u0, lane);
      count = at.i < 0 ? 0 : range_start(sp, blockIdx.x + 1) - u0;
    }
    if (lane == 0) {
      sched[0] = at.i;
      sched[1] = at.g;
      sched[2] = at.grp;
      sched[3] = at.at;
      sched[4] = count;
      sched[5] = u0;
      sched[6] = sp.q;
      sched[7] = sp.r;
      sched[8] = sp.cost;
    }
  }
  // The merge's words: of each pair, by the CTA that has its first unit, or of the pair whose first part this CTA has
  if (threadIdx.x == 0 && !p.by_pair) p.joins[blockIdx.x].parts = 0;
  if (warp == Ro::CLEAN && blockIdx.x == 0) {
    bool bad = false;  // lengths out of range, reported once a launch
    for (int i = lane; i < p.nb; i += 32) {
      if (p.by_pair && clamp_nodes(p, i) == 0)  // pairs without units
        for (int k = 0; k < p.Hkv * p.groups; ++k) p.joins[i * p.Hkv * p.groups + k].parts = 0;
      const int n = p.n_rows ? p.n_rows[i] : p.m, c = p.ctx_len[i];
      bad |= n < 0 || n > p.m || c < 0 || c > p.max_ctx || c > p.Cmax - clamp_nodes(p, i);
    }
    if (bad) flag_status(p.status, kStatusCheck);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  Seg e = seg_begin(p, seqs, sched);

  auto load_q = [&](const Seg &s) {
    const uint64_t pol_q = policy_evict_last();
    const int node0 = s.grp * C::TILES * p.npt;
    const int tiles = TWO && node0 + p.npt < p.m ? 2 : 1;  // a last group may have one tile
    mbar_arrive_expect_tx(q_full, static_cast<uint32_t>(tiles * C::ATOMS * R * 128));
    for (int h = 0; h < tiles; ++h)
#pragma unroll
      for (int a = 0; a < C::ATOMS; ++a)
        tma_load_3d(sQ + h * C::Q_TILE + a * C::ATOM_Q, &p.tmQ, q_full, a * 64, s.g * G, s.i * p.m + node0 + h * p.npt,
                    pol_q);
  };
  if (warp == Ro::PRODUCER) {
    if (e.left > 0 && !p.stall) {
      // K and V of one pair are read by its groups of tiles one after another
      const uint64_t pol_kv = p.groups > 1 ? policy_evict_last() : policy_evict_first();
      bool ok = true;
      int q_loads = 1, loads = 0, st = 0;
      uint32_t ph = 0;
      for (; e.left > 0 && ok; seg_next(e, p, seqs)) {
        // a lane finds the cache row of a unit: 32 pages are looked up in the time of one (trees of 16 nodes
        // 192.8 us, by one thread four at a time 193.4)
        auto row_of = [&](int u) {
          if (u >= e.u1) return 0;
          const int base = unit_base(e.s, u);
          if (p.page_table == nullptr) return p.layer_row0 + (e.i * p.Hkv + e.g) * p.Cmax + base;
          int pg = p.page_table[(long long)e.i * p.pages_per_seq + base / kKeys];
          if (pg < 0 || pg >= p.num_pages) {
            flag_status(p.status, kStatusCheck);
            pg = 0;
          }
          return p.layer_row0 + (pg * p.Hkv + e.g) * kPageRows;
        };
        int row = row_of(e.u0 + lane);
        if (e.index > 0) {  // the first segment's is loaded by the PV issuer, which has the time
          // the place is free when the one tile is in tensor memory; the second is read where it lies
          ok = mbar_wait_warp(C::TILES > C::QT ? q_free : q_ready, (e.index - 1) & 1, p.max_spin);
          if (!ok) break;
          if (lane == 0) load_q(e);
          ++q_loads;
        }
        for (int u = e.u0, k = 0; u < e.u1; ++u, ++k) {
          if (k == 32) {
            k = 0;
            row = row_of(u + lane);
          }
          const int at = __shfl_sync(0xffffffffu, row, k);
          ok = loads < ST || mbar_wait_warp(&kv_empty[st], ph ^ 1, p.max_spin);
          if (!ok) break;
          if (lane == 0) {
            uint8_t *kt = sKV + st * C::STAGE;
            mbar_arrive_expect_tx(&kv_full[st], C::STAGE);
            tma_load_3d(kt, &p.tmK, &kv_full[st], 0, at, 0, pol_kv);
            tma_load_3d(kt + C::KV_TILE, &p.tmV, &kv_full[st], 0, at, 0, pol_kv);
          }
          __syncwarp();
          ++loads;
          ring_next<ST>(st, ph);
        }
      }
      if (lane == 0) {
        if (!ok) flag_status(p.status, kStatusTimeout);
        for (int k = max(0, loads - ST); k < loads; ++k)  // every copy lands before the CTA ends
          mbar_wait(&kv_full[k % ST], (k / ST) & 1, kDrainSpin);
        mbar_wait(q_full, (q_loads - 1) & 1, kDrainSpin);
      }
    }
  } else if (warp == Ro::S) {
    if (__any_sync(0xffffffffu, e.left > 0)) {
      constexpr uint32_t id_s = idesc_bf16_f32(kTileRows, kKeys);
      const uint64_t q_desc0 = sw128_kmajor_desc(smem_u32(sQ));
      const uint64_t k_desc0 = sw128_kmajor_desc(smem_u32(sKV));
      const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem_base);
      bool ok = true;
      int step = 0, st = 0;
      uint32_t ph = 0;
      for (; ok && __any_sync(0xffffffffu, e.left > 0); seg_next(e, p, seqs)) {
        ok = mbar_wait_warp(q_ready, e.index & 1, p.max_spin);
        if (C::TILES > C::QT && ok) ok = mbar_wait_warp(q_full, e.index & 1, p.max_spin);
        const int n = __reduce_max_sync(0xffffffffu, e.u1 - e.u0);
        for (int k = 0; k < n && ok; ++k) {
          ok = mbar_wait_warp(&kv_full[st], ph, p.max_spin);
          const uint64_t kd = k_desc0 + static_cast<uint64_t>((st * C::STAGE) >> 4);
#pragma unroll
          for (int h = 0; h < C::TILES; ++h) {
            const int sb = step & 1;
            if (ok && step >= 2) ok = mbar_wait_warp(&s_empty[sb], ((step >> 1) - 1) & 1, p.max_spin);
            if (!ok) break;
            tc_fence_after();
            const uint32_t d_s = tm + C::S_COL + sb * kKeys;
            const uint64_t qd = q_desc0 + static_cast<uint64_t>((h * C::Q_TILE) >> 4);
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < HD / 16; ++kk) {
                const uint64_t kkd = kd + static_cast<uint64_t>(((kk >> 2) * C::ATOM_KV + (kk & 3) * 32) >> 4);
                if (h < C::QT)
                  tc_mma_bf16_tmem_a(d_s, tm + C::Q_COL + h * (HD / 2) + kk * 8, kkd, id_s, kk > 0 ? 1u : 0u);
                else
                  tc_mma_bf16(d_s, qd + static_cast<uint64_t>(((kk >> 2) * C::ATOM_Q + (kk & 3) * 32) >> 4), kkd, id_s,
                              kk > 0 ? 1u : 0u);
              }
              tc_commit(&s_full[sb]);
            }
            __syncwarp();
            ++step;
          }
          ring_next<ST>(st, ph);
        }
        if (ok && elect_one()) tc_commit(q_free);
        __syncwarp();
      }
      if (elect_one()) {
        if (!ok) flag_status(p.status, kStatusTimeout);
        tc_commit(&mma_done[0]);  // every product completes before tensor memory is freed
        mbar_wait(&mma_done[0], 0, kDrainSpin);
      }
    }
  } else if (warp == Ro::PV) {
    // a warp with an elected lane, or a thread: of 64 channels, whose units come sooner than a warp's votes, 64 single
    // tokens take 102 us with a thread, 108 with a warp; of 128, 64 x 64 rows 250 with a warp, 252 with a thread
    constexpr bool WARP = HD == 128;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      return WARP ? mbar_wait_warp(bar, parity, p.max_spin) : mbar_wait(bar, parity, p.max_spin);
    };
    if (WARP ? __any_sync(0xffffffffu, e.left > 0) != 0 : lane == 0 && e.left > 0) {
      if (lane == 0 && !p.stall) load_q(e);
      if (WARP) __syncwarp();
      constexpr uint32_t id_pv = idesc_bf16_f32(kTileRows, HD) | kIdescBMajorMN;
      const uint64_t v_desc0 = sw128_mnmajor_desc(smem_u32(sKV + C::KV_TILE), C::ATOM_KV);
      const uint32_t tm = WARP ? __reduce_max_sync(0xffffffffu, tmem_base) : tmem_base;
      bool ok = true;
      int step = 0, st = 0;
      uint32_t ph = 0;
      for (; ok && (WARP ? __any_sync(0xffffffffu, e.left > 0) != 0 : e.left > 0); seg_next(e, p, seqs)) {
        const int first = step;
        const int n = WARP ? __reduce_max_sync(0xffffffffu, e.u1 - e.u0) : e.u1 - e.u0;
        for (int k = 0; k < n && ok; ++k) {
          const uint64_t vd = v_desc0 + static_cast<uint64_t>((st * C::STAGE) >> 4);
#pragma unroll
          for (int h = 0; h < C::TILES; ++h) {
            const int half = step & 1;
            const bool start = step < first + 2;  // the half's first unit of the segment
            ok = wait(&p_full[half], (step >> 1) & 1);
            if (ok && start && e.index > 0) ok = wait(&o_free[TWO ? half : 0], (e.index - 1) & 1);
            if (!ok) break;
            tc_fence_after();
            const uint32_t d_o = tm + C::O_COL + half * HD;
            const uint32_t a_p = tm + C::P_COL + half * 32;
            if (!WARP || elect_one()) {
#pragma unroll
              for (int kk = 0; kk < kKeys / 16; ++kk)
                tc_mma_bf16_tmem_a(d_o, a_p + kk * 8, vd + static_cast<uint64_t>((kk * 16 * 128) >> 4), id_pv,
                                   (!start || kk > 0) ? 1u : 0u);
              tc_commit(&p_empty[half]);
              if (h == C::TILES - 1) tc_commit(&kv_empty[st]);
            }
            if (WARP) __syncwarp();
            ++step;
          }
          ring_next<ST>(st, ph);
        }
      }
      if (!WARP || elect_one()) {
        if (!ok) flag_status(p.status, kStatusTimeout);
        tc_commit(&mma_done[1]);
        mbar_wait(&mma_done[1], 0, kDrainSpin);
      }
    }
  } else if (warp == Ro::CLEAN) {
    bool ok = true;
    int st = 0;
    uint32_t ph = 0;
    for (; e.left > 0 && ok; seg_next(e, p, seqs)) {
      const Plain plain = plain_units(p, e.s);
      for (int u = e.u0; u < e.u1; ++u) {
        ok = mbar_wait_warp(&kv_full[st], ph, p.max_spin);
        if (!ok) break;
        if (!unit_plain(plain, u)) {
          const unsigned long long found = clean_values<C::ATOMS>(
              sKV + st * C::STAGE + C::KV_TILE, e.s.ctx + e.s.n - unit_base(e.s, u), lane);
          if (lane == 0) poison[st] = found;
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&clean[st]);
          mbar_arrive(&kv_empty[st]);
        }
        ring_next<ST>(st, ph);
      }
    }
    if (!ok && lane == 0) flag_status(p.status, kStatusTimeout);
  } else if ((warp & 3) < NQ) {
    // ---------------- softmax
    constexpr int STRIDE = TWO ? 1 : 2;  // units between two of this half's
    const int half = warp >> 2;
    const int q = warp & 3;
    const int r = q * 32 + lane;
    const int jr = r / G, hq = r - jr * G;  // node of the tile and head of its group
    const uint32_t trow = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    const uint32_t o_mine = trow + C::O_COL + half * HD;
    const float sl2 = rsqrtf(static_cast<float>(HD)) * 1.4426950408889634f;
    // The first QT tiles of a segment's Q to tensor memory, by half 1, or with two tiles by the halves whose rows they
    // are. One tile's place in shared memory is free for the next segment's then, and the products do not read it from
    // there beside the keys (262147 rows under 64 nodes: 203 us then, both tiles from shared memory 219; of 64
    // channels, where tensor memory has the columns, 173 with both in it, 179 with one).
    const bool copies = TWO ? half < C::QT : half == 1;
    const int tile = TWO ? half : 0;
    auto copy_q = [&](int index) {
      bool good = index == 0 || mbar_wait_warp(q_free, (index - 1) & 1, p.max_spin);
      if (good) good = mbar_wait_warp(q_full, index & 1, p.max_spin);
      if (!good) return false;
      tc_fence_after();
#pragma unroll 1
      for (int a = 0; a < HD / 32; ++a) {
        uint32_t v[16];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint4 x = *reinterpret_cast<const uint4 *>(sQ + tile * C::Q_TILE + (a >> 1) * C::ATOM_Q + r * 128 +
                                                           ((((a & 1) * 4 + c) ^ (r & 7)) << 4));
          v[4 * c] = x.x, v[4 * c + 1] = x.y, v[4 * c + 2] = x.z, v[4 * c + 3] = x.w;
        }
        tmem_st16_raw(trow + C::Q_COL + tile * (HD / 2) + a * 16, v);
      }
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(q_ready, lane);
      return true;
    };
    bool ok = true;
    if (copies && e.left > 0) ok = copy_q(0);
    int units = 0;  // of the segments before
    for (; e.left > 0 && ok; seg_next(e, p, seqs)) {
      const bool more = seg_more(e);
      const int node = (e.grp * C::TILES + (TWO ? half : 0)) * p.npt + jr;
      const bool real = r < R && node < e.s.n;
      const bool warp_real = __any_sync(0xffffffffu, real);
      float m_run = -FLT_MAX, l_run = 0.f;
      unsigned long long line = 0;  // nodes this row sees
      int lo = 0;                   // its first context row behind the sinks
      bool have_line = false;
      int up0 = -1, up1 = -1;       // parents of nodes `lane` and lane + 32, for the masks to come
      if (p.parent) {
        const int *up = p.parent + (long long)e.i * p.m;
        if (lane < p.m) up0 = up[lane];
        if (lane + 32 < p.m) up1 = up[lane + 32];
      }
      const int u_first = TWO ? e.u0 : e.u0 + ((units ^ half) & 1);
      const Plain plain = plain_units(p, e.s);
      int step = 0;
#pragma unroll 1
      for (int u = u_first; u < e.u1; u += STRIDE) {
        const int stage = units + u - e.u0;
        step = TWO ? 2 * stage + half : stage;
        const bool start = u == u_first;
        ok = mbar_wait_warp(&s_full[half], (step >> 1) & 1, p.max_spin);
        if (!ok) break;
        tc_fence_after();
        float sv[kKeys];
        if (warp_real) tmem_ld64(trow + C::S_COL + half * kKeys, sv);
        tc_fence_before();
        warp_arrive(&s_empty[half], lane);

        unsigned long long bad = 0;
        if (!unit_plain(plain, u)) {
          const int base = unit_base(e.s, u);
          if (!have_line) {
            int depth = 0;
            line = line_of(p, e.s, real ? node : -1, up0, up1, lane, &depth);
            lo = p.window > 0 ? max(0, e.s.ctx + depth + 1 - p.window) : 0;
            have_line = true;
          }
          unsigned long long keep = low_bits(e.s.ctx - base);
          if (p.window > 0) keep &= ~low_bits(lo - base) | low_bits(p.sinks - base);
          const int sh = base - e.s.ctx;  // key k of the unit is node k + sh
          keep |= sh >= 64 || sh <= -64 ? 0ull : sh >= 0 ? line >> sh : line << -sh;
          const uint32_t k0 = static_cast<uint32_t>(keep), k1 = static_cast<uint32_t>(keep >> 32);
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            sv[c] = k0 >> c & 1 ? sv[c] : -INFINITY;
            sv[c + 32] = k1 >> c & 1 ? sv[c + 32] : -INFINITY;
          }
          const int st = stage % ST;
          ok = mbar_wait_warp(&clean[st], (stage / ST) & 1, p.max_spin);
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
          need = (mx - m_run) * sl2 > kGrowLog2;
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
        // P's place is free, and O at rest, once the half's product before is done. Asked for here and not behind the
        // exponentials, where it would be there already, it keeps the halves' exponentials apart (262147 rows under 64
        // nodes 196 us then, behind them 216).
        ok = step < 2 || mbar_wait_warp(&p_empty[half], ((step >> 1) - 1) & 1, p.max_spin);
        if (!ok) break;
        tc_fence_after();  // behind that product come what is written of O, and P
        if (!start && __any_sync(0xffffffffu, need)) {
#pragma unroll 1
          for (int cc = 0; cc < HD / 32; ++cc) {
            float ov[32];
            tmem_ld32(o_mine + cc * 32, ov);
#pragma unroll
            for (int c = 0; c < 32; ++c) ov[c] *= alpha;
            tmem_st32(o_mine + cc * 32, ov);
          }
        }
        if (warp_real) {
          const float2 sc = make_float2(sl2, sl2), nm = make_float2(-m_run * sl2, -m_run * sl2);
          float2 sum[2] = {make_float2(l_run, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            uint32_t pk[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              float2 x = fma2(make_float2(sv[32 * cc + 2 * c], sv[32 * cc + 2 * c + 1]), sc, nm);
              x.x = ex2(x.x);
              x.y = ex2(x.y);
              sum[c & 1] = add2(sum[c & 1], x);
              pk[c] = pack_bf16x2(x.x, x.y);
            }
            tmem_st16_raw(trow + C::P_COL + half * 32 + cc * 16, pk);
          }
          l_run = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          tmem_wait_st();
        }
        tc_fence_before();
        warp_arrive(&p_full[half], lane);
      }
      if (!ok) break;

      // ---------------- the segment's end
      const bool whole = e.u0 == 0 && e.u1 == e.s.U;
      const bool mine = u_first < e.u1;  // this half had units of it, the last one at `step`
      units += e.u1 - e.u0;
      const int slot = 2 * static_cast<int>(blockIdx.x) + (e.index > 0);
      float M = m_run, L = l_run, a0 = 1.f, a1 = 0.f;
      if (!TWO && e.index > 0) ok = mbar_wait_warp(&o_free[0], (e.index - 1) & 1, p.max_spin);  // ml was read
      if (ok && mine) ok = mbar_wait_warp(&p_empty[half], (step >> 1) & 1, p.max_spin);
      if (!ok) break;
      if (!TWO) {  // each half ends half of the channels, of both O
        ml[half * kTileRows + r] = mine ? make_float2(M, L) : make_float2(-FLT_MAX, -1.f);
        tc_fence_before();
        warp_arrive(&ml_ready[half], lane);
        if (half == 1 && more) ok = copy_q(e.index + 1);
        if (ok) ok = mbar_wait_warp(&ml_ready[half ^ 1], e.index & 1, p.max_spin);
        if (!ok) break;
        const float2 h0 = ml[r], h1 = ml[kTileRows + r];
        M = fmaxf(h0.x, h1.x);
        a0 = h0.y < 0.f ? 0.f : ex2((h0.x - M) * sl2);
        a1 = h1.y < 0.f ? 0.f : ex2((h1.x - M) * sl2);
        L = (h0.y < 0.f ? 0.f : h0.y * a0) + (h1.y < 0.f ? 0.f : h1.y * a1);
      }
      tc_fence_after();
      if (threadIdx.x == 0 && e.u0 == 0 && (p.by_pair || !whole)) {  // what the merge has to know
        const Split sp = {0, 0, sched[6], sched[7], e.cost};
        const int c0 = blockIdx.x, last = range_of(sp, e.pos + e.cost + e.s.U - 1);
        const int word = p.by_pair ? (e.i * p.Hkv + e.g) * p.groups + e.grp : c0;
        p.joins[word] = {e.i, e.g, e.grp, c0, slot, last - c0 + 1, e.s.n};
      }
      if (warp_real) {
        const float inv = 1.0f / L;
        const int prow = (TWO ? half * R : 0) + r;
        // with one unit only, one of the two O was not begun
        const int first0 = TWO || e.u1 - e.u0 > 1 ? -1 : (units - (e.u1 - e.u0)) & 1;
        const int c0 = TWO ? 0 : half * (HD / 2), cn = TWO ? HD : HD / 2;
#pragma unroll 2
        for (int cc = c0; cc < c0 + cn; cc += 16) {
          float ov[16];
          if (TWO) {
            tmem_ld16(o_mine + cc, ov);
          } else if (first0 < 0) {
            float o1[16];
            tmem_ld16_two(trow + C::O_COL + cc, ov, trow + C::O_COL + HD + cc, o1);
#pragma unroll
            for (int c = 0; c < 16; ++c) ov[c] = ov[c] * a0 + o1[c] * a1;
          } else {
            tmem_ld16(trow + C::O_COL + (first0 == 1 ? HD : 0) + cc, ov);
          }
          if (real && whole) {
            uint16_t *dst = p.o + (((long long)e.i * p.m + node) * p.Hq + e.g * G + hq) * HD + cc;
#pragma unroll
            for (int v = 0; v < 2; ++v)
              reinterpret_cast<uint4 *>(dst)[v] =
                  make_uint4(pack_bf16x2(ov[8 * v] * inv, ov[8 * v + 1] * inv),
                             pack_bf16x2(ov[8 * v + 2] * inv, ov[8 * v + 3] * inv),
                             pack_bf16x2(ov[8 * v + 4] * inv, ov[8 * v + 5] * inv),
                             pack_bf16x2(ov[8 * v + 6] * inv, ov[8 * v + 7] * inv));
          } else if (real) {
            // rows side by side, four channels each: a warp's store is four lines, with a row's channels side by side
            // it was 32 (64 x 64 rows 293 us, so 286)
            float4 *dst =
                reinterpret_cast<float4 *>(p.part_o) + ((long long)slot * (HD / 4) + cc / 4) * p.part_rows + prow;
#pragma unroll
            for (int v = 0; v < 4; ++v)
              dst[v * p.part_rows] = make_float4(ov[4 * v], ov[4 * v + 1], ov[4 * v + 2], ov[4 * v + 3]);
          }
          __syncwarp();  // the next load is the whole warp's
        }
        if (real && !whole && (TWO || half == 0))
          reinterpret_cast<float2 *>(p.part_ml)[(long long)slot * p.part_rows + prow] = make_float2(M, L);
      }
      tc_fence_before();
      warp_arrive(&o_free[TWO ? half : 0], lane);
      if (TWO && copies && more) ok = copy_q(e.index + 1);
    }
    if (!ok && lane == 0) flag_status(p.status, kStatusTimeout);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == Ro::S) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// Warp-collective: the place of the first of pair x's units (or cost), 0 <= x < pairs; *start is where it lies.
__device__ __forceinline__ Place find_pair(const AttnTreeParams &p, const int2 *seqs, const Split &s, int x, int lane,
                                           int *start) {
  const int per = p.Hkv * p.groups;
  Place f = {x / per, 0, 0, 0, 0};
  const int k = x - f.i * per;
  f.g = k / p.groups;
  f.grp = k - f.g * p.groups;
  int before = 0;
  for (int i = lane; i <= f.i; i += 32) {
    const int U = span_of(p, seqs, i).U;
    if (i == f.i)
      f.U = U;
    else
      before += U > 0 ? U + s.cost : 0;
  }
  f.U = __shfl_sync(0xffffffffu, f.U, f.i & 31);
  *start = __reduce_add_sync(0xffffffffu, before) * per + k * (f.U + s.cost);
  return f;
}

// Joins the partials of a pair that several CTAs share: block x those of pair x, or where there are more pairs than
// CTAs of the pair whose first part CTA x has, from the attention's word about it, which spares some 2000 blocks the
// search for it (64 x 64 rows 277 us, with it 287). A lane has four channels of a row, as the partials lie. Bound by the
// latency of the parts' loads: with up to 16 rows eight warps share a lane's parts (WPR), and the blocks, which are few
// then and may stand by next to the attention, find their pair's parts while they wait (one token 9.4 us, by its word
// 9.9).
constexpr int kMergeWarps = 8;

template <int HD, int WPR>
__global__ void __launch_bounds__(kMergeWarps * 32) attn_tree_merge_kernel(const __grid_constant__ AttnTreeParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv, R = p.npt * G, rows = p.part_rows;
  const int f = (blockIdx.y * (kMergeWarps / WPR) + warp / WPR) * 32 + lane;  // four channels of a slot
  const int sub = warp % WPR;
  const int chunk = f / rows, r = f - chunk * rows;
  const int tile = r / R, rt = r - tile * R, jr = rt / G;
  griddep_launch();  // the next launch may begin: it waits for this grid's end
  TreeJoin at = {0, 0, 0, 0, 0, 0, 0};
  if (WPR > 1 && p.by_pair) {
    // the lengths are older than the attention, which lets this launch begin once it waited itself
    __shared__ int2 seqs[kSeqCache];  // every warp writes the same
    const Split sp = make_split(p, seqs, lane);
    int start = 0;
    const Place f = find_pair(p, seqs, sp, blockIdx.x, lane, &start);
    if (f.U > 0) {
      const int c0 = range_of(sp, start + sp.cost), last = range_of(sp, start + sp.cost + f.U - 1);
      at = {f.i, f.g, f.grp, c0, 2 * c0 + (range_start(sp, c0) < start), last - c0 + 1, clamp_nodes(p, f.i)};
    }
    griddep_wait();  // every block: this grid's end has to imply the attention's
  } else {
    griddep_wait();
    at = p.joins[blockIdx.x];
    // an attention whose waits ran out leaves words of before
    if (p.by_pair && (at.c0 < 0 || at.parts > p.grid - at.c0 || (at.slot & ~1) != 2 * at.c0 || at.i < 0 ||
                      at.i >= p.nb || at.g < 0 || at.g >= p.Hkv || at.grp < 0 || at.grp >= p.groups || at.nodes > p.m))
      return;
  }
  const int n = at.parts, c0 = at.c0;
  if (n < 2) return;
  const int node = (at.grp * (rows / R) + tile) * p.npt + jr;
  const bool real = chunk < HD / 4 && node < at.nodes;
  const float sl2 = rsqrtf(static_cast<float>(HD)) * 1.4426950408889634f;
  float M = -FLT_MAX, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float w, float l, const float4 &x) {
    L = fmaf(w, l, L);
    acc.x = fmaf(w, x.x, acc.x), acc.y = fmaf(w, x.y, acc.y);
    acc.z = fmaf(w, x.z, acc.z), acc.w = fmaf(w, x.w, acc.w);
  };
  auto grow = [&](float m) {
    const float a = ex2((M - m) * sl2);
    M = m;
    L *= a;
    acc.x *= a, acc.y *= a, acc.z *= a, acc.w *= a;
  };
  if (real) {
    constexpr int AT = 4;  // parts at a time
    for (int k0 = sub; k0 < n; k0 += AT * WPR) {
      float2 ml[AT];
      float4 x[AT];
#pragma unroll
      for (int j = 0; j < AT; ++j) {
        const int k = k0 + j * WPR;
        const long long slot = k == 0 ? at.slot : 2 * (c0 + min(k, n - 1));
        ml[j] = reinterpret_cast<const float2 *>(p.part_ml)[slot * rows + r];
        x[j] = reinterpret_cast<const float4 *>(p.part_o)[(slot * (HD / 4) + chunk) * rows + r];
      }
      float m = M;
#pragma unroll
      for (int j = 0; j < AT; ++j) m = fmaxf(m, ml[j].x);
      grow(m);
#pragma unroll
      for (int j = 0; j < AT; ++j)
        if (k0 + j * WPR < n) add(ex2((ml[j].x - M) * sl2), ml[j].y, x[j]);
    }
  }
  if constexpr (WPR > 1) {
    __shared__ float4 part[kMergeWarps][32];
    __shared__ float2 part_ml[kMergeWarps][32];
    part[warp][lane] = acc;
    part_ml[warp][lane] = make_float2(M, L);
    __syncthreads();
    if (sub > 0) return;
    float m = M;
#pragma unroll
    for (int k = 1; k < WPR; ++k) m = fmaxf(m, part_ml[warp + k][lane].x);
    grow(m);
#pragma unroll
    for (int k = 1; k < WPR; ++k) {
      const float2 ml = part_ml[warp + k][lane];
      add(ex2((ml.x - M) * sl2), ml.y, part[warp + k][lane]);
    }
  }
  if (!real) return;
  const float inv = 1.0f / L;
  uint16_t *dst = p.o + (((long long)at.i * p.m + node) * p.Hq + at.g * G + rt - jr * G) * HD + chunk * 4;
  *reinterpret_cast<uint2 *>(dst) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

template <int HD, int WPR>
cudaError_t launch_merge(const AttnTreeParams &p, cudaStream_t s) {
  // the attention's split of the SM's memory, so that this grid's CTAs may stand by next to it
  static OncePerDevice once;
  const cudaError_t e = once([] {
    return cudaFuncSetAttribute(attn_tree_merge_kernel<HD, WPR>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                cudaSharedmemCarveoutMaxShared);
  });
  if (e != cudaSuccess) return e;
  constexpr int per = kMergeWarps / WPR * 32;
  const dim3 grid(p.by_pair ? p.nb * p.Hkv * p.groups : p.grid, (p.part_rows * (HD / 4) + per - 1) / per);
  return launch_pdl(attn_tree_merge_kernel<HD, WPR>, grid, dim3(kMergeWarps * 32), 0, s, p);
}

template <int HD, int NQ, bool TWO>
cudaError_t launch(const AttnTreeParams &p, cudaStream_t s) {
  using C = Cfg<HD, NQ, TWO>;
  static OncePerDevice once;
  cudaError_t e = once([] {
    return cudaFuncSetAttribute(attn_tree_kernel<HD, NQ, TWO>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)C::SMEM);
  });
  if (e != cudaSuccess) return e;
  e = launch_pdl(attn_tree_kernel<HD, NQ, TWO>, dim3(p.grid), dim3(Roles<NQ>::THREADS), C::SMEM, s, p);
  if (e != cudaSuccess) return e;
  return p.part_rows <= 16 ? launch_merge<HD, kMergeWarps>(p, s) : launch_merge<HD, 1>(p, s);
}

template <int HD>
cudaError_t launch_form(const AttnTreeParams &p, cudaStream_t s) {
  const int R = p.npt * (p.Hq / p.Hkv);
  if (p.part_rows > R) return launch<HD, 4, true>(p, s);
  if (R > 64) return launch<HD, 4, false>(p, s);
  return R > 32 ? launch<HD, 2, false>(p, s) : launch<HD, 1, false>(p, s);
}

}  // namespace

// Nodes per tile and groups of tiles for m nodes of G <= 64 query heads (dflash_create takes no more): one tile where
// all rows fit, else pairs of tiles of about the same size.
void attention_tree_plan(int m, int G, int *npt, int *groups, int *part_rows) {
  const int most = kTileRows / G;  // nodes of a tile
  if (m <= most) {
    *npt = m;
    *groups = 1;
    *part_rows = m * G;
    return;
  }
  *groups = (m + 2 * most - 1) / (2 * most);
  *npt = (m + 2 * *groups - 1) / (2 * *groups);
  *part_rows = 2 * *npt * G;
}

int attention_tree_part_rows(int m, int G) {
  int most = 0;
  for (int k = 1; k <= m; ++k) {
    int npt, groups, rows;
    attention_tree_plan(k, G, &npt, &groups, &rows);
    most = rows > most ? rows : most;
  }
  return most;
}

cudaError_t launch_attention_tree(AttnTreeParams &p, cudaStream_t s) {
  p.by_pair = p.nb * p.Hkv * p.groups <= p.grid;
  // Set-up, masks and output of a segment in units of the loads' time, by measurement: 64 x 16 rows of 4 heads 194.7 us
  // without, 191.3 with 4, 193.0 with 12; 32 x 25 rows under a window 38.5 with 4, 37.7 with 6; 64 x 64 rows (two tiles)
  // 255 with 4, 246 with 6, 250 with 8. A unit of 64 channels takes half the time.
  p.pair_cost = (p.npt * (p.Hq / p.Hkv) > 64 ? 6 : 4) * (128 / p.hd);
  switch (p.hd) {
    case 64: return launch_form<64>(p, s);
    case 128: return launch_form<128>(p, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace df
