// Penalties for repeated tokens, biases and masks on rows of fp32 logits, with the greedy token of each
// row, and the counts of tokens those penalties read.
//
//   c      times the token was generated: counts[i][v] & 0x7fffffff, and once for every drafted node
//          from row j's own node up to the root (the root's token is counted already)
//   seen   c > 0, or bit 31 of counts[i][v]: the prompt has it
//   y    = x / rep where seen and x > 0, x * rep where seen and x <= 0, else x
//   y   -= freq * c + pres * [c > 0]
//   y   += the token's biases, summed in the order of their list
//   y    = -inf where the row's mask does not allow the token
//   id   = argmax y, the lowest id of equals, -1 where nothing is above -inf (a NaN never is)
//
// One pass over the logits: 8 bytes a value (4 where only ids are asked for), 4 more a sequence for its
// counts, a bit a value for the mask: 1024 rows of 151936 under all of it 232 us, 1.306 GB at 5.6 TB/s; ids alone
// 125 us, 5.3 TB/s. A warp takes up to 1024 tokens for rows of one sequence, RPC of them
// at a time: the tokens that are counted, biased or drafted are found once, as a bit each in a word a
// lane, and every lane's copies of the rows' values run ahead of it through its own places in shared
// memory, so that a warp waits for nobody. The counts of a sequence with one row run through the same places (64
// rows 24.6 us, read before the row 28.8). Bound by HBM for many rows; one row a sequence
// by what a CTA begins with, lists and first copies, in two waves; a single row (5.8 us) by that and two
// launches. Rows of odd strides or vocabularies go value by value, bound by their instructions (265 us).
// Few tokens are listed so, but next to every row of a warp's values has one, and in line they would cost the
// warp their division and look-ups for one lane's sake (1159 us for 1024 rows of 151936). So the pass masks
// and takes the maximum of the others, and behind it the warp works its listed tokens off, a lane a
// token. Biased and drafted tokens are marked in a bitmap of the CTA; only marked ones look their biases
// up (a hash has the ids' sums) and the nodes they are drafted by. Where ids are asked for, a second
// launch picks each row's among its slices'.
#include <algorithm>
#include <cfloat>

#include "common.cuh"
#include "kernels.h"

namespace df {

namespace {

constexpr int kWarps = 8;                // of a CTA
constexpr int kTiles = 8;                // most of a warp: 128 tokens each, four of them a lane's
static_assert(kLogitSlice == 128 * kWarps, "one tile a warp");
static_assert((kMaxVocab - 1) / (kTiles * kLogitSlice) < kLogitSlots, "the largest vocabulary in the largest slices");

// Pieces of 128 values of a warp's stage: the rows', and for one row its counts.
__host__ __device__ constexpr int ring_slots(int rpc) { return rpc == 1 ? 2 : rpc; }

__device__ __forceinline__ uint32_t id_hash(int id, uint32_t mask) {
  return (static_cast<uint32_t>(id) * 2654435761u >> 12) & mask;
}

// Better of two (value, id) pairs: larger value, then lower id; id -1: none.
__device__ __forceinline__ void take_best(float &v, int &id, float w, int wid) {
  const bool better = w > v || (w == v && wid >= 0 && (id < 0 || wid < id));
  v = better ? w : v;
  id = better ? wid : id;
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// A bit for each of four counts that is not zero.
__device__ __forceinline__ uint32_t some_of(const int4 &c) {
  return (c.x ? 1u : 0u) | (c.y ? 2u : 0u) | (c.z ? 4u : 0u) | (c.w ? 8u : 0u);
}

struct RowRules {
  float rep, freq, pres;
};

__device__ __forceinline__ float adjust(float x, int count, int drafted, const RowRules &r) {
  if (count | drafted) {
    x = x > 0.f ? x / r.rep : x * r.rep;
    const int c = (count & 0x7fffffff) + drafted;
    x -= fmaf(r.freq, static_cast<float>(c), c > 0 ? r.pres : 0.f);
  }
  return x;
}

// RPC rows at a time, S stages of a tile of theirs in flight. VEC: rows of 16-byte pieces, a lane's four
// values side by side; else they lie 32 apart and are loaded as they are needed. MASK: the rows have masks.
template <int RPC, int S, bool VEC, bool MASK>
__global__ void __launch_bounds__(32 * kWarps, RPC == 1 ? 4 : 3) logits_adjust_kernel(const LogitsParams p) {
  constexpr int T = 32 * kWarps;
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ int s_token[kTreeMax];
  __shared__ int s_parent[kTreeMax];
  __shared__ unsigned long long s_line[kTreeMax];  // drafted nodes from a node up
  __shared__ float s_val[kTreeMax][kWarps];
  __shared__ int s_id[kTreeMax][kWarps];
  __shared__ uint32_t marked[kWarps * 32];         // biased tokens
  __shared__ uint32_t drafted[kWarps * 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int SLOTS = ring_slots(RPC);
  float *ring = reinterpret_cast<float *>(dyn) + warp * (S * SLOTS * 128) + (VEC ? 4 : 1) * lane;
  int *hkey = reinterpret_cast<int *>(dyn + kWarps * S * SLOTS * 512);  // [hash]: id, -1 free
  float *hsum = reinterpret_cast<float *>(hkey + p.hash);
  int *hcount = reinterpret_cast<int *>(hsum + p.hash);
  const int slice = blockIdx.x % p.slices;
  const int at = blockIdx.x / p.slices;
  const int i = at / p.splits, split = at % p.splits;
  const int v0 = slice * p.chunk, v1 = min(p.V, v0 + p.chunk);
  const bool special = p.n_bias > 0 || p.parent != nullptr;
  if (special) {
    marked[tid] = drafted[tid] = 0;
    for (int e = tid; e < p.hash; e += T) {
      hkey[e] = -1;
      hcount[e] = 0;
    }
  }
  griddep_wait();
  griddep_launch();
  int n = p.n_rows ? p.n_rows[i] : p.m;
  if ((n < 0 || n > p.m) && slice == 0 && split == 0 && tid == 0) flag_status(p.status, kStatusCheck);
  n = max(0, min(n, p.m));
  const int j0 = split * p.rows, j1 = min(n, j0 + p.rows);  // this CTA's rows
  if (j0 >= j1) return;

  // ---- the pass begins: the first tiles' copies, the counts
  const int wt = p.chunk / (128 * kWarps);           // tiles of a warp
  const int base = v0 + warp * wt * 128;             // its first token
  const int tiles = base < v1 ? min(wt, (v1 - base + 127) / 128) : 0;
  const int steps = tiles * ((j1 - j0 + RPC - 1) / RPC);
  const long long seq = (long long)i * p.m;
  const float *x0 = p.x + seq * p.ldx + base + (VEC ? 4 : 1) * lane;
  const int *counts = p.counts ? p.counts + (long long)i * p.V + base : nullptr;
  // copies of a tile of 128 values, the lane's four
  auto copy = [&](const void *src, float *place, int tile) {
    const float *from = static_cast<const float *>(src) + 128 * tile;
    const uint32_t to = smem_u32(place);
    if (VEC) {
      if (base + 128 * tile + 4 * lane < v1) cp_async16(to, from);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (base + 128 * tile + 32 * q + lane < v1) cp_async4(to + 128 * q, from + 32 * q);
    }
  };
  // rows behind the last repeat it: the same values go to the same places
  int f_row = j0, f_tile = 0;
  auto fetch = [&](int step) {
    if (step < steps) {
#pragma unroll
      for (int r = 0; r < RPC; ++r)
        copy(x0 + min(f_row + r, j1 - 1) * p.ldx, ring + (step % S * SLOTS + r) * 128, f_tile);
      if (RPC == 1 && counts) copy(counts + (VEC ? 4 : 1) * lane, ring + (step % S * SLOTS + 1) * 128, f_tile);
      if (++f_tile == tiles) {
        f_tile = 0;
        f_row += RPC;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int k = 0; k < S - 1; ++k) fetch(k);
  uint32_t listed = 0;  // bit 4 t + q: the lane's q'th token of tile t
  if (RPC > 1 && counts) {
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      if (t >= tiles) break;
      if (VEC) {
        if (base + 128 * t + 4 * lane < v1)
          listed |= some_of(__ldg(reinterpret_cast<const int4 *>(counts + 128 * t) + lane)) << 4 * t;
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int e = 128 * t + 32 * q + lane;
          if (base + e < v1) listed |= (__ldg(counts + e) != 0 ? 1u : 0u) << (4 * t + q);
        }
      }
    }
  }
  RowRules rules = {1.f, 0.f, 0.f};
  if (p.penalties) {
    rules.rep = p.penalties[3 * i];
    rules.freq = p.penalties[3 * i + 1];
    rules.pres = p.penalties[3 * i + 2];
  }

  // ---- biased and drafted tokens
  const uint32_t hmask = p.hash - 1;
  if (special) {
    if (p.parent)
      for (int j = tid; j < n; j += T) {
        s_token[j] = p.tokens[seq + j];
        const int up = p.parent[seq + j];
        const bool ok = j == 0 ? up == -1 : up >= 0 && up < j;
        if (!ok && slice == 0 && split == 0) flag_status(p.status, kStatusCheck);
        s_parent[j] = ok ? up : -1;
      }
    __syncthreads();
    const int *ids = p.bias_ids + (long long)i * p.n_bias;
    const float *bias = p.bias + (long long)i * p.n_bias;
    for (int e = tid; e < p.n_bias; e += T) {
      const int id = ids[e];
      if (id < v0 || id >= v1) continue;
      atomicOr(&marked[(id - v0) >> 5], 1u << ((id - v0) & 31));
      uint32_t h = id_hash(id, hmask);
      while (true) {  // at most half of the slots are taken
        const int was = atomicCAS(&hkey[h], -1, id);
        if (was == -1 || was == id) break;
        h = (h + 1) & hmask;
      }
      atomicAdd(&hcount[h], 1);
    }
    if (p.parent)
      for (int j = tid; j < n; j += T) {
        unsigned long long line = 0;
        for (int a = j; s_parent[a] >= 0; a = s_parent[a]) line |= 1ull << a;
        s_line[j] = line;
        const int id = s_token[j];
        if (line >> j & 1 && id >= v0 && id < v1) atomicOr(&drafted[(id - v0) >> 5], 1u << ((id - v0) & 31));
      }
    __syncthreads();
    // An id that comes once has its bias; a warp together adds up what another id has, in the list's order,
    // whoever of its entries asks.
    for (int e0 = 32 * warp; e0 < p.n_bias; e0 += T) {
      const int e = e0 + lane;
      const int id = e < p.n_bias ? ids[e] : -1;
      const bool mine = id >= v0 && id < v1;
      uint32_t h = 0;
      if (mine) {
        h = id_hash(id, hmask);
        while (hkey[h] != id) h = (h + 1) & hmask;
        if (hcount[h] == 1) hsum[h] = bias[e];
      }
      unsigned again = __ballot_sync(0xffffffffu, mine && hcount[h] > 1);
      while (again) {
        const int from = __ffs(again) - 1;
        const int want = __shfl_sync(0xffffffffu, id, from);
        again &= ~__ballot_sync(0xffffffffu, id == want);
        float sum = 0.f;
        for (int q0 = 0; q0 < p.n_bias; q0 += 32) {
          const int q = q0 + lane;
          const bool same = q < p.n_bias && ids[q] == want;
          const float b = same ? bias[q] : 0.f;
          for (unsigned hit = __ballot_sync(0xffffffffu, same); hit; hit &= hit - 1)
            sum += __shfl_sync(0xffffffffu, b, __ffs(hit) - 1);
        }
        if (lane == from) hsum[h] = sum;  // other warps may write the same
      }
    }
    __syncthreads();
    for (int t = 0; t < tiles; ++t) {
      const int at0 = 4 * (warp * wt + t);  // the tile's words
      if (VEC) {
        const int w = at0 + (lane >> 3);
        listed |= ((marked[w] | drafted[w]) >> 4 * (lane & 7) & 15u) << 4 * t;
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) listed |= ((marked[at0 + q] | drafted[at0 + q]) >> lane & 1) << (4 * t + q);
      }
    }
  }

  // ---- rows
  const float *x = p.x + seq * p.ldx + base;
  float *y = p.y ? p.y + seq * p.ldy + base : nullptr;
  const uint32_t *allowed = MASK ? p.allowed + seq * p.words + (base >> 5) : nullptr;
  const int left = (v1 - base + 31) >> 5;  // words of the warp
  uint32_t words = 0;                      // the lane's word of listed tokens
  int before = 0, total = 0;               // of the lanes before, and of all
  int step = 0;
  for (int j = j0; j < j1; j += RPC) {
    uint32_t may[RPC];  // word `lane` of a row's mask
#pragma unroll
    for (int r = 0; r < RPC; ++r)
      if (MASK) may[r] = lane < left ? __ldg(allowed + (long long)min(j + r, j1 - 1) * p.words + lane) : 0u;
    float best[RPC];   // of the values that are not listed, and where: VEC, the first of their four
    int best_at[RPC];
#pragma unroll
    for (int r = 0; r < RPC; ++r) {
      best[r] = -INFINITY;
      best_at[r] = -1;
    }
    for (int t = 0; t < tiles; ++t, ++step) {
      const int e = 128 * t + (VEC ? 4 : 1) * lane;
      const bool in = base + e < v1;
      uint32_t ok[RPC];  // bits of this lane's four values
      if (VEC) {
        const int from = 4 * t + (lane >> 3), sh = 4 * (lane & 7);
#pragma unroll
        for (int r = 0; r < RPC; ++r)
          if (MASK) ok[r] = __shfl_sync(0xffffffffu, may[r], from) >> sh;
      } else {
#pragma unroll
        for (int r = 0; r < RPC; ++r) {
          ok[r] = 0;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (MASK) ok[r] |= (__shfl_sync(0xffffffffu, may[r], 4 * t + q) >> lane & 1) << q;
        }
      }
      float z[RPC][4];
      fetch(step + S - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
      if (RPC == 1 && counts && (in || !VEC)) {
        const int *c = reinterpret_cast<const int *>(ring + (step % S * SLOTS + 1) * 128);
        if (VEC) {
          listed |= some_of(*reinterpret_cast<const int4 *>(c)) << 4 * t;
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (base + e + 32 * q < v1) listed |= (c[32 * q] != 0 ? 1u : 0u) << (4 * t + q);
        }
      }
      const uint32_t sp = listed >> 4 * t;
      float out[4];  // takes listed values from the maximum, and keeps a NaN one
#pragma unroll
      for (int q = 0; q < 4; ++q) out[q] = sp >> q & 1 ? -INFINITY : 0.f;
#pragma unroll
      for (int r = 0; r < RPC; ++r) {
        const float *at_r = ring + (step % S * SLOTS + r) * 128;
        if (VEC) {
          const float4 w = *reinterpret_cast<const float4 *>(at_r);
          z[r][0] = w.x, z[r][1] = w.y, z[r][2] = w.z, z[r][3] = w.w;
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) z[r][q] = base + e + 32 * q < v1 ? at_r[32 * q] : -INFINITY;
        }
      }
#pragma unroll
      for (int r = 0; r < RPC; ++r) {
        if (MASK) {
#pragma unroll
          for (int q = 0; q < 4; ++q) z[r][q] = ok[r] >> q & 1 ? z[r][q] : -INFINITY;
        }
        if (y) {
          float *to = y + min(j + r, j1 - 1) * p.ldy + e;
          if (VEC) {
            if (in) *reinterpret_cast<float4 *>(to) = make_float4(z[r][0], z[r][1], z[r][2], z[r][3]);
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (base + e + 32 * q < v1) to[32 * q] = z[r][q];
          }
        }
        // places rise here, so the first of equals stays
        if (VEC) {
          const float m = fmaxf(fmaxf(z[r][0] + out[0], z[r][1] + out[1]), fmaxf(z[r][2] + out[2], z[r][3] + out[3]));
          const bool more = in && m > best[r];
          best[r] = more ? m : best[r];
          best_at[r] = more ? e : best_at[r];
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float m = z[r][q] + out[q];
            const bool more = m > best[r];
            best[r] = more ? m : best[r];
            best_at[r] = more ? e + 32 * q : best_at[r];
          }
        }
      }
    }
    __syncwarp();  // the listed values of y are written again by other lanes
    if (j == j0) {
      // the same by words of 32 tokens in a row, one a lane: neighbours are worked off together
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        if (t >= tiles) break;
        if (VEC) {
          uint32_t w = (listed >> 4 * t & 15u) << 4 * (lane & 7);
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) w |= __shfl_xor_sync(0xffffffffu, w, o);
          w = __shfl_sync(0xffffffffu, w, 8 * (lane & 3));
          if (lane >> 2 == t) words = w;
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t w = __ballot_sync(0xffffffffu, listed >> (4 * t + q) & 1);
            if (lane == 4 * t + q) words = w;
          }
        }
      }
      const int ones = __popc(words);
      before = ones;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += up;
      }
      total = __shfl_sync(0xffffffffu, before, 31);
      before -= ones;
    }
    float top[RPC];
    int top_at[RPC];
#pragma unroll
    for (int r = 0; r < RPC; ++r) {
      top[r] = -INFINITY;
      top_at[r] = -1;
    }
    for (int k0 = 0; k0 < total; k0 += 32) {
      // lane k takes the listed token of number k: in the last word with fewer before it
      const int k = k0 + lane;
      int from = 0;
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const int b = __shfl_sync(0xffffffffu, before, from + o);
        if (b <= k) from += o;
      }
      uint32_t w = __shfl_sync(0xffffffffu, words, from);
      const int skip = k - __shfl_sync(0xffffffffu, before, from);
      uint32_t mw[RPC];
#pragma unroll
      for (int r = 0; r < RPC; ++r)
        if (MASK) mw[r] = __shfl_sync(0xffffffffu, may[r], from);
      if (k >= total) continue;
      for (int s = 0; s < skip; ++s) w &= w - 1;
      const int bit = __ffs(w) - 1;
      const int e = 32 * from + bit, id = base + e;
      float z[RPC];
#pragma unroll
      for (int r = 0; r < RPC; ++r) z[r] = x[min(j + r, j1 - 1) * p.ldx + e];
      const int count = counts ? __ldg(counts + e) : 0;
      float add = 0.f;
      unsigned long long nodes = 0;  // with this token
      if (p.parent && drafted[(id - v0) >> 5] >> bit & 1)
        for (int a = 1; a < n; ++a) nodes |= static_cast<unsigned long long>(s_token[a] == id) << a;
      if (p.n_bias && marked[(id - v0) >> 5] >> bit & 1) {
        uint32_t h = id_hash(id, hmask);
        while (hkey[h] != id) h = (h + 1) & hmask;
        add = hsum[h];
      }
#pragma unroll
      for (int r = 0; r < RPC; ++r) {
        const int again = nodes ? __popcll(s_line[min(j + r, j1 - 1)] & nodes) : 0;
        const float v = !MASK || mw[r] >> bit & 1 ? adjust(z[r], count, again, rules) + add : -INFINITY;
        if (y) y[min(j + r, j1 - 1) * p.ldy + e] = v;
        if (v > top[r]) {  // places rise
          top[r] = v;
          top_at[r] = e;
        }
      }
    }
    __syncwarp();
    if (p.ids) {
#pragma unroll
      for (int r = 0; r < RPC; ++r) {
        const float b = warp_max(best[r]), w = warp_max(top[r]);
        unsigned at_b = __reduce_min_sync(0xffffffffu, best[r] == b ? static_cast<unsigned>(best_at[r]) : 0xffffffffu);
        const unsigned at_w =
            __reduce_min_sync(0xffffffffu, top[r] == w ? static_cast<unsigned>(top_at[r]) : 0xffffffffu);
        if (VEC && at_b != 0xffffffffu) {  // which of the four: the first that is the maximum, allowed and not listed
          const uint32_t good = (MASK ? __shfl_sync(0xffffffffu, may[r], at_b >> 5) : ~0u) &
                                ~__shfl_sync(0xffffffffu, words, at_b >> 5);
          const float mine = lane < 4 ? x[min(j + r, j1 - 1) * p.ldx + at_b + lane] : 0.f;
          const unsigned hit = __ballot_sync(0xffffffffu, lane < 4 && mine == b && (good >> ((at_b & 31) + lane) & 1));
          at_b += __ffs(hit) - 1;
        }
        float v = b;
        int id = at_b == 0xffffffffu ? -1 : base + static_cast<int>(at_b);
        take_best(v, id, w, at_w == 0xffffffffu ? -1 : base + static_cast<int>(at_w));
        if (lane == 0 && j + r < j1) {
          s_val[j + r][warp] = v;
          s_id[j + r][warp] = id;
        }
      }
    }
  }
  if (!p.ids) return;
  __syncthreads();
  for (int j = j0 + tid; j < j1; j += T) {
    float b = -INFINITY;
    int id = -1;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) take_best(b, id, s_val[j][k], s_id[j][k]);
    p.part[(seq + j) * p.slices + slice] = make_float2(b, __int_as_float(id));
  }
}

// The id of each row among its slices' best: one warp a row.
__global__ void __launch_bounds__(128) logits_ids_kernel(const LogitsParams p) {
  const int lane = threadIdx.x & 31;
  const long long r = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  griddep_wait();
  griddep_launch();
  if (r >= (long long)p.nb * p.m) return;
  if (p.n_rows && static_cast<int>(r % p.m) >= p.n_rows[r / p.m]) return;
  float b = -INFINITY;
  int id = -1;
  for (int s = lane; s < p.slices; s += 32) {
    const float2 o = p.part[r * p.slices + s];
    take_best(b, id, o.x, __float_as_int(o.y));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1)
    take_best(b, id, __shfl_xor_sync(0xffffffffu, b, o), __shfl_xor_sync(0xffffffffu, id, o));
  if (lane == 0) p.ids[r] = id;
}

// counts[i][token] += 1, or its top bit set. Lanes of a warp with the same token send one update of
// their number: frequent tokens would queue up at one address. Sums of whole numbers: any order. Latency: a launch,
// the tokens, an update each (64 sequences of 5 tokens 1.1 us, 8 prompts of 8189 2.0).
__global__ void __launch_bounds__(256) token_counts_kernel(const TokenCountsParams p) {
  griddep_wait();
  griddep_launch();
  const int i = blockIdx.y;
  const int t = blockIdx.x * 256 + threadIdx.x;
  int n = p.n_tokens ? p.n_tokens[i] : p.n;
  bool bad = n < 0 || n > p.n;
  n = max(0, min(n, p.n));
  const bool live = t < n;
  const int id = t < p.n ? p.tokens[(long long)i * p.ld + t] : -1;
  const bool fits = live && id >= 0 && id < p.V;
  bad |= live && !fits;
  if (__any_sync(0xffffffffu, bad) && (threadIdx.x & 31) == 0) flag_status(p.status, kStatusCheck);
  const unsigned same = __match_any_sync(0xffffffffu, fits ? id : -1);
  if (fits && (threadIdx.x & 31) == __ffs(same) - 1) {
    int *at = p.counts + (long long)i * p.V + id;
    if (p.prompt)
      atomicOr(at, static_cast<int>(0x80000000u));
    else
      atomicAdd(at, __popc(same));
  }
}

template <int RPC, int S, bool VEC, bool MASK>
cudaError_t launch_adjust(LogitsParams &p, int tiles, int rows, cudaStream_t s) {
  p.chunk = tiles * 128 * kWarps;
  p.slices = (p.V + p.chunk - 1) / p.chunk;
  p.rows = rows;
  p.splits = (p.m + rows - 1) / rows;
  p.hash = 0;
  if (p.n_bias > 0)
    for (p.hash = 32; p.hash < 2 * p.n_bias;) p.hash *= 2;
  const size_t smem = kWarps * S * ring_slots(RPC) * 512 + (size_t)p.hash * 12;
  static OncePerDevice once;
  cudaError_t e = once([] {
    return cudaFuncSetAttribute(logits_adjust_kernel<RPC, S, VEC, MASK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                100 * 1024);
  });
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>((long long)p.nb * p.splits * p.slices));
  e = launch_pdl(logits_adjust_kernel<RPC, S, VEC, MASK>, grid, dim3(32 * kWarps), smem, s, p);
  if (e != cudaSuccess || !p.ids) return e;
  const long long all = (long long)p.nb * p.m;
  return launch_pdl(logits_ids_kernel, dim3(static_cast<unsigned>((all + 3) / 4)), dim3(128), 0, s, p);
}

template <int RPC, int S>
cudaError_t launch_adjust(LogitsParams &p, bool vec, int tiles, int rows, cudaStream_t s) {
  if (vec)
    return p.allowed ? launch_adjust<RPC, S, true, true>(p, tiles, rows, s)
                     : launch_adjust<RPC, S, true, false>(p, tiles, rows, s);
  return p.allowed ? launch_adjust<RPC, S, false, true>(p, tiles, rows, s)
                   : launch_adjust<RPC, S, false, false>(p, tiles, rows, s);
}

}  // namespace

cudaError_t launch_logits_adjust(LogitsParams &p, int num_sms, cudaStream_t s) {
  auto aligned = [](const void *q, long long ld) { return reinterpret_cast<uintptr_t>(q) % 16 == 0 && ld % 4 == 0; };
  const bool vec = aligned(p.x, p.ldx) && (!p.y || aligned(p.y, p.ldy)) && (!p.counts || aligned(p.counts, p.V)) &&
                   p.V % 4 == 0;
  // Two rows at a time, a warp of 1024 tokens for as many rows of a sequence as leave two CTAs a SM (1024 rows of
  // 151936: 232 us, one at a time 240, four 251; 8 x 16 rows 40, in 1216 CTAs 48), six where values come one by one
  // (1024 rows of 32003: 51 us, with two 81). Fewer tokens a warp where there are fewer CTAs, or tokens (16 rows:
  // 11.7 us, with 1024 tokens 12.4; one row 6, with 1024 9).
  const int at_once = p.m > 1 ? 2 : 1;
  int tiles = kTiles;
  auto slices = [&] { return ((long long)p.V + tiles * 128 * kWarps - 1) / (tiles * 128 * kWarps); };
  while (tiles > 1 && slices() == 1 && tiles / 2 * 128 * kWarps >= p.V) tiles /= 2;
  const long long want = (vec ? 2LL : 6LL) * num_sms, have = p.nb * slices();
  const int parts = static_cast<int>(std::min<long long>(p.m, (want + have - 1) / have));
  const int rows = ((p.m + parts - 1) / parts + at_once - 1) / at_once * at_once;
  while (tiles > 1 && p.nb * slices() * ((p.m + rows - 1) / rows) < 7LL * num_sms / 4) {
    tiles /= 2;
    if (slices() > logit_slots(p.V)) {
      tiles *= 2;
      break;
    }
  }
  // Four stages: the ids of 1024 rows alone 125 us, with three 130; under all rules a row of 64 sequences 32 us, with
  // six 38.
  return at_once == 2 ? launch_adjust<2, 4>(p, vec, tiles, rows, s) : launch_adjust<1, 4>(p, vec, tiles, rows, s);
}

cudaError_t launch_token_counts(const TokenCountsParams &p, cudaStream_t s) {
  return launch_pdl(token_counts_kernel, dim3((p.n - 1) / 256 + 1, p.nb), dim3(256), 0, s, p);
}

}  // namespace df
