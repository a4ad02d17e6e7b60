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
// counts, a bit a value for the mask. A CTA takes a slice of the vocabulary for a few rows of one
// sequence, so that the counts are loaded once for them; the CTAs of a row are a cluster, whose first
// one picks the row's id through distributed shared memory, without scratch or a second launch.
// Biased and drafted tokens are few: a bitmap of the slice in shared memory marks them, and only marked
// values look their biases up (a hash of the slice's biased ids) and count the drafted nodes.
#include <cfloat>

#include "common.cuh"
#include "kernels.h"

namespace df {

namespace {

constexpr int kMaxSlice = 152 * 1024;    // values of a slice: the bitmap's 19 KB
constexpr int kSlices = 8;               // CTAs of a row: a portable cluster

__device__ __forceinline__ uint32_t id_hash(int id, uint32_t mask) { return (static_cast<uint32_t>(id) * 2654435761u >> 12) & mask; }

// Better of two (value, id) pairs: larger value, then lower id; id -1: none.
__device__ __forceinline__ void take_best(float &v, int &id, float w, int wid) {
  const bool better = w > v || (w == v && wid >= 0 && (id < 0 || wid < id));
  v = better ? w : v;
  id = better ? wid : id;
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

template <int T, int RPC, int U, bool VEC>
__global__ void __launch_bounds__(T) logits_adjust_kernel(const LogitsParams p) {
  extern __shared__ uint32_t dyn[];
  __shared__ int s_token[kTreeMax];
  __shared__ int s_parent[kTreeMax];
  __shared__ unsigned long long s_line[kTreeMax];  // drafted nodes from a node up
  __shared__ float s_val[RPC][T / 32];
  __shared__ int s_id[RPC][T / 32];
  __shared__ float4 s_best[RPC];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int slice = blockIdx.x % p.slices;
  const int at = blockIdx.x / p.slices;
  const int i = at / p.groups, grp = at % p.groups;
  const int v0 = min(p.V, slice * p.chunk), v1 = min(p.V, v0 + p.chunk);
  const int nwords = (p.chunk + 31) / 32;
  uint32_t *marked = dyn;                                     // [nwords]
  int *hkey = reinterpret_cast<int *>(dyn + nwords);          // [hash]: id, -1 free
  int *hfirst = hkey + p.hash;                                // first place in the list
  int *hcount = hfirst + p.hash;
  float *hsum = reinterpret_cast<float *>(hcount + p.hash);
  const bool special = p.n_bias > 0 || p.parent != nullptr;
  if (special) {
    for (int e = tid; e < nwords; e += T) marked[e] = 0;
    for (int e = tid; e < p.hash; e += T) {
      hkey[e] = -1;
      hfirst[e] = 0x7fffffff;
      hcount[e] = 0;
    }
  }
  griddep_wait();
  griddep_launch();
  int n = p.n_rows ? p.n_rows[i] : p.m;
  if ((n < 0 || n > p.m) && slice == 0 && grp == 0 && tid == 0) flag_status(p.status, kStatusCheck);
  n = max(0, min(n, p.m));
  const int j0 = grp * RPC;
  const int rows = min(RPC, n - j0);
  if (rows <= 0) return;  // the same for a whole cluster
  RowRules rules = {1.f, 0.f, 0.f};
  if (p.penalties) {
    rules.rep = p.penalties[3 * i];
    rules.freq = p.penalties[3 * i + 1];
    rules.pres = p.penalties[3 * i + 2];
  }
  const uint32_t hmask = p.hash - 1;
  if (special) {
    if (p.parent)
      for (int j = tid; j < n; j += T) {
        s_token[j] = p.tokens[(long long)i * p.m + j];
        const int up = p.parent[(long long)i * p.m + j];
        const bool ok = j == 0 ? up == -1 : up >= 0 && up < j;
        if (!ok && slice == 0 && grp == 0) flag_status(p.status, kStatusCheck);
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
      atomicMin(&hfirst[h], e);
    }
    if (p.parent)
      for (int j = tid; j < n; j += T) {
        unsigned long long line = 0;
        for (int a = j; s_parent[a] >= 0; a = s_parent[a]) line |= 1ull << a;
        s_line[j] = line;
        const int id = s_token[j];
        if (line >> j & 1 && id >= v0 && id < v1) atomicOr(&marked[(id - v0) >> 5], 1u << ((id - v0) & 31));
      }
    __syncthreads();
    // an id's first entry adds the others up, in the list's order
    for (int e = tid; e < p.n_bias; e += T) {
      const int id = ids[e];
      if (id < v0 || id >= v1) continue;
      uint32_t h = id_hash(id, hmask);
      while (hkey[h] != id) h = (h + 1) & hmask;
      if (hfirst[h] != e) continue;
      float sum = bias[e];
      for (int left = hcount[h] - 1, q = e + 1; left > 0 && q < p.n_bias; ++q)
        if (ids[q] == id) {
          sum += bias[q];
          --left;
        }
      hsum[h] = sum;
    }
    __syncthreads();
  }

  const long long row0 = (long long)i * p.m + j0;
  const float *x = p.x + row0 * p.ldx;
  float *y = p.y ? p.y + row0 * p.ldy : nullptr;
  const int *counts = p.counts ? p.counts + (long long)i * p.V : nullptr;
  const uint32_t *allowed = p.allowed ? p.allowed + row0 * p.words : nullptr;
  float best[RPC];
  int best_id[RPC];
#pragma unroll
  for (int r = 0; r < RPC; ++r) {
    best[r] = -INFINITY;
    best_id[r] = -1;
  }
  for (int v = v0 + 4 * tid; v < v1; v += 4 * T * U) {
    float a[U][RPC][4];
    int c[U][4];
    uint32_t ok[U][RPC];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = v + u * 4 * T;
      if (g >= v1) continue;
      if (VEC) {
        const int4 w = counts ? __ldg(reinterpret_cast<const int4 *>(counts + g)) : make_int4(0, 0, 0, 0);
        c[u][0] = w.x, c[u][1] = w.y, c[u][2] = w.z, c[u][3] = w.w;
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) c[u][q] = counts && g + q < v1 ? __ldg(counts + g + q) : 0;
      }
#pragma unroll
      for (int r = 0; r < RPC; ++r) {
        if (r >= rows) continue;
        ok[u][r] = allowed ? __ldg(allowed + (long long)r * p.words + (g >> 5)) >> (g & 31) : ~0u;
        const float *from = x + r * p.ldx + g;
        if (VEC) {
          const float4 w = *reinterpret_cast<const float4 *>(from);
          a[u][r][0] = w.x, a[u][r][1] = w.y, a[u][r][2] = w.z, a[u][r][3] = w.w;
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) a[u][r][q] = g + q < v1 ? from[q] : -INFINITY;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = v + u * 4 * T;
      if (g >= v1) continue;
      const uint32_t sp = special ? marked[(g - v0) >> 5] >> ((g - v0) & 31) & 15u : 0u;
      const bool heard = (c[u][0] | c[u][1] | c[u][2] | c[u][3]) != 0;
#pragma unroll
      for (int r = 0; r < RPC; ++r) {
        if (r >= rows) continue;
        float(&z)[4] = a[u][r];
        if (sp) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            int drafted = 0;
            float add = 0.f;
            if (sp >> q & 1) {
              if (p.parent)
                for (unsigned long long line = s_line[j0 + r]; line; line &= line - 1)
                  drafted += s_token[__ffsll(line) - 1] == g + q;
              if (p.n_bias) {
                uint32_t h = id_hash(g + q, hmask);
                while (hkey[h] != -1 && hkey[h] != g + q) h = (h + 1) & hmask;
                if (hkey[h] != -1) add = hsum[h];
              }
            }
            z[q] = adjust(z[q], c[u][q], drafted, rules) + add;
          }
        } else if (heard) {
#pragma unroll
          for (int q = 0; q < 4; ++q) z[q] = adjust(z[q], c[u][q], 0, rules);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (!(ok[u][r] >> q & 1)) z[q] = -INFINITY;
        if (y) {
          float *to = y + r * p.ldy + g;
          if (VEC) {
            *reinterpret_cast<float4 *>(to) = make_float4(z[0], z[1], z[2], z[3]);
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (g + q < v1) to[q] = z[q];
          }
        }
        const float top = fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]));
        if (top > best[r]) {  // a thread's ids rise, so the first of equals stays
          best[r] = top;
          best_id[r] = g + (z[0] == top ? 0 : z[1] == top ? 1 : z[2] == top ? 2 : 3);
        }
      }
    }
  }
  if (!p.ids) return;
#pragma unroll
  for (int r = 0; r < RPC; ++r) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
      take_best(best[r], best_id[r], __shfl_xor_sync(0xffffffffu, best[r], o), __shfl_xor_sync(0xffffffffu, best_id[r], o));
    if (lane == 0) {
      s_val[r][warp] = best[r];
      s_id[r][warp] = best_id[r];
    }
  }
  __syncthreads();
  if (tid < rows) {
    float b = -INFINITY;
    int id = -1;
    for (int w = 0; w < T / 32; ++w) take_best(b, id, s_val[tid][w], s_id[tid][w]);
    s_best[tid] = make_float4(b, __int_as_float(id), 0.f, 0.f);
  }
  cluster_sync_all();
  if (slice == 0 && tid < rows) {
    float b = -INFINITY;
    int id = -1;
    for (int q = 0; q < p.slices; ++q) {
      const float4 o = ld_cluster_f4(cluster_map(smem_u32(&s_best[tid]), q));
      take_best(b, id, o.x, __float_as_int(o.y));
    }
    p.ids[row0 + tid] = id;
  }
  cluster_sync_all();  // the others' shared memory stays until it was read
}

// counts[i][token] += 1, or its top bit set. Lanes of a warp with the same token send one update of
// their number: frequent tokens would queue up at one address. Sums of whole numbers: any order.
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

template <int T, int RPC, int U, bool VEC>
cudaError_t launch_adjust(LogitsParams &p, cudaStream_t s) {
  p.groups = (p.m + RPC - 1) / RPC;
  p.slices = kSlices;
  // slices of whole mask words, the same length but for the last
  p.chunk = ((p.V + p.slices - 1) / p.slices + 31) / 32 * 32;
  p.hash = 0;
  if (p.n_bias > 0)
    for (p.hash = 32; p.hash < 2 * p.n_bias;) p.hash *= 2;
  size_t smem = 0;
  if (p.n_bias > 0 || p.parent) smem = (size_t)(p.chunk / 32 + 4 * p.hash) * 4;
  if (smem > 40 * 1024) {
    static const cudaError_t configured = cudaFuncSetAttribute(
        logits_adjust_kernel<T, RPC, U, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize, 96 * 1024);
    if (configured != cudaSuccess) return configured;
  }
  const dim3 grid(static_cast<unsigned>((long long)p.nb * p.groups * p.slices));
  return launch_pdl_cluster(logits_adjust_kernel<T, RPC, U, VEC>, grid, dim3(T), smem, s, p.slices, p);
}

template <int T, int RPC, int U>
cudaError_t launch_adjust(LogitsParams &p, bool vec, cudaStream_t s) {
  return vec ? launch_adjust<T, RPC, U, true>(p, s) : launch_adjust<T, RPC, U, false>(p, s);
}

}  // namespace

int logits_max_vocab() { return kSlices * kMaxSlice; }

cudaError_t launch_logits_adjust(LogitsParams &p, int num_sms, cudaStream_t s) {
  auto aligned = [](const void *q, long long ld) { return reinterpret_cast<uintptr_t>(q) % 16 == 0 && ld % 4 == 0; };
  const bool vec = aligned(p.x, p.ldx) && (!p.y || aligned(p.y, p.ldy)) && (!p.counts || aligned(p.counts, p.V)) &&
                   p.V % 4 == 0;
  // rows of one sequence that share the loads of its counts, where enough CTAs remain
  const long long ctas = (long long)p.nb * p.m * kSlices;
  if (p.m >= 4 && ctas >= 16LL * num_sms) return launch_adjust<256, 8, 1>(p, vec, s);
  return launch_adjust<512, 1, 4>(p, vec, s);
}

cudaError_t launch_token_counts(const TokenCountsParams &p, cudaStream_t s) {
  return launch_pdl(token_counts_kernel, dim3((p.n + 255) / 256, p.nb), dim3(256), 0, s, p);
}

}  // namespace df
