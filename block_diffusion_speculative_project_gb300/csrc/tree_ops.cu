// Walk of a drafted tree along the target's tokens, and the move of the accepted path's cache rows.
//
// A tree has up to kTreeMax nodes; node 0 is its root, the last committed token, and every other
// node's parent has a lower index. The greedy walk is the tree form of the accept rule of
// "DFlash 投机解码：块扩散草稿与 KV 注入" (符号约定: tau counts the bonus token).
#include "common.cuh"
#include "kernels.h"

namespace df {

namespace {

// Register k of lane j % 32 holds node j = 32 k + lane.
__device__ __forceinline__ int node_value(const int (&v)[2], int j) {
  const int a = __shfl_sync(0xffffffffu, v[0], j & 31), b = __shfl_sync(0xffffffffu, v[1], j & 31);
  return j < 32 ? a : b;
}

constexpr int kAcceptWarps = 4;

// One warp per sequence, two nodes per lane: every load first, then a step of the walk is two ballots
// (the lowest child whose token is the target's). Latency: a launch, one round of loads, depth * ~30 cycles
// (one tree of 16 nodes 1.4 us, 64 of 64 nodes 1.8 in a graph).
// It lets the next launch begin only at its end: a call's kernels may read lengths before they wait.
__global__ void __launch_bounds__(kAcceptWarps * 32) accept_tree_kernel(const AcceptTreeParams p) {
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * kAcceptWarps + (threadIdx.x >> 5);
  if (i >= p.nb) return;
  int n = p.m, ctx = 0;
  if (p.n_rows) n = p.n_rows[i];
  if (p.ctx_len && lane == 0) ctx = p.ctx_len[i];
  int parent[2], token[2], target[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int j = lane + 32 * k;
    const long long at = (long long)i * p.m + j;
    parent[k] = j < p.m ? p.parent[at] : -1;
    token[k] = j < p.m ? p.tokens[at] : -1;
    target[k] = j < p.m ? p.target[at] : -1;
  }
  bool bad = n < 0 || n > p.m;
  n = max(0, min(n, p.m));
  bool fits[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int j = lane + 32 * k;
    const bool has = j > 0 && j < n && parent[k] >= 0 && parent[k] < j;
    bad |= j < n && (j == 0 ? parent[k] != -1 : !has);
    const int want = node_value(target, has ? parent[k] : 0);
    fits[k] = has && token[k] >= 0 && token[k] == want;
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) flag_status(p.status, kStatusCheck);
  int path[2] = {-1, -1};
  int tau = 0, cur = n > 0 ? 0 : -1, last = 0;
  while (cur >= 0) {  // a child's index is above its parent's: at most n steps
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (lane + 32 * k == tau) path[k] = cur;
    ++tau;
    last = cur;
    const unsigned b0 = __ballot_sync(0xffffffffu, fits[0] && parent[0] == cur);
    const unsigned b1 = __ballot_sync(0xffffffffu, fits[1] && parent[1] == cur);
    cur = b0 ? __ffs(b0) - 1 : b1 ? 31 + __ffs(b1) : -1;
  }
  const int bonus = node_value(target, last);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int j = lane + 32 * k;
    // an accepted node's token is the one the target gave behind its parent
    const int out = node_value(target, max(0, path[k]));
    if (j < p.m) {
      if (p.out_path) p.out_path[(long long)i * p.m + j] = path[k];
      if (p.out_tokens) p.out_tokens[(long long)i * p.m + j] = path[k] >= 0 ? out : -1;
    }
  }
  if (lane == 0) {
    p.out_tau[i] = tau;
    p.out_bonus[i] = n > 0 ? bonus : -1;
    if (p.ctx_len) p.ctx_len[i] = ctx + tau;
  }
}

constexpr int kCommitWarps = 4;
constexpr int kCommitLoads = 8;  // 16-byte loads of a lane in flight

// One warp per (sequence, layer, kv head, K or V): rows base + path[t] move to base + t. Rows go in
// batches of kCommitLoads loads a lane, a batch read whole before it is written: a later batch reads
// rows path[t] >= t, behind everything that an earlier one wrote. The tree's rows lie in two pages at
// most, so the table's entries come with two loads. Latency: lengths and path, table, rows (one sequence's path of
// 5 layers 2.0 us, of 64 sequences 4.7, 17 MB).
template <int HD>
__global__ void __launch_bounds__(kCommitWarps * 32) kv_commit_kernel(const KvCommitParams p) {
  constexpr int LPR = HD / 8;      // lanes of a row
  constexpr int RPI = 32 / LPR;    // rows of a warp's load
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31;
  const int slices = 2 * p.layers * p.Hkv;
  const long long w = (long long)blockIdx.x * kCommitWarps + (threadIdx.x >> 5);
  const int i = static_cast<int>(w / slices), s = static_cast<int>(w % slices);
  if (i >= p.nb) return;
  int tau = p.tau[i];
  const int len = p.ctx_len[i];
  int path[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) path[k] = lane + 32 * k < p.m ? p.path[(long long)i * p.m + lane + 32 * k] : -1;
  bool bad = tau < 0 || tau > p.m || len < tau || len > p.Cmax;
  tau = max(0, min(tau, p.m));
  const int base = len - tau;
  if (bad) tau = 0;
  // row t moves if its source lies behind it: t < path[t] < m, rising
  int moves[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int t = lane + 32 * k;
    int before = __shfl_up_sync(0xffffffffu, path[k], 1);
    const int carry = __shfl_sync(0xffffffffu, path[0], 31);
    if (lane == 0) before = k ? carry : -1;
    const bool ok = t >= tau || (path[k] >= t && path[k] < p.m && path[k] > before && base + path[k] < p.Cmax);
    bad |= !ok;
    moves[k] = ok && t < tau && path[k] > t ? path[k] : -1;
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0 && s == 0) flag_status(p.status, kStatusCheck);
  const unsigned any0 = __ballot_sync(0xffffffffu, moves[0] >= 0), any1 = __ballot_sync(0xffffffffu, moves[1] >= 0);
  if (!(any0 | any1)) return;
  const int first = any0 ? __ffs(any0) - 1 : 31 + __ffs(any1);
  const int g = (s >> 1) % p.Hkv, layer = (s >> 1) / p.Hkv;
  uint16_t *cache = p.cache[s & 1] + (long long)layer * p.layer_rows * HD;
  long long block[2];  // row of the cache where each of the two pages begins, for this kv head
  int page0 = 0;
  if (p.page_table) {
    page0 = base / kPageRows;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int pg = page0 + k < p.pages_per_seq ? p.page_table[(long long)i * p.pages_per_seq + page0 + k] : -1;
      block[k] = pg >= 0 && pg < p.num_pages ? ((long long)pg * p.Hkv + g) * kPageRows : -1;
    }
  } else {
    block[0] = ((long long)i * p.Hkv + g) * p.Cmax;
    block[1] = block[0] + kPageRows;
  }
  const int row0 = base - page0 * kPageRows;  // base counted from block[0]
  auto row = [&](int t) -> uint16_t * {
    const int r = row0 + t;
    if (!p.page_table) return cache + (block[0] + r) * HD;
    const long long b = block[r >= kPageRows];
    return b < 0 ? nullptr : cache + (b + r % kPageRows) * HD;
  };
  const int col = lane % LPR * 8, sub = lane / LPR;
  bool lost = false;
  for (int t0 = first; t0 < tau; t0 += RPI * kCommitLoads) {
    uint4 v[kCommitLoads];
    bool live[kCommitLoads];
#pragma unroll
    for (int q = 0; q < kCommitLoads; ++q) {
      const int t = t0 + q * RPI + sub;
      const int src = node_value(moves, min(t, kTreeMax - 1));
      live[q] = t < tau && src >= 0;
      if (live[q]) {
        const uint16_t *from = row(src);
        live[q] = from != nullptr && row(t) != nullptr;
        lost |= !live[q];
        if (live[q]) v[q] = *reinterpret_cast<const uint4 *>(from + col);
      }
    }
    __syncwarp();
#pragma unroll
    for (int q = 0; q < kCommitLoads; ++q)
      if (live[q]) *reinterpret_cast<uint4 *>(row(t0 + q * RPI + sub) + col) = v[q];
    __syncwarp();
  }
  if (lost) flag_status(p.status, kStatusCheck);
}

}  // namespace

cudaError_t launch_accept_tree(const AcceptTreeParams &p, cudaStream_t s) {
  return launch_pdl(accept_tree_kernel, dim3((p.nb - 1) / kAcceptWarps + 1), dim3(kAcceptWarps * 32), 0, s,
                    p);
}

cudaError_t launch_kv_commit(const KvCommitParams &p, cudaStream_t s) {
  const long long warps = 2LL * p.layers * p.Hkv * p.nb;
  const dim3 grid(static_cast<unsigned>((warps + kCommitWarps - 1) / kCommitWarps));
  switch (p.hd) {
    case 64: return launch_pdl(kv_commit_kernel<64>, grid, dim3(kCommitWarps * 32), 0, s, p);
    case 128: return launch_pdl(kv_commit_kernel<128>, grid, dim3(kCommitWarps * 32), 0, s, p);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace df
