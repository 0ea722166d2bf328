// Bookkeeping of a draft tree on the device: ancestor masks, the accepted
// path, and the move of that path's K/V rows to the end of the cache.
//
// The tree form of the accepted prefix and the rewind of "cortiq-engine
// 0.8.49 src/mimo_mtp.rs" (mimo_spec_round, mimo_verify_rewind): node 0 is the
// pending token, a node's child is kept while its token equals the verifier's
// greedy token on the node's row, and rows off the kept path leave the cache.
// All three are a few hundred bytes of control data (or a few rows a head):
// one launch each, bound by launch latency.
#include <algorithm>

#include "tree.cuh"

namespace mtp {

// One thread a node.  A parent outside [-1, node) counts as -1 (code 5).
__global__ void __launch_bounds__(kTreeMax)
    tree_plan_kernel(const int* parents, int n, unsigned long long* mask, int* depth, int* err) {
  __shared__ int par[kTreeMax];
  pdl_wait();
  pdl_launch_dependents();
  const int i = threadIdx.x;
  if (i < n) {
    int p = parents[i];
    if (p < -1 || p >= i) {
      set_dev_error(err, kErrBadTree);
      p = -1;
    }
    par[i] = p;
  }
  __syncthreads();
  if (i >= n) return;
  unsigned long long m = 1ull << i;
  int d = 0;
  for (int p = par[i]; p >= 0; p = par[p]) {  // parents come before children: ends
    m |= 1ull << p;
    ++d;
  }
  mask[i] = m;
  depth[i] = d;
}

// One warp walks from node 0 to the lowest-index child that matches.
__global__ void __launch_bounds__(32)
    tree_accept_kernel(const int* parents, const int* tokens, const int* verify, int n, int* path,
                       int* emitted, int* count) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x;
  int par[2], tok[2], ver[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = lane + 32 * j;
    par[j] = i < n ? parents[i] : -2;
    tok[j] = i < n ? tokens[i] : 0;
    ver[j] = i < n ? verify[i] : 0;
  }
  int cur = 0, k = 0;
  int pth[2] = {-1, -1}, em[2] = {-1, -1};
  while (true) {
    const int v = __shfl_sync(0xffffffffu, cur < 32 ? ver[0] : ver[1], cur & 31);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (lane + 32 * j == k) {
        pth[j] = cur;
        em[j] = v;
      }
    ++k;
    const unsigned lo = __ballot_sync(0xffffffffu, par[0] == cur && tok[0] == v && lane > cur);
    const unsigned hi = __ballot_sync(0xffffffffu, par[1] == cur && tok[1] == v && lane + 32 > cur);
    if (!(lo | hi)) break;
    cur = lo ? __ffs(lo) - 1 : 31 + __ffs(hi);  // above the old one: at most n rounds
  }
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (lane + 32 * j < n) {
      path[lane + 32 * j] = pth[j];
      emitted[lane + 32 * j] = em[j];
    }
  if (lane == 0) *count = k;
}

constexpr int kCommitLayers = 64;  // layers of one launch
struct CommitArgs {
  float* k[kCommitLayers];
  float* v[kCommitLayers];
  const int* path;
  int n;
  int nkv, dqk, dv;
  int L;
  long long cap;
  int* err;
};

// grid (KV heads, layers, K or V); one thread a 16-byte column.  Path entries
// satisfy path[j] >= j, so a row is read before any later step writes it.  Rows
// go one after another, each a read from memory behind the last one's write:
// 48 layers of 8 heads of 2 x 128 take 5, 12 and 19 us for 5, 32 and 60 rows.
__global__ void __launch_bounds__(64) kv_commit_kernel(const __grid_constant__ CommitArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int d = blockIdx.z ? a.dv : a.dqk;
  const int c = threadIdx.x * 4;
  if (c >= d) return;
  float* base = (blockIdx.z ? a.v[blockIdx.y] : a.k[blockIdx.y]) +
                ((size_t)blockIdx.x * a.cap + a.L) * d + c;
  for (int j = 0; j < a.n; ++j) {
    const int p = a.path[j];
    if (p < 0) break;
    if (p < j || p >= a.n) {
      set_dev_error(a.err, kErrBadTree);
      break;
    }
    if (p != j)
      *reinterpret_cast<float4*>(base + (size_t)j * d) =
          *reinterpret_cast<const float4*>(base + (size_t)p * d);
  }
}

static mtp_status check_nodes(int n, const char* who) {
  if (n < 1 || n > kTreeMax)
    return fail(MTP_ERR_UNSUPPORTED, std::string(who) + ": 1..64 nodes");
  return MTP_OK;
}

static bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace mtp

using namespace mtp;

extern "C" {

size_t mtp_tree_workspace_bytes(void) { return sizeof(WsHeader); }

mtp_status mtp_tree_plan(const int32_t* d_parents, int32_t n, uint64_t* d_mask, int32_t* d_depth,
                         void* d_ws, size_t ws_bytes, void* stream) {
  mtp_status s = check_nodes(n, "mtp_tree_plan");
  if (s != MTP_OK) return s;
  if (!d_parents || !d_mask || !d_depth)
    return fail(MTP_ERR_INVALID_ARG, "mtp_tree_plan: null pointer");
  if (!aligned4(d_parents) || !aligned4(d_depth) || (reinterpret_cast<uintptr_t>(d_mask) & 7))
    return fail(MTP_ERR_INVALID_ARG, "mtp_tree_plan: misaligned pointer");
  if (!d_ws || !aligned16(d_ws) || ws_bytes < sizeof(WsHeader))
    return fail(MTP_ERR_WORKSPACE, "mtp_tree_plan: workspace too small or misaligned");
  cudaError_t e = launch_pdl(tree_plan_kernel, dim3(1), kTreeMax, 0, static_cast<cudaStream_t>(stream),
                             d_parents, n, reinterpret_cast<unsigned long long*>(d_mask), d_depth,
                             &static_cast<WsHeader*>(d_ws)->err);
  if (e != cudaSuccess) return cuda_fail(e, "mtp_tree_plan launch");
  return MTP_OK;
}

mtp_status mtp_tree_accept(const int32_t* d_parents, const int32_t* d_tokens,
                           const int32_t* d_verify, int32_t n, int32_t* d_path, int32_t* d_emitted,
                           int32_t* d_count, void* stream) {
  mtp_status s = check_nodes(n, "mtp_tree_accept");
  if (s != MTP_OK) return s;
  if (!d_parents || !d_tokens || !d_verify || !d_path || !d_emitted || !d_count)
    return fail(MTP_ERR_INVALID_ARG, "mtp_tree_accept: null pointer");
  if (!aligned4(d_parents) || !aligned4(d_tokens) || !aligned4(d_verify) || !aligned4(d_path) ||
      !aligned4(d_emitted) || !aligned4(d_count))
    return fail(MTP_ERR_INVALID_ARG, "mtp_tree_accept: misaligned pointer");
  cudaError_t e = launch_pdl(tree_accept_kernel, dim3(1), 32, 0, static_cast<cudaStream_t>(stream),
                             d_parents, d_tokens, d_verify, n, d_path, d_emitted, d_count);
  if (e != cudaSuccess) return cuda_fail(e, "mtp_tree_accept launch");
  return MTP_OK;
}

mtp_status kv_tree_commit(const mtp_kv_caches* C, const int32_t* d_path, int32_t n,
                          int32_t cache_len, void* d_ws, size_t ws_bytes, void* stream) {
  mtp_status s = check_nodes(n, "kv_tree_commit");
  if (s != MTP_OK) return s;
  if (!C || !C->h_k || !C->h_v || !d_path)
    return fail(MTP_ERR_INVALID_ARG, "kv_tree_commit: null pointer");
  if (C->n_layers < 1 || C->n_layers > 4096 || C->n_kv_heads < 1 || C->n_kv_heads > 64)
    return fail(MTP_ERR_UNSUPPORTED, "kv_tree_commit: 1..4096 layers, 1..64 KV heads");
  if (C->head_dim_qk < 4 || C->head_dim_qk % 4 || C->head_dim_qk > 256 || C->head_dim_v < 4 ||
      C->head_dim_v % 4 || C->head_dim_v > 256)
    return fail(MTP_ERR_UNSUPPORTED, "kv_tree_commit: head dims must be multiples of 4, <= 256");
  if (cache_len < 0 || C->cache_cap < 1)
    return fail(MTP_ERR_INVALID_ARG, "kv_tree_commit: bad cache length");
  if ((int64_t)cache_len + n > C->cache_cap)
    return fail(MTP_ERR_CAPACITY, "kv_tree_commit: cache_len + n exceeds the cache capacity");
  for (int l = 0; l < C->n_layers; ++l)
    if (!C->h_k[l] || !C->h_v[l] || !aligned16(C->h_k[l]) || !aligned16(C->h_v[l]))
      return fail(MTP_ERR_INVALID_ARG, "kv_tree_commit: null or misaligned cache");
  if (!aligned4(d_path)) return fail(MTP_ERR_INVALID_ARG, "kv_tree_commit: misaligned path");
  if (!d_ws || !aligned16(d_ws) || ws_bytes < sizeof(WsHeader))
    return fail(MTP_ERR_WORKSPACE, "kv_tree_commit: workspace too small or misaligned");
  CommitArgs a = {};
  a.path = d_path;
  a.n = n;
  a.nkv = C->n_kv_heads;
  a.dqk = C->head_dim_qk;
  a.dv = C->head_dim_v;
  a.L = cache_len;
  a.cap = C->cache_cap;
  a.err = &static_cast<WsHeader*>(d_ws)->err;
  for (int l0 = 0; l0 < C->n_layers; l0 += kCommitLayers) {
    const int nl = std::min(kCommitLayers, C->n_layers - l0);
    for (int l = 0; l < nl; ++l) {
      a.k[l] = C->h_k[l0 + l];
      a.v[l] = C->h_v[l0 + l];
    }
    cudaError_t e = launch_pdl(kv_commit_kernel, dim3(a.nkv, nl, 2), 64, 0,
                               static_cast<cudaStream_t>(stream), a);
    if (e != cudaSuccess) return cuda_fail(e, "kv_tree_commit launch");
  }
  return MTP_OK;
}

}  // extern "C"
