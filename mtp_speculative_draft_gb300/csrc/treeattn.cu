// Attention of a tree of drafted tokens over a cache.
//
// "hf2q 0.1.13 src/inference/models/qwen35/mtp.rs", forward_full_attention
// (per-head norm, rotation, cache append, attention, sigmoid gate) and
// "cortiq-engine 0.8.49 src/mimo_mtp.rs" (window, sinks), with the new rows'
// causal order replaced by the tree's: node i, at sequence position
// L + depth_i, sees the cached keys of its window and the new rows whose bit
// is set in its ancestor word.
//
// Three launches:
//   1. prep:   q heads normalised, rotated and scaled (log2 domain) to the
//              workspace; k heads normalised and rotated, v heads, appended to
//              cache rows L .. L + n - 1;
//   2. split:  every query row against the cached keys that all rows see,
//              [max(0, L + n - W), L) for a window W (a node's depth is below
//              n), split over CTAs: no mask at all.  Partials (m, l, o);
//   3. finish: one CTA a (node, head) joins the partials, the cached keys at
//              the window's edge (fewer than n, each row its own) and the
//              node's ancestors, read key by key, so a row that a mask hides
//              never enters any arithmetic; sink, gate, output.
#include <algorithm>
#include <cmath>

#include "tree.cuh"

namespace mtp {

constexpr float kLog2e = 1.4426950408889634f;

struct TreeAttnArgs {
  int nh, nkv, G, dqk, dv, n, L, window, gated;
  long long cap;
  float eps, qscale;  // qscale: logit scale times log2(e)
  const float *qp, *kp, *vp, *qn, *kn, *sinks;
  long long ldq, ldk, ldv;
  RopePos rope;
  float *kc, *vc;
  const unsigned long long* mask;
  const int* depth;
  float* out;
  float* qf;       // [nkv][R][dqk] scaled queries, row r = i * G + g
  int* dep;        // [n] depths inside [0, n)
  float* part_o;   // [nkv][ns][R][dv]
  float2* part_ml; // [nkv][ns][R] running maximum and sum
  int R, ns, kbeg, kper;  // query rows of a KV head, splits, first split key, keys a split
  int* err;
};

// ------------------------------------------------------------------ prep
constexpr int kPrepThreads = 128;

// One warp an item: n * nh query heads, then n * nkv key heads, then values.
__global__ void __launch_bounds__(kPrepThreads) tree_prep_kernel(const TreeAttnArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ int dep[kTreeMax];
  if (threadIdx.x < a.n) {
    int d = a.depth[threadIdx.x];
    if (d < 0 || d >= a.n) {
      set_dev_error(a.err, kErrBadTree);
      d = d < 0 ? 0 : a.n - 1;
    }
    dep[threadIdx.x] = d;
    if (blockIdx.x == 0) a.dep[threadIdx.x] = d;
  }
  __syncthreads();
  RopePos rp = a.rope;
  rp.depth = dep;
  const int lane = threadIdx.x & 31;
  int it = blockIdx.x * (kPrepThreads / 32) + (threadIdx.x >> 5);
  HeadVals v;
  if (it < a.n * a.nh) {
    const int i = it / a.nh, h = it % a.nh;
    const float* src = a.qp + (size_t)i * a.ldq + (size_t)h * a.dqk * (a.gated ? 2 : 1);
    head_norm_rope(v, src, a.dqk, a.qn, a.eps, rp, i, a.err, lane);
    const int kv = h / a.G, r = i * a.G + h % a.G;
    head_store(v, a.qf + ((size_t)kv * a.R + r) * a.dqk, a.dqk, rp.half, a.qscale, lane);
    return;
  }
  it -= a.n * a.nh;
  if (it < a.n * a.nkv) {
    const int i = it / a.nkv, kv = it % a.nkv;
    head_norm_rope(v, a.kp + (size_t)i * a.ldk + (size_t)kv * a.dqk, a.dqk, a.kn, a.eps, rp, i,
                   a.err, lane);
    head_store(v, a.kc + ((size_t)kv * a.cap + a.L + i) * a.dqk, a.dqk, rp.half, 1.f, lane);
    return;
  }
  it -= a.n * a.nkv;
  if (it < a.n * a.nkv) {
    const int i = it / a.nkv, kv = it % a.nkv;
    const float* src = a.vp + (size_t)i * a.ldv + (size_t)kv * a.dv;
    float* dst = a.vc + ((size_t)kv * a.cap + a.L + i) * a.dv;
    for (int c = lane; c < a.dv; c += 32) dst[c] = src[c];
  }
}

// A warp's running softmax state over up to 256 output dims: lane l holds dims
// l + 32 j.
struct RowState {
  float m, l;
  float o[8];
};

// One key against a warp's query row (dims lane + 32 j in q).
__device__ __forceinline__ void row_step(RowState& s, const float (&q)[8], const float* k,
                                         const float* v, int dqk, int dv, int lane) {
  float dot = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (32 * j < dqk) dot += q[j] * k[lane + 32 * j];
  dot = warp_sum(dot);
  if (!(dot <= s.m)) {  // a larger logit, or NaN, which then stays
    const float c = exp2f(s.m - dot);  // 0 at the first key (m = -inf)
    s.m = dot;
    s.l *= c;
#pragma unroll
    for (int j = 0; j < 8; ++j) s.o[j] *= c;
  }
  const float p = dot == -INFINITY ? 0.f : exp2f(dot - s.m);
  s.l += p;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (32 * j < dv) s.o[j] += p * v[lane + 32 * j];
}

// ------------------------------------------------------------------ split
constexpr int kSplitWarps = 8;

__global__ void __launch_bounds__(kSplitWarps * 32) tree_split_kernel(const TreeAttnArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int sp = blockIdx.x, kv = blockIdx.y, lane = threadIdx.x & 31;
  const int k0 = a.kbeg + sp * a.kper, k1 = min(a.L, k0 + a.kper);
  for (int r = threadIdx.x >> 5; r < a.R; r += kSplitWarps) {
    float q[8];
    RowState s;
    s.m = -INFINITY;
    s.l = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      q[j] = 32 * j < a.dqk ? a.qf[((size_t)kv * a.R + r) * a.dqk + lane + 32 * j] : 0.f;
      s.o[j] = 0.f;
    }
    for (int k = k0; k < k1; ++k)
      row_step(s, q, a.kc + ((size_t)kv * a.cap + k) * a.dqk, a.vc + ((size_t)kv * a.cap + k) * a.dv,
               a.dqk, a.dv, lane);
    const size_t at = ((size_t)kv * a.ns + sp) * a.R + r;
    if (lane == 0) a.part_ml[at] = make_float2(s.m, s.l);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (32 * j < a.dv) a.part_o[at * a.dv + lane + 32 * j] = s.o[j];
  }
}

// ------------------------------------------------------------------ finish
constexpr int kFinishWarps = 4;

__global__ void __launch_bounds__(kFinishWarps * 32) tree_finish_kernel(const TreeAttnArgs a) {
  __shared__ float sm_m[kFinishWarps], sm_l[kFinishWarps];
  __shared__ float sm_o[kFinishWarps][256];
  pdl_wait();
  pdl_launch_dependents();
  const int h = blockIdx.x, i = blockIdx.y, kv = h / a.G, r = i * a.G + h % a.G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float q[8];
  RowState s;
  s.m = -INFINITY;
  s.l = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    q[j] = 32 * j < a.dqk ? a.qf[((size_t)kv * a.R + r) * a.dqk + lane + 32 * j] : 0.f;
    s.o[j] = 0.f;
  }
  const float* kc = a.kc + (size_t)kv * a.cap * a.dqk;
  const float* vc = a.vc + (size_t)kv * a.cap * a.dv;
  const int dep = a.dep[i];
  // cached keys at the window's edge: seen by this row, not by every row
  if (a.window > 0) {
    const int e0 = max(0, a.L + dep - a.window + 1), e1 = min(a.L, a.kbeg);
    for (int k = e0 + warp; k < e1; k += kFinishWarps)
      row_step(s, q, kc + (size_t)k * a.dqk, vc + (size_t)k * a.dv, a.dqk, a.dv, lane);
  }
  // the node's ancestors
  unsigned long long m = a.mask[i];
  if (a.n < 64) m &= (1ull << a.n) - 1;
  for (int c = 0; m; ++c) {
    const int j = __ffsll(m) - 1;
    m &= m - 1;
    if (c % kFinishWarps != warp) continue;
    if (a.window > 0 && a.dep[j] <= dep - a.window) continue;
    row_step(s, q, kc + (size_t)(a.L + j) * a.dqk, vc + (size_t)(a.L + j) * a.dv, a.dqk, a.dv, lane);
  }
  // the splits' partials
  for (int sp = warp; sp < a.ns; sp += kFinishWarps) {
    const size_t at = ((size_t)kv * a.ns + sp) * a.R + r;
    const float2 ml = a.part_ml[at];
    if (ml.x == -INFINITY) continue;
    const float mn = fmaxf(s.m, ml.x);
    const float c0 = exp2f(s.m - mn), c1 = exp2f(ml.x - mn);
    s.m = mn;
    s.l = s.l * c0 + ml.y * c1;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (32 * j < a.dv) s.o[j] = s.o[j] * c0 + a.part_o[at * a.dv + lane + 32 * j] * c1;
  }
  if (lane == 0) {
    sm_m[warp] = s.m;
    sm_l[warp] = s.l;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (32 * j < a.dv) sm_o[warp][lane + 32 * j] = s.o[j];
  __syncthreads();
  const float sink = a.sinks ? a.sinks[h] * kLog2e : -INFINITY;
  float M = sink;
  for (int w = 0; w < kFinishWarps; ++w) M = fmaxf(M, sm_m[w]);
  float den = sink == -INFINITY ? 0.f : exp2f(sink - M);
  float wt[kFinishWarps];
#pragma unroll
  for (int w = 0; w < kFinishWarps; ++w) {
    wt[w] = sm_m[w] == -INFINITY ? 0.f : exp2f(sm_m[w] - M);
    den += wt[w] * sm_l[w];
  }
  const float inv = den > 0.f ? 1.f / den : den == 0.f ? 0.f : den;  // empty row: 0; NaN stays
  for (int c = threadIdx.x; c < a.dv; c += kFinishWarps * 32) {
    float o = 0.f;
#pragma unroll
    for (int w = 0; w < kFinishWarps; ++w) o += wt[w] * sm_o[w][c];
    o *= inv;
    if (a.gated) {
      const float g = a.qp[(size_t)i * a.ldq + ((size_t)2 * h + 1) * a.dqk + c];
      o *= 1.f / (1.f + expf(-g));
    }
    a.out[((size_t)i * a.nh + h) * a.dv + c] = o;
  }
}

// ------------------------------------------------------------------ host
struct TreePlan {
  int kbeg, ns, kper;
};

// Splits of the cached keys all rows see: about one CTA per SM.
static TreePlan tree_plan_splits(int nkv, int L, int window, int n) {
  TreePlan p;
  p.kbeg = window > 0 ? (int)std::min<int64_t>(L, std::max<int64_t>(0, (int64_t)L + n - window)) : 0;
  const int keys = L - p.kbeg;
  p.ns = 0;
  p.kper = 0;
  if (keys > 0) {
    int want = std::max(1, sm_count() / nkv);
    want = std::min(want, (keys + 31) / 32);
    p.kper = (keys + want - 1) / want;
    p.ns = (keys + p.kper - 1) / p.kper;
  }
  return p;
}

struct TreeWs {
  float* qf;
  int* dep;
  float2* ml;
  float* o;
  size_t bytes;
};

static TreeWs tree_ws(void* ws, const mtp_attn_geom* g, int n, int ns) {
  TreeWs w = {};
  size_t off = sizeof(WsHeader);
  uint8_t* b = static_cast<uint8_t*>(ws);
  auto take = [&](size_t bytes) {
    uint8_t* p = b ? b + off : nullptr;
    off = (off + bytes + 255) & ~size_t(255);
    return p;
  };
  const size_t rows = (size_t)n * g->n_heads;
  w.dep = reinterpret_cast<int*>(take(sizeof(int) * kTreeMax));
  w.qf = reinterpret_cast<float*>(take(4 * rows * g->head_dim_qk));
  w.ml = reinterpret_cast<float2*>(take(8 * rows * ns));
  w.o = reinterpret_cast<float*>(take(4 * rows * ns * g->head_dim_v));
  w.bytes = off;
  return w;
}

static mtp_status check_tree_geom(const mtp_attn_geom* g, int n) {
  if (!g) return fail(MTP_ERR_INVALID_ARG, "attn_tree_sink: null geometry");
  if (g->n_heads < 1 || g->n_kv_heads < 1 || g->n_heads % g->n_kv_heads)
    return fail(MTP_ERR_INVALID_ARG, "attn_tree_sink: n_kv_heads must divide n_heads");
  if (g->n_kv_heads > 64 || g->n_heads / g->n_kv_heads > 64)
    return fail(MTP_ERR_UNSUPPORTED, "attn_tree_sink: at most 64 KV heads of 64 query heads each");
  if (g->head_dim_qk < 32 || g->head_dim_qk % 32 || g->head_dim_qk > 256 || g->head_dim_v < 32 ||
      g->head_dim_v % 32 || g->head_dim_v > 256)
    return fail(MTP_ERR_UNSUPPORTED, "attn_tree_sink: head dims must be multiples of 32, <= 256");
  if (g->rot_dim < 0 || g->rot_dim % 2 || g->rot_dim > g->head_dim_qk)
    return fail(MTP_ERR_INVALID_ARG, "attn_tree_sink: rot_dim must be even and <= head_dim_qk");
  if (g->gated_q != 0 && g->gated_q != 1)
    return fail(MTP_ERR_INVALID_ARG, "attn_tree_sink: gated_q must be 0 or 1");
  if (g->gated_q && g->head_dim_v != g->head_dim_qk)
    return fail(MTP_ERR_UNSUPPORTED, "attn_tree_sink: gated q needs head_dim_v == head_dim_qk");
  if (!(g->eps >= 0.f) || !(g->scale >= 0.f) || !std::isfinite(g->scale))
    return fail(MTP_ERR_INVALID_ARG, "attn_tree_sink: eps and scale must be >= 0");
  if (n < 1 || n > kTreeMax) return fail(MTP_ERR_UNSUPPORTED, "attn_tree_sink: 1..64 nodes");
  return MTP_OK;
}

}  // namespace mtp

using namespace mtp;

extern "C" {

size_t attn_tree_sink_workspace_bytes(const mtp_attn_geom* g, int32_t n, int32_t cache_len) {
  if (!g || n < 1 || n > kTreeMax || cache_len < 0 || g->n_heads < 1 || g->n_kv_heads < 1 ||
      g->n_kv_heads > 64 || g->n_heads > 4096 || g->head_dim_qk < 1 || g->head_dim_qk > 256 ||
      g->head_dim_v < 1 || g->head_dim_v > 256)
    return 0;
  return tree_ws(nullptr, g, n, tree_plan_splits(g->n_kv_heads, cache_len, g->window, n).ns).bytes;
}

mtp_status attn_tree_sink(const mtp_attn_geom* g, const mtp_draft_tree* tree, const float* d_qp,
                          const float* d_kp, const float* d_vp, const float* d_q_norm,
                          const float* d_k_norm, const float* d_rope, int32_t rope_rows,
                          const float* d_sinks, float* d_k_cache, float* d_v_cache,
                          int32_t cache_len, int32_t cache_cap, float* d_out, void* d_ws,
                          size_t ws_bytes, void* stream) {
  if (!tree || !tree->d_mask || !tree->d_depth)
    return fail(MTP_ERR_INVALID_ARG, "attn_tree_sink: null tree");
  const int n = tree->n;
  mtp_status s = check_tree_geom(g, n);
  if (s != MTP_OK) return s;
  if (!d_qp || !d_kp || !d_vp || !d_k_cache || !d_v_cache || !d_out)
    return fail(MTP_ERR_INVALID_ARG, "attn_tree_sink: null pointer");
  if (!aligned16(d_qp) || !aligned16(d_kp) || !aligned16(d_vp) || !aligned16(d_k_cache) ||
      !aligned16(d_v_cache) || !aligned16(d_out) || !aligned16(d_q_norm) || !aligned16(d_k_norm) ||
      !aligned16(d_rope) || (reinterpret_cast<uintptr_t>(d_sinks) & 3) ||
      (reinterpret_cast<uintptr_t>(tree->d_mask) & 7) || (reinterpret_cast<uintptr_t>(tree->d_depth) & 3))
    return fail(MTP_ERR_INVALID_ARG, "attn_tree_sink: misaligned pointer");
  if (cache_len < 0 || cache_cap <= 0)
    return fail(MTP_ERR_INVALID_ARG, "attn_tree_sink: bad cache length");
  if ((int64_t)cache_len + n > cache_cap)
    return fail(MTP_ERR_CAPACITY, "attn_tree_sink: cache_len + n exceeds the cache capacity");
  TreeAttnArgs a = {};
  a.nh = g->n_heads;
  a.nkv = g->n_kv_heads;
  a.G = a.nh / a.nkv;
  a.dqk = g->head_dim_qk;
  a.dv = g->head_dim_v;
  a.n = n;
  a.L = cache_len;
  a.cap = cache_cap;
  a.window = g->window > 0 ? g->window : 0;
  a.gated = g->gated_q;
  a.eps = g->eps;
  a.qscale = (float)((g->scale > 0.f ? (double)g->scale : 1.0 / std::sqrt((double)a.dqk)) *
                     1.4426950408889634);
  const int64_t wq = (int64_t)a.nh * a.dqk * (a.gated ? 2 : 1), wk = (int64_t)a.nkv * a.dqk,
                wv = (int64_t)a.nkv * a.dv;
  a.ldq = tree->ld_q ? tree->ld_q : wq;
  a.ldk = tree->ld_k ? tree->ld_k : wk;
  a.ldv = tree->ld_v ? tree->ld_v : wv;
  if (a.ldq < wq || a.ldk < wk || a.ldv < wv || a.ldq % 4 || a.ldk % 4 || a.ldv % 4)
    return fail(MTP_ERR_INVALID_ARG,
                "attn_tree_sink: row strides must hold a row and be multiples of 4 floats");
  if (g->rot_dim == 0) {
    a.rope = RopePos{};
  } else if (tree->axes) {
    s = fill_rope_axes(&a.rope, tree->axes, g->rot_dim / 2, n, "attn_tree_sink");
    if (s != MTP_OK) return s;
  } else {
    if (!d_rope) return fail(MTP_ERR_INVALID_ARG, "attn_tree_sink: null rotary table");
    if (tree->pos_base < 0 || (int64_t)tree->pos_base + cache_len + n > rope_rows)
      return fail(MTP_ERR_INVALID_ARG, "attn_tree_sink: the rotary table is too short");
    a.rope.table = d_rope;
    a.rope.base = tree->pos_base + cache_len;
    a.rope.max_pos = rope_rows;
    a.rope.n_axes = 1;
    a.rope.half = g->rot_dim / 2;
  }
  const TreePlan pl = tree_plan_splits(a.nkv, cache_len, a.window, n);
  const TreeWs w = tree_ws(d_ws, g, n, pl.ns);
  if (!d_ws || !aligned16(d_ws) || ws_bytes < w.bytes)
    return fail(MTP_ERR_WORKSPACE, "attn_tree_sink: workspace too small");
  a.qp = d_qp;
  a.kp = d_kp;
  a.vp = d_vp;
  a.qn = d_q_norm;
  a.kn = d_k_norm;
  a.sinks = d_sinks;
  a.kc = d_k_cache;
  a.vc = d_v_cache;
  a.mask = reinterpret_cast<const unsigned long long*>(tree->d_mask);
  a.depth = tree->d_depth;
  a.out = d_out;
  a.qf = w.qf;
  a.dep = w.dep;
  a.part_o = w.o;
  a.part_ml = w.ml;
  a.R = n * a.G;
  a.ns = pl.ns;
  a.kbeg = pl.kbeg;
  a.kper = pl.kper;
  a.err = &static_cast<WsHeader*>(d_ws)->err;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int items = n * (a.nh + 2 * a.nkv);
  cudaError_t e = launch_pdl(tree_prep_kernel, dim3((items + kPrepThreads / 32 - 1) / (kPrepThreads / 32)),
                             kPrepThreads, 0, st, a);
  if (e == cudaSuccess && a.ns > 0)
    e = launch_pdl(tree_split_kernel, dim3(a.ns, a.nkv), kSplitWarps * 32, 0, st, a);
  if (e == cudaSuccess)
    e = launch_pdl(tree_finish_kernel, dim3(a.nh, n), kFinishWarps * 32, 0, st, a);
  if (e != cudaSuccess) return cuda_fail(e, "attn_tree_sink launch");
  return MTP_OK;
}

}  // extern "C"
