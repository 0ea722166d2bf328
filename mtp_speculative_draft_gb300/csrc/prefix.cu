// Attention of sequences that share prompts: beams, samples of one prompt, or
// the chains of drafts of several requests with one system prompt.
//
// "hf2q 0.1.13 src/inference/models/qwen35/mtp.rs", forward_full_attention
// (per-head norm, rotation, cache append, attention, sigmoid gate) and
// "cortiq-engine 0.8.49 src/mimo_mtp.rs" (window, sinks), for m new rows of each
// of many sequences.  Sequence b has P cached rows of its prompt, which its
// prompt's other sequences read too, and t_b rows of its own (its tail); its new
// row i sits at position P + t_b + i and sees
//   prompt keys j < P and tail keys j <= t_b + i, inside a window W those at
//   positions above P + t_b + i - W.
//
// Three launches:
//   1. prep:  q heads normalised, rotated and scaled (log2 domain) to the
//             workspace, in float32 and as tensor-core operand tiles; k heads
//             normalised and rotated, v heads, appended to the tails;
//   2. split: all query rows of a prompt's KV head against the prompt's keys
//             that every one of them sees, on tcgen05 (tree_split_kernel): the
//             prompt is read once for all its sequences;
//   3. tail:  a cluster of CTAs a (sequence, KV head, new row) reads the
//             sequence's own keys (and a window's edge in the prompt), joins
//             the splits' partials; sink, gate, output.
// Without a long prompt the second launch is left out and the third reads the
// prompt too.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "prefix.cuh"

namespace mtp {

// ------------------------------------------------------------------ prep
constexpr int kPrefixPrepThreads = 128;

// One warp an item: the q heads of all new rows, then k heads, then v heads.
__global__ void __launch_bounds__(kPrefixPrepThreads) prefix_prep_kernel(const __grid_constant__ PrefixArgs a) {
  __shared__ int zero;
  const int lane = threadIdx.x & 31, half = a.rope.half;
  const int it = blockIdx.x * (kPrefixPrepThreads / 32) + (threadIdx.x >> 5);
  const int rows = a.groups * a.per * a.m, nq = rows * a.nh, nk = rows * a.nkv;
  const bool is_q = it < nq, is_k = !is_q && it < nq + nk;
  const int h = is_q ? it % a.nh : (it - nq) % a.nkv;
  const int row = is_q ? it / a.nh : (is_k ? it - nq : it - nq - nk) / a.nkv;
  pdl_wait();
  pdl_launch_dependents();
  HeadVals v, w;
  const float* norm = is_q ? a.qn : a.kn;
  if (is_q || is_k) {
    head_load(v, is_q ? a.qp + (size_t)row * a.ldq + (size_t)h * a.dqk * (a.gated ? 2 : 1)
                      : a.kp + (size_t)row * a.ldk + (size_t)h * a.dqk, a.dqk, half, lane);
    head_load(w, norm, a.dqk, half, lane);
  }
  if (threadIdx.x == 0) zero = 0;
  __syncthreads();
  if (it >= nq + 2 * nk) return;
  const int b = row / a.m, i = row % a.m, p = b / a.per;
  const int P = a.pmax > 0 ? a.plen[p] : 0, t0 = a.tlen[b];
  if (lane == 0 && (P < 0 || P > a.pmax || t0 > a.tmax)) set_dev_error(a.err, kErrBadLength);
  const int t = min(t0, a.tmax);
  RopePos rp = a.rope;
  if (!rp.pos) {  // the row's own position
    rp.base += prompt_len(a, p) + max(t, 0) + i;
    rp.depth = &zero;
  }
  const int at = rp.pos ? row : 0;
  if (is_q) {
    const int kv = h / a.G, r = ((b - p * a.per) * a.m + i) * a.G + h % a.G, head = p * a.nkv + kv;
    if (t < 0) {  // no sequence: rows of zeros, so that the split meets no stale values
      v = HeadVals{};
    } else {
      head_norm_rope(v, w, norm != nullptr, a.dqk, a.eps, rp, at, a.err, lane);
      head_store(v, a.qf + ((size_t)head * a.R + r) * a.dqk, a.dqk, half, a.qscale, lane);
    }
    if (a.ns > 0) store_q_tile(a, v, head, r, half, lane);
  } else if (t < 0) {
    return;
  } else if (is_k) {
    head_norm_rope(v, w, norm != nullptr, a.dqk, a.eps, rp, at, a.err, lane);
    head_store(v, a.kt + (((size_t)b * a.nkv + h) * a.tcap + t + i) * a.dqk, a.dqk, half, 1.f, lane);
  } else {
    const float* src = a.vp + (size_t)row * a.ldv + (size_t)h * a.dv;
    float* dst = a.vt + (((size_t)b * a.nkv + h) * a.tcap + t + i) * a.dv;
    for (int c = 4 * lane; c < a.dv; c += 128)
      *reinterpret_cast<float4*>(dst + c) = *reinterpret_cast<const float4*>(src + c);
  }
}

// ------------------------------------------------------------------ tail
// Warps take steps of 8 keys in turn; a step's K and V rows come by bulk copy
// into the warp's ring of buffers.  Lane (ks, l) has keys ks and ks + 4 of the
// step and dims 32 j + 4 l .. + 3, for q.k as for p.v, so both are read from
// shared memory without bank conflicts and a lane's part of the output covers
// its keys alone; the four key groups' outputs meet once, at the end.  The eight
// lanes' parts of the 2 RG products are summed by halves, so that each lane ends
// with one or two of them and no exponential is taken twice.  All query rows of
// a CTA are heads of one new row: they see the same keys, and no mask is needed.
// RG: query rows (heads) a CTA; C: 32-dim blocks a head at most.
//
// float32 throughout (packed pairs).  Weights are relative to a reference that
// moves only when a logit passes it by 2^8.
constexpr int kTailWarps = 4;
constexpr int kTailKeys = 8;
constexpr float kTailMove = 8.f;
constexpr int kTailStages = 3;  // buffers a warp at most

struct alignas(16) TailSmem {
  uint64_t full[kTailWarps][kTailStages];
  float m[kTailWarps][8], l[kTailWarps][8];  // a warp's state of each row
};

__device__ __forceinline__ void bulk_load_keep(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n barrier.cluster.wait.aligned;" ::: "memory");
}
// Shared memory of CTA `rank` of the cluster at this CTA's address.
__device__ __forceinline__ uint32_t peer(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_peer(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_peer4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

template <int RG, int C>
__global__ void __launch_bounds__(kTailWarps * 32, 2) prefix_tail_kernel(const __grid_constant__ PrefixArgs a, int stages) {
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ TailSmem sh;
  static_assert(RG * C >= 4 && RG * C <= 32, "outputs in registers, at least one block a key group");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ks = lane >> 3, l8 = lane & 7;
  const int rank = (int)cluster_rank(), csize = (int)cluster_size();
  const int b = blockIdx.z, kv = blockIdx.y, item = blockIdx.x / csize;
  const int blocks = (a.G + RG - 1) / RG, i = item / blocks, g0 = item % blocks * RG;
  const int p = b / a.per, head = p * a.nkv + kv, nr = min(RG, a.G - g0);
  const int cq = a.dqk / 32, cv = a.dv / 32;
  const int r0 = ((b - p * a.per) * a.m + i) * a.G + g0;  // first query row
  float* qs = reinterpret_cast<float*>(sm);               // [RG][dqk]
  const uint32_t kbytes = kTailKeys * a.dqk * 4, vbytes = kTailKeys * a.dv * 4;
  uint8_t* ring = sm + RG * a.dqk * 4 + (size_t)warp * stages * (kbytes + vbytes);
  if (lane == 0) {
    for (int s = 0; s < kTailStages; ++s) mbar_init(&sh.full[warp][s], 1);
    mbar_fence_init();
  }
  __syncwarp();
  // lengths and earlier rows were final before the call's first launch
  const int P = prompt_len(a, p), t = tail_len(a, b);
  const int first = first_shared_key(a, p, P);
  const int sees = a.window > 0 ? (int)max(0ll, (long long)P + t + i + 1 - a.window) : 0;  // lowest position
  const int e0 = min(sees, P), e1 = a.ns > 0 ? max(first, e0) : P;    // keys of the prompt
  const int t0 = max(0, sees - P), t1 = t + i + 1;                   // and of the tail
  const int ne = (e1 - e0 + kTailKeys - 1) / kTailKeys, nt = t < 0 ? 0 : ne + (t1 - t0 + kTailKeys - 1) / kTailKeys;
  const int w0 = rank * kTailWarps + warp, stride = csize * kTailWarps;  // this warp's steps: w0, w0 + stride, ..
  Waiter wait{a.err, false};
  auto step_keys = [&](int s, const float*& k, const float*& v) {
    if (s < ne) {
      const int k0 = e0 + s * kTailKeys;
      k = a.keys + ((size_t)head * a.cap + k0) * a.dqk;
      v = a.values + ((size_t)head * a.cap + k0) * a.dv;
      return min(kTailKeys, e1 - k0);
    }
    const int k0 = t0 + (s - ne) * kTailKeys;
    k = a.kt + (((size_t)b * a.nkv + kv) * a.tcap + k0) * a.dqk;
    v = a.vt + (((size_t)b * a.nkv + kv) * a.tcap + k0) * a.dv;
    return min(kTailKeys, t1 - k0);
  };
  auto fetch = [&](int s, int slot) {
    if (s >= nt || lane != 0) return;
    const float *k, *v;
    const int n = step_keys(s, k, v);
    uint8_t* dst = ring + (size_t)slot * (kbytes + vbytes);
    mbar_arrive_expect_tx(&sh.full[warp][slot], (uint32_t)n * (a.dqk + a.dv) * 4);
    bulk_load_keep(dst, k, (uint32_t)n * a.dqk * 4, &sh.full[warp][slot]);
    bulk_load_keep(dst + kbytes, v, (uint32_t)n * a.dv * 4, &sh.full[warp][slot]);
  };
  pdl_wait();
  pdl_launch_dependents();
  fence_proxy_async_global();
  for (int s = 0; s < stages; ++s) fetch(w0 + s * stride, s);
  for (int c = 4 * threadIdx.x; c < RG * a.dqk; c += 4 * kTailWarps * 32) {
    const bool in = c < nr * a.dqk && t >= 0;
    *reinterpret_cast<float4*>(qs + c) =
        in ? *reinterpret_cast<const float4*>(a.qf + ((size_t)head * a.R + r0) * a.dqk + c) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __syncthreads();

  uint64_t o[RG][C][2];
#pragma unroll
  for (int r = 0; r < RG; ++r)
#pragma unroll
    for (int j = 0; j < C; ++j) o[r][j][0] = o[r][j][1] = 0ull;
  constexpr int PL = RG * 2 / 8 > 0 ? RG * 2 / 8 : 1;  // products a lane ends with
  float ref = -INFINITY, l = 0.f;
  int slot = 0;
  uint32_t phase = 0;
#pragma unroll 1
  for (int s = w0; s < nt; s += stride) {
    const float *kg, *vg;
    const int n = step_keys(s, kg, vg);
    float* kb = reinterpret_cast<float*>(ring + (size_t)slot * (kbytes + vbytes));
    float* vb = reinterpret_cast<float*>(ring + (size_t)slot * (kbytes + vbytes) + kbytes);
    wait(&sh.full[warp][slot], phase);
    if (n < kTailKeys) {  // rows behind the last key take part with weight 0
      for (int c = n * a.dv + 4 * lane; c < kTailKeys * a.dv; c += 128)
        *reinterpret_cast<float4*>(vb + c) = make_float4(0.f, 0.f, 0.f, 0.f);
      __syncwarp();
    }
    uint64_t acc[RG][2];
#pragma unroll
    for (int r = 0; r < RG; ++r) acc[r][0] = acc[r][1] = 0ull;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      if (j < cq) {
        const int c = 32 * j + 4 * l8;
        const ulonglong2 k0 = *reinterpret_cast<const ulonglong2*>(kb + ks * a.dqk + c);
        const ulonglong2 k1 = *reinterpret_cast<const ulonglong2*>(kb + (ks + 4) * a.dqk + c);
#pragma unroll
        for (int r = 0; r < RG; ++r) {
          const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(qs + r * a.dqk + c);
          acc[r][0] = fma2(q.x, k0.x, acc[r][0]);
          acc[r][1] = fma2(q.x, k1.x, acc[r][1]);
          acc[r][0] = fma2(q.y, k0.y, acc[r][0]);
          acc[r][1] = fma2(q.y, k1.y, acc[r][1]);
        }
      }
    }
    // product 2 r + k of row r and key ks + 4 k, summed over the eight lanes
    float x[2 * RG];
#pragma unroll
    for (int r = 0; r < RG; ++r)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float2 f = unpack2(acc[r][k]);
        x[2 * r + k] = f.x + f.y;
      }
    {
      int left = 2 * RG;
#pragma unroll
      for (int d = 4; d > 0; d >>= 1) {
        if (left > 1) {
          left /= 2;
          const bool upper = l8 & d;
#pragma unroll
          for (int y = 0; y < RG; ++y)
            if (y < left) {
              const float give = upper ? x[y] : x[y + left], keep = upper ? x[y + left] : x[y];
              x[y] = keep + __shfl_xor_sync(0xffffffffu, give, d);
            }
        } else {
          x[0] += __shfl_xor_sync(0xffffffffu, x[0], d);
        }
      }
    }
    // this lane's row and keys: RG = 8: row l8, both keys; 4: row l8 / 2, key
    // l8 % 2; 2: row l8 / 4, key l8 / 2 % 2 (twice)
    const int mine = ks + 4 * (RG == 8 ? 0 : RG == 4 ? l8 & 1 : l8 >> 1 & 1);
    float mx;
    if (RG == 8) {
      if (mine >= n) x[0] = -INFINITY;
      if (mine + 4 >= n) x[PL - 1] = -INFINITY;
      mx = fmaxf(x[0], x[PL - 1]);
    } else {
      if (mine >= n) x[0] = -INFINITY;
      mx = fmaxf(x[0], __shfl_xor_sync(0xffffffffu, x[0], RG == 4 ? 1 : 2));
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
    const bool move = mx > ref + kTailMove || (ref == -INFINITY && mx > ref);
    if (__any_sync(0xffffffffu, move)) {
      const float to = move ? mx : ref;
      const float corr = ref == -INFINITY ? 1.f : ex2(ref - to);  // nothing was summed without a reference
      ref = to;
      l *= corr;
#pragma unroll
      for (int r = 0; r < RG; ++r) {
        const float f = __shfl_sync(0xffffffffu, corr, r * (8 / RG), 8);
        const uint64_t f2 = pack2(f, f);
#pragma unroll
        for (int j = 0; j < C; ++j) {
          o[r][j][0] = mul2(o[r][j][0], f2);
          o[r][j][1] = mul2(o[r][j][1], f2);
        }
      }
    }
    const float nref = ref == -INFINITY ? 0.f : ref;
    float pr[PL];
#pragma unroll
    for (int k = 0; k < PL; ++k) {
      pr[k] = ex2(x[k] - nref);
      l += pr[k];
    }
    uint64_t w[RG][2];
#pragma unroll
    for (int r = 0; r < RG; ++r)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float f = RG == 8 ? __shfl_sync(0xffffffffu, pr[PL == 2 ? k : 0], r, 8)
                                : __shfl_sync(0xffffffffu, pr[0], RG == 4 ? 2 * r + k : 4 * r + 2 * k, 8);
        w[r][k] = pack2(f, f);
      }
#pragma unroll
    for (int j = 0; j < C; ++j) {
      if (j < cv) {
        const int c = 32 * j + 4 * l8;
        const ulonglong2 v0 = *reinterpret_cast<const ulonglong2*>(vb + ks * a.dv + c);
        const ulonglong2 v1 = *reinterpret_cast<const ulonglong2*>(vb + (ks + 4) * a.dv + c);
#pragma unroll
        for (int r = 0; r < RG; ++r) {
          o[r][j][0] = fma2(w[r][0], v0.x, o[r][j][0]);
          o[r][j][1] = fma2(w[r][0], v0.y, o[r][j][1]);
          o[r][j][0] = fma2(w[r][1], v1.x, o[r][j][0]);
          o[r][j][1] = fma2(w[r][1], v1.y, o[r][j][1]);
        }
      }
    }
    // every lane has read the buffer before it is filled anew
    fence_proxy_async_shared_cta();
    __syncwarp();
    fetch(s + stages * stride, slot);
    if (++slot == stages) {
      slot = 0;
      phase ^= 1u;
    }
  }
  // the warp's state: sums over the key groups, each lane keeping a quarter of
  // its blocks
  l += __shfl_xor_sync(0xffffffffu, l, 8);
  l += __shfl_xor_sync(0xffffffffu, l, 16);
  if (RG == 4) l += __shfl_xor_sync(0xffffffffu, l, 1);
  if (RG == 2) l += __shfl_xor_sync(0xffffffffu, l, 2);
  if (ks == 0 && l8 % (8 / RG) == 0) {
    sh.m[warp][l8 / (8 / RG)] = ref;
    sh.l[warp][l8 / (8 / RG)] = l;
  }
  {
    float y[RG * C * 4];
#pragma unroll
    for (int r = 0; r < RG; ++r)
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const float2 u = unpack2(o[r][j][0]), v = unpack2(o[r][j][1]);
        y[(r * C + j) * 4] = u.x;
        y[(r * C + j) * 4 + 1] = u.y;
        y[(r * C + j) * 4 + 2] = v.x;
        y[(r * C + j) * 4 + 3] = v.y;
      }
    constexpr int N = RG * C * 4;
#pragma unroll
    for (int e = 0; e < N / 2; ++e) {
      const float give = lane & 16 ? y[e] : y[e + N / 2], keep = lane & 16 ? y[e + N / 2] : y[e];
      y[e] = keep + __shfl_xor_sync(0xffffffffu, give, 16);
    }
#pragma unroll
    for (int e = 0; e < N / 4; ++e) {
      const float give = lane & 8 ? y[e] : y[e + N / 4], keep = lane & 8 ? y[e + N / 4] : y[e];
      y[e] = keep + __shfl_xor_sync(0xffffffffu, give, 8);
    }
    float* st = reinterpret_cast<float*>(ring);  // [RG][dv]
    const int from = (lane >> 4) * (RG * C / 2) + (lane >> 3 & 1) * (RG * C / 4);
#pragma unroll
    for (int e = 0; e < RG * C / 4; ++e) {
      const int r = (from + e) / C, j = (from + e) % C;
      if (j < cv)
        *reinterpret_cast<float4*>(st + r * a.dv + 32 * j + 4 * l8) = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
    }
  }
  cluster_sync();

  // Join: a warp a row, over the cluster; lane l has dims 4 l .. and 128 + 4 l ..
  constexpr int H = C / 4;
  const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
  const uint32_t ring_at = smem_u32(sm) + RG * a.dqk * 4, ring_step = stages * (kbytes + vbytes);
  const int states = csize * kTailWarps;
#pragma unroll 1
  for (int r = w0; r < nr && t >= 0; r += stride) {
    const int h = kv * a.G + g0 + r;
    const float sink = a.sinks ? a.sinks[h] * kLog2e : -INFINITY;
    float4 gate[H];
    if (a.gated)
#pragma unroll
      for (int x = 0; x < H; ++x)
        gate[x] = dims4(a.qp + (size_t)(b * a.m + i) * a.ldq + ((size_t)2 * h + 1) * a.dqk, a.dqk, lane, x);
    float sm_ = -INFINITY, sl = 0.f;
    if (lane < states) {
      sm_ = ld_peer(peer(smem_u32(&sh.m[lane % kTailWarps][r]), lane / kTailWarps));
      sl = ld_peer(peer(smem_u32(&sh.l[lane % kTailWarps][r]), lane / kTailWarps));
    }
    float M = fmaxf(sink, warp_max(sm_));
    const size_t at = (size_t)head * a.ns * a.R + r0 + r;
    for (int s = lane; s < a.ns; s += 32) M = fmaxf(M, a.part_ml[at + (size_t)s * a.R].x);
    M = warp_max(M);
    // a state of NaN logits alone has no maximum, and its sum is NaN
    auto weight = [&](float m, float sum) { return m == -INFINITY ? (sum == 0.f ? 0.f : 1.f) : ex2(m - M); };
    float den = 0.f;
    float4 y[H];
#pragma unroll
    for (int x = 0; x < H; ++x) y[x] = none;
    {
      const float f = lane < states ? weight(sm_, sl) : 0.f;
      den += warp_sum(f * sl);
      unsigned there = __ballot_sync(0xffffffffu, lane < states && !(sl == 0.f));
#pragma unroll 1
      while (there) {
        const int s = __ffs(there) - 1;
        there &= there - 1;
        const float w = __shfl_sync(0xffffffffu, f, s);
        const uint32_t src = peer(ring_at + (uint32_t)(s % kTailWarps) * ring_step + (uint32_t)r * a.dv * 4, s / kTailWarps);
#pragma unroll
        for (int x = 0; x < H; ++x)
          if (128 * x + 4 * lane < a.dv) add4(y[x], w, ld_peer4(src + (128 * x + 4 * lane) * 4));
      }
    }
#pragma unroll 1
    for (int s0 = 0; s0 < a.ns; s0 += 32) {
      const float2 ml = s0 + lane < a.ns ? a.part_ml[at + (size_t)(s0 + lane) * a.R] : make_float2(-INFINITY, 0.f);
      const float f = weight(ml.x, ml.y);
      den += warp_sum(f * ml.y);
      const float* po = a.part_o + (at + (size_t)s0 * a.R) * a.dv;
      const int n = min(32, a.ns - s0);
#pragma unroll 4
      for (int s = 0; s < n; ++s) {
        const float w = __shfl_sync(0xffffffffu, f, s);
#pragma unroll
        for (int x = 0; x < H; ++x) add4(y[x], w, dims4(po + (size_t)s * a.R * a.dv, a.dv, lane, x));
      }
    }
    if (sink != -INFINITY) den += ex2(sink - M);
    const float inv = den == 0.f ? 0.f : 1.f / den;
#pragma unroll
    for (int x = 0; x < H; ++x) {
      const int c = 128 * x + 4 * lane;
      scale4(y[x], inv);
      if (a.gated) {
        y[x].x /= 1.f + expf(-gate[x].x);
        y[x].y /= 1.f + expf(-gate[x].y);
        y[x].z /= 1.f + expf(-gate[x].z);
        y[x].w /= 1.f + expf(-gate[x].w);
      }
      if (c < a.dv) *reinterpret_cast<float4*>(a.out + ((size_t)(b * a.m + i) * a.nh + h) * a.dv + c) = y[x];
    }
  }
  cluster_sync();  // the peers have read this CTA's states
  wait.settle();
}

// ------------------------------------------------------------------ host
static size_t tail_smem(int rg, int dqk, int dv, int stages) {
  return (size_t)rg * dqk * 4 + (size_t)kTailWarps * stages * kTailKeys * (dqk + dv) * 4;
}

template <int RG, int C>
static cudaError_t launch_tail_as(const PrefixArgs& a, int csize, cudaStream_t st) {
  const int stages = tail_smem(RG, a.dqk, a.dv, kTailStages) <= 112 * 1024 ? kTailStages : 2;
  const size_t smem = tail_smem(RG, a.dqk, a.dv, stages);
  static std::atomic<bool> attr[64];  // per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !attr[dev]) {
    e = cudaFuncSetAttribute(prefix_tail_kernel<RG, C>, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(csize * a.m * ((a.G + RG - 1) / RG), a.nkv, a.groups * a.per);
  cfg.blockDim = dim3(kTailWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = csize;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = csize > 1 ? 2 : 1;
  launch_mark(st);
  return cudaLaunchKernelEx(&cfg, prefix_tail_kernel<RG, C>, a, stages);
}

static cudaError_t launch_tail(const PrefixArgs& a, int csize, cudaStream_t st) {
  if (a.dqk <= 128 && a.dv <= 128) {
    if (a.G <= 2) return launch_tail_as<2, 4>(a, csize, st);
    return a.G <= 4 ? launch_tail_as<4, 4>(a, csize, st) : launch_tail_as<8, 4>(a, csize, st);
  }
  return a.G <= 2 ? launch_tail_as<2, 8>(a, csize, st) : launch_tail_as<4, 8>(a, csize, st);
}

// Query heads a CTA of the tail launch.
static int tail_rows(int dqk, int dv, int G) {
  return G <= 2 ? 2 : G <= 4 || dqk > 128 || dv > 128 ? 4 : 8;
}

// Splits of a prompt's keys: the fewest waves of CTAs (one a SM) times the keys
// of a split and a CTA's fixed cost, about 192 keys.
constexpr int kSplitCost = 192;
constexpr int kSplitKeys = 64;   // of a split at least
constexpr int kSplitWaves = 3;   // CTAs a SM at most, where a prompt has several splits

static int prefix_splits(int heads_tiles, int keys, int sms) {
  if (keys <= 0) return 0;
  const int most = std::min((keys + kSplitKeys - 1) / kSplitKeys, std::max(1, kSplitWaves * sms / heads_tiles));
  int best = 1;
  long long cost = -1;
  for (int ns = 1; ns <= most; ++ns) {
    const long long waves = ((long long)heads_tiles * ns + sms - 1) / sms;
    const long long c = waves * ((keys + ns - 1) / ns + kSplitCost);
    if (cost < 0 || c < cost) {
      cost = c;
      best = ns;
    }
  }
  return best;
}

// Keys of a prompt that all rows can see: a window's rows have at most
// window - m in common (empty tails).
static int shared_keys(const mtp_attn_geom* g, int m, int pmax) {
  return g->window > 0 ? std::max(0, std::min(pmax, g->window - m)) : pmax;
}

// Prompts of this many keys are read by the tail launch, once a sequence.
constexpr int kTailPrompt = 64;

struct PrefixWs {
  float* qf;
  uint8_t* qt;
  float* qinv;
  float2* ml;
  float* o;
  size_t bytes;
};

// Partials of any call of up to these sizes: splits times query rows, where
// several splits fill at most kSplitWaves CTAs of 128 rows a SM.
static size_t most_partials(const mtp_attn_geom* g, size_t tiles, size_t rows, int pmax, int sms) {
  const size_t keys = shared_keys(g, 1, pmax);
  if (keys == 0) return 0;
  return std::min(rows * ((keys + kSplitKeys - 1) / kSplitKeys), 128 * std::max(tiles, (size_t)kSplitWaves * sms));
}

static PrefixWs prefix_ws(void* ws, const mtp_attn_geom* g, int groups, int seqs, int m, size_t partials) {
  PrefixWs w = {};
  size_t off = sizeof(WsHeader) + kRuleJoinBytes;
  uint8_t* b = static_cast<uint8_t*>(ws);
  auto take = [&](size_t bytes) {
    uint8_t* p = b ? b + off : nullptr;
    off = (off + bytes + 255) & ~size_t(255);
    return p;
  };
  const size_t rows = (size_t)seqs * m * g->n_heads;
  // tiles of 128 rows of each prompt's KV heads: fewer than one more than the rows fill
  const size_t tiles = rows / 128 + (size_t)groups * g->n_kv_heads;
  w.qf = reinterpret_cast<float*>(take(4 * rows * g->head_dim_qk));
  w.qt = take(tiles * 512 * g->head_dim_qk);
  w.qinv = reinterpret_cast<float*>(take(tiles * 128 * 4));
  w.ml = reinterpret_cast<float2*>(take(8 * partials));
  w.o = reinterpret_cast<float*>(take(4 * partials * g->head_dim_v));
  w.bytes = off;
  return w;
}

static size_t prefix_ws_bound(const mtp_attn_geom* g, int groups, int seqs, int m, int pmax) {
  const size_t rows = (size_t)seqs * m * g->n_heads, tiles = rows / 128 + (size_t)groups * g->n_kv_heads;
  return prefix_ws(nullptr, g, groups, seqs, m, most_partials(g, tiles, rows, pmax, sm_count())).bytes;
}

static mtp_status check_prefix_geom(const mtp_attn_geom* g) {
  if (!g) return fail(MTP_ERR_INVALID_ARG, "attn_prefix_sink: null geometry");
  if (g->n_heads < 1 || g->n_kv_heads < 1 || g->n_heads % g->n_kv_heads)
    return fail(MTP_ERR_INVALID_ARG, "attn_prefix_sink: n_kv_heads must divide n_heads");
  if (g->n_kv_heads > 64 || g->n_heads / g->n_kv_heads > 64)
    return fail(MTP_ERR_UNSUPPORTED, "attn_prefix_sink: at most 64 KV heads of 64 query heads each");
  if (g->head_dim_qk < 32 || g->head_dim_qk % 32 || g->head_dim_qk > 256 || g->head_dim_v < 32 ||
      g->head_dim_v % 32 || g->head_dim_v > 256)
    return fail(MTP_ERR_UNSUPPORTED, "attn_prefix_sink: head dims must be multiples of 32, <= 256");
  if (g->rot_dim < 0 || g->rot_dim % 2 || g->rot_dim > g->head_dim_qk)
    return fail(MTP_ERR_INVALID_ARG, "attn_prefix_sink: rot_dim must be even and <= head_dim_qk");
  if (g->gated_q != 0 && g->gated_q != 1)
    return fail(MTP_ERR_INVALID_ARG, "attn_prefix_sink: gated_q must be 0 or 1");
  if (g->gated_q && g->head_dim_v != g->head_dim_qk)
    return fail(MTP_ERR_UNSUPPORTED, "attn_prefix_sink: gated q needs head_dim_v == head_dim_qk");
  if (!(g->eps >= 0.f) || !(g->scale >= 0.f) || !std::isfinite(g->scale))
    return fail(MTP_ERR_INVALID_ARG, "attn_prefix_sink: eps and scale must be >= 0");
  return MTP_OK;
}

static bool good_batch(int groups, int seqs, int m) {
  return groups >= 1 && seqs >= groups && seqs <= kPrefixSeqs && seqs % groups == 0 && m >= 1 && m <= kPrefixRows;
}

}  // namespace mtp

using namespace mtp;

extern "C" {

size_t attn_prefix_sink_workspace_bytes(const mtp_attn_geom* g, int32_t n_groups, int32_t n_seqs, int32_t m,
                                        int32_t prefix_max) {
  if (!g || !good_batch(n_groups, n_seqs, m) || prefix_max < 0 || g->n_heads < 1 || g->n_kv_heads < 1 ||
      g->n_kv_heads > 64 || g->n_heads > 4096 || g->n_heads % g->n_kv_heads || g->head_dim_qk < 1 ||
      g->head_dim_qk > 256 || g->head_dim_v < 1 || g->head_dim_v > 256)
    return 0;
  return prefix_ws_bound(g, n_groups, n_seqs, m, prefix_max);
}

mtp_status attn_prefix_sink(const mtp_attn_geom* g, const mtp_prefix_batch* B, const float* d_qp, const float* d_kp,
                            const float* d_vp, const float* d_q_norm, const float* d_k_norm, const float* d_rope,
                            int32_t rope_rows, const float* d_sinks, const float* d_k_prefix,
                            const float* d_v_prefix, int32_t prefix_cap, float* d_k_tail, float* d_v_tail,
                            int32_t tail_cap, float* d_out, void* d_ws, size_t ws_bytes, void* stream) {
  mtp_status s = check_prefix_geom(g);
  if (s != MTP_OK) return s;
  if (!B || !B->d_tail_len) return fail(MTP_ERR_INVALID_ARG, "attn_prefix_sink: null batch");
  if (!good_batch(B->n_groups, B->n_seqs, B->m))
    return fail(MTP_ERR_UNSUPPORTED,
                "attn_prefix_sink: 1..1024 sequences, as many for each prompt, of 1..16 new rows");
  const int m = B->m, pmax = B->prefix_max, tmax = B->tail_max;
  if (pmax < 0 || tmax < 0 || tail_cap < 1 || prefix_cap < 0)
    return fail(MTP_ERR_INVALID_ARG, "attn_prefix_sink: bad length or capacity");
  if (pmax > prefix_cap) return fail(MTP_ERR_CAPACITY, "attn_prefix_sink: prefix_max exceeds the prompts' capacity");
  if ((int64_t)tmax + m > tail_cap)
    return fail(MTP_ERR_CAPACITY, "attn_prefix_sink: tail_max + m exceeds the tails' capacity");
  if (!d_qp || !d_kp || !d_vp || !d_k_tail || !d_v_tail || !d_out ||
      (pmax > 0 && (!d_k_prefix || !d_v_prefix || !B->d_prefix_len)))
    return fail(MTP_ERR_INVALID_ARG, "attn_prefix_sink: null pointer");
  if (!aligned16(d_qp) || !aligned16(d_kp) || !aligned16(d_vp) || !aligned16(d_k_prefix) || !aligned16(d_v_prefix) ||
      !aligned16(d_k_tail) || !aligned16(d_v_tail) || !aligned16(d_out) || !aligned16(d_q_norm) ||
      !aligned16(d_k_norm) || !aligned16(d_rope) || (reinterpret_cast<uintptr_t>(d_sinks) & 3) ||
      (reinterpret_cast<uintptr_t>(B->d_prefix_len) & 3) || (reinterpret_cast<uintptr_t>(B->d_tail_len) & 3))
    return fail(MTP_ERR_INVALID_ARG, "attn_prefix_sink: misaligned pointer");
  PrefixArgs a = {};
  a.nh = g->n_heads;
  a.nkv = g->n_kv_heads;
  a.G = a.nh / a.nkv;
  a.dqk = g->head_dim_qk;
  a.dv = g->head_dim_v;
  a.m = m;
  a.groups = B->n_groups;
  a.per = B->n_seqs / B->n_groups;
  a.window = g->window > 0 ? g->window : 0;
  a.gated = g->gated_q;
  a.pmax = pmax;
  a.tmax = tmax;
  a.eps = g->eps;
  a.qscale = (float)((g->scale > 0.f ? (double)g->scale : 1.0 / std::sqrt((double)a.dqk)) * 1.4426950408889634);
  const int64_t wq = (int64_t)a.nh * a.dqk * (a.gated ? 2 : 1), wk = (int64_t)a.nkv * a.dqk,
                wv = (int64_t)a.nkv * a.dv;
  a.ldq = B->ld_q ? B->ld_q : wq;
  a.ldk = B->ld_k ? B->ld_k : wk;
  a.ldv = B->ld_v ? B->ld_v : wv;
  if (a.ldq < wq || a.ldk < wk || a.ldv < wv || a.ldq % 4 || a.ldk % 4 || a.ldv % 4)
    return fail(MTP_ERR_INVALID_ARG,
                "attn_prefix_sink: row strides must hold a row and be multiples of 4 floats");
  if (g->rot_dim == 0) {
    a.rope = RopePos{};
  } else if (B->axes) {
    s = fill_rope_axes(&a.rope, B->axes, g->rot_dim / 2, B->n_seqs * m, "attn_prefix_sink");
    if (s != MTP_OK) return s;
  } else {
    if (!d_rope) return fail(MTP_ERR_INVALID_ARG, "attn_prefix_sink: null rotary table");
    if (B->pos_base < 0 || (int64_t)B->pos_base + pmax + tmax + m > rope_rows)
      return fail(MTP_ERR_INVALID_ARG, "attn_prefix_sink: the rotary table is too short");
    a.rope.table = d_rope;
    a.rope.base = B->pos_base;
    a.rope.max_pos = rope_rows;
    a.rope.n_axes = 1;
    a.rope.half = g->rot_dim / 2;
  }
  a.R = a.per * m * a.G;
  const bool wide = split_tile_keys(a.dqk, a.dv) != 64;
  a.rep = a.dv > 128 || a.R > 64 ? 1 : a.R <= 32 && !wide ? 4 : 2;
  a.mt = (a.R + 127) / 128;  // 1 where rows are repeated
  const int sms = sm_count(), heads = a.groups * a.nkv;
  const int keys = shared_keys(g, m, pmax);
  a.ns = pmax <= kTailPrompt ? 0 : prefix_splits(heads * a.mt, keys, sms);
  const PrefixWs w = prefix_ws(d_ws, g, a.groups, B->n_seqs, m, (size_t)heads * a.R * a.ns);
  if (!d_ws || !aligned16(d_ws) || ws_bytes < w.bytes)
    return fail(MTP_ERR_WORKSPACE, "attn_prefix_sink: workspace too small or misaligned");
  a.keys = d_k_prefix;
  a.values = d_v_prefix;
  a.cap = prefix_cap;
  a.kt = d_k_tail;
  a.vt = d_v_tail;
  a.tcap = tail_cap;
  a.plen = B->d_prefix_len;
  a.tlen = B->d_tail_len;
  a.qp = d_qp;
  a.kp = d_kp;
  a.vp = d_vp;
  a.qn = d_q_norm;
  a.kn = d_k_norm;
  a.sinks = d_sinks;
  a.out = d_out;
  a.qf = w.qf;
  a.qt = w.qt;
  a.qinv = w.qinv;
  a.part_o = w.o;
  a.part_ml = w.ml;
  a.err = &static_cast<WsHeader*>(d_ws)->err;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const long long items = (long long)B->n_seqs * m * (a.nh + 2 * a.nkv);
  // CTAs of a sequence's keys: two a SM in all, of 64 keys or more each
  const int edge = a.ns > 0 ? (a.window > 0 ? std::min(pmax, tmax + m) : 0) : pmax;
  const long long own = a.window > 0 ? std::min<long long>((long long)edge + tmax + m, a.window) : (long long)edge + tmax + m;
  const long long ctas = (long long)B->n_seqs * a.nkv * m * ((a.G + tail_rows(a.dqk, a.dv, a.G) - 1) / tail_rows(a.dqk, a.dv, a.G));
  int csize = 1;
  while (csize < 8 && ctas * csize < 2 * sms && own > 64 * csize) csize *= 2;
  cudaError_t e = launch_pdl(prefix_prep_kernel, dim3((unsigned)((items + kPrefixPrepThreads / 32 - 1) / (kPrefixPrepThreads / 32))),
                             kPrefixPrepThreads, 0, st, a);
  if (e == cudaSuccess && a.ns > 0) e = launch_prefix_split(a, st);
  if (e == cudaSuccess) e = launch_tail(a, csize, st);
  if (e != cudaSuccess) return cuda_fail(e, "attn_prefix_sink launch");
  return MTP_OK;
}

}  // extern "C"
