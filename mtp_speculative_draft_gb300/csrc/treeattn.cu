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
//              workspace, in float32 and as tensor-core operand tiles; k heads
//              normalised and rotated, v heads, appended to cache rows
//              L .. L + n - 1;
//   2. split:  every query row against the cached keys that all rows see,
//              [max(0, L + D + 1 - W), L) for a window W and the tree's
//              largest depth D, split over CTAs, on tcgen05: no mask at all.
//              Partials (m, l, o);
//   3. finish: one CTA a (node, head) joins the partials, the cached keys at
//              the window's edge (fewer than n, each row its own) and the
//              node's ancestors, read key by key, so a row that a mask hides
//              never enters any arithmetic; sink, gate, output.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "prefix.cuh"

namespace mtp {

struct TreeAttnArgs : SplitArgs {
  int nh, nkv, G, n, L, window, gated;
  float eps;
  const float *qp, *kp, *vp, *qn, *kn, *sinks;
  long long ldq, ldk, ldv;
  RopePos rope;
  float *kc, *vc;
  const unsigned long long* mask;
  const int* depth;
  float* out;
  float* qf;       // [nkv][R][dqk] scaled queries, row r = i * G + g
  int* dep;        // [n] depths inside [0, n), then at kTreeMax the largest
  int kper;        // keys a split
};

// First cached key that every row sees (the prep launch has left the depths).
__device__ __forceinline__ int first_common_key(const TreeAttnArgs& a) {
  if (a.window <= 0) return 0;
  const long long k = (long long)a.L + __ldcg(a.dep + kTreeMax) + 1 - a.window;
  return k <= 0 ? 0 : k < a.L ? (int)k : a.L;
}

// Keys [k0, k1) of a split.
__device__ __forceinline__ void split_keys(const TreeAttnArgs& a, int, int sp, int& k0, int& k1) {
  if (a.window > 0) pdl_wait();  // the first key comes from the depths
  k0 = first_common_key(a) + sp * a.kper;
  k1 = min(a.L, k0 + a.kper);
}

// ------------------------------------------------------------------ prep
constexpr int kPrepThreads = 128;

// One warp an item: n * nh query heads, then n * nkv key heads, then values.
// Bound by its dependent reads; a row's values are on their way before the
// depths, which the rotary positions need, are waited for.
__global__ void __launch_bounds__(kPrepThreads) tree_prep_kernel(const __grid_constant__ TreeAttnArgs a) {
  __shared__ int dep[kTreeMax];
  const int lane = threadIdx.x & 31, half = a.rope.half;
  const int it = blockIdx.x * (kPrepThreads / 32) + (threadIdx.x >> 5);
  const int nq = a.n * a.nh, nk = a.n * a.nkv;
  const bool is_q = it < nq, is_k = !is_q && it < nq + nk;
  const int h = is_q ? it % a.nh : (it - nq) % a.nkv;
  const int i = is_q ? it / a.nh : (is_k ? it - nq : it - nq - nk) / a.nkv;
  pdl_wait();
  pdl_launch_dependents();
  HeadVals v, w;
  const float* norm = is_q ? a.qn : a.kn;
  if (is_q || is_k) {
    head_load(v, is_q ? a.qp + (size_t)i * a.ldq + (size_t)h * a.dqk * (a.gated ? 2 : 1)
                      : a.kp + (size_t)i * a.ldk + (size_t)h * a.dqk, a.dqk, half, lane);
    head_load(w, norm, a.dqk, half, lane);
  }
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
  if (blockIdx.x == 0 && threadIdx.x < 32) {
    int d = max(threadIdx.x < a.n ? dep[threadIdx.x] : 0, threadIdx.x + 32 < a.n ? dep[threadIdx.x + 32] : 0);
    d = __reduce_max_sync(0xffffffffu, d);
    if (threadIdx.x == 0) a.dep[kTreeMax] = d;
  }
  RopePos rp = a.rope;
  rp.depth = dep;
  if (is_q) {
    head_norm_rope(v, w, norm != nullptr, a.dqk, a.eps, rp, i, a.err, lane);
    const int kv = h / a.G, r = i * a.G + h % a.G;
    head_store(v, a.qf + ((size_t)kv * a.R + r) * a.dqk, a.dqk, half, a.qscale, lane);
    if (a.ns > 0) store_q_tile(a, v, kv, r, half, lane);
  } else if (is_k) {
    head_norm_rope(v, w, norm != nullptr, a.dqk, a.eps, rp, i, a.err, lane);
    head_store(v, a.kc + ((size_t)h * a.cap + a.L + i) * a.dqk, a.dqk, half, 1.f, lane);
  } else if (it < nq + 2 * nk) {
    const float* src = a.vp + (size_t)i * a.ldv + (size_t)h * a.dv;
    float* dst = a.vc + ((size_t)h * a.cap + a.L + i) * a.dv;
    for (int c = 4 * lane; c < a.dv; c += 128)
      *reinterpret_cast<float4*>(dst + c) = *reinterpret_cast<const float4*>(src + c);
  }
}

// ------------------------------------------------------------------ split
// One CTA: 128 query rows of a KV head against the keys [k0, k1) in tiles of NK.
//
// float32 products on f16 tensor cores: each query row, K tile and V tile is
// scaled by a power of two and split into f16 hi + lo parts (22 bits); q.k and
// p.v are three products each (lo.hi, hi.lo, hi.hi; lo.lo is below 2^-22).  A
// tile's small products are accumulated before the large ones, and P V of a tile
// is added to the running output in float32 registers, so tensor-core
// accumulation chains stay short.  A tile's largest |x| becomes [2^14, 2^15):
// elements keep 22 bits down to 2^-16 of it and an absolute error of 2^-39 of it
// below that.
// Weights are relative to a reference `ref`, set so that the first tile's largest
// weight is 2^8; it moves only when a weight would pass 2^15.5 (f16 ends at
// 2^16), so later tiles need no maximum before their exponentials and no
// rescaling of the output.
//
// Warps: 8 converters (global float32 rows -> f16 hi/lo operand tiles in shared
// memory with the tile's scale), and two warpgroups that each run softmax on
// whole rows (thread = row); a warpgroup's first warp issues P V.
//   COL = false (dv <= 128): the warpgroups take alternate tiles, each with its
//     own (ref, l, o), merged at the end: one's softmax overlaps the other's MMAs.
//     The first warp issues Q K^T too (a converter warp would hold up every tile:
//     230 us, not 191, at 64 nodes and 32768 keys);
//   COL = true: they share every tile, each with half of its keys and half of the
//     output columns, as 256 do not fit a thread's registers.  A K converter warp
//     issues Q K^T (both warpgroups would wait for a softmax warp in the issue
//     queue: 74 us, not 67, at 16 nodes and 32768 keys of 2 x 256).
// Few query rows (64 or less) are repeated `rep` times in the 128 lanes: each
// copy takes its own NK / rep keys of a tile (its P is 0 elsewhere), so all four
// warps of a warpgroup share the exponentials; the copies' states are merged at
// the end like the warpgroups'.
// Shared memory feeds the MMAs at 128 bytes a cycle and is what they wait for, so
// Q and P are operands in tensor memory: P takes the place of S, column by
// column (16 keys: 8 columns of hi parts, 8 of lo parts), and Q hi and lo lie
// behind the outputs (Q lo in shared memory where they do not fit).
//
// Measured: 40/8 heads of 128, 64 nodes, 32768 keys: 170 us, 3.7k cycles a tile of
// 64 keys x 128 rows, of which the tensor pipe works 1.5k (its three products of
// three row tiles are 81 us at 1904 TFLOP/s); the chain scores -> weights -> P V -> output of a
// warpgroup's tile bounds it (issue slots 51 %).  16 nodes: 72 us, 3.7 TB/s of
// cache.  A tile is 64 keys, as two of them, their raw rows and the states fit
// beside 512 tensor-memory columns (32 where a head size passes 128).
constexpr int kSplitThreads = 512;
// Registers a thread at launch, and after the warpgroups share them out anew.
constexpr int kSplitRegs = 128, kSoftmaxRegs = 168, kConvertRegs = 88;
constexpr int kConvWarps = 8;
constexpr int kAhead = 2;  // tiles prefetched to L2 (1 to 4 measure alike; none: +2 % on long caches)
// Tiles whose scales are kept.  Tile t's scale is written once its buffer is free, that is once the scores of
// tile t - kStages are done.  The warpgroup that takes tile t - kStages issues them after its previous tile,
// t - kStages - 2, so the scales up to that one have been read.  (Written before the wait, tile t's scale could
// take the place of t - kStages - 2's while that tile still waits for its V.)
constexpr int kScaleRing = 4;
constexpr float kRefBits = 8.f;   // log2 of the largest weight when the reference is set
constexpr float kRefMost = 15.5f; // log2 of the largest weight before it moves
constexpr int kLaneStride = 132;  // floats of a lane's state: 16-byte accesses without bank conflicts
constexpr int kStages = 2;        // K tile buffers (V: two, or one where COL's do not fit)
constexpr int kRawBytes = 8192;   // a converter warp's rows of a tile: NK / 4 rows of up to 128 or 256 floats

// f16 A and B, f32 accumulator, M = 128; B is MN-major when mn is set (bit 16).
__device__ __forceinline__ uint32_t idesc_f16(int N, bool mn) {
  return (1u << 4) | (mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
}

// Shared-memory operand descriptors as two words: the low one holds the address
// (and the leading offset), the high one is a constant (group offset 1024 bytes,
// 128-byte swizzle), so a step along an operand is one 32-bit addition.
// K-major tiles: rows of 128 bytes.  MN-major tiles: 64 values of MN a block,
// blocks `lead` bytes apart, groups of 8 K rows 1024 bytes apart.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_k(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_mn(uint32_t saddr, uint32_t lead) {
  return ((saddr & 0x3FFFFu) >> 4) | ((lead >> 4) << 16);
}

// One lane of a converged warp, chosen by the hardware: the compiler knows that
// the branch on it is taken by one lane and keeps operands in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(p));
  return p != 0;
}
// D[tmem] (+)= A[smem] * B[smem]^T, by one thread
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %4, 0;\n"
      " mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHi)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %4, 0;\n"
      " mov.b64 b, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHi)
      : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

__device__ __forceinline__ uint32_t half2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// Two values as packed f16 hi and lo parts.
__device__ __forceinline__ void split_f16x2(uint64_t v, uint32_t& hi, uint32_t& lo) {
  const float2 x = unpack2(v);
  const __half2 h = __floats2half2_rn(x.x, x.y);
  const float2 f = __half22float2(h);
  const float2 d = unpack2(fma2(pack2(f.x, f.y), pack2(-1.f, -1.f), v));
  hi = half2_bits(h);
  lo = half2_bits(__floats2half2_rn(d.x, d.y));
}

__device__ __forceinline__ float max16(const float (&v)[16]) {
  float t[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) t[j] = fmaxf(v[j], v[j + 8]);
  return fmaxf(fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])), fmaxf(fmaxf(t[4], t[5]), fmaxf(t[6], t[7])));
}
__device__ __forceinline__ float sum16(const float (&v)[16]) {
  float t[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) t[j] = v[j] + v[j + 8];
  return ((t[0] + t[1]) + (t[2] + t[3])) + ((t[4] + t[5]) + (t[6] + t[7]));
}

struct SplitSmem {
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2], sfull[2], ofull[2];
  uint64_t qready, raw[kConvWarps], top[2];          // a warp's rows have arrived; the K or V warps' largest |x| are there
  uint32_t tmem;
  float kinv[kScaleRing], vinv[kScaleRing];  // a tile's inverse scales
  alignas(16) float wmax[2][2][4];           // largest |x| of each converter warp's rows: K or V, odd or even tile
  float smax[2][128];                        // COL: largest S of each warpgroup's keys
};
// At the end, behind the lane states: m, l and weight of each lane of both
// warpgroups.
struct SplitStates {
  float m[2][128], l[2][128], w[2][128];
};

// First tensor-memory column of the queries (hi parts, then lo parts) behind two
// S tiles and the outputs; whether the lo parts fit too.
__host__ __device__ constexpr int split_q_col(int NK, bool col, int dv) { return 2 * NK + (col ? dv : 2 * dv); }
__host__ __device__ constexpr bool split_q_lo_fits(int NK, bool col, int dqk, int dv) {
  return split_q_col(NK, col, dv) + dqk <= 512;
}

template <int NK, bool COL, class Args>
__global__ void __launch_bounds__(kSplitThreads, 1) tree_split_kernel(const Args a) {
  extern __shared__ __align__(1024) uint8_t smraw[];
  __shared__ SplitSmem sh;
  const uint32_t base = (smem_u32(smraw) + 1023u) & ~1023u;
  uint8_t* sm = smraw + (base - smem_u32(smraw));
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform
  const int sp = blockIdx.x, mt = blockIdx.y, kv = blockIdx.z;
  int k0, k1;
  split_keys(a, kv, sp, k0, k1);
  const int nt = max(0, (k1 - k0 + NK - 1) / NK);  // 0 at a window's end: an empty partial
  const int qb = (a.dqk + 63) / 64, vb = (a.dv + 63) / 64;  // blocks of 64 values
  const uint32_t kpart = (uint32_t)qb * NK * 128, vpart = (uint32_t)vb * NK * 128;
  // one V buffer is for COL alone: warpgroups on alternate tiles would wait for one phase of its barrier on each
  // of their tiles, which passes before the tile's V is there
  const int VS = COL ? a.vstages : 2;
  const uint32_t voff = kStages * 2 * kpart, qoff = voff + (uint32_t)VS * 2 * vpart;
  const bool qlo_tm = split_q_lo_fits(NK, COL, a.dqk, a.dv);
  const uint32_t roff = qoff + (qlo_tm ? 0u : (uint32_t)qb * 128 * 128);  // raw rows

  // tiles on their way to L2 while earlier ones are converted
  auto prefetch = [&](int t) {
    if (t >= nt) return;
    const int row0 = k0 + t * NK, n = min(NK, k1 - row0);
    l2_prefetch(a.keys + ((size_t)kv * a.cap + row0) * a.dqk, (uint32_t)n * a.dqk * 4);
    l2_prefetch(a.values + ((size_t)kv * a.cap + row0) * a.dv, (uint32_t)n * a.dv * 4);
  };
  const bool fetcher = tid == 9 * 32;
  if (fetcher)
    for (int t = 0; t < kAhead; ++t) prefetch(t);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.kfull[i], kConvWarps / 2);
      mbar_init(&sh.kempty[i], 1);
      mbar_init(&sh.vfull[i], kConvWarps / 2);
      mbar_init(&sh.vempty[i], 1);
      mbar_init(&sh.sfull[i], 1);
      mbar_init(&sh.ofull[i], 1);
      mbar_init(&sh.top[i], kConvWarps / 2);
    }
    mbar_init(&sh.qready, 8);
    for (int w = 0; w < kConvWarps; ++w) mbar_init(&sh.raw[w], 1);
    mbar_fence_init();
  }
  if (warp == 0) tc5::alloc(&sh.tmem, 512);
  tc5::fence_before_sync();
  __syncthreads();
  tc5::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem, 0);
  Waiter wait{a.err, false};
  // every MMA has completed and its operands' memory is free
  auto block_sync = [&]() { asm volatile("bar.sync 0, 512;" ::: "memory"); };

  const uint32_t qhi = tmem + split_q_col(NK, COL, a.dv), qlo = qhi + a.dqk / 2;
  // S(t) = Q K(t)^T into S tile `slot`
  auto issue_qk = [&](int t, int slot) {
    const int s = t & 1;
    const uint32_t id = idesc_f16(NK, false), d = tmem + NK * (uint32_t)slot;
    const uint32_t kh = desc_k(base + (uint32_t)s * 2 * kpart), kl = kpart >> 4;
    const int n2 = a.dqk / 32;
    // pairs of 16-dim steps (dims come in 32s): the small products, then the
    // large
    const uint32_t q = desc_k(base + qoff);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      if (b >= n2) break;
      // byte offsets / 16: half of a 128-byte row, or a block of 64 dims
      const uint32_t k = kh + (b >> 1) * (NK * 8) + (b & 1) * 4, ql = q + (b >> 1) * 1024 + (b & 1) * 4;
      if (qlo_tm) {
        mma_f16_ts(d, qlo + 16 * b, k, id, b > 0);
        mma_f16_ts(d, qlo + 16 * b + 8, k + 2, id, 1u);
      } else {
        mma_f16_ss(d, ql, k, id, b > 0);
        mma_f16_ss(d, ql + 2, k + 2, id, 1u);
      }
      mma_f16_ts(d, qhi + 16 * b, k + kl, id, 1u);
      mma_f16_ts(d, qhi + 16 * b + 8, k + kl + 2, id, 1u);
    }
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      if (b >= n2) break;
      const uint32_t k = kh + (b >> 1) * (NK * 8) + (b & 1) * 4;
      mma_f16_ts(d, qhi + 16 * b, k, id, 1u);
      mma_f16_ts(d, qhi + 16 * b + 8, k + 2, id, 1u);
    }
    tc5::commit(&sh.sfull[slot]);
    tc5::commit(&sh.kempty[s]);
  };

  if (warp >= 8) {
    // ---------------- converters: four warps for K, four for V
    const int cw = warp - 8, v = cw >> 2, w4 = cw & 3;
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvertRegs));
    constexpr int RPW = NK / 4;           // rows a warp of a tile
    constexpr int SL = NK == 64 ? 1 : 2;  // 16-byte words a lane of a row
    static_assert(RPW * SL == 16, "sixteen words a lane");
    const int d = v ? a.dv : a.dqk, r0 = w4 * RPW;
    const float* src = v ? a.values + (size_t)kv * a.cap * a.dv : a.keys + (size_t)kv * a.cap * a.dqk;
    const uint32_t part = v ? vpart : kpart, off = v ? voff : 0u;
    uint64_t* full = v ? sh.vfull : sh.kfull;
    uint64_t* empty = v ? sh.vempty : sh.kempty;
    float* inv = v ? sh.vinv : sh.kinv;
    const int ns = v ? VS : kStages;
    uint8_t* raw = sm + roff + (size_t)cw * kRawBytes;
    const uint64_t pol = l2_policy_evict_first();
    auto rows_of = [&](int t) { return min(RPW, k1 - (k0 + t * NK) - r0); };
    // A warp's rows of a tile come by bulk copy into its raw buffer, which is
    // filled anew as soon as the rows are in registers.
    auto fetch = [&](int t) {
      const int n = rows_of(t);
      if (t >= nt || n <= 0 || lane != 0) return;
      mbar_arrive_expect_tx(&sh.raw[cw], (uint32_t)n * d * 4);
      bulk_load(raw, src + (size_t)(k0 + t * NK + r0) * d, (uint32_t)n * d * 4, &sh.raw[cw], pol);
    };
    fetch(0);
#pragma unroll 1
    for (int t = 0; t < nt; ++t) {
      if (fetcher) prefetch(t + kAhead);
      const int n = rows_of(t);
      if (n > 0) wait(&sh.raw[cw], (uint32_t)t & 1u);
      float4 x[16];
      float mx = 0.f;
#pragma unroll
      for (int i = 0; i < RPW; ++i)
#pragma unroll
        for (int s = 0; s < SL; ++s) {
          float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i < n && 4 * (lane + 32 * s) < d)
            q = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(raw) + i * d + 4 * lane + 128 * s);
          x[i * SL + s] = q;
        }
#pragma unroll
      for (int i = 0; i < 16; ++i)
        mx = fmaxf(fmaxf(fmaxf(mx, fabsf(x[i].x)), fabsf(x[i].y)), fmaxf(fabsf(x[i].z), fabsf(x[i].w)));
      mx = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)));
      if (lane == 0) {
        sh.wmax[v][t & 1][w4] = mx;
        tc5::mbar_arrive(&sh.top[v]);
        fence_proxy_async_shared_cta();
      }
      fetch(t + 1);
      // the tile's scale: the largest |x| of the four warps' rows
      __syncwarp();
      wait(&sh.top[v], (uint32_t)t & 1u);
      const float4 m4 = *reinterpret_cast<const float4*>(sh.wmax[v][t & 1]);
      float scale;
      const float iv = f16_scale(fmaxf(fmaxf(m4.x, m4.y), fmaxf(m4.z, m4.w)), scale);
      const int s = ns == 1 ? 0 : t & 1, use = ns == 1 ? t : t >> 1;
      if (use > 0) wait(&empty[s], (uint32_t)(use - 1) & 1u);
      if (w4 == 0 && lane == 0) inv[t % kScaleRing] = iv;
      uint8_t* dst = sm + off + (uint32_t)s * 2 * part;
      const uint64_t s2 = pack2(scale, scale);
#pragma unroll
      for (int i = 0; i < RPW; ++i)
#pragma unroll
        for (int k = 0; k < SL; ++k) {
          const int c = 4 * (lane + 32 * k);
          const float4 q = x[i * SL + k];
          uint2 hi, lo;
          split_f16x2(mul2(pack2(q.x, q.y), s2), hi.x, lo.x);
          split_f16x2(mul2(pack2(q.z, q.w), s2), hi.y, lo.y);
          uint8_t* p = dst + tile_off(r0 + i, c, NK);
          if (c < d) {
            *reinterpret_cast<uint2*>(p) = hi;
            *reinterpret_cast<uint2*>(p + part) = lo;
          }
        }
      tc5::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc5::mbar_arrive(&full[s]);
      if (COL && cw == 0) {
        // the tile's scores, once its S tile is free: P(t - 2) V has completed
        if (t == 0) wait(&sh.qready, 0u);
        if (t >= 2) wait(&sh.ofull[t & 1], (uint32_t)((t - 2) >> 1) & 1u);
        wait(&sh.kfull[s], (uint32_t)use & 1u);
        tc5::fence_after_sync();
        if (elect_one()) issue_qk(t, t & 1);
        __syncwarp();
      }
    }
    block_sync();
  } else {
    // ---------------- softmax and MMA issue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    float o[128];
    float ref = 0.f, l = 0.f;
    SplitStates* states = reinterpret_cast<SplitStates*>(sm + 256 * kLaneStride * 4);
    const int wg = warp >> 2;
    const int row = tid & 127;
    const bool issuer = (warp & 3) == 0 && (!COL || wg == 0);  // the warp that issues P V
    const int lane_rows = 128 / a.rep;       // rows of a copy
    const int qrow = row & (lane_rows - 1);  // this lane's row of the tile
    // this lane's keys of a tile
    const int kw = COL ? 16 : NK / a.rep, kb = COL ? 16 * wg : row / lane_rows * kw;
    // warps of padding rows only keep step
    const bool active = mt * 128 + (qrow & ~31) < a.R;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const int cols = COL ? (wg == 0 ? 128 : a.dv - 128) : a.dv;  // this warpgroup's
    const uint32_t ocol = tmem + 2 * NK + (COL ? 0u : (uint32_t)(wg * a.dv));

    // the queries come from the previous launch (cached rows were final before
    // it released this one): the first warpgroup brings the hi parts, the second
    // the lo parts
    pdl_wait();
    const float qinv = __ldcg(a.qinv + ((size_t)kv * a.mt + mt) * 128 + qrow);
    {
      const uint4* src = reinterpret_cast<const uint4*>(a.qt + ((size_t)kv * a.mt + mt) * 512 * a.dqk) +
                         wg * 16 * a.dqk + row;
      // all reads of 128 dims go out before the first store
#pragma unroll 1
      for (int c0 = 0; c0 < a.dqk; c0 += 128) {
        uint4 u[16];
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (c0 + 8 * k < a.dqk) u[k] = __ldcg(src + (c0 + 8 * k) * 16);
#pragma unroll
        for (int k = 0; k < 16; k += 2) {
          const int c = c0 + 8 * k;
          if (c >= a.dqk) break;
          if (wg == 0 || qlo_tm) {
            const uint32_t r[8] = {u[k].x, u[k].y, u[k].z, u[k].w, u[k + 1].x, u[k + 1].y, u[k + 1].z, u[k + 1].w};
            tmem_st8((wg == 0 ? qhi : qlo) + lanes + c / 2, r);
          } else {
            *reinterpret_cast<uint4*>(sm + qoff + tile_off(row, c, 128)) = u[k];
            *reinterpret_cast<uint4*>(sm + qoff + tile_off(row, c + 8, 128)) = u[k + 1];
          }
        }
      }
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      tc5::fence_proxy_async_smem();
      tc5::fence_before_sync();
    }
    auto pair_sync = [&]() { asm volatile("bar.sync 4, 256;" ::: "memory"); };
    __syncwarp();
    if (lane == 0) tc5::mbar_arrive(&sh.qready);
#pragma unroll
    for (int c = 0; c < 128; ++c) o[c] = 0.f;

    // the tile's P V into this warpgroup's output columns
    auto issue_pv = [&](int t, int slot) {
      const int s = VS == 1 ? 0 : t & 1;
      const uint32_t id = idesc_f16(a.dv, true), p = tmem + NK * (uint32_t)slot;
      const uint32_t v = desc_mn(base + voff + (uint32_t)s * 2 * vpart, NK * 128), vl = vpart >> 4;
#pragma unroll
      for (int k = 0; k < NK / 16; ++k) {
        mma_f16_ts(ocol, p + 16 * k + 8, v + 128 * k, id, k > 0);
        mma_f16_ts(ocol, p + 16 * k, v + vl + 128 * k, id, 1u);
      }
#pragma unroll
      for (int k = 0; k < NK / 16; ++k) mma_f16_ts(ocol, p + 16 * k, v + 128 * k, id, 1u);
      tc5::commit(&sh.ofull[slot]);
      tc5::commit(&sh.vempty[s]);
    };
    auto group_sync = [&]() {
      if (COL)
        pair_sync();
      else
        asm volatile("bar.sync %0, 128;" ::"r"(1 + wg) : "memory");
    };

    const int step = COL ? 1 : 2;
    const int first = COL ? 0 : wg;
    auto scores = [&](int t) {
      if (!issuer || t >= nt) return;
      wait(&sh.kfull[t & 1], (uint32_t)(t >> 1) & 1u);
      tc5::fence_after_sync();
      if (elect_one()) issue_qk(t, t & 1);
      __syncwarp();
    };
    if (issuer && !COL) wait(&sh.qready, 0u);
    if (!COL) scores(first);
#pragma unroll 1
    for (int t = first, it = 0; t < nt; t += step, ++it) {
      const int slot = t & 1;
      const uint32_t ph2 = COL ? (uint32_t)(t >> 1) & 1u : (uint32_t)it & 1u;  // phase of the slot
      const int s = VS == 1 ? 0 : t & 1, use = VS == 1 ? t : t >> 1;  // of V
      wait(&sh.vfull[s], (uint32_t)use & 1u);  // the tile's scales (and V)
      wait(&sh.sfull[slot], ph2);
      tc5::fence_after_sync();
      const int nv = min(NK, k1 - (k0 + t * NK));  // keys before the padding
      const float cs = sh.kinv[t % kScaleRing] * qinv;   // S to logits: a power of two
      const float oscale = sh.vinv[t % kScaleRing];
      const uint32_t st = tmem + lanes + NK * (uint32_t)slot;
      float mx = -INFINITY;
      if (active) {
        // largest S of this lane's keys
#pragma unroll 1
        for (int c = kb; c < kb + kw; c += 16) {
          uint32_t x[16];
          float f[16];
          tc5::ld16(st + c, x);
          tc5::ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) f[j] = __uint_as_float(x[j]);
          if (c + 16 > nv) {  // the tile's last keys are padding
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (c + j >= nv) f[j] = -INFINITY;
          }
          mx = fmaxf(mx, max16(f));
        }
      }
      if (COL) {
        sh.smax[wg][row] = mx;
        pair_sync();
        mx = fmaxf(mx, sh.smax[wg ^ 1][row]);
      }
      if (active) {
        if (it == 0) ref = mx == -INFINITY ? 0.f : mx * cs - kRefBits;  // no key, or NaN logits alone: any
        const float top = mx * cs;
        const bool move = top - ref > kRefMost;
        if (__any_sync(0xffffffffu, move)) {
          const float to = move ? top - kRefBits : ref, corr = ex2(ref - to);
          ref = to;
          l *= corr;
#pragma unroll
          for (int c = 0; c < 128; ++c) o[c] *= corr;
        }
        // P = 2^(logit - ref) as f16 parts in the place of S
        const float nref = -ref;
        float sum = 0.f;
#pragma unroll 1
        for (int c = kb; c < kb + kw; c += 16) {
          uint32_t x[16], hi[8];
          float p[16];
          tc5::ld16(st + c, x);
          tc5::ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) p[j] = ex2(fmaf(__uint_as_float(x[j]), cs, nref));
          if (c + 16 > nv) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (c + j >= nv) p[j] = 0.f;
          }
          sum += sum16(p);
#pragma unroll
          for (int j = 0; j < 8; ++j) split_f16x2(pack2(p[2 * j], p[2 * j + 1]), hi[j], x[j]);
          const uint32_t lo[8] = {x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]};
          tmem_st8(st + c, hi);
          tmem_st8(st + c + 8, lo);
        }
        if (!COL && a.rep > 1) {  // the other copies' keys
          const uint32_t z[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 1
          for (int c = 0; c < NK; c += 8)
            if ((uint32_t)(c - kb) >= (uint32_t)kw) tmem_st8(st + c, z);
        }
        l += sum;
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      }
      tc5::fence_before_sync();
      group_sync();
      if (issuer) {
        tc5::fence_after_sync();
        if (elect_one()) issue_pv(t, slot);
      }
      __syncwarp();
      wait(&sh.ofull[slot], ph2);
      tc5::fence_after_sync();
      if (!COL) scores(t + 2);
      if (active) {
        const uint32_t ot = ocol + lanes + (COL ? 128u * (uint32_t)wg : 0u);
#pragma unroll
        for (int c = 0; c < 128; c += 16) {
          if (c < cols) {
            uint32_t x[16];
            tc5::ld16(ot + c, x);
            tc5::ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) o[c + j] = fmaf(__uint_as_float(x[j]), oscale, o[c + j]);
          }
        }
      }
      tc5::fence_before_sync();
    }
    pdl_launch_dependents();  // by warps that have waited for the launch before: it is through when the next begins
    block_sync();
    // Lane states to shared memory (lane i of a warpgroup at i * kLaneStride),
    // then a row's states weighted and summed.  The code that runs once is kept
    // short: its instructions come from L2 at hundreds of cycles a line.
    float* xo = reinterpret_cast<float*>(sm) + (wg * 128 + row) * kLaneStride;
#pragma unroll
    for (int c = 0; c < 128; c += 4)
      *reinterpret_cast<float4*>(xo + c) = make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]);
    states->m[wg][row] = l == 0.f ? -INFINITY : ref;  // no reference without a key
    states->l[wg][row] = l;
  }
  block_sync();
  const int lane_rows = 128 / a.rep, rows = min(lane_rows, a.R - mt * 128);
  const size_t at0 = ((size_t)kv * a.ns + sp) * a.R + mt * 128;
  SplitStates* states = reinterpret_cast<SplitStates*>(sm + 256 * kLaneStride * 4);
  if (tid < rows) {
    float mr = -INFINITY, lr = 0.f;
#pragma unroll 1
    for (int g = 0; g < 2 * a.rep; ++g) mr = fmaxf(mr, states->m[g & 1][(g >> 1) * lane_rows + tid]);
#pragma unroll 1
    for (int g = 0; g < 2 * a.rep; ++g) {
      const int w = g & 1, i = (g >> 1) * lane_rows + tid;
      // COL: both halves of the columns have one reference
      const float f = COL || states->m[w][i] == -INFINITY ? 1.f : ex2(states->m[w][i] - mr);
      states->w[w][i] = f;
      lr += f * states->l[w][i];
    }
    a.part_ml[at0 + tid] = make_float2(mr, lr);
  }
  block_sync();
  const float* xs = reinterpret_cast<const float*>(sm);
  const int words = a.dv / 4;
#pragma unroll 2
  for (int e = tid; e < rows * words; e += kSplitThreads) {
    const int i = e / words, c = e % words * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int g = 0; g < (COL ? 1 : 2 * a.rep); ++g) {
      const int w = COL ? c >> 7 : g & 1, ln = (g >> 1) * lane_rows + i;
      const float f = states->w[w][ln];
      const float4 x = *reinterpret_cast<const float4*>(xs + (w * 128 + ln) * kLaneStride + (c & 127));
      v.x = fmaf(f, x.x, v.x);
      v.y = fmaf(f, x.y, v.y);
      v.z = fmaf(f, x.z, v.z);
      v.w = fmaf(f, x.w, v.w);
    }
    *reinterpret_cast<float4*>(a.part_o + (at0 + i) * a.dv + c) = v;
  }
  wait.settle();
  if (warp == 0) {
    tc5::fence_after_sync();
    tc5::dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ finish
// One CTA a (node, head), its four warps sharing the splits and the keys read one
// by one; lane l holds dims 4 l .. 4 l + 3 and, past 128 dims, 128 + 4 l ...
// Bound by the latency of a few dependent reads from L2, so keys go four at a
// time (the whole call of 13 nodes of 16 heads of 256: 39 -> 31 us) and 8 CTAs
// share an SM (64 nodes of 40 heads: 2560 CTAs, 19 us).
// H: 128-dim halves of the wider of the two head sizes.
constexpr int kFinishWarps = 4;
constexpr int kFinishKeys = 4;  // keys of a step

template <int H>
struct RowState {
  float m, l;
  float4 o[H];
};

// Cache rows at[0 .. n) (n <= kFinishKeys) against a warp's query row.
template <int H>
__device__ __forceinline__ void keys_step(RowState<H>& s, const float4 (&q)[H], const float* kc,
                                          const float* vc, const int (&at)[kFinishKeys], int n, int dqk,
                                          int dv, int lane) {
  float dot[kFinishKeys];
  float4 v[kFinishKeys][H];
#pragma unroll
  for (int i = 0; i < kFinishKeys; ++i) {
    dot[i] = 0.f;
#pragma unroll
    for (int h = 0; h < H; ++h) {
      v[i][h] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < n) {
        const float4 k = dims4(kc + (size_t)at[i] * dqk, dqk, lane, h);
        v[i][h] = dims4(vc + (size_t)at[i] * dv, dv, lane, h);
        dot[i] += q[h].x * k.x + q[h].y * k.y + q[h].z * k.z + q[h].w * k.w;
      }
    }
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1)
#pragma unroll
    for (int i = 0; i < kFinishKeys; ++i) dot[i] += __shfl_xor_sync(0xffffffffu, dot[i], x);
  float mn = s.m;
#pragma unroll
  for (int i = 0; i < kFinishKeys; ++i)
    if (i < n) mn = fmaxf(mn, dot[i]);
  const float c = mn == -INFINITY ? 1.f : exp2f(s.m - mn);  // 0 at the first keys
  s.m = mn;
  s.l *= c;
#pragma unroll
  for (int h = 0; h < H; ++h) scale4(s.o[h], c);
#pragma unroll
  for (int i = 0; i < kFinishKeys; ++i)
    if (i < n) {
      const float p = dot[i] == -INFINITY ? 0.f : exp2f(dot[i] - mn);  // NaN stays
      s.l += p;
#pragma unroll
      for (int h = 0; h < H; ++h) add4(s.o[h], p, v[i][h]);
    }
}

template <int H>
__global__ void __launch_bounds__(kFinishWarps * 32, H == 1 ? 8 : 6) tree_finish_kernel(const TreeAttnArgs a) {
  __shared__ float sm_m[kFinishWarps], sm_l[kFinishWarps];
  __shared__ float4 sm_o[kFinishWarps][32 * H];
  pdl_wait();
  pdl_launch_dependents();
  const int h = blockIdx.x, i = blockIdx.y, kv = h / a.G, r = i * a.G + h % a.G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // every read that depends on nothing goes out first
  const int dep = a.dep[i];
  unsigned long long m = a.mask[i];
  const int e1 = first_common_key(a);
  const int dep0 = lane < a.n ? a.dep[lane] : 0, dep1 = lane + 32 < a.n ? a.dep[lane + 32] : 0;
  const float sink = a.sinks ? a.sinks[h] * kLog2e : -INFINITY;
  const int c4 = 4 * threadIdx.x;  // this thread's dims of the output
  float4 gate = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.gated && c4 < a.dv)
    gate = *reinterpret_cast<const float4*>(a.qp + (size_t)i * a.ldq + ((size_t)2 * h + 1) * a.dqk + c4);
  const float* qrow = a.qf + ((size_t)kv * a.R + r) * a.dqk;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  float4 q[H];
  RowState<H> s;
  s.m = -INFINITY;
  s.l = 0.f;
#pragma unroll
  for (int x = 0; x < H; ++x) {
    q[x] = dims4(qrow, a.dqk, lane, x);
    s.o[x] = zero;
  }
  // the splits' partials: warp w takes splits w, w + 4, ...; lane l has the
  // weight of the l-th of them
#pragma unroll 1
  for (int s0 = warp; s0 < a.ns; s0 += 32 * kFinishWarps) {
    const int sp = s0 + lane * kFinishWarps;
    const size_t at = ((size_t)kv * a.ns + sp) * a.R + r;
    const float2 ml = sp < a.ns ? a.part_ml[at] : make_float2(-INFINITY, 0.f);
    const float mn = fmaxf(s.m, warp_max(ml.x));
    const float c = s.m == -INFINITY ? 1.f : exp2f(s.m - mn);
    // a partial of NaN logits alone has no maximum, and its sum is NaN
    const float f = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : exp2f(ml.x - mn);
    s.m = mn;
    s.l = s.l * c + warp_sum(f * ml.y);
#pragma unroll
    for (int x = 0; x < H; ++x) scale4(s.o[x], c);
    const int n = min(32, (a.ns - s0 + kFinishWarps - 1) / kFinishWarps);
    const float* po = a.part_o + (((size_t)kv * a.ns + s0) * a.R + r) * a.dv;
    const size_t step = (size_t)kFinishWarps * a.R * a.dv;
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
      const float w = __shfl_sync(0xffffffffu, f, j);
#pragma unroll
      for (int x = 0; x < H; ++x) add4(s.o[x], w, dims4(po + j * step, a.dv, lane, x));
    }
  }
  const float* kc = a.kc + (size_t)kv * a.cap * a.dqk;
  const float* vc = a.vc + (size_t)kv * a.cap * a.dv;
  int at[kFinishKeys];
  // cached keys at the window's edge: seen by this row, not by every row
  if (a.window > 0) {
    const int e0 = max(0, a.L + dep - a.window + 1);
#pragma unroll 1
    for (int k = e0 + warp * kFinishKeys; k < e1; k += kFinishWarps * kFinishKeys) {
#pragma unroll
      for (int j = 0; j < kFinishKeys; ++j) at[j] = k + j;
      keys_step(s, q, kc, vc, at, min(kFinishKeys, e1 - k), a.dqk, a.dv, lane);
    }
  }
  // the node's ancestors inside the window
  if (a.n < 64) m &= (1ull << a.n) - 1;
  if (a.window > 0)
    m &= __ballot_sync(0xffffffffu, dep0 > dep - a.window) |
         (unsigned long long)__ballot_sync(0xffffffffu, dep1 > dep - a.window) << 32;
#pragma unroll 1
  for (int b = 0; m; ++b) {
    int n = 0;
#pragma unroll
    for (int j = 0; j < kFinishKeys; ++j)
      if (m) {
        at[j] = a.L + __ffsll(m) - 1;
        m &= m - 1;
        n = j + 1;
      }
    if (b % kFinishWarps == warp) keys_step(s, q, kc, vc, at, n, a.dqk, a.dv, lane);
  }
  if (lane == 0) {
    sm_m[warp] = s.m;
    sm_l[warp] = s.l;
  }
#pragma unroll
  for (int x = 0; x < H; ++x) sm_o[warp][lane + 32 * x] = s.o[x];
  __syncthreads();
  if (c4 >= a.dv) return;
  float M = sink;
#pragma unroll
  for (int w = 0; w < kFinishWarps; ++w) M = fmaxf(M, sm_m[w]);
  float den = sink == -INFINITY ? 0.f : exp2f(sink - M);
  float4 o = zero;
#pragma unroll
  for (int w = 0; w < kFinishWarps; ++w) {
    const float f = sm_m[w] == -INFINITY ? 1.f : exp2f(sm_m[w] - M);  // none or NaN: 0 or NaN stays
    den += f * sm_l[w];
    add4(o, f, sm_o[w][threadIdx.x]);
  }
  scale4(o, den == 0.f ? 0.f : 1.f / den);  // a row that sees nothing: 0
  if (a.gated) {
    o.x /= 1.f + expf(-gate.x);
    o.y /= 1.f + expf(-gate.y);
    o.z /= 1.f + expf(-gate.z);
    o.w /= 1.f + expf(-gate.w);
  }
  *reinterpret_cast<float4*>(a.out + ((size_t)i * a.nh + h) * a.dv + c4) = o;
}

// ------------------------------------------------------------------ host
struct TreePlan {
  int ns, kper;
};

// Keys of a tile of the split kernel: operand tiles of 64 keys fit beside the
// queries up to 128 dims, 32 above.
static int split_nk(int dqk, int dv) { return dqk <= 128 && dv <= 128 ? 64 : 32; }

// Keys of a split at least: 32, 64 and 128 take 32.6, 32.1 and 36.9 us on 2047 keys
// of two heads of 256 dims; 64 writes half of 32's partials (and leaves SMs without
// a split there: 64 splits for 152).
constexpr int kMinKeys = 64;

// Cached keys that all rows can see: a window's rows have at most window - 1 in
// common (depth 0 alone).
static int common_keys(const mtp_attn_geom* g, int L) { return g->window > 0 ? std::min(L, g->window - 1) : L; }

// Splits of these keys at most: about one CTA per SM.
static int most_splits(const mtp_attn_geom* g, int keys, int n, int sms) {
  const int mt = (n * (g->n_heads / g->n_kv_heads) + 127) / 128;
  return std::min(std::max(1, sms / (g->n_kv_heads * mt)), (keys + kMinKeys - 1) / kMinKeys);
}

static TreePlan tree_plan_splits(const mtp_attn_geom* g, int L, int n) {
  TreePlan p;
  const int keys = common_keys(g, L);
  p.ns = 0;
  p.kper = 0;
  if (keys > 0) {
    const int want = most_splits(g, keys, n, sm_count());
    p.kper = ((keys + want - 1) / want + 15) / 16 * 16;
    p.ns = (keys + p.kper - 1) / p.kper;
  }
  return p;
}

struct TreeWs {
  float* qf;
  uint8_t* qt;
  float* qinv;
  int* dep;
  float2* ml;
  float* o;
  size_t bytes;
};

// `partials`: query rows times splits.
static TreeWs tree_ws(void* ws, const mtp_attn_geom* g, int n, size_t partials) {
  TreeWs w = {};
  size_t off = sizeof(WsHeader) + kRuleJoinBytes;
  uint8_t* b = static_cast<uint8_t*>(ws);
  auto take = [&](size_t bytes) {
    uint8_t* p = b ? b + off : nullptr;
    off = (off + bytes + 255) & ~size_t(255);
    return p;
  };
  const size_t rows = (size_t)n * g->n_heads;
  w.dep = reinterpret_cast<int*>(take(sizeof(int) * (kTreeMax + 1)));
  w.qf = reinterpret_cast<float*>(take(4 * rows * g->head_dim_qk));
  const size_t tiles = (size_t)g->n_kv_heads * ((n * (g->n_heads / g->n_kv_heads) + 127) / 128);
  w.qt = take(tiles * 512 * g->head_dim_qk);
  w.qinv = reinterpret_cast<float*>(take(tiles * 128 * 4));
  w.ml = reinterpret_cast<float2*>(take(8 * partials));
  w.o = reinterpret_cast<float*>(take(4 * partials * g->head_dim_v));
  w.bytes = off;
  return w;
}

// Partials of any call of up to n nodes and L cached keys.  A call's own number falls where its rows fill one
// more tile of 128, and where its keys a split are rounded up; a workspace of the largest call has to do for all.
static size_t most_partials(const mtp_attn_geom* g, int n, int L) {
  const int keys = common_keys(g, L), sms = sm_count();
  size_t most = 0;
  for (int i = 1; i <= n && keys > 0; ++i)
    most = std::max(most, (size_t)i * g->n_heads * most_splits(g, keys, i, sms));
  return most;
}

// Dynamic shared memory of the split kernel: operand tiles, the queries' lo parts where tensor memory has no room
// for them, raw rows, 1024 bytes to align the buffers; and its limit, beside SplitSmem.
constexpr size_t kSplitSmemLimit = 227 * 1024 - 2048;
static constexpr size_t split_smem(int NK, bool col, int dqk, int dv, int vstages) {
  const size_t kstage = (size_t)NK * 256 * ((dqk + 63) / 64), vstage = (size_t)NK * 256 * ((dv + 63) / 64);
  const size_t qlo = split_q_lo_fits(NK, col, dqk, dv) ? 0 : (size_t)((dqk + 63) / 64) * 128 * 128;
  return 1024 + kStages * kstage + vstages * vstage + qlo + kConvWarps * kRawBytes;
}

template <int NK, bool COL, class Args>
static cudaError_t launch_split_as(Args a, int heads, cudaStream_t st) {
  static_assert(kScaleRing >= kStages + 2, "a tile's scale stays until its warpgroup has read it");
  static_assert(sizeof(SplitSmem) <= 2048, "beside the dynamic shared memory");
  // the widest heads of each form (the lo parts are in shared memory at the widest only)
  static_assert(COL || split_smem(NK, false, NK == 64 ? 128 : 256, 128, 2) <= kSplitSmemLimit,
                "warpgroups on alternate tiles need two V buffers");
  constexpr size_t limit = kSplitSmemLimit;
  a.vstages = split_smem(NK, COL, a.dqk, a.dv, 2) <= limit ? 2 : 1;
  const size_t smem = std::max(split_smem(NK, COL, a.dqk, a.dv, a.vstages),
                               1024 + (size_t)256 * kLaneStride * 4 + sizeof(SplitStates));
  if (smem > limit) return cudaErrorInvalidConfiguration;
  static std::atomic<bool> attr[64];  // per device
  static_assert(256 * (kSoftmaxRegs + kConvertRegs) == kSplitThreads * kSplitRegs, "register shares");
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !attr[dev]) {
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, tree_split_kernel<NK, COL, Args>);
    if (e != cudaSuccess) return e;
    if (fa.numRegs != kSplitRegs) return cudaErrorInvalidKernelImage;  // the shares would wait forever
    e = cudaFuncSetAttribute(tree_split_kernel<NK, COL, Args>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)limit);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr[dev] = true;
  }
  return launch_pdl(tree_split_kernel<NK, COL, Args>, dim3(a.ns, a.mt, heads), kSplitThreads, smem, st, a);
}

template <class Args>
static cudaError_t launch_split(const Args& a, int heads, cudaStream_t st) {
  if (split_nk(a.dqk, a.dv) == 64) return launch_split_as<64, false>(a, heads, st);
  return a.dv > 128 ? launch_split_as<32, true>(a, heads, st) : launch_split_as<32, false>(a, heads, st);
}

int split_tile_keys(int dqk, int dv) { return split_nk(dqk, dv); }
cudaError_t launch_prefix_split(const PrefixArgs& a, cudaStream_t st) { return launch_split(a, a.groups * a.nkv, st); }

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
      g->n_kv_heads > 64 || g->n_heads > 4096 || g->n_heads % g->n_kv_heads || g->head_dim_qk < 1 ||
      g->head_dim_qk > 256 || g->head_dim_v < 1 || g->head_dim_v > 256)
    return 0;
  return tree_ws(nullptr, g, n, most_partials(g, n, cache_len)).bytes;
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
  const TreePlan pl = tree_plan_splits(g, cache_len, n);
  const TreeWs w = tree_ws(d_ws, g, n, (size_t)n * g->n_heads * pl.ns);
  if (!d_ws || !aligned16(d_ws) || ws_bytes < w.bytes)
    return fail(MTP_ERR_WORKSPACE, "attn_tree_sink: workspace too small or misaligned");
  a.qp = d_qp;
  a.kp = d_kp;
  a.vp = d_vp;
  a.qn = d_q_norm;
  a.kn = d_k_norm;
  a.sinks = d_sinks;
  a.kc = d_k_cache;
  a.vc = d_v_cache;
  a.keys = d_k_cache;
  a.values = d_v_cache;
  a.mask = reinterpret_cast<const unsigned long long*>(tree->d_mask);
  a.depth = tree->d_depth;
  a.out = d_out;
  a.qf = w.qf;
  a.qt = w.qt;
  a.qinv = w.qinv;
  a.dep = w.dep;
  a.part_o = w.o;
  a.part_ml = w.ml;
  a.R = n * a.G;
  a.rep = a.dv > 128 || a.R > 64 ? 1 : a.R <= 32 && split_nk(a.dqk, a.dv) == 64 ? 4 : 2;
  a.mt = (a.R + 127) / 128;  // 1 where rows are repeated
  a.ns = pl.ns;
  a.kper = pl.kper;
  a.err = &static_cast<WsHeader*>(d_ws)->err;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int items = n * (a.nh + 2 * a.nkv);
  cudaError_t e = launch_pdl(tree_prep_kernel, dim3((items + kPrepThreads / 32 - 1) / (kPrepThreads / 32)),
                             kPrepThreads, 0, st, a);
  if (e == cudaSuccess && a.ns > 0)
    e = launch_split(a, a.nkv, st);
  if (e == cudaSuccess)
    e = launch_pdl(std::max(a.dqk, a.dv) > 128 ? tree_finish_kernel<2> : tree_finish_kernel<1>, dim3(a.nh, n),
                   kFinishWarps * 32, 0, st, a);
  if (e != cudaSuccess) return cuda_fail(e, "attn_tree_sink launch");
  return MTP_OK;
}

}  // extern "C"
