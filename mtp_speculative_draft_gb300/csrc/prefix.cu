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
//   3. tail:  a few CTAs a (sequence, KV head, new row) read the sequence's own
//             keys (and a window's edge in the prompt) and the splits' partials;
//             the last of them joins their parts; sink, gate, output.
// Where there is little of the prompt to share, the third launch reads it too,
// prepares its queries and new keys itself, and is the only one.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "prefix.cuh"

namespace mtp {

// ------------------------------------------------------------------ prep
constexpr int kPrefixPrepThreads = 128;

// One warp an item: the q heads of all new rows, then k heads, then v heads.  Bound by
// its dependent reads (3 us).
__global__ void __launch_bounds__(kPrefixPrepThreads) prefix_prep_kernel(const __grid_constant__ PrefixArgs a) {
  const int lane = threadIdx.x & 31, half = a.rope.half;
  const int it = blockIdx.x * (kPrefixPrepThreads / 32) + (threadIdx.x >> 5);
  const int rows = a.groups * a.per * a.m, nq = rows * a.nh, nk = rows * a.nkv;
  if (it >= nq + 2 * nk) return;
  const bool is_q = it < nq, is_k = !is_q && it < nq + nk;
  const int h = is_q ? it % a.nh : (it - nq) % a.nkv;
  const int row = is_q ? it / a.nh : (is_k ? it - nq : it - nq - nk) / a.nkv;
  const int b = row / a.m, i = row % a.m, p = b / a.per;
  pdl_wait();
  pdl_launch_dependents();
  HeadVals v, w;
  const float* norm = is_q ? a.qn : a.kn;
  if (is_q || is_k) {
    head_load(v, is_q ? a.qp + (size_t)row * a.ldq + (size_t)h * a.dqk * (a.gated ? 2 : 1)
                      : a.kp + (size_t)row * a.ldk + (size_t)h * a.dqk, a.dqk, half, lane);
    head_load(w, norm, a.dqk, half, lane);
  }
  const int P = prompt_len(a, p), t = tail_len(a, b);
  const size_t to = ((size_t)b * a.nkv + h) * a.tcap + t + i;  // in the tails
  if (is_q) {
    const int r = ((b - p * a.per) * a.m + i) * a.G + h % a.G, head = p * a.nkv + h / a.G;
    if (t < 0) {  // no sequence: rows of zeros, so that the split meets no stale values
      v = HeadVals{};
    } else {
      head_norm_rope(v, w, norm != nullptr, a.dqk, a.eps, a.rope, row, a.err, lane, P + t + i);
      head_store(v, a.qf + ((size_t)head * a.R + r) * a.dqk, a.dqk, half, a.qscale, lane);
    }
    store_q_tile(a, v, head, r, half, lane);
  } else if (t < 0) {
    return;
  } else if (is_k) {
    head_norm_rope(v, w, norm != nullptr, a.dqk, a.eps, a.rope, row, a.err, lane, P + t + i);
    head_store(v, a.kt + to * a.dqk, a.dqk, half, 1.f, lane);
  } else {
    const float* src = a.vp + (size_t)row * a.ldv + (size_t)h * a.dv;
    for (int c = 4 * lane; c < a.dv; c += 128)
      *reinterpret_cast<float4*>(a.vt + to * a.dv + c) = *reinterpret_cast<const float4*>(src + c);
  }
}

// ------------------------------------------------------------------ tail
// Warps take steps of 8 keys in turn; a step's K and V rows come by bulk copy
// into the warp's buffers, the next step's while this one's are worked on.  For q.k lane (ks, l) has keys ks and ks + 4 of the
// step and dims 32 j + 4 l .. + 3; the eight lanes' parts of the 2 RG products are
// summed by halves, so that each lane ends with one or two of them and no
// exponential is taken twice.  The weights go through shared memory; for p.v a
// lane has dims 4 l .. and 128 + 4 l .. of every key, so the output takes few
// registers, many warps share an SM and hide each other's waits.  All query rows
// of a CTA are heads of one new row, which see the same keys; MANY: of several new
// rows, whose masks differ in a few steps at the ends of what they see, and a
// sequence's keys are read once for them (8/8 heads of 128, 8 sequences of 8 new rows,
// tails of 512: 32 us, one row a CTA 46).
// RG: query rows (heads) a CTA; H: 128-dim halves of the wider head size; ALONE:
// without a split launch.
//
// float32 throughout (packed pairs).  Weights are relative to a reference that
// moves only when a logit passes it by 2^8.
//
// A step of 8 keys is 400 warp instructions for 5 rows of 128 dims, about 1000 to 2500
// cycles of one warp's waits, so 16 warps share an SM: 24 sequences of up to 2048 rows,
// 40/8 heads of 128, take 44 us (219 MB at 5 TB/s; shared memory's pipe 49 % busy, issue
// slots 34 %), 64 of up to 256 take 22 (two waves; 79 MB).  Outputs by key groups
// (half as many warps) took 76 and 35 us, clusters over long tails 53 and 28.  One
// buffer of keys and one of values a warp do as well as two of each.  At 128 (168)
// registers for four (three) CTAs an SM, 19 of the 28 forms spill 4 to 28 bytes a thread.
constexpr int kTailWarps = 4;
constexpr int kTailKeys = 8;
constexpr float kTailMove = 8.f;

struct alignas(16) TailSmem {
  float2 p[kTailWarps][kTailKeys][8];        // a step's weights, each twice
  uint64_t kfull[kTailWarps], vfull[kTailWarps];  // a warp's keys, values have arrived
  float m[kTailWarps][8], l[kTailWarps][8];  // a warp's state of each row
  int last;                                  // this part is the last to arrive
};

__device__ __forceinline__ void bulk_load_keep(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
// Lane's part of the products: PR rows (a power of two, RG or more), rows RG .. are 0.
__host__ __device__ constexpr int tail_padded(int rg) { return rg <= 2 ? 2 : rg <= 4 ? 4 : 8; }

// CTAs a SM that the registers allow.
__host__ __device__ constexpr int tail_ctas(int rg, int h) { return h == 1 || rg <= 4 ? 4 : 3; }

template <int RG, int H, bool ALONE, bool MANY>
__global__ void __launch_bounds__(kTailWarps * 32, tail_ctas(RG, H))
    prefix_tail_kernel(const __grid_constant__ PrefixArgs a) {
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ TailSmem sh;
  constexpr int PR = tail_padded(RG);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ks = lane >> 3, l8 = lane & 7;
  const int b = blockIdx.z, kv = blockIdx.y, part = blockIdx.x / a.items, item = blockIdx.x % a.items;
  const int blocks = (a.G + RG - 1) / RG, g0 = item % blocks * RG;
  const int i = item / blocks * (MANY ? a.mrows : 1), last = MANY ? min(i + a.mrows, a.m) - 1 : i;  // new rows i .. last
  const int p = b / a.per, head = p * a.nkv + kv, nr = MANY ? (last + 1 - i) * a.G : min(RG, a.G - g0);
  // query row r of the CTA: head g0 + head_of(r) of the KV head's, new row i + row_of(r)
  auto row_of = [&](int r) { return MANY ? r / a.G : 0; };
  auto head_of = [&](int r) { return MANY ? r % a.G : r; };
  const int cq = a.dqk / 32;
  const int r0 = ((b - p * a.per) * a.m + i) * a.G + g0;  // first query row
  float* qs = reinterpret_cast<float*>(sm);               // [RG][dqk]
  const uint32_t kbytes = kTailKeys * a.dqk * 4, wbytes = kbytes + kTailKeys * a.dv * 4;
  float* const kb = reinterpret_cast<float*>(sm + RG * a.dqk * 4 + warp * wbytes);  // [8][dqk]
  float* const vb = kb + kTailKeys * a.dqk;                                          // [8][dv]
  if (lane == 0) {
    mbar_init(&sh.kfull[warp], 1);
    mbar_init(&sh.vfull[warp], 1);
    mbar_fence_init();
  }
  __syncwarp();
  // Behind a split launch, that launch has released this one after its own wait for
  // the prep launch, so all that both wait for is through, queries and appended rows
  // among it; the splits' partials are waited for below, behind the own keys.
  if (ALONE) pdl_wait();
  const int P = prompt_len(a, p), t = tail_len(a, b);
  if (blockIdx.x == 0 && kv == 0 && threadIdx.x == 0) {
    const int P0 = a.pmax > 0 ? a.plen[p] : 0;
    if (P0 < 0 || P0 > a.pmax || a.tlen[b] > a.tmax) set_dev_error(a.err, kErrBadLength);
  }
  if (t < 0) {  // no sequence
    if (!ALONE) pdl_wait();  // a launch ends behind the ones before it
    return;
  }
  const int first = ALONE ? P : first_shared_key(a, p, P);
  // Keys: without a split launch the new rows j0 .. last, which are prepared below; the
  // prompt's e0 .. e1; the tail's t0 .. t2; in steps of their own.
  const int sees = a.window > 0 ? (int)max(0ll, (long long)P + t + i + 1 - a.window) : 0;  // lowest position
  const int e0 = min(sees, P), e1 = ALONE ? P : max(first, e0);
  const int t2 = ALONE ? t : t + last + 1, t0 = min(max(0, sees - P), t2), j0 = max(0, sees - P - t);
  auto steps_of = [](int n) { return (n + kTailKeys - 1) / kTailKeys; };
  const int nn = ALONE ? steps_of(last + 1 - j0) : 0, ne = nn + steps_of(e1 - e0), nt = ne + steps_of(t2 - t0);
  // the sequence's parts: as many as its keys need, each with every parts-th of
  // the steps and of the splits' partials
  const int parts = max(1, min(a.parts, (nt * kTailKeys + a.part_keys - 1) / a.part_keys));
  if (part >= parts) return;
  const int w0 = part * kTailWarps + warp, stride = parts * kTailWarps;  // this warp's steps: w0, w0 + stride, ..
  const float* const kpre = a.keys + ((size_t)head * a.cap + e0) * a.dqk;
  const float* const vpre = a.values + ((size_t)head * a.cap + e0) * a.dv;
  const size_t own_row = ((size_t)b * a.nkv + kv) * a.tcap;
  const float* const kown = a.kt + (own_row + t0) * a.dqk;
  const float* const vown = a.vt + (own_row + t0) * a.dv;
  Waiter wait{a.err, false};
  auto step_size = [&](int s) {
    return min(kTailKeys, s < nn ? last + 1 - j0 - s * kTailKeys : s < ne ? e1 - e0 - (s - nn) * kTailKeys : t2 - t0 - (s - ne) * kTailKeys);
  };
  auto fetch_k = [&](int s) {
    if (lane != 0) return;
    const uint32_t bytes = (uint32_t)step_size(s) * a.dqk * 4;
    mbar_arrive_expect_tx(&sh.kfull[warp], bytes);
    bulk_load_keep(kb, (s < ne ? kpre : kown) + (size_t)(s < ne ? s - nn : s - ne) * kTailKeys * a.dqk, bytes, &sh.kfull[warp]);
  };
  auto fetch_v = [&](int s) {
    if (lane != 0) return;
    const uint32_t bytes = (uint32_t)step_size(s) * a.dv * 4;
    mbar_arrive_expect_tx(&sh.vfull[warp], bytes);
    bulk_load_keep(vb, (s < ne ? vpre : vown) + (size_t)(s < ne ? s - nn : s - ne) * kTailKeys * a.dv, bytes, &sh.vfull[warp]);
  };
  fence_proxy_async_global();
  if (w0 >= nn && w0 < nt) {
    fetch_k(w0);
    fetch_v(w0);
  }
  const int half = a.rope.half;
  if (!ALONE) {
    const float* src = a.qf + ((size_t)head * a.R + r0) * a.dqk;
    for (int c = 4 * threadIdx.x; c < RG * a.dqk; c += 4 * kTailWarps * 32)
      *reinterpret_cast<float4*>(qs + c) = c < nr * a.dqk ? __ldcg(reinterpret_cast<const float4*>(src + c)) : make_float4(0.f, 0.f, 0.f, 0.f);
  } else {
    // The query rows, normalised, rotated and scaled (log2 domain): up to two a warp,
    // whose reads go out together.  Warp 0, which has the new key, comes last.
    HeadVals hv[2], hw;
    const int rq = (warp + kTailWarps - 1) % kTailWarps;
#pragma unroll
    for (int x = 0; x < (RG + kTailWarps - 1) / kTailWarps; ++x) {
      const int r = rq + x * kTailWarps;
      hv[x] = HeadVals{};
      if (r < nr)
        head_load(hv[x], a.qp + (size_t)(b * a.m + i + row_of(r)) * a.ldq + (size_t)(kv * a.G + g0 + head_of(r)) * a.dqk * (a.gated ? 2 : 1), a.dqk, half, lane);
    }
    head_load(hw, a.qn, a.dqk, half, lane);
#pragma unroll
    for (int x = 0; x < (RG + kTailWarps - 1) / kTailWarps; ++x) {
      const int r = rq + x * kTailWarps;
      if (r < nr) head_norm_rope(hv[x], hw, a.qn != nullptr, a.dqk, a.eps, a.rope, b * a.m + i + row_of(r), a.err, lane, P + t + i + row_of(r));
      if (r < RG) head_store(hv[x], qs + r * a.dqk, a.dqk, half, a.qscale, lane);
    }
    // A step of new rows, which is a warp's first, is written into its buffers; the
    // CTA that has a row's first heads appends it to the tail.
    if (w0 < nn) {
#pragma unroll 1
      for (int j = j0 + w0 * kTailKeys, y = 0; j <= last && y < kTailKeys; ++j, ++y) {
        const size_t row = (size_t)b * a.m + j;
        head_load(hv[0], a.kp + row * a.ldk + (size_t)kv * a.dqk, a.dqk, half, lane);
        head_load(hw, a.kn, a.dqk, half, lane);
        head_norm_rope(hv[0], hw, a.kn != nullptr, a.dqk, a.eps, a.rope, (int)row, a.err, lane, P + t + j);
        head_store(hv[0], kb + y * a.dqk, a.dqk, half, 1.f, lane);
        const bool append = j >= i && g0 == 0;
        if (append) head_store(hv[0], a.kt + (own_row + t + j) * a.dqk, a.dqk, half, 1.f, lane);
        const float* src = a.vp + row * a.ldv + (size_t)kv * a.dv;
        for (int c = 4 * lane; c < a.dv; c += 128) {
          const float4 x = *reinterpret_cast<const float4*>(src + c);
          *reinterpret_cast<float4*>(vb + y * a.dv + c) = x;
          if (append) *reinterpret_cast<float4*>(a.vt + (own_row + t + j) * a.dv + c) = x;
        }
      }
      fence_proxy_async_shared_cta();  // before a later copy into the buffers
      __syncwarp();
      if (lane == 0) {
        tc5::mbar_arrive(&sh.kfull[warp]);
        tc5::mbar_arrive(&sh.vfull[warp]);
      }
    }
  }
  if (ALONE) pdl_launch_dependents();
  __syncthreads();

  uint64_t o[RG][H][2];
#pragma unroll
  for (int r = 0; r < RG; ++r)
#pragma unroll
    for (int h = 0; h < H; ++h) o[r][h][0] = o[r][h][1] = 0ull;
  constexpr int PL = PR == 8 ? 2 : 1;  // products a lane ends with
  // this lane's row and keys: PR = 8: row l8, keys ks and ks + 4; 4: row l8 / 2,
  // key ks + 4 (l8 % 2); 2: row l8 / 4, key ks + 4 (l8 / 2 % 2), twice
  const int mine = ks + 4 * (PR == 8 ? 0 : PR == 4 ? l8 & 1 : l8 >> 1 & 1), row = l8 / (8 / PR);
  int vcol[H];  // this lane's dims of a value (past the last one: any, and not stored)
#pragma unroll
  for (int h = 0; h < H; ++h) vcol[h] = min(128 * h + 4 * lane, a.dv - 4);
  const int own_pos = P + t + min(i + row_of(row), last);  // position of this lane's row
  float ref = -INFINITY, l = 0.f;
  uint32_t phase = 0;
#pragma unroll 1
  for (int s = w0; s < nt; s += stride) {
    const int n = step_size(s);
    const int pos = s < nn ? P + t + j0 + s * kTailKeys : s < ne ? e0 + (s - nn) * kTailKeys : P + t0 + (s - ne) * kTailKeys;
    auto hidden = [&](int key) { return MANY && (unsigned)(own_pos - pos - key) >= (a.window > 0 ? (unsigned)a.window : 0x80000000u); };
    const bool edge = MANY && __any_sync(0xffffffffu, hidden(0) || hidden(n - 1));  // some row does not see some key
    wait(&sh.kfull[warp], phase);
    uint64_t acc[RG][2];
#pragma unroll
    for (int r = 0; r < RG; ++r) acc[r][0] = acc[r][1] = 0ull;
    // blocks of 128, 64 and 32 dims, each without a branch, so that its reads go out together
    auto dots = [&](int c, auto blocks) {
      constexpr int N = decltype(blocks)::value;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const ulonglong2 k0 = *reinterpret_cast<const ulonglong2*>(kb + ks * a.dqk + c + 32 * j);
        const ulonglong2 k1 = *reinterpret_cast<const ulonglong2*>(kb + (ks + 4) * a.dqk + c + 32 * j);
#pragma unroll
        for (int r = 0; r < RG; ++r) {
          const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(qs + r * a.dqk + c + 32 * j);
          acc[r][0] = fma2(q.x, k0.x, acc[r][0]);
          acc[r][1] = fma2(q.x, k1.x, acc[r][1]);
          acc[r][0] = fma2(q.y, k0.y, acc[r][0]);
          acc[r][1] = fma2(q.y, k1.y, acc[r][1]);
        }
      }
    };
    int c = 4 * l8;
    if (cq >= 4) dots(c, std::integral_constant<int, 4>{}), c += 128;
    if (H == 2 && cq >= 8) dots(c, std::integral_constant<int, 4>{}), c += 128;
    if (cq & 2) dots(c, std::integral_constant<int, 2>{}), c += 64;
    if (cq & 1) dots(c, std::integral_constant<int, 1>{});
    __syncwarp();  // every lane has read the keys before their buffer is filled anew
    if (s + stride < nt) fetch_k(s + stride);
    // product 2 r + k of row r and key ks + 4 k, summed over the eight lanes
    float x[2 * PR];
#pragma unroll
    for (int r = 0; r < PR; ++r)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        x[2 * r + k] = 0.f;
        if (r < RG) {
          const float2 f = unpack2(acc[r][k]);
          x[2 * r + k] = f.x + f.y;
        }
      }
    {
      int left = 2 * PR;
#pragma unroll
      for (int d = 4; d > 0; d >>= 1) {
        if (left > 1) {
          left /= 2;
          const bool upper = l8 & d;
#pragma unroll
          for (int y = 0; y < PR; ++y)
            if (y < left) {
              const float give = upper ? x[y] : x[y + left], keep = upper ? x[y + left] : x[y];
              x[y] = keep + __shfl_xor_sync(0xffffffffu, give, d);
            }
        } else {
          x[0] += __shfl_xor_sync(0xffffffffu, x[0], d);
        }
      }
    }
    float mx;
    if (mine >= n || hidden(mine)) x[0] = -INFINITY;
    if (PR == 8) {
      if (mine + 4 >= n || hidden(mine + 4)) x[PL - 1] = -INFINITY;
      mx = fmaxf(x[0], x[PL - 1]);
    } else {
      mx = fmaxf(x[0], __shfl_xor_sync(0xffffffffu, x[0], PR == 4 ? 1 : 2));
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
        const float f = __shfl_sync(0xffffffffu, corr, r * (8 / PR), 8);
        const uint64_t f2 = pack2(f, f);
#pragma unroll
        for (int h = 0; h < H; ++h) {
          o[r][h][0] = mul2(o[r][h][0], f2);
          o[r][h][1] = mul2(o[r][h][1], f2);
        }
      }
    }
    const float nref = ref == -INFINITY ? 0.f : ref;
#pragma unroll
    for (int k = 0; k < PL; ++k) {
      const float w = ex2(x[k] - nref);
      l += w;
      sh.p[warp][mine + 4 * k][row] = edge && hidden(mine + 4 * k) ? make_float2(-1.f, -1.f) : make_float2(w, w);
    }
    wait(&sh.vfull[warp], phase);
    phase ^= 1u;
    if (n < kTailKeys) {  // rows behind the last key take part with weight 0
      for (int c = n * a.dv + 4 * lane; c < kTailKeys * a.dv; c += 128)
        *reinterpret_cast<float4*>(vb + c) = make_float4(0.f, 0.f, 0.f, 0.f);
      fence_proxy_async_shared_cta();  // before a later copy into the buffer
    }
    __syncwarp();
    if (edge) {  // a weight of -1: the row does not see the key, whose value may be anything
#pragma unroll 1
      for (int k = 0; k < n; ++k) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(vb + k * a.dv + vcol[h]);
#pragma unroll
          for (int r = 0; r < RG; ++r) {
            const float f = sh.p[warp][k][r].x;
            if (f != -1.f) {
              const uint64_t f2 = pack2(f, f);
              o[r][h][0] = fma2(f2, v.x, o[r][h][0]);
              o[r][h][1] = fma2(f2, v.y, o[r][h][1]);
            }
          }
        }
      }
    } else {
#pragma unroll
    for (int k = 0; k < kTailKeys; ++k) {
      uint64_t w[8];
#pragma unroll
      for (int r = 0; r < RG; r += 2) {
        const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(&sh.p[warp][k][r]);
        w[r] = u.x;
        w[r + 1] = u.y;
      }
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(vb + k * a.dv + vcol[h]);
#pragma unroll
        for (int r = 0; r < RG; ++r) {
          o[r][h][0] = fma2(w[r], v.x, o[r][h][0]);
          o[r][h][1] = fma2(w[r], v.y, o[r][h][1]);
        }
      }
    }
    }
    __syncwarp();  // every lane has read the values
    if (s + stride < nt) fetch_v(s + stride);
  }
  // the warp's share of the splits' partials, in the layout of its own output
  if (!ALONE) {
    pdl_wait();
    pdl_launch_dependents();
    const size_t at = (size_t)head * a.ns * a.R + r0;
    const float2* ml_at = a.part_ml + at + min(row, nr - 1);
    constexpr int NB = RG * H <= 5 ? 3 : RG * H <= 8 ? 2 : 1;  // splits at once: their reads wait together
#pragma unroll 1
    for (int s0 = w0; s0 < a.ns; s0 += NB * stride) {
      ulonglong2 v[NB][RG][H];
      float2 ml[NB];
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const int s = s0 + k * stride;
        ml[k] = make_float2(-INFINITY, 0.f);
        if (s < a.ns) ml[k] = ml_at[(size_t)s * a.R];
        const float* po = a.part_o + (at + (size_t)s * a.R) * a.dv;
#pragma unroll
        for (int r = 0; r < RG; ++r)
#pragma unroll
          for (int h = 0; h < H; ++h) {
            v[k][r][h] = make_ulonglong2(0ull, 0ull);
            if (s < a.ns) v[k][r][h] = *reinterpret_cast<const ulonglong2*>(po + (size_t)min(r, nr - 1) * a.dv + vcol[h]);
          }
      }
      float to = ref;
#pragma unroll
      for (int k = 0; k < NB; ++k) to = fmaxf(to, ml[k].x);
      const float corr = ref == -INFINITY ? 1.f : ex2(ref - to);  // nothing, or NaN, was summed without a reference
      ref = to;
      l *= corr;
      float f[NB];
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        // a partial of NaN logits alone has no maximum, and its sum is NaN
        f[k] = ml[k].x == -INFINITY ? (ml[k].y == 0.f ? 0.f : 1.f) : ex2(ml[k].x - ref);
        if (mine == 0) l += f[k] * ml[k].y;
      }
#pragma unroll
      for (int r = 0; r < RG; ++r) {
        const float c1 = __shfl_sync(0xffffffffu, corr, r * (8 / PR), 8);
        const uint64_t c2 = pack2(c1, c1);
#pragma unroll
        for (int h = 0; h < H; ++h) {
          o[r][h][0] = mul2(o[r][h][0], c2);
          o[r][h][1] = mul2(o[r][h][1], c2);
        }
#pragma unroll
        for (int k = 0; k < NB; ++k) {
          const float w = __shfl_sync(0xffffffffu, f[k], r * (8 / PR), 8);
          const uint64_t w2 = pack2(w, w);
#pragma unroll
          for (int h = 0; h < H; ++h) {
            o[r][h][0] = fma2(w2, v[k][r][h].x, o[r][h][0]);
            o[r][h][1] = fma2(w2, v[k][r][h].y, o[r][h][1]);
          }
        }
      }
    }
  }
  // the warp's state
  l += __shfl_xor_sync(0xffffffffu, l, 8);
  l += __shfl_xor_sync(0xffffffffu, l, 16);
  if (PR == 4) l += __shfl_xor_sync(0xffffffffu, l, 1);
  if (PR == 2) l += __shfl_xor_sync(0xffffffffu, l, 2);
  if (ks == 0 && l8 % (8 / PR) == 0) {
    sh.m[warp][row] = ref;
    sh.l[warp][row] = l;
  }
  float* const states = reinterpret_cast<float*>(sm + RG * a.dqk * 4);  // a warp's at the start of its buffers
  const int wstep = wbytes / 4;
#pragma unroll
  for (int r = 0; r < RG; ++r)
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int c = 128 * h + 4 * lane;
      if (c < a.dv) *reinterpret_cast<ulonglong2*>(states + warp * wstep + r * a.dv + c) = make_ulonglong2(o[r][h][0], o[r][h][1]);
    }
  __syncthreads();

  // Join: a warp a row; lane l has dims 4 l .. and 128 + 4 l ..  A state of NaN
  // logits alone has no maximum, and its sum is NaN.
  auto weight = [](float m, float sum, float top) { return m == -INFINITY ? (sum == 0.f ? 0.f : 1.f) : ex2(m - top); };
  float4 y[H];
  auto finish = [&](int r, float M, float den) {
    const int h = kv * a.G + g0 + head_of(r);
    if (a.sinks) {
      const float sink = a.sinks[h] * kLog2e, to = fmaxf(M, sink);
      if (to != M) {  // M may be -infinity: then nothing was summed
        const float f = weight(M, den, to);
        den *= f;
#pragma unroll
        for (int x = 0; x < H; ++x) scale4(y[x], f);
      }
      if (sink != -INFINITY) den += ex2(sink - to);
    }
    const float inv = den == 0.f ? 0.f : 1.f / den;
    const size_t at = (size_t)(b * a.m + i + row_of(r));
#pragma unroll
    for (int x = 0; x < H; ++x) {
      const int c = 128 * x + 4 * lane;
      scale4(y[x], inv);
      if (a.gated) {
        const float4 g = dims4(a.qp + at * a.ldq + ((size_t)2 * h + 1) * a.dqk, a.dqk, lane, x);
        y[x].x *= __frcp_rn(1.f + expf(-g.x));
        y[x].y *= __frcp_rn(1.f + expf(-g.y));
        y[x].z *= __frcp_rn(1.f + expf(-g.z));
        y[x].w *= __frcp_rn(1.f + expf(-g.w));
      }
      if (c < a.dv) *reinterpret_cast<float4*>(a.out + (at * a.nh + h) * a.dv + c) = y[x];
    }
  };
  // the four warps' states of a row
  auto own = [&](int r, float& M, float& den) {
    M = -INFINITY;
    den = 0.f;
#pragma unroll
    for (int w = 0; w < kTailWarps; ++w) M = fmaxf(M, sh.m[w][r]);
#pragma unroll
    for (int x = 0; x < H; ++x) y[x] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kTailWarps; ++w) {
      const float f = weight(sh.m[w][r], sh.l[w][r], M);
      den += f * sh.l[w][r];
#pragma unroll
      for (int x = 0; x < H; ++x) add4(y[x], f, dims4(states + w * wstep + r * a.dv, a.dv, lane, x));
    }
  };
  if (parts == 1) {
#pragma unroll 1
    for (int r = warp; r < nr; r += kTailWarps) {
      float M, den;
      own(r, M, den);
      finish(r, M, den);
    }
  } else {
    // the part's state to memory; the last part to arrive joins them all
    const size_t unit = ((size_t)b * a.nkv + kv) * a.items + item;
    float2* const ml = a.tail_ml + (unit * a.parts + part) * RG;
    float* const po = a.tail_o + (unit * a.parts + part) * RG * a.dv;
#pragma unroll 1
    for (int r = warp; r < nr; r += kTailWarps) {
      float M, den;
      own(r, M, den);
      if (lane == 0) __stcg(ml + r, make_float2(M, den));
#pragma unroll
      for (int x = 0; x < H; ++x)
        if (128 * x + 4 * lane < a.dv) __stcg(reinterpret_cast<float4*>(po + r * a.dv + 128 * x + 4 * lane), y[x]);
    }
    __syncthreads();
    if (threadIdx.x == 0) sh.last = atom_add_acq_rel_gpu(a.tail_count + unit, 1u) == (unsigned)parts - 1;
    __syncthreads();
    if (sh.last) {
      if (threadIdx.x == 0) a.tail_count[unit] = 0;  // for the next call
      const float2* const ml0 = a.tail_ml + unit * a.parts * RG;
      const float* const po0 = a.tail_o + unit * a.parts * RG * a.dv;
#pragma unroll 1
      for (int r = warp; r < nr; r += kTailWarps) {
        const float2 m = lane < parts ? __ldcg(ml0 + lane * RG + r) : make_float2(-INFINITY, 0.f);  // lane s has part s's
        const float M = warp_max(m.x), f = weight(m.x, m.y, M), den = warp_sum(f * m.y);
#pragma unroll
        for (int x = 0; x < H; ++x) y[x] = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int NB = 16 / H;  // parts at once: their reads wait together
#pragma unroll 1
        for (int s0 = 0; s0 < parts; s0 += NB) {
          float4 v[NB][H];
#pragma unroll
          for (int k = 0; k < NB; ++k)
#pragma unroll
            for (int x = 0; x < H; ++x) {
              v[k][x] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (s0 + k < parts && 128 * x + 4 * lane < a.dv)
                v[k][x] = __ldcg(reinterpret_cast<const float4*>(po0 + ((size_t)(s0 + k) * RG + r) * a.dv + 128 * x + 4 * lane));
            }
#pragma unroll
          for (int k = 0; k < NB; ++k) {
            const float w = __shfl_sync(0xffffffffu, f, (s0 + k) & 31);  // 0 past the parts
#pragma unroll
            for (int x = 0; x < H; ++x) add4(y[x], w, v[k][x]);
          }
        }
        finish(r, M, den);
      }
    }
  }
  wait.settle();
}

// ------------------------------------------------------------------ host
// Query rows a CTA of the tail launch: a KV head's heads in as few CTAs as 8 a CTA
// allow, as even as they go, of `mrows` new rows (more than one: at most 4 in all).
static int tail_rows(int G, int mrows) {
  const int blocks = (G + 7) / 8, each = mrows * ((G + blocks - 1) / blocks);
  return each <= 2 ? 2 : each <= 4 ? 4 : each == 7 ? 8 : each;
}
// New rows a CTA, where reading a sequence's keys once for several pays: with one or
// two heads a KV head, up to 4 query rows (up to 8: 34 us, not 32, in the case above;
// 32/8 heads, 2 new rows a CTA 55 us, one 47).  Not where the keys of all rows are few:
// then more CTAs read them sooner (16 MB: 8/8 heads of 64, 4 x 8 rows 16 us, not 18).
constexpr long long kManyBytes = 64 << 20;
static int tail_new_rows(int G, int m) {
  if (G > 2) return 1;
  const int most = 4 / G, groups = (m + most - 1) / most;
  return (m + groups - 1) / groups;
}
static size_t tail_smem(int rg, int dqk, int dv) { return (size_t)rg * dqk * 4 + (size_t)kTailWarps * kTailKeys * (dqk + dv) * 4; }

template <int RG, int H, bool ALONE, bool MANY = false>
static cudaError_t launch_tail_as(const PrefixArgs& a, cudaStream_t st) {
  static_assert(RG <= kTailKeys, "a warp's state fits one buffer of values");
  static std::atomic<bool> attr[64];  // per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !attr[dev]) {
    e = cudaFuncSetAttribute(prefix_tail_kernel<RG, H, ALONE, MANY>, cudaFuncAttributeMaxDynamicSharedMemorySize, 80 * 1024);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr[dev] = true;
  }
  return launch_pdl(prefix_tail_kernel<RG, H, ALONE, MANY>, dim3(a.parts * a.items, a.nkv, a.groups * a.per), kTailWarps * 32,
                    tail_smem(RG, a.dqk, a.dv), st, a);
}

template <int H, bool ALONE>
static cudaError_t launch_tail_h(const PrefixArgs& a, cudaStream_t st) {
  const int rg = tail_rows(a.G, a.mrows);
  if (a.mrows > 1) return rg == 2 ? launch_tail_as<2, H, ALONE, true>(a, st) : launch_tail_as<4, H, ALONE, true>(a, st);
  switch (rg) {
    case 2: return launch_tail_as<2, H, ALONE>(a, st);
    case 4: return launch_tail_as<4, H, ALONE>(a, st);
    case 5: return launch_tail_as<5, H, ALONE>(a, st);
    case 6: return launch_tail_as<6, H, ALONE>(a, st);
    default: return launch_tail_as<8, H, ALONE>(a, st);
  }
}

static cudaError_t launch_tail(const PrefixArgs& a, cudaStream_t st) {
  if (a.dqk <= 128 && a.dv <= 128) return a.ns > 0 ? launch_tail_h<1, false>(a, st) : launch_tail_h<1, true>(a, st);
  return a.ns > 0 ? launch_tail_h<2, false>(a, st) : launch_tail_h<2, true>(a, st);
}

// Parts of a sequence's keys, for `units` (sequence, KV head, new row, block of
// heads): as many as the SMs hold at once (`ctas`), of kPartBytes of keys and values
// or more; tails that differ in length get a third more (24 of up to 2048 rows: 60
// us, 66 without, 68 with twice as many).  One warp joins them.  us with parts of 32,
// 64 and 128 KB at least: 40/8 heads of 128, 8 beams, 4096 keys 28.3, 27.3, 27.3; 32
// samples, 1024 keys 25.6, 24.0, 24.0; 16/2 heads of 256, 3 x 5 samples 32.0, 32.1,
// 35.1; alone, 8/2 heads of 64, 4 sequences, 3000 keys 11.1, 11.6, 13.9.
constexpr int kTailCtas = 6, kPartBytes = 64 * 1024;  // CTAs a SM at most

// CTAs of the tail launch that an SM holds.
static int tail_resident(int rg, int dqk, int dv) {
  const size_t smem = tail_smem(rg, dqk, dv) + sizeof(TailSmem) + 1024;
  return std::min(tail_ctas(rg, dqk <= 128 && dv <= 128 ? 1 : 2), (int)(228 * 1024 / smem));
}

struct TailPlan {
  int parts, keys;  // keys a part
};
static TailPlan tail_plan(long long units, long long own, int dims, long long ctas, bool even) {
  static_assert(3 * kTailCtas >= 4 * 4, "four CTAs a SM at most, and a third more");
  static_assert(kTailCtas * 256 / 2 <= kPartCounts, "a counter a unit, where units have several parts");
  const long long most = std::min<long long>(32, std::max<long long>(1, (even ? ctas : ctas * 4 / 3) / units));
  TailPlan p;
  p.keys = (int)std::min<long long>(1 << 30, (std::max<long long>(kPartBytes / (4 * dims), (own + most - 1) / most) + 31) / 32 * 32);
  p.parts = (int)std::max<long long>(1, (own + p.keys - 1) / p.keys);
  return p;
}

// Splits of a prompt's keys: the fewest waves of CTAs (one a SM) times the keys
// of a split and a CTA's fixed cost, about 192 keys (48: 64 samples of 32768 keys 200
// us, not 190, 64/8 heads, 64 x 4096 62, not 53; 512: no change there).  A split has 64
// keys at least: with 32 and 128, 16/2 heads of 256, 3 x 5 samples 32.1 and 33.2 us, 32.1
// with 64; 8 x 4096 32.8 and 30.3, 31.3; 40/8 heads of 128, 8 x 2048 23.5 and 20.9, 23.1.
// Up to three waves: 32/8 heads of 128, 13 x 4 sequences, 4096 keys 113 us, 117 with up to
// one or two; 12 x 4, 8192 keys 160, 212 with one; 16/2 heads of 256, 50 x 4, 2048 keys
// 130, 194 with one; up to six: 20 x 4, 2048 keys 110, not 107.
constexpr int kSplitCost = 192;
constexpr int kSplitKeys = 64;   // of a split at least
constexpr int kSplitWaves = 3;   // CTAs a SM at most, where a prompt has several splits

static int prefix_splits(int heads_tiles, int keys, int sms) {
  if (keys <= 0) return 0;
  const int most = (keys + kSplitKeys - 1) / kSplitKeys;
  int best = 1;
  long long cost = -1;
  for (int waves = 1; waves <= kSplitWaves; ++waves) {  // as many splits as the waves hold
    const int ns = std::min(most, std::max(1, waves * sms / heads_tiles));
    const long long w = ((long long)heads_tiles * ns + sms - 1) / sms, c = w * ((keys + ns - 1) / ns + kSplitCost);
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

// Whether the tail launch reads the prompts itself: `keys` of a prompt that a split
// launch would take (with a window: beside the longest tail), once for each of `units` (sequence, KV head, new row, block of up to `rg`
// heads) rather than once for each of `heads` (prompts' KV heads).  It is then the
// only launch, which saves 6 us, and reads what is not shared at about 5.5 TB/s from
// L2.  us alone, and as three launches, 40/8 heads of 128:
//   2 sequences  4096 keys 21, 22   8192 30, 28
//   8            512 keys 14, 16    1024 18, 18    2048 26, 20
//   32           128 keys 15, 17    256 19, 18
// 16/2 heads of 256, 8 sequences: 1024 keys 19, 21, 2048 24, 24, 4096 31, 29.  Few
// heads a KV head cost the one launch less: 32/8 heads, 8 sequences, 1024 keys 15, 17,
// 2048 21, 20.  A CTA's share grows with the keys: 4/2 heads of 64, one sequence, 8192
// keys 13, 14, 32768 keys 32, 23.
constexpr long long kAloneBytes = 52 << 20, kAloneBytesFew = 72 << 20;
constexpr int kAloneKeys = 12288;
// A split launch has prompts times KV heads along a grid's third axis, which ends at
// 65535: 1024 prompts of 64 KV heads are one more.
constexpr int kSplitHeads = 65535;
static bool tail_alone(long long units, long long heads, long long keys, int dims, int rg) {
  return keys <= kAloneKeys && (units - heads) * keys * dims * 4 <= (rg <= 4 ? kAloneBytesFew : kAloneBytes);
}

struct PrefixWs {
  float* qf;
  uint8_t* qt;
  float* qinv;
  float2 *ml, *tail_ml;
  float *o, *tail_o;
  size_t bytes;
};

// Partials of any call of up to these sizes: splits times query rows, where
// several splits fill at most kSplitWaves CTAs of 128 rows a SM.
static size_t most_partials(const mtp_attn_geom* g, size_t tiles, size_t rows, int pmax, int sms) {
  const size_t keys = shared_keys(g, 1, pmax);
  if (keys == 0) return 0;
  return std::min(rows * ((keys + kSplitKeys - 1) / kSplitKeys), 128 * std::max(tiles, (size_t)kSplitWaves * sms));
}

// `partials`, `tails`: rows of split partials, and of the tail launch's parts where it joins several.
static PrefixWs prefix_ws(void* ws, const mtp_attn_geom* g, int groups, int seqs, int m, size_t partials, size_t tails) {
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
  w.tail_ml = reinterpret_cast<float2*>(take(8 * tails));
  w.tail_o = reinterpret_cast<float*>(take(4 * tails * g->head_dim_v));
  w.bytes = off;
  return w;
}

static size_t prefix_ws_bound(const mtp_attn_geom* g, int groups, int seqs, int m, int pmax) {
  const size_t rows = (size_t)seqs * m * g->n_heads, tiles = rows / 128 + (size_t)groups * g->n_kv_heads;
  // several parts: at most kTailCtas CTAs a SM, of at most 8 rows
  const size_t ctas = (size_t)kTailCtas * sm_count();
  return prefix_ws(nullptr, g, groups, seqs, m, most_partials(g, tiles, rows, pmax, sm_count()), 8 * ctas).bytes;
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
  const long long common = a.window > 0 ? std::min<long long>(pmax, std::max<long long>(0, (long long)a.window - m - tmax)) : pmax;
  int rg;
  long long units, own;
  for (a.mrows = tail_new_rows(a.G, m);; a.mrows = 1) {
    rg = tail_rows(a.G, a.mrows);
    a.items = (m + a.mrows - 1) / a.mrows * ((a.G + rg - 1) / rg);
    units = (long long)B->n_seqs * a.nkv * a.items;
    const bool alone = heads > kSplitHeads || tail_alone(units, heads, common, a.dqk + a.dv, rg);
    a.ns = alone ? 0 : prefix_splits(heads * a.mt, keys, sms);
    // a sequence's own keys: its tail, a window's edge in the prompt, or all of the prompt
    const int edge = a.ns > 0 ? (a.window > 0 ? (int)std::min<long long>(pmax, (long long)tmax + m) : 0) : pmax;
    own = (long long)edge + tmax + m;
    if (a.window > 0) own = std::min<long long>(own, a.window);
    if (a.mrows == 1 || (long long)B->n_seqs * a.nkv * m * own * (a.dqk + a.dv) * 4 >= kManyBytes) break;
  }
  const TailPlan tp = tail_plan(units, own, a.dqk + a.dv, (long long)tail_resident(rg, a.dqk, a.dv) * sms, a.ns == 0);
  a.parts = tp.parts;
  a.part_keys = tp.keys;
  const PrefixWs w = prefix_ws(d_ws, g, a.groups, B->n_seqs, m, (size_t)heads * a.R * a.ns,
                               tp.parts > 1 ? (size_t)units * tp.parts * rg : 0);
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
  a.tail_count = reinterpret_cast<unsigned*>(static_cast<uint8_t*>(d_ws) + sizeof(WsHeader) + kPartCountAt);
  a.tail_ml = w.tail_ml;
  a.tail_o = w.tail_o;
  a.err = &static_cast<WsHeader*>(d_ws)->err;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const long long items = (long long)B->n_seqs * m * (a.nh + 2 * a.nkv);
  cudaError_t e = cudaSuccess;
  if (a.ns > 0) {
    e = launch_pdl(prefix_prep_kernel, dim3((unsigned)((items + kPrefixPrepThreads / 32 - 1) / (kPrefixPrepThreads / 32))),
                   kPrefixPrepThreads, 0, st, a);
    if (e == cudaSuccess) e = launch_prefix_split(a, st);
  }
  if (e == cudaSuccess) e = launch_tail(a, st);
  if (e != cudaSuccess) return cuda_fail(e, "attn_prefix_sink launch");
  return MTP_OK;
}

}  // extern "C"
