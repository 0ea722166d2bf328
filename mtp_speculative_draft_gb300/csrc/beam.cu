// A beam search's selection over beams and vocabulary, and the move of the
// surviving beams' K/V tails.
//
// "cortiq-engine 0.8.49 src/mimo_mtp.rs" keeps one hypothesis (mimo_spec_round
// takes each row's argmax, mimo_verify_rewind cuts the caches back); here a
// prompt has several, as its target's logits allow:
//   candidate (b, v) of a prompt: s = score_b + l_bv - log sum_u exp(l_bu),
//   ranked by s / length^alpha; a finished beam's only candidate is itself.
// Two launches for the selection:
//   1. rows:   a CTA a chunk of a row: its largest logit, the sum of
//              exponentials, and a few logits among which are its k largest;
//   2. merge:  a CTA a prompt: the rows' normalisers, the candidates' ranks, the
//              best k in order.
// Within a row candidates go by their logits, between rows by ranks in 64 bits:
// float32 scores of about -30 are 2e-6 apart, and candidates that close are
// common among 150k tokens.  Sums of exponentials: 32 terms in float32 a thread.  In
// units of 2^-24 a term d below its chunk's largest is off by 2 d (difference, product
// with log2 e) + 0.23 d (log2 e in float32) + 4 (2^x) + 6 (additions), a chunk D below
// the row's by D + 4 (weight); under the softmax d is 6.2 and d + D 17 in the mean at
// most (8192 and 2^30 tokens), so a row's log sum is off by 39 units, 2^-18.7, at most.
// Measured on normal logits of deviation 0.5 to 3: 6e-8 at most, and 3e-8 in the mean
// (log2 e is 1.3e-8 short and 2^x errs by -5e-8 in the mean: they work against each
// other); 1e-7 where a few tokens have the most (deviation 6).
//
// Measured (graph): 4 x 4096, 4 candidates 8.2 us; 8 x 151936, 16 candidates 10.8 us;
// 16 prompts of 4 x 152577, 8 candidates 15.9 us (33 MB, without the finished beams'
// rows: 2.1 TB/s).
#include <algorithm>
#include <cmath>

#include "move.h"
#include "prefix.cuh"

namespace mtp {

constexpr int kSelThreads = 256;
constexpr int kSelPer = 32;                         // logits a thread
constexpr int kSelChunk = kSelThreads * kSelPer;    // logits a CTA
constexpr int kBeamsMost = 64, kBeamTop = 128;      // beams and candidates of a prompt
constexpr int kBeamRows = 1024;                     // beams of a call
constexpr int kSelVocab = 1 << 30;                  // tokens
constexpr int kMergeThreads = 1024;
constexpr int kMergeList = 1024;                    // candidates that are put in order at once
constexpr int kMergeSort = 192;                     // and without a closer look first
constexpr int kMergeChunks = 1024;                  // chunks in a list

struct SelArgs {
  const float* x;
  long long ld;
  int beams, V, k, chunks, cap, eos;
  int units;                  // warps' loads of a chunk's candidates
  unsigned long long magic_chunks, magic_units;  // 2^64 / chunks and 2^32 / units, rounded up: quotients by products
  float alpha;
  const float* score;
  const int *len, *done;
  int *parent, *token, *len_out, *done_out;
  float* score_out;
  unsigned long long* sum;    // [rows][chunks] sum of exponentials relative to the largest logit, in 2^-40
  float* top;                 // [rows][chunks] (below 2^53; all ones: NaN), the largest logit
  unsigned long long* cand;   // [rows][chunks][cap] logit key, ~token; 0: none
  unsigned long long* ranks;  // [rows][chunks][cap] their ranks, where many are equal
};

// Floats as unsigned integers in the same order (-0 and 0 alike; NaN below all
// others, with -infinity).
__device__ __forceinline__ uint32_t float_key(float x) {
  x = x == x ? x + 0.f : -INFINITY;
  const uint32_t u = __float_as_uint(x);
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float key_float(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
constexpr uint32_t kNoKey = 0x007FFFFFu;  // of -infinity
__device__ __forceinline__ unsigned long long double_key(double x) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(x + 0.0);
  return u ^ ((u >> 63) ? 0xFFFFFFFFFFFFFFFFull : 0x8000000000000000ull);
}

// A beam that offers candidates of its row: not finished, with a finite score.
__device__ __forceinline__ bool beam_live(const SelArgs& a, int r) {
  return (!a.done || a.done[r] == 0) && fabsf(a.score[r]) < INFINITY;
}

// About the k-th largest of 32 P keys in shared memory, from below (between k and
// k + k / 16 are at or above it, or it is exact): one warp, bit by bit behind those
// that all have in common.  (Each key's place by counting the larger ones took 1 us
// more for 8 rows of 151936 and 16 candidates, 15 us more for 64 rows and 64.)
template <int P>
__device__ __forceinline__ void near_kth_largest(const uint32_t* keys, int k, uint32_t* found) {
  const int lane = threadIdx.x & 31;
  uint32_t mine[P], least = ~0u, most = 0;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    mine[i] = keys[lane + 32 * i];
    least = min(least, mine[i]);
    most = max(most, mine[i]);
  }
  least = __reduce_min_sync(0xffffffffu, least);
  most = __reduce_max_sync(0xffffffffu, most);
  uint32_t t = most;
  if (least != most) {
    uint32_t bit = 0x80000000u >> __clz(least ^ most);
    t &= ~(2 * bit - 1);
#pragma unroll 1
    for (; bit; bit >>= 1) {
      int m = 0;
#pragma unroll
      for (int i = 0; i < P; ++i) m += mine[i] >= (t | bit);
      m = __reduce_add_sync(0xffffffffu, m);
      if (m >= k) t |= bit;
      if (m >= k && m <= k + k / 16) break;
    }
  }
  if (lane == 0) *found = t;
}

struct RowsSmem {
  uint32_t group[kSelThreads];        // largest keys of groups of threads
  uint32_t wmax[kSelThreads / 32];    // and of warps
  uint32_t sum[kSelThreads / 32][2];              // a warp's sum, in 2^-20 and 2^-40
  uint32_t low;
  int n;
};

// grid (chunks, rows).  Bound by HBM on many rows; a row's logits are read once
// and stay in registers.  Which thread has a token does not depend on where the row
// lies, so equal rows get equal sums to the bit, and equal ranks go to the lower beam
// (16-byte reads from the row's first aligned word on did not have that, and took 17.4
// us, not 15.9, for all of 64 rows of 152577).  The k-th largest of the largest logits
// of groups of threads bounds the chunk's k-th largest from below, so the few logits
// at or above it hold the chunk's k largest; where equal logits make them more than
// `cap`, the k largest are found exactly (lower tokens first among equals).
// A thread's sum of exponentials has 6 roundings a term; the threads' are cut off at
// 2^-40 of the chunk's largest and added exactly, in integers of 2^-20 and 2^-40 (a
// 64-bit floating addition costs a warp 16 cycles of an SM).
// 64 rows of 152577: two waves of CTAs, 3 us apart, each 1.3 us until its logits are
// there and 1 to 1.7 us of work behind them.  (With 16-byte reads the second wave's
// sent to L2 ahead changed nothing; 512 threads of 16 logits took 20 us in all, not
// 17.5, chunks of 4096 19.5.)  64 registers, four CTAs an SM: 40 bytes a thread are
// spilled.
__global__ void __launch_bounds__(kSelThreads, 4) beam_rows_kernel(const __grid_constant__ SelArgs a) {
  __shared__ RowsSmem sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = blockIdx.x, r = blockIdx.y;
  constexpr int kWarps = kSelThreads / 32;
  pdl_wait();
  pdl_launch_dependents();
  const size_t slot = (size_t)r * a.chunks + c;
  if (!beam_live(a, r)) return;  // the row is not read
  unsigned long long* const out = a.cand + slot * a.cap;
  for (int i = tid; i < a.cap; i += kSelThreads) out[i] = 0;  // no candidate, until one is written below
  const float* x = a.x + (size_t)r * a.ld + (size_t)c * kSelChunk;
  const int e0 = c * kSelChunk + tid, left = a.V - c * kSelChunk;  // this thread has logits e0 + j kSelThreads
  float v[kSelPer];
  if (left >= kSelChunk) {
#pragma unroll
    for (int j = 0; j < kSelPer; ++j) v[j] = __ldcs(x + tid + j * kSelThreads);
  } else {
#pragma unroll
    for (int j = 0; j < kSelPer; ++j) v[j] = tid + j * kSelThreads < left ? __ldcs(x + tid + j * kSelThreads) : -INFINITY;
  }
#pragma unroll
  for (int j = 0; j < kSelPer; ++j) v[j] = fmaxf(v[j], -INFINITY);  // NaN counts as -infinity
  if (tid == 0) sh.n = 0;
  float mx = -INFINITY;
#pragma unroll
  for (int j = 0; j < kSelPer; ++j) mx = fmaxf(mx, v[j]);
  const uint32_t top = float_key(mx), wtop = __reduce_max_sync(0xffffffffu, top);
  // groups of 4 threads do for few candidates (64 groups, 18 logits at or above
  // the 16th's), of 2 for up to 32 (128; 39 at or above the 32nd's), single threads for
  // more (64 rows, 64 candidates: with 2 the chunks that keep more than `cap` took 64 us
  // more)
  uint32_t gtop = top;
  const int group = a.k <= 16 ? 2 : a.k <= 32 ? 1 : 0;  // log2 of a group's threads
  if (group > 0) gtop = max(gtop, __shfl_xor_sync(0xffffffffu, gtop, 1));
  if (group > 1) gtop = max(gtop, __shfl_xor_sync(0xffffffffu, gtop, 2));
  if ((lane & ((1 << group) - 1)) == 0) sh.group[tid >> group] = gtop;
  if (lane == 0) sh.wmax[warp] = wtop;
  __syncthreads();
  uint32_t mtop = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) mtop = max(mtop, sh.wmax[w]);
  const float M = key_float(mtop), ref = M == -INFINITY ? 0.f : M;  // the chunk's largest logit
  if (warp == 0 && group == 2)
    near_kth_largest<kSelThreads / 128>(sh.group, a.k, &sh.low);
  else if (warp == 0 && group == 1)
    near_kth_largest<kSelThreads / 64>(sh.group, a.k, &sh.low);
  else if (warp == 0)
    near_kth_largest<kSelThreads / 32>(sh.group, a.k, &sh.low);
  float s8[8] = {};
#pragma unroll
  for (int j = 0; j < kSelPer; ++j) s8[j & 7] += ex2((v[j] - ref) * kLog2e);
  const float s = ((s8[0] + s8[1]) + (s8[2] + s8[3])) + ((s8[4] + s8[5]) + (s8[6] + s8[7]));
  // at most 32; NaN (+infinity in the row) is marked by a sum that no row has
  const bool bad = __any_sync(0xffffffffu, s != s);
  const uint32_t s1 = (uint32_t)(s * 0x1p20f), s2 = (uint32_t)((s * 0x1p20f - (float)s1) * 0x1p20f);
  const uint32_t t1 = __reduce_add_sync(0xffffffffu, s1), t2 = __reduce_add_sync(0xffffffffu, s2);
  if (lane == 0) {
    sh.sum[warp][0] = bad ? 0xFFFFFFFFu : t1;
    sh.sum[warp][1] = t2;
  }
  __syncthreads();
  const float low = key_float(max(sh.low, kNoKey + 1));
  if (mx >= low) {
    uint32_t mask = 0;
#pragma unroll
    for (int j = 0; j < kSelPer; ++j) mask |= v[j] >= low ? 1u << j : 0u;
    int at = atomicAdd(&sh.n, __popc(mask));
#pragma unroll 1
    for (; mask; mask &= mask - 1, ++at) {
      const int j = __ffs(mask) - 1, tok = e0 + j * kSelThreads;
      if (at < a.cap) out[at] = (unsigned long long)float_key(x[tid + j * kSelThreads]) << 32 | (0xFFFFFFFFu - (uint32_t)tok);
    }
  }
  if (warp == kWarps - 1) {
    unsigned long long t = 0;
    bool nan = false;
    if (lane < kWarps) {
      nan = sh.sum[lane][0] == 0xFFFFFFFFu;
      t = ((unsigned long long)sh.sum[lane][0] << 20) + sh.sum[lane][1];
    }
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    nan = __any_sync(0xffffffffu, nan);
    if (lane == 0) {
      a.top[slot] = M;
      a.sum[slot] = nan ? ~0ull : t;
    }
  }
  __syncthreads();
  if (sh.n > a.cap) {
    // the k-th largest key, then how many of that key are wanted, and up to which token
    uint32_t kth = 0;
#pragma unroll 1
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t t = kth | 1u << bit;
      int m = 0;
#pragma unroll
      for (int j = 0; j < kSelPer; ++j) m += float_key(v[j]) >= t;
      __syncthreads();
      if (tid == 0) sh.n = 0;
      __syncthreads();
      m = __reduce_add_sync(0xffffffffu, m);
      if (lane == 0) atomicAdd(&sh.n, m);
      __syncthreads();
      if (sh.n >= a.k) kth = t;
    }
    // of the tokens with that key, those up to `end` are taken: the least end at
    // which k tokens are there
    int end = 0;
#pragma unroll 1
    for (int bit = 30; bit >= 0; --bit) {
      const int t = end + (1 << bit);  // end stays below 2^30, t below 2^31
      int m = 0;
#pragma unroll
      for (int j = 0; j < kSelPer; ++j) {
        const int tok = e0 + j * kSelThreads;
        const uint32_t key = float_key(v[j]);
        m += key > kth || (key == kth && tok < t);
      }
      __syncthreads();
      if (tid == 0) sh.n = 0;
      __syncthreads();
      m = __reduce_add_sync(0xffffffffu, m);
      if (lane == 0) atomicAdd(&sh.n, m);
      __syncthreads();
      if (sh.n < a.k) end = t;
    }
    __syncthreads();
    if (tid == 0) sh.n = 0;
    __syncthreads();
#pragma unroll 1
    for (int j = 0; j < kSelPer; ++j) {
      float f = 0.f;
#pragma unroll
      for (int i = 0; i < kSelPer; ++i)
        if (i == j) f = v[i];
      const int tok = e0 + j * kSelThreads;
      const uint32_t key = float_key(f);
      if (key > kth || (key == kth && tok <= end))
        out[atomicAdd(&sh.n, 1)] = (unsigned long long)key << 32 | (0xFFFFFFFFu - (uint32_t)tok);
    }
    for (int i = a.k + tid; i < a.cap; i += kSelThreads) out[i] = 0;
  }
}

// Tables of logarithms and powers, worked out by the compiler: of the middles
// c = 1 + (i + 1/2) / 128, log c = 2 artanh((c - 1) / (c + 1)) and 1 / c; of
// exponents i / 32, exp(i / 32 log 2) by its series.
constexpr int kLogSteps = 128, kExpSteps = 32;
constexpr double kLn2 = 0.69314718055994530942;
struct MathTables {
  double logs[kLogSteps], inverse[kLogSteps], powers[kExpSteps];
};
constexpr MathTables make_tables() {
  MathTables t = {};
  for (int i = 0; i < kLogSteps; ++i) {
    const double c = 1.0 + (i + 0.5) / kLogSteps, z = (c - 1) / (c + 1);
    double sum = 0.0, term = z;
    for (int n = 1; n < 60; n += 2, term *= z * z) sum += term / n;
    t.logs[i] = 2 * sum;
    t.inverse[i] = 1 / c;
  }
  for (int i = 0; i < kExpSteps; ++i) {
    double sum = 0.0, term = 1.0;
    for (int n = 1; n < 30; ++n) {
      sum += term;
      term *= i * kLn2 / kExpSteps / n;
    }
    t.powers[i] = sum;
  }
  return t;
}
__device__ const MathTables kTables = make_tables();

struct MergeSmem {
  double lse[kBeamsMost], score[kBeamsMost];
  double norm[kBeamsMost], inverse[kBeamsMost];  // length^alpha of a candidate, and its inverse
  MathTables math;
  double least[2];
  float base[kBeamsMost], inv[kBeamsMost];       // score - lse, and inverse / the largest inverse
  int len[kBeamsMost], kind[kBeamsMost];         // 0 nothing, 1 tokens, 2 itself
  uint32_t group[256];
  uint32_t low;
  unsigned long long key[kMergeList];            // ranks
  uint32_t beam[kMergeList], tok[kMergeList];
  float logit[kMergeList];
  unsigned long long best_key[kMergeThreads / 32];
  unsigned long long best_id[kMergeThreads / 32];
  unsigned long long last_key, last_id;
  uint32_t slot[kMergeChunks];                   // chunks that may hold one of the k best, and their beams
  uint8_t slot_beam[kMergeChunks];
  int n, slots;
};

// log of a finite s >= 2^-1022 after P. T. P. Tang's table-driven method (1990):
// s = 2^e f, f = c (1 + u) with c the middle of f's step, |u| <= 2^-8; the series of
// log(1 + u) up to u^5 leaves less than 2^-50.
__device__ __forceinline__ double table_log(const MathTables& t, double s) {
  const unsigned long long w = (unsigned long long)__double_as_longlong(s);
  const int e = (int)(w >> 52) - 1023, i = (int)(w >> 45) & (kLogSteps - 1);
  const double f = __longlong_as_double((long long)((w & 0xFFFFFFFFFFFFFull) | 0x3FF0000000000000ull));
  const double u = (f - (1.0 + (i + 0.5) / kLogSteps)) * t.inverse[i];
  return e * kLn2 + (t.logs[i] + u * (1.0 + u * (-1.0 / 2 + u * (1.0 / 3 + u * (-1.0 / 4 + u * (1.0 / 5))))));
}
// exp of |x| < 700 after his method for exponentials (1989): x = (32 e + i) log 2 / 32
// + u, |u| <= 0.0109; the series of exp u up to u^6 leaves less than 2^-57.
__device__ __forceinline__ double table_exp(const MathTables& t, double x) {
  const int n = __float2int_rn((float)x * (float)(kExpSteps / kLn2));
  const double u = x - n * (kLn2 / kExpSteps);
  const double p = 1.0 + u * (1.0 + u * (1.0 / 2 + u * (1.0 / 6 + u * (1.0 / 24 + u * (1.0 / 120 + u * (1.0 / 720))))));
  const int e = n >> 5;  // rounded down
  return t.powers[n & (kExpSteps - 1)] * p * __longlong_as_double((long long)(e + 1023) << 52);
}

// One CTA a prompt.  64-bit arithmetic is slow here (two products a cycle and SM),
// so candidates are first compared by float32 ranks with a bound of their error;
// only those that may be among the k best get a rank in 64 bits.  What depends on
// the beams alone is worked out while the rows are still being read.  Bound by the
// latency of its steps and of fetching its instructions, which are few for that: 8
// rows of 151936 take 6 us from the rows' end (all ranks, logarithms and powers in
// 64 bits took 45).  Candidates are read a chunk by a warp: chunk and beam are then
// known without a division a candidate.
__global__ void __launch_bounds__(kMergeThreads) beam_merge_kernel(const __grid_constant__ SelArgs a) {
  __shared__ MergeSmem sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int seq = blockIdx.x, row0 = seq * a.beams;
  constexpr int kWarps = kMergeThreads / 32;
  if (tid == 0) sh.n = sh.slots = 0;
  if (tid < (int)(sizeof(MathTables) / 8)) reinterpret_cast<double*>(&sh.math)[tid] = reinterpret_cast<const double*>(&kTables)[tid];
  // scores, lengths and flags were final before the call's first launch
  int next = 1, kind = 0;
  if (tid < a.beams) {
    const int r = row0 + tid;
    const float score = a.score[r];
    const bool done = a.done && a.done[r] != 0;
    kind = fabsf(score) < INFINITY ? (done ? 2 : 1) : 0;
    next = a.len ? a.len[r] : 0;
    if (kind == 1 && next < 0x7FFFFFFF) ++next;
    sh.score[tid] = (double)score;
    sh.base[tid] = score;  // of a finished beam
    sh.kind[tid] = kind;
    sh.len[tid] = next;
    sh.lse[tid] = 0.0;
    sh.norm[tid] = sh.inverse[tid] = 1.0;
    sh.inv[tid] = 1.f;
  }
  __syncthreads();
  if (a.alpha != 0.f && tid < kBeamsMost) {  // two whole warps
    // within 1e+-200, so that a rank times it is the score again
    double most = 0.0, inverse = 0.0;
    if (tid < a.beams) {
      const double x = fmin(fmax((double)a.alpha * table_log(sh.math, (double)max(next, 1)), -460.5), 460.5);
      sh.norm[tid] = table_exp(sh.math, x);
      sh.inverse[tid] = inverse = table_exp(sh.math, -x);
      if (kind) most = inverse;
    }
    for (int o = 16; o > 0; o >>= 1) most = fmax(most, __shfl_xor_sync(0xffffffffu, most, o));
    if (lane == 0) sh.least[warp] = most;
    asm volatile("bar.sync 1, 64;" ::: "memory");
    most = fmax(sh.least[0], sh.least[1]);
    if (tid < a.beams && kind) sh.inv[tid] = (float)(inverse / most);
  }
  // A warp reads 32 candidates of one chunk at a time, a unit of all chunks or of the
  // listed ones: unit u's beam, and where this lane's candidate is; ~0: none.  (64
  // beams of 2^30 tokens: just below 2^31 candidates, 2^26 units.)
  const uint32_t all_slots = (uint32_t)a.beams * a.chunks;
  const unsigned long long* cand = a.cand + (size_t)row0 * a.chunks * a.cap;
  uint32_t n_units = all_slots * a.units;
  bool listed = false;
  auto beam_of = [&](uint32_t slot) {
    return a.chunks > 1 ? (int)__umul64hi((unsigned long long)slot, a.magic_chunks) : (int)slot;
  };
  auto locate = [&](uint32_t u, int& b) {
    const uint32_t i = (uint32_t)((unsigned long long)u * a.magic_units >> 32), slot = listed ? sh.slot[i] : i;
    const int j = (int)(u - i * a.units) * 32 + lane;
    b = listed ? (int)sh.slot_beam[i] : beam_of(slot);
    return j < a.cap ? slot * (uint32_t)a.cap + j : ~0u;
  };
  constexpr int kRound = 4;  // units of a warp at once
  uint32_t rounds = (n_units + kRound * kWarps - 1) / (kRound * kWarps);
  unsigned long long w[kRound];
  int beam[kRound];
  auto load_round = [&](uint32_t q) {
#pragma unroll
    for (int i = 0; i < kRound; ++i) {
      const uint32_t u = (q * kRound + i) * kWarps + warp;
      w[i] = 0;  // also 0: no candidate; anything where a row was not read
      beam[i] = 0;
      if (u < n_units) {
        const uint32_t at = locate(u, beam[i]);
        if (at != ~0u) w[i] = cand[at];
      }
    }
  };
  pdl_wait();
  pdl_launch_dependents();
  if (rounds == 1) load_round(0);  // on their way while the rows' normalisers are worked out
#pragma unroll 1
  for (int b = warp; b < a.beams; b += kWarps) {
    if (sh.kind[b] != 1) continue;
    const size_t at = (size_t)(row0 + b) * a.chunks;
    float m = -INFINITY;
    double s = 0.0;
    bool nan = false;
    auto part = [&](int c) {
      const unsigned long long w = a.sum[at + c];
      nan |= w == ~0ull;
      return (double)w * 0x1p-40;
    };
    if (lane < a.chunks) {
      m = a.top[at + lane];
      s = part(lane);
    }
    float M = m;
    for (int c = lane + 32; c < a.chunks; c += 32) M = fmaxf(M, a.top[at + c]);
    M = warp_max(M);
    s = m == -INFINITY ? 0.0 : s * (double)expf(m - M);
    for (int c = lane + 32; c < a.chunks; c += 32) {
      m = a.top[at + c];
      if (m != -INFINITY) s += part(c) * (double)expf(m - M);
    }
    nan = __any_sync(0xffffffffu, nan);
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) {
      if (fabsf(M) < INFINITY && !nan) {
        const double lse = (double)M + table_log(sh.math, s);
        sh.lse[b] = lse;
        sh.base[b] = (float)(sh.score[b] - lse);
      } else {
        sh.kind[b] = 0;  // no token, or +infinity
      }
    }
  }
  __syncthreads();

  // float32 rank (in units of the largest inverse) from below and from above: four
  // roundings of numbers up to |base| + |logit|, and what is too small for a float
  auto bounds = [&](int b, float logit, float& lo, float& hi) {
    const float inv = sh.inv[b], base = sh.base[b], size = fabsf(base) + fabsf(logit), rank = (base + logit) * inv;
    const float e = size * (inv * 0x1p-21f + 0x1p-100f) + 0x1p-120f;
    lo = rank - e;
    hi = rank + e;
  };
  auto rank = [&](int b, float logit) {
    const double s = sh.kind[b] == 1 ? sh.score[b] + ((double)logit - sh.lse[b]) : sh.score[b];
    return double_key(s * sh.inverse[b]);
  };
  auto collect = [&](int b, uint32_t tok, float logit) {
    const int i = atomicAdd(&sh.n, 1);
    if (i < kMergeList) {
      sh.beam[i] = b;
      sh.tok[i] = tok;
      sh.logit[i] = logit;
    }
  };
  // first the threads' best from below, of which the k-th largest bounds the k best;
  // then every candidate that may reach it
  const bool itself = tid < a.beams && sh.kind[tid] == 2;  // a finished beam
  float self_lo = -INFINITY, self_hi = -INFINITY;
  if (itself) bounds(tid, 0.f, self_lo, self_hi);
  uint32_t low = 0;
  bool direct = false;
  if (rounds > 1 && all_slots > (uint32_t)a.k) {
    // many candidates: first the chunks whose largest logit may be among the k best,
    // by the k-th largest of theirs and of the finished beams (16 rows of 151936, 32
    // candidates: 15 us in all, 10 more without; 64 rows, 64 candidates: 38, 78 more)
    const float* tops = a.top + (size_t)row0 * a.chunks;
    if (tid < 256) sh.group[tid] = 0;
    __syncthreads();
    auto chunk_bounds = [&](uint32_t c, float& lo, float& hi) {
      const int b = beam_of(c);
      if (sh.kind[b] != 1) return false;
      const float t = tops[c];
      bounds(b, t, lo, hi);
      return t != -INFINITY;
    };
    if (itself && self_lo == self_lo) atomicMax(&sh.group[255 - tid], float_key(self_lo));
    for (uint32_t c = tid; c < all_slots; c += kMergeThreads) {
      float lo, hi;
      if (chunk_bounds(c, lo, hi) && lo == lo) atomicMax(&sh.group[c & 255], float_key(lo));
    }
    __syncthreads();
    if (warp == 0) near_kth_largest<8>(sh.group, a.k, &sh.low);
    __syncthreads();
    low = sh.low;  // 0: fewer than k
    direct = low != 0 && a.k <= 64;
    for (uint32_t c = tid; c < all_slots; c += kMergeThreads) {
      float lo, hi;
      if (!chunk_bounds(c, lo, hi) || (hi == hi && float_key(hi) < low)) continue;
      const int i = atomicAdd(&sh.slots, 1);
      if (i < kMergeChunks) {
        sh.slot[i] = c;
        sh.slot_beam[i] = beam_of(c);
      }
    }
    __syncthreads();
    if (sh.slots <= kMergeChunks) {  // else all of them
      listed = true;
      n_units = sh.slots * a.units;
      rounds = (n_units + kRound * kWarps - 1) / (kRound * kWarps);
      load_round(0);
    }
  }
  // the candidates that reach `low`; without one, or if they are too many, first the
  // threads' best from below, of which the k-th largest is a (better) `low`.  (For
  // more than 64 they often are: 8 rows, 128 candidates took 12 us more in one pass at
  // first; 16 rows, 32 candidates 3 us less.)
#pragma unroll 1
  for (int pass = direct ? 1 : 0; pass < 2; ++pass) {
    float best = self_lo;
#pragma unroll 1
    for (uint32_t q = 0; q < rounds; ++q) {
      if (rounds > 1) load_round(q);
#pragma unroll
      for (int i = 0; i < kRound; ++i) {
        if (w[i] == 0 || sh.kind[beam[i]] != 1) continue;
        const float logit = key_float((uint32_t)(w[i] >> 32));
        float lo, hi;
        bounds(beam[i], logit, lo, hi);
        best = fmaxf(best, lo);  // NaN takes no part
        if (pass == 1 && (hi != hi || float_key(hi) >= low)) collect(beam[i], 0xFFFFFFFFu - (uint32_t)w[i], logit);
      }
    }
    if (pass == 0) {
      uint32_t top = float_key(best);
      const int share = a.k <= 16 ? kMergeThreads / 64 : kMergeThreads / 256;  // threads a group
      for (int o = 1; o < share; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (tid % share == 0) sh.group[tid / share] = top;
      __syncthreads();
      if (warp == 0 && a.k <= 16)
        near_kth_largest<2>(sh.group, a.k, &sh.low);
      else if (warp == 0)
        near_kth_largest<8>(sh.group, a.k, &sh.low);
      __syncthreads();
      low = max(sh.low, 1u);
      direct = false;
    } else {
      if (itself && (self_hi != self_hi || float_key(self_hi) >= low)) collect(tid, (uint32_t)a.eos, 0.f);
      __syncthreads();
      if (sh.n > kMergeList && direct) {
        __syncthreads();
        if (tid == 0) sh.n = 0;
        pass = -1;
      }
    }
  }
  __syncthreads();
  int n = sh.n;
  if (n > kMergeSort && n <= kMergeList) {
    // of many, only those that reach the k-th largest from below, found bit by bit:
    // their order takes n^2 comparisons
    float lo = -INFINITY, hi = -INFINITY;
    uint32_t b = 0, t = 0;
    float logit = 0.f;
    if (tid < n) {
      b = sh.beam[tid];
      t = sh.tok[tid];
      logit = sh.logit[tid];
      bounds(b, logit, lo, hi);
    }
    const uint32_t mine = tid < n ? float_key(lo) : 0u;
    uint32_t kth = 0;
#pragma unroll 1
    for (uint32_t bit = 0x80000000u; bit; bit >>= 1) {
      const int m = __syncthreads_count(mine >= (kth | bit));
      if (m >= a.k) kth |= bit;
      if (m >= a.k && m <= a.k + a.k / 8) break;
    }
    if (tid == 0) sh.n = 0;
    __syncthreads();
    if (tid < n && (hi != hi || float_key(hi) >= kth)) collect(b, t, logit);
    __syncthreads();
    n = sh.n;
  }
  auto put = [&](int at, uint32_t b, uint32_t tok, unsigned long long key) {
    const size_t o = (size_t)seq * a.k + at;
    const bool none = b == 0xFFFFFFFFu;
    a.parent[o] = none ? -1 : (int)b;
    a.token[o] = none ? -1 : (int)tok;
    float score = -INFINITY;
    if (!none) {
      const unsigned long long u = key ^ ((key >> 63) ? 0x8000000000000000ull : 0xFFFFFFFFFFFFFFFFull);
      score = (float)(__longlong_as_double((long long)u) * sh.norm[b]);
    }
    a.score_out[o] = score;
    if (a.len_out) a.len_out[o] = none ? 0 : sh.len[b];
    if (a.done_out) a.done_out[o] = none ? 0 : (sh.kind[b] == 2 || (int)tok == a.eos);
  };
  if (n <= kMergeList) {
    for (int i = tid; i < n; i += kMergeThreads) sh.key[i] = rank(sh.beam[i], sh.logit[i]);
    __syncthreads();
    // a candidate's place is the number of better ones: a warp a candidate
    for (int i = warp; i < n; i += kWarps) {
      const unsigned long long key = sh.key[i];
      const uint32_t b = sh.beam[i], t = sh.tok[i];
      int at = 0;
      for (int j = lane; j < n; j += 32)
        at += sh.key[j] > key || (sh.key[j] == key && (sh.beam[j] < b || (sh.beam[j] == b && sh.tok[j] < t)));
      at = __reduce_add_sync(0xffffffffu, at);
      if (lane == 0 && at < a.k) put(at, b, t, key);
    }
    for (int i = n + tid; i < a.k; i += kMergeThreads) put(i, 0xFFFFFFFFu, 0, 0);
    return;
  }
  // many (nearly) equal ranks: all of them in 64 bits, then one candidate after
  // another, each the best behind the last
  unsigned long long* ranks = a.ranks + (size_t)row0 * a.chunks * a.cap;
  for (uint32_t u = warp; u < n_units; u += kWarps) {
    int b;
    const uint32_t at = locate(u, b);
    if (at == ~0u) continue;
    const unsigned long long x = sh.kind[b] == 1 ? cand[at] : 0ull;
    ranks[at] = x ? rank(b, key_float((uint32_t)(x >> 32))) : 0ull;
  }
  const unsigned long long self_key = itself ? rank(tid, 0.f) : 0ull;
  if (tid == 0) {
    sh.last_key = ~0ull;
    sh.last_id = 0;
  }
  __syncthreads();
  for (int i = 0; i < a.k; ++i) {
    const unsigned long long lk = sh.last_key, li = sh.last_id;
    unsigned long long bk = 0, bi = ~0ull;  // best rank, then lowest beam and token
    auto see = [&](unsigned long long key, unsigned long long id) {
      if (key == 0 || key > lk || (key == lk && id <= li)) return;  // lk starts above every rank
      if (key > bk || (key == bk && id < bi)) {
        bk = key;
        bi = id;
      }
    };
    for (uint32_t u = warp; u < n_units; u += kWarps) {
      int b;
      const uint32_t at = locate(u, b);
      const unsigned long long key = at != ~0u ? ranks[at] : 0ull;
      if (key >= bk && key != 0) see(key, (unsigned long long)b << 32 | (0xFFFFFFFFu - (uint32_t)cand[at]));
    }
    see(self_key, (unsigned long long)tid << 32 | (uint32_t)a.eos);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long k2 = __shfl_xor_sync(0xffffffffu, bk, o), i2 = __shfl_xor_sync(0xffffffffu, bi, o);
      if (k2 > bk || (k2 == bk && i2 < bi)) {
        bk = k2;
        bi = i2;
      }
    }
    if (lane == 0) {
      sh.best_key[warp] = bk;
      sh.best_id[warp] = bi;
    }
    __syncthreads();
    if (tid == 0) {
      for (int x = 0; x < kWarps; ++x)
        if (sh.best_key[x] > bk || (sh.best_key[x] == bk && sh.best_id[x] < bi)) {
          bk = sh.best_key[x];
          bi = sh.best_id[x];
        }
      sh.last_key = bk;
      sh.last_id = bi;
      put(i, (uint32_t)(bi >> 32), (uint32_t)bi, bk);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ reorder
constexpr int kMoveLayers = 64;  // layers of one launch

struct MoveArgs {
  float* k[kMoveLayers];
  float* v[kMoveLayers];
  const int *parent, *len;
  int seqs, beams, nkv, dqk, dv, most, rows, tiles;  // rows a tile
  int shift;                                         // of a beam's 2^shift 16-byte words of a tile
  long long cap;
  int* err;
};

// grid (row tiles x prompts, KV heads x K or V, layers).  In place: a CTA reads
// its rows of every beam that changes into registers before it writes any of
// them, so beams may exchange places, or several take one beam's tail.  Bound by
// HBM: 8 prompts of 4 beams, tails of 94 to 101 rows, 48 layers of 8 heads of 2 x 128:
// 239 us, 1.59 GB at 6.6 TB/s with three CTAs an SM; 257 with CTAs of 512 threads of 8
// words, 273 with two of this one, 275 with four, which spill.
__global__ void __launch_bounds__(kMoveThreads, 3) kv_beam_kernel(const __grid_constant__ MoveArgs a) {
  __shared__ float *to[kBeamsMost], *from[kBeamsMost];
  __shared__ int words[kBeamsMost];
  __shared__ int n;
  const int tid = threadIdx.x;
  const int seq = blockIdx.x / a.tiles, r0 = blockIdx.x % a.tiles * a.rows;
  const int kv = blockIdx.y >> 1, d = blockIdx.y & 1 ? a.dv : a.dqk;
  float* base = (blockIdx.y & 1 ? a.v[blockIdx.z] : a.k[blockIdx.z]) +
                (((size_t)seq * a.beams * a.nkv + kv) * a.cap + r0) * d;
  const size_t beam_step = (size_t)a.nkv * a.cap * d;
  pdl_wait();
  pdl_launch_dependents();
  if (tid < 32) {
    int have = 0;
    for (int b0 = 0; b0 < a.beams; b0 += 32) {
      const int b = b0 + tid;
      int p = -1, len = 0;
      if (b < a.beams) {
        p = a.parent[seq * a.beams + b];
        len = a.len[seq * a.beams + b];
        if (p >= a.beams || len > a.most) {
          set_dev_error(a.err, kErrBadLength);
          if (p >= a.beams) p = -1;
          len = min(len, a.most);
        }
      }
      const int rows = min(a.rows, max(len, 0) - r0);
      const bool moves = p >= 0 && p != b && rows > 0;
      const unsigned m = __ballot_sync(0xffffffffu, moves);
      if (moves) {
        const int i = have + __popc(m & ((1u << tid) - 1));
        to[i] = base + b * beam_step;
        from[i] = base + p * beam_step;
        words[i] = rows * d / 4;
      }
      have += __popc(m);
    }
    if (tid == 0) n = have;
  }
  __syncthreads();
  // word w of the j-th beam that changes is number j 2^shift + w
  const int all = n << a.shift, mask = (1 << a.shift) - 1;
  float4 x[kMoveWords];
#pragma unroll
  for (int i = 0; i < kMoveWords; ++i) {
    if (i * kMoveThreads >= all) break;
    const int e = tid + i * kMoveThreads, j = e >> a.shift, w = e & mask;
    if (e < all && w < words[j]) x[i] = *reinterpret_cast<const float4*>(from[j] + 4 * w);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kMoveWords; ++i) {
    if (i * kMoveThreads >= all) break;
    const int e = tid + i * kMoveThreads, j = e >> a.shift, w = e & mask;
    if (e < all && w < words[j]) *reinterpret_cast<float4*>(to[j] + 4 * w) = x[i];
  }
}

// ------------------------------------------------------------------ host
struct SelWs {
  unsigned long long* sum;
  unsigned long long* cand;
  unsigned long long* ranks;
  float* top;
  size_t bytes;
};

// Candidates of a chunk that are kept: about as many as reach the k-th largest of
// the groups' largest (18 for 16 candidates, 73 for 64, 176 for 128), and some.
static int sel_cap(int k) { return k + k / 4 + k * k / 256 + 8; }

// Chunks of a row of V logits.
static int sel_chunks(int V) { return (V + kSelChunk - 1) / kSelChunk; }

static SelWs sel_ws(void* ws, int rows, int V, int k) {
  SelWs w = {};
  size_t off = sizeof(WsHeader) + kRuleJoinBytes;
  uint8_t* b = static_cast<uint8_t*>(ws);
  auto take = [&](size_t bytes) {
    uint8_t* p = b ? b + off : nullptr;
    off = (off + bytes + 255) & ~size_t(255);
    return p;
  };
  const size_t slots = (size_t)rows * sel_chunks(V);
  w.sum = reinterpret_cast<unsigned long long*>(take(8 * slots));
  w.cand = reinterpret_cast<unsigned long long*>(take(8 * slots * sel_cap(k)));
  w.ranks = reinterpret_cast<unsigned long long*>(take(8 * slots * sel_cap(k)));
  w.top = reinterpret_cast<float*>(take(4 * slots));
  w.bytes = off;
  return w;
}

static bool sel_sizes(int64_t seqs, int64_t beams, int V, int k) {
  return seqs >= 1 && beams >= 1 && beams <= kBeamsMost && seqs * beams <= kBeamRows && V >= 1 &&
         V <= kSelVocab && k >= 1 && k <= kBeamTop;
}

static bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

static bool overlap(const void* p, size_t pn, const void* q, size_t qn) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p && q && a < b + qn && b < a + pn;
}

}  // namespace mtp

using namespace mtp;

extern "C" {

size_t beam_select_workspace_bytes(int32_t n_seqs, int32_t beams, int32_t vocab, int32_t k) {
  return sel_sizes(n_seqs, beams, vocab, k) ? sel_ws(nullptr, n_seqs * beams, vocab, k).bytes : 0;
}

mtp_status beam_select(const mtp_beam_set* B, const float* d_logits, int64_t ld, int32_t k, int32_t* d_parent,
                       int32_t* d_token, float* d_score_out, int32_t* d_len_out, int32_t* d_done_out, void* d_ws,
                       size_t ws_bytes, void* stream) {
  if (!B || !B->d_score || !d_logits || !d_parent || !d_token || !d_score_out)
    return fail(MTP_ERR_INVALID_ARG, "beam_select: null pointer");
  if (!sel_sizes(B->n_seqs, B->beams, B->vocab, k))
    return fail(MTP_ERR_UNSUPPORTED,
                "beam_select: 1..64 beams a prompt, 1..1024 in all, 1..2^30 tokens, 1..128 candidates");
  if (ld < B->vocab) return fail(MTP_ERR_INVALID_ARG, "beam_select: row stride below the vocabulary");
  if (B->eos < -1 || B->eos >= B->vocab || (B->d_done && B->eos < 0))
    return fail(MTP_ERR_INVALID_ARG, "beam_select: finished beams need an eos token of the vocabulary");
  if (!std::isfinite(B->length_penalty) || (!B->d_len && (B->length_penalty != 0.f || d_len_out)))
    return fail(MTP_ERR_INVALID_ARG, "beam_select: a length penalty and new lengths need the beams' lengths");
  const void* in[3] = {B->d_score, B->d_len, B->d_done};
  const void* out[5] = {d_score_out, d_len_out, d_done_out, d_parent, d_token};
  for (const void* p : in)
    if (!aligned4(p)) return fail(MTP_ERR_INVALID_ARG, "beam_select: misaligned pointer");
  for (const void* p : out)
    if (!aligned4(p)) return fail(MTP_ERR_INVALID_ARG, "beam_select: misaligned pointer");
  if (!aligned4(d_logits)) return fail(MTP_ERR_INVALID_ARG, "beam_select: misaligned pointer");
  const int rows = B->n_seqs * B->beams;
  const size_t nin = 4 * (size_t)rows, nout = 4 * (size_t)B->n_seqs * k;
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < 3; ++j)
      if (overlap(out[i], nout, in[j], nin) && !(i == j && out[i] == in[j] && k == B->beams))
        return fail(MTP_ERR_INVALID_ARG,
                    "beam_select: an output overlaps an input (in place: its own, with as many candidates as beams)");
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], nout, out[j], nout))
        return fail(MTP_ERR_INVALID_ARG, "beam_select: outputs overlap");
    if (overlap(out[i], nout, d_logits, 4 * ((size_t)(rows - 1) * ld + B->vocab)))
      return fail(MTP_ERR_INVALID_ARG, "beam_select: an output overlaps the logits");
  }
  const SelWs w = sel_ws(d_ws, rows, B->vocab, k);
  if (!d_ws || !aligned16(d_ws) || ws_bytes < w.bytes)
    return fail(MTP_ERR_WORKSPACE, "beam_select: workspace too small or misaligned");
  SelArgs a = {};
  a.x = d_logits;
  a.ld = ld;
  a.beams = B->beams;
  a.V = B->vocab;
  a.k = k;
  a.chunks = sel_chunks(B->vocab);
  a.cap = sel_cap(k);
  a.units = (a.cap + 31) / 32;
  a.magic_chunks = a.chunks > 1 ? ~0ull / (unsigned long long)a.chunks + 1 : 0;
  a.magic_units = ((1ull << 32) + a.units - 1) / a.units;
  a.eos = B->eos;
  a.alpha = B->length_penalty;
  a.score = B->d_score;
  a.len = B->d_len;
  a.done = B->d_done;
  a.parent = d_parent;
  a.token = d_token;
  a.score_out = d_score_out;
  a.len_out = d_len_out;
  a.done_out = d_done_out;
  a.sum = w.sum;
  a.top = w.top;
  a.ranks = w.ranks;
  a.cand = w.cand;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_pdl(beam_rows_kernel, dim3(a.chunks, rows), kSelThreads, 0, st, a);
  if (e == cudaSuccess) e = launch_pdl(beam_merge_kernel, dim3(B->n_seqs), kMergeThreads, 0, st, a);
  if (e != cudaSuccess) return cuda_fail(e, "beam_select launch");
  return MTP_OK;
}

size_t kv_beam_workspace_bytes(void) { return sizeof(WsHeader); }

mtp_status kv_beam_reorder(const mtp_kv_caches* C, const int32_t* d_parent, int32_t n_seqs, int32_t beams,
                           const int32_t* d_len, int32_t max_len, void* d_ws, size_t ws_bytes, void* stream) {
  if (!C || !C->h_k || !C->h_v || !d_parent || !d_len)
    return fail(MTP_ERR_INVALID_ARG, "kv_beam_reorder: null pointer");
  if (n_seqs < 1 || beams < 1 || beams > kBeamsMost || (int64_t)n_seqs * beams > kBeamRows)
    return fail(MTP_ERR_UNSUPPORTED, "kv_beam_reorder: 1..64 beams a prompt, 1..1024 in all");
  if (C->n_layers < 1 || C->n_layers > 4096 || C->n_kv_heads < 1 || C->n_kv_heads > 64)
    return fail(MTP_ERR_UNSUPPORTED, "kv_beam_reorder: 1..4096 layers, 1..64 KV heads");
  if (C->head_dim_qk < 4 || C->head_dim_qk % 4 || C->head_dim_qk > 256 || C->head_dim_v < 4 ||
      C->head_dim_v % 4 || C->head_dim_v > 256)
    return fail(MTP_ERR_UNSUPPORTED, "kv_beam_reorder: head dims must be multiples of 4, <= 256");
  if (max_len < 0 || C->cache_cap < 1) return fail(MTP_ERR_INVALID_ARG, "kv_beam_reorder: bad length");
  if (max_len > C->cache_cap)
    return fail(MTP_ERR_CAPACITY, "kv_beam_reorder: max_len exceeds the tails' capacity");
  for (int l = 0; l < C->n_layers; ++l)
    if (!C->h_k[l] || !C->h_v[l] || !aligned16(C->h_k[l]) || !aligned16(C->h_v[l]))
      return fail(MTP_ERR_INVALID_ARG, "kv_beam_reorder: null or misaligned tails");
  if (!aligned4(d_parent) || !aligned4(d_len)) return fail(MTP_ERR_INVALID_ARG, "kv_beam_reorder: misaligned pointer");
  if (!d_ws || !aligned16(d_ws) || ws_bytes < kv_beam_workspace_bytes())
    return fail(MTP_ERR_WORKSPACE, "kv_beam_reorder: workspace too small or misaligned");
  if (max_len == 0) return MTP_OK;
  MoveArgs a = {};
  a.parent = d_parent;
  a.len = d_len;
  a.seqs = n_seqs;
  a.beams = beams;
  a.nkv = C->n_kv_heads;
  a.dqk = C->head_dim_qk;
  a.dv = C->head_dim_v;
  a.most = max_len;
  const MovePlan plan = move_plan(beams, std::max(a.dqk, a.dv), (int64_t)n_seqs * 2 * a.nkv * C->n_layers, max_len, sm_count());
  a.shift = plan.shift;
  a.rows = plan.rows;
  if (plan.tiles * n_seqs > 0x7FFFFFFF)
    return fail(MTP_ERR_UNSUPPORTED, "kv_beam_reorder: more than 2^31 tiles of rows");
  a.tiles = (int)plan.tiles;
  a.cap = C->cache_cap;
  a.err = &static_cast<WsHeader*>(d_ws)->err;
  for (int l0 = 0; l0 < C->n_layers; l0 += kMoveLayers) {
    const int nl = std::min(kMoveLayers, C->n_layers - l0);
    for (int l = 0; l < nl; ++l) {
      a.k[l] = C->h_k[l0 + l];
      a.v[l] = C->h_v[l0 + l];
    }
    cudaError_t e = launch_pdl(kv_beam_kernel, dim3((unsigned)a.tiles * n_seqs, 2 * a.nkv, nl), kMoveThreads, 0,
                               static_cast<cudaStream_t>(stream), a);
    if (e != cudaSuccess) return cuda_fail(e, "kv_beam_reorder launch");
  }
  return MTP_OK;
}

}  // extern "C"
