// Arguments of the attention of sequences that share prompts (prefix.cu), and
// the keys that its split launch (treeattn.cu) takes.
#pragma once

#include "split.cuh"

namespace mtp {

constexpr int kErrBadLength = 7;  // a length of a batch outside its range (the nearest value was used)
constexpr int kPrefixRows = 16;   // new rows a sequence
constexpr int kPrefixSeqs = 1024;

// Query row ((b * m + i) * G + g) of prompt p and KV head h, b among the
// prompt's sequences, is row of "head" p * nkv + h in SplitArgs.
struct PrefixArgs : SplitArgs {
  int nh, nkv, G, m, groups, per, window, gated;
  int pmax, tmax;                // most rows of a prompt, of a tail
  float eps;
  const float *qp, *kp, *vp, *qn, *kn, *sinks;
  long long ldq, ldk, ldv;
  RopePos rope;
  float *kt, *vt;                // tails [seqs][nkv][tcap][dim]
  long long tcap;
  const int *plen, *tlen;
  float* out;
  float* qf;                     // [groups * nkv][R][dqk] scaled queries
  int mrows;                     // new rows of a CTA of the tail launch
  int items;                     // CTAs of a sequence's KV head: groups of new rows times blocks of query heads
  int parts, part_keys;          // parts of a sequence's own keys at most, keys of a part
  unsigned* tail_count;          // [seqs][nkv][items] parts that have arrived, zero at rest
  float2* tail_ml;               // [seqs][nkv][items][parts][rows] their states
  float* tail_o;                 // [seqs][nkv][items][parts][rows][dv]
};

__device__ __forceinline__ int prompt_len(const PrefixArgs& a, int p) {
  return a.pmax > 0 ? min(max(a.plen[p], 0), a.pmax) : 0;
}
__device__ __forceinline__ int tail_len(const PrefixArgs& a, int b) { return min(a.tlen[b], a.tmax); }

// First key of prompt p that every row of its sequences sees: row i of a tail of
// t rows sees keys above P + t + i - window.  Called by whole warps.
__device__ __forceinline__ int first_shared_key(const PrefixArgs& a, int p, int P) {
  if (a.window <= 0) return 0;
  int t = 0;
  for (int b = threadIdx.x & 31; b < a.per; b += 32) t = max(t, tail_len(a, p * a.per + b));
  const long long k = (long long)P + __reduce_max_sync(0xffffffffu, t) + a.m - a.window;
  return k <= 0 ? 0 : k < P ? (int)k : P;
}

// Keys [k0, k1) of a split.  The lengths were final before the call's first
// launch, which releases this one after its own wait.
__device__ __forceinline__ void split_keys(const PrefixArgs& a, int head, int sp, int& k0, int& k1) {
  const int p = head / a.nkv, P = prompt_len(a, p), first = first_shared_key(a, p, P);
  const int each = ((P - first + a.ns - 1) / a.ns + 15) / 16 * 16;
  k0 = (int)min((long long)P, first + (long long)sp * each);
  k1 = (int)min((long long)P, (long long)k0 + each);
}

// Keys of a tile of the split kernel, and its launch.
int split_tile_keys(int dqk, int dv);
cudaError_t launch_prefix_split(const PrefixArgs& a, cudaStream_t st);

}  // namespace mtp
