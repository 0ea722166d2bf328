// A request's rules on logits, and each row's argmax: penalties for repeated
// tokens, additive biases and a grammar's mask, in this order.
//
// For row r and token v, with c the times v was generated (count table) plus
// its occurrences on the row's path in the draft tree, and `seen` when v is in
// the count table's prompt or c > 0:
//   l <- seen ? (l > 0 ? l / repetition : l * repetition) : l
//   l <- l - (frequency * c + presence * [c > 0])
//   l <- l + sum of v's bias entries (in list order)
//   l <- -inf where the row's mask bit of v is 0
// Every step rounds once to float32, so equal inputs give equal outputs bit
// for bit; the argmax takes the lowest index among equal values and -1 where
// nothing is above -inf (NaN never wins).
#include <algorithm>
#include <cmath>

#include "tree.cuh"

namespace mtp {

constexpr int kRuleThreads = 256;
constexpr int kRulePer = 8;                          // tokens a thread of a chunk
constexpr int kRuleChunk = kRuleThreads * kRulePer;  // tokens a CTA
// CTAs a SM at which a CTA takes further rows: fewer repeat the list building
// less, more hide the row loop's waits better (64 x 152577: 3 gave 32 us, 2 gave
// 38, 5 gave 36, one row a CTA 39; 16 x 151936: 13 us against 13, 16 and 16; with
// the mask words handed over too, 3 gives 30 us).
constexpr int kRuleCtas = 3;
// Bias entries of a chunk kept at hand.  With more, each biased token of the chunk scans the whole list: 64 rows
// of 151936 tokens take 27, 29 and 43 us with 300, 1000 and 5000 entries, and 1.8, 5.9 and 22 ms with 10000, 30000
// and 65536 (the torch form: 0.65 ms whatever the list).
constexpr int kRuleHits = 128;
constexpr int kRuleRows = 16;                        // rows a CTA, at most

struct RuleArgs {
  const float* x;
  long long ld;
  float* y;  // or null
  long long ldy;
  int rows, V;
  int rows_per_cta;
  float rep, freq, pres;
  const uint32_t* counts;  // or null
  const int* bias_tok;
  const float* bias;
  int n_bias;
  const uint32_t* allow;  // or null
  int allow_ld;
  const int* path_tok;
  const unsigned long long* path_mask;
  int n_path;
  int* tok;
  float* val;
  unsigned long long* keys;  // [rows], zero at rest
  unsigned* cnt;             // [rows], zero at rest
};

// grid (chunks, row groups).  Few tokens have a count, a bias or a place on a
// path.  A CTA lists its chunk's once for all its rows; a row's listed tokens go
// to as many threads as there are (a division for one lane holds up its warp),
// the rest need the mask and the maximum alone.  The rows' argmax joins the other
// chunks' at the end, a thread a row.  Bound by HBM on many rows (the logits read
// and written once) and by a few dependent reads on few; the code before the row
// loop is rolled up, as a CTA runs it once and fetches its instructions from L2.
__global__ void __launch_bounds__(kRuleThreads, 4) logit_rules_kernel(const __grid_constant__ RuleArgs a) {
  constexpr int kWarps = kRuleThreads / 32;
  __shared__ uint32_t biased[kRuleChunk / 32], on_path[kRuleChunk / 32];  // a bit a token
  __shared__ uint16_t list[kRuleChunk];               // the listed tokens, their count words, summed
  __shared__ uint32_t cnt[kRuleChunk];                // biases and path nodes
  __shared__ float adj[kRuleChunk];
  __shared__ uint8_t slot[kRuleChunk];                // first path node of the token, or kTreeMax
  __shared__ unsigned long long nodes[kTreeMax + 1];  // the nodes of a slot's token
  __shared__ float hand[2][kRuleChunk];               // their logits of a row and the next
  __shared__ uint32_t words[2][kRuleChunk / 32];      // and the mask words
  __shared__ int ptok[kTreeMax];
  __shared__ int hit_i[kRuleHits], hit_t[kRuleHits];  // bias entries of the chunk, in any order
  __shared__ float hit_b[kRuleHits];
  __shared__ unsigned long long best[kRuleRows][kWarps];
  __shared__ int nlist, nhits;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int v0 = blockIdx.x * kRuleChunk;
  const int row0 = blockIdx.y * a.rows_per_cta, nrows = min(a.rows - row0, a.rows_per_cta);
  if (tid < kRuleChunk / 32) biased[tid] = on_path[tid] = 0u;
  if (tid == 0) {
    nlist = nhits = 0;
    nodes[kTreeMax] = 0ull;
  }
  pdl_wait();
  pdl_launch_dependents();
  uint32_t cw[kRulePer];
#pragma unroll
  for (int k = 0; k < kRulePer; ++k) {
    const int v = v0 + tid + k * kRuleThreads;
    cw[k] = a.counts && v < a.V ? a.counts[v] : 0u;
  }
  float l[kRulePer];
  uint32_t w[kRulePer];
  unsigned long long pm = 0ull;
  // a row's logits, mask words (one a warp and word) and path
  auto load = [&](int r) {
    const float* src = a.x + (size_t)r * a.ld + v0 + tid;
    const uint32_t* ok = a.allow + (size_t)r * a.allow_ld + ((v0 + tid) >> 5);
#pragma unroll
    for (int k = 0; k < kRulePer; ++k) {
      const bool in = v0 + tid + k * kRuleThreads < a.V;
      l[k] = in ? src[k * kRuleThreads] : 0.f;
      w[k] = a.allow && in ? ok[k * kWarps] : 0xFFFFFFFFu;
    }
    pm = a.n_path ? a.path_mask[r] : 0ull;
  };
  load(row0);
  const int pt = tid < a.n_path ? a.path_tok[tid] : 0;
  int bt = tid < a.n_bias ? a.bias_tok[tid] : 0;
  float bv = tid < a.n_bias ? a.bias[tid] : 0.f;
  __syncthreads();
  if (tid < a.n_path) {
    const int t = pt - v0;
    ptok[tid] = t;
    if (t >= 0 && t < kRuleChunk) atomicOr(&on_path[t >> 5], 1u << (t & 31));
  }
#pragma unroll 1
  for (int i = tid; i < a.n_bias; i += kRuleThreads) {
    const int t = bt - v0;
    const float b = bv;
    if (i + kRuleThreads < a.n_bias) {
      bt = a.bias_tok[i + kRuleThreads];
      bv = a.bias[i + kRuleThreads];
    }
    if (t >= 0 && t < kRuleChunk) {
      atomicOr(&biased[t >> 5], 1u << (t & 31));
      const int at = atomicAdd(&nhits, 1);
      if (at < kRuleHits) {
        hit_i[at] = i;
        hit_t[at] = t;
        hit_b[at] = b;
      }
    }
  }
  __syncthreads();
  const uint32_t bit = 1u << lane;  // a word holds the 32 tokens of a warp
  unsigned listed = 0;  // bit k: this thread's token k is listed (or past the vocabulary)
  unsigned marks = 0;
#pragma unroll
  for (int k = 0; k < kRulePer; ++k) {
    const int i = tid + k * kRuleThreads;
    if (cw[k] || (biased[i >> 5] | on_path[i >> 5]) & bit) marks |= 1u << k;
    if (v0 + i >= a.V) listed |= 1u << k;
  }
  listed |= marks;
  {
    const int mine = __popc(marks);
    int at = mine;  // inclusive sum over the warp's lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) at += x;
    }
    int base = 0;
    if (lane == 31 && at > 0) base = atomicAdd(&nlist, at);
    at += __shfl_sync(0xffffffffu, base, 31) - mine;
#pragma unroll
    for (int k = 0; k < kRulePer; ++k)
      if ((marks >> k) & 1u) {
        list[at] = (uint16_t)(tid + k * kRuleThreads);
        cnt[at++] = cw[k];
      }
  }
  __syncthreads();
#pragma unroll 1
  for (int e = tid; e < nlist; e += kRuleThreads) {
    const int t = list[e];
    int first = kTreeMax;
    if ((on_path[t >> 5] >> (t & 31)) & 1u) {
      unsigned long long m = 0ull;
#pragma unroll 1
      for (int x = a.n_path - 1; x >= 0; --x)
        if (ptok[x] == t) {
          m |= 1ull << x;
          first = x;
        }
      nodes[first] = m;
    }
    slot[e] = (uint8_t)first;
    // the token's biases in list order: the next entry after the last one taken
    float sum = 0.f;
    if (!((biased[t >> 5] >> (t & 31)) & 1u)) {
    } else if (nhits <= kRuleHits) {
#pragma unroll 1
      for (int last = -1;;) {
        int next = a.n_bias, at = 0;
#pragma unroll 1
        for (int x = 0; x < nhits; ++x)
          if (hit_t[x] == t && hit_i[x] > last && hit_i[x] < next) {
            next = hit_i[x];
            at = x;
          }
        if (next == a.n_bias) break;
        sum += hit_b[at];
        last = next;
      }
    } else {
#pragma unroll 1
      for (int i = 0; i < a.n_bias; ++i)
        if (a.bias_tok[i] - v0 == t) sum += a.bias[i];
    }
    adj[e] = sum;
  }
  __syncthreads();
  const int nl = nlist;
  float* y = a.y ? a.y + (size_t)row0 * a.ldy + v0 : nullptr;
#pragma unroll 1
  for (int q = 0; q < nrows; ++q) {
    const int r = row0 + q;
    float top = -INFINITY;
    int at = 0x7FFFFFFF;
    // listed tokens to the threads that serve them, the others here
    float* xs = hand[q & 1];
    uint32_t* ok = words[q & 1];
#pragma unroll
    for (int k = 0; k < kRulePer; ++k) {
      const int i = tid + k * kRuleThreads;
      if (lane == 0) ok[i >> 5] = w[k];
      if ((listed >> k) & 1u) {
        xs[i] = l[k];
        continue;
      }
      const float t = w[k] & bit ? l[k] : -INFINITY;
      if (y) y[i] = t;
      if (t > top) {
        top = t;
        at = v0 + i;
      }
    }
    const unsigned long long path = pm;
    if (q + 1 < nrows) load(r + 1);  // on its way while the listed tokens are served
    if (nl > 0) __syncthreads();
#pragma unroll 1
    for (int e = tid; e < nl; e += kRuleThreads) {
      const int i = list[e], v = v0 + i;
      if (v >= a.V) continue;
      float t = xs[i];
      const uint32_t word = cnt[e], c = (word & 0x7FFFFFFFu) + __popcll(nodes[slot[e]] & path);  // up to 2^31 + 63
      if (word | c) {  // seen
        t = t > 0.f ? __fdiv_rn(t, a.rep) : __fmul_rn(t, a.rep);
        t = __fsub_rn(t, __fadd_rn(__fmul_rn((float)c, a.freq), c ? a.pres : 0.f));
      }
      const float b = adj[e];
      if (b != 0.f) t = __fadd_rn(t, b);
      if (!((ok[i >> 5] >> (i & 31)) & 1u)) t = -INFINITY;
      if (y) y[i] = t;
      if (t > top || (t == top && t > -INFINITY && v < at)) {
        top = t;
        at = v;
      }
    }
    if (y) y += a.ldy;
    // the warp's largest value, then the lowest index that has it; + 0 makes -0
    // equal +0 (a zero's sign does not order it)
    const uint32_t u = (uint32_t)(argmax_key(top + 0.f, 0) >> 32);
    const uint32_t most = __reduce_max_sync(0xffffffffu, u);
    const int lowest = __reduce_min_sync(0xffffffffu, u == most ? at : 0x7FFFFFFF);
    if (lane == 0)
      best[q][warp] = lowest == 0x7FFFFFFF ? 0ull
                                           : (unsigned long long)most << 32 | (0xFFFFFFFFu - (uint32_t)lowest);
  }
  __syncthreads();
  if (tid < nrows) {
    const int r = row0 + tid;
    unsigned long long key = best[tid][0];
#pragma unroll
    for (int x = 1; x < kWarps; ++x) key = best[tid][x] > key ? best[tid][x] : key;
    if (gridDim.x > 1) {
      if (key) atomicMax(a.keys + r, key);
      __threadfence();
      if (atomicAdd(a.cnt + r, 1u) != gridDim.x - 1) return;
      __threadfence();  // every chunk of the row has merged
      key = atomicMax(a.keys + r, 0ull);
      a.keys[r] = 0ull;  // leave the workspace cleared for the next call
      a.cnt[r] = 0u;
    }
    a.tok[r] = key ? argmax_key_index(key) : -1;
    a.val[r] = key ? argmax_key_value(key) : -INFINITY;
  }
}

// Adds a list of token ids to the count table.
__global__ void __launch_bounds__(256)
    token_counts_kernel(uint32_t* counts, int V, const int* tok, int n, int prompt, int* err) {
  pdl_wait();
  pdl_launch_dependents();
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const int t = tok[i];
  if (t < 0) return;
  if (t >= V) {
    set_dev_error(err, kErrBadToken);
    return;
  }
  if (prompt)
    atomicOr(counts + t, 0x80000000u);
  else
    atomicAdd(counts + t, 1u);
}

}  // namespace mtp

using namespace mtp;

extern "C" {

size_t logit_rules_argmax_workspace_bytes(int32_t rows) {
  if (rows < 1 || rows > kRuleRowsMax) return 0;
  return sizeof(WsHeader) + (size_t)rows * 16 + 256;
}

mtp_status logit_rules_argmax(const mtp_logit_rules* R, const float* d_logits, int64_t ld,
                              int32_t rows, int32_t* d_tokens, float* d_values, float* d_out,
                              int64_t ld_out, void* d_ws, size_t ws_bytes, void* stream) {
  if (!R || !d_logits || !d_tokens || !d_values)
    return fail(MTP_ERR_INVALID_ARG, "logit_rules_argmax: null pointer");
  if (rows < 1 || rows > kRuleRowsMax)
    return fail(MTP_ERR_UNSUPPORTED, "logit_rules_argmax: rows must be in 1..1024");
  if (R->vocab < 1 || R->vocab > (1 << 28))
    return fail(MTP_ERR_UNSUPPORTED, "logit_rules_argmax: vocab must be in 1..2^28");
  if (ld < R->vocab || (d_out && ld_out < R->vocab))
    return fail(MTP_ERR_INVALID_ARG, "logit_rules_argmax: row stride below the vocabulary");
  if (d_out == d_logits && ld_out != ld)
    return fail(MTP_ERR_INVALID_ARG, "logit_rules_argmax: in place needs equal row strides");
  if (!(R->repetition > 0.f) || !std::isfinite(R->repetition) || !std::isfinite(R->frequency) ||
      !std::isfinite(R->presence))
    return fail(MTP_ERR_INVALID_ARG, "logit_rules_argmax: repetition must be > 0, penalties finite");
  if (R->n_bias < 0 || R->n_bias > 65536 || (R->n_bias > 0 && (!R->d_bias_tokens || !R->d_bias)))
    return fail(MTP_ERR_INVALID_ARG, "logit_rules_argmax: 0..65536 bias entries");
  if (R->n_path < 0 || R->n_path > kTreeMax || (R->n_path > 0 && (!R->d_path_tokens || !R->d_path_mask)))
    return fail(MTP_ERR_INVALID_ARG, "logit_rules_argmax: 0..64 path tokens");
  const int words = (R->vocab + 31) / 32;
  if (R->d_allow && R->allow_ld != 0 && R->allow_ld < words)
    return fail(MTP_ERR_INVALID_ARG, "logit_rules_argmax: mask rows shorter than the vocabulary");
  if ((reinterpret_cast<uintptr_t>(R->d_path_mask) & 7) ||
      ((reinterpret_cast<uintptr_t>(d_logits) | reinterpret_cast<uintptr_t>(d_out) |
        reinterpret_cast<uintptr_t>(R->d_counts) | reinterpret_cast<uintptr_t>(R->d_allow) |
        reinterpret_cast<uintptr_t>(R->d_path_tokens) | reinterpret_cast<uintptr_t>(R->d_bias_tokens) |
        reinterpret_cast<uintptr_t>(R->d_bias) | reinterpret_cast<uintptr_t>(d_tokens) |
        reinterpret_cast<uintptr_t>(d_values)) & 3))
    return fail(MTP_ERR_INVALID_ARG, "logit_rules_argmax: misaligned pointer");
  if (!d_ws || !aligned16(d_ws) || ws_bytes < logit_rules_argmax_workspace_bytes(rows))
    return fail(MTP_ERR_WORKSPACE, "logit_rules_argmax: workspace too small or misaligned");
  RuleArgs a = {};
  a.x = d_logits;
  a.ld = ld;
  a.y = d_out;
  a.ldy = ld_out;
  a.rows = rows;
  a.V = R->vocab;
  a.rep = R->repetition;
  a.freq = R->frequency;
  a.pres = R->presence;
  a.counts = R->d_counts;
  a.bias_tok = R->d_bias_tokens;
  a.bias = R->d_bias;
  a.n_bias = R->n_bias;
  a.allow = R->d_allow;
  a.allow_ld = R->allow_ld;
  a.path_tok = R->d_path_tokens;
  a.path_mask = reinterpret_cast<const unsigned long long*>(R->d_path_mask);
  a.n_path = R->n_path;
  a.tok = d_tokens;
  a.val = d_values;
  uint8_t* body = static_cast<uint8_t*>(d_ws) + sizeof(WsHeader);
  a.keys = reinterpret_cast<unsigned long long*>(body);
  a.cnt = reinterpret_cast<unsigned*>(body + (size_t)rows * 8);
  const int chunks = (R->vocab + kRuleChunk - 1) / kRuleChunk;
  a.rows_per_cta = std::min(kRuleRows, std::max(1, (int)((long long)chunks * rows / (sm_count() * kRuleCtas))));
  cudaError_t e = launch_pdl(logit_rules_kernel, dim3(chunks, (rows + a.rows_per_cta - 1) / a.rows_per_cta), kRuleThreads, 0,
                             static_cast<cudaStream_t>(stream), a);
  if (e != cudaSuccess) return cuda_fail(e, "logit_rules_argmax launch");
  return MTP_OK;
}

mtp_status mtp_token_counts(uint32_t* d_counts, int32_t vocab, const int32_t* d_tokens, int32_t n,
                            int32_t prompt, void* d_ws, size_t ws_bytes, void* stream) {
  if (!d_counts || !d_tokens) return fail(MTP_ERR_INVALID_ARG, "mtp_token_counts: null pointer");
  if ((reinterpret_cast<uintptr_t>(d_counts) | reinterpret_cast<uintptr_t>(d_tokens)) & 3)
    return fail(MTP_ERR_INVALID_ARG, "mtp_token_counts: misaligned pointer");
  if (vocab < 1 || n < 1 || (prompt != 0 && prompt != 1))
    return fail(MTP_ERR_INVALID_ARG, "mtp_token_counts: vocab and n must be >= 1, prompt 0 or 1");
  if (!d_ws || !aligned16(d_ws) || ws_bytes < sizeof(WsHeader))
    return fail(MTP_ERR_WORKSPACE, "mtp_token_counts: workspace too small or misaligned");
  cudaError_t e = launch_pdl(token_counts_kernel, dim3((n - 1) / 256 + 1), 256, 0,
                             static_cast<cudaStream_t>(stream), d_counts, vocab, d_tokens, n, prompt,
                             &static_cast<WsHeader*>(d_ws)->err);
  if (e != cudaSuccess) return cuda_fail(e, "mtp_token_counts launch");
  return MTP_OK;
}

}  // extern "C"
