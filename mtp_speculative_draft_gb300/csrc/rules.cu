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
#include <cmath>

#include "tree.cuh"

namespace mtp {

constexpr int kRuleThreads = 256;
constexpr int kRulePer = 8;                          // tokens a thread of a chunk
constexpr int kRuleChunk = kRuleThreads * kRulePer;  // tokens a CTA

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

// grid (chunks, row groups).  The CTA's chunk of the biases and of the count
// table is gathered once for its rows.
__global__ void __launch_bounds__(kRuleThreads) logit_rules_kernel(const RuleArgs a) {
  __shared__ float adj[kRuleChunk];
  __shared__ unsigned long long extra[kRuleChunk];  // which path nodes hold the token
  __shared__ unsigned long long red[kRuleThreads / 32];
  __shared__ int any_path;
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int v0 = blockIdx.x * kRuleChunk;
  for (int i = tid; i < kRuleChunk; i += kRuleThreads) {
    adj[i] = 0.f;
    extra[i] = 0ull;
  }
  if (tid == 0) any_path = 0;
  __syncthreads();
  // path tokens of the chunk: node j sets bit j of its token's word
  if (tid < a.n_path) {
    const int t = a.path_tok[tid] - v0;
    if (t >= 0 && t < kRuleChunk) {
      atomicOr(&extra[t], 1ull << tid);
      any_path = 1;
    }
  }
  // biases of the chunk in list order: hits are added one after another
  if (warp == kRuleThreads / 32 - 1) {
    for (int i0 = 0; i0 < a.n_bias; i0 += 32) {
      const int i = i0 + lane;
      const int t = i < a.n_bias ? a.bias_tok[i] - v0 : -1;
      unsigned hit = __ballot_sync(0xffffffffu, t >= 0 && t < kRuleChunk);
      const float b = t >= 0 && t < kRuleChunk ? a.bias[i] : 0.f;
      while (hit) {
        const int l = __ffs(hit) - 1;
        hit &= hit - 1;
        if (lane == l) adj[t] += b;
        __syncwarp();
      }
    }
  }
  uint32_t cw[kRulePer];
#pragma unroll
  for (int k = 0; k < kRulePer; ++k) {
    const int v = v0 + tid + k * kRuleThreads;
    cw[k] = a.counts && v < a.V ? a.counts[v] : 0u;
  }
  __syncthreads();
  const bool path = any_path != 0;
  const int r1 = min(a.rows, ((int)blockIdx.y + 1) * a.rows_per_cta);
  for (int r = blockIdx.y * a.rows_per_cta; r < r1; ++r) {
    const float* x = a.x + (size_t)r * a.ld;
    float l[kRulePer];
#pragma unroll
    for (int k = 0; k < kRulePer; ++k) {
      const int v = v0 + tid + k * kRuleThreads;
      l[k] = v < a.V ? x[v] : -INFINITY;
    }
    const unsigned long long pm = path ? a.path_mask[r] : 0ull;
    float best = -INFINITY;
    int at = -1;
#pragma unroll
    for (int k = 0; k < kRulePer; ++k) {
      const int i = tid + k * kRuleThreads, v = v0 + i;
      if (v >= a.V) continue;
      float t = l[k];
      uint32_t w = cw[k];
      if (path) w += __popcll(extra[i] & pm);
      if (w) {
        const uint32_t c = w & 0x7FFFFFFFu;
        t = t > 0.f ? __fdiv_rn(t, a.rep) : __fmul_rn(t, a.rep);
        t = __fsub_rn(t, __fadd_rn(__fmul_rn((float)c, a.freq), c ? a.pres : 0.f));
      }
      const float b = adj[i];
      if (b != 0.f) t = __fadd_rn(t, b);
      if (a.allow && !((a.allow[(size_t)r * a.allow_ld + (v >> 5)] >> (v & 31)) & 1u)) t = -INFINITY;
      if (a.y) a.y[(size_t)r * a.ldy + v] = t;
      if (t > best) {
        best = t;
        at = v;
      }
    }
    // a zero's sign does not order it; v + 0 makes -0 equal +0
    unsigned long long key = at < 0 ? 0ull : argmax_key(best + 0.f, at);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long other = __shfl_xor_sync(0xffffffffu, key, o);
      key = other > key ? other : key;
    }
    if (lane == 0) red[warp] = key;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kRuleThreads / 32; ++w) key = red[w] > key ? red[w] : key;
      if (key) atomicMax(a.keys + r, key);
      __threadfence();
      if (atomicAdd(a.cnt + r, 1u) == gridDim.x - 1) {  // every chunk of the row has merged
        __threadfence();
        const unsigned long long best_key = atomicMax(a.keys + r, 0ull);
        a.tok[r] = best_key ? argmax_key_index(best_key) : -1;
        a.val[r] = best_key ? argmax_key_value(best_key) : -INFINITY;
        a.keys[r] = 0ull;  // leave the workspace cleared for the next call
        a.cnt[r] = 0u;
      }
    }
    __syncthreads();
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
  if (rows < 1 || rows > 1024) return 0;
  return sizeof(WsHeader) + (size_t)rows * 16 + 256;
}

mtp_status logit_rules_argmax(const mtp_logit_rules* R, const float* d_logits, int64_t ld,
                              int32_t rows, int32_t* d_tokens, float* d_values, float* d_out,
                              int64_t ld_out, void* d_ws, size_t ws_bytes, void* stream) {
  if (!R || !d_logits || !d_tokens || !d_values)
    return fail(MTP_ERR_INVALID_ARG, "logit_rules_argmax: null pointer");
  if (rows < 1 || rows > 1024)
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
  if ((reinterpret_cast<uintptr_t>(d_logits) | reinterpret_cast<uintptr_t>(d_out) |
       reinterpret_cast<uintptr_t>(R->d_counts) | reinterpret_cast<uintptr_t>(R->d_allow)) & 15 ||
      (reinterpret_cast<uintptr_t>(R->d_path_mask) & 7) ||
      ((reinterpret_cast<uintptr_t>(R->d_path_tokens) | reinterpret_cast<uintptr_t>(R->d_bias_tokens) |
        reinterpret_cast<uintptr_t>(R->d_bias) | reinterpret_cast<uintptr_t>(d_tokens) |
        reinterpret_cast<uintptr_t>(d_values)) & 3))
    return fail(MTP_ERR_INVALID_ARG, "logit_rules_argmax: misaligned pointer");
  if (!d_ws || !aligned16(d_ws) || ws_bytes < logit_rules_argmax_workspace_bytes(rows))
    return fail(MTP_ERR_WORKSPACE, "logit_rules_argmax: workspace too small");
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
  a.rows_per_cta = 1;
  const int chunks = (R->vocab + kRuleChunk - 1) / kRuleChunk;
  cudaError_t e = launch_pdl(logit_rules_kernel, dim3(chunks, rows), kRuleThreads, 0,
                             static_cast<cudaStream_t>(stream), a);
  if (e != cudaSuccess) return cuda_fail(e, "logit_rules_argmax launch");
  return MTP_OK;
}

mtp_status mtp_token_counts(uint32_t* d_counts, int32_t vocab, const int32_t* d_tokens, int32_t n,
                            int32_t prompt, void* d_ws, size_t ws_bytes, void* stream) {
  if (!d_counts || !d_tokens) return fail(MTP_ERR_INVALID_ARG, "mtp_token_counts: null pointer");
  if (((reinterpret_cast<uintptr_t>(d_counts)) & 15) || (reinterpret_cast<uintptr_t>(d_tokens) & 3))
    return fail(MTP_ERR_INVALID_ARG, "mtp_token_counts: misaligned pointer");
  if (vocab < 1 || n < 1 || (prompt != 0 && prompt != 1))
    return fail(MTP_ERR_INVALID_ARG, "mtp_token_counts: vocab and n must be >= 1, prompt 0 or 1");
  if (!d_ws || ws_bytes < sizeof(WsHeader))
    return fail(MTP_ERR_WORKSPACE, "mtp_token_counts: workspace too small");
  cudaError_t e = launch_pdl(token_counts_kernel, dim3((n + 255) / 256), 256, 0,
                             static_cast<cudaStream_t>(stream), d_counts, vocab, d_tokens, n, prompt,
                             &static_cast<WsHeader*>(d_ws)->err);
  if (e != cudaSuccess) return cuda_fail(e, "mtp_token_counts launch");
  return MTP_OK;
}

}  // extern "C"
