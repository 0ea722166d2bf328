// Shared pieces of the draft-tree operators: rotary positions on several
// axes, the per-head norm and rotation of one row, bounds of a tree.
#pragma once

#include "host.h"

namespace mtp {

constexpr int kTreeMax = 64;  // nodes of a tree: one 64-bit ancestor word per node
// Behind a workspace's header the joins of logit_rules_argmax, a 64-bit key and a 32-bit counter a row, which are
// zero between calls.  Other calls of a round that use a workspace's body start behind them, so one workspace
// serves them all in turn.
constexpr int kRuleRowsMax = 1024;
constexpr size_t kRuleJoinBytes = (size_t)kRuleRowsMax * 16;

// Device error codes of these operators (after the ones in common.cuh).
enum TreeErr : int {
  kErrBadTree = 5,      // a parent, depth or path entry outside its range
  kErrBadPosition = 6,  // a rotary position outside the table (position 0 was used)
};

// Rotary positions of `rows` rows.  Pair i of a row takes its angle from the
// table row pos[axis(i)][row].  pos == nullptr: every pair of row r sits at
// base + depth[r].
struct RopePos {
  const float* table;  // [max_pos][half][2] cos, sin
  const int* pos;      // [n_axes][pos_ld] or null
  const int* depth;    // [rows], used when pos is null (values checked by the caller's kernel)
  int base;
  int pos_ld;
  int max_pos;
  int n_axes;
  int sec[4];
  int inter;
  int half;
};

// Axis of rotary pair i: sections one after another, or dealt in turn (pair i
// goes to axis i mod n while that axis has pairs left, else to axis 0).
__device__ __forceinline__ int rope_axis(const RopePos& r, int i) {
  if (r.n_axes == 1) return 0;
  if (r.inter) {
    const int a = i % r.n_axes;
    return a != 0 && i < r.n_axes * r.sec[a] ? a : 0;
  }
  int a = 0, end = r.sec[0];
  while (a < r.n_axes - 1 && i >= end) end += r.sec[++a];
  return a;
}

// Table entry (cos, sin) of pair i of row `row`.
__device__ __forceinline__ float2 rope_entry(const RopePos& r, int row, int i, int* err) {
  int p = r.pos ? r.pos[(size_t)rope_axis(r, i) * r.pos_ld + row] : r.base + r.depth[row];
  if (p < 0 || p >= r.max_pos) {
    set_dev_error(err, kErrBadPosition);
    p = 0;
  }
  return *reinterpret_cast<const float2*>(r.table + 2 * ((size_t)p * r.half + i));
}

// One head row of d <= 256 values held by a warp: lane l has pairs
// (i, i + half) for i = l + 32 j in a[j], b[j] and the values past the
// rotated ones, rot + l + 32 j, in c[j].
struct HeadVals {
  float a[4], b[4], c[8];
};

// The values of a head row, or of a norm weight (1 when null), in that layout.
__device__ __forceinline__ void head_load(HeadVals& h, const float* src, int d, int half, int lane) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int i = lane + 32 * j;
    const bool in = i < half;
    h.a[j] = src ? (in ? src[i] : 0.f) : 1.f;
    h.b[j] = src ? (in ? src[i + half] : 0.f) : 1.f;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int i = 2 * half + lane + 32 * j;
    h.c[j] = src ? (i < d ? src[i] : 0.f) : 1.f;
  }
}

// RMS-normalises a loaded head row (with its loaded weight, when norm) and
// rotates its pairs.
__device__ __forceinline__ void head_norm_rope(HeadVals& h, const HeadVals& w, bool norm, int d, float eps,
                                               const RopePos& r, int row, int* err, int lane) {
  float2 cs[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    cs[j] = lane + 32 * j < r.half ? rope_entry(r, row, lane + 32 * j, err) : make_float2(1.f, 0.f);
  if (norm) {
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) ss += h.a[j] * h.a[j] + h.b[j] * h.b[j];
#pragma unroll
    for (int j = 0; j < 8; ++j) ss += h.c[j] * h.c[j];
    const float inv = rsqrtf(warp_sum(ss) / (float)d + eps);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h.a[j] = h.a[j] * inv * w.a[j];
      h.b[j] = h.b[j] * inv * w.b[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) h.c[j] = h.c[j] * inv * w.c[j];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float a = h.a[j], b = h.b[j];
    h.a[j] = a * cs[j].x - b * cs[j].y;
    h.b[j] = a * cs[j].y + b * cs[j].x;
  }
}

__device__ __forceinline__ void head_store(const HeadVals& h, float* dst, int d, int half,
                                           float mul, int lane) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int i = lane + 32 * j;
    if (i < half) {
      dst[i] = h.a[j] * mul;
      dst[i + half] = h.b[j] * mul;
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int i = 2 * half + lane + 32 * j;
    if (i < d) dst[i] = h.c[j] * mul;
  }
}

// Host side: checks an axes descriptor for `half` rotary pairs (half < 0: any)
// and `rows` rows and fills the device view.
mtp_status fill_rope_axes(RopePos* out, const mtp_rope_axes* ax, int half, int rows,
                          const char* who);

// One launch with programmatic dependent launch, marked for timing sessions.
template <class... P, class... A>
cudaError_t launch_pdl(void (*k)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                       A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  launch_mark(st);
  return cudaLaunchKernelEx(&cfg, k, static_cast<P>(args)...);
}

}  // namespace mtp
