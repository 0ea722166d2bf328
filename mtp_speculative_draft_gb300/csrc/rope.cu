// Per-head RMSNorm and rotary positions on several axes (time, height,
// width), for rows of query and key heads.
//
// "hf2q 0.1.13 src/inference/models/qwen35/mtp.rs", apply_imrope: several
// position ids a token, mrope_section pairs of each axis dealt in turn.  Pair
// (i, i + rot/2) of a head turns by the angle of pair i at the position that
// its axis has for the row; the angles come from the table of mtp_rope_table.
#include "tree.cuh"

namespace mtp {

struct RopeRowsArgs {
  mtp_head_rows t[4];
  int head_end[4];  // running sum of the tensors' heads
  int nt;
  int d;
  int rows;
  float eps;
  RopePos r;
  int* err;
};

constexpr int kRopeThreads = 256;

// grid (rows, head groups): one warp per head row.
__global__ void __launch_bounds__(kRopeThreads) rope_rows_kernel(const RopeRowsArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x;
  const int heads = a.head_end[a.nt - 1];
  for (int h = blockIdx.y * (kRopeThreads / 32) + (threadIdx.x >> 5); h < heads;
       h += gridDim.y * (kRopeThreads / 32)) {
    int ti = 0;
    while (h >= a.head_end[ti]) ++ti;
    const mtp_head_rows& t = a.t[ti];
    const int hh = h - (ti ? a.head_end[ti - 1] : 0);
    HeadVals v;
    head_norm_rope(v, t.x + (size_t)row * t.x_ld + (size_t)hh * t.x_hs, a.d, t.norm_w, a.eps, a.r,
                   row, a.err, lane);
    head_store(v, t.y + (size_t)row * t.y_ld + (size_t)hh * t.y_hs, a.d, a.r.half, 1.f, lane);
  }
}

mtp_status fill_rope_axes(RopePos* out, const mtp_rope_axes* ax, int half, int rows,
                          const char* who) {
  const std::string w(who);
  if (!ax) return fail(MTP_ERR_INVALID_ARG, w + ": null rotary axes");
  if (!ax->d_pos || !ax->d_rope) return fail(MTP_ERR_INVALID_ARG, w + ": null positions or rotary table");
  if ((reinterpret_cast<uintptr_t>(ax->d_rope) & 15) || (reinterpret_cast<uintptr_t>(ax->d_pos) & 3))
    return fail(MTP_ERR_INVALID_ARG, w + ": rotary table or positions misaligned");
  if (ax->n_axes < 1 || ax->n_axes > 4)
    return fail(MTP_ERR_UNSUPPORTED, w + ": rotary axes must be 1..4");
  if (ax->max_pos < 1 || ax->pos_ld < rows)
    return fail(MTP_ERR_INVALID_ARG, w + ": max_pos < 1 or fewer positions than rows");
  if (ax->interleaved != 0 && ax->interleaved != 1)
    return fail(MTP_ERR_INVALID_ARG, w + ": interleaved must be 0 or 1");
  int64_t sum = 0;
  for (int a = 0; a < ax->n_axes; ++a) {
    if (ax->section[a] < 0 || ax->section[a] > 128)
      return fail(MTP_ERR_INVALID_ARG, w + ": sections must hold 0..128 rotary pairs");
    sum += ax->section[a];
  }
  if (sum < 1 || sum > 128 || (half >= 0 && sum != half))
    return fail(MTP_ERR_INVALID_ARG, w + ": the sections' pairs must add up to rot_dim / 2");
  if (ax->interleaved)
    for (int a = 1; a < ax->n_axes; ++a)
      if (ax->section[a] > 0 && a + (int64_t)ax->n_axes * (ax->section[a] - 1) >= sum)
        return fail(MTP_ERR_INVALID_ARG,
                    w + ": a section has more pairs than its turns in rot_dim / 2 pairs");
  *out = RopePos{};
  out->table = ax->d_rope;
  out->pos = ax->d_pos;
  out->pos_ld = ax->pos_ld;
  out->max_pos = ax->max_pos;
  out->n_axes = ax->n_axes;
  for (int a = 0; a < ax->n_axes; ++a) out->sec[a] = ax->section[a];
  out->inter = ax->interleaved;
  out->half = (int)sum;
  return MTP_OK;
}

}  // namespace mtp

using namespace mtp;

extern "C" {

size_t rope_axes_rows_workspace_bytes(void) { return sizeof(WsHeader); }

mtp_status rope_axes_rows(const mtp_rope_axes* axes, const mtp_head_rows* t, int32_t n_t,
                          int32_t rows, int32_t head_dim, float eps, void* d_ws, size_t ws_bytes,
                          void* stream) {
  if (rows < 1) return fail(MTP_ERR_INVALID_ARG, "rope_axes_rows: rows must be >= 1");
  if (head_dim < 32 || head_dim > 256 || head_dim % 32)
    return fail(MTP_ERR_UNSUPPORTED, "rope_axes_rows: head_dim must be a multiple of 32, <= 256");
  if (!t || n_t < 1 || n_t > 4) return fail(MTP_ERR_INVALID_ARG, "rope_axes_rows: 1..4 tensors");
  if (!(eps >= 0.f)) return fail(MTP_ERR_INVALID_ARG, "rope_axes_rows: eps must be >= 0");
  RopeRowsArgs a = {};
  mtp_status s = fill_rope_axes(&a.r, axes, -1, rows, "rope_axes_rows");
  if (s != MTP_OK) return s;
  if (2 * a.r.half > head_dim)
    return fail(MTP_ERR_INVALID_ARG, "rope_axes_rows: more rotary pairs than head_dim / 2");
  int heads = 0;
  for (int i = 0; i < n_t; ++i) {
    const mtp_head_rows& x = t[i];
    if (!x.x || !x.y) return fail(MTP_ERR_INVALID_ARG, "rope_axes_rows: null pointer");
    if (!aligned16(x.x) || !aligned16(x.y) || (x.norm_w && !aligned16(x.norm_w)))
      return fail(MTP_ERR_INVALID_ARG, "rope_axes_rows: pointers must be 16-byte aligned");
    if (x.n_heads < 1 || x.n_heads > 4096)
      return fail(MTP_ERR_UNSUPPORTED, "rope_axes_rows: 1..4096 heads a tensor");
    if (x.x_hs < head_dim || x.y_hs < head_dim || x.x_ld < (int64_t)(x.n_heads - 1) * x.x_hs + head_dim ||
        x.y_ld < (int64_t)(x.n_heads - 1) * x.y_hs + head_dim)
      return fail(MTP_ERR_INVALID_ARG, "rope_axes_rows: strides let heads or rows overlap");
    if (x.x_ld % 4 || x.y_ld % 4 || x.x_hs % 4 || x.y_hs % 4)
      return fail(MTP_ERR_INVALID_ARG, "rope_axes_rows: strides must be multiples of 4 floats");
    heads += x.n_heads;
    a.t[i] = x;
    a.head_end[i] = heads;
  }
  if (!d_ws || ws_bytes < rope_axes_rows_workspace_bytes())
    return fail(MTP_ERR_WORKSPACE, "rope_axes_rows: workspace too small");
  a.nt = n_t;
  a.d = head_dim;
  a.rows = rows;
  a.eps = eps;
  a.err = &static_cast<WsHeader*>(d_ws)->err;
  const int groups = (heads + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  cudaError_t e = launch_pdl(rope_rows_kernel, dim3(rows, groups < 64 ? groups : 64), kRopeThreads,
                             0, static_cast<cudaStream_t>(stream), a);
  if (e != cudaSuccess) return cuda_fail(e, "rope_axes_rows launch");
  return MTP_OK;
}

}  // extern "C"
