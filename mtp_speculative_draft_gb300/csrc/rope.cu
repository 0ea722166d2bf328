// Per-head RMSNorm and rotary positions on several axes (time, height,
// width), for rows of query and key heads.
//
// "hf2q 0.1.13 src/inference/models/qwen35/mtp.rs", apply_imrope: several
// position ids a token, mrope_section pairs of each axis dealt in turn.  Pair
// (i, i + rot/2) of a head turns by the angle of pair i at the position that
// its axis has for the row; the angles come from the table of mtp_rope_table.
#include <algorithm>

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

// Any even rotation: grid (head groups, rows), one warp per head row, 4-byte
// accesses and the table read anew for each head: 8192 rows of 40 + 8 heads of 128
// with 30, 37 and 50 pairs take 213, 242 and 248 us, three times the kernel below.
__global__ void __launch_bounds__(kRopeThreads) rope_rows_any_kernel(const __grid_constant__ RopeRowsArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int heads = a.head_end[a.nt - 1];
  const int h = blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
  if (h >= heads) return;
  int ti = 0;
  while (h >= a.head_end[ti]) ++ti;
  const mtp_head_rows& t = a.t[ti];
  const int hh = h - (ti ? a.head_end[ti - 1] : 0);
  for (int row = blockIdx.y; row < a.rows; row += gridDim.y) {
    HeadVals v, w;
    head_load(v, t.x + (size_t)row * t.x_ld + (size_t)hh * t.x_hs, a.d, a.r.half, lane);
    head_load(w, t.norm_w, a.d, a.r.half, lane);
    head_norm_rope(v, w, t.norm_w != nullptr, a.d, a.eps, a.r, row, a.err, lane);
    head_store(v, t.y + (size_t)row * t.y_ld + (size_t)hh * t.y_hs, a.d, a.r.half, 1.f, lane);
  }
}

// Rotations whose half is a multiple of 4 dims, in 16-byte words.  LP lanes a
// head row (d <= 8 LP), each with up to two units; a unit is a pair of words
// (dims 4u .. and half + 4u ..) while u < half / 4, else one word past the
// rotated dims.  A CTA takes one row (and some of its heads, when rows are few);
// a lane's units are the same in each of its heads, so it reads the table once a
// row and keeps the angles in registers.  Bound by HBM: each value is read and
// written once, and KH heads' loads go out before any arithmetic (8192 rows of
// 40 + 8 heads of 128: 69 us without the replay, 5.8 TB/s, 0.87 of a copy; one
// warp a head with 4-byte accesses: 210 us).  Unequal sizes: 48 heads are one step
// of 16 x 3; single rows spread their heads over CTAs.
template <int LP, int KH, bool TWO>
__global__ void __launch_bounds__(kRopeThreads) rope_rows_kernel(const __grid_constant__ RopeRowsArgs a) {
  constexpr int G = kRopeThreads / LP;  // heads of a step
  constexpr int NU = TWO ? 2 : 1;
  const int l = threadIdx.x % LP, g = threadIdx.x / LP;
  const int row = blockIdx.x, heads = a.head_end[a.nt - 1];
  const int half = a.r.half, pairs = half / 4, units = pairs + (a.d - 2 * half) / 4;
  pdl_wait();
  pdl_launch_dependents();
  float cs[NU][4], sn[NU][4];
  int c0[NU], c1[NU];  // the unit's first dims (c1 < 0: no second word, c0 < 0: no unit)
#pragma unroll
  for (int k = 0; k < NU; ++k) {
    const int u = l + k * LP;
    c0[k] = u < pairs ? 4 * u : u < units ? 2 * half + 4 * (u - pairs) : -1;
    c1[k] = u < pairs ? half + 4 * u : -1;
  }
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  float4 x[KH][NU], y[KH][NU];
  auto load = [&](int h0) {
#pragma unroll
    for (int i = 0; i < KH; ++i) {
      const int h = h0 + i * G + g;
      int ti = 0;
      while (ti < a.nt && h >= a.head_end[ti]) ++ti;
      const bool in = ti < a.nt;
      const mtp_head_rows& t = a.t[in ? ti : 0];
      const float* src = t.x + (size_t)row * t.x_ld + (size_t)(h - (ti ? a.head_end[ti - 1] : 0)) * t.x_hs;
#pragma unroll
      for (int k = 0; k < NU; ++k) {
        x[i][k] = in && c0[k] >= 0 ? *reinterpret_cast<const float4*>(src + c0[k]) : zero;
        y[i][k] = in && c1[k] >= 0 ? *reinterpret_cast<const float4*>(src + c1[k]) : zero;
      }
    }
  };
  load(blockIdx.y * G * KH);
#pragma unroll
  for (int k = 0; k < NU; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 e = c1[k] >= 0 ? rope_entry(a.r, row, 4 * (l + k * LP) + j, a.err) : make_float2(1.f, 0.f);
      cs[k][j] = e.x;
      sn[k][j] = e.y;
    }
#pragma unroll 1
  for (int h0 = blockIdx.y * G * KH; h0 < heads; h0 += gridDim.y * G * KH) {
    if (h0 != (int)blockIdx.y * G * KH) load(h0);
#pragma unroll
    for (int i = 0; i < KH; ++i) {
      const int h = h0 + i * G + g;
      int ti = 0;
      while (ti < a.nt && h >= a.head_end[ti]) ++ti;
      const bool in = ti < a.nt;
      const mtp_head_rows& t = a.t[in ? ti : 0];
      float inv = 1.f;
      float ss = 0.f;
#pragma unroll
      for (int k = 0; k < NU; ++k) {
        const float4 p = x[i][k], q = y[i][k];
        ss += p.x * p.x + p.y * p.y + p.z * p.z + p.w * p.w + q.x * q.x + q.y * q.y + q.z * q.z + q.w * q.w;
      }
#pragma unroll
      for (int o = LP / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (!in) continue;
      const float* w = t.norm_w;
      if (w) inv = rsqrtf(ss / (float)a.d + a.eps);
      float* dst = t.y + (size_t)row * t.y_ld + (size_t)(h - (ti ? a.head_end[ti - 1] : 0)) * t.y_hs;
#pragma unroll
      for (int k = 0; k < NU; ++k) {
        if (c0[k] < 0) continue;
        float p[4] = {x[i][k].x, x[i][k].y, x[i][k].z, x[i][k].w};
        float q[4] = {y[i][k].x, y[i][k].y, y[i][k].z, y[i][k].w};
        if (w) {
          const float4 wp = __ldg(reinterpret_cast<const float4*>(w + c0[k]));
          const float4 wq = c1[k] >= 0 ? __ldg(reinterpret_cast<const float4*>(w + c1[k])) : zero;
          const float vp[4] = {wp.x, wp.y, wp.z, wp.w}, vq[4] = {wq.x, wq.y, wq.z, wq.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            p[j] = p[j] * inv * vp[j];
            q[j] = q[j] * inv * vq[j];
          }
        }
        float4 r0, r1;
        r0.x = p[0] * cs[k][0] - q[0] * sn[k][0];
        r0.y = p[1] * cs[k][1] - q[1] * sn[k][1];
        r0.z = p[2] * cs[k][2] - q[2] * sn[k][2];
        r0.w = p[3] * cs[k][3] - q[3] * sn[k][3];
        r1.x = p[0] * sn[k][0] + q[0] * cs[k][0];
        r1.y = p[1] * sn[k][1] + q[1] * cs[k][1];
        r1.z = p[2] * sn[k][2] + q[2] * cs[k][2];
        r1.w = p[3] * sn[k][3] + q[3] * cs[k][3];
        *reinterpret_cast<float4*>(dst + c0[k]) = r0;
        if (c1[k] >= 0) *reinterpret_cast<float4*>(dst + c1[k]) = r1;
      }
    }
  }
}

template <int LP, int KH>
static cudaError_t launch_rope_rows(const RopeRowsArgs& a, cudaStream_t st) {
  const int heads = a.head_end[a.nt - 1], per = kRopeThreads / LP * KH;
  // few rows: their heads go to CTAs of their own
  int split = 1;
  while (split * per < heads && (long long)a.rows * split < sm_count()) ++split;
  const int units = a.r.half / 4 + (a.d - 2 * a.r.half) / 4;
  return launch_pdl(units > LP ? rope_rows_kernel<LP, KH, true> : rope_rows_kernel<LP, KH, false>,
                    dim3(a.rows, split), kRopeThreads, 0, st, a);
}

// Whether no two head rows share a value: a row's heads between two rows, or a
// head's rows between two heads.
static bool rows_apart(int64_t ld, int32_t hs, int rows, int heads, int d) {
  if (hs < d || ld < d) return false;
  return ld >= (int64_t)(heads - 1) * hs + d || rows == 1 || ld <= (hs - d) / (rows - 1);
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
    if (!rows_apart(x.x_ld, x.x_hs, rows, x.n_heads, head_dim) || !rows_apart(x.y_ld, x.y_hs, rows, x.n_heads, head_dim))
      return fail(MTP_ERR_INVALID_ARG, "rope_axes_rows: strides let heads or rows overlap");
    if (x.x_ld % 4 || x.y_ld % 4 || x.x_hs % 4 || x.y_hs % 4)
      return fail(MTP_ERR_INVALID_ARG, "rope_axes_rows: strides must be multiples of 4 floats");
    if (x.x == x.y && (x.x_ld != x.y_ld || x.x_hs != x.y_hs))
      return fail(MTP_ERR_INVALID_ARG, "rope_axes_rows: in place needs equal strides");
    heads += x.n_heads;
    a.t[i] = x;
    a.head_end[i] = heads;
  }
  if (!d_ws || !aligned16(d_ws) || ws_bytes < rope_axes_rows_workspace_bytes())
    return fail(MTP_ERR_WORKSPACE, "rope_axes_rows: workspace too small or misaligned");
  a.nt = n_t;
  a.d = head_dim;
  a.rows = rows;
  a.eps = eps;
  a.err = &static_cast<WsHeader*>(d_ws)->err;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (a.r.half % 4) {
    const int groups = (heads + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
    e = launch_pdl(rope_rows_any_kernel, dim3(groups, std::min(rows, 65535)), kRopeThreads, 0, st, a);
  } else if (head_dim <= 64) {
    e = launch_rope_rows<8, 2>(a, st);
  } else if (head_dim <= 128) {
    e = launch_rope_rows<16, 3>(a, st);
  } else {
    e = launch_rope_rows<32, 3>(a, st);
  }
  if (e != cudaSuccess) return cuda_fail(e, "rope_axes_rows launch");
  return MTP_OK;
}

}  // extern "C"
