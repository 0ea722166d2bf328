// Pieces that the attention kernels over caches share: powers-of-two scales and
// f16 operand tiles of the split kernel (treeattn.cu), packed float32
// arithmetic, bounded waits.
#pragma once

#include "tc5.cuh"
#include "tree.cuh"

namespace mtp {

constexpr float kLog2e = 1.4426950408889634f;

// What the split kernel reads and writes: every query row of a KV head against
// cached keys that all of them see.  "Head" is a KV head of a cache, or of one of
// several caches that lie one after another.
struct SplitArgs {
  int dqk, dv;
  long long cap;           // rows a head
  const float *keys, *values;  // [heads][cap][dqk], [heads][cap][dv]
  uint8_t* qt;             // [heads][mt] tiles of 128 rows: f16 hi parts, then lo parts
  float* qinv;             // [heads][mt * 128] power of two that undoes a row's f16 scale
  float* part_o;           // [heads][ns][R][dv]
  float2* part_ml;         // [heads][ns][R] running maximum and sum
  float qscale;            // logit scale times log2(e)
  int R, mt;               // query rows of a head, tiles of 128 of them
  int ns;                  // splits
  int vstages;             // V tile buffers of the split kernel's COL form (1 or 2)
  int rep;                 // copies of the query rows in a tile (see the split kernel)
  int* err;
};

// Power-of-two scale of values for their f16 parts: the largest |x| lands in
// [2^14, 2^15), so hi + lo hold 22 bits of every element down to 2^-16 of the
// largest.  Infinity keeps scale 1; values below 2^-95 are scaled by at most
// 2^109.  Returns the inverse, exactly.
__device__ __forceinline__ float f16_scale(float largest, float& scale) {
  uint32_t e = __float_as_uint(largest) >> 23;
  e = e == 255u ? 141u : max(e, 32u);
  scale = __uint_as_float((268u - e) << 23);
  return __uint_as_float((e - 14u) << 23);
}

// Byte offset of value c of row r in an operand tile of `rows` rows: blocks of
// 64 values, rows of 128 bytes, 16-byte chunks swizzled by the row (the layout
// of a K-major operand with c along K, and of an MN-major one with r along K).
__device__ __forceinline__ uint32_t tile_off(int r, int c, int rows) {
  return (uint32_t)((c >> 6) * rows * 128 + r * 128 + ((((c >> 3) & 7) ^ (r & 7)) << 4) + (c & 7) * 2);
}

// Writes a query row's f16 hi and lo parts for the split kernel: 16-byte chunks
// of 8 dims, a chunk's 128 rows consecutive, hi chunks then lo chunks.
__device__ __forceinline__ void store_q_tile(const SplitArgs& a, const HeadVals& v, int kv, int r,
                                             int half, int lane) {
  float mx = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) mx = fmaxf(mx, fmaxf(fabsf(v.a[j]), fabsf(v.b[j])));
#pragma unroll
  for (int j = 0; j < 8; ++j) mx = fmaxf(mx, fabsf(v.c[j]));
  float scale;
  const float inv = f16_scale(warp_max(mx * a.qscale), scale);
  const int rr = r & 127, tile = r >> 7, rows = 128 / a.rep;
  __half* hi = reinterpret_cast<__half*>(a.qt + ((size_t)kv * a.mt + tile) * 512 * a.dqk);
  if (lane == 0) a.qinv[((size_t)kv * a.mt + tile) * 128 + rr] = inv;
  auto put = [&](int c, float x) {
    x = x * a.qscale * scale;
    const __half h = __float2half_rn(x), l = __float2half_rn(x - __half2float(h));
    for (int i = rr; i < 128; i += rows) {
      const int at = ((c >> 3) * 128 + i) * 8 + (c & 7);
      hi[at] = h;
      hi[128 * a.dqk + at] = l;
    }
  };
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (lane + 32 * j < half) {
      put(lane + 32 * j, v.a[j]);
      put(lane + 32 * j + half, v.b[j]);
    }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (2 * half + lane + 32 * j < a.dqk) put(2 * half + lane + 32 * j, v.c[j]);
}

// Two floats in one 64-bit register pair (packed float32 arithmetic).
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ void l2_prefetch(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// A wait that gives up marks the launch (error 1) and lets every later wait of
// the thread through, so the barriers below are still met by every thread.
struct Waiter {
  int* err;
  bool dead;
  __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) {
    if (!dead && !mbar_wait_bounded(bar, parity)) {
      dead = true;
      set_dev_error(err, kErrMbarTimeout);
    }
  }
  // After a wait that gave up (the outputs are not valid): time for copies and
  // MMAs in flight to land, a few milliseconds, before the memory is freed.
  __device__ __noinline__ void settle() {
    if (dead)
      for (int i = 0; i < 2000; ++i) __nanosleep(1000);
  }
};

__device__ __forceinline__ float4 dims4(const float* row, int d, int lane, int h) {
  const int c = 128 * h + 4 * lane;
  return c < d ? *reinterpret_cast<const float4*>(row + c) : make_float4(0.f, 0.f, 0.f, 0.f);
}

__device__ __forceinline__ void scale4(float4& v, float f) {
  v.x *= f;
  v.y *= f;
  v.z *= f;
  v.w *= f;
}

__device__ __forceinline__ void add4(float4& v, float f, const float4& x) {
  v.x = fmaf(f, x.x, v.x);
  v.y = fmaf(f, x.y, v.y);
  v.z = fmaf(f, x.z, v.z);
  v.w = fmaf(f, x.w, v.w);
}

}  // namespace mtp
