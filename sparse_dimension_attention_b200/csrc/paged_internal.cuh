// Shared pieces of the paged 8-bit cache kernels: e4m3 conversions, the scale
// rule, the rotation of one row, and the checks of device-side batch data.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "aqua_internal.cuh"

namespace aqua {

// Smallest scale a page is given: amax / 448 below it would only be zeros and
// subnormals of a value range no model produces, and a scale of 0 cannot be
// divided by.
constexpr int kScaleMinExp = -60;

// The fields of aqua_paged_cache the kernels use (descriptor copied by value).
struct PagedView {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  const int32_t* table;
  int32_t* ctrl;
  int B, Hkv, m, page, page_log2, n_pages, max_pages;

  __device__ __forceinline__ long long capacity() const { return (long long)max_pages * page; }
  // byte offset of the key / value block of (page, head)
  __device__ __forceinline__ size_t kblock(int pid, int h) const { return ((size_t)pid * Hkv + h) * (size_t)(m << page_log2); }
  __device__ __forceinline__ size_t vblock(int pid, int h) const {
    return ((size_t)pid * Hkv + h) * (size_t)(kHeadDim << page_log2);
  }
};

// Elements between rows and between heads of an input [rows][heads][128].
struct Strides {
  long long row, head;
};

struct RopeView {
  const float* cs;   // nullptr: no rotation
  int n_pos, rot, interleaved;
};

// Tokens of a sequence that a kernel reads: a length that is negative, beyond
// the block table or beyond the rotation table counts as 0 (and is reported).
__device__ __forceinline__ int checked_len(int len, const PagedView& c, int n_pos_limit, bool& bad) {
  bad = len < 0 || len > c.capacity() || len > n_pos_limit;
  return bad ? 0 : len;
}

// two e4m3 codes (low byte first) -> two f16, exact (NaN codes give NaN)
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}

// two f32 -> two e4m3 codes, nearest even, saturating (inf too), NaN kept; lo in the low byte
__device__ __forceinline__ uint16_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t f32x4_to_e4m3x4(float a, float b, float c, float d) {
  return (uint32_t)f32x2_to_e4m3x2(a, b) | ((uint32_t)f32x2_to_e4m3x2(c, d) << 16);
}

__device__ __forceinline__ float2 e4m3x2_to_f32x2(uint16_t c) {
  const uint32_t h = e4m3x2_to_f16x2(c);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// |x| for the page maximum: infinities and NaN do not set the scale
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.f;
}

// Smallest power of two s >= 2^kScaleMinExp with amax <= 448 s.  448 = 1.75 * 2^8,
// so with amax = f * 2^E (1 <= f < 2) s is 2^(E-8), or 2^(E-7) when f > 1.75.  A power of two keeps
// every code's mantissa when the scale of a page grows, and e4m3's relative step does not
// depend on it, so nothing is lost against amax / 448.
__device__ __forceinline__ float pow2_scale(float amax) {
  const uint32_t b = __float_as_uint(amax);
  int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);   // subnormals: below the minimum anyway
  e = max(e, kScaleMinExp);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Element i of a row rotated to its position; row: the raw 128 elements (shared
// memory), cs: the position's rot / 2 cosines, then its sines.
// F: the type it is computed in.
template <typename F>
__device__ __forceinline__ F rotated(const float* row, int i, const float* cs, int rot, bool interleaved) {
  const F x = (F)row[i];
  if (i >= rot) return x;
  const int half = rot >> 1;
  int j, o;       // angle index, partner
  bool first;
  if (interleaved) {
    j = i >> 1;
    first = (i & 1) == 0;
    o = i ^ 1;
  } else {
    first = i < half;
    j = first ? i : i - half;
    o = first ? i + half : i - half;
  }
  const F c = (F)__ldg(cs + j), s = (F)__ldg(cs + half + j);
  const F y = (F)row[o];
  return first ? x * c - y * s : x * c + y * s;
}

// Has P of one head (64 KB) brought to L2, 128 bytes a thread and turn.  Before the wait on the previous kernel: that
// kernel may be what writes P, so it is read only after the wait, which alone makes the writes visible.
__device__ __forceinline__ void prefetch_head(const float* P, int tid, int nthreads) {
  for (int i = tid; i < kHeadDim * kHeadDim / 32; i += nthreads)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(P + 32 * i));
}

__device__ __forceinline__ void report_arg(const PagedView& c) { record_status(c.ctrl, AQUA_ERR_ARG); }

}  // namespace aqua
