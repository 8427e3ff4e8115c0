// Device-side building blocks of the attention kernels for gfx950.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attn_internal.h"

namespace dosa {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef int i4 __attribute__((ext_vector_type(4)));
typedef int i2 __attribute__((ext_vector_type(2)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// Exponents are taken as s c - m c in one multiply-add, c = scale log2(e), with
// m c rounded to fp32.  Up to this magnitude that shifts an exponent by 2^-15 at
// most, no more than fp32 scores of the size are off; beyond it the shift would
// grow into the weights (2^31: into infinity), and m is subtracted first.  The
// accumulated weights of bf16 prompts do the same with the normaliser in m's
// place; the other weights kernels always subtract first.
constexpr float kFar = 1024.f;

typedef __attribute__((address_space(4))) const int32_t scalar_i32;      // read through the scalar cache

__device__ __forceinline__ int lane64() { return (int)__lane_id(); }
__device__ __forceinline__ int below(uint64_t mask) {        // lanes of the mask in front of this one
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0u));
}

// The record of the launch that unit `u` belongs to: `first` of the records
// ascends.  Uniform.
template <class Seq, class First>
__device__ __forceinline__ int find_seq(const Seq* s, int n, int u, First first) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first(s[mid]) <= u) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ f4 mfma_bf16(b8 a, b8 b, f4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f4 mfma_f32(float a, float b, f4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// Two 4-bit codes (byte SEL of w) times the power of two in `scale`'s exponent
// bits -> two bf16: exact, a code has two significant bits.
template <int SEL>
__device__ __forceinline__ uint32_t mx2(uint32_t w, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, SEL));
}
__device__ __forceinline__ b8 mx8(uint32_t w, float scale) {
  return __builtin_bit_cast(b8, i4{(int)mx2<0>(w, scale), (int)mx2<1>(w, scale), (int)mx2<2>(w, scale), (int)mx2<3>(w, scale)});
}

// Scale byte `blk` of a row's scale bytes -> the float with that exponent.
__device__ __forceinline__ float mx_scale(uint32_t bytes, int blk8) {
  return __uint_as_float(((bytes >> blk8) & 255u) << 23);
}

// Low (high) halves of two words, first word in the low half.
__device__ __forceinline__ uint32_t lows(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); }
__device__ __forceinline__ uint32_t highs(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  b2 r;
  r[0] = (__bf16)a;
  r[1] = (__bf16)b;
  return __builtin_bit_cast(uint32_t, r);
}

// x = t0 + t1 + t2 in bf16 terms: 24 significant bits, so products of the
// terms with exact bf16 operands, summed in fp32, are fp32 products.  The terms
// are cut off, not rounded: eight bits each suffice, and a number next to the
// largest would round to infinity.
__device__ __forceinline__ float top_bits(float x) { return __uint_as_float(__float_as_uint(x) & 0xffff0000u); }
__device__ __forceinline__ void split3(float x, float* t) {
  t[0] = top_bits(x);
  const float r = x - t[0];
  t[1] = top_bits(r);
  t[2] = r - t[1];
}

// exp(scale s - lse): the normaliser is taken off before the change of base, so
// that its own rounding to fp32 is all that a large one costs.  lse = INFINITY:
// a row that gives nothing.
__device__ __forceinline__ float weight_of(float s, float scale, float lse) {
  return __builtin_amdgcn_exp2f(fmaf(s, scale, -lse) * kLog2e);
}

// 16-byte chunk of a key tile's row `r` in LDS that holds logical chunk c: 16
// lanes read one chunk of 16 rows.
template <int D>
__device__ __forceinline__ int k_chunk(int r, int c) {
  return D == 128 ? c ^ (r & 15) : c ^ ((r >> 1) & 7);
}

// Maximum / sum over the four 16-lane groups (lanes l, l^16, l^32, l^48).
__device__ __forceinline__ float max_groups(float x) {
  const uint32_t u = __float_as_uint(x);
  auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const float y = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  const uint32_t w = __float_as_uint(y);
  auto q = __builtin_amdgcn_permlane16_swap(w, w, false, false);
  return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}
__device__ __forceinline__ float sum_groups(float x) {
  const uint32_t u = __float_as_uint(x);
  auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const float y = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  const uint32_t w = __float_as_uint(y);
  auto q = __builtin_amdgcn_permlane16_swap(w, w, false, false);
  return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

// Order LDS accesses of one wavefront against each other (the hardware keeps
// a wavefront's LDS operations in order; this keeps the compiler from moving
// them).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Pool slot of a logical position, or -1 when its table entry names no page.
__device__ __forceinline__ int cache_slot(const int32_t* table, int b, int max_pages, int page_size, int num_pages,
                                          int pos) {
  const int pg = pos / page_size;
  if (pg >= max_pages) return -1;
  const int page = table[(int64_t)b * max_pages + pg];
  if ((uint32_t)page >= (uint32_t)num_pages) return -1;
  return page * page_size + (pos - pg * page_size);
}

}  // namespace dosa
