// Write and read-back of the paged 4-bit cache.
//
// A row (one token, one kv head) is cut into blocks of 32 elements.  A block's
// scale is 2^e with the smallest e for which every |x| < 7 * 2^e: the largest
// code is 6, and up to 7 its distance to x is at most the half step 1 of that
// binade, so no element is off by more than half a step.  In bits: adding
// 2^21 to a float carries into the exponent exactly from mantissa 1.75 on,
// and 1.75 * 4 = 7.  The codes are the converter's, to nearest with ties to
// the even code.
//
// Bound by memory: 2 (4) bytes in and 17/32 byte out per element.  Four lanes
// share a block, eight elements each: 16-byte loads and 4-byte stores without
// gaps, the block maximum from two lane swaps.
#include "attn_device.h"

namespace dosa {

namespace {

constexpr int kTokens = 16;    // tokens of a workgroup

struct Where {
  int seq, tok0, n;            // record, first token of the workgroup within it, tokens
};

// Slots of the workgroup's tokens, and its place in the launch.
__device__ __forceinline__ Where place(const CacheIoArgs& p, int* slots) {
  int u = blockIdx.x, i = 0;
  for (; i < p.n_seq - 1; ++i) {
    const int nb = (p.s[i].n + kTokens - 1) / kTokens;
    if (u < nb) break;
    u -= nb;
  }
  const CacheSeq& s = p.s[i];
  Where w{i, u * kTokens, min(kTokens, s.n - u * kTokens)};
  if ((int)threadIdx.x < w.n)
    slots[threadIdx.x] = cache_slot(p.cache.table, s.b, p.cache.max_pages, p.cache.page_size, p.cache.num_pages,
                                    s.pos0 + w.tok0 + (int)threadIdx.x);
  __syncthreads();
  return w;
}

template <bool F32>
__device__ __forceinline__ void load8(const void* base, int64_t at, float* x) {
  if constexpr (F32) {
    const f4* s = reinterpret_cast<const f4*>(static_cast<const float*>(base) + at);
    const f4 a = s[0], b = s[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = a[i];
      x[4 + i] = b[i];
    }
  } else {
    const i4 a = *reinterpret_cast<const i4*>(static_cast<const uint16_t*>(base) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float((uint32_t)a[i] << 16);
      x[2 * i + 1] = __uint_as_float((uint32_t)a[i] & 0xffff0000u);
    }
  }
}

// Eight elements of a lane -> their codes; the block's scale byte.
__device__ __forceinline__ uint32_t encode8(const float* x, uint32_t* scale_byte) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));
  top = fmaxf(top, __shfl_xor(top, 1));
  top = fmaxf(top, __shfl_xor(top, 2));
  int e = (int)((__float_as_uint(top) + 0x00200000u) >> 23) - 2;
  e = e < 1 ? 1 : (e > 254 ? 254 : e);
  *scale_byte = (uint32_t)e;
  const float scale = __uint_as_float((uint32_t)e << 23);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], scale, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], scale, 3);
  return w;
}

template <bool F32, int D>
__global__ __launch_bounds__(256) void cache_append_kernel(const CacheIoArgs p) {
  __shared__ int slots[kTokens];
  const Where w = place(p, slots);
  const CacheSeq& s = p.s[w.seq];
  const int tid = threadIdx.x, Hkv = p.cache.Hkv;
  if (p.pos != nullptr && tid < w.n && slots[tid] >= 0) p.pos[slots[tid]] = s.seen0 + w.tok0 + tid;
  const int cols = Hkv * (D / 8);            // lanes of a token
  const int per = cols < 256 ? 256 / cols : 1;
  const int sub = cols < 256 ? tid / cols : 0;
  if (sub >= per) return;
  for (int col = cols < 256 ? tid - sub * cols : tid; col < cols; col += 256) {
    for (int t = sub; t < w.n; t += per) {
      const int slot = slots[t];
      const int64_t row = s.row0 + w.tok0 + t;
      float xk[8], xv[8];
      load8<F32>(p.k, row * p.k_stride + col * 8, xk);
      load8<F32>(p.v, row * p.v_stride + col * 8, xv);
      uint32_t ek, ev;
      const uint32_t ck = encode8(xk, &ek), cv = encode8(xv, &ev);
      if (slot < 0) continue;
      reinterpret_cast<uint32_t*>(p.cache.k_codes)[(int64_t)slot * cols + col] = ck;
      reinterpret_cast<uint32_t*>(p.cache.v_codes)[(int64_t)slot * cols + col] = cv;
      if ((col & 3) == 0) {
        p.cache.k_scales[(int64_t)slot * (cols / 4) + col / 4] = (uint8_t)ek;
        p.cache.v_scales[(int64_t)slot * (cols / 4) + col / 4] = (uint8_t)ev;
      }
    }
  }
}

template <bool F32>
__device__ __forceinline__ void store8(void* base, int64_t at, uint32_t codes, uint32_t e) {
  const i4 x = __builtin_bit_cast(i4, mx8(codes, __uint_as_float(e << 23)));
  if constexpr (F32) {
    f4* d = reinterpret_cast<f4*>(static_cast<float*>(base) + at);
#pragma unroll
    for (int h = 0; h < 2; ++h)
      d[h] = f4{__uint_as_float((uint32_t)x[2 * h] << 16), __uint_as_float((uint32_t)x[2 * h] & 0xffff0000u),
                __uint_as_float((uint32_t)x[2 * h + 1] << 16), __uint_as_float((uint32_t)x[2 * h + 1] & 0xffff0000u)};
  } else {
    *reinterpret_cast<i4*>(static_cast<uint16_t*>(base) + at) = x;
  }
}

template <bool F32, int D>
__global__ __launch_bounds__(256) void cache_read_kernel(const CacheIoArgs p) {
  __shared__ int slots[kTokens];
  const Where w = place(p, slots);
  const CacheSeq& s = p.s[w.seq];
  const int tid = threadIdx.x, Hkv = p.cache.Hkv;
  const int cols = Hkv * (D / 8);
  const int per = cols < 256 ? 256 / cols : 1;
  const int sub = cols < 256 ? tid / cols : 0;
  if (sub >= per) return;
  for (int col = cols < 256 ? tid - sub * cols : tid; col < cols; col += 256) {
    for (int t = sub; t < w.n; t += per) {
      const int slot = slots[t];
      const int64_t at = slot < 0 ? 0 : slot;
      const int64_t row = s.row0 + w.tok0 + t;
      uint32_t ck = 0, cv = 0, ek = 1, ev = 1;      // a token without a page reads as zeros
      if (slot >= 0) {
        ck = reinterpret_cast<const uint32_t*>(p.cache.k_codes)[at * cols + col];
        cv = reinterpret_cast<const uint32_t*>(p.cache.v_codes)[at * cols + col];
        ek = p.cache.k_scales[at * (cols / 4) + col / 4];
        ev = p.cache.v_scales[at * (cols / 4) + col / 4];
      }
      store8<F32>(p.k, row * p.k_stride + col * 8, ck, ek);
      store8<F32>(p.v, row * p.v_stride + col * 8, cv, ev);
    }
  }
}

int blocks(const CacheIoArgs& p) {
  int n = 0;
  for (int i = 0; i < p.n_seq; ++i) n += (p.s[i].n + kTokens - 1) / kTokens;
  return n;
}

}  // namespace

hipError_t launch_cache_append(bool f32, int d, const CacheIoArgs& p, hipStream_t s) {
  const dim3 grid((unsigned)blocks(p)), block(256);
  if (grid.x == 0) return hipSuccess;
  if (f32 && d == 128) cache_append_kernel<true, 128><<<grid, block, 0, s>>>(p);
  else if (f32) cache_append_kernel<true, 64><<<grid, block, 0, s>>>(p);
  else if (d == 128) cache_append_kernel<false, 128><<<grid, block, 0, s>>>(p);
  else cache_append_kernel<false, 64><<<grid, block, 0, s>>>(p);
  return hipGetLastError();
}

hipError_t launch_cache_read(bool f32, int d, const CacheIoArgs& p, hipStream_t s) {
  const dim3 grid((unsigned)blocks(p)), block(256);
  if (grid.x == 0) return hipSuccess;
  if (f32 && d == 128) cache_read_kernel<true, 128><<<grid, block, 0, s>>>(p);
  else if (f32) cache_read_kernel<true, 64><<<grid, block, 0, s>>>(p);
  else if (d == 128) cache_read_kernel<false, 128><<<grid, block, 0, s>>>(p);
  else cache_read_kernel<false, 64><<<grid, block, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace dosa
