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
// Bound by memory: 2 (4) bytes in and 17/32 byte out per element (42395 tokens
// of 8 heads, d = 128, bf16: 220 MB in 37-69 us, the longer when the cache in
// front of the memory is full of someone's writes; read back in fp32, 393 MB in
// 73 us).  A decode step's 128 tokens take 5 us, latency.  Four lanes
// share a block, eight elements each: 16-byte loads and 4-byte stores without
// gaps (fp32: eight lanes of four elements), the block maximum from two lane swaps.
#include "attn_device.h"

namespace dosa {

namespace {

constexpr int kTokens = kCacheTokens;

struct Where {
  int seq, tok0, n;            // record, first token of the workgroup within it, tokens
};

// Slots of the workgroup's tokens, and its place in the launch.
__device__ __forceinline__ Where place(const CacheIoArgs& p, int* slots) {
  const int i = find_seq(p.s, p.n_seq, (int)blockIdx.x, [](const CacheSeq& s) { return s.unit0; });
  const CacheSeq& s = p.s[i];
  const int tok0 = ((int)blockIdx.x - s.unit0) * kTokens;
  Where w{i, tok0, min(kTokens, s.n - tok0)};
  if ((int)threadIdx.x < kTokens)
    slots[threadIdx.x] = (int)threadIdx.x < w.n ? cache_slot(p.cache.table, s.b, p.cache.max_pages, p.cache.page_size,
                                                             p.cache.num_pages, s.pos0 + tok0 + (int)threadIdx.x)
                                                : -1;
  __syncthreads();
  return w;
}

// A lane's share of a row: 16 bytes of the packed operand.
template <bool F32>
struct Share {
  static constexpr int E = F32 ? 4 : 8;      // elements
};

template <bool F32>
__device__ __forceinline__ void widen(i4 a, float* x) {
  if constexpr (F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __int_as_float(a[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float((uint32_t)a[i] << 16);
      x[2 * i + 1] = __uint_as_float((uint32_t)a[i] & 0xffff0000u);
    }
  }
}

// A lane's elements -> their codes and the block's scale byte (the block is
// 32 / E neighbouring lanes).
template <bool F32>
__device__ __forceinline__ uint32_t encode(i4 raw, uint32_t* scale_byte) {
  constexpr int E = Share<F32>::E;
  float x[E];
  widen<F32>(raw, x);
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) top = fmaxf(top, fabsf(x[i]));
#pragma unroll
  for (int m = 1; m < 32 / E; m <<= 1) top = fmaxf(top, __shfl_xor(top, m));
  int e = (int)((__float_as_uint(top) + 0x00200000u) >> 23) - 2;
  e = e < 1 ? 1 : (e > 254 ? 254 : e);
  *scale_byte = (uint32_t)e;
  const float scale = __uint_as_float((uint32_t)e << 23);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], scale, 1);
  if constexpr (!F32) {
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], scale, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], scale, 3);
  }
  return w;
}

template <bool F32>
__device__ __forceinline__ void put(uint8_t* codes, uint8_t* scales, int64_t at, uint32_t w, uint32_t e) {
  constexpr int E = Share<F32>::E;
  if constexpr (F32) reinterpret_cast<uint16_t*>(codes)[at] = (uint16_t)w;
  else reinterpret_cast<uint32_t*>(codes)[at] = w;
  if ((at & (32 / E - 1)) == 0) scales[at / (32 / E)] = (uint8_t)e;
}

// kUnroll tokens at a time, so that their loads are in flight together.
constexpr int kUnroll = 4;

template <bool F32, int D>
__global__ __launch_bounds__(256) void cache_append_kernel(const CacheIoArgs p) {
  constexpr int E = Share<F32>::E;
  __shared__ int slots[kTokens];
  const Where w = place(p, slots);
  const CacheSeq& s = p.s[w.seq];
  const int tid = threadIdx.x, Hkv = p.cache.Hkv;
  if (p.pos != nullptr && tid < w.n && slots[tid] >= 0) p.pos[slots[tid]] = s.seen0 + w.tok0 + tid;
  const int cols = Hkv * (D / E);            // lanes of a token
  const int per = cols < 256 ? 256 / cols : 1;
  const int sub = cols < 256 ? tid / cols : 0;
  if (sub >= per) return;
  const int64_t row0 = s.row0 + w.tok0;
  for (int col = cols < 256 ? tid - sub * cols : tid; col < cols; col += 256) {
    for (int t0 = sub; t0 < w.n; t0 += kUnroll * per) {
      i4 xk[kUnroll], xv[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int64_t row = row0 + min(t0 + i * per, w.n - 1);
        xk[i] = *reinterpret_cast<const i4*>(static_cast<const char*>(p.k) + (row * p.k_stride + col * E) * (16 / E));
        xv[i] = *reinterpret_cast<const i4*>(static_cast<const char*>(p.v) + (row * p.v_stride + col * E) * (16 / E));
      }
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int t = t0 + i * per;
        const int slot = t < w.n ? slots[t] : -1;
        uint32_t ek, ev;
        const uint32_t ck = encode<F32>(xk[i], &ek), cv = encode<F32>(xv[i], &ev);
        if (slot >= 0) {
          put<F32>(p.cache.k_codes, p.cache.k_scales, (int64_t)slot * cols + col, ck, ek);
          put<F32>(p.cache.v_codes, p.cache.v_scales, (int64_t)slot * cols + col, cv, ev);
        }
      }
    }
  }
}

// A lane's codes -> 16 bytes of the packed operand.
template <bool F32>
__device__ __forceinline__ void store_row(void* base, int64_t at, uint32_t codes, uint32_t e) {
  const float sc = __uint_as_float(e << 23);
  if constexpr (F32) {
    const uint32_t a = mx2<0>(codes, sc), b = mx2<1>(codes, sc);
    *reinterpret_cast<i4*>(static_cast<float*>(base) + at) =
        i4{(int)(a << 16), (int)(a & 0xffff0000u), (int)(b << 16), (int)(b & 0xffff0000u)};
  } else {
    *reinterpret_cast<i4*>(static_cast<uint16_t*>(base) + at) = __builtin_bit_cast(i4, mx8(codes, sc));
  }
}

template <bool F32, int D>
__global__ __launch_bounds__(256) void cache_read_kernel(const CacheIoArgs p) {
  constexpr int E = Share<F32>::E;
  __shared__ int slots[kTokens];
  const Where w = place(p, slots);
  const CacheSeq& s = p.s[w.seq];
  const int tid = threadIdx.x, Hkv = p.cache.Hkv;
  const int cols = Hkv * (D / E);
  const int per = cols < 256 ? 256 / cols : 1;
  const int sub = cols < 256 ? tid / cols : 0;
  if (sub >= per) return;
  const int64_t row0 = s.row0 + w.tok0;
  auto codes = [&](const uint8_t* base, int64_t at) -> uint32_t {
    if constexpr (F32) return reinterpret_cast<const uint16_t*>(base)[at];
    else return reinterpret_cast<const uint32_t*>(base)[at];
  };
  for (int col = cols < 256 ? tid - sub * cols : tid; col < cols; col += 256) {
    for (int t0 = sub; t0 < w.n; t0 += kUnroll * per) {
      uint32_t ck[kUnroll], cv[kUnroll], ek[kUnroll], ev[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int slot = slots[min(t0 + i * per, w.n - 1)];
        const int64_t at = (int64_t)(slot < 0 ? 0 : slot) * cols + col;
        ck[i] = codes(p.cache.k_codes, at);
        cv[i] = codes(p.cache.v_codes, at);
        ek[i] = p.cache.k_scales[at / (32 / E)];
        ev[i] = p.cache.v_scales[at / (32 / E)];
        if (slot < 0) {          // a token without a page reads as zeros
          ck[i] = cv[i] = 0;
          ek[i] = ev[i] = 1;
        }
      }
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int t = t0 + i * per;
        if (t < w.n) {
          store_row<F32>(p.k, (row0 + t) * p.k_stride + col * E, ck[i], ek[i]);
          store_row<F32>(p.v, (row0 + t) * p.v_stride + col * E, cv[i], ev[i]);
        }
      }
    }
  }
}

int blocks(const CacheIoArgs& p) {
  const CacheSeq& s = p.s[p.n_seq - 1];
  return s.unit0 + (s.n + kTokens - 1) / kTokens;
}

}  // namespace

hipError_t launch_cache_append(bool f32, int d, const CacheIoArgs& p, hipStream_t s) {
  if (p.n_seq == 0) return hipSuccess;
  const dim3 grid((unsigned)blocks(p)), block(256);
  if (f32 && d == 128) cache_append_kernel<true, 128><<<grid, block, 0, s>>>(p);
  else if (f32) cache_append_kernel<true, 64><<<grid, block, 0, s>>>(p);
  else if (d == 128) cache_append_kernel<false, 128><<<grid, block, 0, s>>>(p);
  else cache_append_kernel<false, 64><<<grid, block, 0, s>>>(p);
  return hipGetLastError();
}

hipError_t launch_cache_read(bool f32, int d, const CacheIoArgs& p, hipStream_t s) {
  if (p.n_seq == 0) return hipSuccess;
  const dim3 grid((unsigned)blocks(p)), block(256);
  if (f32 && d == 128) cache_read_kernel<true, 128><<<grid, block, 0, s>>>(p);
  else if (f32) cache_read_kernel<true, 64><<<grid, block, 0, s>>>(p);
  else if (d == 128) cache_read_kernel<false, 128><<<grid, block, 0, s>>>(p);
  else cache_read_kernel<false, 64><<<grid, block, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace dosa
