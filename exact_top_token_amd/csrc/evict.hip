// Eviction: the choice of the keys that stay, and the move of their rows.
//
// A key's rank is its accumulated weight, above all others if it is protected
// (one of the first `prefix` or the latest `window` tokens of the text); the
// new_len keys of highest rank stay, ties to the lower index.  Kept keys in
// front of the new end do not move; the n-th kept key behind it (in order)
// moves into the n-th hole in front of it.  So a periodic eviction of a few
// keys moves a few rows, and no row is read from a place another is written
// to: the moves are independent.
#include "attn_device.h"

namespace dosa {

namespace {

constexpr int kThreads = 1024, kEvWaves = kThreads / 64;

__device__ __forceinline__ uint32_t rank_of(const EvictArgs& p, const EvictSeq& s, int key) {
  const int slot = cache_slot(p.table, s.b, p.max_pages, p.page_size, p.num_pages, key);
  if (slot < 0) return 0u;
  const int pos = p.pos != nullptr ? p.pos[slot] : key;
  if (pos < p.prefix || (int64_t)pos >= (int64_t)s.seen - p.window) return 0xffffffffu;
  const float a = p.acc[slot] + 0.f;        // -0 ranks as 0
  const uint32_t u = __float_as_uint(a);
  const uint32_t r = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
  return r < 1u ? 1u : (r > 0xfffffffeu ? 0xfffffffeu : r);
}

// Exclusive sum over the workgroup of a 0/1 flag; *total gets the whole sum.
__device__ __forceinline__ int block_rank(bool f, int* sh, int* total) {
  const unsigned long long b = __ballot(f);
  const int lane = lane64(), wave = threadIdx.x >> 6;
  if (lane == 0) sh[wave] = __popcll(b);
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kEvWaves; ++i) {
    const int c = sh[i];
    before += i < wave ? c : 0;
    all += c;
  }
  __syncthreads();
  *total = all;
  return before + __popcll(b & ((1ull << lane) - 1ull));
}

__global__ __launch_bounds__(kThreads) void evict_select_kernel(const EvictArgs p) {
  __shared__ uint32_t hist[256];
  __shared__ int sh[kEvWaves];
  __shared__ uint32_t sel[2];
  const EvictSeq& s = p.s[blockIdx.x];
  const int tid = threadIdx.x;
  int32_t* out = p.out_src + (int64_t)s.b * p.out_stride;
  int32_t* movers = p.moves + (int64_t)s.b * p.move_stride;
  // threshold: the new_len-th largest rank, digit by digit
  uint32_t pre = 0, need = (uint32_t)s.new_len;
  if (s.new_len > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      for (int k = tid; k < s.kv_len; k += kThreads) {
        const uint32_t r = rank_of(p, s, k);
        if (shift == 24 || (r >> (shift + 8)) == (pre >> (shift + 8))) atomicAdd(&hist[(r >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (tid == 0) {
        uint32_t left = need;
        int d = 255;
        for (; d > 0 && hist[d] < left; --d) left -= hist[d];
        sel[0] = pre | ((uint32_t)d << shift);
        sel[1] = left;
      }
      __syncthreads();
      pre = sel[0];
      need = sel[1];
      __syncthreads();
    }
  }
  // ranks above `pre` stay, and the first `need` equal to it
  int equal0 = 0, mover0 = 0, hole0 = 0;
  for (int k0 = 0; k0 < s.kv_len; k0 += kThreads) {
    const int k = k0 + tid;
    const bool in = k < s.kv_len;
    const uint32_t r = in && s.new_len > 0 ? rank_of(p, s, k) : 0u;
    int n_eq, n_mv, n_ho;
    const bool eq = in && s.new_len > 0 && r == pre;
    const int er = equal0 + block_rank(eq, sh, &n_eq);
    const bool keep = in && s.new_len > 0 && (r > pre || (eq && er < (int)need));
    const bool mv = keep && k >= s.new_len, ho = in && !keep && k < s.new_len;
    const int mr = mover0 + block_rank(mv, sh, &n_mv), hr = hole0 + block_rank(ho, sh, &n_ho);
    if (mv) movers[mr] = k;
    if (in && k < s.new_len) out[k] = keep ? k : -2 - hr;
    equal0 += n_eq;
    mover0 += n_mv;
    hole0 += n_ho;
  }
  __threadfence_block();
  __syncthreads();
  for (int k = tid; k < p.out_stride; k += kThreads) {
    if (k >= s.new_len) out[k] = -1;
    else if (out[k] <= -2) out[k] = movers[-2 - out[k]];
  }
}

constexpr int kRows = 64;     // rows of a workgroup

template <class V>
__device__ __forceinline__ void copy_rows(const EvictArray& a, const int* from, const int* to, int n, bool in_place) {
  const int cols = a.row_bytes / (int)sizeof(V);
  const V* src = reinterpret_cast<const V*>(a.src);
  V* dst = reinterpret_cast<V*>(a.dst);
  for (int i = threadIdx.x; i < n * cols; i += (int)blockDim.x) {
    const int r = i / cols, c = i - r * cols;
    const int f = from[r], t = to[r];
    if (f < 0 || t < 0 || (in_place && f == t)) continue;
    dst[(int64_t)t * cols + c] = src[(int64_t)f * cols + c];
  }
}

__global__ __launch_bounds__(256) void evict_move_kernel(const EvictMoveArgs p) {
  __shared__ int from[kRows], to[kRows];
  const EvictSeq& s = p.s[blockIdx.y];
  const int j0 = blockIdx.x * kRows;
  const int n = min(kRows, s.new_len - j0);
  if (n <= 0) return;
  if ((int)threadIdx.x < n) {
    const int j = j0 + (int)threadIdx.x;
    const int src = p.out_src[(int64_t)s.b * p.out_stride + j];
    to[threadIdx.x] = cache_slot(p.table, s.b, p.max_pages, p.page_size, p.num_pages, j);
    from[threadIdx.x] = src < 0 ? -1 : cache_slot(p.table, s.b, p.max_pages, p.page_size, p.num_pages, src);
  }
  __syncthreads();
  for (int i = 0; i < p.n_arr; ++i) {
    const EvictArray& a = p.a[i];
    const bool in_place = a.src == a.dst;
    if (a.gran == 16) copy_rows<i4>(a, from, to, n, in_place);
    else if (a.gran == 4) copy_rows<uint32_t>(a, from, to, n, in_place);
    else copy_rows<uint8_t>(a, from, to, n, in_place);
  }
}

}  // namespace

hipError_t launch_evict_select(const EvictArgs& p, hipStream_t s) {
  if (p.n_seq == 0) return hipSuccess;
  evict_select_kernel<<<dim3((unsigned)p.n_seq), dim3(kThreads), 0, s>>>(p);
  return hipGetLastError();
}

hipError_t launch_evict_move(const EvictMoveArgs& p, hipStream_t s) {
  if (p.n_seq == 0 || p.n_arr == 0 || p.max_new == 0) return hipSuccess;
  evict_move_kernel<<<dim3((unsigned)((p.max_new + kRows - 1) / kRows), (unsigned)p.n_seq), dim3(256), 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace dosa
