// Attention weight every cached key received, summed over queries and heads:
//   w_s = sum over queries i that see s and query heads h of exp(scale q_ih . k_s - lse_ih),
//   acc_out[s] = (acc[s], or 0 for the call's own tokens) + w_s.
// The normalisers come from an attention call, so one pass suffices and every
// key is summed by itself: no atomics, and the result does not change from run
// to run.
//
// This is the kernel for fp32 queries of more than 32 rows; the others are in
// weights_tiles.hip.  A workgroup owns 64 keys, its wavefronts share the (kv
// head, query row) work between them, and the sums meet in LDS and, where
// several workgroups share 64 keys, in a buffer that a second launch adds up
// in a fixed order.  A wavefront holds the 64 keys of a head as bf16 matrix
// operands (decoded once) and streams the query rows past them as three bf16
// terms each: S^T = K Q^T leaves a lane with one query row and 16 keys, whose
// weights it adds to 16 running sums.  Bound by the products (three for one).
#include "attn_device.h"

namespace dosa {

namespace {

constexpr int kWaves = 8;

template <int D>
__global__ __launch_bounds__(64 * kWaves) void weights_kernel(const WeightArgs p) {
  constexpr int NS = D / 32, TERMS = 3;
  __shared__ __attribute__((aligned(16))) uint32_t sc[kWaves][64];
  __shared__ float sums[kWaves][64];
  __shared__ int slots[64];
  const CacheView& cv = p.cache;
  const WeightSeq& sq = p.s[find_seq(p.s, p.n_seq, (int)blockIdx.x, [](const WeightSeq& s) { return s.unit0; })];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = lane64(), n = lane & 15, g = lane >> 4;
  const int u = (int)blockIdx.x - sq.unit0;
  const int tile = u / sq.n_part, part = u - tile * sq.n_part;
  const int key0 = tile * 64;
  if (threadIdx.x < 64)
    slots[threadIdx.x] = key0 + (int)threadIdx.x < sq.kv_len
                             ? cache_slot(cv.table, sq.b, cv.max_pages, cv.page_size, cv.num_pages, key0 + (int)threadIdx.x)
                             : -1;
  __syncthreads();
  const int row_b = cv.Hkv * (D / 2), row_s = cv.Hkv * (D / 32);
  const int before = sq.kv_len - sq.q_len;
  const int i0 = key0 > before ? key0 - before : 0;           // first query that sees any of the keys
  const int rows = (sq.q_len - i0) * p.group;
  const int n_rt = (rows + 15) >> 4;
  // wavefronts of all the parts share (head, row tile): heads first, then slices of the row tiles
  const int all = sq.n_part * kWaves, w = part * kWaves + wave;
  const int nh = cv.Hkv < all ? cv.Hkv : all;
  const int slices = all / nh;
  f4 acc[4];
#pragma unroll
  for (int a = 0; a < 4; ++a) acc[a] = f4{0.f, 0.f, 0.f, 0.f};

  if (w < nh * slices) {
    const int rs = w / nh;
    for (int head = w - rs * nh; head < cv.Hkv; head += nh) {
      b8 kf[4][NS];
      {
        typedef uint32_t kvec __attribute__((ext_vector_type(NS)));
        const int sl = slots[lane];
        uint32_t by = 0;
        if (sl >= 0) {
          const uint8_t* a = cv.k_scales + (int64_t)sl * row_s + head * (D / 32);
          if constexpr (D == 128) by = *reinterpret_cast<const uint32_t*>(a);
          else by = *reinterpret_cast<const uint16_t*>(a);
        }
        wave_sync();
        sc[wave][lane] = by;
        wave_sync();
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          const int ks = slots[16 * a + n];
          const kvec x = *reinterpret_cast<const kvec*>(cv.k_codes + (int64_t)(ks < 0 ? 0 : ks) * row_b + head * (D / 2) +
                                                        g * (D / 8));
          const float s = mx_scale(sc[wave][16 * a + n], 8 * (D == 128 ? g : g >> 1));
#pragma unroll
          for (int e = 0; e < NS; ++e) kf[a][e] = mx8(x[e], s);
        }
      }
      for (int rt = rs; rt < n_rt; rt += slices) {
        int r = rt * 16 + n;
        const bool ok = r < rows;
        r = ok ? r : rows - 1;
        const int query = i0 + r / p.group, qh = head * p.group + r % p.group;
        const int64_t tok = sq.q_row0 + query;
        const float lse = p.lse[tok * p.Hq + qh];
        // a row without a normaliser (it saw no key) gives nothing
        const float ls = ok && lse > -INFINITY ? lse : INFINITY;
        b8 qf[TERMS][NS];
        const int64_t at = tok * p.q_stride + (int64_t)qh * D + g * (D / 4);
        const f4* src = reinterpret_cast<const f4*>(static_cast<const float*>(p.q) + at);
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          const f4 x0 = src[2 * s], x1 = src[2 * s + 1];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float tt[3];
            split3(e < 4 ? x0[e & 3] : x1[e & 3], tt);
#pragma unroll
            for (int k = 0; k < TERMS; ++k) qf[k][s][e] = (__bf16)tt[k];
          }
        }
        f4 s4[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          s4[a] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = TERMS - 1; k >= 0; --k)
#pragma unroll
            for (int s = 0; s < NS; ++s) s4[a] = mfma_bf16(kf[a][s], qf[k][s], s4[a]);
        }
        const int pos = before + query;
        // the first row of the tile sees the fewest keys
        if (before + i0 + (rt * 16) / p.group < key0 + 63) {
#pragma unroll
          for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int e = 0; e < 4; ++e) s4[a][e] = key0 + 16 * a + 4 * g + e > pos ? -INFINITY : s4[a][e];
        }
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[a][e] += weight_of(s4[a][e], p.scale, ls);
      }
    }
  }
  // rows of the wavefront sit in the 16 lanes of a group
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float x = acc[a][e];
#pragma unroll
      for (int m = 1; m < 16; m <<= 1) x += __shfl_xor(x, m);
      if (n == 0) sums[wave][16 * a + 4 * g + e] = x;
    }
  __syncthreads();
  if (threadIdx.x >= 64) return;
  float x = 0.f;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) x += sums[i][threadIdx.x];
  if (sq.n_part > 1) {
    p.part[((int64_t)sq.part0 + u) * 64 + threadIdx.x] = x;
  } else {
    const int key = key0 + (int)threadIdx.x, sl = slots[threadIdx.x];
    if (sl >= 0) p.acc_out[sl] = (key < before && p.acc != nullptr ? p.acc[sl] : 0.f) + x;
  }
}

__global__ __launch_bounds__(64) void weights_join_kernel(const WeightArgs p) {
  const CacheView& cv = p.cache;
  const WeightSeq& sq = p.s[find_seq(p.s, p.n_seq, (int)blockIdx.x, [](const WeightSeq& s) { return s.tile0; })];
  if (sq.n_part <= 1) return;
  const int tile = (int)blockIdx.x - sq.tile0, key = tile * 64 + (int)threadIdx.x;
  if (key >= sq.kv_len) return;
  const int sl = cache_slot(cv.table, sq.b, cv.max_pages, cv.page_size, cv.num_pages, key);
  if (sl < 0) return;
  float x = 0.f;
  for (int i = 0; i < sq.n_part; ++i) x += p.part[((int64_t)sq.part0 + (int64_t)tile * sq.n_part + i) * 64 + threadIdx.x];
  p.acc_out[sl] = (key < sq.kv_len - sq.q_len && p.acc != nullptr ? p.acc[sl] : 0.f) + x;
}

}  // namespace

hipError_t launch_weights(int d, const WeightArgs& p, hipStream_t s) {
  const dim3 grid((unsigned)p.n_units), block(64 * kWaves);
  if (d == 128) weights_kernel<128><<<grid, block, 0, s>>>(p);
  else weights_kernel<64><<<grid, block, 0, s>>>(p);
  return hipGetLastError();
}

hipError_t launch_weights_join(const WeightArgs& p, hipStream_t s) {
  weights_join_kernel<<<dim3((unsigned)p.n_tiles), dim3(64), 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace dosa
