// Choice of a few blocks per query and kv head by a cheap score.
//
//   score_j = 2^(e_j - 142) max_h 2^max(f_h - f, -100) <a_h, c_j>
//
// over the group's query heads h: c_j, 2^(e_j - 127) the summary of block j
// (integers and a scale), a_h, 2^f_h the query rounded the same way, f = max f_h.
// Only the order of the scores of a row matters, so the queries' common factor
// 2^f is left out and 2^-15 keeps every finite summary's score finite.  A dot is
// an integer below 2^21 and all factors are powers of two: the fp32 score is exact
// (one rounding where it is subnormal), whatever the order of the sums, and so is
// the choice.
//
// A workgroup takes a few tokens of one kv head.  Their heads, padded to a power
// of two by repeating the last (which leaves the maximum alone), are the rows of
// 16x16x64 products of 8-bit integers, the blocks their columns; the scores go to
// LDS as unsigned numbers of the same order.  Then a wavefront takes a token:
// the threshold is built bit by bit from above until exactly the wanted number of
// scores reaches it, and the chosen blocks are written in ascending order by
// counting lanes.  Of scores equal to the threshold the lowest blocks are taken.
#include "attn_device.h"
#include "pages_internal.h"

namespace dosa {

namespace {

constexpr int kWavesS = 4;
constexpr int kCols = 4;                 // column tiles a wavefront has in flight
constexpr int kRegs = 16;                // scores of a lane in registers

__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ int below(uint64_t mask) {        // lanes of the mask in front of this one
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0u));
}

// 16 elements of a query row as floats.
template <bool F32>
__device__ __forceinline__ void row16(const void* q, int64_t at, float* x) {
  if constexpr (F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f4 y = reinterpret_cast<const f4*>(static_cast<const float*>(q) + at)[i];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[4 * i + e] = y[e];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const i4 y = reinterpret_cast<const i4*>(static_cast<const uint16_t*>(q) + at)[i];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[8 * i + 2 * e] = __uint_as_float((uint32_t)y[e] << 16);
        x[8 * i + 2 * e + 1] = __uint_as_float((uint32_t)y[e] & 0xffff0000u);
      }
    }
  }
}

template <bool F32, int D, int MT>
__global__ __launch_bounds__(64 * kWavesS) void select_kernel(const SelectArgs p) {
  constexpr int KS = D / 64;
  extern __shared__ uint32_t scores[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = lane64(), n = lane & 15, g = lane >> 4;
  const SelectSeq& sq = p.s[find_seq(p.s, p.n_seq, (int)blockIdx.x, [](const SelectSeq& s) { return s.unit0; })];
  const int per = 16 / p.pad, TW = per * MT;
  const int u = (int)blockIdx.x - sq.unit0, head = u % p.Hkv;
  const int tiles = (sq.q_len + TW - 1) / TW, tok0 = (tiles - 1 - u / p.Hkv) * TW;   // last tokens first: they see the most blocks
  const int n_tok = min(TW, sq.q_len - tok0), pos0 = sq.kv_len - sq.q_len + tok0;
  const int own_last = (pos0 + n_tok - 1) >> p.lb;
  const int col0 = p.sinks & ~15, col_end = own_last - p.local + 1;

  if (own_last >= p.topn) {
    // ---- scores of blocks col0..col_end-1 ----
    auto q_at = [&](int i, int pass) -> int64_t {
      const int tok = min(i * per + n / p.pad, n_tok - 1), h = min(16 * pass + n % p.pad, p.group - 1);
      return (int64_t)(sq.q_row0 + tok0 + tok) * p.q_stride + (int64_t)(head * p.group + h) * D + 16 * g;
    };
    // exponent of row n of tile i
    auto exponent = [&](int i, int pass, float x[KS][16]) -> int {
      float top = 0.f;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        row16<F32>(p.q, q_at(i, pass) + 64 * s, x[s]);
#pragma unroll
        for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(x[s][e]));
      }
      top = max_groups(top);
      const int e = (int)((__float_as_uint(top) + (1u << 16)) >> 23) - 127 - 6;
      return e < -126 ? -126 : e;
    };
    int most[MT];                        // largest exponent of the token's heads
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      most[i] = -126;
      for (int pass = 0; pass < p.passes; ++pass) {
        float x[KS][16];
        most[i] = max(most[i], exponent(i, pass, x));
      }
      for (int w = 1; w < p.pad; w <<= 1) most[i] = max(most[i], __shfl_xor(most[i], w));
    }
    for (int pass = 0; pass < p.passes; ++pass) {
      i4 qa[MT][KS];
      float rs[MT][4];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        float x[KS][16];
        const int e = exponent(i, pass, x);
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t y = 0;
#pragma unroll
            for (int b = 0; b < 4; ++b) y |= ((uint32_t)(int)rintf(x[s][4 * w + b] * inv) & 255u) << (8 * b);
            qa[i][s][w] = (int)y;
          }
        const int rel = e - most[i];
        const float f = __uint_as_float((uint32_t)(127 + (rel < -100 ? -100 : rel)) << 23);
#pragma unroll
        for (int r = 0; r < 4; ++r) rs[i][r] = __shfl(f, 4 * g + r);
      }
      for (int ct = col0 + 16 * kCols * wave; ct < col_end; ct += 16 * kCols * kWavesS) {
        i4 kb[kCols][KS];
        int sb[kCols];
        bool bad[kCols];
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const int j = min(ct + 16 * c + n, col_end - 1), pg = p.div.quot(j);
          int page = p.table[(int64_t)sq.b * p.max_pages + pg];
          bad[c] = (uint32_t)page >= (uint32_t)p.num_pages;
          page = bad[c] ? 0 : page;
          const int64_t at = ((int64_t)page * p.div.by + (j - pg * (int)p.div.by)) * p.Hkv + head;
          sb[c] = p.scales[at];
#pragma unroll
          for (int s = 0; s < KS; ++s) kb[c][s] = *reinterpret_cast<const i4*>(p.codes + at * D + 64 * s + 16 * g);
        }
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const int j = ct + 16 * c + n;
          if (ct + 16 * c >= col_end) break;
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            i4 acc = {0, 0, 0, 0};
#pragma unroll
            for (int s = 0; s < KS; ++s) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(qa[i][s], kb[c][s], acc, 0, 0, 0);
            // rows 4g..4g+3 of the tile, block j: the maximum over a token's rows
            float v[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = (float)acc[r] * rs[i][r];
            if (p.pad >= 2) v[0] = fmaxf(v[0], v[1]), v[2] = fmaxf(v[2], v[3]);
            if (p.pad >= 4) v[0] = fmaxf(v[0], v[2]);
            if (p.pad >= 8) v[0] = fmaxf(v[0], __shfl_xor(v[0], 16));
            if (p.pad >= 16) v[0] = fmaxf(v[0], __shfl_xor(v[0], 32));
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              if ((r & (p.pad - 1)) != 0) continue;
              const float x = bad[c] ? -INFINITY : ldexpf(v[r], sb[c] - 142) + 0.f;     // -0 is 0
              uint32_t key = ordered(x);
              uint32_t* to = scores + (i * per + (4 * g + r) / p.pad) * p.stride + (j - col0);
              if (((4 * g + r) & (p.pad - 1)) == 0 && j < col_end) {
                if (pass > 0) key = max(key, *to);
                *to = key;
              }
            }
          }
        }
      }
    }
  }
  __syncthreads();

  // ---- a wavefront a token ----
  for (int tok = wave; tok < n_tok; tok += kWavesS) {
    const int own = (pos0 + tok) >> p.lb;
    int32_t* out = p.idx + ((int64_t)(sq.q_row0 + tok0 + tok) * p.Hkv + head) * p.topn;
    if (own < p.topn) {
      for (int i = lane; i < p.topn; i += 64) out[i] = i <= own ? i : -1;
      continue;
    }
    const int lo = p.sinks, hi = own - p.local + 1, need = p.topn - p.sinks - p.local, chunks = (hi - lo + 63) >> 6;
    const uint32_t* row = scores + tok * p.stride + (lo - col0) + lane;
    uint32_t v[kRegs];
#pragma unroll
    for (int i = 0; i < kRegs; ++i) v[i] = lo + 64 * i + lane < hi ? row[64 * i] : 0u;     // 0 is below every score
    auto at = [&](int i) -> uint32_t { return lo + 64 * i + lane < hi ? row[64 * i] : 0u; };
    auto count = [&](uint32_t least) -> int {
      int c = 0;
#pragma unroll
      for (int i = 0; i < kRegs; ++i)
        if (i < chunks) c += __popcll(__ballot(v[i] >= least));
      for (int i = kRegs; i < chunks; ++i) c += __popcll(__ballot(at(i) >= least));
      return c;
    };
    uint32_t least = 0;                  // the largest number that `need` scores reach
    int reach = hi - lo;
    for (int b = 31; b >= 0 && reach != need; --b) {
      const int c = count(least | (1u << b));
      if (c >= need) {
        least |= 1u << b;
        reach = c;
      }
    }
    int ties = reach == need ? need : need - count(least + 1);     // of the scores equal to `least`
    int done = p.sinks;
    auto put = [&](uint32_t x, int i) {
      const uint64_t eq = __ballot(x == least && x != 0u);
      const bool take = x > least || (x == least && x != 0u && below(eq) < ties);
      const uint64_t all = __ballot(take);
      if (take) out[done + below(all)] = lo + 64 * i + lane;
      done += __popcll(all);
      ties -= __popcll(eq);
    };
    if (need > 0) {
#pragma unroll
      for (int i = 0; i < kRegs; ++i)
        if (i < chunks) put(v[i], i);
      for (int i = kRegs; i < chunks; ++i) put(at(i), i);
    }
    for (int i = lane; i < p.sinks; i += 64) out[i] = i;
    for (int i = lane; i < p.local; i += 64) out[p.topn - p.local + i] = own - p.local + 1 + i;
  }
}

template <bool F32, int D, int MT>
hipError_t go(const SelectArgs& p, hipStream_t s) {
  const unsigned lds = (unsigned)(16 / p.pad * MT) * (unsigned)p.stride * 4u;
  if (lds > (64u << 10)) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&select_kernel<F32, D, MT>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  select_kernel<F32, D, MT><<<dim3((unsigned)p.n_units), dim3(64 * kWavesS), lds, s>>>(p);
  return hipGetLastError();
}

template <bool F32, int D>
hipError_t go_tiles(int tiles, const SelectArgs& p, hipStream_t s) {
  return tiles == 4 ? go<F32, D, 4>(p, s) : tiles == 2 ? go<F32, D, 2>(p, s) : go<F32, D, 1>(p, s);
}

}  // namespace

hipError_t launch_block_select(bool f32, int d, int tiles, const SelectArgs& p, hipStream_t s) {
  if (p.n_units == 0) return hipSuccess;
  if (f32) return d == 128 ? go_tiles<true, 128>(tiles, p, s) : go_tiles<true, 64>(tiles, p, s);
  return d == 128 ? go_tiles<false, 128>(tiles, p, s) : go_tiles<false, 64>(tiles, p, s);
}

}  // namespace dosa
