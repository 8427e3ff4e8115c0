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
// a lower bound of the threshold from the lanes' largest scores leaves few
// candidates, a few a lane, among which the threshold is built bit by bit; the
// chosen blocks are written in ascending order by counting lanes.  Of scores equal
// to the threshold the lowest blocks are taken.
//
// 4096 queries, 32 heads on 8, d = 128, 16 of up to 1024 blocks: 93 to 104 us, of
// which the scores take 70.  Their bound is the first-level cache: the product
// wants 16 bytes of 16 rows at a time, and each of those counts as an access of its
// own (3.9e7 in all, 64 us at one a cycle and CU; which is why a wavefront's pages and
// scales are read a block a lane and exchanged).  Four row tiles a workgroup would halve them, but their scores leave
// half the wavefronts (125 us).  Decode of 32 sequences x 2 queries, 64 heads on 8, 32
// of up to 1600 blocks: 17 us, latency: pages, scales and codes in turn.  One query
// over 16384 blocks 94 us: a kv head is one workgroup's.  Choices of more than 64 of
// the scored blocks have no lower bound and build the threshold over all scores: 4096
// queries over 2048 blocks in groups of 8, 63 of them 0.32 ms, 128 0.74, 256 0.77.
#include <atomic>

#include "attn_device.h"
#include "pages_internal.h"

namespace dosa {

namespace {

constexpr float kLargest = 0x1.fffffep127f;
constexpr int kFew = 256;                // scores that a wavefront chooses from in registers
constexpr int kCols = 4;                 // column tiles a wavefront has in flight, one block a lane

__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// The value of lane l^16 (l^32).
__device__ __forceinline__ float other_half16(float x) {
  const uint32_t u = __float_as_uint(x);
  auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return (lane64() & 16) != 0 ? __uint_as_float(r[0]) : __uint_as_float(r[1]);
}
__device__ __forceinline__ float other_half32(float x) {
  const uint32_t u = __float_as_uint(x);
  auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return (lane64() & 32) != 0 ? __uint_as_float(r[0]) : __uint_as_float(r[1]);
}

// 16 elements of a query row as floats.
__device__ __forceinline__ void row16(bool f32, const void* q, int64_t at, float* x) {
  if (f32) {
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

// The largest number that `need` scores reach, built bit by bit from above;
// count(x): scores that reach x; reach: how many reach 0.  Stops where exactly
// `need` reach what there is of it.
template <class Count>
__device__ __forceinline__ uint32_t kth(Count count, int need, int reach) {
  uint32_t t = 0;
  for (int b = 31; b >= 0; --b) {
    const int c = count(t | (1u << b));
    if (c >= need) {
      t |= 1u << b;
      reach = c;
      if (reach == need) break;
    }
  }
  return t;
}

// Wavefronts of a workgroup of MT row tiles: with few tokens they are there for
// the loads.
constexpr int select_waves(int mt) { return mt == 1 ? 16 : 8; }

// MT: 16-row tiles of the workgroup; PAD: rows of a token; MANY: groups of more than 16 heads, several
// products of one tile.
template <int D, int MT, int PAD, bool MANY>
__global__ __launch_bounds__(64 * select_waves(MT)) void select_kernel(const SelectArgs p) {
  constexpr int KS = D / 64, kWaves = select_waves(MT);
  extern __shared__ uint32_t scores[];
  __shared__ i4 qcodes[MANY ? 1 : MT][KS][64];
  __shared__ __attribute__((aligned(16))) float qfactor[MANY ? 1 : MT][16];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = lane64(), n = lane & 15, g = lane >> 4, waves = kWaves;
  const SelectSeq& sq = p.s[find_seq(p.s, p.n_seq, (int)blockIdx.x, [](const SelectSeq& s) { return s.unit0; })];
  constexpr int PER = 16 / PAD, TW = PER * MT;
  const int u = (int)blockIdx.x - sq.unit0, head = u % p.Hkv;
  const int tiles = (sq.q_len + TW - 1) / TW, tok0 = (tiles - 1 - u / p.Hkv) * TW;   // last tokens first: they see the most blocks
  const int n_tok = min(TW, sq.q_len - tok0), pos0 = sq.kv_len - sq.q_len + tok0;
  const int own_last = (pos0 + n_tok - 1) >> p.lb;
  const int col0 = p.sinks & ~15, col_end = own_last - p.local + 1;

  if (own_last >= p.topn) {
    // ---- scores of blocks col0..col_end-1 ----
    auto q_at = [&](int i, int pass) -> int64_t {
      const int tok = min(i * PER + n / PAD, n_tok - 1), h = min(16 * pass + n % PAD, p.group - 1);
      return (int64_t)(sq.q_row0 + tok0 + tok) * p.q_stride + (int64_t)(head * p.group + h) * D + 16 * g;
    };
    // exponent of row n of tile i, its elements
    auto exponent = [&](int i, int pass, float x[KS][16]) -> int {
      float top = 0.f;                   // a maximum that a NaN goes through, two elements an instruction
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        row16(p.f32 != 0, p.q, q_at(i, pass) + 64 * s, x[s]);
#pragma unroll
        for (int e = 0; e < 16; ++e) top = __builtin_elementwise_maximum(top, fabsf(x[s][e]));
      }
      if (!(top <= kLargest)) {          // some element is not finite
        top = 0.f;
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            x[s][e] = x[s][e] == x[s][e] ? fminf(fmaxf(x[s][e], -kLargest), kLargest) : 0.f;
            top = fmaxf(top, fabsf(x[s][e]));
          }
      }
      top = max_groups(top);
      const int e = (int)((__float_as_uint(top) + (1u << 16)) >> 23) - 127 - 6;
      return e < -126 ? -126 : e;
    };
    auto round8 = [&](const float x[KS][16], int e, i4* codes) {
      const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t y = 0;
#pragma unroll
          for (int b = 0; b < 4; ++b) y |= ((uint32_t)(int)rintf(x[s][4 * w + b] * inv) & 255u) << (8 * b);
          codes[s][w] = (int)y;
        }
    };
    auto factor = [&](int e, int most) -> float {      // of a head whose exponent is e
      const int rel = e - most;
      return __uint_as_float((uint32_t)(127 + (rel < -100 ? -100 : rel)) << 23);
    };
    int most = -126;                     // MANY: largest exponent of the token's heads
    if constexpr (MANY) {
      for (int pass = 0; pass < p.passes; ++pass) {
        float x[KS][16];
        most = max(most, exponent(0, pass, x));
      }
      for (int w = 1; w < 16; w <<= 1) most = max(most, __shfl_xor(most, w));
    } else {
      // a wavefront rounds the rows of a tile for all of them
      for (int i = wave; i < MT; i += waves) {
        float x[KS][16];
        i4 codes[KS];
        const int e = exponent(i, 0, x);
        int m = e;
        for (int w = 1; w < PAD; w <<= 1) m = max(m, __shfl_xor(m, w));
        round8(x, e, codes);
#pragma unroll
        for (int s = 0; s < KS; ++s) qcodes[i][s][lane] = codes[s];
        if (g == 0) qfactor[i][n] = factor(e, m);
      }
      __syncthreads();
    }
    for (int pass = 0; pass < (MANY ? p.passes : 1); ++pass) {
      i4 qa[MT][KS];
      f4 rs[MT];
      if constexpr (MANY) {
        float x[KS][16];
        const int e = exponent(0, pass, x);
        round8(x, e, qa[0]);
        const float f = factor(e, most);
#pragma unroll
        for (int r = 0; r < 4; ++r) rs[0][r] = __shfl(f, 4 * g + r);
      } else {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
          for (int s = 0; s < KS; ++s) qa[i][s] = qcodes[i][s][lane];
          rs[i] = *reinterpret_cast<const f4*>(&qfactor[i][4 * g]);
        }
      }
      for (int ct = col0 + 16 * kCols * wave; ct < col_end; ct += 16 * kCols * waves) {
        // a lane a block: its page and scale, which the lanes of its column then get
        i4 kb[kCols][KS];
        int sb[kCols], e;
        {
          const int j = min(ct + lane, col_end - 1), pg = p.div.quot(j);
          const int page = p.table[(int64_t)sq.b * p.max_pages + pg];
          const bool there = (uint32_t)page < (uint32_t)p.num_pages;
          const int at = (there ? page : 0) * (int)p.div.by + (j - pg * (int)p.div.by);
          e = there ? (int)p.scales[(int64_t)at * p.Hkv + head] : -1;
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            const int64_t row = (int64_t)__shfl(at, 16 * c + n) * p.Hkv + head;
#pragma unroll
            for (int s = 0; s < KS; ++s) kb[c][s] = *reinterpret_cast<const i4*>(p.codes + row * D + 64 * s + 16 * g);
          }
        }
#pragma unroll
        for (int c = 0; c < kCols; ++c) sb[c] = __shfl(e, 16 * c + n);
#pragma unroll
        for (int c0 = 0; c0 < kCols; c0 += 2) {
          i4 acc[2][MT];
#pragma unroll
          for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int i = 0; i < MT; ++i)
                acc[c][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(qa[i][s], kb[c0 + c][s], s == 0 ? i4{0, 0, 0, 0} : acc[c][i], 0, 0, 0);
          // rows 4g..4g+3 of a tile, block j: the maximum over a token's rows
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int j = ct + 16 * (c0 + c) + n;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              float v[4];
#pragma unroll
              for (int r = 0; r < 4; ++r) v[r] = (float)acc[c][i][r] * rs[i][r];
              if constexpr (PAD >= 2) v[0] = fmaxf(v[0], v[1]), v[2] = fmaxf(v[2], v[3]);
              if constexpr (PAD >= 4) v[0] = fmaxf(v[0], v[2]);
              if constexpr (PAD >= 8) v[0] = fmaxf(v[0], other_half16(v[0]));
              if constexpr (PAD >= 16) v[0] = fmaxf(v[0], other_half32(v[0]));
#pragma unroll
              for (int r = 0; r < 4; r += (PAD < 4 ? PAD : 4)) {
                const float x = sb[c0 + c] < 0 ? -INFINITY : ldexpf(v[r], sb[c0 + c] - 142) + 0.f;     // -0 is 0
                uint32_t key = ordered(x);
                uint32_t* to = scores + (i * PER + (4 * g + r) / PAD) * p.stride + (j - col0);
                if ((PAD <= 4 || ((4 * g) & (PAD - 1)) == 0) && j < col_end) {
                  if (MANY && pass > 0) key = max(key, *to);
                  *to = key;
                }
              }
            }
          }
        }
      }
    }
  }
  __syncthreads();

  // ---- a wavefront a token ----
  __shared__ uint32_t few[kWaves][kFew];           // scores that may be chosen
  __shared__ uint16_t few_at[kWaves][kFew];        // their blocks, from `lo` on
  for (int tok = wave; tok < n_tok; tok += waves) {
    const int own = (pos0 + tok) >> p.lb;
    int32_t* out = p.idx + ((int64_t)(sq.q_row0 + tok0 + tok) * p.Hkv + head) * p.topn;
    if (own < p.topn) {
      for (int i = lane; i < p.topn; i += 64) out[i] = i <= own ? i : -1;
      continue;
    }
    const int lo = p.sinks, hi = own - p.local + 1, need = p.topn - p.sinks - p.local, chunks = (hi - lo + 63) >> 6;
    for (int i = lane; i < p.sinks; i += 64) out[i] = i;
    for (int i = lane; i < p.local; i += 64) out[p.topn - p.local + i] = own - p.local + 1 + i;
    if (need == 0) continue;
    out += p.sinks;
    const uint32_t* row = scores + tok * p.stride + (lo - col0) + lane;
    auto at = [&](int i) -> uint32_t { return lo + 64 * i + lane < hi ? row[64 * i] : 0u; };   // 0 is below every score
    auto each = [&](auto use) {          // four reads under way
      for (int i0 = 0; i0 < chunks; i0 += 4) {
        uint32_t x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) x[u] = at(i0 + u);
#pragma unroll
        for (int u = 0; u < 4; ++u) use(x[u], i0 + u);
      }
    };
    // Of the lanes' largest scores the need-th largest is reached by `need` scores at least: a lower bound of
    // the threshold, and one that few others reach.
    uint32_t least = 0;
    if (need <= 64) {
      uint32_t top = 0;
      each([&](uint32_t x, int) { top = max(top, x); });
      least = kth([&](uint32_t x) -> int { return __popcll(__ballot(top >= x)); }, need, need);
    }
    int n_few = 0;
    if (least != 0) {
      each([&](uint32_t x, int i) {
        const uint64_t in = __ballot(x >= least);
        const int to = n_few + below(in);
        if (x >= least && to < kFew) {
          few[wave][to] = x;
          few_at[wave][to] = (uint16_t)(64 * i + lane);
        }
        n_few += __popcll(in);
      });
    }
    if (least != 0 && n_few <= kFew) {
      wave_sync();
      uint32_t v[kFew / 64], blk[kFew / 64];
#pragma unroll
      for (int i = 0; i < kFew / 64; ++i) {
        const bool in = 64 * i + lane < n_few;
        v[i] = in ? few[wave][64 * i + lane] : 0u;
        blk[i] = in ? few_at[wave][64 * i + lane] : 0u;
      }
      wave_sync();
      auto reach = [&](uint32_t y) -> int {
        int c = __popcll(__ballot(v[0] >= y));
#pragma unroll
        for (int i = 1; i < kFew / 64; ++i)
          if (n_few > 64 * i) c += __popcll(__ballot(v[i] >= y));
        return c;
      };
      const uint32_t t = kth(reach, need, n_few);
      int ties = need - (t == 0xffffffffu ? 0 : reach(t + 1)), done = 0;
#pragma unroll
      for (int i = 0; i < kFew / 64; ++i) {
        if (n_few <= 64 * i) break;
        const uint64_t eq = __ballot(v[i] == t);
        const bool take = v[i] > t || (v[i] == t && below(eq) < ties);
        const uint64_t all = __ballot(take);
        if (take) out[done + below(all)] = lo + (int)blk[i];
        done += __popcll(all);
        ties -= __popcll(eq);
      }
      continue;
    }
    // many blocks to choose, or many equal scores
    auto count = [&](uint32_t y) -> int {
      int c = 0;
      each([&](uint32_t x, int) { c += __popcll(__ballot(x >= y)); });
      return c;
    };
    const uint32_t t = kth(count, need, hi - lo);
    int ties = need - (t == 0xffffffffu ? 0 : count(t + 1)), done = 0;
    for (int i = 0; i < chunks; ++i) {
      const uint32_t x = at(i);
      const uint64_t eq = __ballot(x == t);
      const bool take = x > t || (x == t && below(eq) < ties);
      const uint64_t all = __ballot(take);
      if (take) out[done + below(all)] = lo + 64 * i + lane;
      done += __popcll(all);
      ties -= __popcll(eq);
    }
  }
}

template <int D, int MT, int PAD, bool MANY>
hipError_t go(const SelectArgs& p, hipStream_t s) {
  const unsigned lds = (unsigned)(16 / PAD * MT) * (unsigned)p.stride * 4u;
  if (lds > (32u << 10)) {
    // The limit is the function's, not the launch's: it is raised once on each device, to the most that a launch can
    // ask for, so that no call lowers what another thread's is about to use.
    constexpr int most = 16 / PAD * MT == 1 ? (int)(kSelectBlocks + 16) * 4 : (int)kSelectLds;
    static std::atomic<uint64_t> raised{0};
    int dev;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if ((raised.load(std::memory_order_acquire) & bit) == 0) {
      e = hipFuncSetAttribute(reinterpret_cast<const void*>(&select_kernel<D, MT, PAD, MANY>),
                              hipFuncAttributeMaxDynamicSharedMemorySize, most);
      if (e != hipSuccess) return e;
      raised.fetch_or(bit, std::memory_order_release);
    }
  }
  select_kernel<D, MT, PAD, MANY><<<dim3((unsigned)p.n_units), dim3(64 * select_waves(MT)), lds, s>>>(p);
  return hipGetLastError();
}

template <int D, int MT>
hipError_t go_pad(const SelectArgs& p, hipStream_t s) {
  switch (p.pad) {
    case 1: return go<D, MT, 1, false>(p, s);
    case 2: return go<D, MT, 2, false>(p, s);
    case 4: return go<D, MT, 4, false>(p, s);
    case 8: return go<D, MT, 8, false>(p, s);
    default: return go<D, MT, 16, false>(p, s);
  }
}

template <int D>
hipError_t go_tiles(int tiles, const SelectArgs& p, hipStream_t s) {
  if (p.passes > 1) return go<D, 1, 16, true>(p, s);
  return tiles == 2 ? go_pad<D, 2>(p, s) : go_pad<D, 1>(p, s);
}

}  // namespace

hipError_t launch_block_select(int d, int tiles, const SelectArgs& p, hipStream_t s) {
  if (p.n_units == 0) return hipSuccess;
  return d == 128 ? go_tiles<128>(tiles, p, s) : go_tiles<64>(tiles, p, s);
}

}  // namespace dosa
