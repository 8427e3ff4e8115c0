// Eviction: the choice of the keys that stay, and the move of their rows.
//
// A key's rank is its accumulated weight, above all others if it is protected
// (one of the first `prefix` or the latest `window` tokens of the text); the
// new_len keys of highest rank stay, ties to the lower index.  Kept keys in
// front of the new end do not move; the n-th kept key behind it (in order)
// moves into the n-th hole in front of it.  So a periodic eviction of a few
// keys moves a few rows, and no row is read from a place another is written
// to: the moves are independent.  An index in front of the new end whose table
// entry names no page holds nothing and is no hole: it ranks with the protected
// keys, so that no key moves to where it would be lost.
#include "attn_device.h"

namespace dosa {

namespace {

constexpr int kThreads = 1024, kEvWaves = kThreads / 64;

__device__ __forceinline__ uint32_t rank_of(const EvictArgs& p, const EvictSeq& s, float acc, int pos) {
  const uint32_t u = __float_as_uint(acc + 0.f);        // -0 ranks as 0
  uint32_t r = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
  r = r < 1u ? 1u : (r > 0xfffffffeu ? 0xfffffffeu : r);
  return pos < p.prefix || (int64_t)pos >= (int64_t)s.seen - p.window ? 0xffffffffu : r;
}

// Ranks of N rounds from round i0 on, as unsigned numbers: all ones if protected
// or without a page in front of the new end, 0 without a page behind it, else
// the order of the weight's bits.  Each kind of
// load is issued for all rounds before any is used, without branches, since
// the chain page, weight, position is all latency.  With pages of a multiple
// of 64 keys a wavefront's keys of a round lie in one page.
template <int N>
__device__ __forceinline__ void load_ranks(const EvictArgs& p, const EvictSeq& s, int i0, int wave, uint32_t* rk) {
  const int32_t* table = p.table + (int64_t)s.b * p.max_pages;
  const bool whole = (p.page_size & 63) == 0;
  int slot[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int key0 = (i0 + i) * 1024 + 64 * wave, lane = lane64();
    int at = whole ? key0 : key0 + lane;
    at = at < s.kv_len ? at : s.kv_len - 1;
    const int pg = at / p.page_size;
    const int page = whole ? table[__builtin_amdgcn_readfirstlane(pg)] : table[pg];
    const int in = whole ? key0 + lane - pg * p.page_size : at - pg * p.page_size;
    slot[i] = key0 + lane < s.kv_len && (uint32_t)page < (uint32_t)p.num_pages ? page * p.page_size + in : -1;
  }
  float acc[N];
  int pos[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    acc[i] = p.acc[slot[i] < 0 ? 0 : slot[i]];
    pos[i] = (i0 + i) * 1024 + 64 * wave + lane64();
  }
  if (p.pos != nullptr) {
#pragma unroll
    for (int i = 0; i < N; ++i) pos[i] = p.pos[slot[i] < 0 ? 0 : slot[i]];
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const bool front = (i0 + i) * 1024 + 64 * wave + lane64() < s.new_len;
    rk[i] = slot[i] < 0 ? (front ? 0xffffffffu : 0u) : rank_of(p, s, acc[i], pos[i]);
  }
}

// Exclusive sums over cnt[0..n), n <= kThreads, in place; one workgroup.
__device__ __forceinline__ void block_scan(int* cnt, int n, int* sh) {
  const int tid = threadIdx.x, lane = lane64(), wave = tid >> 6;
  const int v = tid < n ? cnt[tid] : 0;
  int x = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(x, d);
    x += lane >= d ? y : 0;
  }
  if (lane == 63) sh[wave] = x;
  __syncthreads();
  int before = 0;
#pragma unroll
  for (int i = 0; i < kEvWaves; ++i) before += i < wave ? sh[i] : 0;
  if (tid < n) cnt[tid] = before + x - v;
  __syncthreads();
}

// One workgroup chooses a sequence's keys.  A wavefront's 64 keys of round i
// are i * 1024 + 64 * wave ..., a thread keeps the ranks of its first PER
// rounds in registers; longer sequences keep theirs in the workspace.  The
// threshold, the new_len-th largest rank, is found digit by digit (8 bits)
// with a histogram of 32 copies, one per LDS bank, so that a lane meets at most
// one other of its wavefront in a counter however the weights are distributed.
// Then a prefix sum over (round, wavefront) counts numbers, in order of the
// index, the holes in front of the new end and the keys that move from behind
// it: as many of one as of the other, holes first, so one list holds both.
// Only if not all keys that equal the threshold stay does another prefix sum
// number those.
// Bound by latency for short sequences (16 of 4160 keys: 16 us, a few dependent
// loads and about twenty barriers), by the one CU's instructions for long ones
// (4 of up to 65536 keys: 86 us).
template <int PER>
__global__ __launch_bounds__(kThreads) void evict_select_kernel(const EvictArgs p) {
  __shared__ uint32_t hist[256 * 32];
  __shared__ uint32_t tot[256];
  __shared__ int sh[kEvWaves];
  __shared__ int carry[2];
  __shared__ uint32_t sel[3];
  const EvictSeq& s = p.s[blockIdx.x];
  const int tid = threadIdx.x, lane = lane64(), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int32_t* out = p.out_src + (int64_t)s.b * p.out_stride;
  int32_t* ws = p.ws + s.ws_off;
  int32_t* list = ws + kEvictHead;         // holes, then keys that move
  uint32_t* far = reinterpret_cast<uint32_t*>(list + 2 * s.cap);    // ranks of the rounds from PER on
  const int rounds = (s.kv_len + kThreads - 1) / kThreads;
  const int near = rounds < PER ? rounds : PER;
  if (s.new_len == 0 || s.new_len == s.kv_len) {       // nothing to choose
    for (int k = tid; k < p.out_stride; k += kThreads) out[k] = k < s.new_len ? k : -1;
    if (tid == 0) ws[0] = 0;
    return;
  }
  uint32_t rk[PER];
#pragma unroll
  for (int i = 0; i < PER; i += 8) {
#pragma unroll
    for (int j = 0; j < 8; ++j) rk[i + j] = 0u;
    if (i < near) load_ranks<8>(p, s, i, wave, rk + i);
  }
  for (int i = PER; i < rounds; i += 8) {
    uint32_t r[8];
    load_ranks<8>(p, s, i, wave, r);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < rounds) far[(i + j - PER) * kThreads + tid] = r[j];
  }

  uint32_t pre = 0, need = (uint32_t)s.new_len;
  for (int shift = 24; shift >= 0; shift -= 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) hist[i * kThreads + tid] = 0;
    __syncthreads();
    const uint32_t above = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
    auto count = [&](int i, uint32_t r) {
      if (i * kThreads + tid < s.kv_len && (r & above) == pre) atomicAdd(&hist[((r >> shift) & 255u) * 32 + (lane & 31)], 1u);
    };
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i < near) count(i, rk[i]);
    for (int i = PER; i < rounds; i += 8) {
      uint32_t r[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] = far[((i + j < rounds ? i + j : rounds - 1) - PER) * kThreads + tid];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i + j < rounds) count(i + j, r[j]);
    }
    __syncthreads();
    {
      // thread t adds up copies 8 (t % 4).. of digit t / 4, starting at its own bank
      uint32_t x = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) x += hist[(tid >> 2) * 32 + 8 * (tid & 3) + ((i + (tid >> 2)) & 7)];
      x += __shfl_xor(x, 1);
      x += __shfl_xor(x, 2);
      if ((tid & 3) == 0) tot[tid >> 2] = x;
    }
    __syncthreads();
    if (wave == 0) {
      // lane l: digits 255 - 4l downwards; the digit at which the count from the top reaches `need`
      uint32_t v[4], x = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = tot[255 - (4 * lane + j)];
        x += v[j];
      }
      uint32_t incl = x;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const uint32_t y = __shfl_up(incl, d);
        incl += lane >= d ? y : 0u;
      }
      uint32_t before = incl - x;
      if (before < need && incl >= need) {
        int j = 0;
        for (; j < 3 && before + v[j] < need; ++j) before += v[j];
        sel[0] = pre | ((uint32_t)(255 - (4 * lane + j)) << shift);
        sel[1] = need - before;
        sel[2] = v[j];                      // keys with this digit
      }
    }
    __syncthreads();
    pre = sel[0];
    need = sel[1];
  }

  // ranks above `pre` stay, and the first `need` equal to it.  64 rounds of
  // 16 wavefronts at a time, the histogram's memory for the counts
  const bool ties = need < sel[2];
  int* eqs = reinterpret_cast<int*>(hist);          // [64 rounds][16 wavefronts]
  int* cnt = eqs + kThreads;
  if (tid < 2) carry[tid] = 0;
  for (int i0 = 0; i0 < rounds; i0 += 64) {
    const int nr = rounds - i0 < 64 ? rounds - i0 : 64, n = nr * kEvWaves;
    auto rank = [&](int i) -> uint32_t { return far[(i - PER) * kThreads + tid]; };
    auto each = [&](auto f) {
      // ranks from memory, eight rounds in flight
      auto batch = [&](int from, int base) {
        for (int i = from; i < nr; i += 8) {
          uint32_t r[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) r[j] = rank(base + (i + j < nr ? i + j : nr - 1));
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (i + j < nr) f(i + j, r[j]);
        }
      };
      if (i0 == 0) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (i < nr) f(i, rk[i]);
        batch(PER, 0);
      } else {
        batch(0, i0);
      }
    };
    auto key = [&](int i) { return (i0 + i) * kThreads + tid; };
    const unsigned long long below = (1ull << lane) - 1ull;
    __syncthreads();
    int eq0 = 0, eq_last = 0;
    if (ties) {
      each([&](int i, uint32_t r) {
        const unsigned long long b = __ballot(key(i) < s.kv_len && r == pre);
        if (lane == 0) eqs[i * kEvWaves + wave] = __popcll(b);
      });
      __syncthreads();
      eq_last = tid == n - 1 ? eqs[n - 1] : 0;
      block_scan(eqs, n, sh);
      eq0 = carry[0];
    }
    // a hole in front of the new end, or a key behind it that stays
    auto listed = [&](int i, uint32_t r) -> bool {
      const int k = key(i);
      bool keep = r >= pre;
      if (ties) {
        const unsigned long long b = __ballot(k < s.kv_len && r == pre);
        if (r == pre) keep = eq0 + eqs[i * kEvWaves + wave] + __popcll(b & below) < (int)need;
      }
      return k < s.kv_len && keep == (k >= s.new_len);
    };
    each([&](int i, uint32_t r) {
      const unsigned long long b = __ballot(listed(i, r));
      if (lane == 0) cnt[i * kEvWaves + wave] = __popcll(b);
    });
    __syncthreads();
    const int last = tid == n - 1 ? cnt[n - 1] : 0;
    block_scan(cnt, n, sh);
    const int at0 = carry[1];
    each([&](int i, uint32_t r) {
      const bool f = listed(i, r);
      const unsigned long long b = __ballot(f);
      if (f) list[at0 + cnt[i * kEvWaves + wave] + __popcll(b & below)] = key(i);
      else if (key(i) < s.new_len) out[key(i)] = key(i);
    });
    __syncthreads();
    if (tid == n - 1) {
      if (ties) carry[0] = eq0 + eqs[n - 1] + eq_last;
      carry[1] = at0 + cnt[n - 1] + last;
    }
    __syncthreads();
  }
  const int moved = carry[1] / 2;
  for (int i = tid; i < moved; i += kThreads) out[list[i]] = list[moved + i];
  for (int k = s.new_len + tid; k < p.out_stride; k += kThreads) out[k] = -1;
  if (tid == 0) ws[0] = moved;
}

// Copies the rows of one array from slots to slots.
template <class V>
__device__ __forceinline__ void copy_rows(const EvictArray& a, const int* from, const int* to, int n) {
  const int cols = a.row_bytes / (int)sizeof(V);
  const V* src = reinterpret_cast<const V*>(a.src);
  V* dst = reinterpret_cast<V*>(a.dst);
  for (int i = threadIdx.x; i < n * cols; i += (int)blockDim.x) {
    const int r = i / cols, c = i - r * cols;
    if (from[r] >= 0 && to[r] >= 0) dst[(int64_t)to[r] * cols + c] = src[(int64_t)from[r] * cols + c];
  }
}

__device__ __forceinline__ void copy_any(const EvictArray& a, const int* from, const int* to, int n) {
  if (a.gran == 16) copy_rows<i4>(a, from, to, n);
  else if (a.gran == 4) copy_rows<uint32_t>(a, from, to, n);
  else copy_rows<uint8_t>(a, from, to, n);
}

// Workgroups 0..in_blocks-1 of a sequence: kMoveRows entries each of its list
// of moves, for the arrays in place; the others: kCopyRows kept rows each of
// the arrays that go elsewhere.  4 KB a key in two arrays: 64 moves in each of
// 16 sequences 6 us, 16 thousand moves 24 us (5.3 TB/s).
__global__ __launch_bounds__(256) void evict_move_kernel(const EvictMoveArgs p) {
  __shared__ int from[kCopyRows], to[kCopyRows];
  const EvictSeq& s = p.s[blockIdx.y];
  auto slot = [&](int key) { return cache_slot(p.table, s.b, p.max_pages, p.page_size, p.num_pages, key); };
  const int tid = threadIdx.x;
  if ((int)blockIdx.x < p.in_blocks) {
    const int32_t* ws = p.ws + s.ws_off;
    const int j0 = blockIdx.x * kMoveRows, n = min(kMoveRows, ws[0] - j0);
    if (n <= 0) return;
    if (tid < n) {
      to[tid] = slot(ws[kEvictHead + j0 + tid]);
      from[tid] = slot(ws[kEvictHead + ws[0] + j0 + tid]);
    }
    __syncthreads();
    for (int i = 0; i < p.n_arr; ++i)
      if (p.a[i].src == p.a[i].dst) copy_any(p.a[i], from, to, n);
  } else {
    const int j0 = ((int)blockIdx.x - p.in_blocks) * kCopyRows, n = min(kCopyRows, s.new_len - j0);
    if (n <= 0) return;
    if (tid < n) {
      const int src = p.out_src[(int64_t)s.b * p.out_stride + j0 + tid];
      to[tid] = slot(j0 + tid);
      from[tid] = src < 0 ? -1 : slot(src);
    }
    __syncthreads();
    for (int i = 0; i < p.n_arr; ++i)
      if (p.a[i].src != p.a[i].dst) copy_any(p.a[i], from, to, n);
  }
}

}  // namespace

hipError_t launch_evict_select(const EvictArgs& p, hipStream_t s) {
  if (p.n_seq == 0) return hipSuccess;
  int most = 0;
  for (int i = 0; i < p.n_seq; ++i) most = most > p.s[i].kv_len ? most : p.s[i].kv_len;
  const dim3 grid((unsigned)p.n_seq), block(kThreads);
  if (most <= 8 * kThreads) evict_select_kernel<8><<<grid, block, 0, s>>>(p);
  else evict_select_kernel<kEvictNear><<<grid, block, 0, s>>>(p);
  return hipGetLastError();
}

hipError_t launch_evict_move(EvictMoveArgs p, hipStream_t s) {
  int most_new = 0, most_cap = 0;
  bool in = false, away = false;
  for (int i = 0; i < p.n_seq; ++i) {
    most_new = most_new > p.s[i].new_len ? most_new : p.s[i].new_len;
    most_cap = most_cap > p.s[i].cap ? most_cap : p.s[i].cap;
  }
  for (int i = 0; i < p.n_arr; ++i) (p.a[i].src == p.a[i].dst ? in : away) = true;
  p.in_blocks = in ? (most_cap + kMoveRows - 1) / kMoveRows : 0;
  const int blocks = p.in_blocks + (away ? (most_new + kCopyRows - 1) / kCopyRows : 0);
  if (p.n_seq == 0 || blocks == 0) return hipSuccess;
  evict_move_kernel<<<dim3((unsigned)blocks, (unsigned)p.n_seq), dim3(256), 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace dosa
