// Page tables and slot maps, and the write of rows into pages with the
// summaries of the blocks that it completes.
#include "attn_device.h"
#include "pages_internal.h"

namespace dosa {

namespace {

// A workgroup takes kSpan tokens (pages): enough that its two searches among the
// records are a small part of it (1.2M tokens of 300 prompts: 10 us, 13 with 256; a
// decode step of 128 sequences 4 us, latency).
// Most lie in one sequence; the others search among the records that they span.
constexpr int kSpan = 1024;
struct Span {
  int lo, hi;            // records of the first and the last
  const int* starts;     // first tokens of the records, in LDS
  __device__ __forceinline__ int find(int t) const {
    int a = lo, b = hi;
    while (a < b) {
      const int mid = (a + b + 1) >> 1;
      if (starts[mid] <= t) a = mid; else b = mid - 1;
    }
    return a;
  }
};
__device__ __forceinline__ Span span_of(const AssignArgs& p, int* starts) {
  const int first = blockIdx.x * kSpan, last = min(first + kSpan - 1, p.n_tok - 1);
  auto tok0 = [](const AssignSeq& s) { return s.tok0; };
  const Span x{find_seq(p.s, p.n_seq, first, tok0), find_seq(p.s, p.n_seq, last, tok0), starts};
  if (x.lo < x.hi) {
    for (int i = x.lo + (int)threadIdx.x; i <= x.hi; i += 256) starts[i] = p.s[i].tok0;
    __syncthreads();
  }
  return x;
}

// A thread a token at a time.  A sequence's n-th new page is read from the free
// list where it is used, so no token waits for another's table write; the token
// that opens a page writes its entry.
__global__ __launch_bounds__(256) void assign_kernel(const AssignArgs p) {
  __shared__ int starts[kAssignSeqs];
  const Span span = span_of(p, starts);
  const int size = p.page_div.by;
#pragma unroll
  for (int u = 0; u < kSpan / 256; ++u) {
    const int t = blockIdx.x * kSpan + u * 256 + threadIdx.x;
    if (t >= p.n_tok) return;
    const int i = span.find(t);
    const AssignSeq s = p.s[i];
    const int pos = s.pos0 + (t - s.tok0), pg = p.page_div.quot(pos), in = pos - pg * size;
    const int first = p.page_div.quot((uint32_t)s.pos0 + (uint32_t)size - 1u);    // first new page
    int32_t* entry = p.table + (int64_t)(p.b0 + i) * p.max_pages + pg;
    const int page = pg >= first ? p.free_pages[p.top - 1 - (s.new0 + pg - first)] : *entry;
    if (pg >= first && in == 0) *entry = page;
    if (p.slots != nullptr) p.slots[t] = (uint32_t)page < (uint32_t)p.num_pages ? page * size + in : -1;
    if (p.positions != nullptr) p.positions[t] = pos;
  }
}

// A thread a page at a time.
__global__ __launch_bounds__(256) void release_kernel(const AssignArgs p) {
  __shared__ int starts[kAssignSeqs];
  const Span span = span_of(p, starts);
  for (int u = 0; u < kSpan / 256; ++u) {
    const int t = blockIdx.x * kSpan + u * 256 + threadIdx.x;
    if (t >= p.n_tok) return;
    const int i = span.find(t);
    int32_t* entry = p.table + (int64_t)(p.b0 + i) * p.max_pages + p.s[i].pos0 + (t - p.s[i].tok0);
    p.free_pages[p.top - 1 - t] = *entry;
    *entry = -1;
  }
}

constexpr double kLargest = 0x1.fffffep127;      // fp32's

// 16 bytes of a row -> its elements in 64 bits.
template <bool F32>
__device__ __forceinline__ void widen64(i4 a, double* x) {
  if constexpr (F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = (double)__int_as_float(a[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = (double)__uint_as_float((uint32_t)a[i] << 16);
      x[2 * i + 1] = (double)__uint_as_float((uint32_t)a[i] & 0xffff0000u);
    }
  }
}

// Bound by memory: 31011 tokens of 8 heads, d = 128, bf16, with their summaries,
// 255 MB, in 43 us (fp32, twice that, 115 us); a decode step's 128 tokens, of which
// two complete a block, 6 us, latency.  A slice of 32 pieces of 16 bytes and eight
// tokens at a time give a block of 64 tokens four workgroups and eight loads a
// thread.
//
// Rows of a run of positions: the call's own go to their slots bit by bit (none
// without k); where the run is a block that is complete now, all its keys are
// summed, those that are not the call's read from the page.
//
// The mean is summed in 64 bits: keys of 8 or 24 significant bits add up without
// rounding, and so in any order, unless their exponents lie 38 (23) apart; the order
// goes by the positions in the block, so the codes do not depend on which calls
// wrote its keys either way.  The scale 2^e is the smallest power of two with max |mean| <
// 127.5 2^e: 127.5 = 2^6 (2 - 2^-7), so adding 2^-7 to the significand carries
// into the exponent exactly where e has to be one more.
template <bool F32, int D>
__global__ __launch_bounds__(256) void rows_append_kernel(const RowsArgs p) {
  constexpr int E = F32 ? 4 : 8, SUBS = 256 / kRowLanes, HL = D / E;   // elements of a piece, tokens at a time, pieces of a head
  __shared__ double sums[SUBS][kRowLanes * E];
  const int tid = threadIdx.x, lane = tid % kRowLanes, sub = tid / kRowLanes;
  const int unit = blockIdx.x / p.slices, slice = blockIdx.x % p.slices;
  const RowsSeq& s = p.s[find_seq(p.s, p.n_seq, unit, [](const RowsSeq& x) { return x.unit0; })];
  const int base = s.pos0 / p.run * p.run + (unit - s.unit0) * p.run;    // first position of the run
  const int pg = p.page_div.quot(base), size = p.page_div.by;
  const int page = p.pages.table[(int64_t)s.b * p.pages.max_pages + pg];
  if ((uint32_t)page >= (uint32_t)p.pages.num_pages) return;
  const int64_t slot0 = (int64_t)page * size + (base - pg * size);
  const int piece = slice * kRowLanes + lane;
  const bool on = piece < p.pieces;
  const int lo = max(s.pos0, base), hi = min(s.end, base + p.run);      // the call's positions
  const int given = p.k != nullptr ? s.pos0 : s.end;                    // rows from here on are the call's own
  const bool whole = p.codes != nullptr && s.end >= base + p.run;
  const int64_t row_b = (int64_t)p.pieces * 16;
  double x[E], sum[E] = {};
  if (on) {
    const uint8_t* kp = p.k_pages + slot0 * row_b + piece * 16;
    const int from = whole ? base : lo;
    constexpr int U = 4;
    for (int t0 = from + sub; t0 < hi; t0 += U * SUBS) {
      i4 k[U], v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = t0 + u * SUBS, c = t < hi ? t : hi - 1;
        const int64_t row = s.row0 + (c - s.pos0);
        k[u] = *reinterpret_cast<const i4*>(c >= given ? p.k + row * p.k_stride + piece * 16 : kp + (c - base) * row_b);
        if (c >= given) v[u] = *reinterpret_cast<const i4*>(p.v + row * p.v_stride + piece * 16);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = t0 + u * SUBS;
        if (t >= hi) break;
        if (t >= given) {
          const int64_t at = (slot0 + t - base) * row_b + piece * 16;
          *reinterpret_cast<i4*>(p.k_pages + at) = k[u];
          *reinterpret_cast<i4*>(p.v_pages + at) = v[u];
        }
        if (whole) {
          widen64<F32>(k[u], x);
#pragma unroll
          for (int e = 0; e < E; ++e) sum[e] += x[e];
        }
      }
    }
  }
  if (!whole) return;
#pragma unroll
  for (int e = 0; e < E; ++e) sums[sub][lane * E + e] = sum[e];
  __syncthreads();
  if (tid >= kRowLanes) return;
  double top = 0.;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    double y = 0.;
#pragma unroll
    for (int w = 0; w < SUBS; ++w) y += sums[w][lane * E + e];
    y *= 1.0 / p.run;                  // a power of two
    x[e] = y == y ? fmin(fmax(y, -kLargest), kLargest) : 0.;     // keys that are not finite
    top = fmax(top, fabs(x[e]));
  }
#pragma unroll
  for (int w = 1; w < HL; w <<= 1) top = fmax(top, __shfl_xor(top, w));
  int e2 = (int)((__double_as_longlong(top) + (1ll << 45)) >> 52) - 1023 - 6;
  e2 = e2 < -126 ? -126 : (e2 > 127 ? 127 : e2);
  const double inv = __longlong_as_double((long long)(1023 - e2) << 52);
  if (!on) return;
  const int64_t blk = slot0 / p.run;
  const int head = piece / HL;
  uint32_t w[E / 4] = {};
#pragma unroll
  for (int e = 0; e < E; ++e) w[e / 4] |= ((uint32_t)(int)rint(x[e] * inv) & 255u) << (8 * (e % 4));
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.codes + blk * (int64_t)(p.pieces * E) + piece * E);
#pragma unroll
  for (int i = 0; i < E / 4; ++i) dst[i] = w[i];
  if (piece % HL == 0) p.scales[blk * (p.pieces / HL) + head] = (uint8_t)(e2 + 127);
}

}  // namespace

hipError_t launch_assign(const AssignArgs& p, hipStream_t s) {
  if (p.n_tok == 0) return hipSuccess;
  assign_kernel<<<dim3((unsigned)(((int64_t)p.n_tok + kSpan - 1) / kSpan)), dim3(256), 0, s>>>(p);
  return hipGetLastError();
}

hipError_t launch_release(const AssignArgs& p, hipStream_t s) {
  if (p.n_tok == 0) return hipSuccess;
  release_kernel<<<dim3((unsigned)(((int64_t)p.n_tok + kSpan - 1) / kSpan)), dim3(256), 0, s>>>(p);
  return hipGetLastError();
}

hipError_t launch_rows_append(bool f32, int d, const RowsArgs& p, hipStream_t s) {
  if (p.n_units == 0) return hipSuccess;
  const dim3 grid((unsigned)(p.n_units * p.slices)), block(256);
  if (f32 && d == 128) rows_append_kernel<true, 128><<<grid, block, 0, s>>>(p);
  else if (f32) rows_append_kernel<true, 64><<<grid, block, 0, s>>>(p);
  else if (d == 128) rows_append_kernel<false, 128><<<grid, block, 0, s>>>(p);
  else rows_append_kernel<false, 64><<<grid, block, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace dosa
