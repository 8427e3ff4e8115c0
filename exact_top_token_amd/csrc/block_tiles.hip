// Attention over listed blocks for many bf16 queries, in two kernels.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = 2^((s_j - m) c),  c = scale log2(e),
//   lse = scale m + ln sum_j p_j,  over the keys j of a row's blocks.
//
// block_merge_kernel: neighbouring queries list many of the same blocks.  A
// wavefront merges the lists of the queries of a workgroup of the second kernel:
// lane t holds the next block of query t, and the smallest is taken for all
// queries whose next it is.  Ascending lists share all that they can; in any
// order every entry counts once.
//
// block_tiles_kernel: eight wavefronts, each with one 16-row tile (the group
// heads of one query or of a few neighbours), walk over the merged blocks.  A
// block's keys and values come to LDS once for all of them; a wavefront whose
// queries do not list the block passes it by.  What bounds a wavefront that
// reads its blocks by itself is the caches' rate.
//
// Scores are computed transposed, S^T = K Q^T, by 16x16x32 products: lane l then
// holds row l%16 and keys 4(l/16)..+3 of each 16 keys, and numbering the
// reduction slots of O^T = V^T P^T the same way makes its right operand without
// moving a value between lanes.  V^T comes out of row-major LDS tiles through the
// transposing LDS read.
//
// 4096 and 1500 queries, 64 heads on 8, d = 128, each 16 blocks of 64 of up to
// 32768 keys, of which neighbours share half (66 different ones of 16 queries):
// 0.56 to 0.59 ms on different boards, of which 30 us the merge (under a trace 0.58
// to 0.62 ms and 31 us); a wavefront a query takes 1.94 ms, merging two queries in
// a wavefront without LDS 1.36.  Reading the blocks alone took 0.46 ms
// (6.2 GB, two thirds from the dies' caches): a workgroup waits for its slowest
// wavefront at every block, and the CU holds two.  Addresses worked out anew for
// every load and scores masked one by one, not rows, cost 0.05 ms.
// Keys and values in five slots of half a tile, twice as much under way but a
// barrier for each half, took 0.62 ms, in four slots 0.63 (against 0.56, merging
// included); tiles of 32 keys with three under way 0.70, sixteen wavefronts of 32
// queries 0.92, the merge by one of the eight wavefronts 1.24.
//
// Weights are rounded to bf16 once for their product with v, their sum is taken
// before: outputs are off by 0.23% of their size (root mean square) where fp32
// weights and the result's rounding leave 0.17%.  Two terms leave 0.17% too, in 0.72
// instead of 0.59 ms (groups of 4, 16 of 512 blocks: 0.48 and 0.41; d = 64, 64 of
// 2048 blocks of 16: 0.72 and 0.59): a third off what the result's type costs anyway
// does not pay for a fifth more time.
#include <type_traits>

#include "attn_device.h"

namespace dosa {

namespace {

typedef short s4v __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t lbyte;
typedef __attribute__((address_space(3))) b8 lds_b8;
typedef __attribute__((address_space(3))) s4v lds_s4;
typedef __attribute__((address_space(4))) const i4 scalar_i4;

constexpr int NW = kBlockTileWaves;
constexpr int kKeys = 64;       // keys of a tile
constexpr int kRing = 2;        // tiles in LDS: one used, the other arriving
constexpr float kSlack = 8.f;   // exponent by which a score may exceed the running maximum

// The part of a sequence's row tiles that a workgroup takes.
struct Share {
  int wg_rt;                    // first row tile
  int split, head;
  int tiles_q;                  // row tiles of a query
  int q0, q_end;                // its queries
};
__device__ __forceinline__ Share share_of(const AttnArgs& p, const AttnSeq& sq, int t) {
  Share s;
  s.head = t % p.Hkv;
  t /= p.Hkv;
  const int n_wg = (sq.n_rt + NW - 1) / NW;
  s.wg_rt = (n_wg - 1 - t % n_wg) * NW;            // last row tiles first
  s.split = t / n_wg;
  s.tiles_q = (p.group + 15) / 16;
  s.q0 = s.wg_rt / s.tiles_q * p.tok;
  s.q_end = min((min(s.wg_rt + NW, sq.n_rt) - 1) / s.tiles_q * p.tok + p.tok, sq.q_len);
  return s;
}

// Smallest of the lanes' values.  Uniform.
__device__ __forceinline__ uint32_t least64(uint32_t x) {
  x = min(x, (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, 0x128, 0xf, 0xf, false));   // rotations within 16
  x = min(x, (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, 0x124, 0xf, 0xf, false));
  x = min(x, (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, 0x122, 0xf, 0xf, false));
  x = min(x, (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, 0x121, 0xf, 0xf, false));
  const uint32_t a = min((uint32_t)__builtin_amdgcn_readlane((int)x, 0), (uint32_t)__builtin_amdgcn_readlane((int)x, 16));
  const uint32_t b = min((uint32_t)__builtin_amdgcn_readlane((int)x, 32), (uint32_t)__builtin_amdgcn_readlane((int)x, 48));
  return min(a, b);
}

constexpr int kMergeWaves = 4;
constexpr int kListed = 2048;   // entries of a unit's lists in LDS

// Merged blocks of a unit: {slot of the first row, position of the first key,
// queries that list it (64 bits)}, kBlockEnds records of position -1 behind.
// Blocks without a page are left out.
__global__ __launch_bounds__(64 * kMergeWaves) void block_merge_kernel(const AttnArgs p) {
  __shared__ int32_t listed_all[kMergeWaves][kListed];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = lane64();
  const int unit = blockIdx.x * kMergeWaves + wave;
  if (unit >= p.n_units) return;
  const AttnSeq& sq = p.s[find_seq(p.s, p.n_seq, unit, [](const AttnSeq& s) { return s.unit0; })];
  const Share sh = share_of(p, sq, unit - sq.unit0);
  int32_t* const listed = listed_all[wave];
  const int n_tok = sh.q_end - sh.q0;                      // at most 64
  const int lb = __builtin_ctz(p.block), topn = p.topk >> lb;
  const int e_lo = (int)((int64_t)sh.split * sq.split_len >> lb);
  const int e_end = (int)min((int64_t)topn, ((int64_t)sh.split + 1) * sq.split_len >> lb);
  // the lists' next `win` entries are in LDS
  const int win = kListed / (n_tok <= 16 ? 16 : n_tok <= 32 ? 32 : 64);
  const int32_t* const lists = p.idx + ((int64_t)(sq.q_row0 + sh.q0) * p.Hkv + sh.head) * topn;
  auto fill = [&](int x, int e) {                          // entries e.. of query x
    for (int y = lane; y < win && e + y < e_end; y += 64) listed[x * win + y] = lists[(int64_t)x * p.Hkv * topn + e + y];
  };
  {
    const int len = min(win, e_end - e_lo), all = n_tok * len;
    constexpr int U = 4;                                   // loads in flight
    for (int i0 = lane; i0 < all; i0 += 64 * U) {
      int y[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = min(i0 + 64 * u, all - 1), x = i / len;
        y[u] = lists[(int64_t)x * p.Hkv * topn + e_lo + (i - x * len)];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = min(i0 + 64 * u, all - 1), x = i / len;
        listed[x * win + (i - x * len)] = y[u];
      }
    }
  }
  wave_sync();
  constexpr uint32_t kEnd = 0xffffffffu, kNone = 0xfffffffeu;      // no more entries; an entry to skip
  const uint32_t own = (uint32_t)(sq.kv_len - sq.q_len + sh.q0 + lane) >> lb;
  int at = e_lo;
  auto front = [&]() -> uint32_t {
    if (lane >= n_tok || at >= e_end) return kEnd;
    const uint32_t y = (uint32_t)listed[lane * win + ((at - e_lo) & (win - 1))];
    return y <= own ? y : kNone;
  };
  uint32_t cur = front();
  i4* out = reinterpret_cast<i4*>(p.merged) + (int64_t)unit * p.merged_stride;
  uint32_t blk = 0;
  while (blk != kEnd) {
    // up to 64 blocks, one a lane
    int n = 0, mine = 0;
    uint64_t of = 0;
    while (n < 64) {
      blk = least64(cur);
      if (blk == kEnd) break;
      const bool take = cur == blk;
      const uint64_t who = __ballot(take);
      if (take) ++at;
      uint64_t dry = __ballot(take && at < e_end && ((at - e_lo) & (win - 1)) == 0);
      if (dry != 0) {
        wave_sync();
        for (; dry != 0; dry &= dry - 1) {
          const int x = __builtin_ctzll(dry);
          fill(x, __builtin_amdgcn_readlane(at, x));
        }
        wave_sync();
      }
      if (take) cur = front();
      if (blk == kNone) continue;
      if (lane == n) {
        mine = (int)blk;
        of = who;
      }
      ++n;
    }
    const int pos = lane < n ? mine << lb : 0, pg = p.page_div.quot(pos);
    const int page = lane < n ? p.cache.table[(int64_t)sq.b * p.cache.max_pages + pg] : -1;
    const bool there = (uint32_t)page < (uint32_t)p.cache.num_pages;
    const uint64_t all = __ballot(there);
    if (there)
      out[below(all)] = i4{page * p.cache.page_size + (pos - pg * p.cache.page_size), pos, (int)(uint32_t)of, (int)(uint32_t)(of >> 32)};
    out += __popcll(all);
  }
  if (lane < kBlockEnds) out[lane] = i4{0, -1, 0, 0};
}

// 16-byte chunk of a value tile's row `r` that holds logical chunk c: 32 lanes
// read 32 bytes of 8 rows.
template <int D>
__device__ __forceinline__ int v_chunk(int r, int c) {
  return D == 128 ? c ^ ((r & 7) << 1) : c ^ (((r >> 1) & 3) << 1);
}

// Transposed value operands of four 16-dimension columns and 32 keys: eight
// transposing reads and the wait for them.  Written out, because in front of the
// builtin the compiler waits for every load to LDS that is under way, the tiles to
// come among them.
template <int AT0, int AT1>
__device__ __forceinline__ void read_values(const uint32_t* va, b8* w) {
  s4v x[8];
  asm volatile(
      "ds_read_b64_tr_b16 %0, %8 offset:%12\n\t"
      "ds_read_b64_tr_b16 %1, %8 offset:%13\n\t"
      "ds_read_b64_tr_b16 %2, %9 offset:%12\n\t"
      "ds_read_b64_tr_b16 %3, %9 offset:%13\n\t"
      "ds_read_b64_tr_b16 %4, %10 offset:%12\n\t"
      "ds_read_b64_tr_b16 %5, %10 offset:%13\n\t"
      "ds_read_b64_tr_b16 %6, %11 offset:%12\n\t"
      "ds_read_b64_tr_b16 %7, %11 offset:%13\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(x[4]), "=&v"(x[5]), "=&v"(x[6]), "=&v"(x[7])
      : "v"(va[0]), "v"(va[1]), "v"(va[2]), "v"(va[3]), "n"(AT0), "n"(AT1)
      : "memory");
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = __builtin_bit_cast(b8, __builtin_shufflevector(x[2 * j], x[2 * j + 1], 0, 1, 2, 3, 4, 5, 6, 7));
}

// RUNS: blocks of a tile, 4 of 16 keys, 2 of 32, 1 (or a part of one) of 64 and 128.
template <int D, int RUNS>
__global__ __launch_bounds__(64 * NW, 4) void block_tiles_kernel(const AttnArgs p) {
  constexpr int CH = D / 8, TILE = kKeys * D * 2, NS = D / 32, NT = D / 16;
  constexpr int RPI = 64 / CH;                     // rows a wavefront's load fills: 4 (8)
  constexpr int LOADS = 2 * kKeys / RPI / NW;      // loads of a wavefront per tile
  constexpr int RUN = kKeys / RUNS;                // keys of a run
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kRing][2][TILE];   // [buffer][k, v]

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = lane64(), n = lane & 15, g = lane >> 4;
  const int unit = blockIdx.x;
  const AttnSeq& sq = p.s[find_seq(p.s, p.n_seq, unit, [](const AttnSeq& s) { return s.unit0; })];
  const Share sh = share_of(p, sq, unit - sq.unit0);

  // the wavefront's row tile: p.tok queries, or a part of one query's heads
  const int rt0 = sh.wg_rt + wave;
  const bool active = rt0 < sq.n_rt;
  const int q_first = (active ? rt0 : sq.n_rt - 1) / sh.tiles_q * p.tok;
  const int row_base = (active ? rt0 : sq.n_rt - 1) % sh.tiles_q * 16;
  const int n_tok = min(p.tok, sq.q_len - q_first);
  const int r0 = row_base + n, n_rows = n_tok * p.group;
  const bool row_ok = active && r0 < n_rows;
  const int r = r0 < n_rows ? r0 : n_rows - 1;
  const int row_q = q_first + r / p.group, row_h = sh.head * p.group + r % p.group;
  const uint32_t bit = 1u << (r / p.group);
  const int before = sq.kv_len - sq.q_len, vis = before + row_q + 1;
  const int vis_first = before + q_first + 1, vis_end = before + sh.q_end;
  const uint32_t mask = active ? (1u << n_tok) - 1u : 0u;
  const int of_shift = q_first - sh.q0;

  b8 qf[NS];
  {
    const i4* src = reinterpret_cast<const i4*>(static_cast<const uint16_t*>(p.q) + (int64_t)(sq.q_row0 + row_q) * p.q_stride +
                                                (int64_t)row_h * D + 8 * g);
#pragma unroll
    for (int s = 0; s < NS; ++s) qf[s] = __builtin_bit_cast(b8, src[4 * s]);
  }
  f4 o[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) o[j] = f4{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;
  const float c = p.scale * kLog2e;

  // ---- the tiles' blocks, through the scalar cache ----
  struct Tile {
    int slot[RUNS], pos[RUNS];                     // of the runs' first keys; position -1: past the last block
    uint32_t of[RUNS];                             // this wavefront's queries that list them
  };
  const scalar_i4* list = (scalar_i4*)(p.merged + (int64_t)unit * p.merged_stride);
  int sub = 0;
  i4 rec[RUNS];                                    // of the tile that `next` describes
#pragma unroll
  for (int x = 0; x < RUNS; ++x) rec[x] = list[x];
  auto next = [&]() -> Tile {
    Tile t;
#pragma unroll
    for (int x = 0; x < RUNS; ++x) {
      // runs behind the last block are the tile's first one again, whose rows are numbers, listed by nobody
      const bool there = x == 0 || rec[x][1] >= 0;
      const i4 y = there ? rec[x] : rec[0];
      t.slot[x] = y[0] + sub;
      t.pos[x] = y[1] < 0 ? -1 : y[1] + sub;
      t.of[x] = there ? (uint32_t)((((uint64_t)(uint32_t)y[3] << 32) | (uint32_t)y[2]) >> of_shift) & mask : 0u;
    }
    if (rec[0][1] >= 0) {
      sub += kKeys;
      if (RUNS > 1 || sub >= p.block) {
        sub = 0;
        list += RUNS;
#pragma unroll
        for (int x = 0; x < RUNS; ++x) rec[x] = list[x];
      }
    }
    return t;
  };

  // ---- tiles to LDS ----
  const uint16_t *kg = static_cast<const uint16_t*>(p.k) + sh.head * D, *vg = static_cast<const uint16_t*>(p.v) + sh.head * D;
  // A load fills RPI rows.  Its rows and a lane's chunk of them do not change: a tile whose rows are all visible
  // needs one scalar base a load, and the vector unit nothing.
  const int lr = lane / CH, lc = lane % CH;
  uint32_t f_row[LOADS], f_chunk[LOADS], f_off[LOADS];     // row within the run, bytes
#pragma unroll
  for (int x = 0; x < LOADS; ++x) {
    const int i = wave * LOADS + x, which = i / (kKeys / RPI), row = i % (kKeys / RPI) * RPI + lr;
    f_row[x] = row % RUN;
    f_chunk[x] = 16 * (which == 0 ? k_chunk<D>(row, lc) : v_chunk<D>(row, lc));
    f_off[x] = f_row[x] * (uint32_t)p.k_stride * 2 + f_chunk[x];
  }
  auto fetch = [&](const Tile& tile, int buf) {
    bool whole = tile.pos[0] >= 0;
#pragma unroll
    for (int y = 0; y < RUNS; ++y) whole = whole && tile.pos[y] + RUN <= vis_end;
#pragma unroll
    for (int x = 0; x < LOADS; ++x) {
      const int i = wave * LOADS + x, which = i / (kKeys / RPI), at = i % (kKeys / RPI) * RPI, run = at / RUN;
      int slot = tile.slot[0], pos = tile.pos[0];
#pragma unroll
      for (int y = 1; y < RUNS; ++y) {
        slot = run == y ? tile.slot[y] : slot;
        pos = run == y ? tile.pos[y] : pos;
      }
      const uint8_t* from = reinterpret_cast<const uint8_t*>((which == 0 ? kg : vg) + (int64_t)slot * p.k_stride);
      uint32_t off = f_off[x];
      if (!whole) {
        // rows behind the last visible key, which may hold anything, are read as it (it may lie in front of the tile)
        const int lim = pos < 0 ? 0 : vis_end - 1 - pos, back = lim < 0 ? lim : 0;
        from += (int64_t)back * p.k_stride * 2;
        off = (uint32_t)(((int)f_row[x] < lim ? (int)f_row[x] : lim) - back) * (uint32_t)p.k_stride * 2 + f_chunk[x];
      }
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(from + off),
                                       (__attribute__((address_space(3))) void*)(&lds[buf][which][at * D * 2]), 16, 0, 0);
    }
  };

  // LDS offsets of a lane's operands
  lbyte* const base = (lbyte*)&lds[0][0][0];
  uint32_t ka[NS], va[NT];
#pragma unroll
  for (int s = 0; s < NS; ++s) ka[s] = n * (D * 2) + 16 * k_chunk<D>(n, 4 * s + g);
  const int vr = 4 * g + (n >> 2), vc = 4 * (n & 3);
#pragma unroll
  for (int j = 0; j < NT; ++j) va[j] = (uint32_t)(uintptr_t)base + vr * (D * 2) + 16 * v_chunk<D>(vr, (16 * j + vc) >> 3) + (vc & 7) * 2;

  auto compute = [&](const Tile& x, auto buf) {
    constexpr int BUF = decltype(buf)::value;
    lbyte* const tile = base + BUF * (2 * TILE);
    f4 sc[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) sc[a] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int a = 0; a < 4; ++a) sc[a] = mfma_bf16(*(lds_b8*)(tile + ka[s] + 16 * a * (D * 2)), qf[s], sc[a]);
    // A tile of one block, or of a part of one: rows that do not list it keep their maximum, and their weights are
    // cleared once they are packed.  Scores are masked one by one only where keys are hidden or blocks are smaller.
    bool on = true;
    bool edge = RUNS > 1;
    if constexpr (RUNS == 1) {
      on = (x.of[0] & bit) != 0;
      edge = x.pos[0] + kKeys > vis_first;
    }
    if (edge) {
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const int pos = x.pos[16 * a / RUN] + 16 * a % RUN;
        const int end = x.of[16 * a / RUN] & bit ? vis - pos : 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[a][e] = 4 * g + e >= end ? -INFINITY : sc[a][e];
      }
    }
    float top = sc[0][0];
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int e = 0; e < 4; ++e) top = fmaxf(top, sc[a][e]);
    top = max_groups(top);
    top = on ? top : -INFINITY;
    if (__any((top - m) * c > kSlack)) {     // (-inf) - (-inf) compares false
      const float mn = fmaxf(m, top);
      const float f = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m - mn) * c);
      m = mn;
      l *= f;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] *= f;
    }
    float mc = m == -INFINITY ? 0.f : m * c;   // a row that has seen nothing: its scores are -inf, or it does not list the tile
    if (__any(fabsf(mc) > kFar)) {
      const float off = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[a][e] -= off;
      mc = 0.f;
    }
    union { b8 b[2]; uint32_t w[8]; } pf;
    float sum = 0.f;
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float w = __builtin_amdgcn_exp2f(fmaf(sc[a][e], c, -mc));
        sum += w;
        pf.b[a >> 1][4 * (a & 1) + e] = (__bf16)w;
      }
    if constexpr (RUNS == 1) {
      sum = on ? sum : 0.f;
      const uint32_t keep = on ? 0xffffffffu : 0u;
#pragma unroll
      for (int x = 0; x < 8; ++x) pf.w[x] &= keep;
    }
    l += sum;
    auto values = [&](auto sel) {
      constexpr int U = decltype(sel)::value & 1, J = decltype(sel)::value >> 1, AT = BUF * 2 * TILE + TILE + 32 * U * D * 2;
      b8 w[4];
      read_values<AT, AT + 16 * D * 2>(va + 4 * J, w);
#pragma unroll
      for (int j = 0; j < 4; ++j) o[4 * J + j] = mfma_bf16(w[j], pf.b[U], o[4 * J + j]);
    };
    values(std::integral_constant<int, 0>{});
    values(std::integral_constant<int, 1>{});
    if constexpr (NT == 8) {
      values(std::integral_constant<int, 2>{});
      values(std::integral_constant<int, 3>{});
    }
  };

  // Turn t: tile t has arrived, tile t + 1 is sent for (past the last one from slot 0).
  Tile ta = next(), tb;
  fetch(ta, 0);
  auto turn = [&](const Tile& now, Tile& fresh, auto buf) {
    __builtin_amdgcn_s_waitcnt(0x0f70);
    __syncthreads();
    fresh = next();
    fetch(fresh, decltype(buf)::value ^ 1);
    uint32_t of = 0;
#pragma unroll
    for (int x = 0; x < RUNS; ++x) of |= now.of[x];
    if (of != 0) compute(now, buf);
  };
#pragma unroll 1
  while (ta.pos[0] >= 0) {
    turn(ta, tb, std::integral_constant<int, 0>{});
    if (tb.pos[0] < 0) break;
    turn(tb, ta, std::integral_constant<int, 1>{});
  }
  __builtin_amdgcn_s_waitcnt(0x0f70);              // nothing may arrive in LDS after the workgroup

  const float tot = sum_groups(l);
  if (!row_ok) return;
  if (sq.n_split > 1) {
    const int64_t part = sq.part0 + ((int64_t)(sq.n_rt - 1 - rt0) * sq.n_split + sh.split) * p.Hkv + sh.head;
    const int64_t row = part * 16 + n;
    float* po = p.part_o + row * D + 4 * g;
#pragma unroll
    for (int j = 0; j < NT; ++j) *reinterpret_cast<f4*>(po + 16 * j) = o[j];
    if (g == 0) {
      p.part_ml[2 * row] = m;
      p.part_ml[2 * row + 1] = tot;
    }
    return;
  }
  const int64_t row = (int64_t)(sq.q_row0 + row_q) * p.Hq + row_h;
  const float inv = tot > 0.f ? 1.f / tot : 0.f;
  if (p.lse != nullptr && g == 0) p.lse[row] = tot > 0.f ? fmaf(m, p.scale, __builtin_amdgcn_logf(tot) * kLn2) : -INFINITY;
  uint16_t* dst = static_cast<uint16_t*>(p.out) + row * D + 4 * g;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    i2 x;
    x[0] = (int)pack_bf16(o[j][0] * inv, o[j][1] * inv);
    x[1] = (int)pack_bf16(o[j][2] * inv, o[j][3] * inv);
    *reinterpret_cast<i2*>(dst + 16 * j) = x;
  }
}

}  // namespace

hipError_t launch_block_merge(const AttnArgs& p, hipStream_t s) {
  if (p.n_units == 0) return hipSuccess;
  block_merge_kernel<<<dim3((unsigned)(p.n_units + kMergeWaves - 1) / kMergeWaves), dim3(64 * kMergeWaves), 0, s>>>(p);
  return hipGetLastError();
}

hipError_t launch_block_tiles(int d, const AttnArgs& p, hipStream_t s) {
  if (p.n_units == 0) return hipSuccess;
  const dim3 grid((unsigned)p.n_units), block(64 * NW);
  if (d == 128) {
    if (p.block >= 64) block_tiles_kernel<128, 1><<<grid, block, 0, s>>>(p);
    else if (p.block == 32) block_tiles_kernel<128, 2><<<grid, block, 0, s>>>(p);
    else block_tiles_kernel<128, 4><<<grid, block, 0, s>>>(p);
  } else {
    if (p.block >= 64) block_tiles_kernel<64, 1><<<grid, block, 0, s>>>(p);
    else if (p.block == 32) block_tiles_kernel<64, 2><<<grid, block, 0, s>>>(p);
    else block_tiles_kernel<64, 4><<<grid, block, 0, s>>>(p);
  }
  return hipGetLastError();
}

}  // namespace dosa
