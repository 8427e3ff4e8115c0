// Attention over pages of bf16 or fp32 rows by independent wavefronts: every
// visible key, or the keys of the blocks that a row of idx lists.  A wavefront
// takes one 16-row tile of a kv head's query rows (or two) and one range of
// keys, and keeps everything in registers.
//
//   s_j = q . k_j,  m = max_j s_j,  p_j = 2^((s_j - m) c),  c = scale log2(e),
//   o = sum_j p_j v_j / sum_j p_j,  lse = scale m + ln sum_j p_j,
//
// in one pass over the keys with the running maximum and sum in fp32.
//
// Scores are computed transposed, S^T = K Q^T: lane l then holds row l%16 and
// keys 4(l/16)..+3 of each 16-key tile, which is what the right operand of O^T =
// V^T P^T wants, so weights stay in their lanes.  A reduction's slots may be
// numbered freely as long as both operands agree, so a key row is read in runs
// of 64 bytes (four lanes of 16), and a value row whole (16 lanes).
//
// A 16-key tile lies in one page and one block.  Its page comes through the
// scalar cache, one step ahead of its rows (a listed block two), and its rows
// through a buffer descriptor that ends behind the tile's last key: rows
// behind it, and all rows of a tile without a page, arrive as zeros whatever
// memory holds there.  (A weight of 0 is still multiplied by a value.)
//
// Bound by memory: decode of 48 sequences, 64 heads on 8, d = 128, bf16, over
// 888K keys, 3.64 GB: 0.62 ms, 5.9 TB/s, and 8 us of join (fp32 keys 6.1 TB/s,
// d = 64 5.6).  32 listed blocks of 64 keys for each of 64 queries, 535 MB: 80 us
// and 7 of join; merging the two queries of a sequence, which share half of their
// blocks, took 10 us more than it saved, since the caches share them anyway.  One
// fp32 token over 5003 keys, d = 64: 6 + 5 us, latency.
#include "attn_device.h"

namespace dosa {

namespace {

constexpr int kWaves = 8;   // largest wavefronts per workgroup

// Exponent by which a score may exceed the running maximum: weights reach 2^8
// at most, and most steps skip the rescaling of the outputs.
constexpr float kSlack = 8.f;

template <bool F32, int D>
struct Row {
  static constexpr int SIZE = F32 ? 4 : 2;
  static constexpr int KT = F32 ? 1 : 2;           // 16-key tiles per step
  static constexpr int NK = D * SIZE / 64;         // 16-byte pieces of a key row a lane reads
  static constexpr int NV = F32 ? D / 16 : D / 32; // dwords of a value row a lane reads
};

// One step's keys and values of a lane, and the keys there are in each tile.
template <bool F32, int D>
struct Stage {
  using R = Row<F32, D>;
  i4 k[R::KT][R::NK];        // key l%16
  uint32_t v[4 * R::KT][R::NV];   // key 16a+4g+r
  int valid[R::KT];
};

typedef __amdgpu_buffer_rsrc_t Rows;
__device__ __forceinline__ Rows rows_at(const uint8_t* p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, bytes, 0x00027000);
}

template <bool F32, int D, int RT, bool SEL>
__global__ __launch_bounds__(64 * kWaves) void pages_kernel(const AttnArgs p) {
  using T = Row<F32, D>;
  constexpr int KT = T::KT, STEP = 16 * KT, NK = T::NK, NV = T::NV, NT = D / 16, SIZE = T::SIZE;
  constexpr int NB = 2;                  // steps in registers: one used, the other loading

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int unit = blockIdx.x * (int)(blockDim.x >> 6) + wave;
  if (unit >= p.n_units) return;
  const AttnSeq& sq = p.s[find_seq(p.s, p.n_seq, unit, [](const AttnSeq& s) { return s.unit0; })];
  const int lane = lane64(), n = lane & 15, g = lane >> 4;
  int t = unit - sq.unit0;
  const int head = t % p.Hkv;
  t /= p.Hkv;
  // last row tile first: under the causal mask it sees the most keys
  const int split = t % sq.n_split, rtu = t / sq.n_split, rt0 = sq.n_rt - 1 - rtu;

  // rows of this unit: dense (query, group head) pairs of the sequence; with
  // listed blocks the group heads of one query
  const int tiles_q = SEL ? (p.group + 16 * RT - 1) / (16 * RT) : 1;
  const int q_first = SEL ? rt0 / tiles_q : 0;
  const int row_base = (SEL ? rt0 % tiles_q : rt0) * (16 * RT);
  const int n_rows = SEL ? p.group : sq.q_len * p.group;
  int row_q[RT], row_h[RT], vis[RT];     // query, head, visible keys of row l%16 of each tile
  bool row_ok[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    int r = row_base + 16 * i + n;
    row_ok[i] = r < n_rows;
    r = r < n_rows ? r : n_rows - 1;
    row_q[i] = q_first + r / p.group;
    row_h[i] = head * p.group + r % p.group;
    vis[i] = sq.kv_len - sq.q_len + row_q[i] + 1;
  }
  const int last_row = (row_base + 16 * RT < n_rows ? row_base + 16 * RT : n_rows) - 1;
  const int vis_last = sq.kv_len - sq.q_len + q_first + last_row / p.group + 1;
  const int vis_first = sq.kv_len - sq.q_len + q_first + row_base / p.group + 1;
  const int key_lo = split * sq.split_len;
  const int all = SEL ? p.topk : vis_last;
  const int key_hi = (int64_t)key_lo + sq.split_len < all ? key_lo + sq.split_len : all;

  // queries: lane (row l%16, g) holds the dimensions of its key pieces
  i4 q[RT][NK];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const uint8_t* src = static_cast<const uint8_t*>(p.q) +
                         ((int64_t)(sq.q_row0 + row_q[i]) * p.q_stride + (int64_t)row_h[i] * D) * SIZE + 16 * g;
#pragma unroll
    for (int s = 0; s < NK; ++s) q[i][s] = *reinterpret_cast<const i4*>(src + 64 * s);
  }

  f4 o[RT][NT];
  float m[RT], l[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int j = 0; j < NT; ++j) o[i][j] = f4{0.f, 0.f, 0.f, 0.f};
  }
  const float c = p.scale * kLog2e;

  // ---- where a step's rows are ----
  const int row_b = p.Hkv * D * SIZE, page_size = p.cache.page_size, num_pages = p.cache.num_pages;
  const uint8_t *kb = static_cast<const uint8_t*>(p.k) + head * D * SIZE, *vb = static_cast<const uint8_t*>(p.v) + head * D * SIZE;
  scalar_i32* const table = (scalar_i32*)(p.cache.table + (int64_t)sq.b * p.cache.max_pages);
  const int lb = SEL ? __builtin_ctz(p.block) : 0, topn = p.topk >> lb;
  scalar_i32* const idx = SEL ? (scalar_i32*)(p.idx + ((int64_t)(sq.q_row0 + q_first) * p.Hkv + head) * topn) : nullptr;
  const int own = SEL ? (vis_first - 1) >> lb : 0;                          // the query's own block
  const int last_pg = SEL ? 0 : (int)p.page_div.quot(key_hi > 0 ? key_hi - 1 : 0);
  const int k_off = n * row_b + 16 * g, v_off = 4 * g * row_b + n * (F32 || D == 128 ? 16 : 8);

  // the next step's tiles: page number, place in the page, keys; listed blocks of the step after
  int n_page[KT], n_off[KT], n_valid[KT], n_blk[KT];
  int at_pg = 0, at_off = 0;             // walk over the pages
  auto block_of = [&](int e) -> int { return idx[(e < key_hi ? e : key_hi - 1) >> lb]; };
  auto place = [&](int key0) {
#pragma unroll
    for (int a = 0; a < KT; ++a) {
      const int e = key0 + 16 * a;
      if constexpr (SEL) {
        const int j = n_blk[a];
        const bool in = e < key_hi && (uint32_t)j <= (uint32_t)own;
        const int pos = in ? (j << lb) + (e & (p.block - 1)) : 0;
        const int left = vis_first - pos, pg = p.page_div.quot(pos);
        n_valid[a] = !in || left < 0 ? 0 : (left < 16 ? left : 16);
        n_off[a] = pos - pg * page_size;
        n_page[a] = table[pg];
        n_blk[a] = block_of(e + STEP);
      } else {
        const int left = key_hi - e;
        n_valid[a] = left < 0 ? 0 : (left < 16 ? left : 16);
        n_off[a] = at_off;
        n_page[a] = table[at_pg < last_pg ? at_pg : last_pg];
        at_off += 16;
        if (at_off == page_size) {
          at_off = 0;
          ++at_pg;
        }
      }
    }
  };
  auto start = [&]() {
    if constexpr (SEL) {
#pragma unroll
      for (int a = 0; a < KT; ++a) n_blk[a] = block_of(key_lo + 16 * a);
    } else {
      at_pg = p.page_div.quot(key_lo);
      at_off = key_lo - at_pg * page_size;
    }
    place(key_lo);
  };

  auto load = [&](Stage<F32, D>& st, int key0) {
    int page[KT], off[KT];
#pragma unroll
    for (int a = 0; a < KT; ++a) {
      const bool bad = (uint32_t)n_page[a] >= (uint32_t)num_pages;
      st.valid[a] = bad ? 0 : n_valid[a];
      page[a] = bad ? 0 : n_page[a];
      off[a] = n_off[a];
    }
    place(key0 + STEP);
#pragma unroll
    for (int a = 0; a < KT; ++a) {
      const int64_t at = ((int64_t)page[a] * page_size + off[a]) * row_b;
      const int bytes = st.valid[a] > 0 ? (st.valid[a] - 1) * row_b + D * SIZE : 0;
      const Rows k1 = rows_at(kb + at, bytes), v1 = rows_at(vb + at, bytes);
#pragma unroll
      for (int s = 0; s < NK; ++s)
        st.k[a][s] = __builtin_bit_cast(i4, __builtin_amdgcn_raw_buffer_load_b128(k1, k_off + 64 * s, 0, 0));
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if constexpr (!F32 && D == 64) {
          const auto x = __builtin_amdgcn_raw_buffer_load_b64(v1, v_off, r * row_b, 0);
          st.v[4 * a + r][0] = x[0];
          st.v[4 * a + r][1] = x[1];
        } else {
#pragma unroll
          for (int y = 0; y < NV / 4; ++y) {
            const auto x = __builtin_amdgcn_raw_buffer_load_b128(v1, v_off + 256 * y, r * row_b, 0);
#pragma unroll
            for (int e = 0; e < 4; ++e) st.v[4 * a + r][4 * y + e] = x[e];
          }
        }
      }
    }
  };

  auto compute = [&](const Stage<F32, D>& st, int key0) {
    f4 sc[RT][KT];
    // ---- scores ----
#pragma unroll
    for (int a = 0; a < KT; ++a) {
#pragma unroll
      for (int i = 0; i < RT; ++i) sc[i][a] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < NK; ++s)
        if constexpr (F32) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < RT; ++i)
              sc[i][a] = mfma_f32(__int_as_float(st.k[a][s][e]), __int_as_float(q[i][s][e]), sc[i][a]);
        } else {
#pragma unroll
          for (int i = 0; i < RT; ++i)
            sc[i][a] = mfma_bf16(__builtin_bit_cast(b8, st.k[a][s]), __builtin_bit_cast(b8, q[i][s]), sc[i][a]);
        }
    }
    // ---- masks: only steps that reach past some row's visible keys ----
    int least = st.valid[0];
#pragma unroll
    for (int a = 1; a < KT; ++a) least = least < st.valid[a] ? least : st.valid[a];
    if (least < 16 || (!SEL && key0 + STEP > vis_first)) {
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int a = 0; a < KT; ++a)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            bool hide = 4 * g + r >= st.valid[a];
            if constexpr (!SEL) hide = hide || key0 + 16 * a + 4 * g + r >= vis[i];
            sc[i][a][r] = hide ? -INFINITY : sc[i][a][r];
          }
    }
    // ---- running maximum and sum ----
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      float top = sc[i][0][0];
#pragma unroll
      for (int a = 0; a < KT; ++a)
#pragma unroll
        for (int r = 0; r < 4; ++r) top = fmaxf(top, sc[i][a][r]);
      top = max_groups(top);
      if (__any((top - m[i]) * c > kSlack)) {     // (-inf) - (-inf) compares false
        const float m_new = fmaxf(m[i], top);
        // a row that has seen nothing yet: weight 1 on empty sums
        const float f = m_new == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m[i] - m_new) * c);
        m[i] = m_new;
        l[i] *= f;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r) o[i][j][r] *= f;
      }
      float mc = m[i] * c;
      if (__any(fabsf(mc) > kFar)) {         // or a row that has seen nothing
        const float off = m[i] == -INFINITY ? 0.f : m[i];
#pragma unroll
        for (int a = 0; a < KT; ++a)
#pragma unroll
          for (int r = 0; r < 4; ++r) sc[i][a][r] -= off;
        mc = 0.f;
      }
#pragma unroll
      for (int a = 0; a < KT; ++a)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float e = __builtin_amdgcn_exp2f(fmaf(sc[i][a][r], c, -mc));
          sc[i][a][r] = e;
          l[i] += e;
        }
    }
    // ---- weighted values ----
    if constexpr (F32) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int i = 0; i < RT; ++i) o[i][j] = mfma_f32(__uint_as_float(st.v[r][j]), sc[i][0][r], o[i][j]);
    } else {
      // one row tile: weights as two bf16 terms, 16 significant bits.  The matrix unit waits for memory here, and
      // the result's rounding stays the only one that shows.  Two row tiles have no registers for that (32
      // sequences x 4 queries in groups of 8 over 871K keys 814 against 744 us): weights rounded to bf16, their
      // sum taken before, and outputs off by 0.23% of their size (root mean square) instead of 0.17%
      constexpr int TERMS = RT == 1 ? 2 : 1;
      b8 pf[RT][TERMS];
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = sc[i][e >> 2][e & 3];
          pf[i][0][e] = (__bf16)x;
          if constexpr (TERMS == 2) pf[i][1][e] = (__bf16)(x - (float)pf[i][0][e]);
        }
#pragma unroll
      for (int b = 0; b < NV; ++b) {
        uint32_t x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = st.v[e][b];
        const b8 lo = __builtin_bit_cast(b8, i4{(int)lows(x[0], x[1]), (int)lows(x[2], x[3]), (int)lows(x[4], x[5]),
                                                (int)lows(x[6], x[7])});
        const b8 hi = __builtin_bit_cast(b8, i4{(int)highs(x[0], x[1]), (int)highs(x[2], x[3]), (int)highs(x[4], x[5]),
                                                (int)highs(x[6], x[7])});
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int y = TERMS - 1; y >= 0; --y) {
            o[i][2 * b] = mfma_bf16(lo, pf[i][y], o[i][2 * b]);
            o[i][2 * b + 1] = mfma_bf16(hi, pf[i][y], o[i][2 * b + 1]);
          }
      }
    }
  };

  if (key_lo < key_hi) {
    Stage<F32, D> st[NB];
    start();
#pragma unroll
    for (int j = 0; j < NB - 1; ++j) load(st[j], key_lo + j * STEP);
    for (int key0 = key_lo; key0 < key_hi;) {
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        if (key0 < key_hi) {
          load(st[(j + NB - 1) % NB], key0 + (NB - 1) * STEP);
          compute(st[j], key0);
          key0 += STEP;
        }
      }
    }
  }

  // ---- results: lane holds, of row l%16, for each r: bf16 dims NT (4g + r) + j,
  // fp32 dims 64 (j / 4) + 4 (4g + r) + j % 4 ----
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const float tot = sum_groups(l[i]);
    if (!row_ok[i]) continue;
    if (sq.n_split > 1) {
      const int64_t part = sq.part0 + ((int64_t)rtu * sq.n_split + split) * p.Hkv + head;
      const int64_t row = part * (16 * RT) + 16 * i + n;
      float* po = p.part_o + row * D;
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int e = 0; e < NT / 4; ++e)
          *reinterpret_cast<f4*>(po + (F32 ? 64 * e + 4 * (4 * g + r) : NT * (4 * g + r) + 4 * e)) =
              f4{o[i][4 * e][r], o[i][4 * e + 1][r], o[i][4 * e + 2][r], o[i][4 * e + 3][r]};
      if (g == 0) {
        p.part_ml[2 * row] = m[i];
        p.part_ml[2 * row + 1] = tot;
      }
    } else {
      const int64_t row = (int64_t)(sq.q_row0 + row_q[i]) * p.Hq + row_h[i];
      const float inv = tot > 0.f ? 1.f / tot : 0.f;
      if (p.lse != nullptr && g == 0)
        p.lse[row] = tot > 0.f ? fmaf(m[i], p.scale, __builtin_amdgcn_logf(tot) * kLn2) : -INFINITY;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if constexpr (F32) {
          float* dst = static_cast<float*>(p.out) + row * D + 4 * (4 * g + r);
#pragma unroll
          for (int e = 0; e < NT / 4; ++e)
            *reinterpret_cast<f4*>(dst + 64 * e) = f4{o[i][4 * e][r] * inv, o[i][4 * e + 1][r] * inv,
                                                      o[i][4 * e + 2][r] * inv, o[i][4 * e + 3][r] * inv};
        } else {
          uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + row * D + NT * (4 * g + r));
#pragma unroll
          for (int e = 0; e < NT / 2; ++e) dst[e] = pack_bf16(o[i][2 * e][r] * inv, o[i][2 * e + 1][r] * inv);
        }
      }
    }
  }
}

template <bool F32, int D, int RT>
hipError_t go(const AttnArgs& p, hipStream_t s) {
  // few units: smaller workgroups, so that they spread over more CUs
  const int waves = p.n_units >= 1024 ? kWaves : (p.n_units >= 512 ? 4 : 2);
  const dim3 grid((unsigned)((p.n_units + waves - 1) / waves)), block(64 * waves);
  if (p.idx != nullptr) pages_kernel<F32, D, RT, true><<<grid, block, 0, s>>>(p);
  else pages_kernel<F32, D, RT, false><<<grid, block, 0, s>>>(p);
  return hipGetLastError();
}

template <bool F32, int D>
hipError_t go_rt(const AttnArgs& p, hipStream_t s) {
  if constexpr (attn_max_rt(F32 ? A_P32 : A_P16, D) == 2)
    if (p.rt == 2) return go<F32, D, 2>(p, s);
  return go<F32, D, 1>(p, s);
}

}  // namespace

hipError_t launch_pages(int src, int d, const AttnArgs& p, hipStream_t s) {
  if (p.n_units == 0) return hipSuccess;
  if (src == A_P32) return d == 128 ? go_rt<true, 128>(p, s) : go_rt<true, 64>(p, s);
  return d == 128 ? go_rt<false, 128>(p, s) : go_rt<false, 64>(p, s);
}

}  // namespace dosa
