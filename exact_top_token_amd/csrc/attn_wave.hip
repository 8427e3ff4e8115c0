// Attention by independent wavefronts: each takes one 16-row tile of a kv
// head's query rows (or two) and one range of keys, and keeps everything in
// registers.  Rows are the queries of a sequence times the query heads that
// share the kv head, so a single token with grouped heads still fills the
// matrix instruction's rows.
//
//   s_j = q . k_j,  m = max_j s_j,  p_j = 2^((s_j - m) c),  c = scale log2(e),
//   o = sum_j p_j v_j / sum_j p_j,  lse = scale m + ln sum_j p_j,
//
// in one pass over the keys with the running maximum and sum in fp32.
//
// Layout.  The scores are computed transposed, S^T = K Q^T: the 16x16 product
// then leaves lane l with row l%16 and keys 4(l/16)..+3 of each 16-key tile,
// which is what the second product, O^T = V^T P^T, wants of its right operand
// when its reduction slots are numbered the same way.  So the weights go from
// one product to the other without leaving their lane, and the running
// statistics of a row sit in the lanes that hold its outputs.  V^T needs, per
// lane, several keys of one dimension: lane n of 16 loads D/16 neighbouring
// dimensions of its keys and swaps halves with v_perm, so value rows stay
// row-major in memory and are read with whole-row bursts.
//
// 4-bit rows become bf16 in the converter (exact), 32-dimension blocks match a
// lane's share of a key row.  The weights are rounded to bf16 before the second
// product (2^-9 relative at most each, which averages out over keys; the sum in
// the denominator is taken before the rounding; two bf16 terms would double
// that product); with fp32 queries both the queries and the weights go as three
// bf16 terms, which keeps fp32 products.
//
// Bound, over a long cache, by the cache lines a CU may wait for at once (a
// wavefront's requests are 64 bytes a row; see HP): decode of 64 sequences x 2
// queries, 64 heads on 8, d = 128, over 2.35M cached keys, 2.56 GB: 0.48 ms, 5.3
// TB/s, and 14 us of join.  2048 selected keys for each of 64 queries, 144 MB
// in 64-byte rows: 38 us and 8 us of join, no unit busy more than two fifths of
// it: a wavefront has eight steps, and waits for an index, a page and a row in
// turn before the first.  One token over 4133 keys (fp32, d = 64): 6 + 6 us,
// latency.
#include <type_traits>

#include "attn_device.h"

namespace dosa {

namespace {

constexpr int kWaves = 8;   // largest wavefronts per workgroup

template <int SRC, int RT, int HP>
struct SrcTraits {
  static constexpr bool MX = SRC == A_MX || SRC == A_MX32;
  static constexpr int KT = MX ? 4 / HP : (SRC == A_BF16 ? 2 : 1);   // 16-key tiles per step
  static constexpr int TERMS = SRC == A_MX32 ? 3 : 1;             // bf16 terms of queries and weights
  // steps in registers: one used, the others loading.  Three where they fit: with
  // fp32 queries they spill at d = 128 (decode of 32 x 2 queries over 870K keys in
  // pages of 16: 278 against 237 us, 2048 selected keys a query: 62 against 49)
  static constexpr int NB = MX && RT * HP == 1 && TERMS == 1 ? 3 : 2;
  static constexpr bool F32IO = SRC == A_F32 || SRC == A_MX32;    // type of q and out
};

// One step's keys and values of a lane.
template <int SRC, int D, int HP>
struct Stage;

template <int D, int HP>
struct MxStage {
  static constexpr int NS = D / 32, KT = 4 / HP;
  uint32_t k[HP][KT][NS];   // per head and 16-key tile: key l%16, dims [g D/4, (g+1) D/4)
  uint32_t v[HP][4 * KT];   // per head and key 16t+4g+r: dims [n D/16, (n+1) D/16)
  uint32_t ks, vs;          // scale bytes of key l % (16 KT), head l / (16 KT)
  uint32_t mask;            // bit 4t+r: key 16t+4g+r is not there
  bool gone;                // key l % (16 KT) is not there (W_RUN: the step's page names none)
};
template <int D, int HP>
struct Stage<A_MX, D, HP> : MxStage<D, HP> {};
template <int D, int HP>
struct Stage<A_MX32, D, HP> : MxStage<D, HP> {};
template <int D, int HP>
struct Stage<A_BF16, D, HP> {
  i4 k[2][D / 32];
  uint32_t v[8][D / 32];
};
template <int D, int HP>
struct Stage<A_F32, D, HP> {
  float k[D / 4];
  float v[4][D / 16];
};

// A buffer descriptor over rows from a wavefront-uniform address on.
typedef __amdgpu_buffer_rsrc_t Rows;
__device__ __forceinline__ Rows rows_at(const uint8_t* p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, 0x7fffffff, 0x00027000);
}

// How a wavefront finds its keys: consecutive slots of one page (or contiguous
// rows) per step, a page look-up per key, or the selected keys.
enum Walk : int { W_RUN = 0, W_PAGES = 1, W_SEL = 2 };

// HP heads a wavefront: with two, a step is 32 keys of a head pair, whose
// 64-byte rows (d = 128) share a 128-byte line.  The lines a CU may wait for
// at once are what bounds this kernel, so they should be used whole: the decode
// step above takes 0.68 ms with one head a wavefront and the same ranges.
// More steps in flight do not help there (0.74 ms).
template <int SRC, int D, int RT, int HP, int WALK>
__global__ __launch_bounds__(64 * kWaves) void attn_kernel(const AttnArgs p) {
  using T = SrcTraits<SRC, RT, HP>;
  static_assert(HP == 1 || RT == 1, "one row tile per head of a pair");
  constexpr int R = RT * HP;             // row tiles of the wavefront
  constexpr int KT = T::KT, STEP = 16 * KT, TERMS = T::TERMS;
  constexpr int NT = D / 16, NS = D / 32;
  constexpr bool MX = T::MX, SEL = WALK == W_SEL;
  constexpr int NB = T::NB;
  __shared__ __attribute__((aligned(16))) uint32_t lds[MX ? kWaves : 1][3][64];   // key scales, value scales, slots

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int unit = blockIdx.x * (int)(blockDim.x >> 6) + wave;
  if (unit >= p.n_units) return;
  const AttnSeq& sq = p.s[find_seq(p.s, p.n_seq, unit, [](const AttnSeq& s) { return s.unit0; })];
  const int lane = lane64(), n = lane & 15, g = lane >> 4;
  int t = unit - sq.unit0;
  const int head = t % (p.Hkv / HP) * HP;
  t /= p.Hkv / HP;
  // last row tile first: under the causal mask it sees the most keys
  const int split = t % sq.n_split, rtu = t / sq.n_split, rt0 = sq.n_rt - 1 - rtu;

  // rows of this unit: dense (query, group head) pairs of the sequence; with
  // selected keys the group heads of one query
  const int tiles_q = SEL ? (p.group + 16 * RT - 1) / (16 * RT) : 1;
  const int q_first = SEL ? rt0 / tiles_q : 0;
  const int row_base = (SEL ? rt0 % tiles_q : rt0) * (16 * RT);
  const int n_rows = SEL ? p.group : sq.q_len * p.group;
  int row_q[R], row_h[R], vis[R];        // query, head, visible keys of row l%16 of each tile
  bool row_ok[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    int r = row_base + (HP == 1 ? 16 * i : 0) + n;
    row_ok[i] = r < n_rows;
    r = r < n_rows ? r : n_rows - 1;
    row_q[i] = q_first + r / p.group;
    row_h[i] = (head + (HP == 1 ? 0 : i)) * p.group + r % p.group;
    vis[i] = sq.kv_len - sq.q_len + row_q[i] + 1;
  }
  const int last_row = (row_base + 16 * RT < n_rows ? row_base + 16 * RT : n_rows) - 1;
  const int vis_last = sq.kv_len - sq.q_len + q_first + last_row / p.group + 1;
  const int vis_first = sq.kv_len - sq.q_len + q_first + row_base / p.group + 1;
  const int key_lo = split * sq.split_len;
  const int all = SEL ? p.topk : vis_last;
  const int key_hi = (int64_t)key_lo + sq.split_len < all ? key_lo + sq.split_len : all;

  // queries: lane (row l%16, g) holds dims [g D/4, (g+1) D/4)
  b8 qf[SRC == A_F32 ? 1 : R][TERMS][NS];
  float qs[SRC == A_F32 ? R : 1][D / 4];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t at = (int64_t)(sq.q_row0 + row_q[i]) * p.q_stride + (int64_t)row_h[i] * D + g * (D / 4);
    if constexpr (T::F32IO) {
      const float* src = static_cast<const float*>(p.q) + at;
      float x[D / 4];
#pragma unroll
      for (int e = 0; e < D / 16; ++e) {
        const f4 y = reinterpret_cast<const f4*>(src)[e];
        x[4 * e] = y[0]; x[4 * e + 1] = y[1]; x[4 * e + 2] = y[2]; x[4 * e + 3] = y[3];
      }
      if constexpr (SRC == A_F32) {
#pragma unroll
        for (int e = 0; e < D / 4; ++e) qs[i][e] = x[e];
      } else {
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float tt[3];
            split3(x[8 * s + e], tt);
#pragma unroll
            for (int w = 0; w < TERMS; ++w) qf[i][w][s][e] = (__bf16)tt[w];
          }
      }
    } else {
      const i4* src = reinterpret_cast<const i4*>(static_cast<const uint16_t*>(p.q) + at);
#pragma unroll
      for (int s = 0; s < NS; ++s) qf[i][0][s] = __builtin_bit_cast(b8, src[s]);
    }
  }

  f4 o[R][NT];
  float m[R], l[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int j = 0; j < NT; ++j) o[i][j] = f4{0.f, 0.f, 0.f, 0.f};
  }
  const float c = p.scale * kLog2e;

  // ---- where a step's rows are ----
  const CacheView& cv = p.cache;
  const int row_b = cv.Hkv * (D / 2), row_s = cv.Hkv * (D / 32);
  const int64_t sel_row = SEL ? (int64_t)(sq.q_row0 + q_first) * p.topk : 0;
  const int32_t* table = MX ? cv.table + (int64_t)sq.b * cv.max_pages : nullptr;
  const uint32_t k_off = n * row_b + g * (D / 8), v_off = 4 * g * row_b + n * (D / 32);
  const int s_key = lane % STEP, s_head = MX ? lane / STEP : 0;      // whose scales this lane loads
  const uint32_t s_off = s_key * row_s + s_head * (D / 32);

  // Loads are issued without branches, for a step past the range too (which
  // repeats its last keys): a wait then counts the younger loads exactly.
  // Selected keys: position and page of a key are loaded one and two steps
  // before its rows.
  int next_pos = -1, next_page = -1, pos2 = -1;
  auto entry = [&](int e) -> int {       // logical position of entry e of the range, -1 behind it
    if constexpr (SEL) {
      const int pos = p.idx[sel_row + (e < key_hi ? e : key_hi - 1)];
      return e < key_hi && pos < vis_first ? pos : -1;
    } else {
      return e < key_hi ? e : -1;
    }
  };
  auto page_of = [&](int pos) -> int {
    const int pg = (pos < 0 ? 0 : pos) / cv.page_size;
    return table[pg];
  };
  // page of the step at key0 (of the last key behind the range), through the
  // scalar cache: a line holds sixteen pages
  auto run_page = [&](int key0) -> int {
    const int at = key0 < key_hi ? key0 : key_hi - 1;
    return ((const __attribute__((address_space(4))) int32_t*)table)[at / cv.page_size];
  };
  auto scale_bytes = [&](const uint8_t* a) -> uint32_t {
    if constexpr (D == 128) return *reinterpret_cast<const uint32_t*>(a);
    else return *reinterpret_cast<const uint16_t*>(a);
  };
  auto start = [&]() {
    if constexpr (MX && WALK != W_RUN) {
      next_pos = entry(key_lo + s_key);
      pos2 = entry(key_lo + STEP + s_key);
      next_page = page_of(next_pos);
    } else if constexpr (MX) {
      next_page = run_page(key_lo);
    }
  };

  auto load = [&](Stage<SRC, D, HP>& st, int key0) {
    if constexpr (MX) {
      typedef uint32_t kvec __attribute__((ext_vector_type(NS)));
      const uint8_t *kb = cv.k_codes + head * (D / 2), *vb = cv.v_codes + head * (D / 2);
      const uint8_t *ksb = cv.k_scales + head * (D / 32), *vsb = cv.v_scales + head * (D / 32);
      if constexpr (WALK == W_RUN) {
        const int from = key0 < key_hi ? key0 : (key_hi - 1) / STEP * STEP;
        int page = next_page;
        const bool bad = (uint32_t)page >= (uint32_t)cv.num_pages;
        page = bad ? 0 : page;
        const int64_t slot = (int64_t)page * cv.page_size + from % cv.page_size;
        next_page = run_page(key0 + STEP);
        // scalar bases, one lane offset per kind, scalar row offsets
        const Rows k1 = rows_at(kb + slot * row_b), v1 = rows_at(vb + slot * row_b);
        const Rows ks1 = rows_at(ksb + slot * row_s), vs1 = rows_at(vsb + slot * row_s);
        // the scales of keys past the range and of a step without a page (which
        // reads page 0) become zero bytes, which keeps whatever their slots hold
        // finite: a masked key's weight of 0 is still multiplied by its values
        st.mask = bad ? 0xffffu : 0u;
        st.gone = bad;
        if constexpr (D == 128) {
          st.ks = __builtin_amdgcn_raw_buffer_load_b32(ks1, s_off, 0, 0);
          st.vs = __builtin_amdgcn_raw_buffer_load_b32(vs1, s_off, 0, 0);
        } else {
          st.ks = __builtin_amdgcn_raw_buffer_load_b16(ks1, s_off, 0, 0);
          st.vs = __builtin_amdgcn_raw_buffer_load_b16(vs1, s_off, 0, 0);
        }
#pragma unroll
        for (int a = 0; a < KT; ++a)
#pragma unroll
          for (int w = 0; w < HP; ++w) {
            const int off = 16 * a * row_b + w * (D / 2);
            if constexpr (D == 128) {
              const auto x = __builtin_amdgcn_raw_buffer_load_b128(k1, k_off, off, 0);
#pragma unroll
              for (int s = 0; s < NS; ++s) st.k[w][a][s] = x[s];
            } else {
              const auto x = __builtin_amdgcn_raw_buffer_load_b64(k1, k_off, off, 0);
#pragma unroll
              for (int s = 0; s < NS; ++s) st.k[w][a][s] = x[s];
            }
          }
#pragma unroll
        for (int a = 0; a < 4 * KT; ++a)
#pragma unroll
          for (int w = 0; w < HP; ++w) {
            const int off = ((a >> 2) * 16 + (a & 3)) * row_b + w * (D / 2);
            if constexpr (D == 128) st.v[w][a] = __builtin_amdgcn_raw_buffer_load_b32(v1, v_off, off, 0);
            else st.v[w][a] = __builtin_amdgcn_raw_buffer_load_b16(v1, v_off, off, 0);
          }
      } else {
        const int pos = next_pos;
        const bool there = pos >= 0 && (uint32_t)next_page < (uint32_t)cv.num_pages;
        const int slot = there ? next_page * cv.page_size + pos % cv.page_size : -1;
        // the next steps' page and position go out before this step's rows, so
        // that waiting for them does not wait for these
        next_pos = pos2;
        next_page = page_of(next_pos);
        pos2 = entry(key0 + 2 * STEP + s_key);
        const int64_t safe = slot < 0 ? 0 : slot;
        st.ks = scale_bytes(ksb + safe * row_s + s_head * (D / 32));
        st.vs = scale_bytes(vsb + safe * row_s + s_head * (D / 32));
        wave_sync();
        lds[wave][2][lane] = (uint32_t)slot;
        wave_sync();
        st.mask = 0;
#pragma unroll
        for (int a = 0; a < KT; ++a) {
          const int ksl = (int)lds[wave][2][16 * a + n];
          const uint8_t* kr = kb + (int64_t)(ksl < 0 ? 0 : ksl) * row_b + g * (D / 8);
#pragma unroll
          for (int w = 0; w < HP; ++w) {
            const kvec x = *reinterpret_cast<const kvec*>(kr + w * (D / 2));
#pragma unroll
            for (int s = 0; s < NS; ++s) st.k[w][a][s] = x[s];
          }
          const i4 vsl = *reinterpret_cast<const i4*>(&lds[wave][2][16 * a + 4 * g]);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            st.mask |= vsl[r] < 0 ? 1u << (4 * a + r) : 0u;
            const uint8_t* y = vb + (int64_t)(vsl[r] < 0 ? 0 : vsl[r]) * row_b + n * (D / 32);
#pragma unroll
            for (int w = 0; w < HP; ++w) {
              if constexpr (D == 128) st.v[w][4 * a + r] = *reinterpret_cast<const uint32_t*>(y + w * (D / 2));
              else st.v[w][4 * a + r] = *reinterpret_cast<const uint16_t*>(y + w * (D / 2));
            }
          }
        }
        st.gone = slot < 0;
      }
    } else {
      // contiguous rows; rows past the range repeat its last one
      const int from = key0 < key_hi ? key0 : key_hi - 1;
      const int last = key_hi - 1 - from;
      const int64_t r0 = sq.key_base + from;
      if constexpr (SRC == A_BF16) {
        const uint16_t* kb = static_cast<const uint16_t*>(p.k) + r0 * p.k_stride + head * D;
        const uint16_t* vb = static_cast<const uint16_t*>(p.v) + r0 * p.v_stride + head * D;
#pragma unroll
        for (int a = 0; a < KT; ++a) {
          const int kr = 16 * a + n < last ? 16 * a + n : last;
          const i4* x = reinterpret_cast<const i4*>(kb + kr * p.k_stride + g * (D / 4));
#pragma unroll
          for (int s = 0; s < NS; ++s) st.k[a][s] = x[s];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int vr = 16 * a + 4 * g + r < last ? 16 * a + 4 * g + r : last;
            const uint16_t* y = vb + vr * p.v_stride + n * NT;
            if constexpr (D == 128) {
              const i4 z = *reinterpret_cast<const i4*>(y);
#pragma unroll
              for (int e = 0; e < 4; ++e) st.v[4 * a + r][e] = (uint32_t)z[e];
            } else {
              const i2 z = *reinterpret_cast<const i2*>(y);
#pragma unroll
              for (int e = 0; e < 2; ++e) st.v[4 * a + r][e] = (uint32_t)z[e];
            }
          }
        }
      } else {
        const float* kb = static_cast<const float*>(p.k) + r0 * p.k_stride + head * D;
        const float* vb = static_cast<const float*>(p.v) + r0 * p.v_stride + head * D;
        const int kr = n < last ? n : last;
        const f4* x = reinterpret_cast<const f4*>(kb + kr * p.k_stride + g * (D / 4));
#pragma unroll
        for (int e = 0; e < D / 16; ++e) {
          const f4 z = x[e];
          st.k[4 * e] = z[0]; st.k[4 * e + 1] = z[1]; st.k[4 * e + 2] = z[2]; st.k[4 * e + 3] = z[3];
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int vr = 4 * g + r < last ? 4 * g + r : last;
          const f4* y = reinterpret_cast<const f4*>(vb + vr * p.v_stride + n * NT);
#pragma unroll
          for (int e = 0; e < NT / 4; ++e) {
            const f4 z = y[e];
            st.v[r][4 * e] = z[0]; st.v[r][4 * e + 1] = z[1]; st.v[r][4 * e + 2] = z[2]; st.v[r][4 * e + 3] = z[3];
          }
        }
      }
    }
  };

  auto compute = [&](const Stage<SRC, D, HP>& st, int key0) {
    f4 sc[R][KT];
    f4 vscale[HP][KT];
    if constexpr (MX) {
      wave_sync();
      const bool in = !st.gone && (WALK != W_RUN || key0 + s_key < key_hi);
      lds[wave][0][lane] = in ? st.ks : 0u;
      lds[wave][1][lane] = in ? st.vs : 0u;
      wave_sync();
    }
    // ---- scores ----
#pragma unroll
    for (int a = 0; a < KT; ++a) {
#pragma unroll
      for (int i = 0; i < R; ++i) sc[i][a] = f4{0.f, 0.f, 0.f, 0.f};
      if constexpr (MX) {
#pragma unroll
        for (int w = 0; w < HP; ++w) {
          const float ksc = mx_scale(lds[wave][0][STEP * w + 16 * a + n], 8 * (D == 128 ? g : g >> 1));
          const i4 vb = *reinterpret_cast<const i4*>(&lds[wave][1][STEP * w + 16 * a + 4 * g]);
#pragma unroll
          for (int r = 0; r < 4; ++r) vscale[w][a][r] = mx_scale((uint32_t)vb[r], 8 * (D == 128 ? n >> 2 : n >> 3));
#pragma unroll
          for (int s = 0; s < NS; ++s) {
            const b8 kf = mx8(st.k[w][a][s], ksc);
#pragma unroll
            for (int x = TERMS - 1; x >= 0; --x)
#pragma unroll
              for (int i = w * RT; i < (w + 1) * RT; ++i) sc[i][a] = mfma_bf16(kf, qf[i][x][s], sc[i][a]);
          }
        }
      } else if constexpr (SRC == A_BF16) {
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
          for (int i = 0; i < RT; ++i) sc[i][a] = mfma_bf16(__builtin_bit_cast(b8, st.k[a][s]), qf[i][0][s], sc[i][a]);
      } else {
#pragma unroll
        for (int s = 0; s < D / 4; ++s)
#pragma unroll
          for (int i = 0; i < RT; ++i) sc[i][a] = mfma_f32(st.k[s], qs[i][s], sc[i][a]);
      }
    }
    // ---- masks: only steps that reach past some row's visible keys ----
    if constexpr (SEL) {
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int a = 0; a < KT; ++a)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if constexpr (MX) sc[i][a][r] = (st.mask >> (4 * a + r)) & 1u ? -INFINITY : sc[i][a][r];
    } else {
      const int edge = vis_first < key_hi ? vis_first : key_hi;
      bool part = key0 + STEP > edge;
      if constexpr (MX) part = part || __any(st.mask != 0u);
      if (part) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const int end = vis[i] < key_hi ? vis[i] : key_hi;
#pragma unroll
          for (int a = 0; a < KT; ++a)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              bool hide = key0 + 16 * a + 4 * g + r >= end;
              if constexpr (MX) hide = hide || ((st.mask >> (4 * a + r)) & 1u);
              sc[i][a][r] = hide ? -INFINITY : sc[i][a][r];
            }
        }
      }
    }
    // ---- running maximum and sum ----
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float top = sc[i][0][0];
#pragma unroll
      for (int a = 0; a < KT; ++a)
#pragma unroll
        for (int r = 0; r < 4; ++r) top = fmaxf(top, sc[i][a][r]);
      top = max_groups(top);
      if (__any(top > m[i])) {
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
    if constexpr (SRC == A_F32) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int i = 0; i < RT; ++i) o[i][j] = mfma_f32(st.v[r][j], sc[i][0][r], o[i][j]);
    } else {
#pragma unroll
      for (int u = 0; u < KT / 2; ++u) {
        b8 pf[R][TERMS];
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float x = sc[i][2 * u + (e >> 2)][e & 3];
            if constexpr (TERMS == 1) {
              pf[i][0][e] = (__bf16)x;
            } else {
              float tt[3];
              split3(x, tt);
#pragma unroll
              for (int w = 0; w < TERMS; ++w) pf[i][w][e] = (__bf16)tt[w];
            }
          }
        auto pair = [&](auto bsel, int w) {
          constexpr int B = decltype(bsel)::value;
          uint32_t x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if constexpr (MX) x[e] = mx2<B>(st.v[w][8 * u + e], vscale[w][2 * u + (e >> 2)][e & 3]);
            else x[e] = st.v[8 * u + e][B];
          }
          const b8 lo = __builtin_bit_cast(b8, i4{(int)lows(x[0], x[1]), (int)lows(x[2], x[3]), (int)lows(x[4], x[5]),
                                                  (int)lows(x[6], x[7])});
          const b8 hi = __builtin_bit_cast(b8, i4{(int)highs(x[0], x[1]), (int)highs(x[2], x[3]),
                                                  (int)highs(x[4], x[5]), (int)highs(x[6], x[7])});
#pragma unroll
          for (int y = TERMS - 1; y >= 0; --y)
#pragma unroll
            for (int i = w * RT; i < (w + 1) * RT; ++i) {
              o[i][2 * B] = mfma_bf16(lo, pf[i][y], o[i][2 * B]);
              o[i][2 * B + 1] = mfma_bf16(hi, pf[i][y], o[i][2 * B + 1]);
            }
        };
#pragma unroll
        for (int w = 0; w < HP; ++w) {
          pair(std::integral_constant<int, 0>{}, w);
          pair(std::integral_constant<int, 1>{}, w);
          if constexpr (NT == 8) {
            pair(std::integral_constant<int, 2>{}, w);
            pair(std::integral_constant<int, 3>{}, w);
          }
        }
      }
    }
  };

  if (key_lo < key_hi) {
    Stage<SRC, D, HP> st[NB];
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

  // ---- results: lane holds, of row l%16, dims NT (4g + r) + j ----
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const float tot = sum_groups(l[i]);
    if (sq.n_split > 1) {
      if (!row_ok[i]) continue;
      const int64_t part = sq.part0 + ((int64_t)rtu * sq.n_split + split) * p.Hkv + head + (HP == 1 ? 0 : i);
      const int64_t row = part * (16 * RT) + (HP == 1 ? 16 * i : 0) + n;
      float* po = p.part_o + row * D;
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int e = 0; e < NT / 4; ++e)
          reinterpret_cast<f4*>(po + NT * (4 * g + r))[e] =
              f4{o[i][4 * e][r], o[i][4 * e + 1][r], o[i][4 * e + 2][r], o[i][4 * e + 3][r]};
      if (g == 0) {
        p.part_ml[2 * row] = m[i];
        p.part_ml[2 * row + 1] = tot;
      }
    } else if (row_ok[i]) {
      const int64_t row = (int64_t)(sq.q_row0 + row_q[i]) * p.Hq + row_h[i];
      const float inv = tot > 0.f ? 1.f / tot : 0.f;
      if (p.lse != nullptr && g == 0)
        p.lse[row] = tot > 0.f ? fmaf(m[i], p.scale, __builtin_amdgcn_logf(tot) * kLn2) : -INFINITY;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if constexpr (T::F32IO) {
          float* dst = static_cast<float*>(p.out) + row * D + NT * (4 * g + r);
#pragma unroll
          for (int e = 0; e < NT / 4; ++e)
            reinterpret_cast<f4*>(dst)[e] = f4{o[i][4 * e][r] * inv, o[i][4 * e + 1][r] * inv, o[i][4 * e + 2][r] * inv,
                                               o[i][4 * e + 3][r] * inv};
        } else {
          uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + row * D + NT * (4 * g + r));
#pragma unroll
          for (int e = 0; e < NT / 2; ++e) dst[e] = pack_bf16(o[i][2 * e][r] * inv, o[i][2 * e + 1][r] * inv);
        }
      }
    }
  }
}

// Join of a row's key ranges: o = sum_s 2^((m_s - M) c) o_s / sum_s 2^((m_s -
// M) c) l_s with M = max m_s.  WPR wavefronts a row (one where there are few
// ranges, so that a launch is not all workgroups of a few loads), which take
// the ranges in turn, kBatch at a time: outputs, maxima and sums are loaded
// together, since the chain of dependent loads is what the launch waits for.
// The outputs of ranges that saw no key (l = 0) are not used.
template <bool F32IO, int D, int WPR, int kBatch>
__global__ __launch_bounds__(256) void attn_join_kernel(const AttnArgs p, int sel) {
  constexpr int PER = D / 64;
  __shared__ float so[4][D];
  __shared__ float sm[4][2];
  const int lane = lane64(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w0 = wave % WPR;
  const int unit = (int)blockIdx.x * (4 / WPR) + wave / WPR;
  if (unit >= p.n_join) return;        // WPR = 4: the whole workgroup
  const AttnSeq& sq = p.s[find_seq(p.s, p.n_seq, unit, [](const AttnSeq& s) { return s.join0; })];
  const int query = (unit - sq.join0) / p.Hq, qh = (unit - sq.join0) % p.Hq;
  const int head = qh / p.group, gh = qh % p.group, rows_u = 16 * p.rt;
  const int tiles_q = (p.group + rows_u - 1) / rows_u;
  const int r = (sel ? query % p.tok : query) * p.group + gh;
  const int rt0 = r / rows_u + (sel ? query / p.tok * tiles_q : 0), r_in = r % rows_u;
  const float c = p.scale * kLog2e;
  const int64_t first = sq.part0 + (int64_t)(sq.n_rt - 1 - rt0) * sq.n_split * p.Hkv + head;
  float M = -INFINITY, L = 0.f, o[PER] = {};
  for (int s0 = w0; s0 < sq.n_split; s0 += WPR * kBatch) {
    float v[kBatch][PER];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int s = s0 + WPR * i < sq.n_split ? s0 + WPR * i : s0;
      const float* src = p.part_o + ((first + (int64_t)s * p.Hkv) * rows_u + r_in) * D + PER * lane;
#pragma unroll
      for (int e = 0; e < PER; ++e) v[i][e] = src[e];
    }
    const int s = s0 + WPR * lane;
    const bool in = lane < kBatch && s < sq.n_split;
    const float* ml = p.part_ml + 2 * ((first + (int64_t)(in ? s : s0) * p.Hkv) * rows_u + r_in);
    float ms = ml[0], ls = in ? ml[1] : 0.f;
    if (!(ls > 0.f)) ms = -INFINITY;
    float top = ms;
#pragma unroll
    for (int x = kBatch / 2; x >= 1; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
    top = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(top)));
    const float Mn = fmaxf(M, top);
    if (Mn == -INFINITY) continue;
    const float f = __builtin_amdgcn_exp2f((M - Mn) * c);
    const float w = ms == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((ms - Mn) * c);
    L = L * f + w * ls;
#pragma unroll
    for (int e = 0; e < PER; ++e) o[e] *= f;
    M = Mn;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const float wi = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), i));
#pragma unroll
      for (int e = 0; e < PER; ++e) o[e] += wi > 0.f ? wi * v[i][e] : 0.f;
    }
  }
#pragma unroll
  for (int x = kBatch / 2; x >= 1; x >>= 1) L += __shfl_xor(L, x);
  L = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(L)));
  if constexpr (WPR > 1) {
    if (lane == 0) {
      sm[wave][0] = M;
      sm[wave][1] = L;
    }
#pragma unroll
    for (int e = 0; e < PER; ++e) so[wave][PER * lane + e] = o[e];
    __syncthreads();
    if (wave != 0) return;
    M = fmaxf(fmaxf(sm[0][0], sm[1][0]), fmaxf(sm[2][0], sm[3][0]));
    L = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) o[e] = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float f = sm[w][0] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((sm[w][0] - M) * c);
      L += f * sm[w][1];
#pragma unroll
      for (int e = 0; e < PER; ++e) o[e] += f * so[w][PER * lane + e];
    }
  }
  const float inv = L > 0.f ? 1.f / L : 0.f;
  const int64_t row = (int64_t)(sq.q_row0 + query) * p.Hq + qh;
  if (p.lse != nullptr && lane == 0)
    p.lse[row] = L > 0.f ? fmaf(M, p.scale, __builtin_amdgcn_logf(L) * kLn2) : -INFINITY;
  if constexpr (F32IO) {
    float* dst = static_cast<float*>(p.out) + row * D + PER * lane;
#pragma unroll
    for (int e = 0; e < PER; ++e) dst[e] = o[e] * inv;
  } else if constexpr (PER == 2) {
    reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + row * D)[lane] = pack_bf16(o[0] * inv, o[1] * inv);
  } else {
    static_cast<__bf16*>(p.out)[row * D + lane] = (__bf16)(o[0] * inv);
  }
}

constexpr bool from_cache(int src) { return src == A_MX || src == A_MX32; }

template <int SRC, int D, int RT, int HP>
hipError_t go(const AttnArgs& p, hipStream_t s) {
  // few units: smaller workgroups, so that they spread over more CUs
  const int waves = p.n_units >= 1024 ? kWaves : (p.n_units >= 512 ? 4 : 2);
  const dim3 grid((unsigned)((p.n_units + waves - 1) / waves)), block(64 * waves);
  if constexpr (from_cache(SRC)) {
    if (p.idx != nullptr) attn_kernel<SRC, D, RT, HP, W_SEL><<<grid, block, 0, s>>>(p);
    else if ((p.cache.page_size & 63) == 0) attn_kernel<SRC, D, RT, HP, W_RUN><<<grid, block, 0, s>>>(p);
    else attn_kernel<SRC, D, RT, HP, W_PAGES><<<grid, block, 0, s>>>(p);
  } else {
    attn_kernel<SRC, D, RT, HP, W_RUN><<<grid, block, 0, s>>>(p);
  }
  return hipGetLastError();
}

template <int SRC, int D>
hipError_t go_rt(const AttnArgs& p, hipStream_t s) {
  if constexpr (SRC == A_MX)
    if (p.hp == 2) return go<SRC, D, 1, 2>(p, s);
  if constexpr (attn_max_rt(SRC, D) == 2)
    if (p.rt == 2) return go<SRC, D, 2, 1>(p, s);
  return go<SRC, D, 1, 1>(p, s);
}

template <int D>
hipError_t go_src(int src, const AttnArgs& p, hipStream_t s) {
  switch (src) {
    case A_F32: return go_rt<A_F32, D>(p, s);
    case A_BF16: return go_rt<A_BF16, D>(p, s);
    case A_MX: return go_rt<A_MX, D>(p, s);
    default: return go_rt<A_MX32, D>(p, s);
  }
}

}  // namespace

hipError_t launch_attn(int src, int d, const AttnArgs& p, hipStream_t s) {
  if (p.n_units == 0) return hipSuccess;
  return d == 128 ? go_src<128>(src, p, s) : go_src<64>(src, p, s);
}

namespace {

template <bool F32IO, int D>
hipError_t join(const AttnArgs& p, hipStream_t s) {
  int most = 0;
  for (int i = 0; i < p.n_seq; ++i) most = most > p.s[i].n_split ? most : p.s[i].n_split;
  const int sel = p.idx != nullptr;
  // (a batch loads its last range again in place of those that are not there: 32768 rows of 2 ranges 32 us
  // sixteen at a time)
  if (most <= 4) attn_join_kernel<F32IO, D, 1, 4><<<dim3((unsigned)(p.n_join + 3) / 4), dim3(256), 0, s>>>(p, sel);
  else if (most <= 16) attn_join_kernel<F32IO, D, 1, 16><<<dim3((unsigned)(p.n_join + 3) / 4), dim3(256), 0, s>>>(p, sel);
  else attn_join_kernel<F32IO, D, 4, 16><<<dim3((unsigned)p.n_join), dim3(256), 0, s>>>(p, sel);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_join(int src, int d, const AttnArgs& p, hipStream_t s) {
  if (p.n_join == 0) return hipSuccess;
  const bool f32 = src == A_F32 || src == A_MX32 || src == A_P32;
  if (d == 128) return f32 ? join<true, 128>(p, s) : join<false, 128>(p, s);
  return f32 ? join<true, 64>(p, s) : join<false, 64>(p, s);
}

}  // namespace dosa
