// Accumulated attention weights, the two kernels for many calls' shapes (see
// cache_weights.hip for what is computed and for the general kernel).
//
// Few rows (a decode step): a workgroup owns a range of keys for all heads.
// Its wavefronts hold the query rows of a kv head (or of a pair, whose 64-byte
// key rows share a line) and stream the keys, S = Q K^T: a lane then has four
// rows of one key, adds their weights, and the four lane groups meet in two
// swaps.  Bound by the key rows' bytes: 16 sequences, 288K cached keys of 8
// heads, 159 MB in 37 us.  The exponent takes one instruction more than a single
// multiply-add would (17 to 32 bf16 rows: 134 against 130 us, fewer rows the
// same), and no rounding of the normaliser comes with it.
//
// Many bf16 rows (a prompt): a wavefront holds 64 keys of a head as matrix
// operands, eight of them make 512 keys, and the query rows go past them in LDS
// tiles of 64 rows loaded one ahead, S^T = K Q^T on the 32x32x16 product: a
// lane has one row and adds the weights of 32 keys, one normaliser a lane.
// Prompts of 8192 and 1031 queries, 32 heads on 8: 0.39 ms, 760 TFLOP/s.  The
// vector units are busy 57% of it, the matrix units 30%, and the two hardly
// overlap: 200 registers leave one workgroup a CU, whose two wavefronts a SIMD
// run in step between barriers, and wait for them and for query tiles 31% of
// their time.  Of 190 vector instructions per 16 products (64 keys x 32 rows)
// 96 are the weights, the others addresses (with divisions by the group) and
// masks.  The chunks' work is uneven (the causal mask), so the rows are cut
// into more shares than the GPU holds at once: 0.46 ms with a quarter of them.
// Computing a block's weights under the next block's scores, or four row tiles
// in flight, did not help.
#include "attn_device.h"

namespace dosa {

namespace {

constexpr int kWaves = 8;

// ---------------------------------------------------------------------------
// few rows
// ---------------------------------------------------------------------------
template <bool F32, int D, int RT, int HP>
__global__ __launch_bounds__(64 * kWaves) void weights_rows_kernel(const WeightArgs p) {
  constexpr int NS = D / 32, TERMS = F32 ? 3 : 1, KT = 4 / HP, STEP = 16 * KT;
  constexpr int NB = F32 && RT == 2 ? 2 : 3;       // steps in registers: three would spill twice as much there
  constexpr int TAB = kWeightRowKeys;
  __shared__ __attribute__((aligned(16))) uint32_t scl[kWaves][64];
  __shared__ int slots[TAB];
  __shared__ float sums[kWaves][TAB];
  const CacheView& cv = p.cache;
  const WeightSeq& sq = p.s[find_seq(p.s, p.n_seq, (int)blockIdx.x, [](const WeightSeq& s) { return s.unit0; })];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = lane64(), n = lane & 15, g = lane >> 4;
  const int lo = ((int)blockIdx.x - sq.unit0) * p.range;
  const int cnt = sq.kv_len - lo < p.range ? sq.kv_len - lo : p.range;
  for (int i = threadIdx.x; i < p.range; i += 64 * kWaves)
    slots[i] = i < cnt ? cache_slot(cv.table, sq.b, cv.max_pages, cv.page_size, cv.num_pages, lo + i) : -1;
  __syncthreads();
  const int row_b = cv.Hkv * (D / 2), row_s = cv.Hkv * (D / 32);
  const int before = sq.kv_len - sq.q_len;
  const int rows = sq.q_len * p.group;
  const int groups = cv.Hkv / HP, nh = groups < kWaves ? groups : kWaves, slices = kWaves / nh;
  const int slice = wave / nh;
  const float scale = p.scale;
  const int s_key = lane % STEP, s_head = lane / STEP;

  if (slice < slices) {
    for (int hg = wave - slice * nh; hg < groups; hg += nh) {
      const int head = hg * HP;
      b8 qf[HP][RT][TERMS][NS];
      float ls[HP][RT][4];
      int pos[RT][4];
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        int r = 16 * i + n;
        r = r < rows ? r : rows - 1;
        const int query = r / p.group, gh = r - query * p.group;
#pragma unroll
        for (int w = 0; w < HP; ++w) {
          const int64_t at = (int64_t)(sq.q_row0 + query) * p.q_stride + (int64_t)((head + w) * p.group + gh) * D + g * (D / 4);
          if constexpr (F32) {
            const f4* src = reinterpret_cast<const f4*>(static_cast<const float*>(p.q) + at);
#pragma unroll
            for (int s = 0; s < NS; ++s) {
              const f4 x0 = src[2 * s], x1 = src[2 * s + 1];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                float tt[3];
                split3(e < 4 ? x0[e & 3] : x1[e & 3], tt);
#pragma unroll
                for (int k = 0; k < TERMS; ++k) qf[w][i][k][s][e] = (__bf16)tt[k];
              }
            }
          } else {
            const i4* src = reinterpret_cast<const i4*>(static_cast<const uint16_t*>(p.q) + at);
#pragma unroll
            for (int s = 0; s < NS; ++s) qf[w][i][0][s] = __builtin_bit_cast(b8, src[s]);
          }
        }
        // the rows whose scores this lane gets
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          int y = 16 * i + 4 * g + e;
          const bool ok = y < rows;
          y = ok ? y : rows - 1;
          const int yq = y / p.group;
          pos[i][e] = before + yq;
#pragma unroll
          for (int w = 0; w < HP; ++w) {
            const float lse = p.lse[(int64_t)(sq.q_row0 + yq) * p.Hq + (head + w) * p.group + (y - yq * p.group)];
            ls[w][i][e] = ok && lse > -INFINITY ? lse : INFINITY;   // no normaliser: gives nothing
          }
        }
      }
      struct Keys {
        uint32_t k[HP][KT][NS];
        uint32_t sc;
      };
      auto load = [&](Keys& st, int j) {       // step j of the range; past it, the last
        typedef uint32_t kvec __attribute__((ext_vector_type(NS)));
        const int last = (cnt - 1) / STEP;
        const int k0 = (j < last ? j : last) * STEP;
        const int ss = slots[k0 + s_key];
        const uint8_t* sb = cv.k_scales + (int64_t)(ss < 0 ? 0 : ss) * row_s + (head + s_head) * (D / 32);
        if constexpr (D == 128) st.sc = *reinterpret_cast<const uint32_t*>(sb);
        else st.sc = *reinterpret_cast<const uint16_t*>(sb);
#pragma unroll
        for (int a = 0; a < KT; ++a) {
          const int ks = slots[k0 + 16 * a + n];
          const uint8_t* kr = cv.k_codes + (int64_t)(ks < 0 ? 0 : ks) * row_b + head * (D / 2) + g * (D / 8);
#pragma unroll
          for (int w = 0; w < HP; ++w) {
            const kvec x = *reinterpret_cast<const kvec*>(kr + w * (D / 2));
#pragma unroll
            for (int s = 0; s < NS; ++s) st.k[w][a][s] = x[s];
          }
        }
      };
      auto compute = [&](const Keys& st, int j) {
        const int k0 = j * STEP;
        wave_sync();
        scl[wave][lane] = st.sc;
        wave_sync();
        const bool edge = lo + k0 + STEP - 1 > before;     // some key is past the first query
        float part[KT];
#pragma unroll
        for (int a = 0; a < KT; ++a) {
          part[a] = 0.f;
#pragma unroll
          for (int w = 0; w < HP; ++w) {
            const float ks = mx_scale(scl[wave][STEP * w + 16 * a + n], 8 * (D == 128 ? g : g >> 1));
            f4 s4[RT];
#pragma unroll
            for (int i = 0; i < RT; ++i) s4[i] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < NS; ++s) {
              const b8 kf = mx8(st.k[w][a][s], ks);
#pragma unroll
              for (int k = TERMS - 1; k >= 0; --k)
#pragma unroll
                for (int i = 0; i < RT; ++i) s4[i] = mfma_bf16(qf[w][i][k][s], kf, s4[i]);
            }
            if (edge) {
              const int key = lo + k0 + 16 * a + n;
#pragma unroll
              for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) s4[i][e] = key > pos[i][e] ? -INFINITY : s4[i][e];
            }
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) part[a] += weight_of(s4[i][e], scale, ls[w][i][e]);
          }
        }
#pragma unroll
        for (int a = 0; a < KT; ++a) {
          const float x = sum_groups(part[a]);
          float* to = &sums[wave][k0 + 16 * a + n];
          if (g == a) *to = hg < nh ? x : *to + x;     // first head group: nothing there yet
        }
      };
      const int n_step = (cnt + STEP - 1) / STEP;
      if (slice < n_step) {
        Keys st[NB];
#pragma unroll
        for (int j = 0; j < NB - 1; ++j) load(st[j], slice + j * slices);
        for (int j = slice; j < n_step;) {
#pragma unroll
          for (int x = 0; x < NB; ++x) {
            if (j < n_step) {
              load(st[(x + NB - 1) % NB], j + (NB - 1) * slices);
              compute(st[x], j);
              j += slices;
            }
          }
        }
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < cnt; i += 64 * kWaves) {
    const int sl = slots[i];
    const int first = (i / STEP) % slices * nh;
    float x = 0.f;
    for (int w = 0; w < nh; ++w) x += sums[first + w][i];
    if (sl >= 0) p.acc_out[sl] = (lo + i < before && p.acc != nullptr ? p.acc[sl] : 0.f) + x;
  }
}

// ---------------------------------------------------------------------------
// many bf16 rows
// ---------------------------------------------------------------------------
typedef float f16v __attribute__((ext_vector_type(16)));
__device__ __forceinline__ f16v mfma32(b8 a, b8 b, f16v c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Sum over the 32 lanes of a half, in every lane: rotations within 16 lanes,
// then a swap of the neighbouring 16.
template <int N>
__device__ __forceinline__ float add_rotated(float x) {
  return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x120 + N, 0xf, 0xf, false));
}
__device__ __forceinline__ float sum_half(float x) {
  x = add_rotated<8>(x);
  x = add_rotated<4>(x);
  x = add_rotated<2>(x);
  x = add_rotated<1>(x);
  const uint32_t u = __float_as_uint(x);
  auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

constexpr int kRowTile = 64;

template <int D>
__device__ __forceinline__ int q_chunk(int r, int c) {
  return D == 128 ? c ^ (r & 15) : c ^ ((r >> 1) & 7);
}

// First row of part `part` of a key chunk, and one behind its last: parts cut
// all the rows of the sequence evenly, so that a chunk's parts in front of
// its first visible row are empty.
__device__ __forceinline__ void part_rows(const WeightArgs& p, const WeightSeq& sq, int chunk, int part, int* r0, int* r1) {
  const int before = sq.kv_len - sq.q_len, key0 = chunk * kWeightChunk;
  const int seen = (key0 > before ? key0 - before : 0) * p.group;       // first row that sees the chunk
  const int rows = sq.q_len * p.group;
  const int64_t a = (int64_t)part * sq.part_rows, b = a + sq.part_rows;
  *r0 = (int)(a > seen ? a : seen);
  *r1 = (int)(b < rows ? b : rows);
}

template <int D>
__global__ __launch_bounds__(64 * kWaves) void weights_tiles_kernel(const WeightArgs p) {
  constexpr int NS = D / 16, CH = D / 8, RPI = 64 / CH, PER = kRowTile / RPI / kWaves;
  __shared__ __attribute__((aligned(1024))) uint8_t qt[2][kRowTile * D * 2];
  const CacheView& cv = p.cache;
  const WeightSeq& sq = p.s[find_seq(p.s, p.n_seq, (int)blockIdx.x, [](const WeightSeq& s) { return s.unit0; })];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = lane64(), n = lane & 31, h = lane >> 5;
  int u = (int)blockIdx.x - sq.unit0;
  const int head = u % cv.Hkv;
  u /= cv.Hkv;
  const int part = u % sq.n_part, chunk = u / sq.n_part;
  int r0, r1;
  part_rows(p, sq, chunk, part, &r0, &r1);
  if (r0 >= r1) return;                    // the join does not read this part
  const int before = sq.kv_len - sq.q_len;
  const int key0 = chunk * kWeightChunk + 64 * wave;       // of the wavefront
  const bool active = key0 < sq.kv_len;
  const float c = p.scale * kLog2e;

  // 64 keys as operands: lane (key l%32, h) holds dims [h D/2, (h+1) D/2)
  b8 kf[2][NS];
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    const int key = key0 + 32 * a + n;
    const int sl = key < sq.kv_len ? cache_slot(cv.table, sq.b, cv.max_pages, cv.page_size, cv.num_pages, key) : -1;
    const int64_t at = (int64_t)(sl < 0 ? 0 : sl) * cv.Hkv + head;
    const uint8_t* kr = cv.k_codes + at * (D / 2) + h * (D / 4);
    const uint8_t* sr = cv.k_scales + at * (D / 32) + h * (D / 64);
    uint32_t w[NS];
#pragma unroll
    for (int x = 0; x < NS / 4; ++x) {
      const i4 y = reinterpret_cast<const i4*>(kr)[x];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[4 * x + e] = (uint32_t)y[e];
    }
    uint32_t by = D == 128 ? *reinterpret_cast<const uint16_t*>(sr) : (uint32_t)*sr;
    by = sl < 0 ? 0u : by;
#pragma unroll
    for (int s = 0; s < NS; ++s) kf[a][s] = mx8(w[s], mx_scale(by, 8 * (s / 4)));
  }
  f16v acc[2];
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[a][e] = 0.f;

  const int lr = lane / CH, lch = lane % CH;
  const uint16_t* qg = static_cast<const uint16_t*>(p.q);
  float lse_n[2];
  auto fetch = [&](int buf, int base) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = (wave * PER + i) * RPI, row = at + lr;
      const int r = base + row < r1 ? base + row : r1 - 1;
      const int query = r / p.group, qh = head * p.group + (r - query * p.group);
      __builtin_amdgcn_global_load_lds(
          (const __attribute__((address_space(1))) void*)(qg + (int64_t)(sq.q_row0 + query) * p.q_stride + (int64_t)qh * D +
                                                          8 * q_chunk<D>(row, lch)),
          (__attribute__((address_space(3))) void*)(&qt[buf][at * D * 2]), 16, 0, 0);
    }
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int rr = base + 32 * y + n, r = rr < r1 ? rr : r1 - 1;
      const int query = r / p.group;
      lse_n[y] = p.lse[(int64_t)(sq.q_row0 + query) * p.Hq + head * p.group + (r - query * p.group)];
    }
  };

  fetch(0, r0);
  int buf = 0;
  for (int base = r0; base < r1; base += kRowTile) {
    __builtin_amdgcn_s_waitcnt(0x0f70);
    float lse[2] = {lse_n[0], lse_n[1]};
    __syncthreads();
    if (base + kRowTile < r1) fetch(buf ^ 1, base + kRowTile);
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int rb = base + 32 * y;
      // positions of the tile's first and last row
      const int p0 = before + rb / p.group, p1 = before + (rb + 31 < r1 ? rb + 31 : r1 - 1) / p.group;
      if (!active || rb >= r1 || p1 < key0) continue;
      const int row = 32 * y + n;
      f16v s[2];
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int e = 0; e < 16; ++e) s[a][e] = 0.f;
#pragma unroll
      for (int x = 0; x < NS; ++x) {
        const b8 qf = *reinterpret_cast<const b8*>(&qt[buf][row * D * 2 + 16 * q_chunk<D>(row, h * (CH / 2) + x)]);
#pragma unroll
        for (int a = 0; a < 2; ++a) s[a] = mfma32(kf[a][x], qf, s[a]);
      }
      const bool ok = rb + n < r1;
      const float ls = ok && lse[y] > -INFINITY ? lse[y] : INFINITY, lc = ls * kLog2e;   // no normaliser: gives nothing
      if (p0 < key0 + 63) {
        const int pos = before + (rb + n) / p.group;
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            s[a][e] = key0 + 32 * a + 8 * (e >> 2) + 4 * h + (e & 3) > pos ? -INFINITY : s[a][e];
      }
      // normalisers of ordinary size: one multiply-add an exponent (0.39 against
      // 0.41 ms); beyond, the normaliser is taken off before the change of base
      const bool far = __any(fabsf(lse[y]) > kFar);
      if (far) {
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int e = 0; e < 16; ++e) s[a][e] = fmaf(s[a][e], p.scale, -ls);
      }
      const float to2 = far ? kLog2e : c, off = far ? 0.f : lc;
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[a][e] += __builtin_amdgcn_exp2f(fmaf(s[a][e], to2, -off));
    }
    buf ^= 1;
  }
  // sum over the 32 rows' lanes (all of them get it); lane n then writes the
  // n-th of the 16 keys its half holds of each 32
  if (!active) return;
  float* out = p.part + ((int64_t)sq.part0 + (((int64_t)chunk * sq.n_part + part) * cv.Hkv + head)) * kWeightChunk + 64 * wave;
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    float mine = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float x = sum_half(acc[a][e]);
      mine = n == e ? x : mine;
    }
    if (n < 16) out[32 * a + 8 * (n >> 2) + 4 * h + (n & 3)] = mine;
  }
}

// Adds up the parts and heads of each key, in order.
__global__ __launch_bounds__(256) void weights_tiles_join_kernel(const WeightArgs p) {
  const CacheView& cv = p.cache;
  const WeightSeq& sq = p.s[find_seq(p.s, p.n_seq, (int)blockIdx.x, [](const WeightSeq& s) { return s.tile0; })];
  const int b = (int)blockIdx.x - sq.tile0, chunk = b / (kWeightChunk / 256);
  const int in = b % (kWeightChunk / 256) * 256 + (int)threadIdx.x, key = chunk * kWeightChunk + in;
  if (key >= sq.kv_len) return;
  const int sl = cache_slot(cv.table, sq.b, cv.max_pages, cv.page_size, cv.num_pages, key);
  // the chunk's shares with work are the last ones, from the one that holds
  // its first visible row on; theirs and their heads' sums lie one after another
  const int before = sq.kv_len - sq.q_len, key0 = chunk * kWeightChunk;
  const int64_t seen = (int64_t)(key0 > before ? key0 - before : 0) * p.group;
  const int first = (int)(seen / sq.part_rows), n = (sq.n_part - first) * cv.Hkv;
  const float* src = p.part + ((int64_t)sq.part0 + ((int64_t)chunk * sq.n_part + first) * cv.Hkv) * kWeightChunk + in;
  float x = 0.f;
  for (int i = 0; i < n; i += 32) {
    float v[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = src[(int64_t)(i + j < n ? i + j : n - 1) * kWeightChunk];
#pragma unroll
    for (int j = 0; j < 32; ++j) x += i + j < n ? v[j] : 0.f;
  }
  if (sl >= 0) p.acc_out[sl] = (key < sq.kv_len - sq.q_len && p.acc != nullptr ? p.acc[sl] : 0.f) + x;
}

template <bool F32, int D, int HP>
hipError_t rows_go(const WeightArgs& p, hipStream_t s) {
  const dim3 grid((unsigned)p.n_units), block(64 * kWaves);
  if (p.rt == 2) weights_rows_kernel<F32, D, 2, HP><<<grid, block, 0, s>>>(p);
  else weights_rows_kernel<F32, D, 1, HP><<<grid, block, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_weights_rows(bool f32, int d, const WeightArgs& p, hipStream_t s) {
  const bool pair = p.cache.Hkv % 2 == 0;
  if (f32) return d == 128 ? rows_go<true, 128, 1>(p, s) : rows_go<true, 64, 1>(p, s);
  if (d == 128) return pair ? rows_go<false, 128, 2>(p, s) : rows_go<false, 128, 1>(p, s);
  return pair ? rows_go<false, 64, 2>(p, s) : rows_go<false, 64, 1>(p, s);
}

hipError_t launch_weights_tiles(int d, const WeightArgs& p, hipStream_t s) {
  const dim3 grid((unsigned)p.n_units), block(64 * kWaves);
  if (d == 128) weights_tiles_kernel<128><<<grid, block, 0, s>>>(p);
  else weights_tiles_kernel<64><<<grid, block, 0, s>>>(p);
  return hipGetLastError();
}

hipError_t launch_weights_tiles_join(const WeightArgs& p, hipStream_t s) {
  weights_tiles_join_kernel<<<dim3((unsigned)p.n_tiles), dim3(256), 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace dosa
