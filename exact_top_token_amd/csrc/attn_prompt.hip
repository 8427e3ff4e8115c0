// Causal attention of bf16 prompts: workgroups of kWaves wavefronts, 32 query
// rows each, over tiles of 64 keys in LDS.
//
//   s_j = q . k_j,  m = max_j s_j,  p_j = 2^((s_j - m) c),  c = scale log2(e),
//   o = sum_j p_j v_j / sum_j p_j,  lse = scale m + ln sum_j p_j.
//
// Rows are the (query, group head) pairs of a kv head, so the heads of a group
// share the tiles.  Scores are computed transposed, S^T = K Q^T, with the
// 32x32x16 product: lane l then holds row l%32 and keys 8i + 4(l/32)..+3, and
// numbering the reduction slots of O^T = V^T P^T the same way makes its right
// operand without moving a value between lanes.  A row's statistics are one
// number a lane (its other half in lane l^32).  V^T comes out of row-major
// LDS tiles through the transposing LDS read.
//
// Tiles go from global memory to LDS without passing registers, key tiles two
// and value tiles one ahead.  A lane writes LDS at its own place in the
// wavefront's kilobyte, so the swizzle that spreads rows over the banks is
// applied to the address it reads from.
//
// A tile's weights are computed while the matrix unit works on the scores of
// the next tile: one block of code in which products, their LDS reads and the
// vector work alternate.  32K causal prompt, 32 heads on 8, d = 128: 7.6 to 8.1
// ms on different boards, 1090 to 1150 TFLOP/s, nine tenths of what a large
// library product reaches here; 2% slower with the two one after the other.
// Splitting the wavefronts of a SIMD into one that multiplies and one that does
// softmax, with a barrier at each change, took 8.8 ms: one wavefront alone
// issues vector work at two thirds of the rate of two.
//
// The running maximum is only moved when a score exceeds it by more than 8 in
// the exponent: weights then reach 2^8 and sums 2^8 n, both far inside fp32,
// and most tiles skip the rescaling of the outputs.  Weights are rounded to
// bf16 for the second product, since two terms of them would double it in a
// kernel that it bounds: outputs are off by 0.19% of their size (root mean
// square) where fp32 weights and one rounding at the end leave 0.14%.  The
// weights' sum is taken before the rounding.
#include "attn_device.h"

namespace dosa {

namespace {

typedef float f16v __attribute__((ext_vector_type(16)));
typedef short s4v __attribute__((ext_vector_type(4)));

typedef __attribute__((address_space(3))) uint8_t lbyte;
typedef __attribute__((address_space(3))) b8 lds_b8;
typedef __attribute__((address_space(3))) s4v lds_s4;

constexpr int kKeys = 64;      // keys of a tile
constexpr float kSlack = 8.f;  // exponent by which a score may exceed the running maximum

__device__ __forceinline__ f16v mfma32(b8 a, b8 b, f16v c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// 16-byte chunk of row `r` that holds logical chunk c.  Key tiles: 16 lanes
// read one chunk of 16 rows; value tiles: 16 lanes read 32 bytes of 4 rows.
template <int D>
__device__ __forceinline__ int k_chunk(int r, int c) {
  return D == 128 ? c ^ (r & 15) : c ^ ((r >> 1) & 7);
}
template <int D>
__device__ __forceinline__ int v_chunk(int r, int c) {
  return D == 128 ? c ^ ((r & 3) << 2) : c ^ (((r >> 1) & 1) << 2);
}

template <int D, int NW>
__global__ __launch_bounds__(64 * NW, 2) void prompt_kernel(const AttnArgs p) {
  constexpr int CH = D / 8;              // 16-byte chunks of a row
  constexpr int TILE = kKeys * D * 2;    // bytes of a tile
  constexpr int NS = D / 16, NT = D / 32;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2][2][TILE];   // [k, v][buffer]

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = lane64(), n = lane & 31, h = lane >> 5;
  const int unit = blockIdx.x;
  const AttnSeq& sq = p.s[find_seq(p.s, p.n_seq, unit, [](const AttnSeq& s) { return s.unit0; })];
  int u = unit - sq.unit0;
  const int head = u % p.Hkv;
  u /= p.Hkv;
  const int split = u % sq.n_split, rt = sq.n_rt - 1 - u / sq.n_split;   // last row tile first: it sees the most keys
  const int n_rows = sq.q_len * p.group;
  const int wg_row = rt * (32 * NW), row0 = wg_row + 32 * wave;
  const int before = sq.kv_len - sq.q_len;
  int r = row0 + n;
  const bool ok = r < n_rows;
  r = ok ? r : n_rows - 1;
  const int query = r / p.group, qh = head * p.group + (r - query * p.group);
  const int vis = before + query + 1;
  auto seen = [&](int row) { return before + (row < n_rows ? row : n_rows - 1) / p.group + 1; };
  const int key_lo = split * sq.split_len;
  int wg_end = seen(wg_row + 32 * NW - 1);
  wg_end = (int64_t)key_lo + sq.split_len < wg_end ? key_lo + sq.split_len : wg_end;
  const int first = __builtin_amdgcn_readfirstlane(seen(row0)), last = __builtin_amdgcn_readfirstlane(seen(row0 + 31));
  const bool active = row0 < n_rows;

  b8 qf[NS];
  {
    const i4* src = reinterpret_cast<const i4*>(static_cast<const uint16_t*>(p.q) + (int64_t)(sq.q_row0 + query) * p.q_stride +
                                                (int64_t)qh * D + 8 * h);
#pragma unroll
    for (int s = 0; s < NS; ++s) qf[s] = __builtin_bit_cast(b8, src[2 * s]);
  }
  f16v o[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[j][e] = 0.f;
  float m = -INFINITY, l = 0.f;
  const float c = p.scale * kLog2e;

  const uint16_t* kg = static_cast<const uint16_t*>(p.k) + sq.key_base * p.k_stride + head * D;
  const uint16_t* vg = static_cast<const uint16_t*>(p.v) + sq.key_base * p.v_stride + head * D;
  // a wavefront instruction fills 1 KB: 64 / CH rows
  constexpr int RPI = 64 / CH, PER = kKeys / RPI / NW;
  const int lr = lane / CH, lc = lane % CH;
  // key or value tile `i` of the range into its buffer; rows past the last
  // visible one repeat it (their scores are masked)
  auto fetch = [&](int which, const uint16_t* base, int64_t stride, int i) {
    const int key0 = key_lo + i * kKeys, lim = wg_end - 1 - key0;
    const uint16_t* from = base + (int64_t)key0 * stride;
#pragma unroll
    for (int x = 0; x < PER; ++x) {
      const int at = (wave * PER + x) * RPI, row = at + lr, src = row < lim ? row : lim;
      const int ch = which == 0 ? k_chunk<D>(row, lc) : v_chunk<D>(row, lc);
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(from + src * (int)stride + 8 * ch),
                                       (__attribute__((address_space(3))) void*)(&lds[which][i & 1][at * D * 2]), 16, 0, 0);
    }
  };

  // LDS addresses of a lane's operands in buffer 0; the rest are constants
  uint32_t ka[NS], va[NT];
#pragma unroll
  for (int s = 0; s < NS; ++s) ka[s] = n * (D * 2) + 16 * k_chunk<D>(n, 2 * s + h);
  // value operand: the lane supplies 8 bytes of one of 4 rows, gets one column of them
  const int i16 = lane & 15, vr = 4 * h + (i16 >> 2), vc = 16 * ((lane >> 4) & 1) + 4 * (i16 & 3);
#pragma unroll
  for (int j = 0; j < NT; ++j) va[j] = 2 * TILE + vr * (D * 2) + 16 * v_chunk<D>(vr, (32 * j + vc) >> 3) + (vc & 7) * 2;

  lbyte* const base = (lbyte*)&lds[0][0][0];
  // tiles of the workgroup, and those that this wavefront's rows see
  const int tiles = key_lo < wg_end ? (wg_end - key_lo + kKeys - 1) / kKeys : 0;
  const int end = last < wg_end ? last : wg_end;
  const int mine = active && key_lo < end ? (end - key_lo + kKeys - 1) / kKeys : 0;
  const int stop = vis < wg_end ? vis : wg_end;      // first key this lane's row does not see

  auto scores = [&](f16v* sc, int t) {
    lbyte* kt = base + (t & 1) * TILE;
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int e = 0; e < 16; ++e) sc[a][e] = 0.f;
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int a = 0; a < 2; ++a)
        sc[a] = mfma32(*(lds_b8*)(kt + ka[s] + 32 * a * (D * 2)), qf[s], sc[a]);
  };
  // One tile: the maximum of its scores, then its weights while the matrix
  // unit works on the next tile's scores, then its weighted values.
  auto step = [&](f16v* sc, f16v* next, int t) {
    const int key0 = key_lo + t * kKeys;
    if (key0 + kKeys > first || key0 + kKeys > wg_end) {
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          sc[a][e] = key0 + 32 * a + 8 * (e >> 2) + 4 * h + (e & 3) >= stop ? -INFINITY : sc[a][e];
    }
    float top = sc[0][0];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, sc[a][e]);
    {
      const uint32_t w = __float_as_uint(top);
      auto x = __builtin_amdgcn_permlane32_swap(w, w, false, false);
      top = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
    }
    if (__any((top - m) * c > kSlack)) {     // (-inf) - (-inf) compares false
      const float mn = fmaxf(m, top);
      const float f = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m - mn) * c);
      m = mn;
      l *= f;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[j][e] *= f;
    }
    float mc = m * c;
    if (__any(fabsf(mc) > kFar)) {         // or a row that has seen nothing
      const float off = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int e = 0; e < 16; ++e) sc[a][e] -= off;
      mc = 0.f;
    }
    // the tile after the wavefront's last is read too (it is there or never
    // filled; its scores are not used), so that this is one block of code
    scores(next, t + 1);
    b8 pf[4];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float x = __builtin_amdgcn_exp2f(fmaf(sc[a][e], c, -mc));
        l += x;
        pf[2 * a + (e >> 3)][e & 7] = (__bf16)x;
      }
    // a product, the operand four products on, and a seventh of the vector work
    __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
    for (int i = 0; i < 2 * NS; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (i < 2 * NS - 4) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x402, 112 / (2 * NS), 0);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        s4v x[2];
#pragma unroll
        for (int y = 0; y < 2; ++y)
          x[y] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (lds_s4*)(base + (t & 1) * TILE + va[j] + (16 * s + 8 * y) * (D * 2)));
        const b8 vf = __builtin_bit_cast(b8, __builtin_shufflevector(x[0], x[1], 0, 1, 2, 3, 4, 5, 6, 7));
        o[j] = mfma32(vf, pf[s], o[j]);
      }
    constexpr int N = 4 * NT, AHEAD = 4;
    __builtin_amdgcn_sched_group_barrier(0x100, 2 * AHEAD, 0);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (i < N - AHEAD) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
    }
  };
  auto ready = [&]() {                       // this wavefront's loads are in LDS, and everyone's
    __builtin_amdgcn_s_waitcnt(0x0f70);
    __syncthreads();
  };

  if (tiles > 0) {
    f16v sa[2], sb[2];
    fetch(0, kg, p.k_stride, 0);
    ready();
    if (tiles > 1) fetch(0, kg, p.k_stride, 1);
    fetch(1, vg, p.v_stride, 0);
    if (mine > 0) scores(sa, 0);
    auto turn = [&](f16v* sc, f16v* next, int t) {
      ready();
      if (t + 2 < tiles) fetch(0, kg, p.k_stride, t + 2);
      if (t + 1 < tiles) fetch(1, vg, p.v_stride, t + 1);
      if (t < mine) step(sc, next, t);
    };
#pragma unroll 1
    for (int t = 0; t < tiles; t += 2) {
      turn(sa, sb, t);
      if (t + 1 < tiles) turn(sb, sa, t + 1);
    }
  }

  {
    const uint32_t w = __float_as_uint(l);
    auto x = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    l = __uint_as_float(x[0]) + __uint_as_float(x[1]);
  }
  if (sq.n_split > 1) {
    const int64_t prow = ((int64_t)sq.part0 + (unit - sq.unit0)) * (32 * NW) + 32 * wave + n;
    float* po = p.part_o + prow * D;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<f4*>(po + 32 * j + 8 * e + 4 * h) =
            f4{o[j][4 * e], o[j][4 * e + 1], o[j][4 * e + 2], o[j][4 * e + 3]};
    if (h == 0) {
      p.part_ml[2 * prow] = m;
      p.part_ml[2 * prow + 1] = l;
    }
    return;
  }
  if (!ok) return;
  const int64_t row = (int64_t)(sq.q_row0 + query) * p.Hq + qh;
  if (p.lse != nullptr && h == 0) p.lse[row] = fmaf(m, p.scale, __builtin_amdgcn_logf(l) * kLn2);
  const float inv = 1.f / l;
  uint16_t* dst = static_cast<uint16_t*>(p.out) + row * D;
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      i2 x;
      x[0] = (int)pack_bf16(o[j][4 * e] * inv, o[j][4 * e + 1] * inv);
      x[1] = (int)pack_bf16(o[j][4 * e + 2] * inv, o[j][4 * e + 3] * inv);
      *reinterpret_cast<i2*>(dst + 32 * j + 8 * e + 4 * h) = x;
    }
}

}  // namespace

hipError_t launch_prompt(int d, const AttnArgs& p, hipStream_t s) {
  if (p.n_units == 0) return hipSuccess;
  const dim3 grid((unsigned)p.n_units), block(64 * kPromptWaves);
  if (d == 128) prompt_kernel<128, kPromptWaves><<<grid, block, 0, s>>>(p);
  else prompt_kernel<64, kPromptWaves><<<grid, block, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace dosa
