// C-ABI entry points of the attention side: argument checks, the split of the
// work over the GPU, and the launches on the caller's stream.  Lengths travel
// as kernel arguments: no call copies to the device, allocates or waits.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>
#include <vector>

#include "attn_internal.h"
#include "host_common.h"

using namespace dosa;

namespace {

constexpr int64_t kMaxInt = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxTokens = (int64_t(1) << 31) - (1 << 16);   // positions a tile or two ahead stay int32

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Lengths, with a <= b for every sequence; total of each.
int check_lens(int32_t batch, const int32_t* a, const int32_t* b, const char* an, const char* bn, int64_t* ta,
               int64_t* tb) {
  if (batch < 0 || (batch > 0 && (a == nullptr || b == nullptr)))
    return fail(DOSA_ERR_INVALID_ARG, std::string("batch < 0 or ") + an + "/" + bn + " NULL");
  *ta = *tb = 0;
  for (int i = 0; i < batch; ++i) {
    if (a[i] < 0 || b[i] < 0 || a[i] > b[i])
      return fail(DOSA_ERR_INVALID_ARG, "sequence " + std::to_string(i) + ": need 0 <= " + an + " <= " + bn);
    *ta += a[i];
    *tb += b[i];
  }
  if (*ta > kMaxTokens || *tb > kMaxTokens) return fail(DOSA_ERR_UNSUPPORTED, "more than 2^31 - 2^16 tokens in a batch");
  return DOSA_OK;
}

int check_heads(int32_t Hq, int32_t Hkv, int32_t d) {
  if (Hq <= 0 || Hkv <= 0 || d <= 0 || Hq % Hkv != 0)
    return fail(DOSA_ERR_INVALID_ARG, "Hq must be a positive multiple of Hkv, d positive");
  if ((d != 64 && d != 128) || Hkv > 128 || Hq > 1024)
    return fail(DOSA_ERR_UNSUPPORTED, "d must be 64 or 128, Hkv at most 128, Hq at most 1024");
  return DOSA_OK;
}

// Rows of a sequence (queries times group heads) are int32 in the kernels.
int check_row_count(int32_t batch, const int32_t* q_lens, int32_t Hq, int32_t Hkv) {
  for (int b = 0; b < batch; ++b)
    if ((int64_t)q_lens[b] * (Hq / Hkv) > (int64_t(1) << 30))
      return fail(DOSA_ERR_UNSUPPORTED, "sequence " + std::to_string(b) + ": more than 2^30 query rows per kv head");
  return DOSA_OK;
}

// The GPU counts a launch's threads in 32 bits.
constexpr int64_t kLaunchThreads = int64_t(1) << 32;

int check_launch(const char* what, int64_t threads) {
  if (threads >= kLaunchThreads)
    return fail(DOSA_ERR_UNSUPPORTED, std::string(what) + ": a launch of 2^32 threads or more, split the call");
  return DOSA_OK;
}

int check_scale(float scale) {
  // a subnormal scale would be flushed, and 0 times a masked score's -inf is not
  // 0; the kernels multiply by scale * log2(e), and infinity times an equal
  // maximum's difference of 0 is not 0 either
  if (!(scale > 0.f) || !std::isnormal(scale) || !std::isfinite(scale * 1.44269504f))
    return fail(DOSA_ERR_INVALID_ARG, "scale must be positive, not subnormal, and scale * log2(e) finite in fp32");
  return DOSA_OK;
}

int check_float(int32_t dtype) {
  if (dtype != DOSA_F32 && dtype != DOSA_BF16) return fail(DOSA_ERR_UNSUPPORTED, "dtype must be fp32 or bf16");
  return DOSA_OK;
}

// A packed operand [tokens, H, d] with a stride between tokens: 16-byte rows,
// offsets within 64 tokens in 31 bits.
int check_rows(const char* name, const void* p, int64_t stride, int32_t H, int32_t d, int32_t dtype, int64_t tokens) {
  if (tokens == 0) return DOSA_OK;
  const int64_t size = dtype == DOSA_F32 ? 4 : 2;
  if (p == nullptr) return fail(DOSA_ERR_INVALID_ARG, std::string(name) + " is NULL");
  if (stride < (int64_t)H * d || (stride * size) % 16 != 0 || !aligned(p, 16))
    return fail(DOSA_ERR_INVALID_ARG, std::string(name) + ": token rows must not overlap and must be 16-byte aligned");
  if (stride > (int64_t(1) << 23)) return fail(DOSA_ERR_UNSUPPORTED, std::string(name) + ": token stride above 2^23");
  return DOSA_OK;
}

int check_pages(const int32_t* table, int32_t num_pages, int32_t page_size, int32_t max_pages, int32_t batch,
                const int32_t* kv_lens) {
  if (page_size <= 0 || page_size % 16 != 0 || num_pages <= 0 || max_pages < 0)
    return fail(DOSA_ERR_INVALID_ARG, "page_size must be a positive multiple of 16, num_pages positive");
  if ((int64_t)num_pages * page_size > kMaxTokens) return fail(DOSA_ERR_UNSUPPORTED, "more than 2^31 - 2^16 cache slots");
  for (int b = 0; b < batch; ++b) {
    if (kv_lens[b] > 0 && table == nullptr) return fail(DOSA_ERR_INVALID_ARG, "page_table is NULL");
    if ((int64_t)max_pages * page_size < kv_lens[b])
      return fail(DOSA_ERR_INVALID_ARG, "sequence " + std::to_string(b) + ": its page table row ends before its keys");
  }
  return DOSA_OK;
}

int check_cache(const dsa_cache* c, int32_t batch, const int32_t* kv_lens) {
  if (c == nullptr || c->k_codes == nullptr || c->k_scales == nullptr || c->v_codes == nullptr ||
      c->v_scales == nullptr)
    return fail(DOSA_ERR_INVALID_ARG, "cache or one of its buffers is NULL");
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 4) || !aligned(c->v_scales, 4))
    return fail(DOSA_ERR_INVALID_ARG, "cache codes must be 16-byte and scales 4-byte aligned");
  if (c->reserved != 0) return fail(DOSA_ERR_INVALID_ARG, "dsa_cache.reserved must be 0");
  return check_pages(c->page_table, c->num_pages, c->page_size, c->max_pages, batch, kv_lens);
}

CacheView view(const dsa_cache* c) {
  return CacheView{static_cast<uint8_t*>(c->k_codes), static_cast<uint8_t*>(c->k_scales),
                   static_cast<uint8_t*>(c->v_codes), static_cast<uint8_t*>(c->v_scales),
                   c->page_table, c->page_size, c->max_pages, c->num_pages, c->Hkv};
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// ---------------------------------------------------------------------------
// Work split of the attention kernels.  A unit is one row tile of one kv head
// over one key range.  The range length is the shortest (kMinKeys at least)
// for which the launch's units fit in kRounds rounds of what the GPU holds at
// once: a launch a little over a whole number of rounds would leave most of
// the GPU idle in its last one.  One round against two: 0.48 and 0.50 ms for a
// decode step of 64 sequences, 38 and 50 us for 2048 selected keys of 64
// queries, whose partial results halve.
// ---------------------------------------------------------------------------
constexpr int64_t kResident = 2048;      // wavefronts at eight a CU
constexpr int64_t kRounds = 1;
constexpr int64_t kMinKeys = 64;

struct AttnChunk {
  AttnArgs a;
  int64_t parts;
};

// Which kernel takes a sequence: bf16 prompts of more than 16 rows (queries
// times group heads) go to the tiled kernel, whose 256 rows share what is read
// of the keys; all else to the wavefront kernel.
constexpr int64_t kTiledRows = 16;
constexpr int64_t kTiledResident = 256;  // workgroups of the tiled kernel: one a CU
constexpr int64_t kTiledMinKeys = 512;

bool takes_tiled(int src, int64_t rows) { return src == A_BF16 && rows > kTiledRows; }

// Sequences b0.. of the batch that the kernel takes, at most kAttnSeqs with
// queries; returns the sequence after the last one seen, or -1 if the launch
// would be too large.
int plan_attn(AttnChunk& ch, int src, int d, bool tiled, int b0, int32_t batch, const int32_t* q_lens, const int32_t* kv_lens,
              int32_t Hq, int32_t Hkv, int32_t topk, int64_t* q_row, int64_t* k_row) {
  AttnArgs& a = ch.a;
  const bool sel = topk > 0;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.group = Hq / Hkv;
  a.topk = topk;
  a.n_seq = 0;
  int b = b0;
  int64_t most = 0;
  for (; b < batch && a.n_seq < kAttnSeqs; ++b) {
    if (q_lens[b] > 0 && takes_tiled(src, (int64_t)q_lens[b] * a.group) == tiled) {
      AttnSeq& s = a.s[a.n_seq++];
      s = AttnSeq{};
      s.q_row0 = (int32_t)*q_row;
      s.q_len = q_lens[b];
      s.kv_len = kv_lens[b];
      s.b = b;
      s.key_base = *k_row;
      most = std::max<int64_t>(most, sel ? a.group : (int64_t)q_lens[b] * a.group);
    }
    *q_row += q_lens[b];
    *k_row += kv_lens[b];
  }
  a.rt = tiled ? 2 * kPromptWaves : (most > 16 ? attn_max_rt(src, d) : 1);
  a.hp = tiled ? 1 : attn_heads(src, a.rt, Hkv);
  const int64_t tile = 16 * a.rt, heads = Hkv / a.hp;
  auto tiles = [&](const AttnSeq& s) -> int64_t {
    return sel ? (int64_t)s.q_len * ((a.group + tile - 1) / tile) : ((int64_t)s.q_len * a.group + tile - 1) / tile;
  };
  auto keys = [&](const AttnSeq& s) -> int64_t { return sel ? topk : s.kv_len; };
  std::stable_sort(a.s, a.s + a.n_seq, [&](const AttnSeq& x, const AttnSeq& y) { return keys(x) > keys(y); });
  const int64_t cap = kRounds * (tiled ? kTiledResident : kResident);
  auto units_at = [&](int64_t len) {
    int64_t n = 0;
    for (int i = 0; i < a.n_seq; ++i) n += tiles(a.s[i]) * heads * ((keys(a.s[i]) + len - 1) / len);
    return n;
  };
  // shortest range length in steps of 64 that keeps to the cap, or one range each
  int64_t lo = (tiled ? kTiledMinKeys : kMinKeys) / 64, hi = lo;
  for (int i = 0; i < a.n_seq; ++i) hi = std::max(hi, (keys(a.s[i]) + 63) / 64);
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (units_at(64 * mid) <= cap) hi = mid; else lo = mid + 1;
  }
  const int64_t len = 64 * lo;
  int64_t units = 0, join = 0, parts = 0;
  for (int i = 0; i < a.n_seq; ++i) {
    AttnSeq& s = a.s[i];
    const int64_t k = keys(s), nrt = tiles(s);
    int64_t n = std::max<int64_t>(1, (k + len - 1) / len);
    const int64_t sl = ((k + n - 1) / n + 63) / 64 * 64;
    n = (k + sl - 1) / sl;
    if (nrt * n * Hkv > kMaxInt || units + nrt * n * Hkv > kMaxInt) return -1;
    s.n_rt = (int32_t)nrt;
    s.n_split = (int32_t)n;
    s.split_len = (int32_t)sl;
    s.unit0 = (int32_t)units;
    s.join0 = (int32_t)join;
    s.part0 = (int32_t)parts;
    units += nrt * n * heads;
    if (n > 1) {
      join += (int64_t)s.q_len * Hq;
      parts += nrt * n * Hkv;
    }
    if (join > kMaxInt) return -1;
  }
  a.n_units = (int32_t)units;
  a.n_join = (int32_t)join;
  ch.parts = parts;
  return b;
}

size_t part_bytes(const AttnChunk& ch, int d) {
  const size_t rows = (size_t)ch.parts * 16 * ch.a.rt;
  return up256(rows * d * sizeof(float)) + up256(rows * 2 * sizeof(float));
}

int64_t attn_threads(const AttnChunk& ch, bool tiled) {
  return ch.a.n_units * int64_t(tiled ? 64 * kPromptWaves : 64);
}

// Bytes of partial results the call's launches need (each launch reuses them);
// 0 if a launch would be too large.  threads: those of the largest launch.
size_t attn_workspace(int src, int32_t batch, const int32_t* q_lens, const int32_t* kv_lens, int32_t Hq, int32_t Hkv,
                      int32_t d, int32_t topk, int64_t* threads = nullptr) {
  size_t most = 256;
  for (int tiled = 0; tiled < (src == A_BF16 ? 2 : 1); ++tiled) {
    int64_t qr = 0, kr = 0;
    for (int b = 0; b < batch;) {
      AttnChunk ch;
      b = plan_attn(ch, src, d, tiled != 0, b, batch, q_lens, kv_lens, Hq, Hkv, topk, &qr, &kr);
      if (b < 0) return 0;
      most = std::max(most, part_bytes(ch, d));
      if (threads != nullptr) *threads = std::max(*threads, attn_threads(ch, tiled != 0));
    }
  }
  return most;
}

int run_attn(int src, const AttnArgs& base, int32_t batch, const int32_t* q_lens, const int32_t* kv_lens, int32_t d,
             void* workspace, size_t workspace_bytes, hipStream_t stream) {
  // each kernel's first launch is planned once, for the size check and the run
  AttnChunk head[2];
  int next[2];
  int64_t qr[2] = {0, 0}, kr[2] = {0, 0}, threads = 0;
  const int classes = src == A_BF16 ? 2 : 1;
  size_t need = 256;
  for (int tiled = 0; tiled < classes; ++tiled) {
    head[tiled].a = base;
    next[tiled] = plan_attn(head[tiled], src, d, tiled != 0, 0, batch, q_lens, kv_lens, base.Hq, base.Hkv, base.topk,
                            &qr[tiled], &kr[tiled]);
    if (next[tiled] < 0) return fail(DOSA_ERR_UNSUPPORTED, "too many row tiles and key ranges for one launch");
    need = std::max(need, part_bytes(head[tiled], d));
    threads = std::max(threads, attn_threads(head[tiled], tiled != 0));
  }
  if (next[0] < batch || next[classes - 1] < batch) {
    need = attn_workspace(src, batch, q_lens, kv_lens, base.Hq, base.Hkv, d, base.topk, &threads);
    if (need == 0) return fail(DOSA_ERR_UNSUPPORTED, "too many row tiles and key ranges for one launch");
  }
  const int st = check_launch("attention", threads + 64 * 8);   // its last workgroup may be partly empty
  if (st != DOSA_OK) return st;
  if (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 16))
    return fail(DOSA_ERR_WORKSPACE, "workspace needs " + std::to_string(need) + " bytes, 16-byte aligned");
  for (int tiled = classes - 1; tiled >= 0; --tiled) {
    AttnChunk& ch = head[tiled];
    AttnArgs& a = ch.a;
    for (int b = next[tiled];;) {
      const size_t rows = (size_t)ch.parts * 16 * a.rt;
      a.part_o = static_cast<float*>(workspace);
      a.part_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + up256(rows * d * sizeof(float)));
      hipError_t e;
      if (a.n_units > 0) {
        PassScope ps(src == A_F32 || src == A_BF16 ? P_PROMPT : P_ATTEND, stream);
        e = tiled ? launch_prompt(d, a, stream) : launch_attn(src, d, a, stream);
        if (e != hipSuccess) return fail_hip(e, "attention kernel launch");
      }
      if (a.n_join > 0) {
        PassScope ps(P_ATTEND_JOIN, stream);
        e = launch_attn_join(src, d, a, stream);
        if (e != hipSuccess) return fail_hip(e, "attention join launch");
      }
      if (b >= batch) break;
      b = plan_attn(ch, src, d, tiled != 0, b, batch, q_lens, kv_lens, base.Hq, base.Hkv, base.topk, &qr[tiled],
                    &kr[tiled]);
    }
  }
  return DOSA_OK;
}

// ---------------------------------------------------------------------------
// Work split of the weights kernels.
//   few rows    ranges of keys, as long as 512 workgroups (two a CU) allow,
//               64..kWeightRowKeys
//   many rows   512-key chunks x heads x shares of the rows, the shares such
//               that about kWeightUnits workgroups have work; the causal half
//               of them has none
//   fp32        64-key tiles x shares
// ---------------------------------------------------------------------------
constexpr int64_t kWeightUnits = 2048;

WeightKind weight_kind(bool f32, int64_t rows) {
  if (rows <= kWeightRows) return WK_ROWS;
  return f32 ? WK_ANY : WK_TILES;
}

// The next launch of a kind: sequences from b0 on, at most kAttnSeqs of the
// kind; floats of partial sums in *floats.  Returns the sequence after the
// last one seen, or -1 if the launch would be too large.
int plan_weights(WeightArgs& a, WeightKind kind, bool f32, int64_t* floats, int b0, int32_t batch,
                 const int32_t* q_lens, const int32_t* kv_lens, int32_t Hq, int32_t Hkv, int64_t* q_row) {
  a.Hq = Hq;
  a.group = Hq / Hkv;
  a.n_seq = 0;
  int b = b0;
  int64_t work = 0, keys = 0, most = 0;
  for (; b < batch && a.n_seq < kAttnSeqs; ++b) {
    const int64_t rows = (int64_t)q_lens[b] * a.group;
    if (q_lens[b] > 0 && weight_kind(f32, rows) == kind) {
      WeightSeq& s = a.s[a.n_seq++];
      s = WeightSeq{};
      s.q_row0 = (int32_t)*q_row;
      s.q_len = q_lens[b];
      s.kv_len = kv_lens[b];
      s.b = b;
      keys += s.kv_len;
      most = std::max(most, rows);
      work += ((int64_t)s.kv_len + 63) / 64 * ((rows + 15) / 16 * Hkv);
    }
    *q_row += q_lens[b];
  }
  *floats = 0;
  a.n_units = a.n_tiles = 0;
  if (a.n_seq == 0) return b;
  std::stable_sort(a.s, a.s + a.n_seq, [](const WeightSeq& x, const WeightSeq& y) {
    return x.q_len != y.q_len ? x.q_len > y.q_len : x.kv_len > y.kv_len;
  });
  int64_t units = 0, tiles = 0, parts = 0;
  if (kind == WK_ROWS) {
    a.rt = most > 16 ? 2 : 1;
    int64_t range = 64;
    auto count = [&](int64_t r) {
      int64_t n = 0;
      for (int i = 0; i < a.n_seq; ++i) n += (a.s[i].kv_len + r - 1) / r;
      return n;
    };
    while (range < kWeightRowKeys && count(range) > 512) range += 64;
    a.range = (int32_t)range;
    for (int i = 0; i < a.n_seq; ++i) {
      a.s[i].unit0 = (int32_t)units;
      units += (a.s[i].kv_len + range - 1) / range;
    }
  } else if (kind == WK_TILES) {
    for (int i = 0; i < a.n_seq; ++i) {
      WeightSeq& s = a.s[i];
      const int64_t rows = (int64_t)s.q_len * a.group, nc = ((int64_t)s.kv_len + kWeightChunk - 1) / kWeightChunk;
      // shares in proportion to the sequence's part of the work
      const int64_t w = ((int64_t)s.kv_len + 63) / 64 * ((rows + 15) / 16 * Hkv);
      const int64_t want = w / std::max<int64_t>(work / (2 * kWeightUnits), 1) / (nc * Hkv);
      const int64_t np = std::min<int64_t>(std::max<int64_t>(want, 1), (rows + 127) / 128);
      s.part_rows = (int32_t)(((rows + np - 1) / np + 63) / 64 * 64);
      s.n_part = (int32_t)((rows + s.part_rows - 1) / s.part_rows);
      s.unit0 = (int32_t)units;
      s.tile0 = (int32_t)tiles;
      s.part0 = (int32_t)parts;
      units += nc * s.n_part * Hkv;
      parts += nc * s.n_part * Hkv;
      tiles += nc * (kWeightChunk / 256);
      if (units > kMaxInt) return -1;
    }
    *floats = parts * kWeightChunk;
    a.n_tiles = (int32_t)tiles;
  } else {
    const int64_t share = std::max<int64_t>(8, (work + kWeightUnits - 1) / kWeightUnits);   // row tiles x heads a workgroup
    for (int i = 0; i < a.n_seq; ++i) {
      WeightSeq& s = a.s[i];
      const int64_t nt = ((int64_t)s.kv_len + 63) / 64;
      const int64_t w = ((int64_t)s.q_len * a.group + 15) / 16 * Hkv;
      const int64_t np = std::min<int64_t>(64, std::max<int64_t>(1, w / share));
      s.n_part = (int32_t)np;
      s.unit0 = (int32_t)units;
      s.tile0 = (int32_t)tiles;
      s.part0 = (int32_t)parts;
      units += nt * np;
      tiles += nt;
      if (np > 1) parts += nt * np;
      if (units > kMaxInt) return -1;
    }
    *floats = parts * 64;
    a.n_tiles = parts > 0 ? (int32_t)tiles : 0;
  }
  if (units > kMaxInt) return -1;
  a.n_units = (int32_t)units;
  return b;
}

size_t weights_workspace(bool f32, int32_t batch, const int32_t* q_lens, const int32_t* kv_lens, int32_t Hq,
                         int32_t Hkv, int64_t* threads = nullptr) {
  size_t most = 256;
  for (int kind = 0; kind < WK_KINDS; ++kind) {
    int64_t qr = 0;
    for (int b = 0; b < batch;) {
      WeightArgs a;
      int64_t floats;
      b = plan_weights(a, (WeightKind)kind, f32, &floats, b, batch, q_lens, kv_lens, Hq, Hkv, &qr);
      if (b < 0) return 0;
      most = std::max(most, up256((size_t)floats * sizeof(float)));
      if (threads != nullptr) *threads = std::max({*threads, int64_t(a.n_units) * 512, int64_t(a.n_tiles) * 256});
    }
  }
  return most;
}

int cache_io(bool write, const dsa_cache* cache, void* k, int64_t k_stride, void* v, int64_t v_stride, int32_t dtype,
             const int32_t* q_lens, const int32_t* kv_lens, int32_t batch, int32_t* pos, const int32_t* seen_lens,
             hipStream_t stream) {
  int64_t tq, tk;
  int st = check_lens(batch, q_lens, kv_lens, "q_len", "kv_len", &tq, &tk);
  if (st == DOSA_OK) st = check_cache(cache, batch, kv_lens);
  if (st == DOSA_OK) st = check_heads(cache->Hkv, cache->Hkv, cache->d);
  if (st == DOSA_OK) st = check_float(dtype);
  if (st == DOSA_OK) st = check_rows("k", k, k_stride, cache->Hkv, cache->d, dtype, tq);
  if (st == DOSA_OK) st = check_rows("v", v, v_stride, cache->Hkv, cache->d, dtype, tq);
  if (st != DOSA_OK) return st;
  for (int b = 0; seen_lens != nullptr && b < batch; ++b)
    if (seen_lens[b] < kv_lens[b])
      return fail(DOSA_ERR_INVALID_ARG, "sequence " + std::to_string(b) + ": need seen_len >= kv_len");
  auto blocks = [&](int b) { return ((int64_t)q_lens[b] + kCacheTokens - 1) / kCacheTokens; };
  for (int b = 0; b < batch; ++b) {
    st = check_launch("cache append or read", blocks(b) * 256);
    if (st != DOSA_OK) return st;
  }
  CacheIoArgs a{};
  a.cache = view(cache);
  a.k = k;
  a.v = v;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.pos = pos;
  int64_t row = 0;
  for (int b = 0; b < batch;) {
    a.n_seq = 0;
    int32_t units = 0;
    for (; b < batch && a.n_seq < kAttnSeqs && (units + blocks(b)) * 256 < kLaunchThreads; ++b) {
      if (q_lens[b] > 0) {
        a.s[a.n_seq++] = CacheSeq{units, (int32_t)row, q_lens[b], kv_lens[b] - q_lens[b],
                                  (seen_lens != nullptr ? seen_lens[b] : kv_lens[b]) - q_lens[b], b};
        units += (int32_t)blocks(b);
      }
      row += q_lens[b];
    }
    if (a.n_seq == 0) continue;
    PassScope ps(write ? P_APPEND : P_READ, stream);
    const hipError_t e = write ? launch_cache_append(dtype == DOSA_F32, cache->d, a, stream)
                               : launch_cache_read(dtype == DOSA_F32, cache->d, a, stream);
    if (e != hipSuccess) return fail_hip(e, write ? "cache append launch" : "cache read launch");
  }
  return DOSA_OK;
}

// Ints of a sequence's eviction workspace.
int64_t evict_ints(int32_t kv_len, int32_t new_len) {
  const int64_t cap = std::min(new_len, kv_len - new_len);
  const int64_t rounds = ((int64_t)kv_len + 1023) / 1024, near = kEvictNear;
  return (kEvictHead + 2 * cap + std::max<int64_t>(0, rounds - near) * 1024 + 15) / 16 * 16;
}

size_t evict_workspace(int32_t batch, const int32_t* kv_lens, const int32_t* new_lens) {
  int64_t n = 0;
  for (int b = 0; b < batch; ++b) n += evict_ints(kv_lens[b], new_lens[b]);
  return up256((size_t)std::max<int64_t>(n, 1) * sizeof(int32_t));
}

template <class F>
int guarded(F f) {
  try {
    return f();
  } catch (...) {
    g_err = "internal error";
    return DOSA_ERR_HIP;
  }
}

template <class F>
size_t guarded_size(F f) {
  try {
    return f();
  } catch (...) {
    g_err = "internal error";
    return 0;
  }
}

}  // namespace

extern "C" {

size_t dsa_prompt_workspace_size(int32_t batch, const int32_t* q_lens, const int32_t* kv_lens, int32_t Hq, int32_t Hkv,
                                 int32_t d, int32_t dtype) {
  return guarded_size([&]() -> size_t {
    int64_t tq, tk;
    if (check_lens(batch, q_lens, kv_lens, "q_len", "kv_len", &tq, &tk) != DOSA_OK ||
        check_heads(Hq, Hkv, d) != DOSA_OK || check_row_count(batch, q_lens, Hq, Hkv) != DOSA_OK ||
        check_float(dtype) != DOSA_OK)
      return 0;
    return attn_workspace(dtype == DOSA_F32 ? A_F32 : A_BF16, batch, q_lens, kv_lens, Hq, Hkv, d, 0);
  });
}

int dsa_prompt_attention(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                         int64_t v_stride, int32_t dtype, const int32_t* q_lens, const int32_t* kv_lens, int32_t batch,
                         int32_t Hq, int32_t Hkv, int32_t d, float scale, void* out, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    int64_t tq, tk;
    int st = check_lens(batch, q_lens, kv_lens, "q_len", "kv_len", &tq, &tk);
    if (st == DOSA_OK) st = check_heads(Hq, Hkv, d);
    if (st == DOSA_OK) st = check_row_count(batch, q_lens, Hq, Hkv);
    if (st == DOSA_OK) st = check_float(dtype);
    if (st == DOSA_OK) st = check_scale(scale);
    if (st == DOSA_OK) st = check_rows("q", q, q_stride, Hq, d, dtype, tq);
    if (st == DOSA_OK) st = check_rows("k", k, k_stride, Hkv, d, dtype, tq > 0 ? tk : 0);
    if (st == DOSA_OK) st = check_rows("v", v, v_stride, Hkv, d, dtype, tq > 0 ? tk : 0);
    if (st == DOSA_OK) st = check_rows("out", out, (int64_t)Hq * d, Hq, d, dtype, tq);
    if (st != DOSA_OK) return st;
    AttnArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.out = out;
    a.lse = lse;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.scale = scale;
    return run_attn(dtype == DOSA_F32 ? A_F32 : A_BF16, a, batch, q_lens, kv_lens, d, workspace, workspace_bytes,
                    static_cast<hipStream_t>(stream));
  });
}

int dsa_cache_append(const dsa_cache* cache, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                     int32_t dtype, const int32_t* q_lens, const int32_t* kv_lens, int32_t batch, int32_t* pos,
                     const int32_t* seen_lens, void* stream) {
  return guarded([&]() -> int {
    return cache_io(true, cache, const_cast<void*>(k), k_stride, const_cast<void*>(v), v_stride, dtype, q_lens,
                    kv_lens, batch, pos, seen_lens, static_cast<hipStream_t>(stream));
  });
}

int dsa_cache_read(const dsa_cache* cache, void* k, int64_t k_stride, void* v, int64_t v_stride, int32_t dtype,
                   const int32_t* q_lens, const int32_t* kv_lens, int32_t batch, void* stream) {
  return guarded([&]() -> int {
    return cache_io(false, cache, k, k_stride, v, v_stride, dtype, q_lens, kv_lens, batch, nullptr, nullptr,
                    static_cast<hipStream_t>(stream));
  });
}

size_t dsa_cache_workspace_size(int32_t batch, const int32_t* q_lens, const int32_t* kv_lens, int32_t Hq, int32_t Hkv,
                                int32_t d, int32_t topk) {
  return guarded_size([&]() -> size_t {
    int64_t tq, tk;
    if (check_lens(batch, q_lens, kv_lens, "q_len", "kv_len", &tq, &tk) != DOSA_OK ||
        check_heads(Hq, Hkv, d) != DOSA_OK || check_row_count(batch, q_lens, Hq, Hkv) != DOSA_OK)
      return 0;
    if (topk < 0 || topk > (1 << 20)) return 0;
    // fp32 queries take more row tiles than bf16 ones: either may be too many
    const size_t a = attn_workspace(A_MX, batch, q_lens, kv_lens, Hq, Hkv, d, topk);
    const size_t b = attn_workspace(A_MX32, batch, q_lens, kv_lens, Hq, Hkv, d, topk);
    return a == 0 || b == 0 ? 0 : std::max(a, b);
  });
}

int dsa_cache_attention(const dsa_cache* cache, const void* q, int64_t q_stride, int32_t q_dtype,
                        const int32_t* q_lens, const int32_t* kv_lens, int32_t batch, int32_t Hq, const int32_t* idx,
                        int32_t topk, float scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                        void* stream) {
  return guarded([&]() -> int {
    int64_t tq, tk;
    int st = check_lens(batch, q_lens, kv_lens, "q_len", "kv_len", &tq, &tk);
    if (st == DOSA_OK) st = check_cache(cache, batch, kv_lens);
    if (st == DOSA_OK) st = check_heads(Hq, cache->Hkv, cache->d);
    if (st == DOSA_OK) st = check_row_count(batch, q_lens, Hq, cache->Hkv);
    if (st == DOSA_OK) st = check_float(q_dtype);
    if (st == DOSA_OK) st = check_scale(scale);
    if (st == DOSA_OK) st = check_rows("q", q, q_stride, Hq, cache->d, q_dtype, tq);
    if (st == DOSA_OK) st = check_rows("out", out, (int64_t)Hq * cache->d, Hq, cache->d, q_dtype, tq);
    if (st != DOSA_OK) return st;
    if (idx == nullptr ? topk != 0 : topk <= 0)
      return fail(DOSA_ERR_INVALID_ARG, "topk must be positive with idx, 0 without");
    if (topk > (1 << 20)) return fail(DOSA_ERR_UNSUPPORTED, "topk above 2^20");
    AttnArgs a{};
    a.q = q;
    a.q_stride = q_stride;
    a.cache = view(cache);
    a.idx = idx;
    a.topk = topk;
    a.out = out;
    a.lse = lse;
    a.Hq = Hq;
    a.Hkv = cache->Hkv;
    a.scale = scale;
    return run_attn(q_dtype == DOSA_F32 ? A_MX32 : A_MX, a, batch, q_lens, kv_lens, cache->d, workspace,
                    workspace_bytes, static_cast<hipStream_t>(stream));
  });
}

size_t dsa_weights_workspace_size(int32_t batch, const int32_t* q_lens, const int32_t* kv_lens, int32_t Hq,
                                  int32_t Hkv, int32_t d) {
  return guarded_size([&]() -> size_t {
    int64_t tq, tk;
    if (check_lens(batch, q_lens, kv_lens, "q_len", "kv_len", &tq, &tk) != DOSA_OK ||
        check_heads(Hq, Hkv, d) != DOSA_OK || check_row_count(batch, q_lens, Hq, Hkv) != DOSA_OK)
      return 0;
    const size_t a = weights_workspace(false, batch, q_lens, kv_lens, Hq, Hkv);
    const size_t b = weights_workspace(true, batch, q_lens, kv_lens, Hq, Hkv);
    return a == 0 || b == 0 ? 0 : std::max(a, b);
  });
}

int dsa_cache_weights(const dsa_cache* cache, const void* q, int64_t q_stride, int32_t q_dtype, const float* lse,
                      const int32_t* q_lens, const int32_t* kv_lens, int32_t batch, int32_t Hq, float scale,
                      const float* acc, float* acc_out, void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    int64_t tq, tk;
    int st = check_lens(batch, q_lens, kv_lens, "q_len", "kv_len", &tq, &tk);
    if (st == DOSA_OK) st = check_cache(cache, batch, kv_lens);
    if (st == DOSA_OK) st = check_heads(Hq, cache->Hkv, cache->d);
    if (st == DOSA_OK) st = check_row_count(batch, q_lens, Hq, cache->Hkv);
    if (st == DOSA_OK) st = check_float(q_dtype);
    if (st == DOSA_OK) st = check_scale(scale);
    if (st == DOSA_OK) st = check_rows("q", q, q_stride, Hq, cache->d, q_dtype, tq);
    if (st != DOSA_OK) return st;
    if (tq > 0 && (lse == nullptr || acc_out == nullptr)) return fail(DOSA_ERR_INVALID_ARG, "lse or acc_out is NULL");
    const bool f32 = q_dtype == DOSA_F32;
    int64_t threads = 0;
    const size_t need = weights_workspace(f32, batch, q_lens, kv_lens, Hq, cache->Hkv, &threads);
    if (need == 0) return fail(DOSA_ERR_UNSUPPORTED, "too many key tiles for one launch");
    st = check_launch("weights", threads);
    if (st != DOSA_OK) return st;
    if (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 16))
      return fail(DOSA_ERR_WORKSPACE, "workspace needs " + std::to_string(need) + " bytes, 16-byte aligned");
    WeightArgs a{};
    a.cache = view(cache);
    a.q = q;
    a.q_stride = q_stride;
    a.lse = lse;
    a.acc = acc;
    a.acc_out = acc_out;
    a.part = static_cast<float*>(workspace);
    a.scale = scale;
    hipStream_t s = static_cast<hipStream_t>(stream);
    for (int k = 0; k < WK_KINDS; ++k) {
      const WeightKind kind = (WeightKind)k;
      int64_t qr = 0;
      for (int b = 0; b < batch;) {
        int64_t floats;
        b = plan_weights(a, kind, f32, &floats, b, batch, q_lens, kv_lens, Hq, cache->Hkv, &qr);
        if (a.n_units == 0) continue;
        hipError_t e;
        {
          PassScope ps(P_WEIGHTS, s);
          e = kind == WK_ROWS ? launch_weights_rows(f32, cache->d, a, s)
                              : (kind == WK_TILES ? launch_weights_tiles(cache->d, a, s) : launch_weights(cache->d, a, s));
        }
        if (e != hipSuccess) return fail_hip(e, "weights kernel launch");
        if (a.n_tiles == 0) continue;
        {
          PassScope ps(P_WEIGHTS_JOIN, s);
          e = kind == WK_TILES ? launch_weights_tiles_join(a, s) : launch_weights_join(a, s);
        }
        if (e != hipSuccess) return fail_hip(e, "weights join launch");
      }
    }
    return DOSA_OK;
  });
}

size_t dsa_evict_workspace_size(int32_t batch, const int32_t* kv_lens, const int32_t* new_lens) {
  return guarded_size([&]() -> size_t {
    int64_t tn, tk;
    if (check_lens(batch, new_lens, kv_lens, "new_len", "kv_len", &tn, &tk) != DOSA_OK) return 0;
    return evict_workspace(batch, kv_lens, new_lens);
  });
}

int dsa_cache_evict(const float* acc, const int32_t* pos, const int32_t* page_table, int32_t page_size,
                    int32_t max_pages, int32_t num_pages, const int32_t* kv_lens, const int32_t* new_lens,
                    const int32_t* seen_lens, int32_t batch, int32_t prefix, int32_t window,
                    const dsa_evict_array* arrays, int32_t n_arrays, int32_t* out_src, int32_t out_stride,
                    void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    int64_t tn, tk;
    int st = check_lens(batch, new_lens, kv_lens, "new_len", "kv_len", &tn, &tk);
    if (st == DOSA_OK) st = check_pages(page_table, num_pages, page_size, max_pages, batch, kv_lens);
    if (st != DOSA_OK) return st;
    if (prefix < 0 || window < 0) return fail(DOSA_ERR_INVALID_ARG, "prefix and window must not be negative");
    if (pos == nullptr && seen_lens != nullptr)
      return fail(DOSA_ERR_INVALID_ARG, "seen_lens without pos: without positions the keys are the whole text");
    for (int b = 0; b < batch; ++b) {
      if (std::min<int64_t>((int64_t)prefix + window, kv_lens[b]) > new_lens[b])
        return fail(DOSA_ERR_INVALID_ARG, "sequence " + std::to_string(b) + ": prefix + window protect more keys than new_len");
      if (new_lens[b] > out_stride) return fail(DOSA_ERR_INVALID_ARG, "out_stride is shorter than a new_len");
      if (seen_lens != nullptr && seen_lens[b] < kv_lens[b])
        return fail(DOSA_ERR_INVALID_ARG, "sequence " + std::to_string(b) + ": need seen_len >= kv_len");
    }
    if (n_arrays < 0 || n_arrays > kEvictArrays || (n_arrays > 0 && arrays == nullptr))
      return fail(DOSA_ERR_INVALID_ARG, "n_arrays must be in 0.." + std::to_string(kEvictArrays) + ", with arrays");
    int64_t cap = 0, kept = 0;
    for (int b = 0; b < batch; ++b) {
      cap = std::max<int64_t>(cap, std::min(new_lens[b], kv_lens[b] - new_lens[b]));
      kept = std::max<int64_t>(kept, new_lens[b]);
    }
    st = check_launch("eviction", evict_move_threads(cap, kept));
    if (st != DOSA_OK) return st;
    if (batch == 0 || out_stride == 0) return DOSA_OK;
    if (acc == nullptr || out_src == nullptr) return fail(DOSA_ERR_INVALID_ARG, "acc or out_src is NULL");
    EvictMoveArgs mv{};
    for (int i = 0; i < n_arrays; ++i) {
      const dsa_evict_array& x = arrays[i];
      if (x.src == nullptr || x.dst == nullptr || x.row_bytes <= 0)
        return fail(DOSA_ERR_INVALID_ARG, "array " + std::to_string(i) + ": NULL pointer or no row bytes");
      if (x.row_bytes > (1 << 20)) return fail(DOSA_ERR_UNSUPPORTED, "array " + std::to_string(i) + ": rows above 2^20 bytes");
      for (int j = 0; j < n_arrays; ++j)
        if (j != i && (arrays[j].dst == x.dst || arrays[j].src == static_cast<const void*>(x.dst)))
          return fail(DOSA_ERR_INVALID_ARG, "array " + std::to_string(i) + " writes where another one reads or writes");
      if (x.dst == static_cast<const void*>(acc) || (pos != nullptr && x.dst == static_cast<const void*>(pos))) {
        // in place only from itself: the choice has read it by then
        if (x.dst != x.src) return fail(DOSA_ERR_INVALID_ARG, "array " + std::to_string(i) + " would overwrite acc or pos");
      }
      int gran = 1;
      for (int g : {16, 4})
        if (gran == 1 && x.row_bytes % g == 0 && aligned(x.src, g) && aligned(x.dst, g)) gran = g;
      mv.a[i] = EvictArray{static_cast<const uint8_t*>(x.src), static_cast<uint8_t*>(x.dst), (int32_t)x.row_bytes, gran};
    }
    EvictArgs a{};
    const size_t need = evict_workspace(batch, kv_lens, new_lens);
    if (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 16))
      return fail(DOSA_ERR_WORKSPACE, "workspace needs " + std::to_string(need) + " bytes, 16-byte aligned");
    hipStream_t s = static_cast<hipStream_t>(stream);
    a.acc = acc;
    a.pos = pos;
    a.table = page_table;
    a.page_size = page_size;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    a.prefix = prefix;
    a.window = window;
    a.out_src = out_src;
    a.out_stride = out_stride;
    a.ws = static_cast<int32_t*>(workspace);
    mv.ws = a.ws;
    mv.out_src = out_src;
    mv.table = page_table;
    mv.out_stride = out_stride;
    mv.page_size = page_size;
    mv.max_pages = max_pages;
    mv.num_pages = num_pages;
    mv.n_arr = n_arrays;
    int64_t off = 0;
    for (int b0 = 0; b0 < batch; b0 += kEvictSeqs) {
      a.n_seq = mv.n_seq = std::min(kEvictSeqs, batch - b0);
      for (int i = 0; i < a.n_seq; ++i) {
        const int b = b0 + i;
        a.s[i] = EvictSeq{off, kv_lens[b], new_lens[b], seen_lens != nullptr ? seen_lens[b] : kv_lens[b], b,
                          std::min(new_lens[b], kv_lens[b] - new_lens[b]), 0};
        mv.s[i] = a.s[i];
        off += evict_ints(kv_lens[b], new_lens[b]);
      }
      hipError_t e;
      {
        PassScope ps(P_EVICT_SELECT, s);
        e = launch_evict_select(a, s);
      }
      if (e != hipSuccess) return fail_hip(e, "eviction select launch");
      {
        PassScope ps(P_EVICT_MOVE, s);
        e = launch_evict_move(mv, s);
      }
      if (e != hipSuccess) return fail_hip(e, "eviction move launch");
    }
    return DOSA_OK;
  });
}

}  // extern "C"
