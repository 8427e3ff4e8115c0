// C-ABI entry points of paged keys and values in 16 or 32 bits: page tables,
// writes, attention, and the choice of blocks with its attention.  Lengths
// travel as kernel arguments: no call copies to the device, allocates or waits.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>

#include "attn_host.h"
#include "pages_internal.h"

using namespace dosa;

namespace {

int check_block(int32_t page_size, int32_t block) {
  if (block != 16 && block != 32 && block != 64 && block != 128)
    return fail(DOSA_ERR_UNSUPPORTED, "block must be 16, 32, 64 or 128");
  if (page_size <= 0 || page_size % block != 0)
    return fail(DOSA_ERR_INVALID_ARG, "page_size must be a multiple of the block");
  return DOSA_OK;
}

int check_paged(const dsa_pages* c, int32_t batch, const int32_t* kv_lens) {
  if (c == nullptr || c->k == nullptr || c->v == nullptr) return fail(DOSA_ERR_INVALID_ARG, "pages or one of their buffers is NULL");
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return fail(DOSA_ERR_INVALID_ARG, "pages must be 16-byte aligned");
  const int st = check_float(c->dtype);
  if (st != DOSA_OK) return st;
  return check_pages(c->page_table, c->num_pages, c->page_size, c->max_pages, batch, kv_lens);
}

int check_blocks(const dsa_blocks* c) {
  if (c == nullptr || c->codes == nullptr || c->scales == nullptr)
    return fail(DOSA_ERR_INVALID_ARG, "blocks or one of their buffers is NULL");
  if (!aligned(c->codes, 16)) return fail(DOSA_ERR_INVALID_ARG, "codes must be 16-byte aligned");
  if (c->reserved != 0) return fail(DOSA_ERR_INVALID_ARG, "dsa_blocks.reserved must be 0");
  return check_block(c->page_size, c->block);
}

CacheView view(const dsa_pages* c) {
  CacheView v{};
  v.table = c->page_table;
  v.page_size = c->page_size;
  v.max_pages = c->max_pages;
  v.num_pages = c->num_pages;
  v.Hkv = c->Hkv;
  return v;
}

int source(int32_t dtype) { return dtype == DOSA_F32 ? A_P32 : A_P16; }

int64_t pages_of(int64_t len, int32_t page_size) { return (len + page_size - 1) / page_size; }

// Table entries from[b] .. to[b] - 1 of each sequence taken from the free list
// or given back to it; assign: tokens of the launch in place of pages.
int move_pages(bool assign, int32_t* table, int32_t max_pages, int32_t page_size, int32_t num_pages, int32_t* free_pages,
               int32_t* free_count, const int32_t* less, const int32_t* kv_lens, int32_t batch, int32_t* slots,
               int32_t* positions, hipStream_t stream) {
  int64_t tl, tk;
  int st = check_lens(batch, less, kv_lens, assign ? "q_len" : "new_len", "kv_len", &tl, &tk);
  if (st == DOSA_OK) st = check_pages(table, num_pages, page_size, max_pages, batch, kv_lens);
  if (st != DOSA_OK) return st;
  if (free_count == nullptr || *free_count < 0 || *free_count > num_pages)
    return fail(DOSA_ERR_INVALID_ARG, "free_count must be in 0..num_pages");
  auto from = [&](int b) { return pages_of(assign ? (int64_t)kv_lens[b] - less[b] : less[b], page_size); };
  int64_t n = 0;
  for (int b = 0; b < batch; ++b) n += pages_of(kv_lens[b], page_size) - from(b);
  if (n > 0 && free_pages == nullptr) return fail(DOSA_ERR_INVALID_ARG, "free_pages is NULL");
  if (assign && n > *free_count)
    return fail(DOSA_ERR_INVALID_ARG, std::to_string(n) + " pages needed, " + std::to_string(*free_count) + " free");
  if (!assign && n > num_pages - *free_count)
    return fail(DOSA_ERR_INVALID_ARG, "more pages given back than are in use");
  const int32_t count = *free_count;
  AssignArgs a{};
  a.table = table;
  a.free_pages = free_pages;
  a.page_div = Div((uint32_t)page_size);
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  int64_t row = 0, moved = 0;
  for (int b = 0; b < batch; b += kAssignSeqs) {
    a.b0 = b;
    a.n_seq = std::min(kAssignSeqs, batch - b);
    a.n_tok = 0;
    a.top = (int32_t)(assign ? count - moved : count + n - moved);
    a.slots = slots == nullptr ? nullptr : slots + row;
    a.positions = positions == nullptr ? nullptr : positions + row;
    int64_t pages = 0;
    for (int i = 0; i < a.n_seq; ++i) {
      const int32_t kv = kv_lens[b + i];
      const int64_t f = from(b + i), l = pages_of(kv, page_size);
      a.s[i] = AssignSeq{a.n_tok, assign ? kv - less[b + i] : (int32_t)f, (int32_t)pages};
      a.n_tok += assign ? less[b + i] : (int32_t)(l - f);
      pages += l - f;
    }
    PassScope ps(assign ? P_PAGES_ASSIGN : P_PAGES_RELEASE, stream);
    const hipError_t e = assign ? launch_assign(a, stream) : launch_release(a, stream);
    if (e != hipSuccess) return fail_hip(e, assign ? "page assignment launch" : "page release launch");
    row += assign ? a.n_tok : 0;
    moved += pages;
  }
  *free_count = (int32_t)(assign ? count - n : count + n);
  return DOSA_OK;
}

// ---------------------------------------------------------------------------
// Work split of the choice of blocks.  LDS holds the scores of a workgroup's
// tokens: up to kSelectLds bytes where several tokens share a workgroup, more for one.
// ---------------------------------------------------------------------------
constexpr int64_t kSelectTiles = 2;

int64_t select_stride(const SelectArgs& a, int32_t kv_len) {
  const int64_t own = ((int64_t)kv_len - 1) >> a.lb;
  if (own < a.topn) return 16;
  // an odd number of 16-word groups: the four tokens of a store lie on different banks
  return (own - a.local + 1 - (a.sinks & ~15) + 63) / 64 * 64 + 16;
}

}  // namespace

extern "C" {

int dsa_pages_assign(int32_t* page_table, int32_t max_pages, int32_t page_size, int32_t num_pages,
                     const int32_t* free_pages, int32_t* free_count, const int32_t* q_lens, const int32_t* kv_lens,
                     int32_t batch, int32_t* slots, int32_t* positions, void* stream) {
  return guarded([&]() -> int {
    return move_pages(true, page_table, max_pages, page_size, num_pages, const_cast<int32_t*>(free_pages), free_count,
                      q_lens, kv_lens, batch, slots, positions, static_cast<hipStream_t>(stream));
  });
}

int dsa_pages_release(int32_t* page_table, int32_t max_pages, int32_t page_size, int32_t num_pages, int32_t* free_pages,
                      int32_t* free_count, const int32_t* new_lens, const int32_t* kv_lens, int32_t batch, void* stream) {
  return guarded([&]() -> int {
    return move_pages(false, page_table, max_pages, page_size, num_pages, free_pages, free_count, new_lens, kv_lens,
                      batch, nullptr, nullptr, static_cast<hipStream_t>(stream));
  });
}

int dsa_pages_append(const dsa_pages* pages, const dsa_blocks* blocks, const void* k, int64_t k_stride, const void* v,
                     int64_t v_stride, const int32_t* q_lens, const int32_t* kv_lens, int32_t batch, void* stream) {
  return guarded([&]() -> int {
    int64_t tq, tk;
    int st = check_lens(batch, q_lens, kv_lens, "q_len", "kv_len", &tq, &tk);
    if (st == DOSA_OK) st = check_paged(pages, batch, kv_lens);
    if (st == DOSA_OK) st = check_heads(pages->Hkv, pages->Hkv, pages->d);
    const bool rows = k != nullptr || v != nullptr || blocks == nullptr;      // else summaries alone
    if (st == DOSA_OK && rows) st = check_rows("k", k, k_stride, pages->Hkv, pages->d, pages->dtype, tq);
    if (st == DOSA_OK && rows) st = check_rows("v", v, v_stride, pages->Hkv, pages->d, pages->dtype, tq);
    if (st == DOSA_OK && blocks != nullptr) st = check_blocks(blocks);
    if (st != DOSA_OK) return st;
    if (blocks != nullptr && (blocks->num_pages != pages->num_pages || blocks->page_size != pages->page_size ||
                              blocks->Hkv != pages->Hkv || blocks->d != pages->d))
      return fail(DOSA_ERR_INVALID_ARG, "blocks are of other pages");
    const int size = pages->dtype == DOSA_F32 ? 4 : 2;
    RowsArgs a{};
    a.pages = view(pages);
    a.k_pages = static_cast<uint8_t*>(pages->k);
    a.v_pages = static_cast<uint8_t*>(pages->v);
    a.k = static_cast<const uint8_t*>(k);
    a.v = static_cast<const uint8_t*>(v);
    a.k_stride = k_stride * size;
    a.v_stride = v_stride * size;
    a.page_div = Div((uint32_t)pages->page_size);
    a.run = kRowRun;
    if (blocks != nullptr) {
      a.codes = blocks->codes;
      a.scales = blocks->scales;
      a.run = blocks->block;
    }
    a.pieces = pages->Hkv * pages->d * size / 16;
    a.slices = (a.pieces + kRowLanes - 1) / kRowLanes;
    auto runs = [&](int b) -> int64_t {
      return q_lens[b] == 0 ? 0 : (kv_lens[b] - 1) / a.run - (kv_lens[b] - q_lens[b]) / a.run + 1;
    };
    for (int b = 0; b < batch; ++b) {
      st = check_launch("append", runs(b) * a.slices * 256);
      if (st != DOSA_OK) return st;
    }
    int64_t row = 0;
    for (int b = 0; b < batch;) {
      a.n_seq = a.n_units = 0;
      for (; b < batch && a.n_seq < kAttnSeqs && (a.n_units + runs(b)) * a.slices * 256 < kLaunchThreads; ++b) {
        if (q_lens[b] > 0) {
          a.s[a.n_seq++] = RowsSeq{a.n_units, (int32_t)row, kv_lens[b] - q_lens[b], kv_lens[b], b};
          a.n_units += (int32_t)runs(b);
        }
        row += q_lens[b];
      }
      if (a.n_seq == 0) continue;
      PassScope ps(P_PAGES_APPEND, static_cast<hipStream_t>(stream));
      const hipError_t e = launch_rows_append(pages->dtype == DOSA_F32, pages->d, a, static_cast<hipStream_t>(stream));
      if (e != hipSuccess) return fail_hip(e, "pages append launch");
    }
    return DOSA_OK;
  });
}

size_t dsa_pages_workspace_size(int32_t batch, const int32_t* q_lens, const int32_t* kv_lens, int32_t Hq, int32_t Hkv,
                                int32_t d, int32_t dtype) {
  return guarded_size([&]() -> size_t {
    int64_t tq, tk;
    if (check_lens(batch, q_lens, kv_lens, "q_len", "kv_len", &tq, &tk) != DOSA_OK ||
        check_heads(Hq, Hkv, d) != DOSA_OK || check_row_count(batch, q_lens, Hq, Hkv) != DOSA_OK ||
        check_float(dtype) != DOSA_OK)
      return 0;
    return attn_workspace(source(dtype), batch, q_lens, kv_lens, Hq, Hkv, d, 0);
  });
}

int dsa_pages_attention(const dsa_pages* pages, const void* q, int64_t q_stride, const int32_t* q_lens,
                        const int32_t* kv_lens, int32_t batch, int32_t Hq, float scale, void* out, float* lse,
                        void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    int64_t tq, tk;
    int st = check_lens(batch, q_lens, kv_lens, "q_len", "kv_len", &tq, &tk);
    if (st == DOSA_OK) st = check_paged(pages, batch, kv_lens);
    if (st == DOSA_OK) st = check_heads(Hq, pages->Hkv, pages->d);
    if (st == DOSA_OK) st = check_row_count(batch, q_lens, Hq, pages->Hkv);
    if (st == DOSA_OK) st = check_scale(scale);
    if (st == DOSA_OK) st = check_rows("q", q, q_stride, Hq, pages->d, pages->dtype, tq);
    if (st == DOSA_OK) st = check_rows("out", out, (int64_t)Hq * pages->d, Hq, pages->d, pages->dtype, tq);
    if (st != DOSA_OK) return st;
    AttnArgs a{};
    a.q = q;
    a.q_stride = q_stride;
    a.k = pages->k;
    a.v = pages->v;
    a.k_stride = a.v_stride = (int64_t)pages->Hkv * pages->d;
    a.cache = view(pages);
    a.page_div = Div((uint32_t)pages->page_size);
    a.out = out;
    a.lse = lse;
    a.Hq = Hq;
    a.Hkv = pages->Hkv;
    a.scale = scale;
    return run_attn(source(pages->dtype), a, batch, q_lens, kv_lens, pages->d, workspace, workspace_bytes,
                    static_cast<hipStream_t>(stream));
  });
}

int dsa_block_select(const dsa_blocks* blocks, const int32_t* page_table, int32_t max_pages, const void* q,
                     int64_t q_stride, int32_t q_dtype, const int32_t* q_lens, const int32_t* kv_lens, int32_t batch,
                     int32_t Hq, int32_t sinks, int32_t local, int32_t* idx, int32_t topn, void* stream) {
  return guarded([&]() -> int {
    int64_t tq, tk;
    int st = check_lens(batch, q_lens, kv_lens, "q_len", "kv_len", &tq, &tk);
    if (st == DOSA_OK) st = check_blocks(blocks);
    if (st == DOSA_OK) st = check_pages(page_table, blocks->num_pages, blocks->page_size, max_pages, batch, kv_lens);
    if (st == DOSA_OK) st = check_heads(Hq, blocks->Hkv, blocks->d);
    if (st == DOSA_OK) st = check_row_count(batch, q_lens, Hq, blocks->Hkv);
    if (st == DOSA_OK) st = check_float(q_dtype);
    if (st == DOSA_OK) st = check_rows("q", q, q_stride, Hq, blocks->d, q_dtype, tq);
    if (st != DOSA_OK) return st;
    if (sinks < 0 || local < 1 || topn < 1 || (int64_t)sinks + local > topn)
      return fail(DOSA_ERR_INVALID_ARG, "need sinks >= 0, local >= 1 and sinks + local <= topn");
    if (topn > 4096) return fail(DOSA_ERR_UNSUPPORTED, "topn above 4096");
    if (tq > 0 && idx == nullptr) return fail(DOSA_ERR_INVALID_ARG, "idx is NULL");
    SelectArgs a{};
    a.q = q;
    a.q_stride = q_stride;
    a.codes = blocks->codes;
    a.scales = blocks->scales;
    a.table = page_table;
    a.idx = idx;
    a.div = Div((uint32_t)(blocks->page_size / blocks->block));
    a.max_pages = max_pages;
    a.num_pages = blocks->num_pages;
    a.Hkv = blocks->Hkv;
    a.group = Hq / blocks->Hkv;
    a.lb = __builtin_ctz((unsigned)blocks->block);
    a.topn = topn;
    a.sinks = sinks;
    a.local = local;
    a.passes = (a.group + 15) / 16;
    a.f32 = q_dtype == DOSA_F32;
    for (int b = 0; b < batch; ++b) {
      if (q_lens[b] == 0) continue;
      if (((int64_t)kv_lens[b] + blocks->block - 1) / blocks->block > kSelectBlocks)
        return fail(DOSA_ERR_UNSUPPORTED, "sequence " + std::to_string(b) + ": more than " + std::to_string(kSelectBlocks) + " blocks");
      st = check_launch("block selection", (int64_t)q_lens[b] * a.Hkv * 1024);
      if (st != DOSA_OK) return st;
    }
    int64_t row = 0;
    for (int b = 0; b < batch;) {
      // the sequences of a launch, then its tokens a workgroup, then its workgroups
      a.n_seq = 0;
      int64_t most_q = 0, stride = 16, most_units = 0;
      for (; b < batch && a.n_seq < kAttnSeqs && (most_units + (int64_t)q_lens[b] * a.Hkv) * 1024 < kLaunchThreads; ++b) {
        if (q_lens[b] > 0) {
          a.s[a.n_seq++] = SelectSeq{0, (int32_t)row, q_lens[b], kv_lens[b], b};
          most_q = std::max<int64_t>(most_q, q_lens[b]);
          stride = std::max(stride, select_stride(a, kv_lens[b]));
          most_units += (int64_t)q_lens[b] * a.Hkv;
        }
        row += q_lens[b];
      }
      if (a.n_seq == 0) continue;
      // most blocks first
      std::stable_sort(a.s, a.s + a.n_seq, [](const SelectSeq& x, const SelectSeq& y) { return x.kv_len > y.kv_len; });
      a.pad = 1;
      while (a.pad < 16 && a.pad < a.group) a.pad *= 2;
      int64_t tiles = a.passes > 1 ? 1 : kSelectTiles;
      auto lds = [&]() { return 16 / a.pad * tiles * stride * 4; };
      while (tiles > 1 && (lds() > kSelectLds || 16 / a.pad * (tiles / 2) >= most_q)) tiles /= 2;
      while (a.pad < 16 && lds() > kSelectLds) a.pad *= 2;
      a.stride = (int32_t)stride;
      const int64_t tw = 16 / a.pad * tiles;
      a.n_units = 0;
      for (int i = 0; i < a.n_seq; ++i) {
        a.s[i].unit0 = a.n_units;
        a.n_units += (int32_t)((a.s[i].q_len + tw - 1) / tw * a.Hkv);
      }
      PassScope ps(P_BLOCK_SELECT, static_cast<hipStream_t>(stream));
      const hipError_t e = launch_block_select(blocks->d, (int)tiles, a, static_cast<hipStream_t>(stream));
      if (e != hipSuccess) return fail_hip(e, "block selection launch");
    }
    return DOSA_OK;
  });
}

size_t dsa_block_workspace_size(int32_t batch, const int32_t* q_lens, const int32_t* kv_lens, int32_t Hq, int32_t Hkv,
                                int32_t d, int32_t dtype, int32_t block, int32_t topn) {
  return guarded_size([&]() -> size_t {
    int64_t tq, tk;
    if (check_lens(batch, q_lens, kv_lens, "q_len", "kv_len", &tq, &tk) != DOSA_OK ||
        check_heads(Hq, Hkv, d) != DOSA_OK || check_row_count(batch, q_lens, Hq, Hkv) != DOSA_OK ||
        check_float(dtype) != DOSA_OK || check_block(block, block) != DOSA_OK)
      return 0;
    if (topn < 1 || (int64_t)topn * block > (1 << 20)) return 0;
    return attn_workspace(source(dtype), batch, q_lens, kv_lens, Hq, Hkv, d, topn * block, block);
  });
}

int dsa_block_attention(const dsa_pages* pages, const void* q, int64_t q_stride, const int32_t* q_lens,
                        const int32_t* kv_lens, int32_t batch, int32_t Hq, const int32_t* idx, int32_t topn,
                        int32_t block, float scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                        void* stream) {
  return guarded([&]() -> int {
    int64_t tq, tk;
    int st = check_lens(batch, q_lens, kv_lens, "q_len", "kv_len", &tq, &tk);
    if (st == DOSA_OK) st = check_paged(pages, batch, kv_lens);
    if (st == DOSA_OK) st = check_heads(Hq, pages->Hkv, pages->d);
    if (st == DOSA_OK) st = check_row_count(batch, q_lens, Hq, pages->Hkv);
    if (st == DOSA_OK) st = check_scale(scale);
    if (st == DOSA_OK) st = check_block(pages->page_size, block);
    if (st == DOSA_OK) st = check_rows("q", q, q_stride, Hq, pages->d, pages->dtype, tq);
    if (st == DOSA_OK) st = check_rows("out", out, (int64_t)Hq * pages->d, Hq, pages->d, pages->dtype, tq);
    if (st != DOSA_OK) return st;
    if (topn < 1) return fail(DOSA_ERR_INVALID_ARG, "topn must be positive");
    if ((int64_t)topn * block > (1 << 20)) return fail(DOSA_ERR_UNSUPPORTED, "topn * block above 2^20");
    if (tq == 0) return DOSA_OK;
    if (idx == nullptr) return fail(DOSA_ERR_INVALID_ARG, "idx is NULL");
    AttnArgs a{};
    a.q = q;
    a.q_stride = q_stride;
    a.k = pages->k;
    a.v = pages->v;
    a.k_stride = a.v_stride = (int64_t)pages->Hkv * pages->d;
    a.cache = view(pages);
    a.page_div = Div((uint32_t)pages->page_size);
    a.idx = idx;
    a.block = block;
    a.topk = topn * block;
    a.out = out;
    a.lse = lse;
    a.Hq = Hq;
    a.Hkv = pages->Hkv;
    a.scale = scale;
    return run_attn(source(pages->dtype), a, batch, q_lens, kv_lens, pages->d, workspace, workspace_bytes,
                    static_cast<hipStream_t>(stream));
  });
}

}  // extern "C"
