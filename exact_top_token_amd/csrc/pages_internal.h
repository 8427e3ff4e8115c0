// Declarations shared by the host code and kernels of the page tables, the
// writes into paged rows and the choice of blocks.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attn_internal.h"

namespace dosa {

// ---- page tables ----
// Sequences of a launch, by the first of their tokens (release: pages) in it.
struct AssignSeq {
  int32_t tok0;       // first token (page) of the sequence, within the launch
  int32_t pos0;       // position of that token (index of that page)
  int32_t new0;       // new pages of the launch's earlier sequences
};
constexpr int kAssignSeqs = 328;        // what 4 KB of kernel arguments hold
struct AssignArgs {
  int32_t* table;
  int32_t* free_pages;
  int32_t* slots;     // of the launch's first token, or NULL
  int32_t* positions;
  Div page_div;
  int32_t max_pages, num_pages;
  int32_t top;        // free pages in front of the launch's (release: held then)
  int32_t b0, n_seq, n_tok;
  AssignSeq s[kAssignSeqs];
};
hipError_t launch_assign(const AssignArgs& p, hipStream_t s);
hipError_t launch_release(const AssignArgs& p, hipStream_t s);

// ---- write ----
// A workgroup takes a run of positions that lies in one page (a block of the
// summaries, or kRowRun positions) and a slice of the row.
constexpr int kRowRun = 16;
constexpr int kRowLanes = 32;          // 16-byte pieces of a slice
struct RowsSeq {
  int32_t unit0;      // first run
  int32_t row0;       // first token row
  int32_t pos0, end;  // positions of the tokens: pos0..end-1
  int32_t b;
};
struct RowsArgs {
  CacheView pages;    // table and geometry
  uint8_t *k_pages, *v_pages;
  const uint8_t *k, *v;
  int64_t k_stride, v_stride;          // bytes
  int8_t* codes;      // [num_pages, page_size / run, Hkv, d] or NULL
  uint8_t* scales;    // [num_pages, page_size / run, Hkv]
  Div page_div;
  int32_t run, pieces, slices, n_units, n_seq;   // pieces: 16-byte pieces of a row
  RowsSeq s[kAttnSeqs];
};
hipError_t launch_rows_append(bool f32, int d, const RowsArgs& p, hipStream_t s);

// ---- choice of blocks ----
constexpr int64_t kSelectLds = 64 << 10;       // bytes of scores where a workgroup takes several tokens
constexpr int64_t kSelectBlocks = 32768;       // of a sequence
struct SelectSeq {
  int32_t unit0;      // first workgroup
  int32_t q_row0, q_len, kv_len, b;
};
struct SelectArgs {
  const void* q;
  const int8_t* codes;
  const uint8_t* scales;
  const int32_t* table;
  int32_t* idx;       // [total_q, Hkv, topn]
  int64_t q_stride;   // elements
  Div div;            // by the blocks of a page
  int32_t max_pages, num_pages, Hkv, group;
  int32_t lb;         // log2 of the block
  int32_t f32;        // queries' type
  int32_t topn, sinks, local;
  int32_t pad;        // rows of the product a token takes: a power of two up to 16
  int32_t passes;     // products of 16 rows a token takes, groups above 16
  int32_t stride;     // scores of a token in LDS
  int32_t n_units, n_seq;
  SelectSeq s[kAttnSeqs];
};
// Tokens of a workgroup: (16 / pad) * tiles.
hipError_t launch_block_select(int d, int tiles, const SelectArgs& p, hipStream_t s);

}  // namespace dosa
