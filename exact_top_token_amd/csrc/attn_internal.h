// Declarations shared by the attention entry points' host code and kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/dosa_indexer.h"

namespace dosa {

// Sequences of one launch.  Their records travel as kernel arguments (which a
// captured graph keeps), so a call copies nothing to the device; a larger
// batch takes several launches.
constexpr int kAttnSeqs = 64;

// The paged 4-bit cache as the kernels see it.
struct CacheView {
  uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  const int32_t* table;    // [batch, max_pages]
  int32_t page_size, max_pages, num_pages, Hkv;
};

// Where an attention kernel finds its keys and values, and its queries' type:
// contiguous fp32 or bf16 rows, the 4-bit cache read for bf16 or for fp32
// queries, or pages of fp32 or bf16 rows.
enum AttnSrc : int { A_F32 = 0, A_BF16 = 1, A_MX = 2, A_MX32 = 3, A_P32 = 4, A_P16 = 5 };
constexpr bool paged_rows(int src) { return src == A_P32 || src == A_P16; }

// Division by a positive 32-bit number: the high half of a product falls short
// of the quotient by at most 1.
struct Div {
  uint32_t by, mul;
  __host__ __device__ Div() : by(1), mul(0xffffffffu) {}
  __host__ explicit Div(uint32_t d) : by(d), mul(d == 1 ? 0xffffffffu : (uint32_t)((uint64_t(1) << 32) / d)) {}
  __device__ __forceinline__ uint32_t quot(uint32_t n) const {
    const uint32_t q = __umulhi(n, mul);
    return n - q * by >= by ? q + 1 : q;
  }
};

struct AttnSeq {
  int32_t unit0;      // first unit (wavefront task) of the sequence in this launch
  int32_t join0;      // first row of the join launch (sequences with n_split > 1)
  int32_t part0;      // first partial result (sequences with n_split > 1)
  int32_t q_row0;     // first query row of the packed queries
  int32_t q_len, kv_len;
  int32_t b;          // row of the page table / of the batch
  int32_t n_split, split_len;   // key ranges, keys of each (a multiple of 64)
  int32_t n_rt;       // row tiles
  int64_t key_base;   // contiguous keys: row of the sequence's key 0
};

struct AttnArgs {
  const void* q;
  const void* k;      // contiguous sources; pools of paged rows
  const void* v;
  CacheView cache;    // cache sources; page table and geometry of paged rows
  const int32_t* idx; // selected keys [total_q, topk], blocks [total_q, Hkv, topk / block], or NULL
  void* out;          // [total_q, Hq, d] of q's type
  float* lse;         // [total_q, Hq] or NULL
  float* part_o;      // partial outputs [parts, 16 * row tiles, d]
  float* part_ml;     // partial maxima and sums [parts, 16 * row tiles, 2]
  int64_t q_stride, k_stride, v_stride;   // elements between token rows
  int32_t topk, Hq, Hkv, group;           // group = Hq / Hkv
  float scale;
  int32_t block;                          // keys of a selected block (a power of two), paged rows only
  int4* merged;                           // merged blocks of the units, merged_stride each
  int32_t merged_stride;
  int32_t tok;                            // queries of a row tile (1 but for merged blocks)
  Div page_div;                           // by page_size, paged rows only
  int32_t n_seq, n_units, n_join, rt, hp; // rt: 16-row tiles per unit and head, hp: heads per unit
  AttnSeq s[kAttnSeqs];
};

// 16-row tiles one wavefront may hold next to the keys in flight (bf16 rows
// beyond 16 go to the tiled kernel).  Two tiles of bf16 rows over the cache take
// all 256 registers at d = 128 and spill 1 of them, 26 to 30 with a page look-up
// per key, and are the faster for it: 32 sequences x 4 queries in groups of 8
// over 871K keys 242 us, 330 us as one tile of a head pair (which does not
// spill).  A launch takes what its largest sequence needs: one such sequence
// among 31 of 2 queries costs 241 instead of 207 us (bf16 pages, whose rounding
// follows the tiles, are launches of one kind of sequence).
constexpr int attn_max_rt(int src, int d) {
  return src == A_MX || src == A_P16 || ((src == A_F32 || src == A_P32) && d == 64) ? 2 : 1;
}

// Bf16 prompts over LDS tiles: units are row tiles of kPromptWaves * 32 rows of
// one kv head, over all their keys.
constexpr int kPromptWaves = 8;
hipError_t launch_prompt(int src, int d, const AttnArgs& p, hipStream_t s);

// Heads one wavefront takes together: pairs where the rows of the call are one
// tile, so that the registers are there.
constexpr int attn_heads(int src, int rt, int Hkv) { return src == A_MX && rt == 1 && Hkv % 2 == 0 ? 2 : 1; }
hipError_t launch_attn(int src, int d, const AttnArgs& p, hipStream_t s);
hipError_t launch_pages(int src, int d, const AttnArgs& p, hipStream_t s);

// Listed blocks of many bf16 queries: units are kBlockTileWaves 16-row tiles of
// one kv head, which share the blocks that they list.
constexpr int kBlockTileWaves = 8;
// Records of a unit's merged blocks: one for every entry of its queries' lists
// and kBlockEnds behind (so many are read ahead).
constexpr int kBlockEnds = 8;
constexpr int kBlockTok = 8;           // queries of a row tile at most: 64 of a unit
hipError_t launch_block_merge(const AttnArgs& p, hipStream_t s);
hipError_t launch_block_tiles(int d, const AttnArgs& p, hipStream_t s);
hipError_t launch_attn_join(int src, int d, const AttnArgs& p, hipStream_t s);

// Cache write and read-back.
struct CacheSeq {
  int32_t unit0;      // first workgroup (kCacheTokens tokens each)
  int32_t row0;       // first token row of the packed tokens
  int32_t n;          // tokens
  int32_t pos0;       // logical position of the first
  int32_t seen0;      // value of pos[] of the first
  int32_t b;
};
constexpr int kCacheTokens = 16;
struct CacheIoArgs {
  CacheView cache;
  void* k;            // [total, Hkv, d]
  void* v;
  int64_t k_stride, v_stride;
  int32_t* pos;       // [num_pages, page_size] or NULL (write only)
  int32_t n_seq;
  CacheSeq s[kAttnSeqs];
};
hipError_t launch_cache_append(bool f32, int d, const CacheIoArgs& p, hipStream_t s);
hipError_t launch_cache_read(bool f32, int d, const CacheIoArgs& p, hipStream_t s);

// Accumulated attention weights.  Three kernels: few rows (queries times group
// heads), many bf16 rows, many fp32 rows.
constexpr int kWeightRows = 32;        // rows of the first
constexpr int kWeightRowKeys = 1024;   // keys of its workgroup at most
constexpr int kWeightChunk = 512;      // keys of a workgroup of the second
enum WeightKind : int { WK_ROWS = 0, WK_TILES = 1, WK_ANY = 2, WK_KINDS = 3 };
struct WeightSeq {
  int32_t unit0;      // first workgroup
  int32_t tile0;      // first workgroup of the join
  int32_t part0;      // first partial (64 floats; kWeightChunk for WK_TILES)
  int32_t q_row0, q_len, kv_len, b;
  int32_t n_part;     // shares of a key tile's work
  int32_t part_rows;  // WK_TILES: rows of a share
};
struct WeightArgs {
  CacheView cache;
  const void* q;
  const float* lse;
  const float* acc;   // or NULL
  float* acc_out;
  float* part;
  int64_t q_stride;
  int32_t Hq, group;
  float scale;
  int32_t n_seq, n_units, n_tiles;
  int32_t range, rt;  // WK_ROWS: keys of a workgroup, 16-row tiles
  WeightSeq s[kAttnSeqs];
};
hipError_t launch_weights(int d, const WeightArgs& p, hipStream_t s);
hipError_t launch_weights_join(const WeightArgs& p, hipStream_t s);
hipError_t launch_weights_rows(bool f32, int d, const WeightArgs& p, hipStream_t s);
hipError_t launch_weights_tiles(int d, const WeightArgs& p, hipStream_t s);
hipError_t launch_weights_tiles_join(const WeightArgs& p, hipStream_t s);

// Eviction.
// A sequence's workspace: the number of moves (in its first kEvictHead ints),
// the indices keys move to and then, directly behind, the keys that move (at
// most cap of each), and the ranks of the keys beyond the kEvictNear * 1024 that its workgroup keeps in registers.
constexpr int kEvictHead = 16;
constexpr int kEvictNear = 16;
struct EvictSeq {
  int64_t ws_off;
  int32_t kv_len, new_len, seen, b;
  int32_t cap;              // moves at most: min(new_len, kv_len - new_len)
  int32_t pad;
};
constexpr int kEvictSeqs = 64;
struct EvictArgs {
  const float* acc;         // [num_pages, page_size]
  const int32_t* pos;       // [num_pages, page_size] or NULL
  const int32_t* table;
  int32_t page_size, max_pages, num_pages;
  int32_t prefix, window;
  int32_t* out_src;         // [batch, out_stride]
  int32_t out_stride;
  int32_t* ws;
  int32_t n_seq;
  EvictSeq s[kEvictSeqs];
};
struct EvictArray {
  const uint8_t* src;
  uint8_t* dst;
  int32_t row_bytes;
  int32_t gran;             // bytes of one access: 16, 4 or 1
};
constexpr int kEvictArrays = 16;
struct EvictMoveArgs {
  const int32_t* out_src;
  const int32_t* table;
  int32_t out_stride, page_size, max_pages, num_pages;
  int32_t n_seq, n_arr;
  int32_t in_blocks;        // set by the launch
  const int32_t* ws;
  EvictSeq s[kEvictSeqs];
  EvictArray a[kEvictArrays];
};
// Rows of a workgroup of the move: entries of the list of moves, rows copied
// elsewhere; and the threads that so many of each take.
constexpr int kMoveRows = 8;
constexpr int kCopyRows = 256;
constexpr int64_t evict_move_threads(int64_t moves, int64_t copies) {
  return ((moves + kMoveRows - 1) / kMoveRows + (copies + kCopyRows - 1) / kCopyRows) * 256;
}
hipError_t launch_evict_select(const EvictArgs& p, hipStream_t s);
hipError_t launch_evict_move(EvictMoveArgs p, hipStream_t s);

}  // namespace dosa
