// Argument checks and small host helpers that the attention and page entry
// points share, and the planned attention run.
#pragma once
#include <algorithm>
#include <cmath>
#include <string>

#include "attn_internal.h"
#include "host_common.h"

namespace dosa {

constexpr int64_t kMaxInt = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxTokens = (int64_t(1) << 31) - (1 << 16);   // positions a tile or two ahead stay int32

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Lengths, with a <= b for every sequence; total of each.
inline int check_lens(int32_t batch, const int32_t* a, const int32_t* b, const char* an, const char* bn, int64_t* ta,
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

inline int check_heads(int32_t Hq, int32_t Hkv, int32_t d) {
  if (Hq <= 0 || Hkv <= 0 || d <= 0 || Hq % Hkv != 0)
    return fail(DOSA_ERR_INVALID_ARG, "Hq must be a positive multiple of Hkv, d positive");
  if ((d != 64 && d != 128) || Hkv > 128 || Hq > 1024)
    return fail(DOSA_ERR_UNSUPPORTED, "d must be 64 or 128, Hkv at most 128, Hq at most 1024");
  return DOSA_OK;
}

// Rows of a sequence (queries times group heads) are int32 in the kernels.
inline int check_row_count(int32_t batch, const int32_t* q_lens, int32_t Hq, int32_t Hkv) {
  for (int b = 0; b < batch; ++b)
    if ((int64_t)q_lens[b] * (Hq / Hkv) > (int64_t(1) << 30))
      return fail(DOSA_ERR_UNSUPPORTED, "sequence " + std::to_string(b) + ": more than 2^30 query rows per kv head");
  return DOSA_OK;
}

// The GPU counts a launch's threads in 32 bits.
constexpr int64_t kLaunchThreads = int64_t(1) << 32;

inline int check_launch(const char* what, int64_t threads) {
  if (threads >= kLaunchThreads)
    return fail(DOSA_ERR_UNSUPPORTED, std::string(what) + ": a launch of 2^32 threads or more, split the call");
  return DOSA_OK;
}

inline int check_scale(float scale) {
  // a subnormal scale would be flushed, and 0 times a masked score's -inf is not
  // 0; the kernels multiply by scale * log2(e), and infinity times an equal
  // maximum's difference of 0 is not 0 either
  if (!(scale > 0.f) || !std::isnormal(scale) || !std::isfinite(scale * 1.44269504f))
    return fail(DOSA_ERR_INVALID_ARG, "scale must be positive, not subnormal, and scale * log2(e) finite in fp32");
  return DOSA_OK;
}

inline int check_float(int32_t dtype) {
  if (dtype != DOSA_F32 && dtype != DOSA_BF16) return fail(DOSA_ERR_UNSUPPORTED, "dtype must be fp32 or bf16");
  return DOSA_OK;
}

// A packed operand [tokens, H, d] with a stride between tokens: 16-byte rows,
// offsets within 64 tokens in 31 bits.
inline int check_rows(const char* name, const void* p, int64_t stride, int32_t H, int32_t d, int32_t dtype, int64_t tokens) {
  if (tokens == 0) return DOSA_OK;
  const int64_t size = dtype == DOSA_F32 ? 4 : 2;
  if (p == nullptr) return fail(DOSA_ERR_INVALID_ARG, std::string(name) + " is NULL");
  if (stride < (int64_t)H * d || (stride * size) % 16 != 0 || !aligned(p, 16))
    return fail(DOSA_ERR_INVALID_ARG, std::string(name) + ": token rows must not overlap and must be 16-byte aligned");
  if (stride > (int64_t(1) << 23)) return fail(DOSA_ERR_UNSUPPORTED, std::string(name) + ": token stride above 2^23");
  return DOSA_OK;
}

inline int check_pages(const int32_t* table, int32_t num_pages, int32_t page_size, int32_t max_pages, int32_t batch,
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

// Bytes of partial results the call's launches need (each launch reuses them);
// 0 if a launch would be too large.  topk: selected keys of a row, or 0; block:
// keys of a selected block, 0 where keys are selected one by one.
// threads: those of the largest launch.
size_t attn_workspace(int src, int32_t batch, const int32_t* q_lens, const int32_t* kv_lens, int32_t Hq, int32_t Hkv,
                      int32_t d, int32_t topk, int32_t block = 0, int64_t* threads = nullptr);
// The attention of base (operands, heads, scale) planned, checked against the
// workspace and enqueued.
int run_attn(int src, const AttnArgs& base, int32_t batch, const int32_t* q_lens, const int32_t* kv_lens, int32_t d,
             void* workspace, size_t workspace_bytes, hipStream_t stream);

inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }

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

}  // namespace dosa
