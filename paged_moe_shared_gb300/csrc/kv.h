// Internals shared by the rotary, KV-cache and attention code.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <string>

#include "internal.h"

namespace rimuru {

struct KvState {
  int device = -1;
  int sms = 0;
  int* d_err = nullptr;  // device error word
  // the pool as bytes [pages][page_bytes / head_dim][head_dim]
  CUtensorMap tm_codes{};   // swizzled boxes of a page's tokens (MMA operands)
  CUtensorMap tm_values{};  // plain boxes, at most a stage of the tile kernel's V
};

// Checks that the current device holds the view's pool, and creates the view's
// device number and error word on first use (*made is then set).
int paged_state_ready(View* v, bool* made);
// Checks that the view has a KV shape and the current device holds its pool,
// and creates the view's device state on first use.
int kv_ready(View* v);
// Checks one activation descriptor; `what` names it in the message.
int check_heads(const rimuru_heads* h, const char* what);
std::string kv_cuda_msg(const char* what, cudaError_t e);

// Tokens of a box of tm_values.
int kv_value_box(int head_dim, int page_tokens);

inline int64_t element_bytes(int dtype) { return dtype == RIMURU_F32 ? 4 : 2; }

// Geometry of a KV view as the kernels see it.
struct KvGeom {
  uint8_t* pool;
  float* scales;  // [num_pages][2][kv_heads]
  uint64_t page_bytes;
  int num_pages;
  int kv_heads, head_dim, page_tokens;
  int* err;
};
inline KvGeom kv_geom(const View& v) {
  return {static_cast<uint8_t*>(v.pool->base), v.scales,   v.page_bytes,    static_cast<int>(v.n_pages),
          v.kv_heads,                          v.head_dim, v.page_tokens, v.kv->d_err};
}

// Where the sequences lie (see the header: page_table, kv_lens).
struct KvSeqs {
  const int32_t* cu;  // row offsets [num_seqs + 1], or null: one row per sequence
  const int32_t* lens;
  const int32_t* table;
  int64_t table_stride;
  int num_seqs;
  int rows;     // rows of all sequences
  int max_len;  // longest sequence that the table and kMostTokens admit
};

// Tokens of the longest sequence: positions, windows and their sums then stay inside an int.
constexpr int64_t kMostTokens = 1 << 30;
inline int max_len(const View& v, int64_t table_stride) {
  return table_stride >= kMostTokens / v.page_tokens ? static_cast<int>(kMostTokens)
                                                    : static_cast<int>(table_stride * v.page_tokens);
}

}  // namespace rimuru
