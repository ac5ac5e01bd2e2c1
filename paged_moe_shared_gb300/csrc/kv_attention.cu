// Attention over the 8-bit paged cache.
#include <algorithm>
#include <cmath>
#include <limits>

#include "kv_attn.h"

namespace rimuru {
// How a call is cut: rows and number of units, and the workspace's two regions.
struct AttnSplit {
  bool decode;
  int unit_rows, units_per_pair;
  uint64_t cut_bytes, part_bytes;
};
AttnSplit split_of(const View& v, int q_heads, int max_q) {
  const int group = q_heads / v.kv_heads;
  AttnSplit w{};
  const int64_t rows = static_cast<int64_t>(max_q) * group;
  // Up to 16 rows take the decode kernel, in units of 8 or 16 rows (32 sequences of 2000 keys,
  // head_dim 128: 8 rows 18.2 us, in units of 16 25.6; 16 rows 26.9 us, with the tile kernel
  // 31.9).  Beyond, a unit is 128 rows, or 256 from 257 rows on where two query tiles fit the
  // tensor memory (eight sequences of 2000 keys: 256 rows 29.0 us in units of 128, 37.9 of 256;
  // 512 rows 38.0 and 38.2; one of 8000 keys: 8192 rows 137 and 121).
  w.decode = rows <= kDecodeMaxRows;
  w.unit_rows = rows <= 8 ? 8 : rows <= kDecodeMaxRows ? 16 : rows <= 256 ? 128 : tile_rows(v.head_dim);
  const int unit_q = std::max(1, w.unit_rows / group);
  w.units_per_pair = std::max(1, max_q / unit_q + (max_q % unit_q != 0));
  w.cut_bytes = (kMaxRuns * sizeof(int4) + 1023) / 1024 * 1024;
  w.part_bytes = 2ull * (w.decode ? kMaxRuns : kMaxTileRuns) * w.unit_rows * (v.head_dim + 1) * sizeof(float);  // and statistics
  return w;
}

}  // namespace rimuru

using rimuru::fail;

extern "C" uint64_t rimuru_kv_attention_workspace_bytes(rimuru_view_t view, int q_heads,
                                                        int num_seqs, int num_q, int max_q) {
  if (!view || !view->v.has_kv || q_heads <= 0 || num_seqs < 0 || num_q < 0 || max_q < 0) return 0;
  if (q_heads % view->v.kv_heads != 0) return 0;
  const rimuru::AttnSplit w = rimuru::split_of(view->v, q_heads, std::min(max_q, num_q));
  return w.cut_bytes + w.part_bytes;
}

extern "C" int rimuru_kv_attention(rimuru_view_t view, const rimuru_heads* q, const rimuru_heads* out,
                                   float* lse, const int32_t* cu_q, const int32_t* kv_lens,
                                   int num_seqs, int num_q, int max_q, const int32_t* page_table,
                                   int64_t table_stride, double scale, int window, void* workspace,
                                   uint64_t workspace_bytes, void* stream) {
  using namespace rimuru;
  clear_error();
  if (!view) return fail(RIMURU_ERR_ARG, "null view");
  View& v = view->v;
  if (!v.has_kv) return fail(RIMURU_ERR_STATE, "view has no KV shape");
  if (num_seqs < 0 || num_q < 0 || max_q < 0 || window < 0)
    return fail(RIMURU_ERR_ARG, "negative count or window");
  const float scale_log2 = static_cast<float>(scale * 1.4426950408889634);
  if (!std::isfinite(scale_log2)) return fail(RIMURU_ERR_ARG, "scale must be finite in fp32");
  if (num_seqs == 0 || num_q == 0) return RIMURU_OK;
  max_q = std::min(max_q, num_q);  // no sequence has more rows than all have together
  int st = check_heads(q, "queries");
  if (st == RIMURU_OK) st = check_heads(out, "output");
  if (st != RIMURU_OK) return st;
  if (q->dtype == RIMURU_F32) return fail(RIMURU_ERR_UNSUPPORTED, "queries must be bf16 or f16");
  if (out->dtype != q->dtype || out->heads != q->heads)
    return fail(RIMURU_ERR_ARG, "output and queries must agree in heads and type");
  if (q->heads % v.kv_heads != 0)
    return fail(RIMURU_ERR_UNSUPPORTED, "query heads must be a multiple of kv_heads");
  if (q->heads / v.kv_heads > 128)
    return fail(RIMURU_ERR_UNSUPPORTED, "at most 128 query heads share a key/value head");
  if (!kv_lens || !page_table || !workspace) return fail(RIMURU_ERR_ARG, "null device pointer");
  if (table_stride <= 0) return fail(RIMURU_ERR_ARG, "table_stride must be positive");
  if (!cu_q && num_q != num_seqs)
    return fail(RIMURU_ERR_ARG, "without row offsets there is one query row per sequence");
  if (reinterpret_cast<uintptr_t>(workspace) % 1024 != 0)
    return fail(RIMURU_ERR_ALIGN, "workspace must be 1024-byte aligned");
  const uint64_t need = rimuru_kv_attention_workspace_bytes(view, q->heads, num_seqs, num_q, max_q);
  if (workspace_bytes < need)
    return fail(RIMURU_ERR_WORKSPACE, "workspace needs " + std::to_string(need) + " bytes");
  const AttnSplit w = split_of(v, q->heads, max_q);
  const int cost = w.decode ? kDecodeUnitCost : kTileUnitCost;
  const double places = (static_cast<double>(table_stride) * v.page_tokens / kTileTokens + 1 + cost) *
                        num_seqs * v.kv_heads * w.units_per_pair;
  if (places > 2e9 || max_q > kMostTokens) return fail(RIMURU_ERR_UNSUPPORTED, "too many keys and queries for one call");
  st = kv_ready(&v);
  if (st != RIMURU_OK) return st;
  AttnArgs a{};
  a.q = q->data;
  a.out = out->data;
  a.lse = lse;
  a.q_ts = q->token_stride;
  a.q_hs = q->head_stride;
  a.o_ts = out->token_stride;
  a.o_hs = out->head_stride;
  a.q_heads = q->heads;
  a.group = q->heads / v.kv_heads;
  a.scale_log2 = scale_log2;
  a.s = {cu_q, kv_lens, page_table, table_stride, num_seqs, num_q, max_len(v, table_stride)};
  a.window = window < a.s.max_len ? window : 0;  // as long as every sequence: none
  a.g = kv_geom(v);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  a.max_q = max_q;
  a.sms = v.kv->sms;
  a.unit_rows = w.unit_rows;
  a.units_per_pair = w.units_per_pair;
  a.unit_cost = cost;
  a.cuts = static_cast<int4*>(workspace);
  a.unit_q = w.unit_rows / a.group;
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + w.cut_bytes);
  a.stat = a.part + 2ll * (w.decode ? kMaxRuns : kMaxTileRuns) * w.unit_rows * v.head_dim;
  const int64_t units = static_cast<int64_t>(num_seqs) * v.kv_heads * w.units_per_pair;
  const int64_t most = (table_stride * v.page_tokens + kTileTokens - 1) / kTileTokens;  // tiles of a unit
  a.runs = w.decode ? std::min(kMaxRuns, kv_decode_runs(v.kv->sms, v.head_dim, w.unit_rows))
                    : std::min(kMaxTileRuns, v.kv->sms);
  a.direct = leave_whole(units, most, a.runs, cost, w.unit_rows, v.head_dim);
  if (a.direct) a.runs = static_cast<int>(units);
  cudaError_t e = w.decode ? launch_kv_decode(a, q->dtype, v.kv->tm_codes, s)
                           : launch_kv_tiles(a, q->dtype, v.kv->tm_codes, v.kv->tm_values, s);
  if (e == cudaSuccess && !a.direct) e = launch_kv_join(a, q->dtype, s);
  if (e != cudaSuccess) return fail(RIMURU_ERR_CUDA, kv_cuda_msg("attention launch", e));
  return RIMURU_OK;
}
