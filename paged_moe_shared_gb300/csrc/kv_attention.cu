// Attention over the 8-bit paged cache.
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>
#include <limits>

#include "kv_attn.h"

namespace rimuru {
namespace {

__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f(float x, __nv_bfloat16* y) { *y = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f(float x, __half* y) { *y = __float2half_rn(x); }

__device__ __forceinline__ float code_to_f(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

// Simple form: one warp per (query row, head) walks the keys one at a time.
template <typename T, int kD>
__global__ void __launch_bounds__(128) kv_attention_rows_kernel(const __grid_constant__ AttnArgs p) {
  constexpr int kPer = kD / 32;
  const int lane = threadIdx.x & 31;
  const int64_t w = blockIdx.x * 4ll + (threadIdx.x >> 5);
  const int row = static_cast<int>(w / p.q_heads), h = static_cast<int>(w % p.q_heads);
  if (row >= p.s.rows) return;
  int b = row, first = row, n = 1;
  if (p.s.cu) {
    int lo = 0, hi = p.s.num_seqs;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (row < p.s.cu[mid + 1]) hi = mid;
      else lo = mid + 1;
    }
    b = lo;
    if (b >= p.s.num_seqs) return;
    first = p.s.cu[b];
    n = p.s.cu[b + 1] - first;
  }
  const int P = p.g.page_tokens;
  int len = p.s.lens[b];
  if (len < 0 || len > p.s.table_stride * P) {
    if (lane == 0) dev::set_error(p.g.err, RIMURU_DEV_BAD_SHAPE);
    len = 0;
  }
  const int pos = len - n + (row - first);
  const int j1 = min(len, pos + 1), j0 = p.window > 0 ? max(0, pos - p.window + 1) : 0;
  const int kvh = h / p.group;
  float q[kPer], o[kPer], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    q[i] = to_f(static_cast<const T*>(p.q)[row * p.q_ts + h * p.q_hs + lane * kPer + i]) * p.scale_log2;
    o[i] = 0.f;
  }
  for (int j = j0; j < j1; ++j) {
    const int page = p.s.table[b * p.s.table_stride + j / P];
    if (page < 0 || page >= p.g.num_pages) {
      if (lane == 0) dev::set_error(p.g.err, RIMURU_DEV_BAD_PAGE);
      continue;
    }
    const uint8_t* kp = p.g.pool + page * p.g.page_bytes + (static_cast<uint64_t>(kvh) * P + j % P) * kD;
    const uint8_t* vp = kp + static_cast<uint64_t>(p.g.kv_heads) * P * kD;
    const float* sc = p.g.scales + static_cast<int64_t>(page) * 2 * p.g.kv_heads + kvh;
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) x += q[i] * code_to_f(kp[lane * kPer + i]);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
    x *= sc[0];
    const float m2 = fmaxf(m, x), a = exp2f(m - m2), e = exp2f(x - m2);
    m = m2;
    l = l * a + e;
    const float ev = e * sc[p.g.kv_heads];
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] = o[i] * a + ev * code_to_f(vp[lane * kPer + i]);
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    from_f(o[i] * inv, static_cast<T*>(p.out) + row * p.o_ts + h * p.o_hs + lane * kPer + i);
  if (p.lse && lane == 0)
    p.lse[static_cast<int64_t>(row) * p.q_heads + h] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

template <typename T>
cudaError_t launch_rows(const AttnArgs& a, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(a.s.rows) * a.q_heads + 3) / 4);
  if (a.g.head_dim == 64) kv_attention_rows_kernel<T, 64><<<grid, 128, 0, s>>>(a);
  else if (a.g.head_dim == 128) kv_attention_rows_kernel<T, 128><<<grid, 128, 0, s>>>(a);
  else kv_attention_rows_kernel<T, 256><<<grid, 128, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

// How a call is cut: rows and number of units, and the workspace's two regions.
struct AttnSplit {
  int unit_rows, units_per_pair;
  uint64_t join_bytes, part_bytes;
};
AttnSplit split_of(const View& v, int q_heads, int num_seqs, int max_q) {
  const int group = q_heads / v.kv_heads;
  AttnSplit w{};
  const int64_t rows = static_cast<int64_t>(max_q) * group;
  w.unit_rows = rows <= 8 ? 8 : kDecodeMaxRows;
  w.units_per_pair = 1;
  const uint64_t units = static_cast<uint64_t>(num_seqs) * v.kv_heads * w.units_per_pair;
  w.join_bytes = (units * sizeof(int2) + 1023) / 1024 * 1024;
  w.part_bytes = 2ull * kMaxRuns * w.unit_rows * (v.head_dim + 1) * sizeof(float);  // and statistics
  return w;
}

}  // namespace rimuru

using rimuru::fail;

extern "C" uint64_t rimuru_kv_attention_workspace_bytes(rimuru_view_t view, int q_heads,
                                                        int num_seqs, int num_q, int max_q) {
  if (!view || !view->v.has_kv || q_heads <= 0 || num_seqs < 0 || num_q < 0 || max_q < 0) return 0;
  if (q_heads % view->v.kv_heads != 0) return 0;
  const rimuru::AttnSplit w = rimuru::split_of(view->v, q_heads, num_seqs, max_q);
  return w.join_bytes + w.part_bytes;
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
  if (!std::isfinite(scale)) return fail(RIMURU_ERR_ARG, "scale must be finite");
  if (num_seqs == 0 || num_q == 0) return RIMURU_OK;
  int st = check_heads(q, "queries");
  if (st == RIMURU_OK) st = check_heads(out, "output");
  if (st != RIMURU_OK) return st;
  if (q->dtype == RIMURU_F32) return fail(RIMURU_ERR_UNSUPPORTED, "queries must be bf16 or f16");
  if (out->dtype != q->dtype || out->heads != q->heads)
    return fail(RIMURU_ERR_ARG, "output and queries must agree in heads and type");
  if (q->heads % v.kv_heads != 0)
    return fail(RIMURU_ERR_UNSUPPORTED, "query heads must be a multiple of kv_heads");
  if (!kv_lens || !page_table || !workspace) return fail(RIMURU_ERR_ARG, "null device pointer");
  if (table_stride <= 0) return fail(RIMURU_ERR_ARG, "table_stride must be positive");
  if (!cu_q && num_q != num_seqs)
    return fail(RIMURU_ERR_ARG, "without row offsets there is one query row per sequence");
  if (reinterpret_cast<uintptr_t>(workspace) % 1024 != 0)
    return fail(RIMURU_ERR_ALIGN, "workspace must be 1024-byte aligned");
  const uint64_t need = rimuru_kv_attention_workspace_bytes(view, q->heads, num_seqs, num_q, max_q);
  if (workspace_bytes < need)
    return fail(RIMURU_ERR_WORKSPACE, "workspace needs " + std::to_string(need) + " bytes");
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
  a.scale_log2 = static_cast<float>(scale * 1.4426950408889634);
  a.window = window;
  a.s = {cu_q, kv_lens, page_table, table_stride, num_seqs, num_q};
  a.g = kv_geom(v);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const AttnSplit w = split_of(v, q->heads, num_seqs, max_q);
  a.max_q = max_q;
  a.unit_rows = w.unit_rows;
  a.units_per_pair = w.units_per_pair;
  a.joins = static_cast<int2*>(workspace);
  a.unit_q = w.unit_rows / a.group;
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + w.join_bytes);
  a.stat = a.part + 2ll * kMaxRuns * w.unit_rows * v.head_dim;
  const double tiles = (static_cast<double>(table_stride) * v.page_tokens / kTileTokens + 1) *
                       num_seqs * v.kv_heads * w.units_per_pair;
  if (tiles > 2e9) return fail(RIMURU_ERR_UNSUPPORTED, "too many keys and queries for one call");
  cudaError_t e;
  if (static_cast<int64_t>(max_q) * a.group <= kDecodeMaxRows) {
    a.runs = std::min(kMaxRuns, kv_decode_runs(v.kv->sms, v.head_dim, w.unit_rows));
    e = launch_kv_decode(a, q->dtype, v.kv->tm_codes, s);
    if (e == cudaSuccess) e = launch_kv_join(a, q->dtype, s);
  } else {
    e = q->dtype == RIMURU_BF16 ? launch_rows<__nv_bfloat16>(a, s) : launch_rows<__half>(a, s);
  }
  if (e != cudaSuccess) return fail(RIMURU_ERR_CUDA, kv_cuda_msg("attention launch", e));
  return RIMURU_OK;
}
