// Linear attention with a decay for each head, on state pages: the view's shape, the
// call, and the kernel that goes token by token.
//
// The recurrent form holds a state, or a slice of its value columns, in the registers of
// one CTA: it is read once, takes all of the sequence's new tokens and is written once.
// A thread holds four neighbouring columns of several key rows; per token it adds k v^T
// and multiplies by q, and the parts of out that the CTA's rows give are added up in
// shared memory.  A decode step moves 8 bytes for each state element and little else: 64
// sequences of 32 heads of 128 x 128 (268 MB) 44.0 us, 0.90 of the copy rate; one sequence 3.2 us;
// 16 sequences of 3 to 5 tokens, 16 heads of 64 x 128, 6.5 us, of which 2.6 are bytes.
#include <algorithm>
#include <cmath>
#include <limits>

#include "device.cuh"
#include "linear.h"

namespace rimuru {
namespace {

using dev::from_f;
using dev::to_f;

constexpr int kStepThreads = 256;
constexpr int kStepTokens = 8;  // tokens between barriers

// kCols value columns of one head's state a CTA.  kStream: states pass through L2 without staying.
template <typename T, int kKey, int kCols, bool kStream>
__global__ void __launch_bounds__(kStepThreads) linear_steps_kernel(const __grid_constant__ LinearArgs a) {
  constexpr int kLanes = kCols / 4;              // threads of a state row
  constexpr int kParts = kStepThreads / kLanes;  // threads that share a column
  constexpr int kRows = kKey / kParts;           // rows of a thread
  constexpr int kSums = kStepThreads / 32;       // partial sums of a column that meet in shared memory: a warp's
  static_assert(kLanes <= 32 && kRows >= 1, "");
  __shared__ alignas(16) float qs[kStepTokens][kKey], ks[kStepTokens][kKey], vs[kStepTokens][kCols];
  __shared__ float decay[kStepTokens];
  __shared__ alignas(16) float sums[kStepTokens][kSums][kCols];
  const int slices = a.value_dim / kCols;
  const int unit = blockIdx.x / slices, col0 = (blockIdx.x - unit * slices) * kCols;
  const int b = unit / a.heads, h = unit - b * a.heads;
  const int tid = threadIdx.x, warp = tid / 32;
  const int part = tid / kLanes, col = 4 * (tid % kLanes);
  const LinearSeq s = linear_seq(a, b, h == 0 && col0 == 0 && tid == 0);
  if (!s.ok) return;
  // row i of this thread: i * kParts + part, so that a warp reads whole rows side by side
  const int64_t at = (static_cast<int64_t>(h) * kKey + part) * a.value_dim + col0 + col;
  const int64_t step = static_cast<int64_t>(kParts) * a.value_dim;
  float4 S[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (s.in) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if constexpr (kStream) S[i] = __ldcs(reinterpret_cast<const float4*>(s.in + at + i * step));
      else S[i] = *reinterpret_cast<const float4*>(s.in + at + i * step);
    }
  }

  const T* q = static_cast<const T*>(a.q) + s.row * a.q_ts + h / a.per_key_head * a.q_hs;
  const T* k = static_cast<const T*>(a.k) + s.row * a.k_ts + h / a.per_key_head * a.k_hs;
  const T* v = static_cast<const T*>(a.v) + s.row * a.v_ts + h * a.v_hs + col0;
  T* o = static_cast<T*>(a.out) + s.row * a.o_ts + h * a.o_hs + col0;
  for (int t0 = 0; t0 < s.n; t0 += kStepTokens) {
    const int n = min(kStepTokens, s.n - t0);
    for (int i = tid; i < n * kKey; i += kStepThreads) {
      const int t = i / kKey, d = i - t * kKey;
      qs[t][d] = to_f(q[(t0 + t) * a.q_ts + d]);
      ks[t][d] = to_f(k[(t0 + t) * a.k_ts + d]);
    }
    for (int i = tid; i < n * kCols; i += kStepThreads) {
      const int t = i / kCols, d = i - t * kCols;
      vs[t][d] = to_f(v[(t0 + t) * a.v_ts + d]);
    }
    if (tid < n) {
      const float g = a.decay[(s.row + t0 + tid) * a.g_ts + h * a.g_hs];
      decay[tid] = expf(g > 0.f ? 0.f : g);  // a NaN stays one
    }
    __syncthreads();
    for (int t = 0; t < n; ++t) {
      const float f = decay[t];
      const float4 x = *reinterpret_cast<const float4*>(&vs[t][col]);
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const float kd = ks[t][i * kParts + part], qd = qs[t][i * kParts + part];
        S[i].x = fmaf(S[i].x, f, kd * x.x);
        S[i].y = fmaf(S[i].y, f, kd * x.y);
        S[i].z = fmaf(S[i].z, f, kd * x.z);
        S[i].w = fmaf(S[i].w, f, kd * x.w);
        y.x = fmaf(S[i].x, qd, y.x);
        y.y = fmaf(S[i].y, qd, y.y);
        y.z = fmaf(S[i].z, qd, y.z);
        y.w = fmaf(S[i].w, qd, y.w);
      }
#pragma unroll
      for (int m = kLanes; m < 32; m <<= 1) {
        y.x += __shfl_xor_sync(~0u, y.x, m);
        y.y += __shfl_xor_sync(~0u, y.y, m);
        y.z += __shfl_xor_sync(~0u, y.z, m);
        y.w += __shfl_xor_sync(~0u, y.w, m);
      }
      if (tid % 32 < kLanes) *reinterpret_cast<float4*>(&sums[t][warp][col]) = y;
    }
    __syncthreads();
    for (int i = tid; i < n * kCols; i += kStepThreads) {
      const int t = i / kCols, d = i - t * kCols;
      float y = 0.f;
#pragma unroll
      for (int w = 0; w < kSums; ++w) y += sums[t][w][d];
      from_f(y * a.scale, &o[(t0 + t) * a.o_ts + d]);
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if constexpr (kStream) __stcs(reinterpret_cast<float4*>(s.out + at + i * step), S[i]);
    else *reinterpret_cast<float4*>(s.out + at + i * step) = S[i];
  }
}

template <typename T, int kKey>
cudaError_t launch_steps(const LinearArgs& a, cudaStream_t s) {
  const int64_t units = static_cast<int64_t>(a.num_seqs) * a.heads;
  // Slices of 64 columns: 64 registers a thread and four CTAs an SM, which take turns loading and
  // storing (64 sequences of 32 heads of 128 x 128: 45.4 us; whole states 50.1, slices of 32 columns
  // 54.8).  Where that leaves SMs without two CTAs, slices of 32.
  const bool wide = units * (a.value_dim / 64) >= 2ll * a.sms;
  const unsigned grid = static_cast<unsigned>(units * (a.value_dim / (wide ? 64 : 32)));
  // States that pass L2 by go faster where there are many (the same 45.4 -> 44.0 us, 16 sequences
  // 15.5 -> 14.5); 17 MB of them, read again soon, slower (6.3 -> 6.8).
  const bool stream = units * kKey * a.value_dim * 8 > 32ll << 20;
  if (!wide) linear_steps_kernel<T, kKey, 32, false><<<grid, kStepThreads, 0, s>>>(a);
  else if (stream) linear_steps_kernel<T, kKey, 64, true><<<grid, kStepThreads, 0, s>>>(a);
  else linear_steps_kernel<T, kKey, 64, false><<<grid, kStepThreads, 0, s>>>(a);
  return cudaGetLastError();
}

// The device's number of SMs, or the usual one without a device.
int sms_here() {
  const int sms = rimuru_device_sm_count();
  return sms > 0 ? sms : 152;
}
bool by_steps(const View& v, int num_seqs, int max_new) {
  return max_new <= steps_most(v.state_heads, v.key_dim, v.value_dim, sms_here(), num_seqs);
}
LinearCut cut_of(const View& v, int num_seqs, int num_tokens, int max_new) {
  if (by_steps(v, num_seqs, max_new)) return {};
  return linear_cut(v.state_heads, v.key_dim, v.value_dim, sms_here(), num_seqs, num_tokens, max_new);
}

int state_ready(View* v) {
  if (!v->has_state) return fail(RIMURU_ERR_STATE, "view has no state shape");
  bool made = false;
  return paged_state_ready(v, &made);
}

}  // namespace

cudaError_t launch_linear_steps(const LinearArgs& a, int dtype, cudaStream_t s) {
  if (dtype == RIMURU_BF16)
    return a.key_dim == 128 ? launch_steps<__nv_bfloat16, 128>(a, s) : launch_steps<__nv_bfloat16, 64>(a, s);
  return a.key_dim == 128 ? launch_steps<__half, 128>(a, s) : launch_steps<__half, 64>(a, s);
}

}  // namespace rimuru

using rimuru::fail;

extern "C" int rimuru_view_set_state_shape(rimuru_view_t view, int heads, int key_dim, int value_dim) {
  rimuru::clear_error();
  if (!view) return fail(RIMURU_ERR_ARG, "null view");
  rimuru::View& v = view->v;
  if (v.has_shape) return fail(RIMURU_ERR_STATE, "view already has an MoE shape");
  if (v.has_kv) return fail(RIMURU_ERR_STATE, "view already has a KV shape");
  if (v.has_state) return fail(RIMURU_ERR_STATE, "view already has a state shape");
  if (heads <= 0 || key_dim <= 0 || value_dim <= 0) return fail(RIMURU_ERR_ARG, "shape values must be positive");
  if ((key_dim != 64 && key_dim != 128) || (value_dim != 64 && value_dim != 128))
    return fail(RIMURU_ERR_UNSUPPORTED, "key_dim and value_dim must be 64 or 128");
  if (heads > 1024 || 4ull * heads * key_dim * value_dim > v.page_bytes)
    return fail(RIMURU_ERR_UNSUPPORTED, "the states of all heads (at most 1024) must fit in one page");
  if (v.n_pages > std::numeric_limits<int32_t>::max())
    return fail(RIMURU_ERR_UNSUPPORTED, "view has too many pages for int32 page ids");
  v.state_heads = heads;
  v.key_dim = key_dim;
  v.value_dim = value_dim;
  v.has_state = true;
  return RIMURU_OK;
}

extern "C" uint64_t rimuru_linear_attention_workspace_bytes(rimuru_view_t view, int num_seqs,
                                                            int num_tokens, int max_new) {
  if (!view || !view->v.has_state || num_seqs < 0 || num_tokens < 0 || max_new < 0) return 0;
  return 1024 + rimuru::cut_of(view->v, num_seqs, num_tokens, std::min(max_new, num_tokens)).state_bytes;
}

extern "C" int rimuru_linear_attention(rimuru_view_t view, const rimuru_heads* q, const rimuru_heads* k,
                                       const rimuru_heads* v_in, const rimuru_heads* out,
                                       const float* log_decay, int64_t decay_token_stride,
                                       int64_t decay_head_stride, const int32_t* cu_new, int num_seqs,
                                       int num_tokens, int max_new, const int32_t* state_in,
                                       const int32_t* state_out, double scale, void* workspace,
                                       uint64_t workspace_bytes, void* stream) {
  using namespace rimuru;
  clear_error();
  if (!view) return fail(RIMURU_ERR_ARG, "null view");
  View& v = view->v;
  if (!v.has_state) return fail(RIMURU_ERR_STATE, "view has no state shape");
  if (num_seqs < 0 || num_tokens < 0 || max_new < 0) return fail(RIMURU_ERR_ARG, "negative count");
  if (!std::isfinite(static_cast<float>(scale))) return fail(RIMURU_ERR_ARG, "scale must be finite in fp32");
  if (num_seqs == 0) return RIMURU_OK;
  max_new = std::min(max_new, num_tokens);
  if (num_tokens > 0) {  // without tokens the states pass from page to page
    const rimuru_heads* all[4] = {q, k, v_in, out};
    const char* names[4] = {"queries", "keys", "values", "output"};
    for (int i = 0; i < 4; ++i) {
      const int st = check_heads(all[i], names[i]);
      if (st != RIMURU_OK) return st;
      if (all[i]->dtype == RIMURU_F32) return fail(RIMURU_ERR_UNSUPPORTED, "activations must be bf16 or f16");
      if (all[i]->dtype != q->dtype) return fail(RIMURU_ERR_ARG, "activations must have one type");
    }
    for (int i = 0; num_tokens > 1 && i < 4; ++i)
      if (all[i]->token_stride == 0 || (i == 3 && out->heads > 1 && out->head_stride == 0))
        return fail(RIMURU_ERR_UNSUPPORTED, std::string(names[i]) + ": elements may not lie on one another");
    if (v_in->heads != v.state_heads || out->heads != v.state_heads)
      return fail(RIMURU_ERR_ARG, "values and output must have the view's heads");
    if (q->heads != k->heads) return fail(RIMURU_ERR_ARG, "queries and keys must have the same heads");
    if (v.state_heads % q->heads != 0)
      return fail(RIMURU_ERR_UNSUPPORTED, "the view's heads must be a multiple of the query/key heads");
  }
  if ((!log_decay && num_tokens > 0) || !state_in || !state_out || !workspace) return fail(RIMURU_ERR_ARG, "null device pointer");
  if (decay_token_stride < 0 || decay_head_stride < 0) return fail(RIMURU_ERR_ARG, "negative stride");
  if (!cu_new && num_tokens != num_seqs)
    return fail(RIMURU_ERR_ARG, "without row offsets there is one token per sequence");
  if (!cu_new) max_new = 1;
  const uintptr_t ints = reinterpret_cast<uintptr_t>(log_decay) | reinterpret_cast<uintptr_t>(cu_new) |
                         reinterpret_cast<uintptr_t>(state_in) | reinterpret_cast<uintptr_t>(state_out);
  if (ints % 4 != 0) return fail(RIMURU_ERR_ALIGN, "decays, offsets and page ids must be 4-byte aligned");
  if (reinterpret_cast<uintptr_t>(workspace) % 1024 != 0)
    return fail(RIMURU_ERR_ALIGN, "workspace must be 1024-byte aligned");
  const uint64_t need = rimuru_linear_attention_workspace_bytes(view, num_seqs, num_tokens, max_new);
  if (workspace_bytes < need)
    return fail(RIMURU_ERR_WORKSPACE, "workspace needs " + std::to_string(need) + " bytes");
  if (4ll * num_seqs * v.state_heads > std::numeric_limits<int32_t>::max())
    return fail(RIMURU_ERR_UNSUPPORTED, "too many sequences for one call");
  if (num_tokens > 0 && (out->data == q->data || out->data == k->data || out->data == v_in->data))
    return fail(RIMURU_ERR_ARG, "the output may not be an input");
  const int st = state_ready(&v);
  if (st != RIMURU_OK) return st;
  LinearArgs a{};
  a.per_key_head = 1;
  if (num_tokens > 0) {
    a.q = q->data, a.k = k->data, a.v = v_in->data, a.out = out->data;
    a.q_ts = q->token_stride, a.q_hs = q->head_stride;
    a.k_ts = k->token_stride, a.k_hs = k->head_stride;
    a.v_ts = v_in->token_stride, a.v_hs = v_in->head_stride;
    a.o_ts = out->token_stride, a.o_hs = out->head_stride;
    a.per_key_head = v.state_heads / q->heads;
  }
  a.decay = log_decay;
  a.g_ts = decay_token_stride, a.g_hs = decay_head_stride;
  a.scale = static_cast<float>(scale);
  a.heads = v.state_heads;
  a.key_dim = v.key_dim, a.value_dim = v.value_dim;
  a.cu = cu_new;
  a.num_seqs = num_seqs, a.num_tokens = num_tokens, a.max_new = max_new;
  a.state_in = state_in, a.state_out = state_out;
  a.pool = static_cast<uint8_t*>(v.pool->base);
  a.page_bytes = v.page_bytes;
  a.num_pages = static_cast<int>(v.n_pages);
  a.err = v.kv->d_err;
  a.sms = v.kv->sms;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int dtype = num_tokens > 0 ? q->dtype : RIMURU_BF16;
  if (!by_steps(v, num_seqs, max_new))
    return launch_linear_chunks(a, cut_of(v, num_seqs, num_tokens, max_new), workspace, dtype, s);
  const cudaError_t e = launch_linear_steps(a, dtype, s);
  if (e != cudaSuccess) return fail(RIMURU_ERR_CUDA, kv_cuda_msg("linear attention launch", e));
  return RIMURU_OK;
}
