// The 8-bit paged key/value cache: the view's KV shape, the append that
// quantises new tokens, page copies, and the host side of forking and
// compaction.
#include <cuda_fp8.h>

#include <algorithm>
#include <limits>
#include <mutex>
#include <new>
#include <unordered_map>
#include <vector>

#include "device.cuh"
#include "kernels.h"
#include "kv.h"

namespace rimuru {

std::string kv_cuda_msg(const char* what, cudaError_t e) {
  return std::string(what) + ": " + cudaGetErrorName(e) + " (" + cudaGetErrorString(e) + ")";
}

int check_heads(const rimuru_heads* h, const char* what) {
  const std::string w(what);
  if (!h || !h->data) return fail(RIMURU_ERR_ARG, w + ": null descriptor or data");
  if (h->heads <= 0) return fail(RIMURU_ERR_ARG, w + ": heads must be positive");
  if (h->dtype != RIMURU_BF16 && h->dtype != RIMURU_F16 && h->dtype != RIMURU_F32)
    return fail(RIMURU_ERR_ARG, w + ": unknown element type");
  if (h->token_stride < 0 || h->head_stride < 0) return fail(RIMURU_ERR_ARG, w + ": negative stride");
  const int64_t unit = 16 / element_bytes(h->dtype);
  if (reinterpret_cast<uintptr_t>(h->data) % 16 != 0 || h->token_stride % unit != 0 ||
      h->head_stride % unit != 0)
    return fail(RIMURU_ERR_ALIGN, w + ": data and strides must be multiples of 16 bytes");
  return RIMURU_OK;
}

int* kv_error_word(const View* v) { return v->kv ? v->kv->d_err : nullptr; }

void destroy_kv_state(View* v) {
  if (!v->kv) return;
  if (v->kv->d_err) cudaFree(v->kv->d_err);
  delete v->kv;
  v->kv = nullptr;
}

int paged_state_ready(View* v, bool* made) {
  int cur = 0;
  cudaError_t e = cudaGetDevice(&cur);
  if (e != cudaSuccess) return fail(RIMURU_ERR_CUDA, kv_cuda_msg("cudaGetDevice", e));
  int st = check_device(v, cur);
  if (st != RIMURU_OK) return st;
  if (v->kv) {
    if (v->kv->device != cur)
      return fail(RIMURU_ERR_ARG, "the view's device state lives on another device");
    return RIMURU_OK;
  }
  auto* k = new (std::nothrow) KvState;
  if (!k) return fail(RIMURU_ERR_OOM, "host allocation failed");
  v->kv = k;
  k->device = cur;
  e = cudaDeviceGetAttribute(&k->sms, cudaDevAttrMultiProcessorCount, cur);
  if (e == cudaSuccess) e = alloc_words(&k->d_err, 1);
  if (e != cudaSuccess) {
    destroy_kv_state(v);
    return fail(RIMURU_ERR_CUDA, kv_cuda_msg("device state of the view", e));
  }
  *made = true;
  return RIMURU_OK;
}

int kv_ready(View* v) {
  if (!v->has_kv) return fail(RIMURU_ERR_STATE, "view has no KV shape");
  bool made = false;
  int st = paged_state_ready(v, &made);
  if (st != RIMURU_OK || !made) return st;
  KvState* k = v->kv;
  // the pool as pages of rows of head_dim codes; a box is one head's tokens of a
  // page, at most 128 bytes of each
  const uint64_t dim = static_cast<uint64_t>(v->head_dim);
  const cuuint32_t inner = static_cast<cuuint32_t>(std::min<uint64_t>(dim, 128));
  const cuuint64_t dims[3] = {dim, v->page_bytes / dim, static_cast<cuuint64_t>(v->n_pages)};
  const cuuint64_t strides[2] = {dim, v->page_bytes};
  const cuuint32_t box[3] = {inner, static_cast<cuuint32_t>(v->page_tokens), 1};
  st = make_byte_map(&k->tm_codes, v->pool->base, dims, strides, box,
                     inner == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
  const cuuint32_t box_v[3] = {static_cast<cuuint32_t>(dim),
                               static_cast<cuuint32_t>(kv_value_box(v->head_dim, v->page_tokens)), 1};
  if (st == RIMURU_OK)
    st = make_byte_map(&k->tm_values, v->pool->base, dims, strides, box_v, CU_TENSOR_MAP_SWIZZLE_NONE);
  if (st != RIMURU_OK) {
    const std::string msg = rimuru_last_error();
    destroy_kv_state(v);
    return fail(st, msg);
  }
  return RIMURU_OK;
}

namespace {

// ------------------------------------------------------------------ append
struct AppendArgs {
  const void* x[2];  // keys, values
  int64_t ts[2], hs[2];
  int warps_per_slice;
  KvSeqs s;
  KvGeom g;
};

__device__ __forceinline__ void load8f(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(v[i] << 16);
    x[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8f(const __half* p, float (&x)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void load8f(const float* p, float (&x)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// Eight codes of x * inv (a power of two, so the product is exact up to fp32
// range): round to nearest even, saturating; NaN becomes 0.
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    float a = x[i], b = x[i + 1];
    a = a == a ? a * inv : 0.f;
    b = b == b ? b * inv : 0.f;
    const uint32_t c = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    w[i >> 2] |= c << (8 * (i & 2));
  }
  return make_uint2(w[0], w[1]);
}

// Smallest power of two s with amax <= 448 s, within [2^-60, 2^60].  448 is
// 1.75 * 2^8: the exponent of amax less 8, plus one when its mantissa is above 1.75.
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t b = __float_as_uint(amax);
  int k = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u);
  k = max(-60, min(60, k));
  return __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
}

// One CTA per unit, a page that one sequence's new tokens touch.  Sequence b has
// at most n_b / P + 2 units, at unit numbers cu[b] / P + 2 b onwards, so a unit
// finds its sequence by bisection and the grid needs no lengths on the host.  The
// units below cu[0] / P have nothing to do.
//
// Bound: HBM (two bytes read and one written per element).  `wps` warps share a
// (K or V, head) slice of the page, a lane has eight elements of a token at a
// time, and everything a warp has to read is in flight at once: up to kHold
// vectors a lane, which stay in registers between the maximum and the encoding
// (a slice with more per warp is read again).  Ragged prompts of 33 MB: 12.0 us,
// 2.8 TB/s (f16 11.7; f32, 56 MB, 22.6: held as four words a vector they spill 244 bytes a
// thread); 64 sequences of one token: 4.0 us.  What is left is the chain length ->
// page table -> values -> scale -> codes, of which each step waits for the last, and
// that two CTAs of 512 threads fit an SM: of the prompts' 354 pages 304 are written at
// the same time and the others after them.
constexpr int kHold = 8;
constexpr int kAppendWarps = 16;

template <typename T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw8<T> load_raw(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) r.w[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}

template <typename T>
__global__ void __launch_bounds__(32 * kAppendWarps, 2)
    kv_append_kernel(const __grid_constant__ AppendArgs p) {
  __shared__ float tops[kAppendWarps];
  const int P = p.g.page_tokens, D = p.g.head_dim;
  const int u = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // first sequence with u < cu[b + 1] / P + 2 (b + 1): by halves, the last 32 at once
  int lo = 0, hi = p.s.num_seqs;
  while (hi - lo > 32) {
    const int mid = (lo + hi) >> 1;
    if (u < p.s.cu[mid + 1] / P + 2 * (mid + 1)) hi = mid;
    else lo = mid + 1;
  }
  const int probe = lo + lane;
  const bool past = probe >= hi || u < p.s.cu[probe + 1] / P + 2 * (probe + 1);
  const uint32_t hits = __ballot_sync(0xffffffffu, past);
  const int b = hits ? lo + __ffs(hits) - 1 : hi;
  if (b >= p.s.num_seqs) return;
  const int r0 = p.s.cu[b], n = p.s.cu[b + 1] - r0;
  const int len = p.s.lens[b], start = len - n;
  if (n <= 0) return;
  if (r0 < 0 || r0 + n > p.s.rows || start < 0 || len > p.s.max_len) {
    if (threadIdx.x == 0) dev::set_error(p.g.err, RIMURU_DEV_BAD_SHAPE);
    return;
  }
  const int d = u - (r0 / P + 2 * b);  // of the sequence's units; below 0 where its rows are not the array's first
  const int c = start / P + d;         // page index within the sequence
  if (d < 0 || c * P >= len) return;
  const int page = p.s.table[b * p.s.table_stride + c];
  if (page < 0 || page >= p.g.num_pages) {
    if (threadIdx.x == 0) dev::set_error(p.g.err, RIMURU_DEV_BAD_PAGE);
    return;
  }
  const int s0 = max(start - c * P, 0), s1 = min(len - c * P, P);  // slots to write
  const int row0 = r0 + c * P - start;                              // row of slot 0
  const int lanes = D / 8, at = lane % lanes, per = 32 / lanes;
  const int slices = 2 * p.g.kv_heads, wps = p.warps_per_slice;
  const int part = warp % wps, team = warp / wps, teams = (blockDim.x >> 5) / wps;
  const int step = per * wps, first = part * per + lane / lanes;  // this lane's rows: first, + step, ...
  for (int w0 = 0; w0 < slices; w0 += teams) {
    const int w = w0 + team;
    const bool busy = w < slices;
    const int kv = w >= p.g.kv_heads, h = w - kv * p.g.kv_heads;
    const T* x = static_cast<const T*>(p.x[kv]) + h * p.hs[kv] + row0 * p.ts[kv] + 8 * at;
    uint8_t* codes = p.g.pool + page * p.g.page_bytes + static_cast<uint64_t>(w) * P * D + 8 * at;
    float* scale = p.g.scales + (static_cast<int64_t>(page) * slices + w);
    float amax = 0.f, s_old = 0.f;
    bool odd = false;  // a NaN or an infinity among the new elements
    const auto look = [&](const Raw8<T>& raw) {
      float v[8];
      load8f(reinterpret_cast<const T*>(&raw), v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float m = fabsf(v[e]);
        if (m <= 3.4028234664e38f) amax = fmaxf(amax, m);
        else odd = true;
      }
    };
    Raw8<T> held[kHold];
    if (busy) {
      if (s0 > 0) s_old = *scale;
#pragma unroll
      for (int i = 0; i < kHold; ++i)
        if (s0 + first + i * step < s1) held[i] = load_raw(x + (s0 + first + i * step) * p.ts[kv]);
#pragma unroll
      for (int i = 0; i < kHold; ++i)
        if (s0 + first + i * step < s1) look(held[i]);
      for (int t = s0 + first + kHold * step; t < s1; t += step) look(load_raw(x + t * p.ts[kv]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (lane == 0) tops[warp] = amax;
    __syncthreads();  // also: every warp of the slice has read the old scale
    for (int i = 0; i < wps; ++i) amax = fmaxf(amax, tops[warp - part + i]);
    if (busy) {
      const float s_new = fmaxf(scale_for(amax), s_old);
      if (s0 > 0 && s_new > s_old) {  // earlier tokens are rounded again at the larger scale
        const float f = s_old / s_new;
        for (int t = first; t < s0; t += step) {
          uint2 q = *reinterpret_cast<uint2*>(codes + t * D);
          const uint32_t in[2] = {q.x, q.y};
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
                static_cast<__nv_fp8x2_storage_t>(in[i >> 2] >> (8 * (i & 2))), __NV_E4M3);
            const float2 g = __half22float2(__half2(hr));
            v[i] = g.x;
            v[i + 1] = g.y;
          }
          *reinterpret_cast<uint2*>(codes + t * D) = encode8(v, f);
        }
      }
      const float inv = 1.f / s_new;
#pragma unroll
      for (int i = 0; i < kHold; ++i) {
        const int t = s0 + first + i * step;
        if (t >= s1) continue;
        float v[8];
        load8f(reinterpret_cast<const T*>(&held[i]), v);
        *reinterpret_cast<uint2*>(codes + t * D) = encode8(v, inv);
      }
      for (int t = s0 + first + kHold * step; t < s1; t += step) {
        float v[8];
        load8f(x + t * p.ts[kv], v);
        *reinterpret_cast<uint2*>(codes + t * D) = encode8(v, inv);
      }
      if (part == 0 && lane == 0) *scale = s_new;
      if (odd) dev::set_error(p.g.err, RIMURU_DEV_NONFINITE);
    }
    __syncthreads();  // `tops` is free again
  }
}

// -------------------------------------------------------------- page copies
// Bound: HBM.  A CTA copies a chunk of a page, four 16-byte vectors a thread in
// flight.  2048 pages of 32 KiB (134 MB): 21.2 us, 6.3 TB/s, 0.95 of the copy rate.
constexpr int kPairsPerLaunch = 448;
struct PairList {  // pairs passed by value (fork, compaction)
  int32_t src[kPairsPerLaunch], dst[kPairsPerLaunch];
};
struct CopyArgs {
  const int32_t* src;
  const int32_t* dst;
  KvGeom g;
  int chunks;  // CTAs a page
  uint32_t chunk_bytes;
};

constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;

__device__ __forceinline__ void copy_page(const CopyArgs& p, int from, int to, int chunk) {
  if (from < 0 || from >= p.g.num_pages || to < 0 || to >= p.g.num_pages) {
    if (threadIdx.x == 0) dev::set_error(p.g.err, RIMURU_DEV_BAD_PAGE);
    return;
  }
  const uint64_t used = 2ull * p.g.kv_heads * p.g.page_tokens * p.g.head_dim;
  const uint64_t b0 = static_cast<uint64_t>(chunk) * p.chunk_bytes;
  const uint64_t b1 = min(used, b0 + p.chunk_bytes);
  const uint8_t* s = p.g.pool + from * p.g.page_bytes;
  uint8_t* d = p.g.pool + to * p.g.page_bytes;
  for (uint64_t i = b0 + threadIdx.x * 16; i < b1; i += kCopyThreads * 16 * kCopyUnroll) {
    uint4 v[kCopyUnroll];
#pragma unroll
    for (int j = 0; j < kCopyUnroll; ++j)
      if (i + j * kCopyThreads * 16 < b1) v[j] = *reinterpret_cast<const uint4*>(s + i + j * kCopyThreads * 16);
#pragma unroll
    for (int j = 0; j < kCopyUnroll; ++j)
      if (i + j * kCopyThreads * 16 < b1) *reinterpret_cast<uint4*>(d + i + j * kCopyThreads * 16) = v[j];
  }
  if (chunk == 0)
    for (int i = threadIdx.x; i < 2 * p.g.kv_heads; i += kCopyThreads)
      p.g.scales[static_cast<int64_t>(to) * 2 * p.g.kv_heads + i] =
          p.g.scales[static_cast<int64_t>(from) * 2 * p.g.kv_heads + i];
}

__global__ void __launch_bounds__(kCopyThreads) kv_copy_kernel(const __grid_constant__ CopyArgs p) {
  const int i = blockIdx.x / p.chunks, chunk = blockIdx.x % p.chunks;
  copy_page(p, p.src[i], p.dst[i], chunk);
}
__global__ void __launch_bounds__(kCopyThreads)
    kv_copy_list_kernel(const __grid_constant__ CopyArgs p, const __grid_constant__ PairList l) {
  const int i = blockIdx.x / p.chunks, chunk = blockIdx.x % p.chunks;
  copy_page(p, l.src[i], l.dst[i], chunk);
}

CopyArgs copy_args(const View& v) {
  CopyArgs a{};
  a.g = kv_geom(v);
  const uint64_t used = 2ull * v.kv_heads * v.page_tokens * v.head_dim;
  a.chunk_bytes = kCopyThreads * 16 * kCopyUnroll;  // 16 KiB
  a.chunks = static_cast<int>((used + a.chunk_bytes - 1) / a.chunk_bytes);
  return a;
}

// Queue copies of (src, dst) page pairs known on the host.
int copy_pairs(View* v, const std::vector<std::pair<int32_t, int32_t>>& pairs, cudaStream_t stream) {
  if (pairs.empty()) return RIMURU_OK;
  CopyArgs a = copy_args(*v);
  PairList l;
  for (size_t i = 0; i < pairs.size(); i += kPairsPerLaunch) {
    const int n = static_cast<int>(std::min<size_t>(kPairsPerLaunch, pairs.size() - i));
    for (int j = 0; j < n; ++j) {
      l.src[j] = pairs[i + j].first;
      l.dst[j] = pairs[i + j].second;
    }
    kv_copy_list_kernel<<<n * a.chunks, kCopyThreads, 0, stream>>>(a, l);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(RIMURU_ERR_CUDA, kv_cuda_msg("page copy launch", e));
  }
  return RIMURU_OK;
}

}  // namespace
}  // namespace rimuru

using rimuru::fail;

extern "C" {

uint64_t rimuru_kv_scale_bytes(rimuru_view_t view, int kv_heads) {
  if (!view || kv_heads <= 0) return 0;
  return static_cast<uint64_t>(view->v.n_pages) * 2u * static_cast<uint64_t>(kv_heads) * sizeof(float);
}

int rimuru_view_set_kv_shape(rimuru_view_t view, int kv_heads, int head_dim, int page_tokens,
                             float* dev_scales, uint64_t scales_bytes) {
  rimuru::clear_error();
  if (!view) return fail(RIMURU_ERR_ARG, "null view");
  rimuru::View& v = view->v;
  if (v.has_shape) return fail(RIMURU_ERR_STATE, "view already has an MoE shape");
  if (v.has_kv) return fail(RIMURU_ERR_STATE, "view already has a KV shape");
  if (v.has_state) return fail(RIMURU_ERR_STATE, "view already has a state shape");
  if (kv_heads <= 0 || head_dim <= 0 || page_tokens <= 0)
    return fail(RIMURU_ERR_ARG, "shape values must be positive");
  if (!dev_scales) return fail(RIMURU_ERR_ARG, "null scales");
  if (reinterpret_cast<uintptr_t>(dev_scales) % 16 != 0)
    return fail(RIMURU_ERR_ALIGN, "scales must be 16-byte aligned");
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return fail(RIMURU_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256");
  if (page_tokens != 16 && page_tokens != 32 && page_tokens != 64)
    return fail(RIMURU_ERR_UNSUPPORTED, "page_tokens must be 16, 32 or 64");
  const uint64_t block = static_cast<uint64_t>(page_tokens) * head_dim;
  if (kv_heads > 1024 || 2u * kv_heads * block > v.page_bytes)
    return fail(RIMURU_ERR_UNSUPPORTED, "page_tokens tokens of all heads must fit in one page");
  if (v.page_bytes % block != 0)
    return fail(RIMURU_ERR_UNSUPPORTED, "page size must be a multiple of page_tokens * head_dim");
  if (v.n_pages > std::numeric_limits<int32_t>::max())
    return fail(RIMURU_ERR_UNSUPPORTED, "view has too many pages for an int32 page table");
  if (scales_bytes < rimuru_kv_scale_bytes(view, kv_heads))
    return fail(RIMURU_ERR_ARG, "scales array smaller than rimuru_kv_scale_bytes()");
  v.kv_heads = kv_heads;
  v.head_dim = head_dim;
  v.page_tokens = page_tokens;
  v.scales = dev_scales;
  v.has_kv = true;
  return RIMURU_OK;
}

int rimuru_kv_append(rimuru_view_t view, const rimuru_heads* k, const rimuru_heads* v_in,
                     const int32_t* cu_new, const int32_t* kv_lens, int num_seqs, int num_tokens,
                     const int32_t* page_table, int64_t table_stride, void* stream) {
  using namespace rimuru;
  clear_error();
  if (!view) return fail(RIMURU_ERR_ARG, "null view");
  View& v = view->v;
  if (!v.has_kv) return fail(RIMURU_ERR_STATE, "view has no KV shape");
  if (num_seqs < 0 || num_tokens < 0) return fail(RIMURU_ERR_ARG, "negative count");
  if (num_seqs == 0 || num_tokens == 0) return RIMURU_OK;
  int st = check_heads(k, "keys");
  if (st == RIMURU_OK) st = check_heads(v_in, "values");
  if (st != RIMURU_OK) return st;
  if (k->heads != v.kv_heads || v_in->heads != v.kv_heads)
    return fail(RIMURU_ERR_ARG, "keys and values must have the view's kv_heads heads");
  if (k->dtype != v_in->dtype) return fail(RIMURU_ERR_ARG, "keys and values must have one type");
  if (!cu_new || !kv_lens || !page_table) return fail(RIMURU_ERR_ARG, "null device pointer");
  if (table_stride <= 0) return fail(RIMURU_ERR_ARG, "table_stride must be positive");
  st = kv_ready(&v);
  if (st != RIMURU_OK) return st;
  AppendArgs a{};
  a.x[0] = k->data;
  a.x[1] = v_in->data;
  a.ts[0] = k->token_stride;
  a.ts[1] = v_in->token_stride;
  a.hs[0] = k->head_stride;
  a.hs[1] = v_in->head_stride;
  a.s = {cu_new, kv_lens, page_table, table_stride, num_seqs, num_tokens, max_len(v, table_stride)};
  a.g = kv_geom(v);
  const int64_t units = num_tokens / v.page_tokens + 2ll * num_seqs;
  if (units > std::numeric_limits<int32_t>::max()) return fail(RIMURU_ERR_ARG, "too many sequences");
  // Sixteen warps, shared out over the slices.  With a token or two a sequence (a
  // decode step) there is nothing to share: one warp a slice, eight at most.
  const int slices = 2 * v.kv_heads;
  const bool few = num_tokens < 4ll * num_seqs;
  a.warps_per_slice = few ? 1 : std::max(1, kAppendWarps / slices);
  const int threads = 32 * std::min(few ? 8 : kAppendWarps, slices * a.warps_per_slice);
  const dim3 grid(static_cast<unsigned>(units));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (k->dtype == RIMURU_BF16) kv_append_kernel<__nv_bfloat16><<<grid, threads, 0, s>>>(a);
  else if (k->dtype == RIMURU_F16) kv_append_kernel<__half><<<grid, threads, 0, s>>>(a);
  else kv_append_kernel<float><<<grid, threads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(RIMURU_ERR_CUDA, kv_cuda_msg("append launch", e));
  return RIMURU_OK;
}

int rimuru_kv_copy_pages(rimuru_view_t view, const int32_t* src, const int32_t* dst, int n,
                         void* stream) {
  using namespace rimuru;
  clear_error();
  if (!view) return fail(RIMURU_ERR_ARG, "null view");
  View& v = view->v;
  if (!v.has_kv) return fail(RIMURU_ERR_STATE, "view has no KV shape");
  if (n < 0) return fail(RIMURU_ERR_ARG, "negative count");
  if (n == 0) return RIMURU_OK;
  if (!src || !dst) return fail(RIMURU_ERR_ARG, "null device pointer");
  int st = kv_ready(&v);
  if (st != RIMURU_OK) return st;
  CopyArgs a = copy_args(v);
  a.src = src;
  a.dst = dst;
  if (static_cast<int64_t>(n) * a.chunks > std::numeric_limits<int32_t>::max())
    return fail(RIMURU_ERR_ARG, "too many pages in one call");
  kv_copy_kernel<<<n * a.chunks, kCopyThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(RIMURU_ERR_CUDA, kv_cuda_msg("page copy launch", e));
  return RIMURU_OK;
}

int rimuru_kv_fork(rimuru_view_t view, const int32_t* pages, int kv_len, int n, int32_t* children,
                   int64_t child_stride, void* stream) {
  using namespace rimuru;
  clear_error();
  if (!view) return fail(RIMURU_ERR_ARG, "null view");
  View& v = view->v;
  if (!v.has_kv) return fail(RIMURU_ERR_STATE, "view has no KV shape");
  if (kv_len < 0 || n < 0) return fail(RIMURU_ERR_ARG, "negative count");
  if (kv_len == 0 || n == 0) return RIMURU_OK;
  if (!pages || !children) return fail(RIMURU_ERR_ARG, "null pointer");
  const int64_t used = (static_cast<int64_t>(kv_len) + v.page_tokens - 1) / v.page_tokens;
  const int64_t full = kv_len / v.page_tokens;
  if (child_stride < used) return fail(RIMURU_ERR_ARG, "child_stride shorter than the sequence");
  std::vector<std::pair<int32_t, int32_t>> copies;
  if (full < used) {  // a copy will be launched: the device has to be right before anything changes
    int st = kv_ready(&v);
    if (st != RIMURU_OK) return st;
  }
  {
    std::lock_guard<std::mutex> g(v.pool->mu);
    const int lvl = v.pool->level_of(v.page_bytes);
    const Level& L = v.pool->levels[lvl];
    for (int64_t i = 0; i < used; ++i) {
      if (pages[i] < 0 || pages[i] >= L.n_pages) return fail(RIMURU_ERR_RANGE, "page id out of range");
      if (L.state[pages[i]] != Level::OWNED || L.owner[pages[i]] != v.id)
        return fail(RIMURU_ERR_STATE, "page is not owned by this view");
    }
    // whatever may fail comes first: entries for the references, and the children's own pages
    const auto undo = [&] {
      for (const auto& p : copies) v.pool->release(lvl, v.id, p.second);
      for (int64_t i = 0; i < full; ++i) {
        auto r = v.extra_refs.find(pages[i]);
        if (r != v.extra_refs.end() && r->second == 0) v.extra_refs.erase(r);
      }
    };
    try {
      for (int64_t i = 0; i < full; ++i) v.extra_refs.try_emplace(pages[i], 0);
      for (int c = 0; full < used && c < n; ++c) {
        copies.emplace_back(pages[used - 1], -1);
        int64_t id = -1;
        int st = v.pool->alloc_near(lvl, v.id, pages[used - 1], &id);
        if (st != RIMURU_OK) {
          copies.pop_back();
          const std::string msg = rimuru_last_error();
          undo();
          return fail(st, msg);
        }
        copies.back().second = static_cast<int32_t>(id);
      }
    } catch (const std::bad_alloc&) {
      if (!copies.empty() && copies.back().second < 0) copies.pop_back();
      undo();
      return fail(RIMURU_ERR_OOM, "host allocation failed");
    }
    for (int64_t i = 0; i < full; ++i) v.extra_refs.find(pages[i])->second += n;
  }
  for (int c = 0; c < n; ++c) {
    int32_t* row = children + c * child_stride;
    for (int64_t i = 0; i < full; ++i) row[i] = pages[i];
    if (full < used) row[full] = copies[c].second;
  }
  return copy_pairs(&v, copies, static_cast<cudaStream_t>(stream));
}

int rimuru_kv_compact(rimuru_view_t view, int32_t* tables, int64_t n_entries, int max_moves,
                      int* moved, void* stream) {
  using namespace rimuru;
  clear_error();
  if (!view || !moved) return fail(RIMURU_ERR_ARG, "null argument");
  View& v = view->v;
  *moved = 0;
  if (!v.has_kv) return fail(RIMURU_ERR_STATE, "view has no KV shape");
  if (n_entries < 0 || max_moves < 0) return fail(RIMURU_ERR_ARG, "negative count");
  if (n_entries == 0 || max_moves == 0) return RIMURU_OK;
  if (!tables) return fail(RIMURU_ERR_ARG, "null tables");
  int st = kv_ready(&v);
  if (st != RIMURU_OK) return st;
  std::vector<std::pair<int32_t, int32_t>> moves;
  try {
    std::lock_guard<std::mutex> g(v.pool->mu);
    const int lvl = v.pool->level_of(v.page_bytes);
    if (lvl == 0) return RIMURU_OK;  // huge pages have no parent to merge into
    Level& L = v.pool->levels[lvl];
    std::unordered_map<int32_t, int32_t> to;  // pages in the tables, and where they go
    for (int64_t i = 0; i < n_entries; ++i) {
      if (tables[i] < 0) continue;
      if (tables[i] >= L.n_pages) return fail(RIMURU_ERR_RANGE, "page id out of range");
      if (L.state[tables[i]] != Level::OWNED || L.owner[tables[i]] != v.id)
        return fail(RIMURU_ERR_STATE, "page is not owned by this view");
      to.emplace(tables[i], -1);
    }
    moves.reserve(std::min<size_t>(max_moves, to.size()));
    // every parent that holds a page of the tables: how many are in use, how many
    // free, and whether all in use can move
    struct Parent {
      int64_t id;
      int used, free;
      bool movable;
    };
    const int64_t per = static_cast<int64_t>(v.pool->levels[lvl - 1].page_bytes / L.page_bytes);
    std::unordered_map<int64_t, char> seen;
    std::vector<Parent> parents;
    for (const auto& e : to) {
      const int64_t q = e.first / per;
      if (!seen.emplace(q, 1).second) continue;
      Parent p{q, 0, 0, true};
      for (int64_t c = q * per; c < (q + 1) * per; ++c) {
        if (L.state[c] == Level::FREE) {
          p.free += 1;
        } else {
          p.used += 1;
          if (L.state[c] != Level::OWNED || L.owner[c] != v.id || !to.count(static_cast<int32_t>(c)))
            p.movable = false;
        }
      }
      if (p.free > 0) parents.push_back(p);
    }
    std::sort(parents.begin(), parents.end(), [](const Parent& a, const Parent& b) {
      return a.used != b.used ? a.used < b.used : a.id > b.id;
    });
    // sources from the sparse end, destinations from the full end, until they meet
    size_t last = parents.size();
    int64_t room = 0;
    for (const Parent& p : parents) room += p.free;
    int64_t slot = 0;
    for (size_t s = 0; s < last; ++s) {
      const Parent& p = parents[s];
      room -= p.free;  // free pages in the parents that stay
      if (!p.movable || p.used > room ||
          static_cast<int64_t>(moves.size()) + p.used > max_moves) {
        if (p.movable) break;  // later sources hold more pages and leave less room
        continue;
      }
      for (int64_t c = p.id * per; c < (p.id + 1) * per; ++c) {
        if (L.state[c] != Level::OWNED) continue;
        // next free page of the fullest destination
        while (parents[last - 1].free == 0) --last, slot = 0;
        Parent& d = parents[last - 1];
        while (L.state[d.id * per + slot] != Level::FREE) ++slot;
        const int64_t dst = d.id * per + slot;
        st = v.pool->place(lvl, v.id, dst);
        if (st != RIMURU_OK) return st;
        d.free -= 1;
        room -= 1;
        moves.emplace_back(static_cast<int32_t>(c), static_cast<int32_t>(dst));
      }
    }
    for (const auto& m : moves) {
      to[m.first] = m.second;
      auto extra = v.extra_refs.extract(m.first);
      if (!extra.empty()) {
        extra.key() = m.second;
        v.extra_refs.insert(std::move(extra));
      }
      v.pool->release(lvl, v.id, m.first);
    }
    for (int64_t i = 0; i < n_entries; ++i) {
      if (tables[i] < 0) continue;
      const int32_t t = to[tables[i]];
      if (t >= 0) tables[i] = t;
    }
  } catch (const std::bad_alloc&) {
    return fail(RIMURU_ERR_OOM, "host allocation failed");
  }
  *moved = static_cast<int>(moves.size());
  return copy_pairs(&v, moves, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
