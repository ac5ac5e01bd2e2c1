// Beam search: the selection over beams and vocabulary, and the reordering of the paged
// cache that follows it.
//
// Selection.  A candidate (beam b, token v) is worth (x_v - m_b) + c_b with m_b
// the row's maximum and c_b = score_b - log(sum exp(x - m_b)), so one row's candidates stand in the order of its logits, and the sum
// and the order need one read of them.  The first kernel streams the logits once: for
// each run of 64 tokens (a group) it keeps the largest logit, for each of its chunks of a
// row the maximum and the sum of exponentials.  The n best candidates lie in the n best
// groups (by value, then by position: whoever is outside has n better group leaders
// before it), so the second kernel, one CTA a batch entry, looks at the group maxima,
// reads n groups of logits again and ranks what may be among the n best.
// Comparisons that decide are made on doubles; fp32 only sieves, with a margin.
#include <algorithm>
#include <cmath>

#include "device.cuh"
#include "kv.h"

namespace rimuru {
namespace {

constexpr int kGroup = 64;             // tokens of a group
constexpr int kChunk = 8192;           // tokens of a first-kernel CTA
constexpr int kScanThreads = 256;
constexpr int kPickThreads = 1024;
constexpr int kLeaders = 256;          // subsets whose best give the sieve
constexpr int kMostSelect = 128;
constexpr int kList = 512;             // candidates that are ranked by counting
constexpr int kMostBeams = 128;
constexpr float kLog2e = 1.4426950408889634f;

struct BeamArgs {
  const void* logits;
  int64_t row_stride;
  int vocab;
  const float* scores;
  const uint8_t* done;
  int groups, beams, pad, n_select;
  float* best;
  int32_t *rows, *tokens;
  int shift_elems;   // elements of 16 bytes
  int n_groups;      // groups of a row
  int n_chunks;
  float* top;        // [rows][n_groups]
  float2* parts;     // [rows][n_chunks] maximum and sum of exp(x - maximum)
};

__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(float x) { return x; }

// 2^x; the instruction is good to 2^-22, far below what a sum of thousands of terms keeps.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A NaN counts as -inf, infinities as the largest finite value.
__device__ __forceinline__ float tame(float x) {
  return x != x ? -INFINITY : fminf(x, 3.402823466e38f);
}

// Row r's first element lies `skip` elements past a 16-byte boundary; places count from there.
template <typename T>
__device__ __forceinline__ const T* row_base(const BeamArgs& a, int row, int* skip) {
  const T* p = static_cast<const T*>(a.logits) + row * a.row_stride;
  *skip = static_cast<int>(reinterpret_cast<uintptr_t>(p) % 16 / sizeof(T));
  return p - *skip;
}

// Eight elements from place `at` (a multiple of 8); places outside [skip, end) are -inf.
template <typename T>
__device__ __forceinline__ void load8(const T* base, int at, int skip, int end, float (&x)[8]) {
  if (at >= skip && at + 8 <= end) {
    uint4 w[sizeof(T) / 2];
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) w[i] = dev::ld_nc_na_v4(base + at + i * (16 / sizeof(T)));
    const T* t = reinterpret_cast<const T*>(w);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = to_f(t[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = at + e >= skip && at + e < end ? to_f(base[at + e]) : -INFINITY;
  }
}

// Maximum and sum of two parts.
__device__ __forceinline__ float2 join(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x);
  float s = 0.f;
  if (a.x > -INFINITY) s += a.y * ex2((a.x - m) * kLog2e);
  if (b.x > -INFINITY) s += b.y * ex2((b.x - m) * kLog2e);
  return make_float2(m, s);
}

template <typename T>
__global__ void __launch_bounds__(kScanThreads) beam_scan_kernel(const __grid_constant__ BeamArgs a) {
  dev::grid_dep_launch();
  __shared__ float2 warp_part[kScanThreads / 32];
  const int row = blockIdx.y, tid = threadIdx.x;
  if (a.done && a.done[row]) return;
  int skip;
  const T* base = row_base<T>(a, row, &skip);
  const int end = skip + a.vocab;
  constexpr int kVec = 4;  // vectors of eight in flight
  float2 part = make_float2(-INFINITY, 0.f);
  const int c0 = blockIdx.x * kChunk;
#pragma unroll 1
  for (int c = c0; c < c0 + kChunk && c < end; c += kScanThreads * 8 * kVec) {
    float x[kVec][8];
#pragma unroll
    for (int j = 0; j < kVec; ++j) load8(base, c + (j * kScanThreads + tid) * 8, skip, end, x[j]);
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      float v = x[j][0];
#pragma unroll
      for (int e = 1; e < 8; ++e) v = fmaxf(v, x[j][e]);
      v = fmaxf(v, -INFINITY);
      m = fmaxf(m, v);
#pragma unroll
      for (int s = 1; s < 8; s <<= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, s));
      const int g = (c + (j * kScanThreads + tid) * 8) / kGroup;
      if (tid % 8 == 0 && g < a.n_groups) a.top[static_cast<int64_t>(row) * a.n_groups + g] = fminf(v, 3.402823466e38f);
    }
    if (m > part.x) {
      part.y = part.x > -INFINITY ? part.y * ex2((part.x - fminf(m, 3.402823466e38f)) * kLog2e) : 0.f;
      part.x = fminf(m, 3.402823466e38f);
    }
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      float u = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) u += ex2((x[j][e] - part.x) * kLog2e);
      s += u;
    }
    if (!(s <= 3.402823466e38f)) {  // a NaN or an infinity among them, or nothing finite so far
      s = 0.f;
#pragma unroll
      for (int j = 0; j < kVec; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float v = tame(x[j][e]);
          if (v > -INFINITY) s += ex2((v - part.x) * kLog2e);
        }
    }
    part.y += s;
  }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1)
    part = join(part, make_float2(__shfl_xor_sync(~0u, part.x, m), __shfl_xor_sync(~0u, part.y, m)));
  if (tid % 32 == 0) warp_part[tid / 32] = part;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kScanThreads / 32; ++w) part = join(part, warp_part[w]);
    a.parts[static_cast<int64_t>(row) * a.n_chunks + blockIdx.x] = part;
  }
}

// Doubles as unsigned numbers in the same order.
__device__ __forceinline__ uint64_t ordered(double x) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x + 0.0));  // -0 and 0 are one value
  return u >> 63 ? ~u : u | 1ull << 63;
}
__device__ __forceinline__ double unordered(uint64_t u) {
  return __longlong_as_double(static_cast<long long>(u >> 63 ? u & ~(1ull << 63) : ~u));
}
constexpr uint64_t kNothing = 0x000FFFFFFFFFFFFFull;  // ordered(-inf)

struct Candidate {
  uint64_t key;  // ordered(worth)
  int index;     // position among the batch entry's, or INT_MAX
};
__device__ __forceinline__ bool before(Candidate a, Candidate b) {
  return a.key > b.key || (a.key == b.key && a.index < b.index);
}

struct PickShared {
  double c[kMostBeams];  // a candidate is worth (x - m) + c
  float c32[kMostBeams], m[kMostBeams];
  uint8_t done[kMostBeams];
  float leader[kLeaders];
  Candidate list[kList], chosen[kMostSelect], next[kPickThreads / 32];
  int count, n_chosen;
  float sieve;
};

// The `want` first candidates of a stream in order, into s.chosen[0 .. s.n_chosen).
// rough(i, &err): fp32 worth of item i and a bound of its error; exact(i): the candidate.
// Candidates worth -inf (in fp32) are left out.  All threads of the CTA call it.
template <typename Rough, typename Exact>
__device__ void pick(PickShared& s, int n, int want, const Rough& rough, const Exact& exact) {
  const int tid = threadIdx.x;
  // The best of each of 256 subsets, from below: the want-th largest of them bounds the
  // want-th best of all.
  float m = -INFINITY;
  for (int i = tid; i < n; i += kPickThreads) {
    float err;
    const float r = rough(i, &err);
    m = fmaxf(m, r - err);
  }
  m = fmaxf(m, __shfl_xor_sync(~0u, m, 1));
  m = fmaxf(m, __shfl_xor_sync(~0u, m, 2));
  if (tid % 4 == 0) s.leader[tid / 4] = m;
  if (tid == 0) s.count = s.n_chosen = 0;
  __syncthreads();
  if (tid < kLeaders) {
    const float mine = s.leader[tid];
    int above = 0;
#pragma unroll 8
    for (int i = 0; i < kLeaders; ++i) above += s.leader[i] > mine || (s.leader[i] == mine && i < tid);
    if (above == want - 1) s.sieve = mine;
  }
  __syncthreads();
  const float sieve = s.sieve;
  const auto passes = [&](int i) {
    float err;
    const float r = rough(i, &err);
    return r > -INFINITY && r + err >= sieve;
  };
  for (int i = tid; i < n; i += kPickThreads)
    if (passes(i)) {
      const int at = atomicAdd(&s.count, 1);
      if (at < kList) s.list[at] = exact(i);
    }
  __syncthreads();
  if (s.count <= kList) {
    const int count = s.count;
    // a warp for each listed candidate: how many come before it
    for (int i = tid / 32; i < count; i += kPickThreads / 32) {
      const Candidate mine = s.list[i];
      int n_before = 0;
      for (int j = tid % 32; j < count; j += 32) n_before += before(s.list[j], mine);
      n_before = __reduce_add_sync(~0u, n_before);
      if (tid % 32 == 0 && n_before < want && mine.key > kNothing) {
        s.chosen[n_before] = mine;
        atomicAdd(&s.n_chosen, 1);
      }
    }
    __syncthreads();
    return;
  }
  // Many candidates near the border (rows that are alike): one at a time.
  Candidate last{~0ull, -1};
  for (int k = 0; k < want; ++k) {
    Candidate mine{0, 0x7FFFFFFF};
    for (int i = tid; i < n; i += kPickThreads) {
      if (!passes(i)) continue;
      const Candidate c = exact(i);
      if (before(last, c) && before(c, mine)) mine = c;
    }
    for (int w = 16; w > 0; w >>= 1) {
      const Candidate c{__shfl_xor_sync(~0u, mine.key, w), __shfl_xor_sync(~0u, mine.index, w)};
      if (before(c, mine)) mine = c;
    }
    if (tid % 32 == 0) s.next[tid / 32] = mine;
    __syncthreads();
    mine = s.next[0];
    for (int w = 1; w < kPickThreads / 32; ++w)
      if (before(s.next[w], mine)) mine = s.next[w];
    __syncthreads();
    if (mine.key <= kNothing) break;
    if (tid == 0) s.chosen[k] = mine, s.n_chosen = k + 1;
    last = mine;
  }
  __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kPickThreads) beam_pick_kernel(const __grid_constant__ BeamArgs a) {
  __shared__ PickShared s;
  __shared__ int group_of[kMostSelect];
  const int entry = blockIdx.x, tid = threadIdx.x;
  const int row0 = entry * a.beams;
  dev::grid_dep_wait();
  // what a beam's logits have to be raised by: a warp for each beam
  for (int b = tid / 32; b < a.beams; b += kPickThreads / 32) {
    const int row = row0 + b;
    const bool done = a.done && a.done[row];
    float2 part = make_float2(-INFINITY, 0.f);
    if (!done)
      for (int c = tid % 32; c < a.n_chunks; c += 32) part = join(part, a.parts[static_cast<int64_t>(row) * a.n_chunks + c]);
    for (int m = 16; m > 0; m >>= 1)
      part = join(part, make_float2(__shfl_xor_sync(~0u, part.x, m), __shfl_xor_sync(~0u, part.y, m)));
    if (tid % 32 == 0) {
      const float score = tame(a.scores[row]);
      double c = static_cast<double>(score);
      if (!done) c = part.y > 0.f ? c - log(static_cast<double>(part.y)) : -INFINITY;
      s.m[b] = done || !(part.x > -INFINITY) ? 0.f : part.x;
      s.c[b] = c;
      s.c32[b] = static_cast<float>(c);
      s.done[b] = done;
    }
  }
  __syncthreads();
  // c32 is off by 2^-24 of c, the difference and the sum by 2^-24 of themselves
  const auto sum32 = [&](int b, float x, float* err) {
    const float d = x - s.m[b];
    *err = (fabsf(s.c32[b]) + fabsf(d)) * 0x1p-22f;
    return s.c32[b] + d;
  };
  const auto worth = [&](int b, float x) {
    return ordered((static_cast<double>(x) - static_cast<double>(s.m[b])) + s.c[b]);
  };
  // A finished beam is one group of one candidate, its pad token.
  const int G = a.n_groups;
  const auto group_top = [&](int i, int b) -> float {
    if (s.done[b]) return i == b * G ? 0.f : -INFINITY;
    return a.top[static_cast<int64_t>(row0) * G + i];
  };
  const int want = a.n_select;
  pick(s, a.beams * G, want,
       [&](int i, float* err) { return sum32(i / G, group_top(i, i / G), err); },
       [&](int i) { return Candidate{worth(i / G, group_top(i, i / G)), i}; });
  const int n_groups = s.n_chosen;
  if (tid < n_groups) group_of[tid] = s.chosen[tid].index;
  __syncthreads();

  // the elements of those groups; an index is beam * vocab + token
  const auto element = [&](int i, int* beam, int* token) -> float {
    const int g = group_of[i / kGroup], e = i % kGroup;
    *beam = g / G;
    const int row = row0 + *beam;
    if (s.done[*beam]) {
      *token = a.pad;
      return e == 0 ? 0.f : -INFINITY;
    }
    int skip;
    const T* base = row_base<T>(a, row, &skip);
    const int at = (g - *beam * G) * kGroup + e;
    *token = at - skip;
    return at >= skip && at < skip + a.vocab ? tame(to_f(base[at])) : -INFINITY;
  };
  pick(s, n_groups * kGroup, want,
       [&](int i, float* err) {
         int b, v;
         const float x = element(i, &b, &v);
         return sum32(b, x, err);
       },
       [&](int i) {
         int b, v;
         const float x = element(i, &b, &v);
         return Candidate{worth(b, x), b * a.vocab + v};
       });
  for (int k = tid; k < want; k += kPickThreads) {
    const int64_t at = static_cast<int64_t>(entry) * want + k;
    const bool live = k < s.n_chosen;
    const Candidate c = s.chosen[live ? k : 0];
    a.best[at] = live ? static_cast<float>(unordered(c.key)) : -INFINITY;
    a.rows[at] = live ? row0 + c.index / a.vocab : -1;
    a.tokens[at] = live ? c.index % a.vocab : -1;
  }
}

template <typename T>
cudaError_t launch(const BeamArgs& a, cudaStream_t s) {
  const int rows = a.groups * a.beams;
  for (int r = 0; r < rows; r += 65535 / a.beams * a.beams) {  // grid.y ends at 65535
    BeamArgs p = a;
    const int n = std::min(65535 / a.beams * a.beams, rows - r);
    p.logits = static_cast<const T*>(a.logits) + r * a.row_stride;
    p.done = a.done ? a.done + r : nullptr;
    p.top += static_cast<int64_t>(r) * a.n_groups;
    p.parts += static_cast<int64_t>(r) * a.n_chunks;
    beam_scan_kernel<T><<<dim3(a.n_chunks, n), kScanThreads, 0, s>>>(p);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.groups);
  cfg.blockDim = dim3(kPickThreads);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, beam_pick_kernel<T>, a);
  const cudaError_t last = cudaGetLastError();
  return e != cudaSuccess ? e : last;
}

// ------------------------------------------------------------------ reordering
struct ReorderArgs {
  const int32_t *parents, *lens, *table_in, *fresh;
  int32_t *table_out, *lens_out;
  int n, n_parents;
  int64_t stride;
  KvGeom g;
  int max_len;
};
constexpr int kReorderThreads = 256;

// One CTA a (layer, child): the row of the table, and the page that is partly filled.
__global__ void __launch_bounds__(kReorderThreads) kv_reorder_kernel(const __grid_constant__ ReorderArgs a) {
  const int layer = blockIdx.y, child = blockIdx.x, tid = threadIdx.x;
  const int64_t out_row = static_cast<int64_t>(layer) * a.n + child;
  const int fresh = a.fresh[out_row];
  const int parent = a.parents[child];
  if (parent == -1) {  // no such child
    if (layer == 0 && tid == 0) a.lens_out[child] = 0;
    return;
  }
  if (parent < 0 || parent >= a.n_parents) {
    if (layer == 0 && tid == 0) {
      a.lens_out[child] = 0;
      dev::set_error(a.g.err, RIMURU_DEV_BAD_SHAPE);
    }
    return;
  }
  const int len = a.lens[parent], P = a.g.page_tokens;
  if (len < 0 || len > a.max_len) {
    if (layer == 0 && tid == 0) {
      a.lens_out[child] = 0;
      dev::set_error(a.g.err, RIMURU_DEV_BAD_SHAPE);
    }
    return;
  }
  const int full = len / P;
  const bool partly = len % P != 0;
  const int32_t* from = a.table_in + (static_cast<int64_t>(layer) * a.n_parents + parent) * a.stride;
  int32_t* to = a.table_out + out_row * a.stride;
  if (layer == 0 && tid == 0) a.lens_out[child] = len;
  if (partly) {
    const int src = from[full];
    if (src < 0 || src >= a.g.num_pages || fresh < 0 || fresh >= a.g.num_pages) {
      if (tid == 0) {
        to[full] = -1;
        dev::set_error(a.g.err, RIMURU_DEV_BAD_PAGE);
      }
    } else {
      const int words = 2 * a.g.kv_heads * P * a.g.head_dim / 16;
      const uint4* x = reinterpret_cast<const uint4*>(a.g.pool + static_cast<uint64_t>(src) * a.g.page_bytes);
      uint4* y = reinterpret_cast<uint4*>(a.g.pool + static_cast<uint64_t>(fresh) * a.g.page_bytes);
      constexpr int kPer = 8;
#pragma unroll 1
      for (int i0 = 0; i0 < words; i0 += kPer * kReorderThreads) {
        uint4 v[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int i = i0 + j * kReorderThreads + tid;
          if (i < words) v[j] = x[i];
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int i = i0 + j * kReorderThreads + tid;
          if (i < words) y[i] = v[j];
        }
      }
      const int n_scales = 2 * a.g.kv_heads;
      for (int i = tid; i < n_scales; i += kReorderThreads)
        a.g.scales[static_cast<int64_t>(fresh) * n_scales + i] = a.g.scales[static_cast<int64_t>(src) * n_scales + i];
      if (tid == 0) to[full] = fresh;
    }
  }
  for (int i = tid; i < full; i += kReorderThreads) to[i] = from[i];
}

}  // namespace
}  // namespace rimuru

using rimuru::fail;

namespace {
// Groups of a row: a row may begin up to eight elements past a 16-byte boundary.
int64_t row_groups(int vocab) { return (static_cast<int64_t>(vocab) + 7 + rimuru::kGroup - 1) / rimuru::kGroup; }
int64_t row_chunks(int vocab) { return (static_cast<int64_t>(vocab) + 7 + rimuru::kChunk - 1) / rimuru::kChunk; }
}  // namespace

extern "C" uint64_t rimuru_beam_select_workspace_bytes(int num_groups, int beams, int vocab, int n_select) {
  if (num_groups < 0 || beams <= 0 || vocab <= 0 || n_select <= 0) return 0;
  const uint64_t rows = static_cast<uint64_t>(num_groups) * beams;
  return (rows * row_groups(vocab) * sizeof(float) + 1023) / 1024 * 1024 + rows * row_chunks(vocab) * sizeof(float2) + 1024;
}

extern "C" int rimuru_beam_select(const rimuru_rows* logits, const float* scores, const uint8_t* done,
                                  int num_groups, int beams, int pad_token, int n_select, float* out_scores,
                                  int32_t* out_rows, int32_t* out_tokens, void* workspace,
                                  uint64_t workspace_bytes, void* stream) {
  using namespace rimuru;
  clear_error();
  if (num_groups < 0) return fail(RIMURU_ERR_ARG, "negative count");
  if (!logits) return fail(RIMURU_ERR_ARG, "logits: null descriptor");
  if (beams <= 0 || n_select <= 0 || logits->cols <= 0)
    return fail(RIMURU_ERR_ARG, "beams, n_select and the vocabulary must be positive");
  if (logits->dtype != RIMURU_BF16 && logits->dtype != RIMURU_F16 && logits->dtype != RIMURU_F32)
    return fail(RIMURU_ERR_ARG, "logits: unknown element type");
  if (beams > kMostBeams || n_select > kMostSelect)
    return fail(RIMURU_ERR_UNSUPPORTED, "at most 128 beams and 128 selected candidates");
  if (static_cast<int64_t>(beams) * (logits->cols + 2ll * kGroup) > (1 << 30) ||
      static_cast<int64_t>(num_groups) * beams > (1 << 24))
    return fail(RIMURU_ERR_UNSUPPORTED, "too many beams and tokens for one call");
  if (num_groups == 0) return RIMURU_OK;
  if (!logits->data || !scores || !out_scores || !out_rows || !out_tokens || !workspace)
    return fail(RIMURU_ERR_ARG, "null device pointer");
  if (logits->row_stride < 0) return fail(RIMURU_ERR_ARG, "logits: negative stride");
  if (done && (pad_token < 0 || pad_token >= logits->cols))
    return fail(RIMURU_ERR_ARG, "pad_token must be a token where beams may be finished");
  if (reinterpret_cast<uintptr_t>(logits->data) % element_bytes(logits->dtype) != 0)
    return fail(RIMURU_ERR_ALIGN, "logits must be aligned to their type");
  const uintptr_t words = reinterpret_cast<uintptr_t>(scores) | reinterpret_cast<uintptr_t>(out_scores) |
                          reinterpret_cast<uintptr_t>(out_rows) | reinterpret_cast<uintptr_t>(out_tokens);
  if (words % 4 != 0) return fail(RIMURU_ERR_ALIGN, "scores and outputs must be 4-byte aligned");
  if (reinterpret_cast<uintptr_t>(workspace) % 1024 != 0)
    return fail(RIMURU_ERR_ALIGN, "workspace must be 1024-byte aligned");
  const uint64_t need = rimuru_beam_select_workspace_bytes(num_groups, beams, logits->cols, n_select);
  if (workspace_bytes < need)
    return fail(RIMURU_ERR_WORKSPACE, "workspace needs " + std::to_string(need) + " bytes");
  BeamArgs a{};
  a.logits = logits->data;
  a.row_stride = logits->row_stride;
  a.vocab = logits->cols;
  a.scores = scores;
  a.done = done;
  a.groups = num_groups, a.beams = beams, a.pad = pad_token, a.n_select = n_select;
  a.best = out_scores, a.rows = out_rows, a.tokens = out_tokens;
  a.n_groups = static_cast<int>(row_groups(logits->cols));
  a.n_chunks = static_cast<int>(row_chunks(logits->cols));
  a.top = static_cast<float*>(workspace);
  const uint64_t rows = static_cast<uint64_t>(num_groups) * beams;
  a.parts = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) +
                                      (rows * a.n_groups * sizeof(float) + 1023) / 1024 * 1024);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = logits->dtype == RIMURU_BF16  ? launch<__nv_bfloat16>(a, s)
                        : logits->dtype == RIMURU_F16 ? launch<__half>(a, s)
                                                      : launch<float>(a, s);
  if (e != cudaSuccess) return fail(RIMURU_ERR_CUDA, kv_cuda_msg("beam selection launch", e));
  return RIMURU_OK;
}

extern "C" int rimuru_kv_reorder(rimuru_view_t view, const int32_t* parents, int num_seqs, const int32_t* kv_lens,
                                 int num_parents, const int32_t* table_in, int32_t* table_out, int num_layers,
                                 int64_t table_stride, const int32_t* fresh, int32_t* lens_out, void* stream) {
  using namespace rimuru;
  clear_error();
  if (!view) return fail(RIMURU_ERR_ARG, "null view");
  View& v = view->v;
  if (!v.has_kv) return fail(RIMURU_ERR_STATE, "view has no KV shape");
  if (num_seqs < 0 || num_parents < 0 || num_layers < 0) return fail(RIMURU_ERR_ARG, "negative count");
  if (num_seqs == 0 || num_layers == 0) return RIMURU_OK;
  if (!parents || !kv_lens || !table_in || !table_out || !fresh || !lens_out)
    return fail(RIMURU_ERR_ARG, "null device pointer");
  if (table_stride <= 0) return fail(RIMURU_ERR_ARG, "table_stride must be positive");
  if (num_layers > 65535) return fail(RIMURU_ERR_UNSUPPORTED, "at most 65535 layers");
  if (table_in == table_out || kv_lens == lens_out)
    return fail(RIMURU_ERR_ARG, "the new tables and lengths need arrays of their own");
  const uintptr_t words = reinterpret_cast<uintptr_t>(parents) | reinterpret_cast<uintptr_t>(kv_lens) |
                          reinterpret_cast<uintptr_t>(table_in) | reinterpret_cast<uintptr_t>(table_out) |
                          reinterpret_cast<uintptr_t>(fresh) | reinterpret_cast<uintptr_t>(lens_out);
  if (words % 4 != 0) return fail(RIMURU_ERR_ALIGN, "arrays must be 4-byte aligned");
  const int st = kv_ready(&v);
  if (st != RIMURU_OK) return st;
  ReorderArgs a{};
  a.parents = parents, a.lens = kv_lens, a.table_in = table_in, a.fresh = fresh;
  a.table_out = table_out, a.lens_out = lens_out;
  a.n = num_seqs, a.n_parents = num_parents;
  a.stride = table_stride;
  a.g = kv_geom(v);
  a.max_len = max_len(v, table_stride);
  kv_reorder_kernel<<<dim3(num_seqs, num_layers), kReorderThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(RIMURU_ERR_CUDA, kv_cuda_msg("reordering launch", e));
  return RIMURU_OK;
}
