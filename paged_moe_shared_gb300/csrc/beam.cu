// Beam search: the selection over beams and vocabulary, and the reordering of the paged
// cache that follows it.
//
// Selection.  A candidate (beam b, token v) is worth (x_v - m_b) + c_b with m_b
// the row's maximum and c_b = score_b - log(sum exp(x - m_b)), so one row's candidates
// stand in the order of its logits, and the sum and the order need one read of them.  The
// first kernel streams the logits once, a warp for each chunk of 1024 tokens, and keeps
// the chunk's maximum and sum of exponentials.  The n best candidates lie in the n best
// chunks (by maximum, then by position: whoever is outside has n better chunk leaders
// before it), so the second kernel, one CTA a batch entry, finds a worth that n leaders
// reach, reads the chunks whose leaders reach it again and ranks what does.  Comparisons that decide are made on
// doubles; fp32 only sieves, with a margin.
//
// 32 entries of 8 beams over 151,936 tokens in bf16 (78 MB), 16 best: 21.7 us, of which the
// scan takes 15.7 (0.73 of the copy rate; 68 % of the issue slots) and the pick 6, a chain of
// a dozen barriers and three dependent loads on one SM an entry.  One entry of 4 beams 8.4 us.  With
// maxima of 64 tokens in place of chunks the scan took 20 us and the pick, which has then
// sixteen times as many, 30.
#include <algorithm>
#include <cmath>

#include "device.cuh"
#include "kv.h"

namespace rimuru {
namespace {

constexpr int kChunk = 1024;           // tokens of a first-kernel warp
constexpr int kScanThreads = 256;
constexpr int kPickThreads = 1024;
constexpr int kLeaders = 256;          // subsets whose best give the sieve, where n_select is above 32; else half
static_assert(kPickThreads == 4 * kLeaders, "");
constexpr int kMostSelect = 128;
constexpr int kList = 1024;            // candidates that are ranked by counting
constexpr int kMostBeams = 128;
constexpr float kLog2e = 1.4426950408889634f;

using dev::ex2;  // far more exact than a sum of thousands of terms
using dev::Raw;
using dev::to_f;
using dev::unpack;

struct BeamArgs {
  const void* logits;
  int64_t row_stride;
  int vocab;
  const float* scores;
  const uint8_t* done;
  int groups, beams, pad, n_select;
  float* best;
  int32_t *rows, *tokens;
  int n_chunks;      // of a row
  float *tops, *sums;  // [rows][n_chunks]: a chunk's maximum, its sum of exp(x - maximum)
};

__device__ __forceinline__ __nv_bfloat16 lowest(__nv_bfloat16) { return __ushort_as_bfloat16(0xFF80); }
__device__ __forceinline__ __half lowest(__half) { return __ushort_as_half(0xFC00); }
__device__ __forceinline__ float lowest(float) { return -INFINITY; }

// A NaN counts as -inf, infinities as the largest finite value.
__device__ __forceinline__ float tame(float x) {
  return x != x ? -INFINITY : fminf(x, 3.402823466e38f);
}

// Row r's first element lies `skip` elements past a 16-byte boundary; places count from that.
template <typename T>
__device__ __forceinline__ const T* row_base(const BeamArgs& a, int row, int* skip) {
  const T* p = static_cast<const T*>(a.logits) + row * a.row_stride;
  *skip = static_cast<int>(reinterpret_cast<uintptr_t>(p) % 16 / sizeof(T));
  return p - *skip;
}

// Eight elements from place `at` (a multiple of 8), as they lie in memory; places outside
// [skip, end) are -inf.
template <typename T>
__device__ __forceinline__ Raw<T> load8(const T* base, int at, int skip, int end) {
  Raw<T> v;
  if (at >= skip && at + 8 <= end) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) v.w[i] = dev::ld_nc_na_v4(base + at + i * (16 / sizeof(T)));
  } else {
    T* t = reinterpret_cast<T*>(&v);
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = at + e >= skip && at + e < end ? base[at + e] : lowest(T());
  }
  return v;
}
// The same for the 16 bytes from place `at`, which is not below `skip`.
template <typename T>
__device__ __forceinline__ uint4 load16(const T* base, int at, int end) {
  constexpr int kN = 16 / sizeof(T);
  if (at + kN <= end) return dev::ld_nc_na_v4(base + at);
  uint4 v;
  T* t = reinterpret_cast<T*>(&v);
#pragma unroll
  for (int e = 0; e < kN; ++e) t[e] = at + e < end ? base[at + e] : lowest(T());
  return v;
}

// A warp's chunk of a row: tokens [kChunk chunk, kChunk (chunk + 1)), 256 j + 8 lane + (0 .. 7) of them in
// vector j of a lane.  Chunks and lanes count tokens and not places, so that a row's sum is the same, to
// the last bit, wherever the row begins, and beams that are alike tie.  Vectors are loaded from places, and
// move down by `skip` elements once they are there (to_tokens): the first ones of the next lane follow a
// lane's own, and lane 0 holds the 16 bytes behind the chunk for the last one.
// kAny: rows may begin off the boundaries (32 x 8 beams over 151,935 tokens 26.8 us; grouped by places and
// without moving, 22.0).  Where none does there is nothing to move (151,936 tokens 21.7; with the registers
// that moving takes 22.8 to 24.7).
constexpr int kVec = kChunk / 256;
template <typename T, bool kAny>
struct Loaded {
  Raw<T> v[kVec];
  uint4 behind;
  int skip;
};
template <typename T>
struct Loaded<T, false> {
  Raw<T> v[kVec];
};
template <typename T, bool kAny>
__device__ __forceinline__ void load_chunk(const BeamArgs& a, int row, int chunk, Loaded<T, kAny>* x) {
  const int lane = threadIdx.x & 31, at = chunk * kChunk + lane * 8;
  int skip = 0;
  const T* base = static_cast<const T*>(a.logits) + row * a.row_stride;
  if constexpr (kAny) {
    base = row_base<T>(a, row, &skip);
    x->skip = skip;
  }
  const int end = skip + a.vocab;
#pragma unroll
  for (int j = 0; j < kVec; ++j) x->v[j] = load8(base, at + j * 256, skip, end);
  if constexpr (kAny) {
    if (skip > 0 && lane == 0) x->behind = load16(base, at + kChunk, end);
  }
}
template <typename T>
__device__ __forceinline__ void to_tokens(Loaded<T, false>*) {}
template <typename T>
__device__ __forceinline__ void to_tokens(Loaded<T, true>* x) {
  constexpr int kOwn = static_cast<int>(sizeof(T)) * 2;   // words of eight elements
  constexpr int kMore = sizeof(T) == 2 ? 4 : 3;           // words of the next eight that may be needed
  const int lane = threadIdx.x & 31, skip = x->skip;
  if (skip == 0) return;  // as one: a warp has one row
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    uint32_t w[kOwn + kMore + 1];
    uint32_t* own = reinterpret_cast<uint32_t*>(&x->v[j]);
    const uint32_t* after = j + 1 < kVec ? reinterpret_cast<const uint32_t*>(&x->v[j + 1 < kVec ? j + 1 : j])
                                         : reinterpret_cast<const uint32_t*>(&x->behind);
#pragma unroll
    for (int i = 0; i < kOwn; ++i) w[i] = own[i];
#pragma unroll
    for (int i = 0; i < kMore; ++i) w[kOwn + i] = __shfl_sync(~0u, lane == 0 ? after[i] : own[i], (lane + 1) & 31);
    w[kOwn + kMore] = 0;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < kOwn + kMore; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], skip % 2 * 16);
    }
    const int words = skip * static_cast<int>(sizeof(T)) / 4;  // 0 to 3
#pragma unroll
    for (int i = 0; i + 1 < kOwn + kMore; ++i) w[i] = words & 1 ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) own[i] = words & 2 ? w[i + 2] : w[i];
  }
}

// Largest of eight elements and `m`, a number where there is one among them.
__device__ __forceinline__ float max8(const Raw<__nv_bfloat16>& r) {
  const __nv_bfloat162* x = reinterpret_cast<const __nv_bfloat162*>(&r);
  const __nv_bfloat162 m = __hmax2(__hmax2(x[0], x[1]), __hmax2(x[2], x[3]));
  return fmaxf(__low2float(m), __high2float(m));
}
__device__ __forceinline__ float max8(const Raw<__half>& r) {
  const __half2* x = reinterpret_cast<const __half2*>(&r);
  const __half2 m = __hmax2(__hmax2(x[0], x[1]), __hmax2(x[2], x[3]));
  return fmaxf(__low2float(m), __high2float(m));
}
__device__ __forceinline__ float max8(const Raw<float>& r) {
  const float* x = reinterpret_cast<const float*>(&r);
  float m = x[0];
#pragma unroll
  for (int e = 1; e < 8; ++e) m = fmaxf(m, x[e]);
  return m;
}

// A bit for each of eight elements that are at least `least`, as numbers that `tame` leaves.
template <typename T>
__device__ __forceinline__ uint32_t reaching(const Raw<T>& r, float least) {
  uint64_t x[4];
  unpack(r, x);
  uint32_t bits = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = dev::split(x[e]);
    if (f.x >= least) bits |= 1u << (2 * e);
    if (f.y >= least) bits |= 2u << (2 * e);
  }
  return bits;
}
// Element `at` of several vectors of eight, by choices between registers.
template <typename T, int kN>
__device__ __forceinline__ float element(const Raw<T> (&r)[kN], int at) {
  constexpr int kWords = kN * static_cast<int>(sizeof(T)) * 2;
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
  const int word = at * static_cast<int>(sizeof(T)) / 4;
  uint32_t v = w[0];
#pragma unroll
  for (int i = 1; i < kWords; ++i) v = i == word ? w[i] : v;
  if constexpr (sizeof(T) == 4) {
    return __uint_as_float(v);
  } else {
    const uint16_t half = static_cast<uint16_t>(at % 2 ? v >> 16 : v);
    return to_f(*reinterpret_cast<const T*>(&half));
  }
}

// A warp goes from chunk to chunk and loads the next one before it works on its own.
// exp(x - m) is 2^(x L - fl(m L)) with L = log2(e) in fp32: one multiply-add; what the
// rounding of m L puts into every term alike is taken out of the sum.
template <typename T, bool kAny>
__global__ void __launch_bounds__(kScanThreads) beam_scan_kernel(const __grid_constant__ BeamArgs a) {
  dev::grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int rows = a.groups * a.beams, stride = gridDim.x * (kScanThreads / 32);
  const int step_rows = stride / a.n_chunks, step_chunks = stride - step_rows * a.n_chunks;
  Loaded<T, kAny> next;
  const int first = blockIdx.x * (kScanThreads / 32) + (threadIdx.x >> 5);
  int row = first / a.n_chunks, chunk = first - row * a.n_chunks;
  const auto load = [&]() {
    if (a.done && a.done[row]) return false;
    load_chunk(a, row, chunk, &next);
    return true;
  };
  bool live = row < rows && load();
  while (row < rows) {
    Loaded<T, kAny> now = next;
    const auto& raw = now.v;
    const bool mine = live;
    const int64_t at = static_cast<int64_t>(row) * a.n_chunks + chunk;
    row += step_rows, chunk += step_chunks;
    if (chunk >= a.n_chunks) chunk -= a.n_chunks, ++row;
    live = row < rows && load();
    if (!mine) continue;
    to_tokens(&now);
    float m = -INFINITY;  // fmaxf takes the number where the other is a NaN
#pragma unroll
    for (int j = 0; j < kVec; ++j) m = fmaxf(m, max8(raw[j]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    m = fminf(m, 3.402823466e38f);
    const float scaled = m * kLog2e;
    uint64_t sums[kVec];
    const uint64_t scale2 = dev::pair(kLog2e, kLog2e), minus2 = dev::pair(-scaled, -scaled);
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      uint64_t x[4];
      unpack(raw[j], x);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 y = dev::split(dev::fma2(x[e], scale2, minus2));
        const uint64_t z = dev::pair(ex2(y.x), ex2(y.y));
        sums[j] = e == 0 ? z : dev::add2(sums[j], z);
      }
    }
#pragma unroll
    for (int j = 1; j < kVec; ++j) sums[0] = dev::add2(sums[0], sums[j]);
    float s = dev::split(sums[0]).x + dev::split(sums[0]).y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    s *= ex2(-fmaf(m, kLog2e, -scaled));
    if (!(s <= 3.402823466e38f)) {  // a NaN or an infinity among them, or nothing above -inf
      s = 0.f;
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const T* x = reinterpret_cast<const T*>(&raw[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float v = tame(to_f(x[e]));
          if (v > -INFINITY) s += ex2((v - m) * kLog2e);
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    }
    if (lane == 0) a.tops[at] = m, a.sums[at] = s;
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

// n + 1 if a is before b, else n: key and index as one number of 96 bits, b less a.
__device__ __forceinline__ int count_before(int n, Candidate a, Candidate b) {
  int next;
  asm("{\n\t.reg .u32 al, ah, bl, bh, t;\n\t"
      "mov.b64 {al, ah}, %1;\n\tmov.b64 {bl, bh}, %2;\n\t"
      "sub.cc.u32 t, %3, %4;\n\t"  // the lower index is the larger number
      "subc.cc.u32 t, bl, al;\n\t"
      "subc.cc.u32 t, bh, ah;\n\t"
      "subc.u32 t, 0, 0;\n\t"  // -1 where that borrowed
      "sub.s32 %0, %5, t;\n\t}\n"
      : "=r"(next)
      : "l"(a.key), "l"(b.key), "r"(a.index), "r"(b.index), "r"(n));
  return next;
}

constexpr int kTops = 4096;  // chunk maxima that are kept in shared memory

struct PickShared {
  double c[kMostBeams];  // a candidate is worth (x - m) + c
  float c32[kMostBeams], m[kMostBeams];
  uint8_t done[kMostBeams];
  float leader[kLeaders];
  int chunks[kList];
  Candidate list[kList], chosen[kMostSelect], next[kPickThreads / 32];
  int n_chunks;  // that pass; `chunks` has the first kList
  int count;     // of listed candidates.  A counter of its own: slow warps still read the other one
  int n_chosen;
  float sieve;
  float tops[kTops];
};

__device__ __forceinline__ void note(PickShared& s, const Candidate& c) {
  const int at = atomicAdd(&s.count, 1);
  if (at < kList) s.list[at] = c;
}

// The `want` first of the listed candidates, if the list holds them all; a warp for each
// of them counts those before it.  256 of the others wait in its lanes' registers instead of
// being read anew for each.  Candidates worth
// -inf are left out.
__device__ bool rank(PickShared& s, int want) {
  constexpr int kHeld = 8;
  const int count = s.count, lane = threadIdx.x % 32;
  if (count > kList) return false;
  int* const places = s.chunks;  // no longer needed; one warp's each
  for (int j0 = 0; j0 < count; j0 += 32 * kHeld) {
    Candidate other[kHeld];
#pragma unroll
    for (int e = 0; e < kHeld; ++e) {
      const int j = j0 + 32 * e + lane;
      other[e] = j < count ? s.list[j] : Candidate{0, 0x7FFFFFFF};  // before none
    }
    for (int i = threadIdx.x / 32; i < count; i += kPickThreads / 32) {
      const Candidate mine = s.list[i];
      int n = 0;
#pragma unroll
      for (int e = 0; e < kHeld; ++e) {
        if (e > 0 && 32 * e >= count - j0) break;
        n = count_before(n, other[e], mine);
      }
      n = __reduce_add_sync(~0u, n);
      if (lane > 0) continue;
      if (j0 > 0) n += places[i];
      if (j0 + 32 * kHeld < count) {
        places[i] = n;
      } else if (n < want && mine.key > kNothing) {
        s.chosen[n] = mine;
        atomicAdd(&s.n_chosen, 1);
      }
    }
    __syncwarp();
  }
  __syncthreads();
  return true;
}

// The same where many candidates are near the border (rows that are alike): one at a time.
// item(i, &c): whether item i passes the sieve, and its candidate.
template <typename Item>
__device__ void one_by_one(PickShared& s, int n, int want, const Item& item) {
  const int tid = threadIdx.x;
  Candidate last{~0ull, -1};
  for (int k = 0; k < want; ++k) {
    Candidate mine{0, 0x7FFFFFFF};
#pragma unroll 1
    for (int i = tid; i < n; i += kPickThreads) {
      Candidate c;
      if (item(i, &c) && before(last, c) && before(c, mine)) mine = c;
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

// A lower bound of the want-th best of a stream of which each thread has seen a part; `m`
// is the best of that part, from below.  The best of 128 or 256 subsets, neighbouring lanes'
// parts, are ranked, so neighbours should have seen things that have little to do with one
// another.
__device__ float bound_of(PickShared& s, float m, int want) {
  const int tid = threadIdx.x;
  const int shift = want > 32 ? 2 : 3, leaders = kPickThreads >> shift, share = 1 << shift;
  for (int o = 1; o < share; o <<= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
  const int me = tid >> shift;
  if ((tid & (share - 1)) == 0) s.leader[me] = m;
  __syncthreads();
  // `share` threads count for a leader, a part of the others each
  int above = 0;
#pragma unroll 8
  for (int i = tid & (share - 1); i < leaders; i += share) above += s.leader[i] > m || (s.leader[i] == m && i < me);
  for (int o = 1; o < share; o <<= 1) above += __shfl_xor_sync(~0u, above, o);
  if (above == want - 1) s.sieve = m;
  __syncthreads();
  return s.sieve;
}

// log(y) of an fp32 y > 0: the exponent's share in a double, the fraction's in fp32.
__device__ __forceinline__ double log_of(float y) {
  int e;
  float f = frexpf(y, &e);  // in [0.5, 1)
  if (f < 0.70710678f) f *= 2.f, --e;
  return fma(static_cast<double>(e), 0.693147180559945309417, static_cast<double>(logf(f)));
}

template <typename T, bool kAny>
__global__ void __launch_bounds__(kPickThreads) beam_pick_kernel(const __grid_constant__ BeamArgs a) {
  __shared__ PickShared s;
  const int entry = blockIdx.x, tid = threadIdx.x, lane = tid % 32;
  const int row0 = entry * a.beams;
  const int N = a.n_chunks, n_tops = a.beams * N;
  if (tid == 0) s.n_chunks = s.count = s.n_chosen = 0;
  dev::grid_dep_wait();
  const float* all_tops = a.tops + static_cast<int64_t>(row0) * N;
  const bool fits = n_tops <= kTops;
  // what a beam's logits have to be raised by: a warp for each beam
  for (int b = tid / 32; b < a.beams; b += kPickThreads / 32) {
    const int row = row0 + b;
    const bool done = a.done && a.done[row];
    const float score = tame(a.scores[row]);
    const float* tops = all_tops + b * N;
    const float* sums = a.sums + static_cast<int64_t>(row) * N;
    float m = -INFINITY, y = 0.f;
    for (int c0 = 0; c0 < N; c0 += 256) {
      float top[8], sum[8], t = m;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int c = c0 + 32 * k + lane;
        const bool in = c < N && !done;
        top[k] = in ? tops[c] : -INFINITY;
        sum[k] = in ? sums[c] : 0.f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int c = c0 + 32 * k + lane;
        t = fmaxf(t, top[k]);
        // a finished beam is one chunk of one candidate, its pad token
        if (fits && c < N) s.tops[b * N + c] = done && c == 0 ? 0.f : top[k];
      }
      if (t > -INFINITY) {
        y *= ex2((m - t) * kLog2e);
#pragma unroll
        for (int k = 0; k < 8; ++k) y = fmaf(sum[k], ex2((top[k] - t) * kLog2e), y);
        m = t;
      }
    }
    float t = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t = fmaxf(t, __shfl_xor_sync(~0u, t, o));
    y = m > -INFINITY ? y * ex2((m - t) * kLog2e) : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) y += __shfl_xor_sync(~0u, y, o);
    if (lane == 0) {
      double c = static_cast<double>(score);
      if (!done) c = y > 0.f ? c - log_of(y) : -INFINITY;
      s.m[b] = t > -INFINITY ? t : 0.f;
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
  const uint32_t per = 0xFFFFFFFFu / static_cast<uint32_t>(N);
  const auto beam_of = [&](int i) {  // i / N
    const int q = static_cast<int>(__umulhi(static_cast<uint32_t>(i), per));
    return q + ((q + 1) * static_cast<int64_t>(N) <= i) + ((q + 2) * static_cast<int64_t>(N) <= i);
  };
  const auto passes = [&](int b, float x, float sieve) {
    float err;
    const float r = sum32(b, x, &err);
    return r > -INFINITY && r + err >= sieve;
  };
  const auto chunk_top = [&](int i, int b) {
    return fits ? s.tops[i] : s.done[b] ? (i == b * N ? 0.f : -INFINITY) : all_tops[i];
  };

  // ---- the chunks that may hold one of the `want` best: those whose leaders pass a sieve that
  // `want` leaders pass.  Lanes that share a leader look at chunks 128 or 256 apart: a beam's own
  // chunks, which may all be good, then count apart.
  const int want = a.n_select, mixed = want > 32 ? (tid & 3) << 8 | tid >> 2 : (tid & 7) << 7 | tid >> 3;
  float sieve = -INFINITY;
  // Few chunks may all: their bound would be one that too many candidates pass.  (8 entries, tops and
  // n_select: 32 and 16 9.3 us, with a sieve 18.2; 128 and 16 9.5, without one 14.8; but 64 and 8 10.9, with one 8.3.)
  if (n_tops > 64) {
    float best = -INFINITY;
    for (int i = mixed; i < n_tops; i += kPickThreads) {
      float err;
      const int b = beam_of(i);
      const float r = sum32(b, chunk_top(i, b), &err);
      best = fmaxf(best, r - err);
    }
    sieve = bound_of(s, best, want);
  }
  const auto chunk = [&](int i, Candidate* c) {
    const int b = beam_of(i);
    const float x = chunk_top(i, b);
    if (!passes(b, x, sieve)) return false;
    *c = Candidate{worth(b, x), i};
    return true;
  };
  for (int i = tid; i < n_tops; i += kPickThreads) {
    const int b = beam_of(i);
    if (passes(b, chunk_top(i, b), sieve)) {
      const int at = atomicAdd(&s.n_chunks, 1);
      if (at < kList) s.chunks[at] = i;
    }
  }
  __syncthreads();
  int n_chosen = s.n_chunks;
  if (n_chosen > kList) {  // chunks that are alike: the `want` best, whose last one's leader is a sieve too
    one_by_one(s, n_tops, want, chunk);
    n_chosen = s.n_chosen;
    if (tid < n_chosen) s.chunks[tid] = s.chosen[tid].index;
    if (n_chosen == want) sieve = fmaxf(sieve, __double2float_rd(unordered(s.chosen[want - 1].key)));
    __syncthreads();  // all have read the number that are chosen
    if (tid == 0) s.n_chosen = 0;
    __syncthreads();
  }

  // ---- the candidates of those chunks, a warp for each; an index is beam * vocab + token.
  // What passes the chunks' sieve is listed.  Where that is too much (one beam far ahead of the
  // others) or there is no such sieve, the candidates themselves give one.
  const auto load = [&](int b, int g, Loaded<T, kAny>* x) {  // this lane's first token
    load_chunk(a, row0 + b, g - b * N, x);
    to_tokens(x);
    return (g - b * N) * kChunk + lane * 8;
  };
  for (int turn = sieve == -INFINITY; turn < 2; ++turn) {
    if (turn == 1) {
      float best = -INFINITY;
      for (int k = tid / 32; k < n_chosen; k += kPickThreads / 32) {
        const int g = s.chunks[k], b = g / N;
        float top = s.done[b] && lane == 0 ? 0.f : -INFINITY;
        if (!s.done[b]) {
          Loaded<T, kAny> x;
          load(b, g, &x);
#pragma unroll
          for (int j = 0; j < kVec; ++j) top = fmaxf(top, max8(x.v[j]));
          top = fminf(top, 3.402823466e38f);
        }
        float err;
        const float r = sum32(b, top, &err);
        best = fmaxf(best, r - err);
      }
      sieve = fmaxf(sieve, bound_of(s, best, want));
      if (tid == 0) s.count = 0;
      __syncthreads();
    }
    for (int k = tid / 32; k < n_chosen; k += kPickThreads / 32) {
      const int g = s.chunks[k], b = g / N;
      if (s.done[b]) {
        if (lane == 0) note(s, Candidate{worth(b, 0.f), b * a.vocab + a.pad});
        continue;
      }
      Loaded<T, kAny> x;
      const int token = load(b, g, &x);
      // what a logit has to reach, from below
      const float least = sieve > -INFINITY ? s.m[b] + (sieve - s.c32[b]) - (fabsf(s.m[b]) + fabsf(sieve) + fabsf(s.c32[b])) * 0x1p-21f
                                            : -3.402823466e38f;
      // a bit for each element that does; the lanes then take one of theirs at a time (128 best of 8
      // beams: 38.7 us; all eight elements of such vectors one by one, indexed in local memory, and
      // ranks by 64-bit comparisons of candidates in shared memory 58.5)
      uint32_t good = 0;
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (max8(x.v[j]) >= least) good |= reaching(x.v[j], least) << (8 * j);
      while (good) {
        const int at = __ffs(good) - 1;
        good &= good - 1;
        const float f = tame(element(x.v, at));
        if (passes(b, f, sieve)) note(s, Candidate{worth(b, f), b * a.vocab + token + 256 * (at / 8) + at % 8});
      }
    }
    __syncthreads();
    if (s.count <= kList) break;
  }
  if (!rank(s, want))
    one_by_one(s, n_chosen * kChunk, want, [&](int i, Candidate* c) {
      const int g = s.chunks[i / kChunk], b = g / N, e = i % kChunk;
      float f = e == 0 ? 0.f : -INFINITY;
      int token = a.pad;
      if (!s.done[b]) {
        token = (g - b * N) * kChunk + e;
        const T* x = static_cast<const T*>(a.logits) + (row0 + b) * a.row_stride;
        f = token < a.vocab ? tame(to_f(x[token])) : -INFINITY;
      }
      if (!passes(b, f, sieve)) return false;
      *c = Candidate{worth(b, f), b * a.vocab + token};
      return true;
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

template <typename T, bool kAny>
cudaError_t launch_rows(const BeamArgs& a, int sms, cudaStream_t s) {
  // Four CTAs an SM, which bf16 has at the same time (fp32 two: 64 x 5 beams 20.7 us, with three 21.9); three
  // where 16-bit rows are moved, which is what their registers allow (26.8 us, with four 28.6).
  const int64_t chunks = static_cast<int64_t>(a.groups) * a.beams * a.n_chunks;
  const int ctas = static_cast<int>(std::min<int64_t>((chunks + 7) / 8, (kAny && sizeof(T) == 2 ? 3ll : 4ll) * sms));
  beam_scan_kernel<T, kAny><<<ctas, kScanThreads, 0, s>>>(a);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.groups);
  cfg.blockDim = dim3(kPickThreads);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, beam_pick_kernel<T, kAny>, a);
  const cudaError_t last = cudaGetLastError();
  return e != cudaSuccess ? e : last;
}
template <typename T>
cudaError_t launch(const BeamArgs& a, int sms, cudaStream_t s) {
  const uint64_t at = reinterpret_cast<uintptr_t>(a.logits) | static_cast<uint64_t>(a.row_stride) * sizeof(T);
  return at % 16 == 0 ? launch_rows<T, false>(a, sms, s) : launch_rows<T, true>(a, sms, s);
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

// One CTA a (layer, child): the row of the table, and the page that is partly filled.  Few CTAs
// have kPer = 8 vectors a thread in flight, a page of 32 KiB at once (one layer of 4 beams 2.7 us,
// with 4 vectors 3.3); many share the SMs better with 4 (48 layers of 32 beams 11.2 us, 11.7 with 8).
template <int kPer>
__global__ void __launch_bounds__(kReorderThreads, kPer == 4 ? 8 : 4) kv_reorder_kernel(const __grid_constant__ ReorderArgs a) {
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
int64_t row_chunks(int vocab) { return (static_cast<int64_t>(vocab) + rimuru::kChunk - 1) / rimuru::kChunk; }
}  // namespace

extern "C" uint64_t rimuru_beam_select_workspace_bytes(int num_groups, int beams, int vocab, int n_select) {
  if (num_groups < 0 || beams <= 0 || vocab <= 0 || n_select <= 0) return 0;
  const uint64_t rows = static_cast<uint64_t>(num_groups) * beams;
  return 2 * rows * row_chunks(vocab) * sizeof(float) + 1024;
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
  if (static_cast<int64_t>(beams) * (logits->cols + 2ll * kChunk) > (1 << 30) ||
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
  // an entry reads its scores before it writes, but not before another entry does
  const uintptr_t s0 = reinterpret_cast<uintptr_t>(scores), o0 = reinterpret_cast<uintptr_t>(out_scores);
  const uintptr_t entries = static_cast<uintptr_t>(num_groups) * sizeof(float);
  if (o0 < s0 + entries * beams && s0 < o0 + entries * n_select && !(o0 == s0 && n_select == beams))
    return fail(RIMURU_ERR_ARG, "out_scores may lie on the scores only where n_select is the number of beams");
  BeamArgs a{};
  a.logits = logits->data;
  a.row_stride = logits->row_stride;
  a.vocab = logits->cols;
  a.scores = scores;
  a.done = done;
  a.groups = num_groups, a.beams = beams, a.pad = pad_token, a.n_select = n_select;
  a.best = out_scores, a.rows = out_rows, a.tokens = out_tokens;
  a.n_chunks = static_cast<int>(row_chunks(logits->cols));
  const int64_t chunks = static_cast<int64_t>(num_groups) * beams * a.n_chunks;
  a.tops = static_cast<float*>(workspace);
  a.sums = a.tops + chunks;
  int sms = 0, device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
  if (e != cudaSuccess) return fail(RIMURU_ERR_CUDA, kv_cuda_msg("device attributes", e));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  e = logits->dtype == RIMURU_BF16  ? launch<__nv_bfloat16>(a, sms, s)
      : logits->dtype == RIMURU_F16 ? launch<__half>(a, sms, s)
                                    : launch<float>(a, sms, s);
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
  const dim3 grid(num_seqs, num_layers);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (static_cast<int64_t>(num_seqs) * num_layers <= 4ll * v.kv->sms) kv_reorder_kernel<8><<<grid, kReorderThreads, 0, s>>>(a);
  else kv_reorder_kernel<4><<<grid, kReorderThreads, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(RIMURU_ERR_CUDA, kv_cuda_msg("reordering launch", e));
  return RIMURU_OK;
}
