// Norms of heads and their rotation in one pass: a head x of a token becomes
// rot_p(x * r * (w + offset)) with r = 1 / sqrt(mean(x^2) + eps).
//
// Each element is read and written once; a head stays in the registers of the lanes
// that loaded it.  A group of 2^n lanes takes some heads of one token: a lane holds two
// vectors of eight elements of a head (in the half layout the two members of eight pairs,
// so that pairs turn within a lane), and the squares are added up over the group by
// shuffles.  A CTA computes its tokens' cosines and sines once, for all heads.
//
// 8192 tokens, 18 heads of 256 of which 64 elements turn (151 MB): 31.7 us, 0.70 of the copy
// rate; the rotation alone takes 30.4.  Bound by instructions and latency together: a group
// that computed its own angles, with all its values in fp32 registers, took 96 us; values as they
// were loaded 55; shared angles, packed products and the next heads loaded ahead 39; fewer
// groups with more heads each 31.8.  One token of 36 heads of 128: 3.7 us.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "device.cuh"
#include "kv.h"
#include "rope.h"

namespace rimuru {
namespace {

constexpr int kMaxArrays = 4;
constexpr int kThreads = 256;

struct NormArray {
  const void* in;
  void* out;
  int64_t in_ts, in_hs, out_ts, out_hs;  // strides in elements
  const void* weight;                    // or null: ones
  int weight_dtype;
  float eps, offset;
};

struct NormArgs {
  RopeTurns rope;
  NormArray arr[kMaxArrays];
  int first_head[kMaxArrays + 1];  // heads of the arrays before this one
  const int32_t* positions;
  int num_tokens, head_dim;
  int lanes_log2;         // of a group
  int heads_per_group;
  int groups, groups_mul; // groups of a token in a CTA; g / groups = g * groups_mul >> 16
  int tokens;             // of a CTA
  int turn_slots, slots;  // of a head: slots whose vectors are a pair's members, and all
};

using dev::fma2;
using dev::mul2;
using dev::pair;
using dev::split;

template <typename T>
struct Raw {  // eight elements as they lie in memory
  uint4 w[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* p) {
  Raw<T> v;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) v.w[i] = reinterpret_cast<const uint4*>(p)[i];
  return v;
}
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16>& r, uint64_t (&x)[4]) {
  const uint32_t v[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = pair(__uint_as_float(v[i] << 16), __uint_as_float(v[i] & 0xFFFF0000u));
}
__device__ __forceinline__ void unpack(const Raw<__half>& r, uint64_t (&x)[4]) {
  const uint32_t v[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v[i]));
    x[i] = pair(f.x, f.y);
  }
}
__device__ __forceinline__ void unpack(const Raw<float>& r, uint64_t (&x)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[2 * i] = pair(__uint_as_float(r.w[i].x), __uint_as_float(r.w[i].y));
    x[2 * i + 1] = pair(__uint_as_float(r.w[i].z), __uint_as_float(r.w[i].w));
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const uint64_t (&x)[4]) {
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = dev::pack_bf16x2(split(x[i]).x, split(x[i]).y);
  *reinterpret_cast<uint4*>(p) = make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store8(__half* p, const uint64_t (&x)[4]) {
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(split(x[i]).x, split(x[i]).y);
    v[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store8(float* p, const uint64_t (&x)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 a = split(x[2 * i]), b = split(x[2 * i + 1]);
    reinterpret_cast<float4*>(p)[i] = make_float4(a.x, a.y, b.x, b.y);
  }
}

// Offsets of a slot's two vectors in a head, -1 where there is none.  Slots below
// turn_slots hold both members of eight pairs (half layout); the vectors that are left
// are shared out so that neighbouring lanes hold neighbouring vectors.
template <bool kHalf>
__device__ __forceinline__ void place(const NormArgs& p, int slot, int (&off)[2]) {
  off[0] = off[1] = -1;
  if (slot >= p.slots) return;
  if (kHalf && slot < p.turn_slots) {
    off[0] = 8 * slot;
    off[1] = 8 * slot + p.rope.pairs;
    return;
  }
  const int first = kHalf ? 16 * p.turn_slots : 0, rest = p.slots - (kHalf ? p.turn_slots : 0);
  off[0] = first + 8 * (slot - (kHalf ? p.turn_slots : 0));
  off[1] = off[0] + 8 * rest;
  if (off[1] >= p.head_dim) off[1] = -1;
}

// A group's place among the heads of the arrays.
template <typename T>
struct Cursor {
  T* at;       // the head's first element
  int64_t hs;
  int left, i; // heads left of array i
};
template <bool kOut, typename T>
__device__ __forceinline__ void begin(const NormArgs& p, Cursor<T>* c, unsigned t, int h) {
  int i = 0;
#pragma unroll
  for (int k = 1; k < kMaxArrays; ++k) i += h >= p.first_head[k];
  const NormArray& A = p.arr[i];
  c->i = i;
  c->left = p.first_head[i + 1] - h;
  c->hs = kOut ? A.out_hs : A.in_hs;
  c->at = static_cast<T*>(kOut ? A.out : const_cast<void*>(A.in)) + static_cast<int64_t>(t) * (kOut ? A.out_ts : A.in_ts) +
          (h - p.first_head[i]) * c->hs;
}
template <bool kOut, typename T>
__device__ __forceinline__ void step(const NormArgs& p, Cursor<T>* c, unsigned t) {
  c->at += c->hs;
  if (--c->left == 0 && c->i + 1 < kMaxArrays) begin<kOut>(p, c, t, p.first_head[c->i + 1]);
}

// kSlots: slots of a lane; kFull: every lane has both vectors of each of its slots.  Heads
// wait as they were loaded and are unpacked twice, for the sum and for the result: half the
// registers for 16-bit types.  The next kRows heads are loaded before these are worked on.
template <typename T, bool kHalf, int kSlots, bool kFull>
__global__ void __launch_bounds__(kThreads, 2)
    norm_rope_kernel(const __grid_constant__ NormArgs p) {
  constexpr int kRows = kSlots == 1 ? 2 : 1;
  extern __shared__ float4 dynamic[];
  float* const weights = reinterpret_cast<float*>(dynamic);  // [arrays][head_dim], the offset added, ones without a weight
  float2* const cosines = reinterpret_cast<float2*>(weights + kMaxArrays * p.head_dim);  // [tokens of the CTA][pairs]
  const int lanes = 1 << p.lanes_log2, lane = threadIdx.x & (lanes - 1);
  const int g = threadIdx.x >> p.lanes_log2, u = g * p.groups_mul >> 16;
  const unsigned t0 = blockIdx.x * p.tokens, t = t0 + u, num_tokens = p.num_tokens;
  const int h0 = (blockIdx.y * p.groups + g - u * p.groups) * p.heads_per_group;
  // groups past the last token or head stay for the shuffles and take none
  const int heads = u < p.tokens && t < num_tokens ? min(p.heads_per_group, p.first_head[kMaxArrays] - h0) : 0;
  const int pairs = p.rope.pairs, rot = 2 * pairs;
  int off[kSlots][2];
#pragma unroll
  for (int s = 0; s < kSlots; ++s) place<kHalf>(p, lane + s * lanes, off[s]);

  Raw<T> next[kRows][kSlots][2];
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int s = 0; s < kSlots; ++s)
#pragma unroll
      for (int v = 0; v < 2; ++v) next[r][s][v] = Raw<T>{};
  Cursor<T> in{}, out{};
  if (heads > 0) {
    begin<false>(p, &in, t, h0);
    begin<true>(p, &out, t, h0);
  }
  const auto load = [&](int h) {
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      if (h + r < heads) {
#pragma unroll
        for (int s = 0; s < kSlots; ++s)
#pragma unroll
          for (int v = 0; v < 2; ++v)
            if (kFull || off[s][v] >= 0) next[r][s][v] = load_raw(in.at + off[s][v]);
        step<false>(p, &in, t);
      }
  };
  load(0);
  if (rot > 0) {
    const int n = min(static_cast<unsigned>(p.tokens), num_tokens - t0);
    for (int k = threadIdx.x; k < n * pairs; k += blockDim.x) {
      const int w = k / pairs, i = k - w * pairs;
      const uint64_t pos = static_cast<uint64_t>(static_cast<int64_t>(p.positions[t0 + w]));
      float sn, c;
      sincospif(__ll2float_rn(static_cast<int64_t>(pos * p.rope.turn[i])) * 0x1p-63f, &sn, &c);
      cosines[k] = make_float2(c * p.rope.mscale, sn * p.rope.mscale);
    }
  }
  for (int i = 0; i < kMaxArrays; ++i) {
    const NormArray& A = p.arr[i];
    if (p.first_head[i] == p.first_head[i + 1]) continue;
    for (int d = threadIdx.x; d < p.head_dim; d += blockDim.x) {
      const float w = !A.weight                        ? 1.f
                      : A.weight_dtype == RIMURU_BF16  ? __bfloat162float(static_cast<const __nv_bfloat16*>(A.weight)[d])
                      : A.weight_dtype == RIMURU_F16 ? __half2float(static_cast<const __half*>(A.weight)[d])
                                                     : static_cast<const float*>(A.weight)[d];
      weights[i * p.head_dim + d] = A.weight ? w + A.offset : w;
    }
  }
  __syncthreads();

  // of the slot's eight pairs: elements (e, e) of its two vectors, or (2 e, 2 e + 1) of one
  uint64_t cs[kSlots][4], sn[kSlots][4];
#pragma unroll
  for (int s = 0; s < kSlots; ++s)
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const int at = kHalf ? (off[s][0] >= 0 && off[s][0] < rot ? off[s][0] + e : -1)
                           : (off[s][e / 4] >= 0 && off[s][e / 4] < rot ? off[s][e / 4] / 2 + e % 4 : -1);
      const float2* w = cosines + u * pairs + at;
      const float2 w0 = at >= 0 && heads > 0 ? w[0] : make_float2(1.f, 0.f), w1 = at >= 0 && heads > 0 ? w[1] : make_float2(1.f, 0.f);
      cs[s][e / 2] = pair(w0.x, w1.x);
      sn[s][e / 2] = pair(w0.y, w1.y);
    }

  const float per_dim = 1.f / p.head_dim;
  const uint64_t minus = pair(-1.f, -1.f);
#pragma unroll 1
  for (int h = 0; h < p.heads_per_group; h += kRows) {  // as often in every group: shuffles take all lanes
    Raw<T> x[kRows][kSlots][2];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int s = 0; s < kSlots; ++s)
#pragma unroll
        for (int v = 0; v < 2; ++v) x[r][s][v] = next[r][s][v];
    load(h + kRows);
    float sum[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      uint64_t acc = 0;
#pragma unroll
      for (int s = 0; s < kSlots; ++s)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          uint64_t y[4];
          unpack(x[r][s][v], y);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc = fma2(y[e], y[e], acc);
        }
      sum[r] = split(acc).x + split(acc).y;
    }
    for (int m = lanes >> 1; m > 0; m >>= 1)
#pragma unroll
      for (int r = 0; r < kRows; ++r) sum[r] += __shfl_xor_sync(~0u, sum[r], m);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      float eps = p.arr[out.i].eps, f = 1.f;
      // squares past fp32: the head is taken 2^-96 times as large, where eps is nothing
      const bool large = !std::is_same<T, __half>::value && isinf(sum[r]);
      if (__any_sync(~0u, large)) {
        float again = 0.f;
#pragma unroll
        for (int s = 0; s < kSlots; ++s)
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            uint64_t y[4];
            unpack(x[r][s][v], y);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 z = split(y[e]);
              again = fmaf(z.x * 0x1p-96f, z.x * 0x1p-96f, again);
              again = fmaf(z.y * 0x1p-96f, z.y * 0x1p-96f, again);
            }
          }
        for (int m = lanes >> 1; m > 0; m >>= 1) again += __shfl_xor_sync(~0u, again, m);
        if (large) sum[r] = again, eps = 0.f, f = 0x1p-96f;
      }
      const float mean = fmaf(sum[r], per_dim, eps);
      float k = rsqrtf(mean);
      if (sizeof(T) == 4) k = isinf(mean) ? 0.f : k * fmaf(-0.5f * mean * k, k, 1.5f);  // to the last bit
      k *= f;
      if (h + r >= heads) continue;
      const uint64_t k2 = pair(k, k);
      const float* weight = weights + out.i * p.head_dim;
#pragma unroll
      for (int s = 0; s < kSlots; ++s) {
        uint64_t y[2][4];
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          unpack(x[r][s][v], y[v]);
          if (kFull || off[s][v] >= 0) {
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(weight + off[s][v] + 2 * e);
              // in this order: k times a weight may leave fp32 where the result does not
              y[v][e] = mul2(mul2(y[v][e], k2), w.x);
              y[v][e + 1] = mul2(mul2(y[v][e + 1], k2), w.y);
            }
          }
        }
        if (kHalf) {
          if (off[s][0] >= 0 && off[s][0] < rot) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint64_t a = y[0][e], b = y[1][e];
              y[0][e] = fma2(mul2(b, sn[s][e]), minus, mul2(a, cs[s][e]));
              y[1][e] = fma2(a, sn[s][e], mul2(b, cs[s][e]));
            }
          }
        } else {
#pragma unroll
          for (int v = 0; v < 2; ++v)
            if (off[s][v] >= 0 && off[s][v] < rot) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 z = split(y[v][e]);
                const float2 c2 = split(cs[s][2 * v + e / 2]), s2 = split(sn[s][2 * v + e / 2]);
                const float c = e % 2 ? c2.y : c2.x, q = e % 2 ? s2.y : s2.x;
                y[v][e] = pair(z.x * c - z.y * q, z.y * c + z.x * q);
              }
            }
        }
#pragma unroll
        for (int v = 0; v < 2; ++v)
          if (kFull || off[s][v] >= 0) store8(out.at + off[s][v], y[v]);
      }
      step<true>(p, &out, t);
    }
  }
}

template <typename T, bool kHalf>
cudaError_t launch_layout(const NormArgs& a, int per_lane, dim3 grid, int block, int smem, cudaStream_t stream) {
  const bool full = a.head_dim == 16 * (per_lane << a.lanes_log2);
  if (per_lane == 1) {
    if (full) norm_rope_kernel<T, kHalf, 1, true><<<grid, block, smem, stream>>>(a);
    else norm_rope_kernel<T, kHalf, 1, false><<<grid, block, smem, stream>>>(a);
  } else {
    if (full) norm_rope_kernel<T, kHalf, 2, true><<<grid, block, smem, stream>>>(a);
    else norm_rope_kernel<T, kHalf, 2, false><<<grid, block, smem, stream>>>(a);
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch(NormArgs a, int per_lane, int heads, int sms, cudaStream_t stream) {
  // A group takes several heads of its token where that leaves 512 threads an SM, else fewer, down
  // to one; more groups pay for the prologue more often (8192 tokens of 18 heads of 256: 31.8 us,
  // 35.8 with 1024 threads; 1000 tokens 8.6 and 9.9).
  const int64_t want = 512ll * sms >> a.lanes_log2;  // groups
  const int64_t per_token = std::max<int64_t>(1, std::min<int64_t>(std::min(heads, 32768), (want + a.num_tokens - 1) / a.num_tokens));
  a.heads_per_group = static_cast<int>((heads + per_token - 1) / per_token);
  const int all = (heads + a.heads_per_group - 1) / a.heads_per_group;  // groups of a token
  // few threads: small CTAs, on many SMs
  const int most = (static_cast<int64_t>(a.num_tokens) * all << a.lanes_log2) < static_cast<int64_t>(sms) * kThreads ? 64 : kThreads;
  const int fit = std::max(1, most >> a.lanes_log2);  // groups of a CTA
  a.groups = std::min(all, fit);
  a.groups_mul = 65536 / a.groups + 1;  // exact for g < 256
  a.tokens = std::max(1, fit / a.groups);
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(a.num_tokens) + a.tokens - 1) / a.tokens), (all + a.groups - 1) / a.groups);
  const int block = (((a.tokens * a.groups) << a.lanes_log2) + 31) / 32 * 32;
  const int smem = kMaxArrays * a.head_dim * static_cast<int>(sizeof(float)) +
                   a.tokens * a.rope.pairs * static_cast<int>(sizeof(float2));
  return a.rope.layout == RIMURU_ROPE_HALF ? launch_layout<T, true>(a, per_lane, grid, block, smem, stream)
                                           : launch_layout<T, false>(a, per_lane, grid, block, smem, stream);
}

}  // namespace
}  // namespace rimuru

using rimuru::fail;

extern "C" int rimuru_norm_rope_apply(rimuru_rope_t rope, const int32_t* positions, int num_tokens,
                                      int head_dim, const rimuru_heads* in, const rimuru_heads* out,
                                      const rimuru_head_norm* norms, int n_arrays, void* stream) {
  using namespace rimuru;
  clear_error();
  if (!in || !out || !norms || n_arrays < 1 || n_arrays > kMaxArrays)
    return fail(RIMURU_ERR_ARG, "between 1 and 4 arrays, each with its norm");
  if (num_tokens < 0) return fail(RIMURU_ERR_ARG, "negative token count");
  NormArgs a{};
  a.rope.layout = RIMURU_ROPE_HALF;
  if (rope) rope_turns(rope, &a.rope);
  const int rot = 2 * a.rope.pairs;
  if (head_dim < std::max(rot, 8) || head_dim % 8 != 0 || head_dim > 1024)
    return fail(RIMURU_ERR_UNSUPPORTED,
                "head_dim must be a multiple of 8, at least rot_dim and at most 1024");
  if (num_tokens == 0) return RIMURU_OK;
  if (rope && !positions) return fail(RIMURU_ERR_ARG, "null positions");
  if (rope && reinterpret_cast<uintptr_t>(positions) % 4 != 0)
    return fail(RIMURU_ERR_ALIGN, "positions must be 4-byte aligned");
  a.positions = positions;
  a.num_tokens = num_tokens;
  a.head_dim = head_dim;
  int64_t heads = 0;
  for (int i = 0; i < n_arrays; ++i) {
    int st = check_heads(&in[i], "norm input");
    if (st == RIMURU_OK) st = check_heads(&out[i], "norm output");
    if (st != RIMURU_OK) return st;
    if (in[i].heads != out[i].heads || in[i].dtype != out[i].dtype || in[i].dtype != in[0].dtype)
      return fail(RIMURU_ERR_ARG, "inputs and outputs must agree in heads and type");
    const rimuru_head_norm& n = norms[i];
    if (!(n.eps >= 1e-20 && n.eps <= 1.0)) return fail(RIMURU_ERR_ARG, "eps must be in [1e-20, 1]");
    if (!std::isfinite(static_cast<float>(n.offset))) return fail(RIMURU_ERR_ARG, "offset must be finite in fp32");
    if (n.weight) {
      if (n.dtype != RIMURU_BF16 && n.dtype != RIMURU_F16 && n.dtype != RIMURU_F32)
        return fail(RIMURU_ERR_ARG, "norm weight: unknown element type");
      if (reinterpret_cast<uintptr_t>(n.weight) % 16 != 0)
        return fail(RIMURU_ERR_ALIGN, "norm weight must be 16-byte aligned");
    }
    a.arr[i] = {in[i].data,         out[i].data,         in[i].token_stride,          in[i].head_stride,
                out[i].token_stride, out[i].head_stride, n.weight, n.dtype, static_cast<float>(n.eps),
                static_cast<float>(n.offset)};
    a.first_head[i] = static_cast<int>(heads);
    heads += in[i].heads;
    if (heads > (1 << 20)) return fail(RIMURU_ERR_UNSUPPORTED, "too many heads");
  }
  for (int i = n_arrays; i <= kMaxArrays; ++i) a.first_head[i] = static_cast<int>(heads);
  const int vectors = head_dim / 8;
  a.turn_slots = a.rope.layout == RIMURU_ROPE_HALF ? a.rope.pairs / 8 : 0;
  a.slots = a.turn_slots + (vectors - 2 * a.turn_slots + 1) / 2;
  while ((1 << a.lanes_log2) < a.slots && a.lanes_log2 < 5) ++a.lanes_log2;
  const int per_lane = a.slots > 32 ? 2 : 1;
  int sms = 0, dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return fail(RIMURU_ERR_CUDA, kv_cuda_msg("device attributes", e));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int n = static_cast<int>(heads);
  e = in[0].dtype == RIMURU_BF16  ? launch<__nv_bfloat16>(a, per_lane, n, sms, s)
      : in[0].dtype == RIMURU_F16 ? launch<__half>(a, per_lane, n, sms, s)
                                  : launch<float>(a, per_lane, n, sms, s);
  if (e != cudaSuccess) return fail(RIMURU_ERR_CUDA, kv_cuda_msg("norm launch", e));
  return RIMURU_OK;
}
