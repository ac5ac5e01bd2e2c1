// Norms of heads and their rotation in one pass: a head x of a token becomes
// rot_p(x * r * (w + offset)) with r = 1 / sqrt(mean(x^2) + eps).
//
// Each element is read and written once; a head stays in the registers of the lanes
// that loaded it.  A group of 2^n lanes takes a run of heads, counted through all tokens: a
// lane holds two vectors of eight elements of a head (in the half layout the two members of
// eight pairs, so that pairs turn within a lane), and the squares are added up over the group
// by shuffles.  A CTA computes its tokens' cosines and sines once, for all heads.
//
// 8192 tokens, 18 heads of 256 of which 64 elements turn (151 MB): 30.0 us, 0.74 of the copy
// rate, 0.84 at 32,768 tokens; the rotation alone takes 30.4.  Bound by instructions and latency
// together: a group that computed its own angles, with all its values in fp32 registers, took
// 96 us; values as they were loaded 55; shared angles, packed products and the next heads loaded
// ahead 39; fewer groups with more heads each 31.8; runs of one length that fill whole rounds
// of CTAs 30.0 (6500 tokens 30.8 -> 25.3, 3000 18.7 -> 14.1).  One token of 36 heads of 128: 3.7 us.
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
constexpr int kLongest = 128;  // heads of a run (32,768 tokens: 105 us; with 24 116, with 64 108)

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
  int run;                // heads of a group, counted through all tokens
  int64_t all_heads;      // of all tokens
  uint32_t heads_mul;     // 2^32 / heads of a token, rounded down
  int turn_slots, slots;  // of a head: slots whose vectors are a pair's members, and all
};

using dev::fma2;
using dev::mul2;
using dev::pair;
using dev::Raw;
using dev::split;
using dev::unpack;

template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* p) {
  Raw<T> v;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) v.w[i] = reinterpret_cast<const uint4*>(p)[i];
  return v;
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
// To the next head; false where that is the first one of the next token.
template <bool kOut, typename T>
__device__ __forceinline__ bool step(const NormArgs& p, Cursor<T>* c, unsigned* t) {
  c->at += c->hs;
  if (--c->left > 0) return true;
  const int h = p.first_head[c->i + 1];
  const bool same = h < p.first_head[kMaxArrays];
  if (!same) ++*t;
  begin<kOut>(p, c, *t, same ? h : 0);
  return same;
}
__device__ __forceinline__ unsigned token_of(const NormArgs& p, int64_t head) {
  const unsigned heads = p.first_head[kMaxArrays];
  if (head >> 32) return static_cast<unsigned>(static_cast<uint64_t>(head) / heads);
  const uint32_t x = static_cast<uint32_t>(head), q = __umulhi(x, p.heads_mul);  // one short at most
  return q + (x - q * heads >= heads);
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
  const int groups = blockDim.x >> p.lanes_log2;  // of the CTA
  const int64_t begin0 = static_cast<int64_t>(blockIdx.x) * groups * p.run, at0 = begin0 + static_cast<int64_t>(threadIdx.x >> p.lanes_log2) * p.run;
  // groups past the last head stay for the shuffles and take none
  int to_load = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(p.run), p.all_heads - at0)));
  const unsigned t0 = token_of(p, begin0);
  unsigned t_in = to_load > 0 ? token_of(p, at0) : t0, t_out = t_in;
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
  if (to_load > 0) {
    const int h = static_cast<int>(at0 - static_cast<int64_t>(t_in) * p.first_head[kMaxArrays]);
    begin<false>(p, &in, t_in, h);
    begin<true>(p, &out, t_out, h);
  }
  // The next heads, kRows of them unless the group's or the token's last comes before.
  const auto load = [&]() {
    int n = 0;
    bool more = true;
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      if (more && to_load > 0) {
#pragma unroll
        for (int s = 0; s < kSlots; ++s)
#pragma unroll
          for (int v = 0; v < 2; ++v)
            if (kFull || off[s][v] >= 0) next[r][s][v] = load_raw(in.at + off[s][v]);
        more = step<false>(p, &in, &t_in);
        --to_load;
        ++n;
      }
    return n;
  };
  int loaded = load();
  if (rot > 0) {
    const int64_t end = min(begin0 + static_cast<int64_t>(groups) * p.run, p.all_heads);
    const int n = static_cast<int>(token_of(p, end - 1) - t0) + 1;
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
  const auto angles = [&]() {
#pragma unroll
    for (int s = 0; s < kSlots; ++s)
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const int at = kHalf ? (off[s][0] >= 0 && off[s][0] < rot ? off[s][0] + e : -1)
                             : (off[s][e / 4] >= 0 && off[s][e / 4] < rot ? off[s][e / 4] / 2 + e % 4 : -1);
        const float2* w = cosines + (t_out - t0) * pairs + at;
        const float2 w0 = at >= 0 ? w[0] : make_float2(1.f, 0.f), w1 = at >= 0 ? w[1] : make_float2(1.f, 0.f);
        cs[s][e / 2] = pair(w0.x, w1.x);
        sn[s][e / 2] = pair(w0.y, w1.y);
      }
  };
  angles();

  const float per_dim = 1.f / p.head_dim;
  const uint64_t minus = pair(-1.f, -1.f);
#pragma unroll 1
  while (__any_sync(~0u, loaded > 0)) {  // as often in every group of a warp: shuffles take all lanes
    const int here = loaded;
    Raw<T> x[kRows][kSlots][2];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int s = 0; s < kSlots; ++s)
#pragma unroll
        for (int v = 0; v < 2; ++v) x[r][s][v] = next[r][s][v];
    loaded = load();
    bool same = true;
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
      if (r >= here) continue;
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
      same = step<true>(p, &out, &t_out);
    }
    if (!same && loaded > 0) angles();  // the next token's
  }
}

template <typename T, bool kHalf>
cudaError_t launch_layout(const NormArgs& a, int per_lane, unsigned grid, int block, int smem, cudaStream_t stream) {
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
  // Groups take equal runs of heads, as long as 512 threads an SM (what their registers allow) make
  // whole rounds of them.
  a.all_heads = static_cast<int64_t>(a.num_tokens) * heads;
  a.heads_mul = static_cast<uint32_t>(std::min<uint64_t>((1ull << 32) / heads, 0xFFFFFFFFu));
  const int64_t slots = 512ll * sms >> a.lanes_log2;  // groups at the same time
  // few threads: small CTAs, on many SMs, but a thread for each angle of two tokens (36 heads of 128,
  // 16 tokens: 4.1 us; 64 threads 4.7, 256 4.4)
  const int block = a.all_heads << a.lanes_log2 < static_cast<int64_t>(sms) * kThreads ? 128 : kThreads;
  const int groups = block >> a.lanes_log2;
  // tokens whose cosines a CTA has room for, at least two: runs begin anywhere
  const int64_t room = a.rope.pairs ? std::max<int64_t>(2, (32 << 10) / (a.rope.pairs * static_cast<int>(sizeof(float2)))) : 1 << 20;
  const int64_t longest = std::max<int64_t>(1, std::min<int64_t>(kLongest, (room - 1) * heads / groups));
  const int64_t rounds = (a.all_heads + slots * longest - 1) / (slots * longest);
  a.run = static_cast<int>((a.all_heads + slots * rounds - 1) / (slots * rounds));
  // kernels that take two heads at once: a token's heads then pair up in every run (30.4 -> 30.0 us)
  if (per_lane == 1 && heads % 2 == 0 && a.run > 2 && a.run < longest) a.run += a.run & 1;
  const int64_t per_cta = static_cast<int64_t>(groups) * a.run;
  const int64_t ctas = (a.all_heads + per_cta - 1) / per_cta;
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  const unsigned grid = static_cast<unsigned>(ctas);
  const int64_t tokens = std::min<int64_t>(a.num_tokens, (per_cta + heads - 2) / heads + 1);
  const int smem = kMaxArrays * a.head_dim * static_cast<int>(sizeof(float)) +
                   static_cast<int>(tokens) * a.rope.pairs * static_cast<int>(sizeof(float2));
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
    if ((num_tokens > 1 && out[i].token_stride == 0) || (out[i].heads > 1 && out[i].head_stride == 0))
      return fail(RIMURU_ERR_UNSUPPORTED, "norm output: elements may not lie on one another");
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
