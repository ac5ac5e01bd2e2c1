// Norms of heads and their rotation in one pass: a head x of a token becomes
// rot_p(x * r * (w + offset)) with r = 1 / sqrt(mean(x^2) + eps).
//
// Each element is read and written once; a head stays in the registers of the lanes
// that loaded it.  A group of 2^n lanes takes one token and some of its heads: a lane
// holds two vectors of eight elements of a head (in the half layout the two members of
// eight pairs, so that pairs turn within a lane), the squares are added up over the
// group by shuffles, and the token's cosines and sines, which a lane computes once for
// the pairs that it holds, serve every head that the group takes.
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
  int lanes_log2;       // of a group
  int heads_per_group, groups_per_token;
  int turn_slots, slots;  // of a head: slots whose vectors are a pair's members, and all
};

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(v[i] << 16);
    x[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const __half* p, float (&x)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(dev::pack_bf16x2(x[0], x[1]), dev::pack_bf16x2(x[2], x[3]),
                                            dev::pack_bf16x2(x[4], x[5]), dev::pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store8(__half* p, const float (&x)[8]) {
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    v[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
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

// kSlots: slots of a lane.
template <typename T, bool kHalf, int kSlots>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NormArgs p) {
  constexpr int kRows = kSlots == 1 ? 4 : 2;  // heads in flight in a group
  __shared__ uint64_t turn[kMaxPairs];
  for (int i = threadIdx.x; i < p.rope.pairs; i += blockDim.x) turn[i] = p.rope.turn[i];
  __syncthreads();
  const int lanes = 1 << p.lanes_log2, lane = threadIdx.x & (lanes - 1);
  const int64_t group = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> p.lanes_log2;
  const int64_t t = group / p.groups_per_token;
  // groups past the last token stay for the shuffles and take no head
  const int h0 = t < p.num_tokens ? static_cast<int>(group - t * p.groups_per_token) * p.heads_per_group : 1 << 30;
  const int rot = 2 * p.rope.pairs;

  int off[kSlots][2];
  float2 cs[kSlots][8];
  const uint64_t pos =
      rot > 0 && t < p.num_tokens ? static_cast<uint64_t>(static_cast<int64_t>(p.positions[t])) : 0;
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    place<kHalf>(p, lane + s * lanes, off[s]);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // pair e of the slot: elements (e, e) of its two vectors, or (2 e, 2 e + 1) of one
      const int at = kHalf ? (off[s][0] >= 0 && off[s][0] < rot ? off[s][0] + e : -1)
                           : (off[s][e / 4] >= 0 && off[s][e / 4] < rot ? off[s][e / 4] / 2 + e % 4 : -1);
      cs[s][e] = make_float2(1.f, 0.f);
      if (at >= 0) {
        float sn, c;
        sincospif(__ll2float_rn(static_cast<int64_t>(pos * turn[at])) * 0x1p-63f, &sn, &c);
        cs[s][e] = make_float2(c * p.rope.mscale, sn * p.rope.mscale);
      }
    }
  }

#pragma unroll 1
  for (int i = 0; i < kMaxArrays; ++i) {
    const int first = p.first_head[i], last = p.first_head[i + 1];
    if (first == last) continue;
    const NormArray& A = p.arr[i];
    const int from = max(h0, first) - first, to = min(h0 + p.heads_per_group, last) - first;
    // the same number of turns in every group of the warp: shuffles take all lanes
    const int turns = __reduce_max_sync(~0u, max(0, to - from));
    if (turns == 0) continue;
    float w[kSlots][2][8];
#pragma unroll
    for (int s = 0; s < kSlots; ++s)
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        if (A.weight && off[s][v] >= 0) {
          if (A.weight_dtype == RIMURU_BF16) load8(static_cast<const __nv_bfloat16*>(A.weight) + off[s][v], w[s][v]);
          else if (A.weight_dtype == RIMURU_F16) load8(static_cast<const __half*>(A.weight) + off[s][v], w[s][v]);
          else load8(static_cast<const float*>(A.weight) + off[s][v], w[s][v]);
#pragma unroll
          for (int e = 0; e < 8; ++e) w[s][v][e] += A.offset;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) w[s][v][e] = 1.f;
        }
      }
    const T* in = static_cast<const T*>(A.in) + t * A.in_ts + from * A.in_hs;
    T* out = static_cast<T*>(A.out) + t * A.out_ts + from * A.out_hs;
#pragma unroll 1
    for (int h = 0; h < turns; h += kRows) {
      float x[kRows][kSlots][2][8], sum[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int s = 0; s < kSlots; ++s)
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            if (from + h + r < to && off[s][v] >= 0) {
              load8(in + (h + r) * A.in_hs + off[s][v], x[r][s][v]);
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e) x[r][s][v][e] = 0.f;
            }
          }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        sum[r] = 0.f;
#pragma unroll
        for (int s = 0; s < kSlots; ++s)
#pragma unroll
          for (int v = 0; v < 2; ++v)
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[r] = fmaf(x[r][s][v][e], x[r][s][v][e], sum[r]);
      }
      for (int m = lanes >> 1; m > 0; m >>= 1)
#pragma unroll
        for (int r = 0; r < kRows; ++r) sum[r] += __shfl_xor_sync(~0u, sum[r], m);
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        float eps = A.eps;
        // squares past fp32: the head is taken 2^-96 times as large, where eps is nothing
        const bool large = !std::is_same<T, __half>::value && isinf(sum[r]);
        if (__any_sync(~0u, large)) {
          float again = 0.f;
          const float f = large ? 0x1p-96f : 1.f;
#pragma unroll
          for (int s = 0; s < kSlots; ++s)
#pragma unroll
            for (int v = 0; v < 2; ++v)
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                x[r][s][v][e] *= f;
                again = fmaf(x[r][s][v][e], x[r][s][v][e], again);
              }
          for (int m = lanes >> 1; m > 0; m >>= 1) again += __shfl_xor_sync(~0u, again, m);
          if (large) sum[r] = again, eps = 0.f;
        }
        const float mean = fmaf(sum[r], 1.f / p.head_dim, eps);
        float k = rsqrtf(mean);
        if (sizeof(T) == 4) k = isinf(mean) ? 0.f : k * fmaf(-0.5f * mean * k, k, 1.5f);  // to the last bit
        if (from + h + r >= to) continue;
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
          float y[2][8];
#pragma unroll
          for (int v = 0; v < 2; ++v)
#pragma unroll
            for (int e = 0; e < 8; ++e) y[v][e] = x[r][s][v][e] * k * w[s][v][e];
          if (kHalf) {
            if (off[s][0] >= 0 && off[s][0] < rot) {
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float a = y[0][e], b = y[1][e];
                y[0][e] = a * cs[s][e].x - b * cs[s][e].y;
                y[1][e] = b * cs[s][e].x + a * cs[s][e].y;
              }
            }
          } else {
#pragma unroll
            for (int v = 0; v < 2; ++v)
              if (off[s][v] >= 0 && off[s][v] < rot) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float a = y[v][2 * e], b = y[v][2 * e + 1];
                  const float2 c = cs[s][4 * v + e];
                  y[v][2 * e] = a * c.x - b * c.y;
                  y[v][2 * e + 1] = b * c.x + a * c.y;
                }
              }
          }
#pragma unroll
          for (int v = 0; v < 2; ++v)
            if (off[s][v] >= 0) store8(out + (h + r) * A.out_hs + off[s][v], y[v]);
        }
      }
    }
  }
}

template <typename T>
cudaError_t launch(const NormArgs& a, int per_lane, cudaStream_t stream) {
  const int64_t threads = static_cast<int64_t>(a.num_tokens) * a.groups_per_token << a.lanes_log2;
  // few threads: small CTAs, on many SMs
  const int block = threads < 152 * kThreads ? 64 : kThreads;
  const unsigned grid = static_cast<unsigned>((threads + block - 1) / block);
  if (a.rope.layout == RIMURU_ROPE_HALF) {
    if (per_lane == 1) norm_rope_kernel<T, true, 1><<<grid, block, 0, stream>>>(a);
    else norm_rope_kernel<T, true, 2><<<grid, block, 0, stream>>>(a);
  } else {
    if (per_lane == 1) norm_rope_kernel<T, false, 1><<<grid, block, 0, stream>>>(a);
    else norm_rope_kernel<T, false, 2><<<grid, block, 0, stream>>>(a);
  }
  return cudaGetLastError();
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
  // A group takes all heads of its token when that leaves 512 threads an SM, else fewer
  // (the angles are then computed by several groups).
  int sms = 0, dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return fail(RIMURU_ERR_CUDA, kv_cuda_msg("device attributes", e));
  const int64_t want = 512ll * sms >> a.lanes_log2;  // groups
  const int64_t per_token = std::max<int64_t>(1, std::min<int64_t>(heads, want / num_tokens));
  a.heads_per_group = static_cast<int>((heads + per_token - 1) / per_token);
  a.groups_per_token = static_cast<int>((heads + a.heads_per_group - 1) / a.heads_per_group);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  e = in[0].dtype == RIMURU_BF16  ? launch<__nv_bfloat16>(a, per_lane, s)
      : in[0].dtype == RIMURU_F16 ? launch<__half>(a, per_lane, s)
                                  : launch<float>(a, per_lane, s);
  if (e != cudaSuccess) return fail(RIMURU_ERR_CUDA, kv_cuda_msg("norm launch", e));
  return RIMURU_OK;
}
