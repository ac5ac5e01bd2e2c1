// Rotary positions: pair (u, v) of a head at position p becomes
// m (u cos a - v sin a, v cos a + u sin a) with a = p f_i.
//
// An fp32 product p * f_i is off by up to half an ulp of the product: 0.004 rad
// at 65536 positions for the fastest pair.  Here f_i is a 64-bit fraction of a
// turn, so p times it modulo 2^64 is the angle modulo one turn.  It is rounded to
// fp32 once, as a signed number, so that a small angle keeps its bits too.  f_i
// itself is a double, good to a few times 2^-53 of itself: at 2^31 positions the
// fastest pair is off by about 2^-24 of a turn.  A negative position is the same
// product modulo 2^64.
//
// Each element is read and written once.  A CTA takes one token, or four of a
// long array: it computes their cosines and sines once into shared memory (they
// serve all heads of all arrays), then every thread loads, turns and stores 64
// bytes (half layout: 128) at a time, without another barrier.
// 8192 tokens in bf16 (151 MB), 18 heads of 256 of which 64 elements turn: 30.4 us, 5.0
// TB/s, 0.74 of the copy rate (35 us with one token a CTA); 36 heads of 128, half layout:
// 33.4 us.  Not HBM alone: with DRAM 44 % busy 62 % of the issue slots are taken, by the
// arithmetic that finds an item's place as much as by the rotation.  One token: 2.9 us, a
// launch.
#include <algorithm>
#include <cmath>
#include <limits>
#include <new>

#include "device.cuh"
#include "kv.h"
#include "rope.h"

namespace rimuru {
namespace {

using dev::from_f;
using dev::to_f;

constexpr int kMaxArrays = 4;
constexpr int kMaxTokens = 4;  // of a CTA

struct RopeArray {
  const void* in;
  void* out;
  int64_t in_ts, in_hs, out_ts, out_hs;  // strides in elements
};

struct RopeArgs {
  uint64_t turn[kMaxPairs];  // 2^-64 turns per position
  RopeArray arr[kMaxArrays];
  int first_item[kMaxArrays + 1];  // items (see kernel) of the arrays before this one
  const int32_t* positions;
  float mscale;
  int pairs, layout, head_dim, num_tokens, tokens_per_cta;
  int turn_items, items_per_head;
  uint64_t head_mul;  // item / items_per_head = item * head_mul >> 32
};

template <typename T>
struct Vec8 {  // eight elements of T
  uint4 w[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Vec8<T> load8(const T* p) {
  Vec8<T> v;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) v.w[i] = reinterpret_cast<const uint4*>(p)[i];
  return v;
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const Vec8<T>& v) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) reinterpret_cast<uint4*>(p)[i] = v.w[i];
}

// An item is one thread's unit of work in a head: items below `turn_items` turn
// pairs (two vectors of eight in the half layout, one in the interleaved one),
// the others copy a vector of eight past the rotated part.
template <typename T, bool kHalf, int kPer>
__global__ void __launch_bounds__(256) rope_kernel(const __grid_constant__ RopeArgs p) {
  __shared__ float2 cosines[kMaxTokens * kMaxPairs];
  const int t0 = blockIdx.x * p.tokens_per_cta, n_tokens = min(p.tokens_per_cta, p.num_tokens - t0);
  const int n_items = p.first_item[kMaxArrays];
  const int rot = 2 * p.pairs;
  for (int k = threadIdx.x; k < n_tokens * p.pairs; k += blockDim.x) {
    const int t = k / p.pairs, i = k - t * p.pairs;
    const uint64_t pos = static_cast<uint64_t>(static_cast<int64_t>(p.positions[t0 + t]));
    const int64_t turn = static_cast<int64_t>(pos * p.turn[i]);  // 2^-64 turns
    float s, c;
    sincospif(__ll2float_rn(turn) * 0x1p-63f, &s, &c);
    cosines[k] = make_float2(c * p.mscale, s * p.mscale);
  }
  __syncthreads();
  for (int t = t0; t < t0 + n_tokens; ++t) {
    const float2* cs = cosines + (t - t0) * p.pairs;
    for (int base = 0; base < n_items; base += kPer * blockDim.x) {
      Vec8<T> a[kPer], b[kHalf ? kPer : 1];
      T* dst[kPer];
      int off[kPer];  // first element of the item in its head
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int item = base + j * blockDim.x + threadIdx.x;
        dst[j] = nullptr;
        if (item >= n_items) continue;
        int s = 0;
#pragma unroll
        for (int i = 1; i < kMaxArrays; ++i) s += item >= p.first_item[i];
        const RopeArray& A = p.arr[s];
        const int local = item - p.first_item[s];
        const int h = static_cast<int>(local * p.head_mul >> 32), i = local - h * p.items_per_head;
        off[j] = i < p.turn_items ? 8 * i : rot + 8 * (i - p.turn_items);
        const T* src = static_cast<const T*>(A.in) + t * A.in_ts + h * A.in_hs + off[j];
        dst[j] = static_cast<T*>(A.out) + t * A.out_ts + h * A.out_hs + off[j];
        a[j] = load8(src);
        if (kHalf && off[j] < rot) b[kHalf ? j : 0] = load8(src + p.pairs);
      }
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        if (!dst[j]) continue;
        if (off[j] < rot) {
          T* x = reinterpret_cast<T*>(&a[j]);
          T* y = reinterpret_cast<T*>(&b[kHalf ? j : 0]);
          if (kHalf) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float2 w = cs[off[j] + e];
              const float u = to_f(x[e]), v = to_f(y[e]);
              from_f(u * w.x - v * w.y, &x[e]);
              from_f(v * w.x + u * w.y, &y[e]);
            }
            store8(dst[j] + p.pairs, b[kHalf ? j : 0]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 w = cs[off[j] / 2 + e];
              const float u = to_f(x[2 * e]), v = to_f(x[2 * e + 1]);
              from_f(u * w.x - v * w.y, &x[2 * e]);
              from_f(v * w.x + u * w.y, &x[2 * e + 1]);
            }
          }
        }
        store8(dst[j], a[j]);
      }
    }
  }
}

template <typename T>
cudaError_t launch(const RopeArgs& a, cudaStream_t stream) {
  const int items = a.first_item[kMaxArrays];
  // four items a thread, so that a thread has 64 bytes (half layout: 128) in flight
  const int threads = std::min(256, ((items + 3) / 4 + 31) / 32 * 32);
  const int grid = (a.num_tokens + a.tokens_per_cta - 1) / a.tokens_per_cta;
  if (a.layout == RIMURU_ROPE_HALF) rope_kernel<T, true, 4><<<grid, threads, 0, stream>>>(a);
  else rope_kernel<T, false, 4><<<grid, threads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace rimuru

struct rimuru_rope_s {
  rimuru::RopeArgs a;  // turn, mscale, pairs and layout filled in
};

using rimuru::fail;

void rimuru::rope_turns(rimuru_rope_t rope, RopeTurns* out) {
  for (int i = 0; i < rope->a.pairs; ++i) out->turn[i] = rope->a.turn[i];
  out->mscale = rope->a.mscale;
  out->pairs = rope->a.pairs;
  out->layout = rope->a.layout;
}

extern "C" int rimuru_rope_create(int rot_dim, int layout, double base, int scaling, double factor,
                                  double orig_len, double low, double high, double mscale,
                                  rimuru_rope_t* out) {
  rimuru::clear_error();
  if (!out) return fail(RIMURU_ERR_ARG, "null output handle");
  if (layout != RIMURU_ROPE_HALF && layout != RIMURU_ROPE_INTERLEAVED)
    return fail(RIMURU_ERR_ARG, "unknown rotary layout");
  if (scaling < RIMURU_ROPE_PLAIN || scaling > RIMURU_ROPE_BY_PARTS)
    return fail(RIMURU_ERR_ARG, "unknown rotary scaling");
  if (!(base > 1.0) || !std::isfinite(base) || !std::isfinite(static_cast<float>(mscale)))
    return fail(RIMURU_ERR_ARG, "base must be finite and above 1, mscale finite in fp32");
  const bool scaled = scaling != RIMURU_ROPE_PLAIN;
  if (scaled && !(factor > 0.0 && std::isfinite(factor)))
    return fail(RIMURU_ERR_ARG, "factor must be finite and positive");
  if (rot_dim <= 0 || rot_dim > 2 * rimuru::kMaxPairs ||
      rot_dim % (layout == RIMURU_ROPE_HALF ? 16 : 8) != 0)
    return fail(RIMURU_ERR_UNSUPPORTED,
                "rot_dim must be in (0, 256] and a multiple of 16 (half) or 8 (interleaved)");
  if (scaling == RIMURU_ROPE_BY_PARTS &&
      !(orig_len > 0.0 && std::isfinite(orig_len) && std::isfinite(high - low) && high > low))
    return fail(RIMURU_ERR_ARG, "by-parts scaling needs orig_len > 0 and high > low");
  if (scaling == RIMURU_ROPE_BASE) base *= std::pow(factor, rot_dim / (rot_dim - 2.0));
  if (!(base > 0.0 && std::isfinite(base))) return fail(RIMURU_ERR_ARG, "scaled base out of range");
  auto* r = new (std::nothrow) rimuru_rope_s{};
  if (!r) return fail(RIMURU_ERR_OOM, "host allocation failed");
  const double two_pi = 6.283185307179586476925;
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot_dim);
    if (scaling == RIMURU_ROPE_LINEAR) f /= factor;
    if (scaling == RIMURU_ROPE_BY_PARTS) {
      const double g = std::min(1.0, std::max(0.0, (orig_len * f / two_pi - low) / (high - low)));
      f = (1.0 - g) * f / factor + g * f;
    }
    if (!std::isfinite(f)) {
      delete r;
      return fail(RIMURU_ERR_ARG, "scaled frequencies out of range");
    }
    double turns = f / two_pi;
    turns -= std::floor(turns);  // the phase is taken modulo one turn
    r->a.turn[i] = static_cast<uint64_t>(std::ldexp(turns, 63)) << 1;
  }
  r->a.mscale = static_cast<float>(mscale);
  r->a.pairs = rot_dim / 2;
  r->a.layout = layout;
  *out = r;
  return RIMURU_OK;
}

extern "C" int rimuru_rope_destroy(rimuru_rope_t rope) {
  rimuru::clear_error();
  if (!rope) return fail(RIMURU_ERR_ARG, "null rope");
  delete rope;
  return RIMURU_OK;
}

extern "C" int rimuru_rope_apply(rimuru_rope_t rope, const int32_t* positions, int num_tokens,
                                 int head_dim, const rimuru_heads* in, const rimuru_heads* out,
                                 int n_arrays, void* stream) {
  using namespace rimuru;
  clear_error();
  if (!rope) return fail(RIMURU_ERR_ARG, "null rope");
  if (!in || !out || n_arrays < 1 || n_arrays > kMaxArrays)
    return fail(RIMURU_ERR_ARG, "between 1 and 4 arrays");
  if (num_tokens < 0) return fail(RIMURU_ERR_ARG, "negative token count");
  RopeArgs a = rope->a;
  const int rot = 2 * a.pairs;
  if (head_dim < rot || head_dim % 8 != 0 || head_dim > 1024)
    return fail(RIMURU_ERR_UNSUPPORTED,
                "head_dim must be a multiple of 8, at least rot_dim and at most 1024");
  if (num_tokens == 0) return RIMURU_OK;
  if (!positions) return fail(RIMURU_ERR_ARG, "null positions");
  if (reinterpret_cast<uintptr_t>(positions) % 4 != 0)
    return fail(RIMURU_ERR_ALIGN, "positions must be 4-byte aligned");
  a.positions = positions;
  a.head_dim = head_dim;
  a.num_tokens = num_tokens;
  a.tokens_per_cta = num_tokens >= 2048 ? kMaxTokens : 1;  // below, one token a CTA fills the GPU better
  a.turn_items = (a.layout == RIMURU_ROPE_HALF ? a.pairs : rot) / 8;
  int64_t items = 0;
  bool inplace = true;
  for (int i = 0; i < n_arrays; ++i) {
    int st = check_heads(&in[i], "rope input");
    if (st == RIMURU_OK) st = check_heads(&out[i], "rope output");
    if (st != RIMURU_OK) return st;
    if (in[i].heads != out[i].heads || in[i].dtype != out[i].dtype || in[i].dtype != in[0].dtype)
      return fail(RIMURU_ERR_ARG, "inputs and outputs must agree in heads and type");
    inplace &= in[i].data == out[i].data && in[i].token_stride == out[i].token_stride &&
               in[i].head_stride == out[i].head_stride;
    a.arr[i] = {in[i].data,          out[i].data,         in[i].token_stride,
                in[i].head_stride, out[i].token_stride, out[i].head_stride};
  }
  // in place, the elements past the rotated part stay where they are
  a.items_per_head = a.turn_items + (inplace ? 0 : (head_dim - rot) / 8);
  for (int i = 0; i <= kMaxArrays; ++i) {
    a.first_item[i] = static_cast<int>(items);
    if (i < n_arrays) items += static_cast<int64_t>(in[i].heads) * a.items_per_head;
    if (items > (1 << 24)) return fail(RIMURU_ERR_UNSUPPORTED, "too many heads");
  }
  a.head_mul = (1ull << 32) / a.items_per_head + 1;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = in[0].dtype == RIMURU_BF16  ? launch<__nv_bfloat16>(a, s)
                  : in[0].dtype == RIMURU_F16 ? launch<__half>(a, s)
                                              : launch<float>(a, s);
  if (e != cudaSuccess) return fail(RIMURU_ERR_CUDA, kv_cuda_msg("rope launch", e));
  return RIMURU_OK;
}
