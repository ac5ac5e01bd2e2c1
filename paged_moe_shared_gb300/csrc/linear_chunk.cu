// Linear attention over prompts: 64 tokens (a chunk) at a time on the tensor cores.
//
// With G_i the sum of the decays of a chunk's tokens up to i, S the state before it and
// T the state after it, a head's chunk is
//   out_i = scale (exp(G_i) S^T q_i + sum_{j <= i} exp(G_i - G_j) (q_i . k_j) v_j)
//   T     = exp(G_last) S + sum_j exp(G_last - G_j) k_j v_j^T.
// All products are made transposed, with the value columns in the 128 lanes of TMEM and
// 64 tokens or the key columns across, so that every MMA has full height:
//   scores  Q K^T          (64 x 64; the lanes below take K K^T, which nobody reads)
//   inter   S^T Q^T        S^T in TMEM, as two bf16 parts that its owners write there
//   intra   V^T P^T        P = scores * decays, two bf16 parts in shared memory
//   update  V^T Kd         Kd = decayed keys, three bf16 parts: an fp32 number exactly
// S^T itself stays in the registers of eight warps in fp32 and takes each chunk's update
// there: sums inside the tensor cores truncate, and over thousands of tokens that would
// show.  f16 inputs are split into two bf16 parts as they are loaded, exactly.
//
// Differences G_i - G_j are taken on sums in 64-bit fixed point, so that a huge decay
// early in a chunk costs the small ones after it nothing.
//
// Few heads and long sequences leave SMs without work, so sequences can be cut into
// pieces: a first kernel computes what each piece adds to the state and a second one
// starts every piece from the states of the pieces before it.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "device.cuh"
#include "kv_attn.h"
#include "linear.h"

namespace rimuru {
namespace {

using namespace dev;

constexpr int kC = 64;               // tokens of a chunk
constexpr uint32_t kBlock = 8192;    // 64 rows of 128 bytes, swizzled
constexpr int kGates = 4;            // chunks whose decays are ready
constexpr int kThreads = 768;
constexpr int kStateRegs = 112, kProductRegs = 64, kOutRegs = 72, kOtherRegs = 56;
static_assert((2 * kStateRegs + 2 * kProductRegs + kOutRegs + kOtherRegs) * 128 <= 80 * kThreads, "");

struct Gate {
  float2 sum[kC];   // G in two parts whose differences are exact, log2
  float before[kC]; // scale * exp(G)
  float after[kC];  // exp(G_last - G), 0 past the chunk's tokens
  float all;        // exp(G_last)
};

struct ChunkShared {
  Gate gate[kGates];
  uint64_t full[2], empty[2];             // loaded tiles
  uint64_t gate_full[kGates], gate_empty[kGates];
  uint64_t score_full[2], score_empty[2];
  uint64_t key_full[2], key_empty[2];     // decayed keys
  uint64_t p_full, p_empty;
  uint64_t state_full, state_empty;       // parts of S
  uint64_t update_full, update_empty;
  uint64_t out_full, out_empty;
  uint64_t drain;
  int abort;
  uint32_t tmem_base;
};

template <typename T, int kDk, int kDv>
struct Cfg {
  static constexpr int kIn = std::is_same<T, __half>::value ? 2 : 1;  // bf16 parts of an input
  static constexpr int kStages = kIn == 1 ? 2 : 1;
  static constexpr int kKb = kDk / 64, kVb = kDv / 64;
  // a stage: for each part [key block][Q rows, K rows], then for each part [value block]
  static constexpr uint32_t kQk = kKb * 2 * kBlock, kV = kVb * kBlock;
  static constexpr uint32_t kStage = kIn * (kQk + kV);
  static constexpr uint32_t kKeyPart = kKb * kBlock;
  static constexpr uint32_t kKeyAt = kStages * kStage, kPAt = kKeyAt + 2 * 3 * kKeyPart;
  static constexpr uint32_t kSmem = kPAt + 2 * kBlock + 1024;
};

struct ChunkArgs {
  LinearArgs l;
  int piece, units;
  float* states;  // [pieces][heads][key_dim][value_dim]: what pieces add, sequences' first ones whole
  float* firsts;  // [num_seqs][heads][...]: states before sequences that are cut
  float* decays;  // [pieces][heads]
};

// One unit: a piece of a sequence and a head.
struct Unit {
  int b, h, slot;   // slot: the piece's among all
  int64_t row;      // first row
  int n;            // rows
  int seq0;         // the sequence's first row
  bool first, last; // piece of its sequence
  const float* in;  // of the sequence, or null
  float* out;
  bool ok;
};
__device__ __forceinline__ Unit find_unit(const ChunkArgs& p, int u, bool record) {
  const LinearArgs& a = p.l;
  Unit x;
  x.slot = u / a.heads;
  x.h = u - x.slot * a.heads;
  int start;
  if (x.slot < a.num_seqs) {
    x.b = x.slot;
    start = a.cu[x.b];
  } else {
    start = (x.slot - a.num_seqs + 1) * p.piece;
    int lo = 0, hi = a.num_seqs;  // the last sequence that begins at or before the row
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.cu[mid] <= start) lo = mid;
      else hi = mid;
    }
    x.b = lo;
  }
  const LinearSeq s = linear_seq(a, x.b, record && x.slot < a.num_seqs && x.h == 0);
  x.seq0 = static_cast<int>(s.row);
  const int end = x.seq0 + s.n;
  x.ok = s.ok && (x.slot < a.num_seqs || (start > x.seq0 && start < end));
  const int64_t next = p.piece > 0 ? (static_cast<int64_t>(start) / p.piece + 1) * p.piece : end;
  x.row = start;
  x.n = static_cast<int>(min(next, static_cast<int64_t>(end))) - start;
  x.first = start == x.seq0;
  x.last = start + x.n == end;
  x.in = s.in;
  x.out = s.out;
  return x;
}

// Walks the units of this CTA; every warp does so by itself.
template <bool kOut>
struct Walk {
  int u;
  __device__ __forceinline__ bool next(const ChunkArgs& p, Unit* x, bool record = false) {
    for (;; ) {
      u = u < 0 ? static_cast<int>(blockIdx.x) : u + static_cast<int>(gridDim.x);
      if (u >= p.units) return false;
      *x = find_unit(p, u, record);
      // the first kernel is about pieces that others follow
      if (x->ok && (kOut || !x->last)) return true;
    }
  }
};

template <int kRegs>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <uint32_t kAHi, uint32_t kBHi, uint32_t kIdesc>
__device__ __forceinline__ void umma_f16_lo(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %3, 0;\n\t"
      "mov.b64 a, {%1, %4};\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %6, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(accumulate), "n"(kAHi), "n"(kBHi), "n"(kIdesc)
      : "memory");
}
// 16 bytes from global memory, or zeros where `real` is false (nothing is read).
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 16-byte piece `c` of row r in a swizzled block of 128-byte rows.
__device__ __forceinline__ uint32_t place(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }
// The upper halves of two numbers as a pair of bf16: what is below is cut off.
__device__ __forceinline__ uint32_t tops(float lo, float hi) {
  return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}
__device__ __forceinline__ float top(float x) { return __uint_as_float(__float_as_uint(x) & 0xFFFF0000u); }

// Fixed point with 40 bits below the point.
__device__ __forceinline__ int64_t fixed_log2(float g) {
  g = fminf(fmaxf(g, -1400.f), 1400.f);  // 2^2000 either way is 0 or infinity
  constexpr float kHi = 1.4426950408889634f, kLo = 1.925963033500e-8f;  // log2(e)
  const float x = g * kHi;
  const float rest = fmaf(g, kHi, -x) + g * kLo;
  return __float2ll_rn(x * 0x1p40f) + __float2ll_rn(rest * 0x1p40f);
}
__device__ __forceinline__ float exp2_fixed(int64_t d) {
  const int64_t n = (d + (1ll << 39)) >> 40;
  const float f = __ll2float_rn(d - (n << 40)) * 0x1p-40f;
  return ldexpf(exp2f(f), static_cast<int>(n));
}

template <typename T, int kDk, int kDv, bool kOut>
__global__ void __launch_bounds__(kThreads, 1) linear_chunk_kernel(const __grid_constant__ ChunkArgs p) {
  using C = Cfg<T, kDk, kDv>;
  constexpr int kStages = C::kStages, kIn = C::kIn;
  extern __shared__ uint8_t raw_smem[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ ChunkShared sh_;
  ChunkShared* sh = &sh_;
  volatile int* abort = &sh->abort;
  const LinearArgs& a = p.l;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->full[i], 64);
      mbar_init(&sh->empty[i], 1 + 4);   // the MMAs, the warps that decay keys
      mbar_init(&sh->score_full[i], 1);
      mbar_init(&sh->score_empty[i], 4);
      mbar_init(&sh->key_full[i], 4);
      mbar_init(&sh->key_empty[i], 1);
    }
    for (int i = 0; i < kGates; ++i) {
      mbar_init(&sh->gate_full[i], 1);
      mbar_init(&sh->gate_empty[i], kOut ? 8 + 4 + 4 + 4 : 8 + 4);
    }
    mbar_init(&sh->p_full, 4);
    mbar_init(&sh->p_empty, 1);
    mbar_init(&sh->state_full, 8);
    mbar_init(&sh->state_empty, 1);
    mbar_init(&sh->update_full, 1);
    mbar_init(&sh->update_empty, 8);
    mbar_init(&sh->out_full, 1);
    mbar_init(&sh->out_empty, 4);
    mbar_init(&sh->drain, 1);
    sh->abort = 0;
    fence_barrier_init();
  }
  if (warp == 20) {
    tmem_alloc(&sh->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  // columns of TMEM
  constexpr uint32_t kScore = 0, kInter = 128, kIntra = 192, kUpdate = 256, kState = 384;
  bool ok = true;
  const auto wait = [&](uint64_t* bar, uint32_t phase) {
    ok = ok && mbar_wait_idle(bar, phase & 1u, abort);
    ok = __all_sync(0xffffffffu, ok);
  };
  // one arrival of a converged warp
  const auto arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  Walk<kOut> walk{-1};
  Unit x;
  uint32_t it = 0;  // chunks so far

  if (warp >= 20) {
    regs_down<kOtherRegs>();
    if (warp >= 22) {
      // ------------------------------------------------------------------ loads
      const int tid = threadIdx.x - 22 * 32;
      while (ok && walk.next(p, &x)) {
        const T* q = static_cast<const T*>(a.q) + x.row * a.q_ts + x.h / a.per_key_head * a.q_hs;
        const T* k = static_cast<const T*>(a.k) + x.row * a.k_ts + x.h / a.per_key_head * a.k_hs;
        const T* v = static_cast<const T*>(a.v) + x.row * a.v_ts + x.h * a.v_hs;
        for (int c = 0; ok && c < x.n; c += kC, ++it) {
          const uint32_t stage = it % kStages;
          wait(&sh->empty[stage], (it / kStages) ^ 1u);
          if (!ok) break;
          const int n = min(kC, x.n - c);
          uint8_t* base = smem + stage * C::kStage;
          // rows of `src` into blocks `pitch` bytes apart; parts lie `part` bytes apart
          const auto tile = [&](const T* src, int64_t ts, int vectors, uint8_t* dst, uint32_t pitch, uint32_t part) {
            const int per = 64 / vectors;  // rows of a turn
            const int col = tid % vectors, r0 = tid / vectors;
            dst += col / 8 * pitch;
#pragma unroll 8
            for (int r = r0; r < kC; r += per) {
              const T* from = src + (c + r) * ts + 8 * col;
              const uint32_t at = place(r, col & 7);
              if (kIn == 1) {
                cp_async16_or_zero(smem_u32(dst + at), r < n ? from : src, r < n);
              } else {
                uint4 w = make_uint4(0, 0, 0, 0);
                if (r < n) w = ld_nc_na_v4(from);
                uint32_t hi[4], lo[4];
                const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&in[i]));
                  hi[i] = tops(f.x, f.y);
                  lo[i] = tops(f.x - top(f.x), f.y - top(f.y));
                }
                *reinterpret_cast<uint4*>(dst + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4*>(dst + part + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
              }
            }
          };
          tile(k, a.k_ts, kDk / 8, base + kBlock, 2 * kBlock, C::kQk);
          if (kOut) tile(q, a.q_ts, kDk / 8, base, 2 * kBlock, C::kQk);
          tile(v, a.v_ts, kDv / 8, base + kIn * C::kQk, kBlock, C::kV);
          if (kIn == 1) {
            cp_async_arrive_noinc(&sh->full[stage]);
          } else {
            fence_proxy_async_smem();
            mbar_arrive(&sh->full[stage]);
          }
        }
      }
      cp_async_wait_all();
    } else if (warp == 21) {
      // ------------------------------------------------------------------ decays
      while (ok && walk.next(p, &x)) {
        const float* g = a.decay + x.row * a.g_ts + x.h * a.g_hs;
        constexpr int64_t kFar = 1ll << 53;  // 2^8192 either way is 0 or infinity
        int64_t total = 0;
        bool nan = false;
        for (int c = 0; ok && c < x.n; c += kC, ++it) {
          const uint32_t slot = it % kGates;
          const int n = min(kC, x.n - c), i = 2 * lane;
          const float g0 = i < n ? g[(c + i) * a.g_ts] : 0.f, g1 = i + 1 < n ? g[(c + i + 1) * a.g_ts] : 0.f;
          const int64_t x1 = fixed_log2(g1);
          int64_t G1 = fixed_log2(g0) + x1;
#pragma unroll
          for (int m = 1; m < 32; m <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, G1, m);
            if (lane >= m) G1 += up;
          }
          const int64_t G0 = G1 - x1, last = __shfl_sync(0xffffffffu, G1, 31);
          const uint32_t bad0 = __ballot_sync(0xffffffffu, g0 != g0), bad1 = __ballot_sync(0xffffffffu, g0 != g0 || g1 != g1);
          // a NaN counts for every token from its own on
          const uint32_t below = (2u << lane) - 1u;
          const bool nan0 = ((bad0 & below) | (bad1 & (below >> 1))) != 0, nan1 = (bad1 & below) != 0;
          const float none = __int_as_float(0x7FFFFFFF);
          wait(&sh->gate_empty[slot], (it / kGates) ^ 1u);
          if (!ok) break;
          Gate& t = sh->gate[slot];
          if (kOut) {
            const auto parts = [&](int64_t G, bool is_nan) {
              return make_float2(is_nan ? none : __int2float_rn(static_cast<int>(G >> 34)) * 0x1p-6f,
                                 __ll2float_rn(G & ((1ll << 34) - 1)) * 0x1p-40f);
            };
            t.sum[i] = parts(G0, nan0);
            t.sum[i + 1] = parts(G1, nan1);
            t.before[i] = nan0 ? none : exp2_fixed(G0) * a.scale;
            t.before[i + 1] = nan1 ? none : exp2_fixed(G1) * a.scale;
          }
          t.after[i] = i < n ? exp2_fixed(last - G0) : 0.f;
          t.after[i + 1] = i + 1 < n ? exp2_fixed(last - G1) : 0.f;
          if (lane == 0) t.all = bad1 ? none : exp2_fixed(last);
          total = min(max(total + last, -kFar), kFar);
          nan |= bad1 != 0;
          arrive(&sh->gate_full[slot]);
        }
        if (!kOut && lane == 0)
          p.decays[static_cast<int64_t>(x.slot) * a.heads + x.h] =
              nan ? __int_as_float(0x7FFFFFFF) : exp2_fixed(total);
      }
    } else {
      // ------------------------------------------------------------------ MMAs
      constexpr uint32_t kHi = desc_hi(1024, 2);
      constexpr uint32_t id_score = idesc_bf16_f32(128, 64, false, false);
      constexpr uint32_t id_inter = idesc_bf16_f32(128, 64, false, false);
      constexpr uint32_t id_intra = idesc_bf16_f32(128, 64, true, false);
      constexpr uint32_t id_update = idesc_bf16_f32(128, kDk, true, true);
      const uint32_t tb = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t base_lo = __shfl_sync(0xffffffffu, desc_lo(smem_u32(smem), 16), 0);            // K-major tiles
      const uint32_t cols_lo = __shfl_sync(0xffffffffu, desc_lo(smem_u32(smem), kBlock), 0);        // MN-major tiles
      uint32_t scored = 0;
      const auto scores = [&]() {  // of chunk `scored`
        const uint32_t stage = scored % kStages, buffer = scored & 1u;
        wait(&sh->full[stage], scored / kStages);
        wait(&sh->score_empty[buffer], (scored >> 1) ^ 1u);
        tc_fence_after();
        if (ok && elect_one()) {
          fence_proxy_async_smem();
          const uint32_t q0 = base_lo + stage * (C::kStage / 16), k0 = q0 + kBlock / 16;
          uint32_t more = 0;
#pragma unroll
          for (int pair = (kIn == 2 ? 2 : 0); pair >= 0; --pair) {  // parts (0, 1), (1, 0), then (0, 0)
            const uint32_t pa = pair == 1 ? C::kQk / 16 : 0, pb = pair == 2 ? C::kQk / 16 : 0;
#pragma unroll
            for (int s = 0; s < kDk / 16; ++s) {
              const uint32_t at = s / 4 * (2 * kBlock / 16) + s % 4 * 2;
              umma_f16_lo<kHi, kHi, id_score>(tb + kScore + 64 * buffer, q0 + pa + at, k0 + pb + at, more);
              more = 1;
            }
          }
          umma_commit(&sh->score_full[buffer]);
        }
        __syncwarp();
        ++scored;
      };
      while (ok && walk.next(p, &x)) {
        const int chunks = (x.n + kC - 1) / kC;
        if (kOut && chunks > 0) scores();
        for (int c = 0; ok && c < chunks; ++c, ++it) {
          const uint32_t stage = it % kStages, buffer = it & 1u;
          const uint32_t v0 = cols_lo + (stage * C::kStage + kIn * C::kQk) / 16;
          if (!kOut) wait(&sh->full[stage], it / kStages);
          wait(&sh->key_full[buffer], it >> 1);
          wait(&sh->update_empty, it ^ 1u);
          tc_fence_after();
          if (ok && elect_one()) {
            if (!kOut) fence_proxy_async_smem();
            const uint32_t k0 = cols_lo + (C::kKeyAt + buffer * 3 * C::kKeyPart) / 16;
            uint32_t more = 0;
            // small parts first: what the sum cuts off is then small too
#pragma unroll
            for (int pv = kIn - 1; pv >= 0; --pv) {
#pragma unroll
              for (int pk = pv == 1 ? 1 : 2; pk >= 0; --pk) {
#pragma unroll
                for (int s = 0; s < kC / 16; ++s) {
                  umma_f16_lo<kHi, kHi, id_update>(tb + kUpdate, v0 + pv * (C::kV / 16) + 128 * s,
                                                   k0 + pk * (C::kKeyPart / 16) + 128 * s, more);
                  more = 1;
                }
              }
            }
            umma_commit(&sh->update_full);
            umma_commit(&sh->key_empty[buffer]);
            if (!kOut) umma_commit(&sh->empty[stage]);
          }
          __syncwarp();
          if (!kOut) continue;
          if (kStages > 1 && c + 1 < chunks) scores();
          wait(&sh->state_full, it);
          wait(&sh->out_empty, it ^ 1u);
          tc_fence_after();
          if (ok && elect_one()) {
            const uint32_t q0 = base_lo + stage * (C::kStage / 16);
            uint32_t more = 0;
#pragma unroll
            for (int pair = (kIn == 2 ? 2 : 1); pair >= 0; --pair) {  // (lo, 0), (hi, 1), (hi, 0) of S and Q
              const uint32_t ps = pair == 1 ? kDk / 2 : 0, pq = pair == 2 ? C::kQk / 16 : 0;
#pragma unroll
              for (int s = 0; s < kDk / 16; ++s) {
                umma_f16_ts_lo<kHi, id_inter>(tb + kInter, tb + kState + ps + 8 * s,
                                              q0 + pq + s / 4 * (2 * kBlock / 16) + s % 4 * 2, more);
                more = 1;
              }
            }
            umma_commit(&sh->state_empty);
          }
          __syncwarp();
          wait(&sh->p_full, it);
          tc_fence_after();
          if (ok && elect_one()) {
            const uint32_t p0 = base_lo + C::kPAt / 16;
            uint32_t more = 0;
#pragma unroll
            for (int pair = (kIn == 2 ? 2 : 1); pair >= 0; --pair) {  // (0, lo), (1, hi), (0, hi) of V and P
              const uint32_t pp = pair == 1 ? kBlock / 16 : 0, pv = pair == 2 ? C::kV / 16 : 0;
#pragma unroll
              for (int s = 0; s < kC / 16; ++s) {
                umma_f16_lo<kHi, kHi, id_intra>(tb + kIntra, v0 + pv + 128 * s, p0 + pp + 2 * s, more);
                more = 1;
              }
            }
            umma_commit(&sh->p_empty);
            umma_commit(&sh->out_full);
            umma_commit(&sh->empty[stage]);
          }
          __syncwarp();
          if (kStages == 1 && c + 1 < chunks) scores();
        }
      }
      if (elect_one()) umma_commit(&sh->drain);  // all MMAs are finished before TMEM is released
      __syncwarp();
      volatile int never = 0;
      mbar_wait_idle(&sh->drain, 0, &never);
    }
  } else if (warp >= 16) {
    // -------------------------------------------------------------------- outputs
    regs_down<kOutRegs>();
    const int quad = warp & 3, col = quad * 32 + lane;
    const uint32_t at = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    while (kOut && ok && walk.next(p, &x, warp == 16 && lane == 0)) {
      T* out = static_cast<T*>(a.out) + x.row * a.o_ts + x.h * a.o_hs + col;
      for (int c = 0; ok && c < x.n; c += kC, ++it) {
        const uint32_t slot = it % kGates;
        const int n = min(kC, x.n - c);
        wait(&sh->gate_full[slot], it / kGates);
        wait(&sh->out_full, it);
        if (!ok) break;
        tc_fence_after();
        const Gate& t = sh->gate[slot];
#pragma unroll 1
        for (int j0 = 0; j0 < kC; j0 += 16) {
          uint32_t u[16], w[16];
          tmem_ld16(at + kInter + j0, u);
          tmem_ld16(at + kIntra + j0, w);
          tmem_ld_wait();
          if (j0 + 16 == kC) {
            tc_fence_before();
            arrive(&sh->out_empty);
          }
          if (col < kDv) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float y = fmaf(t.before[j0 + j], __uint_as_float(u[j]), a.scale * __uint_as_float(w[j]));
              if (j0 + j < n) {
                T* o = out + (c + j0 + j) * a.o_ts;
                if constexpr (kIn == 2) *o = __float2half_rn(y);
                else *o = __float2bfloat16_rn(y);
              }
            }
          }
        }
        arrive(&sh->gate_empty[slot]);
      }
    }
  } else if (warp >= 8) {
    regs_down<kProductRegs>();
    const int quad = warp & 3, half = (warp - 8) >> 2;
    if (quad < 2) {
      // ------------------------------------------------------------------ P
      const int i = quad * 32 + lane;  // row: token i, columns [32 half, 32 half + 32)
      const uint32_t at = tmem + (static_cast<uint32_t>(quad * 32) << 16) + kScore + 32 * half;
      uint8_t* dst = smem + C::kPAt;
      while (kOut && ok && walk.next(p, &x)) {
        for (int c = 0; ok && c < x.n; c += kC, ++it) {
          const uint32_t slot = it % kGates, buffer = it & 1u;
          wait(&sh->gate_full[slot], it / kGates);
          wait(&sh->score_full[buffer], it >> 1);
          if (!ok) break;
          tc_fence_after();
          uint32_t s[32];
          tmem_ld32(at + 64 * buffer, s);
          tmem_ld_wait32(s);
          tc_fence_before();
          arrive(&sh->score_empty[buffer]);
          const Gate& t = sh->gate[slot];
          const float2 mine = t.sum[i];
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float2 other = t.sum[32 * half + j];
            const float f = ex2((mine.x - other.x) + (mine.y - other.y));
            s[j] = 32 * half + j <= i ? __float_as_uint(__uint_as_float(s[j]) * f) : 0u;
          }
          arrive(&sh->gate_empty[slot]);
          wait(&sh->p_empty, it ^ 1u);
          if (!ok) break;
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float a0 = __uint_as_float(s[8 * v + 2 * e]), a1 = __uint_as_float(s[8 * v + 2 * e + 1]);
              hi[e] = tops(a0, a1);
              lo[e] = pack_bf16x2(a0 - top(a0), a1 - top(a1));
            }
            const uint32_t o = place(i, 4 * half + v);
            *reinterpret_cast<uint4*>(dst + o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(dst + kBlock + o) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
          fence_proxy_async_smem();
          arrive(&sh->p_full);
        }
      }
    } else {
      // ------------------------------------------------------------------ decayed keys
      const int tid = (half * 2 + quad - 2) * 32 + lane;  // of 128
      constexpr int kVec = kDk / 8;
      const int col = tid % kVec, r0 = tid / kVec;
      const uint32_t from = kBlock + col / 8 * (2 * kBlock), to = C::kKeyAt + col / 8 * kBlock;
      while (ok && walk.next(p, &x)) {
        for (int c = 0; ok && c < x.n; c += kC, ++it) {
          const uint32_t slot = it % kGates, stage = it % kStages, buffer = it & 1u;
          wait(&sh->gate_full[slot], it / kGates);
          wait(&sh->full[stage], it / kStages);
          wait(&sh->key_empty[buffer], (it >> 1) ^ 1u);
          if (!ok) break;
          const Gate& t = sh->gate[slot];
          const uint8_t* src = smem + stage * C::kStage + from;
          uint8_t* dst = smem + to + buffer * 3 * C::kKeyPart;
#pragma unroll 2
          for (int r = r0; r < kC; r += 128 / kVec) {
            const uint32_t o = place(r, col & 7);
            const float w = t.after[r];
            const uint4 h = *reinterpret_cast<const uint4*>(src + o);
            const uint4 l = kIn == 2 ? *reinterpret_cast<const uint4*>(src + C::kQk + o) : make_uint4(0, 0, 0, 0);
            const uint32_t in[4] = {h.x, h.y, h.z, h.w}, in_lo[4] = {l.x, l.y, l.z, l.w};
            uint32_t part[3][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float x0 = __uint_as_float(in[e] << 16), x1 = __uint_as_float(in[e] & 0xFFFF0000u);
              if (kIn == 2) {
                x0 += __uint_as_float(in_lo[e] << 16);
                x1 += __uint_as_float(in_lo[e] & 0xFFFF0000u);
              }
              x0 *= w, x1 *= w;
              part[0][e] = tops(x0, x1);
              x0 -= top(x0), x1 -= top(x1);
              part[1][e] = tops(x0, x1);
              x0 -= top(x0), x1 -= top(x1);
              part[2][e] = tops(x0, x1);
            }
#pragma unroll
            for (int k = 0; k < 3; ++k)
              *reinterpret_cast<uint4*>(dst + k * C::kKeyPart + o) = make_uint4(part[k][0], part[k][1], part[k][2], part[k][3]);
          }
          fence_proxy_async_smem();
          arrive(&sh->key_full[buffer]);
          if (lane == 0) {
            mbar_arrive(&sh->empty[stage]);
            mbar_arrive(&sh->gate_empty[slot]);
          }
        }
      }
    }
  } else {
    // -------------------------------------------------------------------- states
    regs_up<kStateRegs>();
    constexpr int kN = kDk / 2;  // key rows of a thread
    const int quad = warp & 3, wg = warp >> 2, col = quad * 32 + lane;
    const uint32_t at = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const bool real = col < kDv;
    const int64_t mine = static_cast<int64_t>(wg) * kN * kDv + col;
    constexpr int64_t kState1 = static_cast<int64_t>(kDk) * kDv;
    while (ok && walk.next(p, &x, !kOut && warp == 0 && lane == 0)) {
      float S[kN];
      const auto load = [&](const float* src) {
#pragma unroll
        for (int d = 0; d < kN; ++d) S[d] = src && real ? src[mine + d * kDv] : 0.f;
      };
      const int64_t head = static_cast<int64_t>(x.h) * kState1;
      const auto slot_state = [&](int slot) { return p.states + (static_cast<int64_t>(slot) * a.heads + x.h) * kState1; };
      if (x.first) {
        float* copy = p.firsts + (static_cast<int64_t>(x.b) * a.heads + x.h) * kState1;
        // a sequence in pieces: its first kernel keeps the state, whose page the second may overwrite early
        load(!x.in ? nullptr : kOut && !x.last ? copy : x.in + head);
        if (!kOut && x.in && real) {
#pragma unroll
          for (int d = 0; d < kN; ++d) copy[mine + d * kDv] = S[d];
        }
      } else if (kOut) {
        load(slot_state(x.b));
        for (int slot = a.num_seqs + x.seq0 / p.piece; slot < x.slot; ++slot) {
          const float f = p.decays[static_cast<int64_t>(slot) * a.heads + x.h];
          const float* src = slot_state(slot);
          if (real) {
#pragma unroll
            for (int d = 0; d < kN; ++d) S[d] = fmaf(S[d], f, src[mine + d * kDv]);
          }
        }
      } else {
        load(nullptr);
      }
      for (int c = 0; ok && c < x.n; c += kC, ++it) {
        const uint32_t slot = it % kGates;
        if (kOut) {
          wait(&sh->state_empty, it ^ 1u);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int d0 = 0; d0 < kN; d0 += 32) {
            uint32_t hi[16], lo[16];
#pragma unroll
            for (int d = 0; d < 16; ++d) {
              const float s0 = S[d0 + 2 * d], s1 = S[d0 + 2 * d + 1];
              hi[d] = tops(s0, s1);
              lo[d] = pack_bf16x2(s0 - top(s0), s1 - top(s1));
            }
            tmem_st16(at + kState + (wg * kN + d0) / 2, hi);
            tmem_st16(at + kState + kDk / 2 + (wg * kN + d0) / 2, lo);
          }
          tmem_st_wait();
          tc_fence_before();
          arrive(&sh->state_full);
        }
        wait(&sh->gate_full[slot], it / kGates);
        wait(&sh->update_full, it);
        if (!ok) break;
        tc_fence_after();
        const float f = sh->gate[slot].all;
#pragma unroll
        for (int d0 = 0; d0 < kN; d0 += 16) {
          uint32_t u[16];
          tmem_ld16(at + kUpdate + wg * kN + d0, u);
          tmem_ld_wait();
          if (d0 + 16 == kN) {
            tc_fence_before();
            arrive(&sh->update_empty);
          }
#pragma unroll
          for (int d = 0; d < 16; ++d) S[d0 + d] = fmaf(S[d0 + d], f, __uint_as_float(u[d]));
        }
        arrive(&sh->gate_empty[slot]);
      }
      float* dst = kOut ? (x.last ? x.out + head : nullptr) : slot_state(x.slot);
      if (ok && dst && real) {
#pragma unroll
        for (int d = 0; d < kN; ++d) dst[mine + d * kDv] = S[d];
      }
    }
  }
  if (!ok && lane == 0) {
    set_error(a.err, RIMURU_DEV_TIMEOUT);
    sh->abort = 1;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 20) tmem_dealloc(tmem, 512);
}

template <typename T, int kDk, int kDv, bool kOut>
cudaError_t launch_one(const ChunkArgs& p, cudaStream_t s) {
  constexpr int smem = Cfg<T, kDk, kDv>::kSmem;
  auto* fn = linear_chunk_kernel<T, kDk, kDv, kOut>;
  static SmemOnce once;
  const cudaError_t e = once.set(reinterpret_cast<const void*>(fn), smem);
  if (e != cudaSuccess) return e;
  fn<<<std::min(p.units, p.l.sms), kThreads, smem, s>>>(p);
  return cudaGetLastError();
}
template <typename T, int kDk, int kDv>
cudaError_t launch(const ChunkArgs& p, cudaStream_t s) {
  if (p.piece > 0) {
    const cudaError_t e = launch_one<T, kDk, kDv, false>(p, s);
    if (e != cudaSuccess) return e;
  }
  return launch_one<T, kDk, kDv, true>(p, s);
}
template <typename T>
cudaError_t launch_dims(const ChunkArgs& p, cudaStream_t s) {
  if (p.l.key_dim == 128) return p.l.value_dim == 128 ? launch<T, 128, 128>(p, s) : launch<T, 128, 64>(p, s);
  return p.l.value_dim == 128 ? launch<T, 64, 128>(p, s) : launch<T, 64, 64>(p, s);
}

}  // namespace

LinearCut linear_cut(int heads, int key_dim, int value_dim, int sms, int num_seqs, int num_tokens, int max_new) {
  // Times in chunks of the second kernel: a chunk of the first costs 0.45, a unit's start one,
  // another kernel four, and a piece reads the states of those before it at about 0.3 each.
  const auto cost = [&](int piece) {
    const int64_t longest = piece > 0 ? std::min(piece, max_new) : max_new;
    const int64_t pieces = piece > 0 ? num_seqs + num_tokens / piece : num_seqs;
    const double chunks = (longest + kC - 1.0) / kC + 1.0;
    const double rounds = std::ceil(static_cast<double>(heads) * std::max<int64_t>(num_seqs, (num_tokens + longest - 1) / longest) / sms);
    const double even = heads * (num_tokens / static_cast<double>(kC) + pieces) / sms;
    const double t = std::max(rounds * chunks * (num_seqs > 1 ? 0.75 : 1.0), std::max(even, chunks));
    return piece > 0 ? 1.45 * t + 4.0 + 0.15 * (max_new / piece) : t;
  };
  LinearCut best;
  double least = cost(0);
  for (int piece = kC; piece < max_new && piece <= 65536; piece += piece < 1024 ? kC : piece / 16 / kC * kC) {
    if (num_tokens / piece > 512) continue;
    const double c = cost(piece);
    if (c < least) least = c, best.piece = piece;
  }
  best.pieces = num_seqs + (best.piece > 0 ? num_tokens / best.piece : 0);
  if (best.piece > 0) {
    const uint64_t state = 4ull * heads * key_dim * value_dim;
    best.state_bytes = (static_cast<uint64_t>(best.pieces) + num_seqs) * state + 4ull * best.pieces * heads;
  }
  return best;
}

cudaError_t launch_linear_chunks(const LinearArgs& a, const LinearCut& cut, void* workspace, int dtype, cudaStream_t s) {
  ChunkArgs p{};
  p.l = a;
  p.piece = cut.piece;
  p.units = cut.pieces * a.heads;
  const int64_t state = static_cast<int64_t>(a.heads) * a.key_dim * a.value_dim;
  p.states = static_cast<float*>(workspace);
  p.firsts = p.states + cut.pieces * state;
  p.decays = p.firsts + a.num_seqs * state;
  return dtype == RIMURU_BF16 ? launch_dims<__nv_bfloat16>(p, s) : launch_dims<__half>(p, s);
}

}  // namespace rimuru
