// Linear attention over prompts: 64 tokens (a chunk) at a time on the tensor cores.
//
// With G_i the sum of the decays of a chunk's tokens up to i, S the state before it and
// T the state after it, a head's chunk is
//   out_i = scale exp(G_i) (S^T q_i + sum_{j <= i} exp(-G_j) (q_i . k_j) v_j)
//   T     = exp(G_last) S + sum_j exp(G_last - G_j) k_j v_j^T.
// exp(-G_j) leaves fp32 where a chunk forgets more than 2^64.  There exp(G_i) outside the bracket is
// held between 2^-64 and 2^-63, and the power of two that is missing goes into the sum's weights and
// into q_i, exactly: what is left of S counts however little that is.
// All products are made transposed, with the value columns in the 128 lanes of TMEM and
// 64 tokens or the key columns across, so that every MMA has full height:
//   scores  Q K^T          (64 x 64; the lanes below take K K^T, which nobody reads)
//   inter   S^T Q^T        S^T in TMEM, as two bf16 parts that its owners write there: 2^-17 of it is lost
//   intra   V^T P^T        onto it; P = scores * decays, two bf16 parts in shared memory
//   update  V^T Kd         Kd = decayed keys, three bf16 parts: an fp32 number exactly
// Products of two lower parts (f16, inter and scores) are left out, 2^-16.
// S^T itself stays in the registers of eight warps in fp32 and takes each chunk's update
// there: sums inside the tensor cores truncate, and over thousands of tokens that would
// show.  f16 inputs are split into two bf16 parts in shared memory, exactly.
//
// Differences G_i - G_j are taken on sums in 64-bit fixed point, so that a huge decay
// early in a chunk costs the small ones after it nothing.
//
// Few heads and long sequences leave SMs without work, so sequences can be cut into
// pieces: a first kernel computes what each piece adds to the state and a second one
// starts every piece from the states of the pieces before it.
//
// Warps: 0-7 hold S; 8, 9, 12, 13 make P and a quarter of the decayed keys, 10, 11, 14, 15
// the rest of them; 16-19 write outputs; 20 and 23 issue MMAs, 21 sums up decays, 22 loads
// by TMA.  One CTA an SM; tiles, scores, outputs and decayed keys have two buffers each
// (f16 has twice the parts: one, and the next tiles behind it).
//
// One prompt of 8192 tokens, 32 heads on 16 key heads of 128 x 128, bf16: 118 us, 45 of
// them in the first kernel (token by token 4550 us); seven prompts of 558 to 1663 tokens 96,
// f16 208 and 170.  What bounds a chunk of the second kernel, 2.4 us, is instructions: 10,400 of them,
// 63 % of the issue slots, half of them in the cutting into parts; the tensor pipe is busy for
// a third.  On the way: loads by two warps of 16-byte copies 220 us, by TMA 150; packed fp32
// 141; 103 KiB of code, which the instruction cache fetched again and again (71 % of its hits
// missed the SM), to 56 KiB by short waits, rolled loops and units in shared memory 137 to 116.
#include <algorithm>
#include <cmath>
#include <cstddef>
#include <type_traits>

#include "device.cuh"
#include "kernels.h"
#include "kv_attn.h"
#include "linear.h"

namespace rimuru {
namespace {

using namespace dev;

constexpr int kC = 64;               // tokens of a chunk
constexpr uint32_t kBlock = 8192;    // 64 rows of 128 bytes, swizzled
constexpr int kGates = 4;            // chunks whose decays are ready
constexpr int kThreads = 768;
constexpr int kKeysByP = 16;         // keys of a chunk that the warps of P decay
constexpr int kStateRegs = 104, kProductRegs = 72, kOutRegs = 72, kOtherRegs = 56;
static_assert((2 * kStateRegs + 2 * kProductRegs + kOutRegs + kOtherRegs) * 128 <= 80 * kThreads, "");

struct alignas(16) Gate {  // read four numbers at a time
  float2 sum[kC];   // G in two parts whose differences are exact, log2
  float col[kC];    // exp(-G)
  float before[kC]; // scale * exp(G), at least 2^-64 of it
  float after[kC];  // exp(G_last - G)
  float all;        // exp(G_last)
  int wide;         // G leaves 2^-64: `col` is of no use, queries are scaled
  int pad[2];
};
static_assert(sizeof(Gate) % 16 == 0 && offsetof(Gate, col) % 16 == 0 && offsetof(Gate, before) % 16 == 0, "");
constexpr float kLeast = -64.f;   // of exp(G) outside the bracket, log2

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
constexpr int kUnits = 64;  // of a CTA

struct ChunkShared {
  Gate gate[kGates];
  Unit units[kUnits];
  uint64_t full[2], empty[2];             // loaded queries and values (f16: all tiles, split)
  uint64_t keys_full[2], keys_empty[2];   // loaded keys
  uint64_t raw, raw_empty;                // f16: all tiles before they are split
  uint64_t values_full, parts_empty;      // f16, second kernel: split values; queries' and keys' parts
  uint64_t gate_full[kGates], gate_empty[kGates];
  uint64_t seen[kGates];                  // second kernel: `bad` is known
  uint64_t safe[kGates];                  // values that are not finite have become zeros
  alignas(4) uint8_t bad[kGates][4];      // whether one may not be, in 32 columns each
  uint8_t bad_from[kGates][128];          // where one was: the column's first token that had one, or kC
  uint64_t score_full[2], score_empty[2];
  uint64_t key_full[2], key_empty[2];     // decayed keys
  uint64_t p_full, p_empty;
  uint64_t state_full, state_empty;       // parts of S
  uint64_t update_full, update_empty;
  uint64_t out_full[2], out_empty[2];
  uint64_t drain;
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
  // decayed keys twice; f16: once, and the next chunk's tiles as they are loaded [keys, queries, values]
  static constexpr int kKeyBufs = kIn == 1 ? 2 : 1;
  static constexpr uint32_t kKeyAt = kStages * kStage, kPAt = kKeyAt + kKeyBufs * 3 * kKeyPart;
  static constexpr uint32_t kRawAt = kPAt + 2 * kBlock;
  static constexpr uint32_t kSmem = kRawAt + (kIn == 1 ? 0 : kQk + kV) + 1024;
};

struct ChunkArgs {
  LinearArgs l;
  int q_one, k_one, v_one;  // heads that lie on one another (a stride of 0)
  int piece, units;
  float* states;  // [pieces][heads][key_dim][value_dim]: what pieces add, sequences' first ones whole
  float* firsts;  // [num_seqs][heads][...]: states before sequences that are cut
  float* decays;  // [pieces][heads]
};

__device__ __forceinline__ Unit find_unit(const ChunkArgs& p, int u, bool record) {
  const LinearArgs& a = p.l;
  Unit x{};
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
// 16-byte piece `c` of row r in a swizzled block of 128-byte rows.
__device__ __forceinline__ uint32_t place(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }
template <typename T>
__device__ __forceinline__ T not_a_number() {
  const uint16_t bits = 0x7FFF;
  return *reinterpret_cast<const T*>(&bits);
}
template <typename T>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    return pack_bf16x2(lo, hi);
  }
}
// The upper halves of two numbers as a pair of bf16: what is below is cut off.
__device__ __forceinline__ uint32_t tops(float lo, float hi) {
  return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}
__device__ __forceinline__ uint32_t tops(uint64_t x) { return tops(split(x).x, split(x).y); }
// The nearest bf16, which leave half as much as `tops` does: with `rest` 2^-17 of a number is lost, and it
// costs nothing (half as many outputs of a prompt are rounded the other way than the exact ones).
__device__ __forceinline__ uint32_t nearest(uint64_t x) { return pack_bf16x2(split(x).x, split(x).y); }
// Two bf16 as fp32.  The lower one moves up by a product, which is not the logic unit's work:
// with the cutting of parts that has more to do than any other here.
__device__ __forceinline__ uint64_t widen(uint32_t two) {
  return pair(__uint_as_float(two * 65536u), __uint_as_float(two & 0xFFFF0000u));
}
// Two numbers less those.
__device__ __forceinline__ uint64_t below(uint64_t x, uint32_t upper) { return fma2(widen(upper), pair(-1.f, -1.f), x); }
// That, as a pair of bf16.
__device__ __forceinline__ uint32_t rest(uint64_t x, uint32_t upper) {
  const float2 r = split(below(x, upper));
  return pack_bf16x2(r.x, r.y);
}

// Eight f16 as two bf16 parts: their 11 bits are 8, to the nearest, and the rest.
__device__ __forceinline__ void split_f16(const uint4& w, uint4* hi, uint4* lo) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&in[i]));
    h[i] = pack_bf16x2(f.x, f.y);
    l[i] = tops(below(pair(f.x, f.y), h[i]));
  }
  *hi = make_uint4(h[0], h[1], h[2], h[3]);
  *lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// Fixed point with 40 bits below the point.
__device__ __forceinline__ int64_t fixed_log2(float g) {
  g = fminf(fmaxf(g, -1400.f), 0.f);  // 2^-2000 is 0; decays above 0 are none
  constexpr float kHi = 1.4426950408889634f, kLo = 1.925963033500e-8f;  // log2(e)
  const float x = g * kHi;
  const float rest = fmaf(g, kHi, -x) + g * kLo;
  return __float2ll_rn(x * 0x1p40f) + __float2ll_rn(rest * 0x1p40f);
}
// In two parts: a multiple of 2^-6 below 2^17, and what is left, below 2^-6.
__device__ __forceinline__ float2 parts_of(int64_t G) {
  return make_float2(__int2float_rn(static_cast<int>(G >> 34)) * 0x1p-6f,
                     __uint2float_rn(static_cast<uint32_t>(static_cast<uint64_t>(G) >> 2)) * 0x1p-38f);
}
// 2^(a - b), of numbers in parts: the first ones' difference is exact.
__device__ __forceinline__ float exp2_of(float2 a, float2 b) {
  const float hi = a.x - b.x, n = rintf(hi);
  const float f = (hi - n) + (a.y - b.y);
  const int e = static_cast<int>(fminf(fmaxf(n, -127.f), 128.f)) + 127;
  // 2^f as its power series up to f^8, |f| <= 0.52: the rest is below 2^-31.  A chunk's whole decay
  // meets the state once a chunk, and the instruction's 2^-22 would add up.
  float y = 1.321548679e-6f;
  y = fmaf(y, f, 1.525273380e-5f);
  y = fmaf(y, f, 1.540353039e-4f);
  y = fmaf(y, f, 1.333355815e-3f);
  y = fmaf(y, f, 9.618129108e-3f);
  y = fmaf(y, f, 5.550410866e-2f);
  y = fmaf(y, f, 2.402265070e-1f);
  y = fmaf(y, f, 6.931471806e-1f);
  return fmaf(y, f, 1.f) * __int_as_float(e << 23);
}

// Waits for a phase in as few instructions as that takes: the loops of six kinds of warps
// together are what the instruction cache has to hold.  A try suspends the warp for up to a
// microsecond, and gives up after a million of them.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity) {
  uint32_t done, left = 1u << 20;
  do {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity), "r"(1000)
        : "memory");
  } while (!done && --left);
  return done;
}

template <typename T, int kDk, int kDv, bool kOut>
__global__ void __launch_bounds__(kThreads, 1)
    linear_chunk_kernel(const __grid_constant__ ChunkArgs p, const __grid_constant__ CUtensorMap tm_q,
                        const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
  using C = Cfg<T, kDk, kDv>;
  constexpr int kStages = C::kStages, kIn = C::kIn;
  constexpr int kKeyWarps = kOut ? 8 : 12;  // the first kernel has no outputs to make
  extern __shared__ uint8_t raw_smem[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ ChunkShared sh_;
  ChunkShared* sh = &sh_;
  const LinearArgs& a = p.l;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->full[i], kIn == 1 ? 1 : kKeyWarps);  // f16: the warps that split the tiles
      mbar_init(&sh->empty[i], kOut ? 2 : 1);      // both MMA warps
      mbar_init(&sh->keys_full[i], 1);
      mbar_init(&sh->keys_empty[i], (kOut ? 1 : 0) + kKeyWarps);
      mbar_init(&sh->score_full[i], 1);
      mbar_init(&sh->score_empty[i], 4);
      mbar_init(&sh->key_full[i], kKeyWarps);
      mbar_init(&sh->key_empty[i], 1);
      mbar_init(&sh->out_full[i], 1);
      mbar_init(&sh->out_empty[i], 4);
    }
    for (int i = 0; i < kGates; ++i) {
      mbar_init(&sh->gate_full[i], 1);
      mbar_init(&sh->seen[i], 4);
      mbar_init(&sh->safe[i], 1);
      mbar_init(&sh->gate_empty[i], kOut ? 8 + 4 + 1 + kKeyWarps : 8 + kKeyWarps);
    }
    mbar_init(&sh->raw, 1);
    mbar_init(&sh->raw_empty, kKeyWarps);
    mbar_init(&sh->values_full, 4);
    mbar_init(&sh->parts_empty, 2);  // scores, inter
    mbar_init(&sh->p_full, 4);
    mbar_init(&sh->p_empty, 1);
    mbar_init(&sh->state_full, 8);
    mbar_init(&sh->state_empty, 1);
    mbar_init(&sh->update_full, 1);
    mbar_init(&sh->update_empty, 8);
    mbar_init(&sh->drain, 2);
    fence_barrier_init();
  }
  if (warp == 20) {
    tmem_alloc(&sh->tmem_base, 512);
    tmem_relinquish();
  }
  // Units, the longest pieces first and every other round backwards: a CTA that got a long one
  // gets a short one next (seven prompts of 558 to 1663 tokens, 32 heads: 96 us, in the order of the
  // sequences 110).  More pieces than threads even out by themselves.
  const int slots = p.units / a.heads, ctas = gridDim.x;
  const bool sorted = slots <= kThreads && p.units > ctas;
  int* const length = reinterpret_cast<int*>(smem);  // nothing has been loaded yet
  int* const order = length + kThreads;
  if (sorted) {
    const int slot = threadIdx.x;
    int mine = 0;
    if (slot < slots) {
      const Unit y = find_unit(p, slot * a.heads, false);
      mine = y.ok && (kOut || !y.last) ? y.n : 0;
      length[slot] = mine;
    }
    __syncthreads();
    if (slot < slots) {
      int before = 0;
      for (int j = 0; j < slots; ++j) before += length[j] > mine || (length[j] == mine && j < slot);
      order[before] = slot;
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < kUnits; i += kThreads) {
    const int64_t u = static_cast<int64_t>(i) * ctas + (sorted && i % 2 ? ctas - 1 - blockIdx.x : blockIdx.x);
    Unit y{};
    if (u < p.units) {
      const int v = static_cast<int>(u);
      y = find_unit(p, sorted ? order[v / a.heads] * a.heads + v % a.heads : v, kOut);
      y.ok = y.ok && (kOut || !y.last);  // the first kernel is about pieces that others follow
    }
    sh->units[i] = y;
  }
  if (sorted) fence_proxy_async_smem();  // the lists lie where TMA is going to write
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  // columns of TMEM
  constexpr uint32_t kScore = 0, kOutAt = 128, kUpdate = 256, kState = 384;  // two buffers of scores and outputs
  bool ok = true;
  const auto wait = [&](uint64_t* bar, uint32_t phase) {
    ok = __all_sync(0xffffffffu, wait_for(bar, phase & 1u)) && ok;
  };
  // one arrival of a converged warp
  const auto arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  // Units of this CTA in order; every warp goes through them by itself.
  int next_unit = 0;
  Unit x{};
  const auto next = [&]() {
    while (next_unit < kUnits) {
      x = sh->units[next_unit++];
      if (x.ok) return true;
    }
    return false;
  };
  uint32_t it = 0;  // chunks so far

  // f16: a loaded block into its parts, 16 bytes a turn of each of `threads`; rows past `n` become zeros.
  const auto split_block = [&](const uint8_t* src, uint8_t* dst, uint32_t part, int n, int tid, int threads) {
#pragma unroll 2
    for (int v = tid; v < static_cast<int>(kBlock / 16); v += threads) {
      uint4 lo, hi = *reinterpret_cast<const uint4*>(src + 16 * v);
      if (v / 8 >= n) hi = make_uint4(0, 0, 0, 0);
      split_f16(hi, &hi, &lo);
      *reinterpret_cast<uint4*>(dst + 16 * v) = hi;
      *reinterpret_cast<uint4*>(dst + part + 16 * v) = lo;
    }
  };
  const uint8_t* const raw_tiles = smem + C::kRawAt;
  constexpr uint32_t kRawQ = C::kKb * kBlock, kRawV = 2 * kRawQ;
  // f16: the tiles have been loaded and the places of the queries' and keys' parts are free, which
  // the outputs of the last chunk need not be for that
  const auto wait_for_raw = [&]() {
    wait(&sh->raw, it);
    if (kOut) wait(&sh->parts_empty, it ^ 1u);
  };
  // Decayed keys of rows [r0, r1) of the chunk that begins at c, by vectors of eight.
  constexpr int kVec = kDk / 8;
  const auto decay_keys = [&](int c, int r0, int r1, int tid, int threads) {
    const uint32_t slot = it % kGates, stage = it % kStages, buffer = it % C::kKeyBufs;
    const int n = min(kC, x.n - c), col = tid % kVec;
    const Gate& t = sh->gate[slot];
    uint8_t* src = smem + stage * C::kStage + kBlock + col / 8 * (2 * kBlock);
    uint8_t* dst = smem + C::kKeyAt + col / 8 * kBlock + buffer * 3 * C::kKeyPart;
#pragma unroll 1
    for (int r = r0 + tid / kVec; r < r1; r += threads / kVec) {
      const uint32_t o = place(r, col & 7);
      const uint64_t w2 = pair(t.after[r], t.after[r]);
      uint4 h = *reinterpret_cast<const uint4*>(kIn == 1 ? src + o : raw_tiles + col / 8 * kBlock + o);
      if (r >= n) h = make_uint4(0, 0, 0, 0);
      uint32_t part[3][4];
      const uint32_t in[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint64_t y;
        if constexpr (kIn == 2) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&in[e]));
          y = pair(f.x, f.y);
        } else {
          y = widen(in[e]);
        }
        y = mul2(y, w2);
        part[0][e] = tops(y);
        y = below(y, part[0][e]);
        part[1][e] = tops(y);
        part[2][e] = tops(below(y, part[1][e]));
      }
#pragma unroll
      for (int k = 0; k < 3; ++k)
        *reinterpret_cast<uint4*>(dst + k * C::kKeyPart + o) = make_uint4(part[k][0], part[k][1], part[k][2], part[k][3]);
      if (kIn == 2 && kOut) {
        uint4 lo;
        split_f16(h, &h, &lo);
        *reinterpret_cast<uint4*>(src + o) = h;
        *reinterpret_cast<uint4*>(src + C::kQk + o) = lo;
      }
    }
  };
  const auto wait_for_keys = [&]() {
    const uint32_t slot = it % kGates;
    wait(&sh->gate_full[slot], it / kGates);
    if (kIn == 1) wait(&sh->keys_full[it % kStages], it / kStages);
    else wait_for_raw();
    wait(&sh->key_empty[it % C::kKeyBufs], (it / C::kKeyBufs) ^ 1u);
  };
  // What this warp wrote of the keys (and, f16, of other tiles) can be used.
  const auto give_keys = [&](bool read_all) {  // f16: whether this warp has read all it will of the loaded tiles
    fence_proxy_async_smem();
    arrive(&sh->key_full[it % C::kKeyBufs]);
    if (lane == 0) {
      mbar_arrive(kIn == 2 ? &sh->full[it % kStages] : &sh->keys_empty[it % kStages]);
      if (kIn == 2 && read_all) mbar_arrive(&sh->raw_empty);
    }
  };

  // Half of query i of a stage, times 2^e.  The state takes no other factor for each token.
  const auto scale_query = [&](uint8_t* base, int i, int half, float e) {
    // in two factors, which fp32 holds; the product then rounds to bf16's smallest numbers at most
    const int k = static_cast<int>(fmaxf(e, -252.f)), k0 = max(k, -126);
    const float f0 = __int_as_float((k0 + 127) << 23), f1 = __int_as_float((k - k0 + 127) << 23);
    const uint64_t f2 = pair(f0, f0), more = pair(f1, f1);
#pragma unroll 1
    for (int v = half; v < kIn * kVec; v += 2) {
      const int part = v / kVec, col = v - part * kVec;
      uint4* at = reinterpret_cast<uint4*>(base + part * C::kQk + col / 8 * (2 * kBlock) + place(i, col & 7));
      const uint4 x = *at;
      const uint32_t in[4] = {x.x, x.y, x.z, x.w};
      uint32_t y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 z = split(mul2(mul2(widen(in[k]), f2), more));
        y[k] = pack_bf16x2(z.x, z.y);
      }
      *at = make_uint4(y[0], y[1], y[2], y[3]);
    }
  };

  const auto products = [&]() {
    // P: a thread has row i (token i) and columns [32 half, 32 half + 32), eight at a time.  These
    // warps also decay some of the keys, so that all four schedulers do, and split the queries (f16).
    const int quad = warp & 3, half = (warp - 8) >> 2, i = quad * 32 + lane;
    const int tid = (half * 2 + quad) * 32 + lane;  // of 128
    const uint32_t at = tmem + (static_cast<uint32_t>(quad * 32) << 16) + kScore + 32 * half;
    uint8_t* dst = smem + C::kPAt;
    while (ok && next()) {
      for (int c = 0; ok && c < x.n; c += kC, ++it) {
        const uint32_t slot = it % kGates, buffer = it & 1u;
        wait_for_keys();
        if (!ok) break;
        decay_keys(c, kC - kKeysByP, kC, tid, 128);
        if (kIn == 2) {
          uint8_t* base = smem + it % kStages * C::kStage;
          for (int b = 0; b < C::kKb; ++b)
            split_block(raw_tiles + kRawQ + b * kBlock, base + 2 * b * kBlock, C::kQk, min(kC, x.n - c), tid, 128);
        }
        give_keys(true);
        wait(&sh->score_full[buffer], it >> 1);
        wait(&sh->p_empty, it ^ 1u);
        if (!ok) break;
        tc_fence_after();
        const Gate& t = sh->gate[slot];
        float2 sum = t.sum[i];
        // what exp(G_i) is held back by, a power of two
        sum = make_float2(sum.x >= kLeast ? 0.f : floorf(sum.x - kLeast), 0.f);
        const bool wide = t.wide;
        // the scores have been made: the query may change for its product with S, which waits for P then
        if (wide && sum.x < 0.f) scale_query(smem + it % kStages * C::kStage, i, half, sum.x);
        uint32_t next[8];
        tmem_ld8(at + 64 * buffer, next);
#pragma unroll 2
        for (int v = 0; v < 4; ++v) {
          uint64_t y[4];
          tmem_ld_wait8(next);
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = pair(__uint_as_float(next[2 * e]), __uint_as_float(next[2 * e + 1]));
          if (v < 3) tmem_ld8(at + 64 * buffer + 8 * (v + 1), next);
          const int j0 = 32 * half + 8 * v;
          if (!wide) {
            const ulonglong2 f0 = *reinterpret_cast<const ulonglong2*>(&t.col[j0]), f1 = *reinterpret_cast<const ulonglong2*>(&t.col[j0 + 4]);
            const uint64_t f[4] = {f0.x, f0.y, f1.x, f1.y};
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = mul2(y[e], f[e]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 o = *reinterpret_cast<const float4*>(&t.sum[j0 + 2 * e]);
              y[e] = mul2(y[e], pair(ex2((sum.x - o.x) + (sum.y - o.y)), ex2((sum.x - o.z) + (sum.y - o.w))));
            }
          }
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 z = split(y[e]);  // later tokens do not count
            const uint64_t w = pair(j0 + 2 * e <= i ? z.x : 0.f, j0 + 2 * e + 1 <= i ? z.y : 0.f);
            hi[e] = nearest(w);
            lo[e] = rest(w, hi[e]);
          }
          const uint32_t o = place(i, 4 * half + v);
          *reinterpret_cast<uint4*>(dst + o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(dst + kBlock + o) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        tc_fence_before();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sh->score_empty[buffer]);
          mbar_arrive(&sh->p_full);
          mbar_arrive(&sh->gate_empty[slot]);
        }
      }
    }
  };
  const auto keys = [&](int which) {
    constexpr int kThreads1 = 32 * (kOut ? 4 : 12);
    const int tid = which * 32 + lane;
    while (ok && next()) {
      for (int c = 0; ok && c < x.n; c += kC, ++it) {
        const int n = min(kC, x.n - c);
        uint8_t* v = smem + it % kStages * C::kStage + kIn * C::kQk;
        wait_for_keys();
        if (!ok) break;
        decay_keys(c, 0, kOut ? kC - kKeysByP : kC, tid, kThreads1);
        if (kIn == 2 && !kOut) {
          wait(&sh->empty[0], it ^ 1u);
          if (!ok) break;
          for (int b = 0; b < C::kVb; ++b) split_block(raw_tiles + kRawV + b * kBlock, v + b * kBlock, C::kV, n, tid, kThreads1);
        }
        if (kIn == 1 && n < kC) {  // values past the piece: 0 times what they hold may be NaN
          wait(&sh->full[it % kStages], it / kStages);
          if (!ok) break;
          for (int i = tid; i < (kC - n) * 8 * C::kVb; i += kThreads1) {
            const int b = i / ((kC - n) * 8), k = i - b * ((kC - n) * 8);
            *reinterpret_cast<uint4*>(v + b * kBlock + n * 128 + 16 * k) = make_uint4(0, 0, 0, 0);
          }
        }
        give_keys(!kOut);
        if (lane == 0) mbar_arrive(&sh->gate_empty[it % kGates]);
        if (kIn == 2 && kOut) {  // the values may come later than the keys
          wait(&sh->empty[0], it ^ 1u);
          if (!ok) break;
          for (int b = 0; b < C::kVb; ++b) split_block(raw_tiles + kRawV + b * kBlock, v + b * kBlock, C::kV, n, tid, kThreads1);
          fence_proxy_async_smem();
          arrive(&sh->values_full);
          if (lane == 0) mbar_arrive(&sh->raw_empty);
        }
      }
    }
  };

  if (warp >= 20) {
    regs_down<kOtherRegs>();
    if (warp == 22) {
      // ------------------------------------------------------------------ loads
      // Rows past the piece come along: their outputs are not written, their scores and decayed
      // keys are replaced by zeros, and the warps that decay keys clear their values.
      // bf16: keys have barriers of their own.  They are needed for less time than the other tiles,
      // and the warps that decay them then run ahead of the MMAs.
      while (ok && next()) {
        const int hq = p.q_one ? 0 : x.h / a.per_key_head, hk = p.k_one ? 0 : x.h / a.per_key_head;
        const int hv = p.v_one ? 0 : x.h;
        for (int c = 0; ok && c < x.n; c += kC, ++it) {
          const uint32_t stage = it % kStages;
          uint8_t* base = smem + stage * C::kStage;
          const int row = static_cast<int>(x.row) + c;
          const uint64_t pol = policy_evict_normal();
          uint64_t* bar = kIn == 2 ? &sh->raw : &sh->keys_full[stage];
          constexpr uint32_t kKeyBytes = C::kKb * kBlock, kRestBytes = ((kOut ? C::kKb : 0) + C::kVb) * kBlock;
          wait(kIn == 2 ? &sh->raw_empty : &sh->keys_empty[stage], (it / kStages) ^ 1u);
          if (!ok) break;
          if (elect_one()) {
            mbar_arrive_expect_tx(bar, kIn == 2 ? kKeyBytes + kRestBytes : kKeyBytes);
#pragma unroll
            for (int b = 0; b < C::kKb; ++b)
              tma_load_3d(kIn == 2 ? smem + C::kRawAt + b * kBlock : base + (2 * b + 1) * kBlock, &tm_k, bar, 64 * b, hk, row, pol);
          }
          __syncwarp();
          if (kIn == 1) {
            bar = &sh->full[stage];
            wait(&sh->empty[stage], (it / kStages) ^ 1u);
            if (!ok) break;
          }
          if (elect_one()) {
            if (kIn == 1) mbar_arrive_expect_tx(bar, kRestBytes);
#pragma unroll
            for (int b = 0; kOut && b < C::kKb; ++b)
              tma_load_3d(kIn == 2 ? smem + C::kRawAt + kRawQ + b * kBlock : base + 2 * b * kBlock, &tm_q, bar, 64 * b, hq, row, pol);
#pragma unroll
            for (int b = 0; b < C::kVb; ++b)
              tma_load_3d(kIn == 2 ? smem + C::kRawAt + kRawV + b * kBlock : base + kIn * C::kQk + b * kBlock, &tm_v, bar, 64 * b, hv, row, pol);
          }
          __syncwarp();
        }
      }
    } else if (warp == 21) {
      // ------------------------------------------------------------------ decays
      while (ok && next()) {
        const float* g = a.decay + x.row * a.g_ts + x.h * a.g_hs;
        constexpr int64_t kFar = 1ll << 50;  // 2^-1024 is 0, and the parts hold 2^17
        int64_t total = 0;
        bool nan = false;
        const int i = 2 * lane;
        float g0 = i < x.n ? g[i * a.g_ts] : 0.f, g1 = i + 1 < x.n ? g[(i + 1) * a.g_ts] : 0.f;
        for (int c = 0; ok && c < x.n; c += kC, ++it) {
          const uint32_t slot = it % kGates;
          const float now0 = g0, now1 = g1;
          const int next = c + kC + i;  // loaded before they are needed
          g0 = next < x.n ? g[next * a.g_ts] : 0.f;
          g1 = next + 1 < x.n ? g[(next + 1) * a.g_ts] : 0.f;
          const int64_t x1 = fixed_log2(now1);
          int64_t G1 = fixed_log2(now0) + x1;
#pragma unroll
          for (int m = 1; m < 32; m <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, G1, m);
            if (lane >= m) G1 += up;
          }
          const int64_t last = __shfl_sync(0xffffffffu, G1, 31);
          const uint32_t bad0 = __ballot_sync(0xffffffffu, now0 != now0);
          const uint32_t bad1 = __ballot_sync(0xffffffffu, now0 != now0 || now1 != now1);
          // a NaN counts for every token from its own on
          const uint32_t below = (2u << lane) - 1u;
          const bool nan0 = ((bad0 & below) | (bad1 & (below >> 1))) != 0, nan1 = (bad1 & below) != 0;
          const float none = __int_as_float(0x7FFFFFFF);
          float2 p0 = parts_of(G1 - x1), p1 = parts_of(G1);
          const float2 end = parts_of(last), zero = make_float2(0.f, 0.f);
          const float after0 = exp2_of(end, p0), after1 = exp2_of(end, p1), all = exp2_of(end, zero);
          wait(&sh->gate_empty[slot], (it / kGates) ^ 1u);
          if (!ok) break;
          Gate& t = sh->gate[slot];
          if (kOut) {
            const bool wide = !(end.x >= kLeast) || bad1 != 0;
            if (nan0) p0.x = none;
            if (nan1) p1.x = none;
            *reinterpret_cast<float4*>(&t.sum[i]) = make_float4(p0.x, p0.y, p1.x, p1.y);
            // less the power of two that P and q take; a NaN stays one
            const auto held = [](float2 x) { return x.x < kLeast ? make_float2(x.x - floorf(x.x - kLeast), x.y) : x; };
            *reinterpret_cast<float2*>(&t.before[i]) = make_float2(exp2_of(held(p0), zero) * a.scale, exp2_of(held(p1), zero) * a.scale);
            *reinterpret_cast<float2*>(&t.col[i]) = make_float2(exp2_of(zero, p0), exp2_of(zero, p1));
            if (lane == 0) t.wide = wide;
          }
          *reinterpret_cast<float2*>(&t.after[i]) = make_float2(after0, after1);
          if (lane == 0) t.all = bad1 ? none : all;
          total = max(total + last, -kFar);
          nan |= bad1 != 0;
          arrive(&sh->gate_full[slot]);
        }
        if (!kOut && lane == 0) {
          p.decays[static_cast<int64_t>(x.slot) * a.heads + x.h] =
              nan ? __int_as_float(0x7FFFFFFF) : exp2_of(parts_of(total), make_float2(0.f, 0.f));
        }
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
        if (kIn == 1) wait(&sh->keys_full[stage], scored / kStages);
        wait(&sh->score_empty[buffer], (scored >> 1) ^ 1u);
        tc_fence_after();
        if (ok && elect_one()) {
          const uint32_t q0 = base_lo + stage * (C::kStage / 16), k0 = q0 + kBlock / 16;
          uint32_t more = 0;
#pragma unroll 1
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
          umma_commit(kIn == 1 ? &sh->keys_empty[stage] : &sh->parts_empty);
        }
        __syncwarp();
        ++scored;
      };
      // Two warps issue, since an MMA of this size takes longer to issue than it runs: one the
      // scores and the updates, which need no state, the other what makes outputs.
      while (warp == 20 && ok && next()) {
        const int chunks = (x.n + kC - 1) / kC;
        if (kOut && chunks > 0) scores();
        for (int c = 0; ok && c < chunks; ++c, ++it) {
          const uint32_t stage = it % kStages, buffer = it % C::kKeyBufs;
          const uint32_t v0 = cols_lo + (stage * C::kStage + kIn * C::kQk) / 16;
          wait(&sh->full[stage], it / kStages);
          wait(&sh->key_full[buffer], it / C::kKeyBufs);
          if (kIn == 2 && kOut) wait(&sh->values_full, it);
          wait(&sh->update_empty, it ^ 1u);
          tc_fence_after();
          if (ok && elect_one()) {
            const uint32_t k0 = cols_lo + (C::kKeyAt + buffer * 3 * C::kKeyPart) / 16;
            uint32_t more = 0;
            // small parts first: what the sum cuts off is then small too
#pragma unroll 1
            for (int pv = kIn - 1; pv >= 0; --pv) {
#pragma unroll 1
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
            umma_commit(&sh->empty[stage]);
          }
          __syncwarp();
          if (kOut && c + 1 < chunks) scores();
        }
      }
      while (kOut && warp == 23 && ok && next()) {
        const int chunks = (x.n + kC - 1) / kC;
        for (int c = 0; ok && c < chunks; ++c, ++it) {
          const uint32_t stage = it % kStages;
          const uint32_t v0 = cols_lo + (stage * C::kStage + kIn * C::kQk) / 16;
          wait(&sh->gate_full[it % kGates], it / kGates);
          if (sh->gate[it % kGates].wide) wait(&sh->p_full, it);  // with P come the scaled queries
          arrive(&sh->gate_empty[it % kGates]);
          wait(&sh->full[stage], it / kStages);
          wait(&sh->state_full, it);
          wait(&sh->out_empty[it & 1u], (it >> 1) ^ 1u);
          tc_fence_after();
          const uint32_t out = tb + kOutAt + 64 * (it & 1u);
          if (ok && elect_one()) {
            const uint32_t q0 = base_lo + stage * (C::kStage / 16);
            uint32_t more = 0;
#pragma unroll 1
            for (int pair = (kIn == 2 ? 2 : 1); pair >= 0; --pair) {  // (hi, 1), (lo, 0), (hi, 0) of S and Q
              const uint32_t ps = pair == 1 ? kDk / 2 : 0, pq = pair == 2 ? C::kQk / 16 : 0;
#pragma unroll
              for (int s = 0; s < kDk / 16; ++s) {
                umma_f16_ts_lo<kHi, id_inter>(out, tb + kState + ps + 8 * s,
                                              q0 + pq + s / 4 * (2 * kBlock / 16) + s % 4 * 2, more);
                more = 1;
              }
            }
            umma_commit(&sh->state_empty);
            if (kIn == 2) umma_commit(&sh->parts_empty);
          }
          __syncwarp();
          wait(&sh->p_full, it);
          // The values past the piece have been cleared.  f16 clears them as it splits them, and its one buffer of
          // keys may be a phase further by now: nothing of the next chunk's keys waits for these products.
          if (kIn == 1) wait(&sh->key_full[it % C::kKeyBufs], it / C::kKeyBufs);
          if (kIn == 2) wait(&sh->values_full, it);
          // P is 0 for tokens to come, and 0 times a NaN or an infinity is NaN.  So values that are not
          // finite, which the update has taken to the state by now, become zeros before the outputs'
          // products, and their columns of the outputs NaN from their tokens on.
          const uint32_t slot = it % kGates;
          wait(&sh->seen[slot], it / kGates);
          if (*reinterpret_cast<const uint32_t*>(sh->bad[slot]) != 0) {
#pragma unroll 1
            for (int col = lane; col < kDv; col += 32) {
              int from = kC;
              uint8_t* const tile = smem + stage * C::kStage + kIn * C::kQk + col / 64 * kBlock + col % 8 * 2;
#pragma unroll 1
              for (int r = min(kC, x.n - c * kC) - 1; r >= 0; --r) {
                auto* const y = reinterpret_cast<uint16_t*>(tile + place(r, col / 8 % 8));
                if ((*y & 0x7F80u) != 0x7F80u) continue;  // f16: of the upper part
                from = r;
                *y = 0;
                if (kIn == 2) y[C::kV / 2] = 0;
              }
              sh->bad_from[slot][col] = static_cast<uint8_t>(from);
            }
            fence_proxy_async_smem();
          }
          arrive(&sh->safe[slot]);
          tc_fence_after();
          if (ok && elect_one()) {
            const uint32_t p0 = base_lo + C::kPAt / 16;
#pragma unroll 1
            for (int pair = (kIn == 2 ? 2 : 1); pair >= 0; --pair) {  // (1, hi), (0, lo), (0, hi) of V and P
              const uint32_t pp = pair == 1 ? kBlock / 16 : 0, pv = pair == 2 ? C::kV / 16 : 0;
#pragma unroll
              for (int s = 0; s < kC / 16; ++s) {
                umma_f16_lo<kHi, kHi, id_intra>(out, v0 + pv + 128 * s, p0 + pp + 2 * s, 1u);
              }
            }
            umma_commit(&sh->p_empty);
            umma_commit(&sh->out_full[it & 1u]);
            umma_commit(&sh->empty[stage]);
          }
          __syncwarp();
        }
      }
      if (elect_one()) umma_commit(&sh->drain);  // all MMAs are finished before TMEM is released
      __syncwarp();
      wait_for(&sh->drain, 0);
    }
  } else if (warp >= 16) {
    // -------------------------------------------------------------------- outputs
    regs_down<kOutRegs>();
    if (!kOut) keys(warp - 8);
    const int quad = warp & 3, col = quad * 32 + lane;
    const uint32_t at = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    while (kOut && ok && next()) {
      // Lanes are value columns.  Four neighbouring lanes change places for four tokens, so that each
      // writes four columns of one token.
      T* out = static_cast<T*>(a.out) + (x.row + (lane & 3)) * a.o_ts + x.h * a.o_hs + (col & ~3);
      for (int c = 0; ok && c < x.n; c += kC, ++it) {
        const uint32_t slot = it % kGates;
        const int n = min(kC, x.n - c) - (lane & 3);
        wait(&sh->gate_full[slot], it / kGates);
        wait(&sh->safe[slot], it / kGates);
        wait(&sh->out_full[it & 1u], it >> 1);
        if (!ok) break;
        tc_fence_after();
        const Gate& t = sh->gate[slot];
        T* o = out + c * a.o_ts;
        const int64_t four = 4 * a.o_ts;
        uint32_t ahead[8];
        tmem_ld8(at + kOutAt + 64 * (it & 1u), ahead);
#pragma unroll 2
        for (int h = 0; h < kC; h += 8) {
          uint32_t u[8];
          tmem_ld_wait8(ahead);
#pragma unroll
          for (int j = 0; j < 8; ++j) u[j] = ahead[j];
          if (h + 8 < kC) tmem_ld8(at + kOutAt + 64 * (it & 1u) + h + 8, ahead);
#pragma unroll
          for (int j = 0; j < 8; j += 4) {
            const ulonglong2 before = *reinterpret_cast<const ulonglong2*>(&t.before[h + j]);
            const auto two = [](uint32_t lo, uint32_t hi) { return pair(__uint_as_float(lo), __uint_as_float(hi)); };
            const float2 f01 = split(mul2(before.x, two(u[j], u[j + 1])));
            const float2 f23 = split(mul2(before.y, two(u[j + 2], u[j + 3])));
            // even lanes take tokens 0 and 2, odd ones 1 and 3
            const bool odd = lane & 1, up = lane & 2;
            const float g0 = __shfl_xor_sync(0xffffffffu, odd ? f01.x : f01.y, 1);
            const float g1 = __shfl_xor_sync(0xffffffffu, odd ? f23.x : f23.y, 1);
            const uint32_t y0 = odd ? pack<T>(g0, f01.y) : pack<T>(f01.x, g0);
            const uint32_t y1 = odd ? pack<T>(g1, f23.y) : pack<T>(f23.x, g1);
            // the lower lanes of each four keep tokens 0 and 1, the upper ones 2 and 3
            const uint32_t mine = up ? y1 : y0, other = __shfl_xor_sync(0xffffffffu, up ? y0 : y1, 2);
            if (col < kDv && h + j < n) *reinterpret_cast<uint2*>(o) = up ? make_uint2(other, mine) : make_uint2(mine, other);
            o += four;
          }
        }
        if (sh->bad[slot][quad] && col < kDv) {  // a warp's lanes alike
          __syncwarp();  // after what the neighbours have written
          const int rows = min(kC, x.n - c);
#pragma unroll 1
          for (int r = sh->bad_from[slot][col]; r < rows; ++r)
            static_cast<T*>(a.out)[(x.row + c + r) * a.o_ts + x.h * a.o_hs + col] = not_a_number<T>();
        }
        tc_fence_before();
        arrive(&sh->out_empty[it & 1u]);
        if (lane == 0) mbar_arrive(&sh->gate_empty[slot]);
      }
    }
  } else if (warp >= 8) {
    regs_down<kProductRegs>();
    if (kOut && (warp & 3) < 2) products();
    else keys(kOut ? (warp - 8) / 4 * 2 + (warp & 1) : warp - 8);
  } else {
    // -------------------------------------------------------------------- states
    regs_up<kStateRegs>();
    constexpr int kN = kDk / 2;  // key rows of a thread
    const int quad = warp & 3, wg = warp >> 2, col = quad * 32 + lane;
    const uint32_t at = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const bool real = col < kDv;
    const int64_t mine = static_cast<int64_t>(wg) * kN * kDv + col;
    constexpr int64_t kState1 = static_cast<int64_t>(kDk) * kDv;
    while (ok && next()) {
      uint64_t S[kN / 2];  // pairs of key rows
      const auto load = [&](const float* src) {
#pragma unroll
        for (int d = 0; d < kN; d += 2)
          S[d / 2] = src && real ? pair(src[mine + d * kDv], src[mine + (d + 1) * kDv]) : 0ull;
      };
      const int64_t head = static_cast<int64_t>(x.h) * kState1;
      const auto store = [&](float* dst) {
#pragma unroll
        for (int d = 0; d < kN; d += 2) {
          const float2 y = split(S[d / 2]);
          dst[mine + d * kDv] = y.x;
          dst[mine + (d + 1) * kDv] = y.y;
        }
      };
      const auto slot_state = [&](int slot) { return p.states + (static_cast<int64_t>(slot) * a.heads + x.h) * kState1; };
      if (x.first) {
        float* copy = p.firsts + (static_cast<int64_t>(x.b) * a.heads + x.h) * kState1;
        // a sequence in pieces: its first kernel keeps the state, whose page the second may overwrite early
        load(!x.in ? nullptr : kOut && !x.last ? copy : x.in + head);
        if (!kOut && x.in && real) store(copy);
      } else if (kOut) {
        load(slot_state(x.b));
        for (int slot = a.num_seqs + x.seq0 / p.piece; slot < x.slot; ++slot) {
          const float f = p.decays[static_cast<int64_t>(slot) * a.heads + x.h];
          const float* src = slot_state(slot);
          if (real) {
#pragma unroll
            for (int d = 0; d < kN; d += 2)
              S[d / 2] = fma2(S[d / 2], pair(f, f), pair(src[mine + d * kDv], src[mine + (d + 1) * kDv]));
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
              hi[d] = nearest(S[d0 / 2 + d]);
              lo[d] = rest(S[d0 / 2 + d], hi[d]);
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
        for (int d0 = 0; d0 < kN; d0 += 32) {
          uint32_t u[32];
          tmem_ld32(at + kUpdate + wg * kN + d0, u);
          tmem_ld_wait32(u);
          if (d0 + 32 == kN) {
            tc_fence_before();
            arrive(&sh->update_empty);
          }
#pragma unroll
          for (int d = 0; d < 32; d += 2)
            S[(d0 + d) / 2] = fma2(S[(d0 + d) / 2], pair(f, f), pair(__uint_as_float(u[d]), __uint_as_float(u[d + 1])));
        }
        if (kOut && wg == 0) {
          // row 0 has a product of every value of the column in it
          const bool bad = __any_sync(0xffffffffu, real && !(fabsf(split(S[0]).x) < INFINITY));
          if (lane == 0) sh->bad[slot][quad] = bad;
          arrive(&sh->seen[slot]);
        }
        arrive(&sh->gate_empty[slot]);
      }
      float* dst = kOut ? (x.last ? x.out + head : nullptr) : slot_state(x.slot);
      if (ok && dst && real) store(dst);
    }
  }
  if (!ok && lane == 0) set_error(a.err, RIMURU_DEV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 20) tmem_dealloc(tmem, 512);
}

template <typename T, int kDk, int kDv, bool kOut>
cudaError_t launch_one(const ChunkArgs& p, const CUtensorMap* tm, cudaStream_t s) {
  constexpr int smem = Cfg<T, kDk, kDv>::kSmem;
  auto* fn = linear_chunk_kernel<T, kDk, kDv, kOut>;
  static SmemOnce once;
  const cudaError_t e = once.set(reinterpret_cast<const void*>(fn), smem);
  if (e != cudaSuccess) return e;
  const int ctas = std::max(std::min(p.units, p.l.sms), (p.units + kUnits - 1) / kUnits);
  fn<<<ctas, kThreads, smem, s>>>(p, tm[0], tm[1], tm[2]);
  return cudaGetLastError();
}
template <typename T, int kDk, int kDv>
cudaError_t launch(const ChunkArgs& p, const CUtensorMap* tm, cudaStream_t s) {
  if (p.piece > 0) {
    const cudaError_t e = launch_one<T, kDk, kDv, false>(p, tm, s);
    if (e != cudaSuccess) return e;
  }
  return launch_one<T, kDk, kDv, true>(p, tm, s);
}
template <typename T>
cudaError_t launch_dims(const ChunkArgs& p, const CUtensorMap* tm, cudaStream_t s) {
  if (p.l.key_dim == 128) return p.l.value_dim == 128 ? launch<T, 128, 128>(p, tm, s) : launch<T, 128, 64>(p, tm, s);
  return p.l.value_dim == 128 ? launch<T, 64, 128>(p, tm, s) : launch<T, 64, 64>(p, tm, s);
}

}  // namespace

LinearCut linear_cut(int heads, int key_dim, int value_dim, int sms, int num_seqs, int num_tokens, int max_new) {
  // Times in chunks of the second kernel: a chunk of the first costs 0.45, a unit's start one,
  // another kernel four, and a piece reads the states of those before it at about 0.3 each.  Several
  // sequences seldom are all as long as the longest: 0.75 of that.  (32 heads of 128: 2048 tokens whole 71.5 us,
  // in pieces of 512 47.3; 3 x 2048 whole 73.3, in pieces of 1408 89; 32,768 whole 1002, pieces of 1728 414; 2 x 4096
  // takes pieces of 1088, 132, where 2048 would take 118.)
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

int launch_linear_chunks(const LinearArgs& a, const LinearCut& cut, void* workspace, int dtype, cudaStream_t s) {
  ChunkArgs p{};
  p.l = a;
  p.piece = cut.piece;
  p.units = cut.pieces * a.heads;
  const int64_t state = static_cast<int64_t>(a.heads) * a.key_dim * a.value_dim;
  p.states = static_cast<float*>(workspace);
  p.firsts = p.states + cut.pieces * state;
  p.decays = p.firsts + a.num_seqs * state;
  CUtensorMap tm[3];
  const int key_heads = a.heads / a.per_key_head;
  const auto map = [&](CUtensorMap* m, const void* x, int64_t ts, int64_t hs, int heads, int dim, int* one) {
    *one = heads == 1 || hs == 0;
    if (ts >= 1ll << 39 || hs >= 1ll << 39)
      return fail(RIMURU_ERR_UNSUPPORTED, "token and head strides must be below 2^39");
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(*one ? 1 : heads),
                                static_cast<cuuint64_t>(a.num_tokens)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(*one ? dim : hs) * 2, static_cast<cuuint64_t>(ts) * 2};
    const cuuint32_t box[3] = {64, 1, kC};
    return make_bf16_map(m, const_cast<void*>(x), 3, dims, strides, box);
  };
  int st = map(&tm[0], a.q, a.q_ts, a.q_hs, key_heads, a.key_dim, &p.q_one);
  if (st == RIMURU_OK) st = map(&tm[1], a.k, a.k_ts, a.k_hs, key_heads, a.key_dim, &p.k_one);
  if (st == RIMURU_OK) st = map(&tm[2], a.v, a.v_ts, a.v_hs, a.heads, a.value_dim, &p.v_one);
  if (st != RIMURU_OK) return st;
  const cudaError_t e = dtype == RIMURU_BF16 ? launch_dims<__nv_bfloat16>(p, tm, s) : launch_dims<__half>(p, tm, s);
  return e == cudaSuccess ? RIMURU_OK : fail(RIMURU_ERR_CUDA, kv_cuda_msg("linear attention launch", e));
}

}  // namespace rimuru
