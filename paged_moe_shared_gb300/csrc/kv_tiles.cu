// Attention of many query rows (prompts, chunks, drafted tokens of wide groups)
// over the 8-bit paged cache.
//
// Bound: the tensor cores (4 head_dim operations per query head and key).  Rows
// are (query, head of the group) pairs, so the heads that share a key/value
// head share its tiles.  Per 128-token tile of keys and 128 rows:
//   S = Q K^T   8 bits x 8 bits: K is multiplied as it lies in the page, Q as a sum
//               of 8-bit parts into one fp32 accumulator: two parts cost what one
//               bf16 product costs, without widening K.  The first part is e4m3 (4
//               significant bits), the rest e5m2 (3 bits, and small enough numbers):
//               with the row scaled to (224, 448], two parts hold a bf16 element
//               exactly down to 2^-6 of that scale and within 2^-14 below, three an
//               f16 element exactly down to 2^-6 and within 2^-17 below;
//   O += P V    f16 x f16: P rounded to f16 stays in TMEM as the A operand; the
//               codes of V are widened (exactly) by four warps on their way to
//               shared memory.
// The V scale 2^k of a page is added to the score, x + k, so that the weight that
// meets the codes stays bounded; the row sum takes the weight without it by an
// exact multiplication.  Weights are relative to a reference that follows the
// row's largest x + k only when 64 weights add up to more than 2^8 times the
// weight at the reference; then the softmax warps rescale O in TMEM.
//
// Two softmax warpgroups alternate on two score buffers ("items"), so that the
// tensor cores work on one while the other is in softmax.  With head_dim <= 128
// and units of 256 rows the items are two query tiles (each K and V tile serves
// 256 rows, a row is a thread).  With one query tile the items are successive key
// tiles: where O fits the tensor memory twice (head_dim <= 128) the warpgroups take
// them in turns, each with a reference, a sum and an O of its own that are added up
// at the end; with head_dim 256 both work on each item and halve its columns.
//
// 2048 rows x 32 heads after 6144 keys, 32/4 heads of 128: 207 us with the join, 1.16
// PFLOP/s (0.59 of cuBLAS bf16; f16 208 us); about 3,500 cycles a 256 x 128 tile whose MMAs take
// 3,072 (of them 1,024 for the second halves of the scores, see the MMA warps).  16
// sequences of 24 to 40 rows over 900 to 6600 keys: 29.4 us (f16 30.9).  What bounds both is the
// chain scores -> softmax -> weights -> MMA, 150 to 300 cycles a hand-over, with the
// two chains in flight that the tensor memory holds.
//
// The block is launched with 128 registers a thread, and every instance spills 168 to 280
// bytes a thread; what that costs was not measured.
//
// Warps 0-3 and 4-7: softmax.  8-11: widening V.  12: K copies, and the pages and
// scales of each key tile for the others.  13 and 15: MMAs.  14: V copies.
#include <cuda_fp8.h>

#include <algorithm>

#include "kv_attn.h"

namespace rimuru {
namespace {

using namespace dev;

constexpr int kThreads = 512;
constexpr int kMetaRing = 8;
constexpr int kGroups = kTileTokens / 16;
constexpr float kWeightTop = 7.f;     // a weight at the reference is 2^7
constexpr float kMostSum = 32768.f;   // of 64 weights, so that none passes 2^15: f16 ends at 2^16
constexpr float kNoRef = -1e30f;     // the reference of a row that has seen no key

template <int kD, int kTiles, int kQParts>
struct TileCfg {
  static constexpr int kRowBytes = kD < 128 ? kD : 128;  // bytes of a K or Q row in one slab
  static constexpr int kSlabs = kD / kRowBytes;
  static constexpr int kSlabBytes = 128 * kRowBytes;
  static constexpr int kKBytes = kSlabs * kSlabBytes;           // one K tile
  // One query tile whose O fits the tensor memory twice: the warpgroups take key tiles in turns.
  static constexpr bool kTurns = kTiles == 1 && kD <= 128;
  // K tiles.  In turns an even number: within a unit a slot then belongs to one of the two MMA warps.
  static constexpr int kKRing = kTurns ? 4 : kD <= 128 ? 3 : 2;
  static constexpr int kQBytes = kQParts * kTiles * kKBytes;    // [part][tile][slab][128 rows]
  static constexpr int kVTok = kD <= 128 ? 64 : 32;             // tokens of a V stage
  static constexpr int kVStages = kTileTokens / kVTok;          // stages of a tile
  static constexpr int kVBytes = kVTok * kD * 2;                // [64 f16 of a token: 128 bytes][tokens]
  static constexpr bool kWide = kQParts == 3 && (kD == 256 || kTiles == 2);  // Q takes 96 KiB
  static constexpr int kVRing = kWide ? 2 : 4;
  static constexpr int kVRaw = kVTok * kD;                      // codes of a stage
  static constexpr int kFifo = kD == 256 ? (kWide ? 2 : 3) : kTiles == 2 || kQParts == 3 ? 4 : 6;  // stages of codes
  static constexpr int kStage = kD == 64 ? 8 * 4096 : 0;        // output staging; else in Q's place
  static constexpr int kSmem =
      1024 + kQBytes + kKRing * kKBytes + kVRing * kVBytes + kFifo * kVRaw + kStage;
  static constexpr uint32_t kO = 256;                           // TMEM column of O; scores are at 0 and 128
  static constexpr int kIssuers = kTiles == 2 || kTurns ? 2 : 1;     // MMA warps
  static constexpr int kScoreN = kTiles == 1 && !kTurns ? 128 : 64;  // keys of one batch of scores
};

struct __align__(16) Meta {  // a 16-token group of a tile
  float k;      // scale of K
  float add;    // log2 of the scale of V
  float inv;    // 1 / scale of V
  int page;     // -1: none
};
struct TileShared {
  uint64_t k_full[4], k_empty[4];
  uint64_t v_full[4], v_empty[4];
  uint64_t raw_full[6], raw_empty[6];
  uint64_t meta_full[kMetaRing];
  uint64_t q_full;
  uint64_t o_full[2];
  uint64_t s_full[2][2], p_full[2][2], o_half[2];  // by halves of the key tile
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  RunStart run;
  uint64_t scratch[16];
  Meta meta[kMetaRing][kGroups];
  uint32_t seen[kMetaRing][4];    // a bit per token of the tile: its group has a page
  int4 span[kMetaRing];           // tokens [x, y) of the tile count (and have pages if z); w: head
  float row_scale[2][128];        // of each row: score per unit of S and K scale
  float other[2][128];            // one query tile: row maxima of the halves
  float row_sum[2][128];          // and their sums
};

// Two 16-bit numbers of type T as floats, and the larger ones of two pairs.
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t x) {
  if constexpr (std::is_same<T, __half>::value) return __half22float2(*reinterpret_cast<const __half2*>(&x));
  else return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
}
template <typename T>
__device__ __forceinline__ uint32_t max2(uint32_t x, uint32_t y) {
  using T2 = std::conditional_t<std::is_same<T, __half>::value, __half2, __nv_bfloat162>;
  const T2 z = __hmax2(*reinterpret_cast<const T2*>(&x), *reinterpret_cast<const T2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&z);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) { return pack_bf16x2(a, b); }
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Score per unit of S: the row's factor times the scale of K.  Both may be tiny (a row of zeros, scale 0,
// a page of zeros: 2^-60), and a masked S, -inf, times a factor that has become 0 would be NaN: 2^-120
// is added, which vanishes beside a factor above 2^-95, and below that no S (at most 2^26) gives a score
// that counts.  (A maximum in its place would cost an instruction: a chunk of 2048 took 207.6 us, not 205.3.)
__device__ __forceinline__ float score_factor(float row, float k) { return fmaf(row, k, 0x1p-120f); }
// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)),
        "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
// Holds in all 256 softmax threads (barrier 2).
__device__ __forceinline__ bool softmax_and(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\t"
      "setp.ne.u32 a, %1, 0;\n\t"
      "bar.red.and.pred b, 2, 256, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}\n"
      : "=r"(r)
      : "r"(v ? 1u : 0u)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ bool softmax_or(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\t"
      "setp.ne.u32 a, %1, 0;\n\t"
      "bar.red.or.pred b, 2, 256, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}\n"
      : "=r"(r)
      : "r"(v ? 1u : 0u)
      : "memory");
  return r != 0;
}
// Registers per thread of a warpgroup; the four groups' shares add up to the 4 x 128
// that the block was launched with (2 x 160 + 2 x 96 = 512).
constexpr int kSoftmaxRegs = 160, kOtherRegs = 96;
template <int kRegs>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
// Byte offset of byte d of row r in a swizzled K-major block.
template <int kRowBytes>
__device__ __forceinline__ int swz(int r, int d) {
  if (kRowBytes == 128) return r * 128 + ((((d >> 4) ^ r) & 7) << 4) + (d & 15);
  return r * 64 + ((((d >> 4) ^ (r >> 1)) & 3) << 4) + (d & 15);
}
// Four e4m3 codes as f16 numbers.
__device__ __forceinline__ uint2 widen(uint32_t w) {
  uint2 r;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}\n"
      : "=r"(r.x), "=r"(r.y)
      : "r"(w));
  return r;
}

template <typename T, int kD, int kTiles>
__global__ void __launch_bounds__(kThreads, 1)
    kv_tiles_kernel(const __grid_constant__ AttnArgs p, const __grid_constant__ CUtensorMap tm,
                    const __grid_constant__ CUtensorMap tm_v) {
  constexpr int kQParts = std::is_same<T, __nv_bfloat16>::value ? 2 : 3;
  using C = TileCfg<kD, kTiles, kQParts>;
  constexpr int kSlabs = C::kSlabs, kRowBytes = C::kRowBytes;
  constexpr uint32_t kSwizzle = kRowBytes == 128 ? 2 : 4;
  constexpr uint32_t kAtom = 8 * kRowBytes;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + C::kQBytes;
  uint8_t* sV = sK + C::kKRing * C::kKBytes;
  uint8_t* sRaw = sV + C::kVRing * C::kVBytes;
  __shared__ TileShared sh_;
  TileShared* sh = &sh_;
  volatile int* abort = &sh->abort;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sh->k_full[i], 1);
      mbar_init(&sh->k_empty[i], kTiles);
      mbar_init(&sh->v_full[i], 4);
      mbar_init(&sh->v_empty[i], kTiles);
    }
    for (int i = 0; i < 6; ++i) {
      mbar_init(&sh->raw_full[i], 1);
      mbar_init(&sh->raw_empty[i], 4);
    }
    for (int i = 0; i < kMetaRing; ++i) mbar_init(&sh->meta_full[i], 1);
    mbar_init(&sh->q_full, C::kTurns ? 9 : 8);  // the softmax warps, and in turns MMA warp 15
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->s_full[i][0], 1);
      mbar_init(&sh->s_full[i][1], 1);
      mbar_init(&sh->p_full[i][0], 4);
      mbar_init(&sh->p_full[i][1], 4);
      mbar_init(&sh->o_half[i], 1);
      mbar_init(&sh->o_full[i], 1);
    }
    mbar_init(&sh->drain, C::kIssuers);
    sh->abort = 0;
    fence_barrier_init();
    prefetch_tmap(&tm);
    prefetch_tmap(&tm_v);
  }
  if (warp == 13) {
    tmem_alloc(&sh->tmem_base, 512);
    tmem_relinquish();
  }
  grid_dep_wait();  // lengths, tables, q and the cache come from earlier kernels
  grid_dep_launch();
  if (p.direct) {
    find_unit<T>(p, blockIdx.x, &sh->run);
  } else {
    find_run(p, blockIdx.x, sh->scratch, &sh->run);
    if (threadIdx.x == 0) p.cuts[blockIdx.x] = make_int4(0, 0, 0, 0);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  const int P = p.g.page_tokens, log_p = 31 - __clz(P);
  RunWalk walk;
  walk.begin_run(p, sh->run);
  Segment g;

  if (warp >= 12) {
    regs_down<kOtherRegs>();
    if (warp == 12) {
      // -------------------------------------------------------------- K copies
      // The warp holds the ids and scales of 32 pages, one per lane (`boxes`
      // pages are a tile), and the ids of the next 32.
      const uint64_t pol = policy_evict_last();  // other query tiles read the same keys
      const int boxes = kTileTokens >> log_p, groups = P / 16;
      uint32_t tile = 0;
      bool ok = true;
      while (ok && walk.next(p, &g)) {
        const int lo = p.window > 0 ? max(0, g.s.len - g.s.n + g.i0 - p.window + 1) : 0;
        const int32_t* row = p.s.table + g.b * p.s.table_stride;
        const auto page_at = [&](int c) {  // page c of the sequence, -1 when none of its tokens count
          int page = -1;
          if (c << log_p < g.s.len && (c + 1) << log_p > lo && c < g.t1 * boxes) {
            page = row[c];
            if (page < 0 || page >= p.g.num_pages) {
              set_error(p.g.err, RIMURU_DEV_BAD_PAGE);
              page = -1;
            }
          }
          return page;
        };
        int c = g.t0 * boxes + lane, at = 32;
        int ahead = page_at(c), page = -1;
        float ks = 0.f, vs = 0.f;
        const int y = g.h << log_p;  // first K row of the head in a page
        for (int t = g.t0; ok && t < g.t1; ++t, ++tile) {
          if (at == 32) {
            page = ahead;
            ks = vs = 0.f;
            if (page >= 0) {
              const float* sc = p.g.scales + static_cast<int64_t>(page) * 2 * p.g.kv_heads + g.h;
              ks = sc[0];
              vs = sc[p.g.kv_heads];
            }
            c += 32;
            ahead = page_at(c);
            at = 0;
          }
          const int mine = __shfl_sync(0xffffffffu, page, (at + lane) & 31);  // for lanes below `boxes`
          const bool copies = lane < boxes && mine >= 0;
          const uint32_t which = __ballot_sync(0xffffffffu, copies);
          const uint32_t i = tile % C::kKRing;
          ok = mbar_wait_idle(&sh->k_empty[i], ((tile / C::kKRing) & 1u) ^ 1u, abort);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&sh->k_full[i], __popc(which) * P * kD);
          __syncwarp();
          if (copies) {
#pragma unroll
            for (int sl = 0; sl < kSlabs; ++sl)
              tma_load_3d(sK + i * C::kKBytes + sl * C::kSlabBytes + (lane << log_p) * kRowBytes, &tm,
                          &sh->k_full[i], sl * kRowBytes, y, mine, pol);
          }
          // The tile's pages and scales by groups of 16 tokens.  Their last readers, eight
          // tiles back, were done before the K tile just waited for could be reused.
          const uint32_t m = tile % kMetaRing;
          if (lane >= at && lane < at + boxes) {
            const int e = static_cast<int>(__float_as_uint(vs) >> 23) - 127;
            const Meta x = {page >= 0 ? ks : 1.f, page >= 0 ? static_cast<float>(e) : 0.f,
                            page >= 0 ? __uint_as_float(static_cast<uint32_t>(127 - e) << 23) : 0.f, page};
            for (int k = 0; k < groups; ++k) sh->meta[m][(lane - at) * groups + k] = x;
          }
          if (lane < 4) {  // 32 tokens a word: a page of 64 fills two, of 16 half of one
            const uint32_t two = log_p == 4 ? which >> (2 * lane) & 3u
                                            : (which >> (lane >> (log_p - 5)) & 1u) * 3u;
            sh->seen[m][lane] = (two & 1u ? 0xFFFFu : 0u) | (two & 2u ? 0xFFFF0000u : 0u);
          }
          if (lane == 0) {
            const int first = max(0, lo - t * kTileTokens), last = min(kTileTokens, g.s.len - t * kTileTokens);
            sh->span[m] = make_int4(first, last, which == (1u << boxes) - 1u, g.h);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh->meta_full[m]);
          at += boxes;
        }
      }
      if (!ok && lane == 0) {
        set_error(p.g.err, RIMURU_DEV_TIMEOUT);
        sh->abort = 1;
      }
      // every copy this warp issued must have landed before the CTA exits
      volatile int never = 0;
      for (uint32_t j = tile > C::kKRing ? tile - C::kKRing : 0u; j < tile; ++j)
        mbar_wait_idle(&sh->k_full[j % C::kKRing], (j / C::kKRing) & 1u, &never);
    } else if (warp == 13 || (C::kIssuers == 2 && warp == 15)) {
      // ------------------------------------------------------------------ MMAs
      // Items: (key tile, query tile) pairs in order; item i uses score buffer i & 1.
      // Weights lie in the same buffer, each half of 64 keys over its own scores, so
      // the scores of half h of item i + 2 follow the output of half h of item i, and
      // are there when its softmax warps come back (with 128 keys at a time they
      // waited 1,250 of 3,900 cycles a tile for them).  MMAs of one thread run in the
      // order they were issued.
      // The whole warp walks and waits, and one lane issues: addresses stay
      // warp-uniform (issued from a one-lane branch, an MMA took 160 cycles to issue
      // instead of the 64 it runs).
      constexpr uint32_t id_s = idesc_f8_f32(128, C::kScoreN, false, false, false);
      constexpr uint32_t id_rest = id_s | kIdescAE5m2;  // the parts of Q after the first
      constexpr uint32_t id_o = idesc_f16_f32(128, kD, false, /*b_mn=*/true);
      constexpr uint32_t kHiQK = desc_hi(kAtom, kSwizzle), kHiV = desc_hi(1024, 2);
      const uint32_t tb = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t q_lo = __shfl_sync(0xffffffffu, desc_lo(smem_u32(sQ), 16), 0);
      const uint32_t k_lo = __shfl_sync(0xffffffffu, desc_lo(smem_u32(sK), 16), 0);
      const uint32_t v_lo = __shfl_sync(0xffffffffu, desc_lo(smem_u32(sV), C::kVTok * 128), 0);
      // Two warps issue, each for one query tile or turn: an MMA takes as long to issue as
      // it runs, and while one warp waits on its barriers the other's are under way.
      const int mine = C::kIssuers == 2 && warp == 15 ? 1 : 0;
      uint32_t item0 = 0, tile = 0, seg = 0;
      bool ok = true;
      const auto wait = [&](uint64_t* bar, uint32_t phase) {
        ok = ok && mbar_wait_idle(bar, phase, abort);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
      };
      // The scores of key tile kt, its half h (128 keys at a time: h is 0), into `buffer`.
      constexpr int kLastHalf = 128 / C::kScoreN - 1;
      const auto scores = [&](uint32_t kt, uint32_t buffer, int h) {
        const uint32_t slot = kt % C::kKRing;
        if (h == 0) wait(&sh->k_full[slot], (kt / C::kKRing) & 1u);
        if (ok && elect_one()) {
          const uint32_t a0 = q_lo + (kTiles == 2 ? mine : 0) * (C::kKBytes / 16);
          const uint32_t b0 = k_lo + slot * (C::kKBytes / 16) + h * (64 * kRowBytes / 16);
          const uint32_t d = tb + 128 * buffer + 64 * h;
#pragma unroll
          for (int part = 0; part < kQParts; ++part) {
#pragma unroll
            for (int sl = 0; sl < kSlabs; ++sl) {
#pragma unroll
              for (int k = 0; k < kRowBytes / 32; ++k) {
                const uint32_t a = a0 + (part * kTiles * C::kKBytes + sl * C::kSlabBytes) / 16 + 2 * k;
                const uint32_t b = b0 + sl * (C::kSlabBytes / 16) + 2 * k;
                if (part == 0) umma_f8_lo<kHiQK, kHiQK, id_s>(d, a, b, (sl | k) != 0 ? 1u : 0u);
                else umma_f8_lo<kHiQK, kHiQK, id_rest>(d, a, b, 1u);
              }
            }
          }
          umma_commit(&sh->s_full[buffer][h]);
          if (h == kLastHalf) umma_commit(&sh->k_empty[slot]);
        }
        __syncwarp();
      };
      constexpr int kStep = C::kTurns ? 2 : 1;       // key tiles from one item of this warp's to the next
      constexpr int kAhead = C::kIssuers == 2 ? kStep : 2;  // from an item to the next one in its buffer
      const auto buffer_of = [&](int n) { return kTiles == 2 ? static_cast<uint32_t>(mine) : (item0 + n) & 1u; };
      while (__any_sync(0xffffffffu, ok && walk.next(p, &g))) {
        const int tiles = __shfl_sync(0xffffffffu, g.t1 - g.t0, 0);
        // In turns this unit may have no key tile for warp 15, and then nobody waits for it.  Its
        // arrival for each unit keeps Q's phases from passing it: a barrier waited for by parity
        // must not be two phases ahead of its waiter, nor may a waiter skip one.
        if (C::kTurns && mine == 1 && lane == 0) mbar_arrive(&sh->q_full);
        wait(&sh->q_full, seg & 1u);
        const int n0 = C::kTurns ? mine : 0;
        for (int n = n0; n < min(tiles, n0 + kAhead); n += kStep) {
#pragma unroll
          for (int h = 0; h <= kLastHalf; ++h) scores(tile + n, buffer_of(n), h);
        }
        for (int n = n0; ok && n < tiles; n += kStep) {
          const uint32_t buffer = buffer_of(n), item = item0 + (kTiles == 2 ? 2 * n + mine : n);
          const uint32_t o = tb + C::kO + (kTiles == 2 || C::kTurns ? mine : 0) * kD;
#pragma unroll
          for (int st = 0; st < C::kVStages; ++st) {
            constexpr int kPer = C::kVStages / 2;  // stages of a half
            const uint32_t v = (tile + n) * C::kVStages + st, slot = v % C::kVRing;
            wait(&sh->v_full[slot], (v / C::kVRing) & 1u);
            if (st % kPer == 0) wait(&sh->p_full[buffer][st / kPer], (item >> 1) & 1u);
            if (ok && elect_one()) {
              const uint32_t b0 = v_lo + slot * (C::kVBytes / 16);
              const uint32_t a0 = tb + 128 * buffer + 64 * (st / kPer) + C::kVTok / 2 * (st % kPer);
#pragma unroll
              for (int k = 0; k < C::kVTok / 16; ++k)  // 16 tokens: eight columns of P, 16 rows of V
                umma_f16_ts_lo<kHiV, id_o>(o, a0 + 8 * k, b0 + 128 * k, (st + k != 0) || n >= kStep ? 1u : 0u);
              umma_commit(&sh->v_empty[slot]);
              if (st == kPer - 1) umma_commit(&sh->o_half[buffer]);
              if (st == C::kVStages - 1) umma_commit(&sh->o_full[buffer]);
            }
            __syncwarp();
            if (kLastHalf == 1 && n + kAhead < tiles) scores(tile + n + kAhead, buffer, st);
          }
          if (kLastHalf == 0 && n + kAhead < tiles) scores(tile + n + kAhead, buffer, 0);
        }
        item0 += tiles * kTiles;
        tile += tiles;
        ++seg;
      }
      if (!ok && lane == 0) {
        set_error(p.g.err, RIMURU_DEV_TIMEOUT);
        sh->abort = 1;
      }
      if (elect_one()) umma_commit(&sh->drain);  // all MMAs are finished before TMEM is released
      __syncwarp();
      volatile int never = 0;
      mbar_wait_idle(&sh->drain, 0, &never);
    } else if (warp == 14) {
      // -------------------------------------------------------------- V copies
      // A box is a page's tokens, at most a stage's; lane l copies box l of a stage.
      const uint64_t pol = policy_evict_last();
      const int per = min(P, C::kVTok), boxes = C::kVTok / per;
      const uint32_t total = sh->run.tiles() * C::kVStages;
      uint32_t slot = 0, phase = 1;
      bool ok = true;
      uint32_t v = 0;
#pragma unroll 1
      for (; v < total; ++v) {
        const uint32_t tile = v / C::kVStages, m = tile % kMetaRing;
        ok = mbar_wait_idle(&sh->meta_full[m], (tile / kMetaRing) & 1u, abort);
        ok = ok && mbar_wait_idle(&sh->raw_empty[slot], phase, abort);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        const int tok = v % C::kVStages * C::kVTok + lane * per;
        const int page = lane < boxes ? sh->meta[m][tok >> 4].page : -1;
        const uint32_t which = __ballot_sync(0xffffffffu, page >= 0);
        if (lane == 0) mbar_arrive_expect_tx(&sh->raw_full[slot], __popc(which) * per * kD);
        __syncwarp();
        if (page >= 0)
          tma_load_3d(sRaw + slot * C::kVRaw + lane * per * kD, &tm_v, &sh->raw_full[slot], 0,
                      ((p.g.kv_heads + sh->span[m].w) << log_p) + (tok & (P - 1)), page, pol);
        if (++slot == C::kFifo) slot = 0, phase ^= 1u;
      }
      if (!ok && lane == 0) {
        set_error(p.g.err, RIMURU_DEV_TIMEOUT);
        sh->abort = 1;
      }
      // every copy this warp issued must have landed before the CTA exits
      volatile int never = 0;
      for (uint32_t j = v > C::kFifo ? v - C::kFifo : 0u; j < v; ++j)
        mbar_wait_idle(&sh->raw_full[j % C::kFifo], (j / C::kFifo) & 1u, &never);
    }
  } else if (warp >= 8) {
    regs_down<kOtherRegs>();
    // --------------------------------------------------------------- widening V
    // A stage is kVTok tokens: thread `t128` takes 16 codes (chunk c) of the tokens
    // r0, r0 + kStep, ...
    constexpr int kChunks = kD / 16, kStep = 128 / kChunks, kPer = C::kVTok / kStep;
    const int t128 = threadIdx.x - 256, c = t128 % kChunks, r0 = t128 / kChunks;
    const int ch = 2 * (c & 3);  // its chunks of eight f16 in a 128-byte row: ch and ch + 1
    uint8_t* const dst0 = sV + (c >> 2) * (C::kVTok * 128) + r0 * 128;
    const uint8_t* const src0 = sRaw + r0 * kD + 16 * c;
    bool ok = true;
    const uint32_t total = sh->run.tiles() * C::kVStages;
    uint32_t v_slot = 0, v_phase = 1, raw_slot = 0, raw_phase = 0;
#pragma unroll 1
    for (uint32_t v = 0; v < total; ++v) {
      ok = mbar_wait_idle(&sh->raw_full[raw_slot], raw_phase, abort);
      ok = ok && mbar_wait_idle(&sh->v_empty[v_slot], v_phase, abort);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      // slots that no counted token owns may hold anything, and 0 * NaN is not 0
      const uint32_t m = v / C::kVStages % kMetaRing;
      const int4 span = sh->span[m];
      const bool all = span.x <= 0 && span.y >= kTileTokens && span.z;
      const int r_tile = v % C::kVStages * C::kVTok + r0;
      uint8_t* const dst = dst0 + v_slot * C::kVBytes;
      const uint8_t* const src = src0 + raw_slot * C::kVRaw;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        uint4 x = *reinterpret_cast<const uint4*>(src + k * kStep * kD);
        if (!all) {
          const int r = r_tile + k * kStep;
          if (r < span.x || r >= span.y || sh->meta[m][r >> 4].page < 0) x = make_uint4(0, 0, 0, 0);
        }
        const uint2 f0 = widen(x.x), f1 = widen(x.y), f2 = widen(x.z), f3 = widen(x.w);
        const int r = r0 + k * kStep;
        *reinterpret_cast<uint4*>(dst + k * kStep * 128 + (((ch ^ r) & 7) << 4)) = make_uint4(f0.x, f0.y, f1.x, f1.y);
        *reinterpret_cast<uint4*>(dst + k * kStep * 128 + ((((ch + 1) ^ r) & 7) << 4)) =
            make_uint4(f2.x, f2.y, f3.x, f3.y);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sh->v_full[v_slot]);
        mbar_arrive(&sh->raw_empty[raw_slot]);
      }
      if (++v_slot == C::kVRing) v_slot = 0, v_phase ^= 1u;
      if (++raw_slot == C::kFifo) raw_slot = 0, raw_phase ^= 1u;
    }
    if (!ok && lane == 0) {
      set_error(p.g.err, RIMURU_DEV_TIMEOUT);
      sh->abort = 1;
    }
  } else {
    // ---------------------------------------------------------------- softmax
    regs_up<kSoftmaxRegs>();
    const int wg = warp >> 2, quad = warp & 3;
    const int row = quad * 32 + lane;  // row of the query tile, and TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const int qt = kTiles == 2 ? wg : 0;             // query tile
    constexpr bool kTurns = C::kTurns, kHalves = kTiles == 1 && !kTurns;  // kHalves: both have a part of each tile
    const uint32_t tO = tmem + C::kO + (kHalves ? 0 : wg) * kD + lane_off;
    const uint32_t group_mul = 65536u / p.group + 1;  // r / group = r * group_mul >> 16 for r < 256
    uint32_t tile = 0, item0 = 0;
    bool ok = true;
    while (ok && walk.next(p, &g)) {
      const int rows = (g.i1 - g.i0) * p.group;
      // keys [j_lo, j_hi) of this thread's row; rows past the unit see every column and are
      // not written
      const int r = qt * 128 + row, qi = static_cast<int>(r * group_mul >> 16), gi = r - qi * p.group;
      const bool real = r < rows;
      // Q of the warp's 32 rows, as parts (with one query tile the two warpgroups take 16
      // each).  A lane holds eight elements; kLanes lanes are a row.  The 16 bytes of a lane
      // come into the places of its first two parts, all rows at once, and are replaced by the
      // parts, four rows at a time so that their shuffles and conversions overlap (one after the
      // other, ragged prompts at head_dim 256 took 115 us instead of 103).
      constexpr int kLanes = kD / 8, kRows = 32 / kLanes;  // rows of one load
      constexpr int kSteps = (kTiles == 2 ? 32 : 16) / kRows;
      constexpr int kPart = kTiles * C::kKBytes;
      const int row0 = quad * 32 + (kTiles == 2 ? 0 : 16 * wg) + lane / kLanes;  // + k * kRows
      const int d0q = lane % kLanes * 8;
      const T* q_base = static_cast<const T*>(p.q) + (g.s.row0 + g.i0) * p.q_ts + g.h * p.group * p.q_hs + d0q;
      uint8_t* const q_dst = sQ + qt * C::kKBytes + d0q / kRowBytes * C::kSlabBytes;
      if (kTiles == 1 && !(ok = softmax_and(ok))) break;  // Q's place has been left by all warps
#pragma unroll 4
      for (int k = 0; k < kSteps; ++k) {
        const int rl = row0 + k * kRows, rr = qt * 128 + rl, i = static_cast<int>(rr * group_mul >> 16);
        uint8_t* dst = q_dst + swz<kRowBytes>(rl, d0q % kRowBytes);
        if (rr < rows) {
          const T* src = q_base + i * p.q_ts + (rr - i * p.group) * p.q_hs;
          cp_async8(smem_u32(dst), src);
          cp_async8(smem_u32(dst + kPart), src + 4);
        } else {
          *reinterpret_cast<uint2*>(dst) = make_uint2(0, 0);
          *reinterpret_cast<uint2*>(dst + kPart) = make_uint2(0, 0);
        }
      }
      cp_async_wait_all();
      constexpr int kBatch = 4;  // rows whose chains of shuffles and conversions overlap
#pragma unroll 1
      for (int k0 = 0; k0 < kSteps; k0 += kBatch) {
        uint32_t raw[kBatch][4], top[kBatch];
        uint8_t* dst[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          dst[k] = q_dst + swz<kRowBytes>(row0 + (k0 + k) * kRows, d0q % kRowBytes);
          const uint2 lo = *reinterpret_cast<const uint2*>(dst[k]), hi = *reinterpret_cast<const uint2*>(dst[k] + kPart);
          raw[k][0] = lo.x, raw[k][1] = lo.y, raw[k][2] = hi.x, raw[k][3] = hi.y;
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          top[k] = max2<T>(max2<T>(raw[k][0] & 0x7FFF7FFFu, raw[k][1] & 0x7FFF7FFFu),
                           max2<T>(raw[k][2] & 0x7FFF7FFFu, raw[k][3] & 0x7FFF7FFFu));
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) {
#pragma unroll
          for (int k = 0; k < kBatch; ++k) top[k] = max2<T>(top[k], __shfl_xor_sync(0xffffffffu, top[k], o));
        }
        __half2 x[kBatch][4];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const float2 both = unpack2<T>(top[k]);
          const float amax = fmaxf(both.x, both.y);
          // power of two that brings the row's largest magnitude into (224, 448]; the sign of
          // the scale goes into Q, so that a larger S is always a larger score
          const uint32_t ab = __float_as_uint(amax);
          const int e = max(-100, min(100, static_cast<int>(ab >> 23) - 127 - 8 + ((ab & 0x7FFFFFu) > 0x600000u)));
          const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23 | (p.scale_log2 < 0.f ? 0x80000000u : 0u));
          if (lane % kLanes == 0)  // an infinite query gives NaN
            sh->row_scale[qt][row0 + (k0 + k) * kRows] =
                amax <= 3.4028234664e38f ? __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * fabsf(p.scale_log2)
                                         : __int_as_float(0x7FFFFFFF);
          // f16 holds the scaled values exactly above 2^-14, and within 2^-25 below
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2<T>(raw[k][i]);
            x[k][i] = __floats2half2_rn(f.x * inv, f.y * inv);
          }
        }
#pragma unroll
        for (int part = 0; part < kQParts; ++part) {
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            uint32_t c[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const __nv_fp8_interpretation_t type = part == 0 ? __NV_E4M3 : __NV_E5M2;
              c[i] = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(x[k][i]), __NV_SATFINITE, type);
              if (part + 1 < kQParts)
                x[k][i] = __hsub2(x[k][i], __half2(__nv_cvt_fp8x2_to_halfraw2(
                                               static_cast<__nv_fp8x2_storage_t>(c[i]), type)));
            }
            *reinterpret_cast<uint2*>(dst[k] + part * kPart) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->q_full);
      if (kTiles == 1 && !(ok = softmax_and(ok))) break;  // the other half of the row scales
      const float c_row = sh->row_scale[qt][row];  // score per unit of S and K scale
      const int pos = g.s.len - g.s.n + g.i0 + qi;
      const int j_hi = real ? min(pos + 1, g.s.len) : 0x7FFFFFFF;
      const int j_lo = real && p.window > 0 ? max(0, pos - p.window + 1) : 0;
      float ref = kNoRef, l = 0.f;
      const int n_tiles = g.t1 - g.t0;
      for (int n = kTurns ? wg : 0; n < n_tiles; n += kTurns ? 2 : 1) {
        const int t = g.t0 + n;
        const uint32_t item = item0 + (kTiles == 2 ? 2 * n + wg : n), slot = item & 1u;
        const uint32_t m = (tile + n) % kMetaRing;
        ok = mbar_wait_idle(&sh->meta_full[m], ((tile + n) / kMetaRing) & 1u, abort) && ok;
        // whether some row of the warp does not see all of a half, by halves
        uint32_t edges = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint2 seen = *reinterpret_cast<const uint2*>(&sh->seen[m][2 * h]);
          const int j0 = t * kTileTokens + 64 * h;
          if (__any_sync(0xffffffffu, j_lo > j0 || j_hi < j0 + 64 || (seen.x & seen.y) != 0xFFFFFFFFu)) edges |= 1u << h;
        }
        const uint32_t tS = tmem + 128 * slot + lane_off;
        // Half a tile, 64 columns, at a time; with kHalves each warpgroup has its half.
        // The loop is kept rolled: past the first 10 KiB of instructions, which the warps of a
        // scheduler share, a warp runs three times slower.
#pragma unroll 1
        for (int h = kHalves ? wg : 0; h < (kHalves ? wg + 1 : 2); ++h) {
          uint32_t v[64], w[32];
          ok = mbar_wait_idle(&sh->s_full[slot][C::kScoreN == 128 ? 0 : h], (item >> 1) & 1u, abort) && ok;
          ok = __all_sync(0xffffffffu, ok);
          if (!kHalves && !ok) break;
          tc_fence_after();
          tmem_ld32(tS + 64 * h, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
          tmem_ld32(tS + 64 * h + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
          tmem_ld_wait32(*reinterpret_cast<uint32_t(*)[32]>(&v[0]));
          tmem_ld_wait32(*reinterpret_cast<uint32_t(*)[32]>(&v[32]));
          bool sees = true;
          if (edges >> h & 1u) {  // -inf where the row does not see
            const int j0 = t * kTileTokens + 64 * h;
            const int lo = max(0, min(64, j_lo - j0)), hi = max(0, min(64, j_hi - j0));
            const uint2 seen = *reinterpret_cast<const uint2*>(&sh->seen[m][2 * h]);
            uint64_t see = (hi == 64 ? ~0ull : (1ull << hi) - 1) & (lo == 64 ? 0ull : ~0ull << lo);
            see &= static_cast<uint64_t>(seen.y) << 32 | seen.x;
            sees = see != 0;
#pragma unroll
            for (int k = 0; k < 64; ++k) v[k] = see >> k & 1u ? v[k] : 0xFF800000u;
          }
          float got;
          for (bool settled = false;; settled = true) {
            // The weights with the reference as it stands: x + k of a 16-column group is S * mul
            // + add.  Their sum says whether a score passes the reference by too much: only then
            // (and for a row's first keys) the largest score is looked for, the reference moved
            // and the weights taken again.
            const float shift = ref == kNoRef ? 0.f : kWeightTop - ref;
            float raw = 0.f;
            got = 0.f;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float4 kv = *reinterpret_cast<const float4*>(&sh->meta[m][4 * h + q]);
              const float mul = score_factor(c_row, kv.x), a = kv.y + shift;
              float2 sum = make_float2(0.f, 0.f);
#pragma unroll
              for (int k = 0; k < 16; k += 2) {
                const float2 x = fma2(make_float2(__uint_as_float(v[16 * q + k]), __uint_as_float(v[16 * q + k + 1])),
                                      make_float2(mul, mul), make_float2(a, a));
                const float2 y = make_float2(ex2(x.x), ex2(x.y));
                sum = add2(sum, y);
                const __half2 hh = __floats2half2_rn(y.x, y.y);
                w[8 * q + k / 2] = *reinterpret_cast<const uint32_t*>(&hh);
              }
              raw += sum.x + sum.y;
              got += (sum.x + sum.y) * kv.z;
            }
            const bool redo = !settled && ((ref == kNoRef && sees) || raw > kMostSum);
            if (!kHalves) {
              if (!__any_sync(0xffffffffu, redo)) break;
            } else {
              if (!softmax_or(redo || !ok)) break;
            }
            float top = -INFINITY;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float4 kv = *reinterpret_cast<const float4*>(&sh->meta[m][4 * h + q]);
              float x = __uint_as_float(v[16 * q]);
#pragma unroll
              for (int k = 1; k < 16; ++k) x = fmaxf(x, __uint_as_float(v[16 * q + k]));
              top = fmaxf(top, x * score_factor(c_row, kv.x) + kv.y);
            }
            if (kHalves) {  // two threads have the row's halves and agree on its reference
              sh->other[wg][row] = top;
              if (!(ok = softmax_and(ok))) break;
              top = fmaxf(top, sh->other[wg ^ 1][row]);
            }
            const float now = fmaxf(top, ref), f = ref == kNoRef ? 1.f : ex2(ref - now);
            ref = now;
            l *= f;
            // O of the row, once the MMAs so far are done: those of the row's tile before, or
            // of this tile's first half
            if (n > (kTurns ? 1 : 0) || (!kHalves && h > 0)) {
              const bool second = !kHalves && h > 0;
              const uint32_t last = second ? item : kHalves ? item - 1 : item - 2;
              ok = mbar_wait_idle(second ? &sh->o_half[slot] : &sh->o_full[last & 1u], (last >> 1) & 1u, abort) && ok;
              ok = __all_sync(0xffffffffu, ok);
              tc_fence_after();
              constexpr int kO = kHalves ? kD / 2 : kD;
#pragma unroll 1
              for (int k = 0; k < kO; k += 16) {
                uint32_t o[16];
                const uint32_t at = tO + (kHalves ? wg * kO : 0) + k;
                tmem_ld16(at, o);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tmem_st16(at, o);
              }
              tmem_st_wait();
            }
          }
          if (kHalves && !ok) break;
          l += got;
          tmem_st32(tS + 64 * h, w);  // over the half's own scores
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh->p_full[slot][h]);  // this half's MMAs may begin
        }
        if (!ok) break;
      }
      const uint32_t items = n_tiles * kTiles;
      if (kTiles == 2 && !ok) break;
      // the rows: O / l, once this warpgroup's last item is done
      if (!kTurns || wg < n_tiles) {
        const uint32_t last = item0 + items - 1 -
                              (kTiles == 2 ? 1 - wg : kTurns ? (n_tiles - 1 - wg) & 1 : 0);
        ok = mbar_wait_idle(&sh->o_full[last & 1u], (last >> 1) & 1u, abort) && ok;
        ok = __all_sync(0xffffffffu, ok);
      }
      float f0 = 1.f, f1 = 0.f;  // of the two O of a row, with kTurns
      if (kTiles == 1) {  // the two parts of the row's sum
        sh->row_sum[wg][row] = l;
        if (kTurns) sh->other[wg][row] = ref;
        ok = softmax_and(ok);
        if (!ok) break;
        const float l0 = sh->row_sum[0][row], l1 = sh->row_sum[1][row];
        if (kTurns) {
          const float r0 = sh->other[0][row], r1 = sh->other[1][row];
          ref = fmaxf(r0, r1);
          f0 = r0 == kNoRef ? 0.f : ex2(r0 - ref);
          f1 = r1 == kNoRef ? 0.f : ex2(r1 - ref);
          l = l0 * f0 + l1 * f1;
        } else {
          l = l0 + l1;
        }
      }
      if (!ok) break;
      tc_fence_after();
      const float inv = l > 0.f ? 1.f / l : l;
      const float stat = l > 0.f ? ref - kWeightTop + __log2f(l) : l == 0.f ? -INFINITY : l;
      const bool whole = g.starts && g.ends;
      const int64_t at = part_slot(p, blockIdx.x, g.starts);
      constexpr int kO = kTiles == 2 ? kD : kD / 2;
      const int d0 = kTiles == 2 ? 0 : wg * kO;
      // 32 columns at a time go through 4 KiB of the warp's own, so that stores are whole
      // row segments: 32 rows x 64 bytes of results or 128 bytes of parts, in 16-byte
      // chunks at the place their row's number turns them to.
      uint8_t* stage = kD == 64 ? sRaw + C::kFifo * C::kVRaw + warp * 4096
                                : sQ + (kTiles == 2 ? qt : wg * kTiles) * C::kKBytes + quad * 4096;
      T* to[4];            // rows 8 i + lane / 4 of the warp, whole results
      bool has[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int rr = qt * 128 + quad * 32 + 8 * i + (lane >> 2), qr = static_cast<int>(rr * group_mul >> 16);
        has[i] = rr < rows;
        to[i] = static_cast<T*>(p.out) + static_cast<int64_t>(g.s.row0 + g.i0 + qr) * p.o_ts +
                (g.h * p.group + rr - qr * p.group) * p.o_hs + d0 + 8 * (lane & 3);
      }
      const int rp = qt * 128 + quad * 32 + (lane >> 3);  // rows 4 i + lane / 8, parts
      float* const part_to = p.part + (at + rp) * kD + d0 + 4 * (lane & 7);
#pragma unroll 1
      for (int k = 0; k < kO; k += 32) {
        uint32_t v[32];
        const uint32_t t0 = kTurns ? tmem + C::kO + lane_off : tO;
        tmem_ld32(t0 + d0 + k, v);
        tmem_ld_wait32(v);
        if (kTurns) {
          if (n_tiles > 1) {  // the other one has held no key otherwise
            uint32_t u[32];
            tmem_ld32(t0 + kD + d0 + k, u);
            tmem_ld_wait32(u);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              v[i] = __float_as_uint(__uint_as_float(v[i]) * f0 + __uint_as_float(u[i]) * f1);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f0);
          }
        }
        __syncwarp();
        if (whole) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t u[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              u[e] = pack2(__uint_as_float(v[8 * i + 2 * e]) * inv, __uint_as_float(v[8 * i + 2 * e + 1]) * inv, T{});
            *reinterpret_cast<uint4*>(stage + lane * 64 + (((i ^ (lane >> 1)) & 3) << 4)) = make_uint4(u[0], u[1], u[2], u[3]);
          }
          __syncwarp();
          const int ch = lane & 3;
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // eight rows a store
            const int rl = 8 * i + (lane >> 2);
            const uint4 x = *reinterpret_cast<const uint4*>(stage + rl * 64 + (((ch ^ (rl >> 1)) & 3) << 4));
            if (has[i]) *reinterpret_cast<uint4*>(to[i] + k) = x;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float4*>(stage + lane * 128 + (((i ^ lane) & 7) << 4)) =
                make_float4(__uint_as_float(v[4 * i]) * inv, __uint_as_float(v[4 * i + 1]) * inv,
                            __uint_as_float(v[4 * i + 2]) * inv, __uint_as_float(v[4 * i + 3]) * inv);
          __syncwarp();
          const int ch = lane & 7;
#pragma unroll
          for (int i = 0; i < 8; ++i) {  // four rows a store
            const int rl = 4 * i + (lane >> 3);
            const float4 x = *reinterpret_cast<const float4*>(stage + rl * 128 + (((ch ^ rl) & 7) << 4));
            if (rp + 4 * i < rows) *reinterpret_cast<float4*>(part_to + 4 * i * kD + k) = x;
          }
        }
      }
      __syncwarp();
      tc_fence_before();
      if (real && (kTiles == 2 || wg == 0)) {
        if (!whole) p.stat[at + r] = stat;
        else if (p.lse)
          p.lse[static_cast<int64_t>(g.s.row0 + g.i0 + qi) * p.q_heads + g.h * p.group + gi] = stat * kLn2;
      }
      if (threadIdx.x == 0) note_cut(p, g, sh->run.cut, blockIdx.x);
      tile += n_tiles;
      item0 += items;
    }
    if (!ok && lane == 0) {
      set_error(p.g.err, RIMURU_DEV_TIMEOUT);
      sh->abort = 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 13) tmem_dealloc(tmem, 512);
}

template <typename T, int kD, int kTiles>
cudaError_t launch(const AttnArgs& a, const CUtensorMap& tm, const CUtensorMap& tm_v, cudaStream_t s) {
  constexpr int kQParts = std::is_same<T, __nv_bfloat16>::value ? 2 : 3;
  constexpr int smem = TileCfg<kD, kTiles, kQParts>::kSmem;
  auto* fn = kv_tiles_kernel<T, kD, kTiles>;
  static SmemOnce once;
  cudaError_t e = once.set(reinterpret_cast<const void*>(fn), smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.runs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, a, tm, tm_v);
}
template <typename T>
cudaError_t launch_dim(const AttnArgs& a, const CUtensorMap& tm, const CUtensorMap& tm_v, cudaStream_t s) {
  const bool two = a.unit_rows == 256;
  if (a.g.head_dim == 64) return two ? launch<T, 64, 2>(a, tm, tm_v, s) : launch<T, 64, 1>(a, tm, tm_v, s);
  if (a.g.head_dim == 128) return two ? launch<T, 128, 2>(a, tm, tm_v, s) : launch<T, 128, 1>(a, tm, tm_v, s);
  return launch<T, 256, 1>(a, tm, tm_v, s);
}

}  // namespace

int kv_value_box(int head_dim, int page_tokens) {
  const int stage = head_dim <= 128 ? 64 : 32;
  return page_tokens < stage ? page_tokens : stage;
}

cudaError_t launch_kv_tiles(const AttnArgs& a, int dtype, const CUtensorMap& tm, const CUtensorMap& tm_v,
                            cudaStream_t s) {
  return dtype == RIMURU_BF16 ? launch_dim<__nv_bfloat16>(a, tm, tm_v, s) : launch_dim<__half>(a, tm, tm_v, s);
}

}  // namespace rimuru
