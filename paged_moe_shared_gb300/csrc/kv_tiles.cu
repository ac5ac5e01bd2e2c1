// Attention of many query rows (prompts, chunks, drafted tokens of wide groups)
// over the 8-bit paged cache.
//
// Bound: the tensor cores (4 head_dim operations per query head and key).  Rows
// are (query, head of the group) pairs, so the heads that share a key/value
// head share its tiles.  Per 128-token tile of keys and 128 rows:
//   S = Q K^T   e4m3 x e4m3: K is multiplied as it lies in the page, Q as a sum
//               of e4m3 parts (two hold a bf16 query exactly, three an f16 one)
//               into one fp32 accumulator: two parts cost what one bf16 product
//               costs, without widening K;
//   O += P V    f16 x f16: P rounded to f16 stays in TMEM as the A operand; V is
//               widened on its way to shared memory by four warps.  An e4m3 code
//               placed in the upper bits of an f16 is that value times 2^-8,
//               exactly, with no conversion instruction (and finite, whatever
//               the byte, so unused slots need no clearing).
// The V scale 2^k of a page is added to the score, x + k, so that the weight that
// meets the codes stays bounded; the row sum takes the weight without it by an
// exact multiplication.  Weights are relative to a reference that follows the
// row's largest x + k only when a tile passes it by more than 2^8; then the
// softmax warps rescale O in TMEM.
//
// Two softmax warpgroups alternate on two score buffers ("items"), so that the
// tensor cores work on one while the other is in softmax.  With head_dim <= 128
// and more than 128 rows the items are two query tiles (each K and V tile serves
// 256 rows, a row is a thread); otherwise successive key tiles of one query
// tile, whose columns the two warpgroups halve.
//
// Warps 0-3 and 4-7: softmax.  8-11: V.  12: K copies and page scales.  13: MMAs.
#include <cuda_fp8.h>

#include <algorithm>

#include "kv_attn.h"

namespace rimuru {
namespace {

using namespace dev;

constexpr int kThreads = 512;
constexpr int kMetaRing = 8;
constexpr int kGroups = kTileTokens / 16;
constexpr float kWeightTop = 7.f;    // a weight at the reference is 2^7
constexpr float kWeightSlack = 8.f;  // and may pass it by 2^8: f16 ends at 2^16
constexpr float kNoRef = -1e30f;     // the reference of a row that has seen no key

template <int kD, int kTiles, int kQParts>
struct TileCfg {
  static constexpr int kRowBytes = kD < 128 ? kD : 128;  // bytes of a K or Q row in one slab
  static constexpr int kSlabs = kD / kRowBytes;
  static constexpr int kSlabBytes = 128 * kRowBytes;
  static constexpr int kKBytes = kSlabs * kSlabBytes;           // one K tile
  static constexpr int kKRing = kD <= 128 ? 3 : 2;              // K tiles
  static constexpr int kQBytes = kQParts * kTiles * kKBytes;    // [part][tile][slab][128 rows]
  static constexpr int kVTok = kD <= 128 ? 64 : 32;             // tokens of a V stage
  static constexpr int kVStages = kTileTokens / kVTok;          // stages of a tile
  static constexpr int kVBytes = kVTok * kD * 2;                // [64 f16 of a token: 128 bytes][tokens]
  static constexpr int kVRing = kD == 256 && kQParts == 3 ? 3 : 4;
  static constexpr int kSmem = 1024 + kQBytes + kKRing * kKBytes + kVRing * kVBytes;
  static constexpr int kCols = kTiles == 2 ? 128 : 64;          // score columns of a thread
  static constexpr uint32_t kO = 256;                           // TMEM column of O; scores are at 0 and 128
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
  uint64_t meta_full[kMetaRing];
  uint64_t q_full;
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  RunStart run;
  int scratch[16];
  Meta meta[kMetaRing][kGroups];
  uint32_t seen[kMetaRing][4];    // a bit per token of the tile: its group has a page
  float row_max[2][128];          // one query tile: largest magnitudes of the halves of Q's rows
  float other[2][128];            // one query tile: row maxima of the halves
  float row_sum[2][128];          // and their sums
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t c) {
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c), __NV_E4M3)));
}
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) { return pack_bf16x2(a, b); }
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
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
// that the block was launched with (2 x 176 + 2 x 80 = 512).
constexpr int kSoftmaxRegs = 176, kOtherRegs = 80;
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
// Two e4m3 codes (bytes 0 and 1 of w, or 2 and 3) as f16 numbers times 2^-8.
__device__ __forceinline__ uint32_t widen(uint32_t w, bool upper) {
  const uint32_t t = __byte_perm(w, 0, upper ? 0x3424 : 0x1404);  // code in the high byte of each half
  return (t & 0x80008000u) | ((t >> 1) & 0x3F803F80u);
}

template <typename T, int kD, int kTiles>
__global__ void __launch_bounds__(kThreads, 1)
    kv_tiles_kernel(const __grid_constant__ AttnArgs p, const __grid_constant__ CUtensorMap tm) {
  constexpr int kQParts = std::is_same<T, __nv_bfloat16>::value ? 2 : 3;
  using C = TileCfg<kD, kTiles, kQParts>;
  constexpr int kSlabs = C::kSlabs, kRowBytes = C::kRowBytes, kCols = C::kCols;
  constexpr uint32_t kSwizzle = kRowBytes == 128 ? 2 : 4;
  constexpr uint32_t kAtom = 8 * kRowBytes;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + C::kQBytes;
  uint8_t* sV = sK + C::kKRing * C::kKBytes;
  __shared__ TileShared sh_;
  TileShared* sh = &sh_;
  volatile int* abort = &sh->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sh->k_full[i], 1);
      mbar_init(&sh->k_empty[i], 1);
      mbar_init(&sh->v_full[i], 4);
      mbar_init(&sh->v_empty[i], 1);
    }
    for (int i = 0; i < kMetaRing; ++i) mbar_init(&sh->meta_full[i], 1);
    mbar_init(&sh->q_full, 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->s_full[i], 1);
      mbar_init(&sh->p_full[i], kTiles == 2 ? 4 : 8);
      mbar_init(&sh->o_full[i], 1);
    }
    mbar_init(&sh->drain, 1);
    sh->abort = 0;
    fence_barrier_init();
    prefetch_tmap(&tm);
  }
  if (warp == 13) {
    tmem_alloc(&sh->tmem_base, 512);
    tmem_relinquish();
  }
  grid_dep_wait();  // lengths, tables, q and the cache come from earlier kernels
  grid_dep_launch();
  find_run(p, blockIdx.x, sh->scratch, &sh->run);
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
          ok = mbar_wait(&sh->k_empty[i], ((tile / C::kKRing) & 1u) ^ 1u, abort);
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
        mbar_wait(&sh->k_full[j % C::kKRing], (j / C::kKRing) & 1u, &never);
    } else if (warp == 13) {
      // ------------------------------------------------------------------ MMAs
      // Items: (key tile, query tile) pairs in order; item i uses score buffer i & 1.
      // The scores of item i + 2 follow the output of item i, whose weights lie in
      // the same buffer; MMAs of one thread run in the order they were issued.
      // The whole warp walks and waits, and one lane issues: addresses stay
      // warp-uniform (issued from a one-lane branch, an MMA took 160 cycles to issue
      // instead of the 64 it runs).
      constexpr uint32_t id_s = idesc_f8_f32(128, 128, false, false, false);
      constexpr uint32_t id_o = idesc_f16_f32(128, kD, false, /*b_mn=*/true);
      const uint32_t tb = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t q_s = smem_u32(sQ), k_s = smem_u32(sK), v_s = smem_u32(sV);
      uint32_t item = 0, k_slot = 0, k_phase = 0, v_slot = 0, v_phase = 0, seg = 0;
      bool ok = true;
      const auto wait = [&](uint64_t* bar, uint32_t phase) {
        ok = ok && mbar_wait(bar, phase, abort);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
      };
      // The next scores go to buffer `item`'s parity; `q`: its query tile.
      const auto scores = [&](uint32_t buffer, uint32_t q) {
        if (q == 0) wait(&sh->k_full[k_slot], k_phase);
        if (ok && elect_one()) {
          const uint32_t a0 = q_s + q * C::kKBytes, b0 = k_s + k_slot * C::kKBytes;
          const uint32_t d = tb + 128 * buffer;
#pragma unroll
          for (int part = 0; part < kQParts; ++part) {
#pragma unroll
            for (int sl = 0; sl < kSlabs; ++sl) {
#pragma unroll
              for (int k = 0; k < kRowBytes / 32; ++k)
                umma_f8(d,
                        smem_desc(a0 + part * kTiles * C::kKBytes + sl * C::kSlabBytes + 32 * k, 16,
                                  kAtom, kSwizzle),
                        smem_desc(b0 + sl * C::kSlabBytes + 32 * k, 16, kAtom, kSwizzle), id_s,
                        (part | sl | k) != 0 ? 1u : 0u);
            }
          }
          umma_commit(&sh->s_full[buffer]);
          if (q == kTiles - 1) umma_commit(&sh->k_empty[k_slot]);
        }
        __syncwarp();
        if (q == kTiles - 1 && ++k_slot == C::kKRing) k_slot = 0, k_phase ^= 1u;
      };
      while (ok && walk.next(p, &g)) {
        const int tiles = __shfl_sync(0xffffffffu, g.t1 - g.t0, 0);
        wait(&sh->q_full, seg & 1u);
        scores(item & 1u, 0);
        if (kTiles == 2) scores((item + 1) & 1u, 1);
        else if (tiles > 1) scores((item + 1) & 1u, 0);
        for (int n = 0; ok && n < tiles; ++n) {
          const uint32_t v_slot0 = v_slot, v_phase0 = v_phase;
#pragma unroll
          for (int q = 0; q < kTiles; ++q, ++item) {
            const uint32_t buffer = item & 1u;
            wait(&sh->p_full[buffer], (item >> 1) & 1u);
            v_slot = v_slot0, v_phase = v_phase0;
#pragma unroll
            for (int h = 0; h < C::kVStages; ++h) {
              if (q == 0) wait(&sh->v_full[v_slot], v_phase);
              if (ok && elect_one()) {
                const uint32_t b0 = v_s + v_slot * C::kVBytes;
#pragma unroll
                for (int k = 0; k < C::kVTok / 16; ++k)  // 16 tokens: eight columns of P, 16 rows of V
                  umma_f16_ts(tb + C::kO + q * kD, tb + 128 * buffer + C::kVTok / 2 * h + 8 * k,
                              smem_desc_sw128(b0 + 2048 * k, C::kVTok * 128, 1024), id_o,
                              (n > 0 || h + k != 0) ? 1u : 0u);
                if (q == kTiles - 1) umma_commit(&sh->v_empty[v_slot]);
                if (h == C::kVStages - 1) umma_commit(&sh->o_full[buffer]);
              }
              __syncwarp();
              if (++v_slot == C::kVRing) v_slot = 0, v_phase ^= 1u;
            }
            if (kTiles == 2 ? n + 1 < tiles : n + 2 < tiles) scores(buffer, q);
          }
        }
        ++seg;
      }
      if (!ok && lane == 0) {
        set_error(p.g.err, RIMURU_DEV_TIMEOUT);
        sh->abort = 1;
      }
      if (elect_one()) umma_commit(&sh->drain);  // all MMAs are finished before TMEM is released
      __syncwarp();
      volatile int never = 0;
      mbar_wait(&sh->drain, 0, &never);
    }
  } else if (warp >= 8) {
    regs_down<kOtherRegs>();
    // ---------------------------------------------------------------------- V
    // A stage is kVTok tokens: thread `t128` takes 16 codes (chunk c) of the
    // tokens r0, r0 + kStep, ...; the next two stages are loaded ahead.
    constexpr int kChunks = kD / 16, kStep = 128 / kChunks, kPer = C::kVTok / kStep;
    const int t128 = threadIdx.x - 256, c = t128 % kChunks, r0 = t128 / kChunks;
    bool ok = true;
    uint4 raw[2][kPer];
    // the load cursor: stage `lh` of key tile lt, tile `ltile` of the run
    int lt = 0, lh = C::kVStages;
    uint32_t ltile = 0xFFFFFFFFu;
    g.t1 = 0;
    const auto load = [&](uint4(&x)[kPer]) {
      if (lh == C::kVStages) {
        lh = 0;
        ++ltile;
        if (++lt >= g.t1) {
          walk.next(p, &g);
          lt = g.t0;
        }
        ok = mbar_wait(&sh->meta_full[ltile % kMetaRing], (ltile / kMetaRing) & 1u, abort) && ok;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
      }
      const uint64_t base = static_cast<uint64_t>(p.g.kv_heads + g.h) * P * kD + 16 * c;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int r = C::kVTok * lh + r0 + k * kStep;
        const int page = sh->meta[ltile % kMetaRing][r >> 4].page;
        x[k] = make_uint4(0, 0, 0, 0);
        if (page >= 0)
          x[k] = *reinterpret_cast<const uint4*>(p.g.pool + page * p.g.page_bytes + base +
                                                 static_cast<uint64_t>(r & (P - 1)) * kD);
      }
      ++lh;
    };
    const auto store = [&](uint32_t v, const uint4(&x)[kPer]) {
      const uint32_t s = v % C::kVRing;
      ok = mbar_wait(&sh->v_empty[s], ((v / C::kVRing) & 1u) ^ 1u, abort) && ok;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      uint8_t* dst = sV + s * C::kVBytes + (c >> 2) * (C::kVTok * 128);
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int r = r0 + k * kStep, ch = 2 * (c & 3);  // chunks of eight f16 in the 128-byte row
        *reinterpret_cast<uint4*>(dst + r * 128 + (((ch ^ r) & 7) << 4)) =
            make_uint4(widen(x[k].x, false), widen(x[k].x, true), widen(x[k].y, false), widen(x[k].y, true));
        *reinterpret_cast<uint4*>(dst + r * 128 + ((((ch + 1) ^ r) & 7) << 4)) =
            make_uint4(widen(x[k].z, false), widen(x[k].z, true), widen(x[k].w, false), widen(x[k].w, true));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->v_full[s]);
    };
    const uint32_t total = C::kVStages * sh->run.tiles;  // even
    if (total > 0) {
      load(raw[0]);
      if (ok) load(raw[1]);
    }
    for (uint32_t v = 0; ok && v < total; v += 2) {
      store(v, raw[0]);
      if (ok && v + 2 < total) load(raw[0]);
      if (ok) store(v + 1, raw[1]);
      if (ok && v + 3 < total) load(raw[1]);
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
    const int col0 = kTiles == 2 ? 0 : 64 * wg;      // first score column of this thread
    const uint32_t tO = tmem + C::kO + qt * kD + lane_off;
    uint32_t tile = 0, item0 = 0;
    bool ok = true;
    while (ok && walk.next(p, &g)) {
      const int rows = (g.i1 - g.i0) * p.group;
      // keys [j_lo, j_hi) of this thread's row; rows past the unit see every column and are
      // not written
      const int r = qt * 128 + row, qi = r / p.group, gi = r - qi * p.group;
      const bool real = r < rows;
      // Q of the row, as parts; with one query tile the two warpgroups halve the row
      constexpr int kQ = kTiles == 2 ? kD : kD / 2;
      const int d0q = kTiles == 2 ? 0 : wg * kQ;
      float c_row;  // score per unit of S and K scale; never 0, so masked scores stay masked
      {
        uint4 raw[kQ / 8];
        const T* src = static_cast<const T*>(p.q) + (g.s.row0 + g.i0 + qi) * p.q_ts +
                       (g.h * p.group + gi) * p.q_hs + d0q;
#pragma unroll
        for (int k = 0; k < kQ / 8; ++k)
          raw[k] = real ? *reinterpret_cast<const uint4*>(src + 8 * k) : make_uint4(0, 0, 0, 0);
        float amax = 0.f;
#pragma unroll
        for (int k = 0; k < kQ / 8; ++k) {
#pragma unroll
          for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(to_f(reinterpret_cast<const T*>(&raw[k])[i])));
        }
        if (kTiles == 1) {
          sh->row_max[wg][row] = amax;
          ok = softmax_and(ok);
          if (!ok) break;
          amax = fmaxf(amax, sh->row_max[wg ^ 1][row]);
        }
        // power of two that brings the row's largest magnitude into (224, 448]; the sign of
        // the scale goes into Q, so that a larger S is always a larger score
        const uint32_t ab = __float_as_uint(amax);
        const int e = max(-100, min(100, static_cast<int>(ab >> 23) - 127 - 8 + ((ab & 0x7FFFFFu) > 0x600000u)));
        const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23 | (p.scale_log2 < 0.f ? 0x80000000u : 0u));
        c_row = fmaxf(__uint_as_float(static_cast<uint32_t>(127 + e) << 23) * fabsf(p.scale_log2), 1e-30f);
        if (!(amax <= 3.4028234664e38f)) c_row = __int_as_float(0x7FFFFFFF);  // an infinite query: NaN
#pragma unroll
        for (int k = 0; k < kQ / 16; ++k) {  // 16 codes of each part at a time
          float x[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = to_f(reinterpret_cast<const T*>(&raw[2 * k])[i]) * inv;
          const int d = d0q + 16 * k;
          uint8_t* dst = sQ + qt * C::kKBytes + d / kRowBytes * C::kSlabBytes + swz<kRowBytes>(row, d % kRowBytes);
#pragma unroll
          for (int part = 0; part < kQParts; ++part) {
            uint32_t c[4];
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              const uint32_t lo2 = e4m3x2(x[i], x[i + 1]), hi2 = e4m3x2(x[i + 2], x[i + 3]);
              c[i / 4] = lo2 | hi2 << 16;
              if (part + 1 < kQParts) {
                const float2 f = from_e4m3x2(lo2), h = from_e4m3x2(hi2);
                x[i] -= f.x, x[i + 1] -= f.y, x[i + 2] -= h.x, x[i + 3] -= h.y;
              }
            }
            *reinterpret_cast<uint4*>(dst + part * kTiles * C::kKBytes) = make_uint4(c[0], c[1], c[2], c[3]);
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->q_full);
      const int pos = g.s.len - g.s.n + g.i0 + qi;
      const int j_hi = real ? min(pos + 1, g.s.len) : 0x7FFFFFFF;
      const int j_lo = real && p.window > 0 ? max(0, pos - p.window + 1) : 0;
      float ref = kNoRef, l = 0.f;
      const int n_tiles = g.t1 - g.t0;
      for (int n = 0; n < n_tiles; ++n) {
        const int t = g.t0 + n;
        const uint32_t item = item0 + (kTiles == 2 ? 2 * n + wg : n), slot = item & 1u;
        const uint32_t m = (tile + n) % kMetaRing;
        ok = mbar_wait(&sh->meta_full[m], ((tile + n) / kMetaRing) & 1u, abort) && ok;
        ok = mbar_wait(&sh->s_full[slot], (item >> 1) & 1u, abort) && ok;
        ok = __all_sync(0xffffffffu, ok);
        if (kTiles == 2 && !ok) break;
        tc_fence_after();
        const uint32_t tS = tmem + 128 * slot + lane_off;
        const int j0 = t * kTileTokens + col0;
        bool edge = j_lo > j0 || j_hi < j0 + kCols;
#pragma unroll
        for (int k = 0; k < kCols / 32; ++k) edge |= sh->seen[m][col0 / 32 + k] != 0xFFFFFFFFu;
        edge = __any_sync(0xffffffffu, edge);
        const auto hide = [&](uint32_t(&v)[32], int k0) {  // -inf where the row does not see
          if (edge) {
            const int lo = max(0, min(32, j_lo - (j0 + k0))), hi = max(0, min(32, j_hi - (j0 + k0)));
            uint32_t see = sh->seen[m][(col0 + k0) / 32];
            see &= static_cast<uint32_t>((1ull << hi) - (1ull << lo)) & (hi > lo ? 0xFFFFFFFFu : 0u);
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = see >> k & 1u ? v[k] : 0xFF800000u;
          }
        };
        // The weights are taken with the reference as it stands, and their maximum on the
        // way: only a tile that passes it by more than the slack is looked through for its
        // largest score, and its weights taken again.  A group's x + k is S * mul + add.
        uint32_t w[kCols / 2];
        float sum_l;
        while (true) {
          const float base = kWeightTop - ref;
          float most = 0.f, most2 = 0.f;
          sum_l = 0.f;
          uint32_t s0[32], s1[32];  // 32 columns at hand, 32 on their way
          tmem_ld32(tS + col0, s0);
#pragma unroll
          for (int c = 0; c < kCols; c += 32) {
            uint32_t(&v)[32] = c & 32 ? s1 : s0;
            tmem_ld_wait32(v);
            if (c + 32 < kCols) tmem_ld32(tS + col0 + c + 32, c & 32 ? s0 : s1);
            hide(v, c);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const float4 kv = *reinterpret_cast<const float4*>(&sh->meta[m][(col0 + c) / 16 + q]);
              const float mul = c_row * kv.x, a = kv.y + base;
              float2 sum = make_float2(0.f, 0.f);
#pragma unroll
              for (int k = 0; k < 16; k += 2) {
                const float2 x = fma2(make_float2(__uint_as_float(v[16 * q + k]), __uint_as_float(v[16 * q + k + 1])),
                                      make_float2(mul, mul), make_float2(a, a));
                const float2 y = make_float2(ex2(x.x), ex2(x.y));
                sum = add2(sum, y);
                if (k & 2) most2 = fmaxf(fmaxf(most2, y.x), y.y);
                else most = fmaxf(fmaxf(most, y.x), y.y);
                const __half2 h = __floats2half2_rn(y.x, y.y);
                w[c / 2 + 8 * q + k / 2] = *reinterpret_cast<const uint32_t*>(&h);
              }
              sum_l += (sum.x + sum.y) * kv.z;
            }
          }
          most = fmaxf(most, most2);
          constexpr float kMost = static_cast<float>(1 << static_cast<int>(kWeightTop + kWeightSlack));
          if (kTiles == 2) {
            if (!__any_sync(0xffffffffu, most > kMost)) break;
          } else {
            if (!softmax_or(most > kMost || !ok)) break;
            if (!(ok = softmax_and(ok))) break;
          }
          float top = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < kCols; c += 32) {
            uint32_t v[32];
            tmem_ld32(tS + col0 + c, v);
            tmem_ld_wait32(v);
            hide(v, c);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const float4 kv = *reinterpret_cast<const float4*>(&sh->meta[m][(col0 + c) / 16 + q]);
              float x = __uint_as_float(v[16 * q]);
#pragma unroll
              for (int k = 1; k < 16; ++k) x = fmaxf(x, __uint_as_float(v[16 * q + k]));
              top = fmaxf(top, x * (c_row * kv.x) + kv.y);
            }
          }
          if (kTiles == 1) {  // the other half of the row
            sh->other[wg][row] = top;
            if (!(ok = softmax_and(ok))) break;
            top = fmaxf(top, sh->other[wg ^ 1][row]);
          }
          const float now = top > ref + kWeightSlack ? top : ref, f = ex2(ref - now);
          ref = now;
          l *= f;
          if (n > 0) {  // O of the row is complete up to the tile before: rescale it
            const uint32_t last = kTiles == 2 ? item - 2 : item - 1;
            ok = mbar_wait(&sh->o_full[last & 1u], (last >> 1) & 1u, abort) && ok;
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
            constexpr int kO = kTiles == 2 ? kD : kD / 2;
#pragma unroll 1
            for (int k = 0; k < kO; k += 32) {
              uint32_t v[32];
              const uint32_t at = tO + (kTiles == 2 ? 0 : wg * kO) + k;
              tmem_ld32(at, v);
              tmem_ld_wait32(v);
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
              tmem_st32(at, v);
            }
            tmem_st_wait();
          }
        }
        if (kTiles == 1 && !ok) break;
        l += sum_l;
        // The weights lie where the scores were (with one query tile, where the other half
        // had its own: it has read them, or the barrier above would not have let go).
#pragma unroll
        for (int c = 0; c < kCols / 2; c += 32)
          tmem_st32(tS + col0 / 2 + c, *reinterpret_cast<const uint32_t(*)[32]>(&w[c]));
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->p_full[slot]);
      }
      const uint32_t items = n_tiles * kTiles;
      if (kTiles == 2 && !ok) break;
      // the rows: O / l, with the 2^8 that V was widened without
      {
        const uint32_t last = item0 + items - 1 - (kTiles == 2 ? 1 - wg : 0);
        ok = mbar_wait(&sh->o_full[last & 1u], (last >> 1) & 1u, abort) && ok;
        ok = __all_sync(0xffffffffu, ok);
      }
      if (kTiles == 1) {  // the two halves of the row's sum
        sh->row_sum[wg][row] = l;
        ok = softmax_and(ok);
        if (!ok) break;
        l = sh->row_sum[0][row] + sh->row_sum[1][row];
      }
      if (!ok) break;
      tc_fence_after();
      const float inv = l > 0.f ? 256.f / l : l;
      const float stat = l > 0.f ? ref - kWeightTop + __log2f(l) : l == 0.f ? -INFINITY : l;
      const bool whole = g.starts && g.ends;
      const int64_t at = part_slot(p, blockIdx.x, g.starts) + r;
      const int64_t orow = g.s.row0 + g.i0 + qi;
      const int head = g.h * p.group + gi;
      constexpr int kO = kTiles == 2 ? kD : kD / 2;
      const int d0 = kTiles == 2 ? 0 : wg * kO;
      T* out = static_cast<T*>(p.out) + orow * p.o_ts + head * p.o_hs + d0;
      float* part = p.part + at * kD + d0;
#pragma unroll 1
      for (int k = 0; k < kO; k += 32) {
        uint32_t v[32];
        tmem_ld32(tO + d0 + k, v);
        tmem_ld_wait();
        if (!real) continue;
        if (whole) {
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            uint32_t u[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              u[e] = pack2(__uint_as_float(v[i + 2 * e]) * inv, __uint_as_float(v[i + 2 * e + 1]) * inv, T{});
            *reinterpret_cast<uint4*>(out + k + i) = make_uint4(u[0], u[1], u[2], u[3]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<float4*>(part + k + i) =
                make_float4(__uint_as_float(v[i]) * inv, __uint_as_float(v[i + 1]) * inv,
                            __uint_as_float(v[i + 2]) * inv, __uint_as_float(v[i + 3]) * inv);
        }
      }
      tc_fence_before();
      if (real && (kTiles == 2 || wg == 0)) {
        if (!whole) p.stat[at] = stat;
        else if (p.lse) p.lse[orow * p.q_heads + head] = stat * kLn2;
      }
      if (g.starts && threadIdx.x == 0) note_join(p, g, sh->run.cut, blockIdx.x);
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
cudaError_t launch(const AttnArgs& a, const CUtensorMap& tm, cudaStream_t s) {
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
  return cudaLaunchKernelEx(&cfg, fn, a, tm);
}
template <typename T>
cudaError_t launch_dim(const AttnArgs& a, const CUtensorMap& tm, cudaStream_t s) {
  const bool two = a.unit_rows == 256;
  if (a.g.head_dim == 64) return two ? launch<T, 64, 2>(a, tm, s) : launch<T, 64, 1>(a, tm, s);
  if (a.g.head_dim == 128) return two ? launch<T, 128, 2>(a, tm, s) : launch<T, 128, 1>(a, tm, s);
  return launch<T, 256, 1>(a, tm, s);
}

}  // namespace

cudaError_t launch_kv_tiles(const AttnArgs& a, int dtype, const CUtensorMap& tm, cudaStream_t s) {
  return dtype == RIMURU_BF16 ? launch_dim<__nv_bfloat16>(a, tm, s) : launch_dim<__half>(a, tm, s);
}

}  // namespace rimuru
