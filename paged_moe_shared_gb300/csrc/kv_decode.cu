// Attention of a few query rows (at most 16 per key/value head) over the 8-bit
// paged cache: decode steps.
//
// Bound: HBM, one read of the codes.  The codes go from the pages to the tensor
// cores as they are: TMA brings 128 tokens of K and V (one box per page) into
// swizzled shared memory, and tcgen05 multiplies them as the M = 128 operand,
//   S^T [tokens x rows] = K Q^T,     O^T [head_dim x rows] = V^T P,
// so nothing is ever widened.  The few-row operands Q and P are 16-bit or fp32
// quantities: each is written as a sum of 8-bit floats (rounded, then the rest
// rounded, ...) and the parts are multiplied one after another into the same
// fp32 accumulator.  Q takes e4m3 parts, 4 significant bits each: two hold a
// bf16 query exactly, three an f16 query.  P takes four e5m2 parts, 12 bits;
// e5m2 spans 2^-16 .. 2^15, so a weight is kept down to 2^-32 of the largest
// (three e4m3 parts flushed below 2^-18, which showed in output elements whose
// heaviest tokens have a V near zero).
//
// Softmax: thread = token.  The V scale of a token is a power of two 2^k and is
// added to its score, x + k, so the weight that meets the code of V is
// 2^(x + k - m) with m the tile's largest x + k: at most one whatever the
// scales, and the row sum takes 2^(x - m) by an exact multiplication.  Weights
// are relative to the tile's own maximum, so no accumulator is ever rescaled:
// tiles are joined in fp32 registers.
//
// Warp 0 issues the copies, warp 1 the MMAs, warps 2-5 do the softmax; S and O
// are double buffered in TMEM, so K Q^T of the next tile runs during the
// softmax of this one.  With 8 rows and head_dim 128 a tile costs the softmax
// warps about 400 instructions each, a third of the time its bytes take.
#include <cuda_fp8.h>

#include <algorithm>

#include "kv_attn.h"

namespace rimuru {
namespace {

using namespace dev;

constexpr int kDecodeThreads = 192;
constexpr int kWeightParts = 4;
constexpr float kWeightTop = 15.f;  // weights are scaled by 2^15: e5m2 ends at 1.75 * 2^15

template <int kD, int kR, int kQParts>
struct DecodeCfg {
  static constexpr int kRowBytes = kD < 128 ? kD : 128;  // bytes of a token in one slab
  static constexpr int kSlabs = kD / kRowBytes;           // slabs of a K or V tile
  static constexpr int kSlabBytes = kTileTokens * kRowBytes;
  static constexpr int kCtas = kD <= 128 ? 2 : 1;  // per SM
  static constexpr int kRing = kD <= 128 ? (kD == 64 ? 10 : 6) : 12;  // slabs
  static constexpr int kN = kR < 16 ? 16 : kR;  // columns of an MMA
  static constexpr int kQBytes = kN * kD;       // one part of Q: kSlabs x [kN][kRowBytes]
  static constexpr int kPBytes = kN * 128;      // one part of P: [kN][128 tokens]
  static constexpr int kTmem = 2 * kN + 2 * kSlabs * kN;  // S twice, O twice
  static constexpr int kTmemCols = kTmem <= 32 ? 32 : kTmem <= 64 ? 64 : kTmem <= 128 ? 128 : 256;
  static constexpr int kSmem =
      1024 + kRing * kSlabBytes + kQParts * kQBytes + kWeightParts * kPBytes + 1024;
};

struct DecodeShared {
  uint64_t full[12], empty[12];
  uint64_t q_full, p_full;
  uint64_t s_full[2], o_full[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  RunStart run;
  int64_t scratch[8];
  float tile_max[2][4][kDecodeMaxRows];
  float row_scale[kDecodeMaxRows];
  float row_sum[4][kDecodeMaxRows];
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
// Two e4m3 codes (a in the low byte).
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t c) {
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c), __NV_E4M3)));
}
// The same in e5m2, whose codes are the upper halves of f16 numbers.
__device__ __forceinline__ uint32_t e5m2x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E5M2);
}
__device__ __forceinline__ float2 from_e5m2x2(uint32_t c) {
  const uint32_t h = __byte_perm(c, 0, 0x1404);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f(float x, __nv_bfloat16* y) { *y = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f(float x, __half* y) { *y = __float2half_rn(x); }

// Byte offset of byte d (of kRowBytes) of row r in a swizzled K-major block.
template <int kRowBytes>
__device__ __forceinline__ int swz(int r, int d) {
  if (kRowBytes == 128) return r * 128 + ((((d >> 4) ^ r) & 7) << 4) + (d & 15);
  return r * 64 + ((((d >> 4) ^ (r >> 1)) & 3) << 4) + (d & 15);
}
template <int kN>
__device__ __forceinline__ void tmem_ld(uint32_t t, uint32_t (&r)[kN]) {
  if constexpr (kN == 8) tmem_ld8(t, r);
  else tmem_ld16(t, r);
}

template <typename T, int kD, int kR>
__global__ void __launch_bounds__(kDecodeThreads, kD <= 128 ? 2 : 1)
    kv_decode_kernel(const __grid_constant__ AttnArgs p, const __grid_constant__ CUtensorMap tm) {
  constexpr int kQParts = sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value ? 2 : 3;
  using C = DecodeCfg<kD, kR, kQParts>;
  constexpr int kN = C::kN, kSlabs = C::kSlabs, kRing = C::kRing, kRowBytes = C::kRowBytes;
  constexpr uint32_t kSwizzle = kRowBytes == 128 ? 2 : 4;
  constexpr uint32_t kAtom = 8 * kRowBytes;  // eight rows
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sRing = smem;
  uint8_t* sQ = sRing + kRing * C::kSlabBytes;
  uint8_t* sP = sQ + kQParts * C::kQBytes;
  __shared__ DecodeShared sh_;
  DecodeShared* sh = &sh_;
  volatile int* abort = &sh->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sh->full[i], 1);
      mbar_init(&sh->empty[i], 1);
    }
    mbar_init(&sh->q_full, 4);
    mbar_init(&sh->p_full, 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->s_full[i], 1);
      mbar_init(&sh->o_full[i], 1);
    }
    mbar_init(&sh->drain, 1);
    sh->abort = 0;
    fence_barrier_init();
    prefetch_tmap(&tm);
  }
  if (warp == 1) {
    tmem_alloc(&sh->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  grid_dep_wait();  // lengths, tables, q and the cache come from earlier kernels
  grid_dep_launch();
  find_run(p, blockIdx.x, sh->scratch, &sh->run);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  const uint32_t tS = tmem, tO = tmem + 2 * kN;
  const int P = p.g.page_tokens;
  RunWalk walk;
  walk.begin(p, sh->run);
  Segment g;

  if (warp == 0) {
    // ---------------------------------------------------------------- copies
    // Unit 2 i is the K tile i of the run, unit 2 i + 1 its V tile; a unit is
    // kSlabs slots of the ring.  Lane l copies page l of the tile.
    const uint64_t pol = policy_evict_first();
    const int boxes = kTileTokens / P;
    uint32_t slot = 0;
    bool ok = true;
    while (ok && walk.next(p, &g)) {
      const int lo = p.window > 0 ? max(0, g.s.len - g.s.n + g.i0 - p.window + 1) : 0;
      for (int t = g.t0; ok && t < g.t1; ++t) {
        const int tok = t * kTileTokens + lane * P;  // first token of this lane's page
        int page = -1;
        if (lane < boxes && tok < g.s.len && tok + P > lo) {
          page = p.s.table[g.b * p.s.table_stride + tok / P];
          if (page < 0 || page >= p.g.num_pages) {
            set_error(p.g.err, RIMURU_DEV_BAD_PAGE);
            page = -1;
          }
        }
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, page >= 0)) * P * kRowBytes;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const int row = (kv * p.g.kv_heads + g.h) * P;  // first row of the head in the page
#pragma unroll
          for (int sl = 0; sl < kSlabs; ++sl, ++slot) {
            const uint32_t i = slot % kRing, ph = (slot / kRing) & 1u;
            ok = ok && mbar_wait(&sh->empty[i], ph ^ 1u, abort);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&sh->full[i], bytes);
            __syncwarp();
            if (page >= 0)
              tma_load_3d(sRing + i * C::kSlabBytes + lane * P * kRowBytes, &tm, &sh->full[i],
                          sl * kRowBytes, row, page, pol);
          }
          if (!ok) break;
        }
      }
    }
    if (!ok && lane == 0) {
      set_error(p.g.err, RIMURU_DEV_TIMEOUT);
      sh->abort = 1;
    }
    // every copy this warp issued must have landed before the CTA exits
    volatile int never = 0;
    for (uint32_t j = slot > kRing ? slot - kRing : 0u; j < slot; ++j)
      mbar_wait(&sh->full[j % kRing], (j / kRing) & 1u, &never);
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMAs
    if (lane == 0) {
      constexpr uint32_t id_s = idesc_f8_f32(128, kN, false, false, false);
      constexpr uint32_t id_o = idesc_f8_f32(128, kN, /*a_mn=*/true, false, /*b_e5m2=*/true);
      uint32_t tile = 0, seg = 0;
      bool ok = true;
      const auto scores = [&](uint32_t i) {  // S^T of the run's tile i
#pragma unroll
        for (int sl = 0; sl < kSlabs; ++sl) {
          const uint32_t u = 2 * i * kSlabs + sl, slot = u % kRing;
          if (!mbar_wait(&sh->full[slot], (u / kRing) & 1u, abort)) return false;
          tc_fence_after();
          const uint32_t a0 = smem_u32(sRing + slot * C::kSlabBytes);
#pragma unroll
          for (int part = 0; part < kQParts; ++part) {
            const uint32_t b0 = smem_u32(sQ + part * C::kQBytes + sl * kN * kRowBytes);
#pragma unroll
            for (int k = 0; k < kRowBytes / 32; ++k)
              umma_f8(tS + (i & 1u) * kN, smem_desc(a0 + 32 * k, 16, kAtom, kSwizzle),
                      smem_desc(b0 + 32 * k, 16, kAtom, kSwizzle), id_s,
                      (sl | part | k) != 0 ? 1u : 0u);
          }
          umma_commit(&sh->empty[slot]);
        }
        umma_commit(&sh->s_full[i & 1u]);
        return true;
      };
      const auto outputs = [&](uint32_t i) {  // O^T of the run's tile i
        if (!mbar_wait(&sh->p_full, i & 1u, abort)) return false;
#pragma unroll
        for (int sl = 0; sl < kSlabs; ++sl) {
          const uint32_t u = (2 * i + 1) * kSlabs + sl, slot = u % kRing;
          if (!mbar_wait(&sh->full[slot], (u / kRing) & 1u, abort)) return false;
          tc_fence_after();
          const uint32_t a0 = smem_u32(sRing + slot * C::kSlabBytes);
#pragma unroll
          for (int part = 0; part < kWeightParts; ++part) {
            const uint32_t b0 = smem_u32(sP + part * C::kPBytes);
#pragma unroll
            for (int k = 0; k < 4; ++k)  // 32 tokens: four groups of eight rows
              umma_f8(tO + ((i & 1u) * kSlabs + sl) * kN,
                      smem_desc(a0 + 4 * k * kAtom, C::kSlabBytes, kAtom, kSwizzle),
                      smem_desc(b0 + 32 * k, 16, 1024, 2), id_o, (part | k) != 0 ? 1u : 0u);
          }
          umma_commit(&sh->empty[slot]);
        }
        umma_commit(&sh->o_full[i & 1u]);
        return true;
      };
      while (ok && walk.next(p, &g)) {
        ok = mbar_wait(&sh->q_full, seg & 1u, abort);
        tc_fence_after();
        ok = ok && scores(tile);
        for (int t = g.t0; ok && t < g.t1; ++t, ++tile) {
          if (t + 1 < g.t1) ok = scores(tile + 1);
          ok = ok && outputs(tile);
        }
        ++seg;
      }
      if (!ok) {
        set_error(p.g.err, RIMURU_DEV_TIMEOUT);
        sh->abort = 1;
      }
      umma_commit(&sh->drain);  // all MMAs are finished before TMEM is released
      volatile int never = 0;
      mbar_wait(&sh->drain, 0, &never);
    }
  } else {
    // --------------------------------------------------------------- softmax
    const int quad = warp & 3;             // TMEM lanes this warp may read
    const int tok = quad * 32 + lane;      // token of the tile, and row of O^T
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    uint32_t tile = 0;
    // `ok`: this warp's waits came through; `all`: the four warps' did, as agreed
    // at the last barrier.  Only `all` leaves the loops, so no warp waits at a
    // barrier for one that has left.
    bool ok = true, all = true;
    while (all && walk.next(p, &g)) {
      // Q of the segment, as parts; warp `quad` takes rows quad, quad + 4, ...
      const int rows = (g.i1 - g.i0) * p.group;
      const int pos0 = g.s.len - g.s.n + g.i0;  // position of the first query row
      for (int r = quad; r < kR; r += 4) {
        constexpr int kPer = kD / 32;
        float x[kPer];
        float amax = 0.f;
        if (r < rows) {
          const int64_t at = (g.s.row0 + g.i0 + r / p.group) * p.q_ts +
                             (g.h * p.group + r % p.group) * p.q_hs + lane * kPer;
#pragma unroll
          for (int i = 0; i < kPer; ++i) x[i] = to_f(static_cast<const T*>(p.q)[at + i]);
        } else {
#pragma unroll
          for (int i = 0; i < kPer; ++i) x[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) amax = fmaxf(amax, fabsf(x[i]));
        amax = warp_max(amax);
        // power of two that brings the row's largest magnitude into (224, 448]
        const uint32_t ab = __float_as_uint(amax);
        const int e = max(-100, min(100, static_cast<int>(ab >> 23) - 127 - 8 + ((ab & 0x7FFFFFu) > 0x600000u)));
        const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
        for (int i = 0; i < kPer; ++i) x[i] *= inv;
        const int d0 = lane * kPer, sl = d0 / kRowBytes;
        uint8_t* dst = sQ + sl * kN * kRowBytes + swz<kRowBytes>(r, d0 % kRowBytes);
#pragma unroll
        for (int part = 0; part < kQParts; ++part) {
#pragma unroll
          for (int i = 0; i < kPer; i += 2) {
            const uint32_t c = e4m3x2(x[i], x[i + 1]);
            const float2 f = from_e4m3x2(c);
            x[i] -= f.x;
            x[i + 1] -= f.y;
            *reinterpret_cast<uint16_t*>(dst + part * C::kQBytes + i) = static_cast<uint16_t>(c);
          }
        }
        // an infinite query has no finite score: its row becomes NaN
        if (lane == 0)
          sh->row_scale[r] = amax <= 3.4028234664e38f
                                 ? __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * p.scale_log2
                                 : __int_as_float(0x7FFFFFFF);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->q_full);
      if (!(all = named_bar_and(ok))) break;
      float rs[kR], m[kR], l[kR], pa[kR], pb[kR], o[kSlabs][kR];
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        rs[r] = sh->row_scale[r];
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int sl = 0; sl < kSlabs; ++sl) o[sl][r] = 0.f;
      }
      // The token's page and scales, fetched a tile ahead.
      const int lo = p.window > 0 ? max(0, pos0 - p.window + 1) : 0;
      float k_next = 0.f, v_next = 0.f;
      const auto fetch = [&](int t) {  // v_next 0: the token does not count
        const int j = t * kTileTokens + tok;
        k_next = v_next = 0.f;
        if (j >= lo && j < g.s.len) {
          const int page = p.s.table[g.b * p.s.table_stride + j / P];
          if (page >= 0 && page < p.g.num_pages) {
            const float* sc = p.g.scales + static_cast<int64_t>(page) * 2 * p.g.kv_heads + g.h;
            k_next = sc[0];
            v_next = sc[p.g.kv_heads];
          }
        }
      };
      const auto take_output = [&](uint32_t i) {  // adds O^T of tile i, scaled by pa and pb
        tc_fence_after();
#pragma unroll
        for (int sl = 0; sl < kSlabs; ++sl) {
          uint32_t v[kR];
          tmem_ld<kR>(tO + ((i & 1u) * kSlabs + sl) * kN + lane_off, v);
          tmem_ld_wait();
#pragma unroll
          for (int r = 0; r < kR; ++r) o[sl][r] = o[sl][r] * pa[r] + __uint_as_float(v[r]) * pb[r];
        }
        tc_fence_before();
      };
      fetch(g.t0);
      for (int t = g.t0; t < g.t1; ++t, ++tile) {
        const float ks = k_next, vs = v_next;
        if (t + 1 < g.t1) fetch(t + 1);
        const int j = t * kTileTokens + tok;
        const bool live = vs != 0.f;
        const float kv = static_cast<float>(static_cast<int>(__float_as_uint(vs) >> 23) - 127);
        const float inv_v = live ? 1.f / vs : 0.f;
        ok = mbar_wait(&sh->s_full[tile & 1u], (tile >> 1) & 1u, abort) && ok;
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        float x[kR];
        {
          uint32_t v[kR];
          tmem_ld<kR>(tS + (tile & 1u) * kN + lane_off, v);
          tmem_ld_wait();
#pragma unroll
          for (int r = 0; r < kR; ++r) x[r] = __uint_as_float(v[r]) * (ks * rs[r]) + kv;
        }
        tc_fence_before();
        // rows see j <= pos and j > pos - window; every row sees a tile inside both
        const bool inside = (t + 1) * kTileTokens <= pos0 + 1 &&
                            (p.window == 0 || t * kTileTokens > pos0 + g.i1 - g.i0 - 1 - p.window);
        if (!inside) {
#pragma unroll
          for (int r = 0; r < kR; ++r) {
            const int pos = pos0 + r / p.group;
            if (j > pos || (p.window > 0 && j <= pos - p.window)) x[r] = -INFINITY;
          }
        }
        float* mine = sh->tile_max[tile & 1u][quad];
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          if (!live) x[r] = -INFINITY;
          const float w = warp_max(x[r]);
          if (lane == 0) mine[r] = w;
        }
        // a wait that gave up in any warp, here or since the last barrier, ends all four
        if (!(all = named_bar_and(ok))) break;
        float mt[kR];
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          mt[r] = fmaxf(fmaxf(sh->tile_max[tile & 1u][0][r], sh->tile_max[tile & 1u][1][r]),
                        fmaxf(sh->tile_max[tile & 1u][2][r], sh->tile_max[tile & 1u][3][r]));
          x[r] = ex2(x[r] - (mt[r] == -INFINITY ? 0.f : mt[r]) + kWeightTop);
        }
        // P of the tile before has been read, and its O is ready
        if (t > g.t0) {
          const uint32_t i = tile - 1;
          ok = ok && mbar_wait(&sh->o_full[i & 1u], (i >> 1) & 1u, abort);
          ok = __all_sync(0xffffffffu, ok);
        }
        // tokens that do not count may hold anything: their rows of V become zero
        if (__any_sync(0xffffffffu, !live)) {
#pragma unroll
          for (int sl = 0; sl < kSlabs; ++sl) {
            const uint32_t u = (2 * tile + 1) * kSlabs + sl, slot = u % kRing;
            ok = ok && mbar_wait(&sh->full[slot], (u / kRing) & 1u, abort);
            ok = __all_sync(0xffffffffu, ok);
            if (ok && !live) {
              uint4* row = reinterpret_cast<uint4*>(sRing + slot * C::kSlabBytes + tok * kRowBytes);
#pragma unroll
              for (int i = 0; i < kRowBytes / 16; ++i) row[i] = make_uint4(0, 0, 0, 0);
            }
          }
        }
        if (!ok) sh->abort = 1;  // found at the next barrier; nothing below waits
        {
          float y[kR];
#pragma unroll
          for (int r = 0; r < kR; ++r) y[r] = x[r];
#pragma unroll
          for (int part = 0; part < kWeightParts; ++part) {
#pragma unroll
            for (int r = 0; r < kR; r += 2) {
              const uint32_t c = e5m2x2(y[r], y[r + 1]);
              const float2 f = from_e5m2x2(c);
              y[r] -= f.x;
              y[r + 1] -= f.y;
              sP[part * C::kPBytes + swz<128>(r, tok)] = static_cast<uint8_t>(c);
              sP[part * C::kPBytes + swz<128>(r + 1, tok)] = static_cast<uint8_t>(c >> 8);
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->p_full);
        if (t > g.t0) take_output(tile - 1);
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          const float mn = fmaxf(m[r], mt[r]), ref = mn == -INFINITY ? 0.f : mn;
          pa[r] = ex2(m[r] - ref);
          pb[r] = ex2(mt[r] - ref);
          m[r] = mn;
          l[r] = l[r] * pa[r] + (x[r] * inv_v) * pb[r];
        }
      }
      if (!all) break;
      const uint32_t i = tile - 1;
      ok = mbar_wait(&sh->o_full[i & 1u], (i >> 1) & 1u, abort);
      ok = __all_sync(0xffffffffu, ok);
      take_output(i);
      // row sums over the tile's tokens, then the rows
#pragma unroll
      for (int r = 0; r < kR; ++r) {
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], s);
        if (lane == 0) sh->row_sum[quad][r] = l[r];
      }
      if (!(all = named_bar_and(ok))) break;
      const bool whole = g.starts && g.ends;
      float* part = part_slot(p, blockIdx.x, g.starts);
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        if (r >= rows) break;
        const float sum = (sh->row_sum[0][r] + sh->row_sum[1][r]) + (sh->row_sum[2][r] + sh->row_sum[3][r]);
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        const float stat = sum > 0.f ? m[r] - kWeightTop + log2f(sum) : -INFINITY;
        const int row = g.s.row0 + g.i0 + r / p.group, head = g.h * p.group + r % p.group;
#pragma unroll
        for (int sl = 0; sl < kSlabs; ++sl) {
          const int d = sl * kRowBytes + tok;
          if (kRowBytes < 128 && tok >= kRowBytes) continue;  // head_dim 64: lanes past the head
          if (whole) from_f(o[sl][r] * inv, static_cast<T*>(p.out) + row * p.o_ts + head * p.o_hs + d);
          else part[r * (kD + 1) + d] = o[sl][r] * inv;
        }
        if (tok == 0) {
          if (!whole) part[r * (kD + 1) + kD] = stat;
          else if (p.lse) p.lse[static_cast<int64_t>(row) * p.q_heads + head] = stat * kLn2;
        }
      }
      if (g.starts && tok == 0) {
        int2 j = make_int2(-1, -1);
        if (!whole) {
          const TileSpan sp = unit_span(p, g.s, g.w);
          // the unit's tiles are contiguous in the total; this run holds the first of them
          const int64_t first = sh->run.begin + (sh->run.tiles - walk.left) - (g.t1 - g.t0);
          j = make_int2(blockIdx.x, run_of(sh->run.total, sh->run.runs, first + (sp.last - sp.first) - 1));
        }
        *join_of(p, g.b, g.h, g.w) = j;
      }
      if (!(all = named_bar_and(ok))) break;  // row_sum and row_scale are free again
    }
    if (!all && lane == 0) {
      set_error(p.g.err, RIMURU_DEV_TIMEOUT);
      sh->abort = 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
}

template <typename T, int kD, int kR>
cudaError_t launch(const AttnArgs& a, const CUtensorMap& tm, cudaStream_t s) {
  constexpr int kQParts = std::is_same<T, __nv_bfloat16>::value ? 2 : 3;
  constexpr int smem = DecodeCfg<kD, kR, kQParts>::kSmem;
  auto* fn = kv_decode_kernel<T, kD, kR>;
  static SmemOnce once;
  cudaError_t e = once.set(reinterpret_cast<const void*>(fn), smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.runs);
  cfg.blockDim = dim3(kDecodeThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, a, tm);
}
template <typename T, int kD>
cudaError_t launch_rows(const AttnArgs& a, const CUtensorMap& tm, cudaStream_t s) {
  return a.unit_rows <= 8 ? launch<T, kD, 8>(a, tm, s) : launch<T, kD, 16>(a, tm, s);
}
template <typename T>
cudaError_t launch_dim(const AttnArgs& a, const CUtensorMap& tm, cudaStream_t s) {
  if (a.g.head_dim == 64) return launch_rows<T, 64>(a, tm, s);
  if (a.g.head_dim == 128) return launch_rows<T, 128>(a, tm, s);
  return launch_rows<T, 256>(a, tm, s);
}

// ---------------------------------------------------------------------- join
// One CTA per (unit, query row x group): adds the runs' partial rows, weighted
// by their share of the softmax sum, in run order.  Rows of sequences without
// any tile become zero here.
template <typename T>
__global__ void __launch_bounds__(128) kv_join_kernel(const __grid_constant__ AttnArgs p) {
  const int r = blockIdx.y, w = blockIdx.x % p.units_per_pair;
  const int pair = blockIdx.x / p.units_per_pair, b = pair / p.g.kv_heads, h = pair % p.g.kv_heads;
  grid_dep_wait();
  const int D = p.g.head_dim;
  int row0 = p.s.cu ? p.s.cu[b] : b;
  int n = p.s.cu ? p.s.cu[b + 1] - row0 : 1;
  const SeqShape s = seq_shape(p, b);
  if (!s.ok) {  // inconsistent arguments: zero what of its rows lies inside the arrays
    n = min(min(n, p.max_q), p.s.rows - row0);
    if (row0 < 0) n = 0;
  }
  const int per = p.unit_rows / p.group, i = w * per + r / p.group;
  if (r >= per * p.group || i >= n) return;
  const int row = row0 + i, head = h * p.group + r % p.group;
  T* out = static_cast<T*>(p.out) + row * p.o_ts + head * p.o_hs;
  float* lse = p.lse ? p.lse + static_cast<int64_t>(row) * p.q_heads + head : nullptr;
  TileSpan t{0, 0};
  if (s.ok) t = unit_span(p, s, w);
  if (t.first >= t.last) {
    for (int d = threadIdx.x; d < D; d += blockDim.x) from_f(0.f, out + d);
    if (lse && threadIdx.x == 0) *lse = -INFINITY;
    return;
  }
  const int2 j = *join_of(p, b, h, w);
  if (j.x < 0) return;  // finished by one run
  float top = -INFINITY;
  const auto slot = [&](int c) { return part_slot(p, c, c == j.x) + static_cast<int64_t>(r) * (D + 1); };
  for (int c = j.x; c <= j.y; ++c) top = fmaxf(top, slot(c)[D]);
  const float ref = top == -INFINITY ? 0.f : top;
  float sum = 0.f, acc[2] = {0.f, 0.f};
#pragma unroll 4
  for (int c = j.x; c <= j.y; ++c) {
    const float* q = slot(c);
    const float e = ex2(q[D] - ref);
    sum += e;
    if (threadIdx.x < D) acc[0] += e * q[threadIdx.x];
    if (threadIdx.x + 128 < D) acc[1] += e * q[threadIdx.x + 128];
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  if (threadIdx.x < D) from_f(acc[0] * inv, out + threadIdx.x);
  if (threadIdx.x + 128 < D) from_f(acc[1] * inv, out + threadIdx.x + 128);
  if (lse && threadIdx.x == 0) *lse = sum > 0.f ? (ref + log2f(sum)) * kLn2 : -INFINITY;
}

}  // namespace

int kv_decode_runs(int sms, int head_dim) { return sms * (head_dim <= 128 ? 2 : 1); }

cudaError_t launch_kv_decode(const AttnArgs& a, int dtype, const CUtensorMap& tm, cudaStream_t s) {
  return dtype == RIMURU_BF16 ? launch_dim<__nv_bfloat16>(a, tm, s) : launch_dim<__half>(a, tm, s);
}

cudaError_t launch_kv_join(const AttnArgs& a, int dtype, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.s.num_seqs * a.g.kv_heads * a.units_per_pair),
                     static_cast<unsigned>(a.unit_rows));
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return dtype == RIMURU_BF16 ? cudaLaunchKernelEx(&cfg, kv_join_kernel<__nv_bfloat16>, a)
                              : cudaLaunchKernelEx(&cfg, kv_join_kernel<__half>, a);
}

}  // namespace rimuru
