// Attention of a few query rows (at most 16 per key/value head) over the 8-bit
// paged cache: decode steps.
//
// Bound: HBM, one read of the codes.  The codes go from the pages to the tensor
// cores as they are: TMA brings 128 tokens of K and V (one box per page) into
// swizzled shared memory, and tcgen05 multiplies them as the M = 128 operand,
//   S^T [tokens x rows] = K Q^T,     O^T [head_dim x rows] = V^T P,
// so nothing is ever widened.  The few-row operands Q and P are 16-bit or fp32
// quantities: each is written as a sum of 8-bit floats and the products of the
// parts are added.  Q takes e4m3 parts, 4 significant bits each: the element
// rounded, then 16 times the rest, and for f16 16 times the rest of that.  With the
// row scaled to (224, 448], two parts hold a bf16 element exactly down to 2^-6 of that
// scale and within 2^-14 below, three an f16 element down to 2^-7 and within 2^-17
// (without the factors both ended at 2^-10, and a score beside one loud channel of
// 4096 was off by 0.03).  P
// is rounded to f16 and cut into four e5m2 parts, which is exact: an e5m2 number
// is the upper byte of an f16 one, so a part is that byte and the rest an exact
// f16 difference.  Weights are kept down to 2^-27 of the reference (three e4m3
// parts flushed below 2^-18, which showed in output elements whose heaviest
// tokens have a V near zero).
//
// Softmax: thread = token.  The V scale of a token is a power of two 2^k and is
// added to its score, x + k, so the weight that meets the code of V is
// 2^(x + k - ref), bounded whatever the scales, and the row sum takes 2^(x - ref)
// by an exact multiplication.  ref follows the largest x + k seen, but only once
// a token passes it by more than 2^4: until then O stays in TMEM and adds up
// there, and a tile costs its barrier one predicate.  When ref moves, O is
// brought into registers, rescaled, and TMEM starts afresh.
//
// The parts of Q and of P lie side by side as columns of one MMA (8 rows: N = 16
// or 32), so each byte of K and V is read from shared memory once, and are
// added up in registers.
//
// Warp 0 copies (it also reads the page table and the scales, 32 pages at a
// time), warp 1 issues the MMAs, warp 2 prepares Q of the next segment, warps
// 3-6 do the softmax.  S and O are double buffered in TMEM, so K Q^T of the next
// tile, of the next segment too, runs during the softmax of this one.
//
// Two sequences of 130,000 keys, 16/2 heads of 256 (264 MB): 50 us with the join,
// 5.3 TB/s; a CTA takes 2,790 cycles a 64 KiB tile, the copy rate, after 5 us to its
// first.  64 sequences of 1 to 4014 keys, 32/4 heads of 128 (32 MB): 16.9 us; in f16
// 27.6, because the third part of Q takes the shared memory of the second CTA an SM.
#include <cuda_fp8.h>

#include <algorithm>

#include "kv_attn.h"

namespace rimuru {
namespace {

using namespace dev;

constexpr int kDecodeThreads = 224;
constexpr int kWeightParts = 4;
constexpr int kRestTimes = 16;       // what a part of Q leaves is multiplied by this: at most 16 of 448
constexpr float kWeightTop = 11.f;   // a weight at the reference is 2^11
constexpr float kWeightSlack = 4.f;  // and may pass it by 2^4: f16 ends at 2^16
constexpr float kNoRef = -1e30f;     // the reference of a row that has seen no key
constexpr int kMetaRing = 8;

constexpr int decode_ctas(int head_dim, int rows) { return head_dim <= 128 && rows <= 8 ? 2 : 1; }

template <int kD, int kR, int kQParts>
struct DecodeCfg {
  static constexpr int kRowBytes = kD < 128 ? kD : 128;  // bytes of a token in one slab
  static constexpr int kSlabs = kD / kRowBytes;           // slabs of a K or V tile
  static constexpr int kSlabBytes = kTileTokens * kRowBytes;
  static constexpr int kCtas = decode_ctas(kD, kR);  // per SM
  static constexpr int kRing = kCtas == 1 ? (kR == 8 ? 12 : 10) : kD == 64 ? 10 : 6;  // slabs
  static constexpr int kNS = (kQParts * kR + 15) / 16 * 16;  // columns of S: part x row
  static constexpr int kNO = kWeightParts * kR;              // columns of O
  static constexpr int kQBytes = kNS * kD;  // Q: kSlabs x [kNS][kRowBytes]
  static constexpr int kPBytes = kNO * 128;  // P: [128 tokens][kNO]
  static constexpr int kTmem = 2 * kNS + kSlabs * kNO;  // S twice, O
  static constexpr int kTmemCols = kTmem <= 64 ? 64 : kTmem <= 128 ? 128 : kTmem <= 256 ? 256 : 512;
  static constexpr int kSmem = 1024 + kRing * kSlabBytes + 2 * kQBytes + 2 * kPBytes;
};

struct DecodeShared {
  uint64_t full[12], empty[12];
  uint64_t meta_full[kMetaRing];
  uint64_t q_full[2], q_empty[2], p_full[2];
  uint64_t s_full[2], o_full[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int fresh[2];  // the tile's O starts afresh
  RunStart run;
  uint64_t scratch[8];
  float2 meta[kMetaRing][8];  // per page of a tile: scales of K and V; V 0: no such page
  float tile_max[4][kDecodeMaxRows];
  float row_scale[2][kDecodeMaxRows];
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
// 1 when the predicate holds in any of the 128 softmax threads (barrier 1).
__device__ __forceinline__ bool named_bar_or(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\t"
      "setp.ne.u32 a, %1, 0;\n\t"
      "bar.red.or.pred b, 1, 128, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}\n"
      : "=r"(r)
      : "r"(v ? 1u : 0u)
      : "memory");
  return r != 0;
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
// Sums of kParts blocks of kR columns of this thread's TMEM lane; every block was
// multiplied by kTimes as often as it is blocks from the first.
template <int kParts, int kR, int kTimes>
__device__ __forceinline__ void tmem_sum(uint32_t t, float (&x)[kR]) {
  uint32_t v[kParts][kR];
#pragma unroll
  for (int part = 0; part < kParts; ++part) {
    if constexpr (kR == 8) tmem_ld8(t + part * kR, v[part]);
    else tmem_ld16(t + part * kR, v[part]);
  }
  tmem_ld_wait();
#pragma unroll
  for (int r = 0; r < kR; ++r) {
    x[r] = __uint_as_float(v[kParts - 1][r]);  // smallest parts first
#pragma unroll
    for (int part = kParts - 2; part >= 0; --part)
      x[r] = kTimes == 1 ? x[r] + __uint_as_float(v[part][r]) : fmaf(x[r], 1.f / kTimes, __uint_as_float(v[part][r]));
  }
}

template <typename T, int kD, int kR>
__global__ void __launch_bounds__(kDecodeThreads, decode_ctas(kD, kR))
    kv_decode_kernel(const __grid_constant__ AttnArgs p, const __grid_constant__ CUtensorMap tm) {
  constexpr int kQParts = std::is_same<T, __nv_bfloat16>::value ? 2 : 3;
  using C = DecodeCfg<kD, kR, kQParts>;
  constexpr int kNS = C::kNS, kNO = C::kNO;
  constexpr int kSlabs = C::kSlabs, kRing = C::kRing, kRowBytes = C::kRowBytes;
  constexpr uint32_t kSwizzle = kRowBytes == 128 ? 2 : 4;
  constexpr uint32_t kAtom = 8 * kRowBytes;  // eight rows
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sRing = smem;
  uint8_t* sQ = sRing + kRing * C::kSlabBytes;
  uint8_t* sP = sQ + 2 * C::kQBytes;
  __shared__ DecodeShared sh_;
  DecodeShared* sh = &sh_;
  volatile int* abort = &sh->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sh->full[i], 1);
      mbar_init(&sh->empty[i], 1);
    }
    for (int i = 0; i < kMetaRing; ++i) mbar_init(&sh->meta_full[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->p_full[i], 4);
      mbar_init(&sh->q_full[i], 1);
      mbar_init(&sh->q_empty[i], 4);
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
  const uint32_t tS = tmem, tO = tmem + 2 * kNS;
  const int P = p.g.page_tokens, log_p = 31 - __clz(P);
  RunWalk walk;
  walk.begin_run(p, sh->run);
  Segment g;

  if (warp == 0) {
    // ---------------------------------------------------------------- copies
    // Unit 2 i is the K tile i of the run, unit 2 i + 1 its V tile; a unit is
    // kSlabs slots of the ring.  The warp holds the ids and scales of 32 pages,
    // one per lane (`boxes` pages are a tile), and the ids of the next 32.
    const uint64_t pol = policy_evict_first();
    const int boxes = kTileTokens >> log_p;
    uint32_t slot = 0, tile = 0;
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
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, copies)) * P * kRowBytes;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const int y = (kv * p.g.kv_heads + g.h) << log_p;  // first row of the head in the page
#pragma unroll
          for (int sl = 0; sl < kSlabs; ++sl) {
            if (!ok) break;
            const uint32_t i = slot % kRing, ph = (slot / kRing) & 1u;
            ok = mbar_wait_idle(&sh->empty[i], ph ^ 1u, abort);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&sh->full[i], bytes);
            __syncwarp();
            if (copies)
              tma_load_3d(sRing + i * C::kSlabBytes + (lane << log_p) * kRowBytes, &tm, &sh->full[i],
                          sl * kRowBytes, y, mine, pol);
            ++slot;
          }
        }
        // The tile's scales.  The entry's last reader was at least eight tiles back, and
        // the slots just waited for were freed by the MMAs of a later tile than that.
        if (lane >= at && lane < at + boxes)
          sh->meta[tile % kMetaRing][lane - at] = make_float2(ks, vs);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->meta_full[tile % kMetaRing]);
        at += boxes;
      }
    }
    if (!ok && lane == 0) {
      set_error(p.g.err, RIMURU_DEV_TIMEOUT);
      sh->abort = 1;
    }
    // every copy this warp issued must have landed before the CTA exits
    volatile int never = 0;
    for (uint32_t j = slot > kRing ? slot - kRing : 0u; j < slot; ++j)
      mbar_wait_idle(&sh->full[j % kRing], (j / kRing) & 1u, &never);
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMAs
    // The whole warp walks and waits, and one lane issues, so that addresses stay
    // warp-uniform.
    constexpr uint32_t id_s = idesc_f8_f32(128, kNS, false, false, false);
    constexpr uint32_t id_o = idesc_f8_f32(128, kNO, /*a_mn=*/true, /*b_mn=*/true, /*b_e5m2=*/true);
    const uint32_t tb = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t ring_s = smem_u32(sRing), q_s = smem_u32(sQ), p_s = smem_u32(sP);
    uint32_t slot = 0, phase = 0;  // the next slot of the ring
    bool ok = true;
    const auto wait = [&](uint64_t* bar, uint32_t ph) {
      ok = ok && mbar_wait_idle(bar, ph, abort);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
    };
    const auto step = [&](uint32_t* at, uint32_t* ph, uint32_t n) {
      *at += n;
      if (*at >= kRing) *at -= kRing, *ph ^= 1u;
    };
    const auto scores = [&](uint32_t i, uint32_t seg) {  // S^T of the run's tile i, in the next K unit
      uint32_t at = slot, ph = phase;
#pragma unroll
      for (int sl = 0; sl < kSlabs; ++sl) {
        wait(&sh->full[at], ph);
        if (ok && elect_one()) {
          const uint32_t a0 = ring_s + at * C::kSlabBytes;
          const uint32_t b0 = q_s + (seg & 1u) * C::kQBytes + sl * kNS * kRowBytes;
#pragma unroll
          for (int k = 0; k < kRowBytes / 32; ++k)
            umma_f8(tb + (i & 1u) * kNS, smem_desc(a0 + 32 * k, 16, kAtom, kSwizzle),
                    smem_desc(b0 + 32 * k, 16, kAtom, kSwizzle), id_s, (sl | k) != 0 ? 1u : 0u);
          umma_commit(&sh->empty[at]);
          if (sl == kSlabs - 1) umma_commit(&sh->s_full[i & 1u]);
        }
        __syncwarp();
        step(&at, &ph, 1);
      }
      step(&slot, &phase, 2 * kSlabs);  // past the tile's V unit
    };
    uint32_t v_slot = kSlabs, v_phase = 0;
    const auto outputs = [&](uint32_t i) {  // O^T of the run's tile i, in the next V unit
      wait(&sh->p_full[i & 1u], (i >> 1) & 1u);
      const uint32_t keep = sh->fresh[i & 1u] ? 0u : 1u;
      uint32_t at = v_slot, ph = v_phase;
#pragma unroll
      for (int sl = 0; sl < kSlabs; ++sl) {
        wait(&sh->full[at], ph);
        if (ok && elect_one()) {
          const uint32_t a0 = ring_s + at * C::kSlabBytes;
#pragma unroll
          for (int k = 0; k < 4; ++k)  // 32 tokens: four groups of eight rows
            umma_f8(tb + 2 * kNS + sl * kNO,
                    smem_desc(a0 + 4 * k * kAtom, C::kSlabBytes, kAtom, kSwizzle),
                    smem_desc(p_s + (i & 1u) * C::kPBytes + 32 * k * kNO, C::kPBytes, 8 * kNO,
                              kNO == 64 ? 4 : 6),
                    id_o, k != 0 ? 1u : keep);
          umma_commit(&sh->empty[at]);
          if (sl == kSlabs - 1) umma_commit(&sh->o_full[i & 1u]);
        }
        __syncwarp();
        step(&at, &ph, 1);
      }
      step(&v_slot, &v_phase, 2 * kSlabs);
    };
    // S of the next tile is issued before O of this one.  Its buffer and this
    // one's are free: the weights of the tile before were written after the
    // softmax warps had read them.
    uint32_t tile = 0, seg = 0;
    if (walk.next(p, &g)) {
      wait(&sh->q_full[0], 0);
      scores(0, 0);
      for (int t = g.t0; ok; ++tile) {
        bool more = true;
        if (++t == g.t1) {
          more = walk.next(p, &g);
          if (more) {
            ++seg;
            t = g.t0;
            wait(&sh->q_full[seg & 1u], (seg >> 1) & 1u);
          }
        }
        if (more) scores(tile + 1, seg);
        outputs(tile);
        if (!more) break;
      }
    }
    if (!ok && lane == 0) {
      set_error(p.g.err, RIMURU_DEV_TIMEOUT);
      sh->abort = 1;
    }
    if (elect_one()) umma_commit(&sh->drain);  // all MMAs are finished before TMEM is released
    __syncwarp();
    volatile int never = 0;
    mbar_wait_idle(&sh->drain, 0, &never);
  } else if (warp == 2) {
    // --------------------------------------------------------------------- Q
    uint32_t seg = 0;
    bool ok = true;
    while (ok && walk.next(p, &g)) {
      constexpr int kPer = kD / 32;
      const uint32_t buf = seg & 1u;
      const int rows = (g.i1 - g.i0) * p.group;
      uint8_t* q_s = sQ + buf * C::kQBytes;
      const T* src = static_cast<const T*>(p.q) + (g.s.row0 + g.i0) * p.q_ts + g.h * p.group * p.q_hs + lane * kPer;
      int of_group = 0;  // the row's place in its group; src is its address
#pragma unroll 1
      for (int half = 0; half < kR; half += 8) {
        T raw[8][kPer];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int r = half + k;
          if (r < rows) {
            if constexpr (kPer == 8) *reinterpret_cast<uint4*>(raw[k]) = *reinterpret_cast<const uint4*>(src);
            else if constexpr (kPer == 4) *reinterpret_cast<uint2*>(raw[k]) = *reinterpret_cast<const uint2*>(src);
            else *reinterpret_cast<uint32_t*>(raw[k]) = *reinterpret_cast<const uint32_t*>(src);
            src += p.q_hs;
            if (++of_group == p.group) of_group = 0, src += p.q_ts - p.group * p.q_hs;
          } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i) from_f(0.f, &raw[k][i]);
          }
        }
        if (half == 0) {
          ok = mbar_wait_idle(&sh->q_empty[buf], ((seg >> 1) & 1u) ^ 1u, abort);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int r = half + k;
          float x[kPer], amax = 0.f;
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            x[i] = to_f(raw[k][i]);
            amax = fmaxf(amax, fabsf(x[i]));
          }
          amax = warp_max(amax);
          // power of two that brings the row's largest magnitude into (224, 448]
          const uint32_t ab = __float_as_uint(amax);
          const int e = max(-100, min(100, static_cast<int>(ab >> 23) - 127 - 8 + ((ab & 0x7FFFFFu) > 0x600000u)));
          const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
          for (int i = 0; i < kPer; ++i) x[i] *= inv;
          const int d0 = lane * kPer, sl = d0 / kRowBytes;
#pragma unroll
          for (int part = 0; part < kQParts; ++part) {
            uint8_t* dst = q_s + sl * kNS * kRowBytes + swz<kRowBytes>(part * kR + r, d0 % kRowBytes);
#pragma unroll
            for (int i = 0; i < kPer; i += 2) {
              const uint32_t c = e4m3x2(x[i], x[i + 1]);
              const float2 f = from_e4m3x2(c);
              x[i] = (x[i] - f.x) * kRestTimes;
              x[i + 1] = (x[i + 1] - f.y) * kRestTimes;
              *reinterpret_cast<uint16_t*>(dst + i) = static_cast<uint16_t>(c);
            }
          }
          // an infinite query has no finite score: its row becomes NaN
          if (lane == 0)
            sh->row_scale[buf][r] =
                amax <= 3.4028234664e38f
                    ? __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * p.scale_log2
                    : __int_as_float(0x7FFFFFFF);
        }
      }
      if (!ok) break;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->q_full[buf]);
      ++seg;
    }
    if (!ok && lane == 0) {
      set_error(p.g.err, RIMURU_DEV_TIMEOUT);
      sh->abort = 1;
    }
  } else {
    // --------------------------------------------------------------- softmax
    const int quad = warp & 3;             // TMEM lanes this warp may read
    const int tok = quad * 32 + lane;      // token of the tile, and row of O^T
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    uint32_t tile = 0, seg = 0;
    // `ok`: this warp's waits came through; `all`: the four warps' did, as agreed
    // at the last barrier.  Only `all` leaves the loops, so no warp waits at a
    // barrier for one that has left.
    bool ok = true, all = true;
    while (all && walk.next(p, &g)) {
      const int rows = (g.i1 - g.i0) * p.group;
      const int pos0 = g.s.len - g.s.n + g.i0;  // position of the first query row
      const int lo = p.window > 0 ? max(0, pos0 - p.window + 1) : 0;
      const uint32_t buf = seg & 1u;
      ok = mbar_wait_idle(&sh->q_full[buf], (seg >> 1) & 1u, abort);
      ok = __all_sync(0xffffffffu, ok);
      // A weight is 2^(x + add) with add = kWeightTop - ref.
      float rs[kR], ref[kR], l[kR], o[kSlabs][kR];
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        rs[r] = sh->row_scale[buf][r];
        ref[r] = kNoRef;
        l[r] = 0.f;
#pragma unroll
        for (int sl = 0; sl < kSlabs; ++sl) o[sl][r] = 0.f;
      }
      const auto add_output = [&]() {  // O of the tiles so far, out of TMEM
        tc_fence_after();
#pragma unroll
        for (int sl = 0; sl < kSlabs; ++sl) {
          float v[kR];
          tmem_sum<kWeightParts, kR, 1>(tO + sl * kNO + lane_off, v);
#pragma unroll
          for (int r = 0; r < kR; ++r) o[sl][r] += v[r];
        }
        tc_fence_before();
      };
      for (int t = g.t0; t < g.t1; ++t, ++tile) {
        ok = mbar_wait_idle(&sh->meta_full[tile % kMetaRing], (tile / kMetaRing) & 1u, abort) && ok;
        ok = __all_sync(0xffffffffu, ok);
        const float2 kvs = sh->meta[tile % kMetaRing][tok >> log_p];
        const int j = t * kTileTokens + tok;
        const bool live = kvs.y != 0.f && j >= lo && j < g.s.len;
        const int ke = static_cast<int>(__float_as_uint(kvs.y) >> 23);  // V scale = 2^(ke - 127)
        const float kv = static_cast<float>(ke - 127);
        const float inv_v = __uint_as_float(static_cast<uint32_t>(254 - ke) << 23);
        ok = mbar_wait_idle(&sh->s_full[tile & 1u], (tile >> 1) & 1u, abort) && ok;
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        float x[kR];
        tmem_sum<kQParts, kR, kRestTimes>(tS + (tile & 1u) * kNS + lane_off, x);
        tc_fence_before();
#pragma unroll
        for (int r = 0; r < kR; ++r) x[r] = live ? x[r] * (kvs.x * rs[r]) + kv : -INFINITY;
        // rows see j <= pos and j > pos - window; every row sees a tile inside both
        const bool inside = (t + 1) * kTileTokens <= pos0 + 1 &&
                            (p.window == 0 || t * kTileTokens > pos0 + g.i1 - g.i0 - 1 - p.window);
        if (!inside) {
          int pos = pos0, of_group = 0;
#pragma unroll
          for (int r = 0; r < kR; ++r) {
            if (j > pos || (p.window > 0 && j <= pos - p.window)) x[r] = -INFINITY;
            if (++of_group == p.group) of_group = 0, ++pos;
          }
        }
        bool raise = !ok;  // a wait that gave up is settled where the reference moves
#pragma unroll
        for (int r = 0; r < kR; ++r) raise |= x[r] > ref[r] + kWeightSlack;
        if (named_bar_or(raise)) {
          float top[kR];
#pragma unroll
          for (int r = 0; r < kR; ++r) top[r] = warp_max(x[r]);
          if (lane == 0) {
#pragma unroll
            for (int r = 0; r < kR; r += 4)
              *reinterpret_cast<float4*>(&sh->tile_max[quad][r]) =
                  make_float4(top[r], top[r + 1], top[r + 2], top[r + 3]);
          }
          if (!(all = named_bar_and(ok))) break;
          if (t > g.t0) {  // every O MMA so far is done
            ok = mbar_wait_idle(&sh->o_full[(tile - 1) & 1u], ((tile - 1) >> 1) & 1u, abort);
            ok = __all_sync(0xffffffffu, ok);
            add_output();
          }
#pragma unroll
          for (int r = 0; r < kR; ++r) {
            const float now = fmaxf(fmaxf(fmaxf(sh->tile_max[0][r], sh->tile_max[1][r]),
                                          fmaxf(sh->tile_max[2][r], sh->tile_max[3][r])),
                                    ref[r]);
            const float f = ex2(ref[r] - now);
            ref[r] = now;
            l[r] *= f;
#pragma unroll
            for (int sl = 0; sl < kSlabs; ++sl) o[sl][r] *= f;
          }
          if (tok == 0) sh->fresh[tile & 1u] = 1;
        } else if (tok == 0) {
          sh->fresh[tile & 1u] = t == g.t0;
        }
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          x[r] = ex2(x[r] + (kWeightTop - ref[r]));
          l[r] += x[r] * inv_v;
        }
        if (t > g.t0 + 1) {  // the weights two tiles back have been read
          ok = mbar_wait_idle(&sh->o_full[tile & 1u], ((tile - 2) >> 1) & 1u, abort) && ok;
          ok = __all_sync(0xffffffffu, ok);
        }
        // tokens that do not count may hold anything: their rows of V become zero
        if (__any_sync(0xffffffffu, !live)) {
#pragma unroll
          for (int sl = 0; sl < kSlabs; ++sl) {
            const uint32_t u = (2 * tile + 1) * kSlabs + sl, slot = u % kRing;
            ok = mbar_wait_idle(&sh->full[slot], (u / kRing) & 1u, abort) && ok;
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
          // the token's row of P: kNO bytes, part x row, in 16-byte chunks
          uint32_t c[kNO / 4];
          __half2 y[kR / 2];
#pragma unroll
          for (int r = 0; r < kR / 2; ++r) y[r] = __floats2half2_rn(x[2 * r], x[2 * r + 1]);
#pragma unroll
          for (int part = 0; part < kWeightParts; ++part) {
#pragma unroll
            for (int r = 0; r < kR / 2; r += 2) {
              const uint32_t a = *reinterpret_cast<const uint32_t*>(&y[r]);
              const uint32_t b = *reinterpret_cast<const uint32_t*>(&y[r + 1]);
              c[(part * kR + 2 * r) / 4] = __byte_perm(a, b, 0x7531);
              if (part + 1 < kWeightParts) {
                const uint32_t ah = a & 0xFF00FF00u, bh = b & 0xFF00FF00u;
                y[r] = __hsub2(y[r], *reinterpret_cast<const __half2*>(&ah));
                y[r + 1] = __hsub2(y[r + 1], *reinterpret_cast<const __half2*>(&bh));
              }
            }
          }
          uint8_t* row = sP + (tile & 1u) * C::kPBytes + tok * kNO;
#pragma unroll
          for (int i = 0; i < kNO / 16; ++i) {
            const int at = kNO == 64 ? (i ^ (tok >> 1)) & 3 : (i ^ (tok >> 2)) & 1;
            *reinterpret_cast<uint4*>(row + 16 * at) =
                make_uint4(c[4 * i], c[4 * i + 1], c[4 * i + 2], c[4 * i + 3]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->p_full[tile & 1u]);
      }
      if (!all) break;
      if (lane == 0) mbar_arrive(&sh->q_empty[buf]);  // S of the segment's last tile is complete
      // Row sums over the tokens: each exchange halves the rows a lane holds, so
      // lane bits 4, 3, (2, 1) name its row in the end.
#pragma unroll
      for (int n = kR / 2, bit = 16; bit > 0; n /= 2, bit /= 2) {
        if (n >= 1) {
#pragma unroll
          for (int r = 0; r < (n >= 1 ? n : 1); ++r) {
            const bool up = lane & bit;
            const float give = up ? l[r] : l[r + n];
            l[r] = (up ? l[r + n] : l[r]) + __shfl_xor_sync(0xffffffffu, give, bit);
          }
        } else {
          l[0] += __shfl_xor_sync(0xffffffffu, l[0], bit);
        }
      }
      constexpr int kLanesPerRow = 32 / kR;
      if (lane % kLanesPerRow == 0) sh->row_sum[quad][lane / kLanesPerRow] = l[0];
      const uint32_t i = tile - 1;
      ok = mbar_wait_idle(&sh->o_full[i & 1u], (i >> 1) & 1u, abort) && ok;
      ok = __all_sync(0xffffffffu, ok);
      add_output();
      if (!(all = named_bar_and(ok))) break;
      const bool whole = g.starts && g.ends;
      // lane r finishes the statistics of row r
      float sum = 0.f, mr = 0.f;
      if (lane < kR)
        sum = (sh->row_sum[0][lane] + sh->row_sum[1][lane]) + (sh->row_sum[2][lane] + sh->row_sum[3][lane]);
#pragma unroll
      for (int r = 0; r < kR; ++r) mr = lane == r ? ref[r] : mr;
      const float inv = sum > 0.f ? 1.f / sum : sum;  // 0 for a row that sees nothing; NaN stays
      const float stat = sum > 0.f ? mr - kWeightTop + __log2f(sum) : sum == 0.f ? -INFINITY : sum;
      const int64_t slot = part_slot(p, blockIdx.x, g.starts);
      const bool has_d = kRowBytes == 128 || tok < kRowBytes;  // head_dim 64: lanes past the head
      if (whole) {
        const int row = g.s.row0 + g.i0, head = g.h * p.group;
        T* dst = static_cast<T*>(p.out) + row * p.o_ts + head * p.o_hs + tok;
        int of_group = 0;
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          const float f = __shfl_sync(0xffffffffu, inv, r);
          if (r >= rows) break;
#pragma unroll
          for (int sl = 0; sl < kSlabs; ++sl)
            if (has_d) from_f(o[sl][r] * f, dst + sl * kRowBytes);
          dst += p.o_hs;
          if (++of_group == p.group) of_group = 0, dst += p.o_ts - p.group * p.o_hs;
        }
        if (p.lse && quad == 0 && lane < rows)
          p.lse[static_cast<int64_t>(row + lane / p.group) * p.q_heads + head + lane % p.group] = stat * kLn2;
      } else {
        float* dst = p.part + slot * kD + tok;
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          const float f = __shfl_sync(0xffffffffu, inv, r);
          if (r >= rows) break;
#pragma unroll
          for (int sl = 0; sl < kSlabs; ++sl)
            if (has_d) dst[r * kD + sl * kRowBytes] = o[sl][r] * f;
        }
        if (quad == 0 && lane < rows) p.stat[slot + lane] = stat;
      }
      if (tok == 0) note_cut(p, g, sh->run.cut, blockIdx.x);
      ++seg;
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
// Adds the runs' partial rows, weighted by their share of the softmax sum, in
// run order.  At most one unit is cut per run, so the grid goes over the runs and
// blocks of rows (over the units, most of which one run has finished, the join
// of a 2048-token chunk took 21 us instead of 15, for 40 MB of parts).  A warp takes
// kRows rows, whose loads it keeps under way together; or, when few units are cut
// into many runs (a long context), a CTA takes one row of a unit, its warps split
// the runs, and their sums meet in shared memory in warp order.
constexpr int kJoinWarps = 8;

template <typename T, int kPer>
__device__ __forceinline__ void store_row(T* out, const float (&x)[kPer]) {
  T v[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) from_f(x[k], v + k);
  if constexpr (kPer == 8) *reinterpret_cast<uint4*>(out) = *reinterpret_cast<uint4*>(v);
  else if constexpr (kPer == 4) *reinterpret_cast<uint2*>(out) = *reinterpret_cast<uint2*>(v);
  else *reinterpret_cast<uint32_t*>(out) = *reinterpret_cast<uint32_t*>(v);
}
template <int kPer>
__device__ __forceinline__ void load_part(const float* q, float (&v)[kPer]) {
  if constexpr (kPer >= 4) {
#pragma unroll
    for (int i = 0; i < kPer; i += 4) *reinterpret_cast<float4*>(v + i) = *reinterpret_cast<const float4*>(q + i);
  } else {
    *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(q);
  }
}

// The rows of units without any tile are zero (every query head's, by the warps
// of the CTAs past the runs): a lane looks at a unit, the warp writes its rows.
template <typename T, int kD>
__device__ void zero_rows(const AttnArgs& p, int first, int step) {
  const int lane = threadIdx.x & 31;
  const int64_t units = static_cast<int64_t>(p.s.num_seqs) * p.units_per_pair;
  for (int64_t at = static_cast<int64_t>(first) * 32; at < units; at += static_cast<int64_t>(step) * 32) {
    int row0 = 0, n = 0;
    if (at + lane < units) {
      const int b = static_cast<int>((at + lane) / p.units_per_pair), w = static_cast<int>((at + lane) % p.units_per_pair);
      const RowSpan r = empty_rows(p, seq_shape(p, b), b, w);
      row0 = r.row0, n = r.n;
    }
    for (uint32_t todo = __ballot_sync(0xffffffffu, n > 0); todo != 0; todo &= todo - 1) {
      const int from = __ffs(todo) - 1;
      const int r0 = __shfl_sync(0xffffffffu, row0, from), m = __shfl_sync(0xffffffffu, n, from);
      const float none[kD / 32] = {};
      for (int i = 0; i < m * p.q_heads; ++i) {
        const int64_t row = r0 + i / p.q_heads, head = i % p.q_heads;
        store_row(static_cast<T*>(p.out) + row * p.o_ts + head * p.o_hs + lane * (kD / 32), none);
        if (p.lse && lane == 0) p.lse[row * p.q_heads + head] = -INFINITY;
      }
    }
  }
}

template <typename T, int kD, int kRows>  // kRows 0: a row per CTA, its runs split over the warps
__global__ void __launch_bounds__(32 * kJoinWarps) kv_join_kernel(const __grid_constant__ AttnArgs p) {
  constexpr int kPer = kD / 32, kN = kRows > 0 ? kRows : 1;
  __shared__ float sums[kRows == 0 ? kJoinWarps : 1][kD];
  __shared__ float weight[kJoinWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int units = kRows == 0 ? p.s.num_seqs * p.g.kv_heads * p.units_per_pair : p.runs;
  grid_dep_wait();
  if (static_cast<int>(blockIdx.x) >= units) {
    if (blockIdx.y == 0)
      zero_rows<T, kD>(p, (blockIdx.x - units) * kJoinWarps + warp, (gridDim.x - units) * kJoinWarps);
    return;
  }
  int c0 = blockIdx.x;
  int4 cut;
  if (kRows == 0) {  // the unit's entry, if it is cut
    __shared__ int4 found;
    __shared__ int where;
    if (threadIdx.x == 0) where = -1;
    __syncthreads();
    for (int c = threadIdx.x; c < p.runs; c += 32 * kJoinWarps) {
      const int4 e = p.cuts[c];
      if (e.y > 0 && e.z == static_cast<int>(blockIdx.x)) found = e, where = c;
    }
    __syncthreads();
    c0 = where;
    if (c0 < 0) return;
    cut = found;
  } else {
    cut = p.cuts[c0];
  }
  const int rows = cut.y % 512, h = cut.y / 512;  // no rows: no entry
  const int r0 = kRows == 0 ? blockIdx.y : (blockIdx.y * kJoinWarps + warp) * kN;
  if (r0 >= rows) return;
  const auto slot = [&](int c, int r) { return part_slot(p, c, c == c0) + min(r, rows - 1); };
  float ref[kN], sum[kN], acc[kN][kPer];
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    float top = -INFINITY;
    for (int c = c0 + lane; c <= cut.w; c += 32) top = fmaxf(top, p.stat[slot(c, r0 + k)]);
    top = warp_max(top);
    ref[k] = top == -INFINITY ? 0.f : top;
    sum[k] = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[k][i] = 0.f;
  }
#pragma unroll 2
  for (int c = c0 + (kRows == 0 ? warp : 0); c <= cut.w; c += kRows == 0 ? kJoinWarps : 1) {
    float v[kN][kPer];
#pragma unroll
    for (int k = 0; k < kN; ++k) load_part(p.part + slot(c, r0 + k) * kD + lane * kPer, v[k]);
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const float e = ex2(p.stat[slot(c, r0 + k)] - ref[k]);
      sum[k] += e;
#pragma unroll
      for (int i = 0; i < kPer; ++i) acc[k][i] += e * v[k][i];
    }
  }
  if (kRows == 0) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) sums[warp][lane * kPer + i] = acc[0][i];
    if (lane == 0) weight[warp] = sum[0];
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int k = 1; k < kJoinWarps; ++k) {
      sum[0] += weight[k];
#pragma unroll
      for (int i = 0; i < kPer; ++i) acc[0][i] += sums[k][lane * kPer + i];
    }
  }
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    const int r = r0 + k;
    if (r >= rows) return;
    const float inv = sum[k] > 0.f ? 1.f / sum[k] : sum[k];
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[k][i] *= inv;
    const int i = r / p.group;
    const int64_t row = cut.x + i, head = h * p.group + r - i * p.group;
    store_row(static_cast<T*>(p.out) + row * p.o_ts + head * p.o_hs + lane * kPer, acc[k]);
    if (p.lse && lane == 0)
      p.lse[row * p.q_heads + head] =
          sum[k] > 0.f ? (ref[k] + __log2f(sum[k])) * kLn2 : sum[k] == 0.f ? -INFINITY : sum[k];
  }
}

template <typename T, int kD>
cudaError_t launch_join(const AttnArgs& a, cudaStream_t s) {
  const int64_t pairs = static_cast<int64_t>(a.s.num_seqs) * a.units_per_pair, units = pairs * a.g.kv_heads;
  // With four runs a unit or more, one CTA per row whose warps split the runs.  Else a row a warp
  // while that fits the 64 warps of the SMs (16 sequences of 40 rows: 35.9 us the call, 40.4 with
  // four rows a warp), four rows beyond.
  const bool split = units * 4 <= a.runs;
  const int64_t bound = std::max<int64_t>(1, std::min<int64_t>(a.unit_rows, static_cast<int64_t>(a.max_q) * a.group));
  const int per = split ? 0 : a.runs * bound <= a.sms * 64 ? 1 : 4;
  const int rows = split ? 1 : per * kJoinWarps;  // of a CTA
  const int64_t zero = std::min<int64_t>(a.runs, (pairs + 32 * kJoinWarps - 1) / (32 * kJoinWarps));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((split ? units : a.runs) + zero),
                     static_cast<unsigned>((bound + rows - 1) / rows));
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return split ? cudaLaunchKernelEx(&cfg, kv_join_kernel<T, kD, 0>, a)
         : per == 1 ? cudaLaunchKernelEx(&cfg, kv_join_kernel<T, kD, 1>, a)
                    : cudaLaunchKernelEx(&cfg, kv_join_kernel<T, kD, 4>, a);
}
template <typename T>
cudaError_t join_dim(const AttnArgs& a, cudaStream_t s) {
  if (a.g.head_dim == 64) return launch_join<T, 64>(a, s);
  if (a.g.head_dim == 128) return launch_join<T, 128>(a, s);
  return launch_join<T, 256>(a, s);
}

}  // namespace

int kv_decode_runs(int sms, int head_dim, int rows) { return sms * decode_ctas(head_dim, rows); }

cudaError_t launch_kv_decode(const AttnArgs& a, int dtype, const CUtensorMap& tm, cudaStream_t s) {
  return dtype == RIMURU_BF16 ? launch_dim<__nv_bfloat16>(a, tm, s) : launch_dim<__half>(a, tm, s);
}

cudaError_t launch_kv_join(const AttnArgs& a, int dtype, cudaStream_t s) {
  return dtype == RIMURU_BF16 ? join_dim<__nv_bfloat16>(a, s) : join_dim<__half>(a, s);
}

}  // namespace rimuru
