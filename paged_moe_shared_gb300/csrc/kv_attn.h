// Shared by the attention kernels: arguments, how the work is cut, and the
// layout of the partial results that are joined afterwards.
//
// A unit is a (sequence, key/value head, block of query rows); its work is the
// 128-token tiles of keys that any of its rows sees.  The tiles of all units,
// laid end to end, are cut into equal runs, one per CTA, so the CTAs finish
// together whatever the lengths are, and no length has to be known on the
// host.  A unit that lies within one run is finished there; the others leave
// one partial result per run (normalised rows and their log2 sums), which the
// join kernel adds up in run order.
#pragma once

#include <atomic>

#include "device.cuh"
#include "kv.h"

namespace rimuru {

constexpr int kTileTokens = 128;

struct AttnArgs {
  const void* q;
  void* out;
  float* lse;  // [rows][q_heads] or null
  int64_t q_ts, q_hs, o_ts, o_hs;
  int q_heads, group;  // group = q_heads / kv_heads
  float scale_log2;    // scale * log2(e): scores are kept in base 2
  int window;          // 0: none
  int max_q;           // no sequence has more query rows
  KvSeqs s;
  KvGeom g;
  // work split
  int runs;            // CTAs that share the tiles
  int unit_rows;       // query rows (query x group) of a unit
  int units_per_pair;  // bound of the units of one (sequence, head)
  int2* joins;         // [num_seqs][kv_heads][units_per_pair]: runs (first, last) of a unit cut up
  float* part;         // [2 runs][unit_rows][head_dim + 1] partial results
};

constexpr float kLn2 = 0.69314718055994531f;

// One sequence: its query rows and cached length.  ok == false: the arguments
// disagree and the sequence has no work (its rows become zero).
struct SeqShape {
  int row0, n, len;
  bool ok;
};
__device__ __forceinline__ SeqShape seq_shape(const AttnArgs& p, int b) {
  SeqShape s;
  s.row0 = p.s.cu ? p.s.cu[b] : b;
  s.n = p.s.cu ? p.s.cu[b + 1] - s.row0 : 1;
  s.len = p.s.lens[b];
  s.ok = s.n >= 0 && s.n <= p.max_q && s.row0 >= 0 && s.row0 <= p.s.rows - s.n && s.len >= 0 &&
         s.len <= p.s.table_stride * p.g.page_tokens;
  if (!s.ok || s.n == 0) s.n = 0, s.len = 0;
  return s;
}
// Tiles [first, last) that the query rows i0 .. i1 - 1 of a sequence see.
struct TileSpan {
  int first, last;
};
__device__ __forceinline__ TileSpan tile_span(const AttnArgs& p, const SeqShape& s, int i0, int i1) {
  const int p0 = s.len - s.n + i0, p1 = s.len - s.n + i1;  // positions p0 .. p1 - 1
  TileSpan t;
  t.last = p1 > 0 ? (p1 + kTileTokens - 1) / kTileTokens : 0;
  t.first = p.window > 0 && p0 >= p.window ? (p0 - p.window + 1) / kTileTokens : 0;
  return t;
}
// Query rows [i0, i1) of unit w of a sequence.  A unit holds unit_rows / group
// whole query rows.
__device__ __forceinline__ int units_of(const AttnArgs& p, const SeqShape& s) {
  const int per = p.unit_rows / p.group;
  return (s.n + per - 1) / per;
}
__device__ __forceinline__ TileSpan unit_span(const AttnArgs& p, const SeqShape& s, int w) {
  const int per = p.unit_rows / p.group;
  return tile_span(p, s, w * per, min(s.n, (w + 1) * per));
}
// Tiles of one head of a sequence, over all its units.
__device__ __forceinline__ int64_t pair_tiles(const AttnArgs& p, const SeqShape& s) {
  int64_t n = 0;
  const int u = units_of(p, s);
  for (int w = 0; w < u; ++w) {
    const TileSpan t = unit_span(p, s, w);
    n += t.last - t.first;
  }
  return n;
}

// Run c holds the tiles [run_start(c), run_start(c + 1)) of the total.
__device__ __forceinline__ int64_t run_start(int64_t total, int runs, int c) {
  return total * c / runs;
}
__device__ __forceinline__ int run_of(int64_t total, int runs, int64_t tile) {
  return static_cast<int>(((tile + 1) * runs + total - 1) / total) - 1;
}

// Where a run begins: sequence, head and tile offset within the head's tiles.
struct RunStart {
  int64_t tiles;  // tiles of this run
  int64_t at;     // first tile within (b, h)
  int64_t begin;  // first tile, counted over all units
  int64_t total;
  int runs;       // runs that have tiles
  int b, h;
};

// Found by the whole CTA (every thread calls it; `scratch` is 40 int64 of
// shared memory): thread t sums the tiles of a contiguous share of the
// sequences, the shares are scanned, and the thread whose share holds the
// run's first tile walks its share.
__device__ __forceinline__ void find_run(const AttnArgs& p, int c, int64_t* scratch, RunStart* out) {
  const int t = threadIdx.x, nt = blockDim.x, lane = t & 31, warp = t >> 5;
  const int b0 = static_cast<int>(static_cast<int64_t>(p.s.num_seqs) * t / nt);
  const int b1 = static_cast<int>(static_cast<int64_t>(p.s.num_seqs) * (t + 1) / nt);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) {
    const SeqShape s = seq_shape(p, b);
    if (!s.ok && c == 0) dev::set_error(p.g.err, RIMURU_DEV_BAD_SHAPE);
    mine += pair_tiles(p, s) * p.g.kv_heads;
  }
  int64_t scan = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += v;
  }
  if (lane == 31) scratch[warp] = scan;
  __syncthreads();
  int64_t before = scan - mine, total = 0;
  for (int w = 0; w < nt / 32; ++w) {
    if (w < warp) before += scratch[w];
    total += scratch[w];
  }
  // no run between the first and the last is empty, so every run of a unit leaves a part
  const int runs = static_cast<int>(min(total, static_cast<int64_t>(p.runs)));
  const int64_t begin = c < runs ? run_start(total, runs, c) : total;
  const int64_t end = c < runs ? run_start(total, runs, c + 1) : total;
  if (t == 0) {
    out->tiles = end - begin;
    out->begin = begin;
    out->total = total;
    out->runs = runs;
  }
  if (begin < end && begin >= before && begin < before + mine) {
    int64_t at = begin - before;
    for (int b = b0; b < b1; ++b) {
      const int64_t n = pair_tiles(p, seq_shape(p, b));
      if (at < n * p.g.kv_heads) {
        out->b = b;
        out->h = static_cast<int>(at / n);
        out->at = at % n;
        break;
      }
      at -= n * p.g.kv_heads;
    }
  }
  __syncthreads();
}

// Walks a run segment by segment: the part of a unit that lies in the run.
struct Segment {
  int b, h, w;          // sequence, head, unit
  SeqShape s;
  int i0, i1;           // query rows of the unit
  int t0, t1;           // its tiles within this run
  bool starts, ends;    // holds the unit's first / last tile
};
struct RunWalk {
  int64_t left, at;
  int b, h, w, u;  // next unit; u: units of sequence b
  SeqShape s;
  __device__ __forceinline__ void begin(const AttnArgs& p, const RunStart& r) {
    left = r.tiles;
    if (left <= 0) return;
    b = r.b;
    h = r.h;
    at = r.at;
    s = seq_shape(p, b);
    u = units_of(p, s);
    w = 0;
    while (true) {  // the unit that holds tile `at`
      const TileSpan t = unit_span(p, s, w);
      if (at < t.last - t.first) break;
      at -= t.last - t.first;
      ++w;
    }
  }
  __device__ __forceinline__ bool next(const AttnArgs& p, Segment* g) {
    if (left <= 0) return false;
    TileSpan t;
    while (true) {
      if (w < u) {
        t = unit_span(p, s, w);
        if (t.last > t.first) break;
        ++w;
      } else if (h + 1 < p.g.kv_heads && u > 0) {
        ++h, w = 0;
      } else {
        if (++b >= p.s.num_seqs) return false;
        h = 0, w = 0;
        s = seq_shape(p, b);
        u = units_of(p, s);
      }
    }
    const int per = p.unit_rows / p.group;
    g->b = b;
    g->h = h;
    g->w = w;
    g->s = s;
    g->i0 = w * per;
    g->i1 = min(s.n, (w + 1) * per);
    g->t0 = t.first + static_cast<int>(at);
    g->t1 = static_cast<int>(min(static_cast<int64_t>(t.last), g->t0 + left));
    g->starts = at == 0;
    g->ends = g->t1 == t.last;
    left -= g->t1 - g->t0;
    at = 0;
    ++w;
    return true;
  }
};

// Slot of a segment that is not a whole unit: the run's first segment when it
// continues a unit, its last one when it begins a unit.
__device__ __forceinline__ float* part_slot(const AttnArgs& p, int run, bool starts) {
  const int64_t slot = 2ll * run + (starts ? 1 : 0);
  return p.part + slot * p.unit_rows * (p.g.head_dim + 1);
}
__device__ __forceinline__ int2* join_of(const AttnArgs& p, int b, int h, int w) {
  return p.joins + (static_cast<int64_t>(b) * p.g.kv_heads + h) * p.units_per_pair + w;
}

// Sets a kernel's dynamic shared memory limit once per device.
struct SmemOnce {
  std::atomic<uint64_t> done{0};
  cudaError_t set(const void* fn, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
  }
};

// No grid has more runs than this, so the workspace has one size on every device.
constexpr int kMaxRuns = 320;

// Launchers (the result is cudaGetLastError's).
cudaError_t launch_kv_decode(const AttnArgs& a, int dtype, const CUtensorMap& tm, cudaStream_t s);
cudaError_t launch_kv_join(const AttnArgs& a, int dtype, cudaStream_t s);
// Rows of a unit of the decode kernel: 8 or 16.
constexpr int kDecodeMaxRows = 16;
int kv_decode_runs(int sms, int head_dim);

}  // namespace rimuru
