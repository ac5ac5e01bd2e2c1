// Shared by the attention kernels: arguments, how the work is cut, and the
// layout of the partial results that are joined afterwards.
//
// A unit is a (sequence, key/value head, block of query rows); its work is the
// 128-token tiles of keys that any of its rows sees, and before them `unit_cost`
// places for what it costs to begin and end one.  The places of all units, laid
// end to end, are cut into equal runs, one per CTA, so the CTAs finish together
// whatever the lengths are, and no length has to be known on the host (with tiles
// alone, the CTAs that had many short units were the last ones).  A unit that lies within one run is finished there; the others leave
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
  int sms;             // of the device
  int runs;            // CTAs that share the tiles
  int unit_rows;       // query rows (query x group) of a unit
  int unit_q;          // whole query rows of a unit: unit_rows / group
  int units_per_pair;  // bound of the units of one (sequence, head)
  int unit_cost;       // places of a unit before its tiles
  bool direct;         // a CTA per unit, none is cut and nothing joined
  int4* cuts;          // [runs] the unit that begins in a run and ends in a later one: first
                       // query row, head * 512 + rows, unit, last run; 0 rows: there is none
  float* part;         // [2 runs][unit_rows][head_dim] partial results, then
  float* stat;         // [2 runs][unit_rows] their log2 sums
};

constexpr float kLn2 = 0.69314718055994531f;

// One sequence: its query rows and cached length.  ok == false: the arguments
// disagree and the sequence has no work (its rows become zero).
struct SeqShape {
  int row0, n, len;
  bool ok;
};
__host__ __device__ __forceinline__ SeqShape seq_shape(const AttnArgs& p, int b) {
  SeqShape s;
  s.row0 = p.s.cu ? p.s.cu[b] : b;
  s.n = p.s.cu ? p.s.cu[b + 1] - s.row0 : 1;
  s.len = p.s.lens[b];
  s.ok = s.n >= 0 && s.n <= p.max_q && s.row0 >= 0 && s.row0 <= p.s.rows - s.n && s.len >= 0 &&
         s.len <= p.s.max_len;
  if (!s.ok || s.n == 0) s.n = 0, s.len = 0;
  return s;
}
// Tiles [first, last) that the query rows i0 .. i1 - 1 of a sequence see.
struct TileSpan {
  int first, last;
};
__host__ __device__ __forceinline__ TileSpan tile_span(const AttnArgs& p, const SeqShape& s, int i0, int i1) {
  const int p0 = s.len - s.n + i0, p1 = s.len - s.n + i1;  // positions p0 .. p1 - 1
  TileSpan t;
  t.last = p1 > 0 ? (p1 + kTileTokens - 1) / kTileTokens : 0;
  t.first = p.window > 0 && p0 >= p.window ? (p0 - p.window + 1) / kTileTokens : 0;
  return t;
}
// A unit holds the query rows [w unit_q, (w + 1) unit_q) of its sequence.
__host__ __device__ __forceinline__ int units_of(const AttnArgs& p, const SeqShape& s) {
  return p.units_per_pair == 1 ? (s.n > 0) : (s.n + p.unit_q - 1) / p.unit_q;
}
__host__ __device__ __forceinline__ TileSpan unit_span(const AttnArgs& p, const SeqShape& s, int w) {
  return tile_span(p, s, w * p.unit_q, min(s.n, (w + 1) * p.unit_q));
}
// Sum of floor((a i + b) / 128) over 0 <= i < n; a > 0, b >= 0.  Whole parts of
// a / m and b / m are taken out, and what is left counts lattice points under a
// line, which are counted along the other axis with smaller numbers.
__host__ __device__ __forceinline__ int floor_sum(uint32_t n, uint32_t a, uint32_t b) {
  uint32_t sum = 0, m = kTileTokens;  // a count of tiles: fits an int (checked on the host)
  while (n > 0) {
    const uint32_t qa = a / m, qb = b / m;
    sum += static_cast<uint32_t>(static_cast<uint64_t>(n) * (n - 1) / 2) * qa + n * qb;
    a -= qa * m;
    b -= qb * m;
    const uint32_t top = a * n + b;
    if (top < m) break;
    n = top / m;
    b = top - n * m;
    const uint32_t x = m;
    m = a;
    a = x;
  }
  return static_cast<int>(sum);
}
// Tiles of the first w units of one head of a sequence (all of them full units).
__host__ __device__ __forceinline__ int tiles_before(const AttnArgs& p, const SeqShape& s, int w) {
  const int q = p.unit_q, base = s.len - s.n;  // unit v: positions base + v q .. base + (v + 1) q - 1
  const int v0 = base + q > 0 ? 0 : -base / q;   // units before end at or below position 0
  int n = 0;
  if (w > v0) n = floor_sum(w - v0, q, base + (v0 + 1) * q + kTileTokens - 1);
  if (p.window > 0) {
    // first position minus `out` leaves the window's reach.  Unsigned: with a large window, or rows
    // before position 0, it passes 2^31.
    const uint32_t out = p.window - 1 > base ? static_cast<uint32_t>(p.window - 1) - static_cast<uint32_t>(base) : 0u;
    const uint32_t v1 = out / q + (out % q != 0);
    if (static_cast<uint32_t>(w) > v1)
      n -= floor_sum(w - v1, q, static_cast<uint32_t>(base) + v1 * q - static_cast<uint32_t>(p.window) + 1u);
  }
  return n;
}
// Tiles of one head of a sequence, over all its units.
__host__ __device__ __forceinline__ int pair_tiles(const AttnArgs& p, const SeqShape& s) {
  const int u = units_of(p, s);
  if (u == 0) return 0;
  const TileSpan t = unit_span(p, s, u - 1);
  return (u > 1 ? tiles_before(p, s, u - 1) : 0) + t.last - t.first;
}

// All places are cut into `runs` runs of base or base + 1 places, the longer first.
struct RunCut {
  int base, longer, runs;
};
__device__ __forceinline__ int run_start(const RunCut& k, int c) { return c * k.base + min(c, k.longer); }
__device__ __forceinline__ int run_of(const RunCut& k, int place) {
  const int head = k.longer * (k.base + 1);
  return place < head ? place / (k.base + 1) : k.longer + (place - head) / k.base;
}

// One run: where its first tile lies, and its tiles.
struct RunStart {
  RunCut cut;
  int before[2];      // tiles before the run's first and after its last place
  int place;          // of its first tile
  int b, h, w, at;    // sequence, head, unit, and the tile within the unit
  SeqShape s;
  struct {            // an end of the run within its (sequence, head): places from there, tiles before
    int at, before;
    SeqShape s;
  } end[2];
  __device__ __forceinline__ int tiles() const { return before[1] - before[0]; }
};

// Found by the whole CTA (every thread calls it; `scratch` has a number per
// warp): thread t sums the tiles and units of a contiguous share of the
// sequences, the shares are scanned, and the thread whose share holds an end of
// the run walks its share.  Totals fit an int (checked on the host).
__device__ __forceinline__ void find_run(const AttnArgs& p, int c, uint64_t* scratch, RunStart* out) {
  const int t = threadIdx.x, nt = blockDim.x, lane = t & 31, warp = t >> 5, cost = p.unit_cost;
  const int share = p.s.num_seqs <= nt ? 1 : (p.s.num_seqs + nt - 1) / nt;
  const int b0 = min(p.s.num_seqs, t * share), b1 = min(p.s.num_seqs, b0 + share);
  uint64_t mine = 0;  // tiles, and units in the upper half
  SeqShape s0{};
  int n0 = 0;
  for (int b = b0; b < b1; ++b) {
    const SeqShape s = seq_shape(p, b);
    if (!s.ok && c == 0) dev::set_error(p.g.err, RIMURU_DEV_BAD_SHAPE);
    const int n = pair_tiles(p, s);
    if (b == b0) s0 = s, n0 = n;
    mine += (static_cast<uint64_t>(units_of(p, s)) << 32 | static_cast<uint32_t>(n)) * p.g.kv_heads;
  }
  uint64_t scan = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t v = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += v;
  }
  if (lane == 31) scratch[warp] = scan;
  __syncthreads();
  uint64_t before = scan - mine, total = 0;
  for (int w = 0; w < nt / 32; ++w) {
    if (w < warp) before += scratch[w];
    total += scratch[w];
  }
  const auto tiles_in = [](uint64_t x) { return static_cast<int>(static_cast<uint32_t>(x)); };
  const auto places_in = [&](uint64_t x) { return tiles_in(x) + static_cast<int>(x >> 32) * cost; };
  // Runs may hold no tile; but those from the first to the last tile of a unit all hold some of
  // it, so every one of them leaves a part.
  const int places = places_in(total), first = places_in(before), own = places_in(mine);
  RunCut k;
  k.runs = min(places, p.runs);
  k.base = k.runs > 0 ? places / k.runs : 0;
  k.longer = places - k.base * k.runs;
  const int ends[2] = {c < k.runs ? run_start(k, c) : places, c < k.runs ? run_start(k, c + 1) : places};
  if (t == 0) {
    out->cut = k;
    for (int e = 0; e < 2; ++e)
      if (ends[e] == places) out->before[e] = tiles_in(total);
  }
#pragma unroll 1
  for (int e = 0; e < 2; ++e) {
    if (ends[e] < first || ends[e] >= first + own) continue;
    int at = ends[e] - first, b = b0, n = n0, sum = tiles_in(before);
    SeqShape s = s0;
    int each = n + units_of(p, s) * cost;
    while (at >= each * p.g.kv_heads) {
      at -= each * p.g.kv_heads;
      sum += n * p.g.kv_heads;
      s = seq_shape(p, ++b);
      n = pair_tiles(p, s);
      each = n + units_of(p, s) * cost;
    }
    int h = 0;
    while (at >= each) at -= each, sum += n, ++h;
    if (p.units_per_pair == 1) {
      const int tile = max(0, at - cost);
      out->before[e] = sum + tile;
      if (e == 0) out->w = 0, out->at = tile, out->place = ends[0] - at + max(at, cost);
    } else {
      out->end[e].at = at;
      out->end[e].before = sum;
      out->end[e].s = s;
    }
    if (e == 0) {
      out->b = b;
      out->h = h;
      out->s = s;
    }
  }
  __syncthreads();
  if (p.units_per_pair == 1) return;
  // the unit: the last one with at most `at` places before it, one thread per group of units;
  // half of the CTA looks for either end
  const int half = nt / 64 * 32, e = t >= half, te = e ? t - half : t, ne = e ? nt - half : half;
  if (ends[e] < places) {
    const SeqShape s = out->end[e].s;
    const int at = out->end[e].at, u = units_of(p, s), per = (u + ne - 1) / ne;
    const int w0 = min(u, te * per), w1 = min(u, w0 + per);
    const auto places_before = [&](int w) { return tiles_before(p, s, w) + w * cost; };
    int n = places_before(w0);
    const int after = w1 < u ? places_before(w1) : at + 1;
    if (w0 < w1 && n <= at && at < after) {
      int w = w0;
      for (; w + 1 < w1; ++w) {
        const TileSpan x = unit_span(p, s, w);
        if (n + cost + max(0, x.last - x.first) > at) break;
        n += cost + max(0, x.last - x.first);
      }
      const int y = at - n, tile = max(0, y - cost);
      out->before[e] = out->end[e].before + n - w * cost + tile;
      if (e == 0) out->w = w, out->at = tile, out->place = ends[0] - y + max(y, cost);
    }
  }
  __syncthreads();
}

// First row and number of the query rows of a unit that has no tile: they become
// zero.  Where the arguments disagree, what of its rows lies inside the arrays.
struct RowSpan {
  int row0, n;
};
__device__ __forceinline__ RowSpan empty_rows(const AttnArgs& p, const SeqShape& s, int b, int w) {
  int n = s.n;
  if (!s.ok) {
    n = p.s.cu ? p.s.cu[b + 1] - s.row0 : 1;
    n = s.row0 < 0 ? 0 : min(min(n, p.max_q), p.s.rows - s.row0);
  }
  const int i0 = w * p.unit_q;
  // one unit a pair holds all of its rows, be they more than a unit's (arguments that disagree)
  n = p.units_per_pair == 1 ? n : min(n - i0, p.unit_q);
  if (n > 0 && s.ok) {
    const TileSpan t = unit_span(p, s, w);
    if (t.first < t.last) n = 0;
  }
  return {s.row0 + i0, n};
}

// The same for a CTA that has one unit, `u` in the order of the cuts; it also
// writes the zeros of a unit without tiles.  T: type of the results.
template <typename T>
__device__ __forceinline__ void find_unit(const AttnArgs& p, int u, RunStart* out) {
  const int w = u % p.units_per_pair, pair = u / p.units_per_pair, b = pair / p.g.kv_heads;
  const int h = pair - b * p.g.kv_heads;
  const SeqShape s = seq_shape(p, b);  // every thread: one broadcast load each
  const bool has = w < units_of(p, s);
  const TileSpan t = has ? unit_span(p, s, w) : TileSpan{0, 0};
  if (threadIdx.x == 0) {
    if (!s.ok) dev::set_error(p.g.err, RIMURU_DEV_BAD_SHAPE);
    out->before[0] = 0;
    out->before[1] = max(0, t.last - t.first);
    out->place = out->at = 0;
    out->b = b;
    out->h = h;
    out->w = w;
    out->s = s;
  }
  const RowSpan r = empty_rows(p, s, b, w);
  const int per = p.g.head_dim / 8;  // 16 bytes a thread
  for (int i = threadIdx.x; i < r.n * p.group * per; i += blockDim.x) {
    const int row = i / per, q = row / p.group;
    const int64_t to = r.row0 + q, head = h * p.group + row - q * p.group;
    *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + to * p.o_ts + head * p.o_hs + (i - row * per) * 8) =
        make_uint4(0, 0, 0, 0);
    if (p.lse && i == row * per) p.lse[to * p.q_heads + head] = -INFINITY;
  }
}

// Walks a run segment by segment: the part of a unit that lies in the run.
struct Segment {
  int b, h, w;        // sequence, head, unit
  SeqShape s;
  int i0, i1;         // query rows of the unit
  int t0, t1;         // its tiles within this run
  int place;          // of the first of them
  int unit_tiles;     // tiles of the whole unit
  bool starts, ends;  // holds the unit's first / last tile
};
struct RunWalk {
  int left, at, place;  // tiles of the run still to come; the next one's within its unit, and its place
  int b, h, w, u;  // next unit; u: units of sequence b
  SeqShape s;
  __device__ __forceinline__ void begin_run(const AttnArgs& p, const RunStart& r) {
    left = r.tiles();
    if (left <= 0) return;
    place = r.place;
    b = r.b;
    h = r.h;
    w = r.w;
    at = r.at;
    s = r.s;
    u = units_of(p, s);
  }
  __device__ __forceinline__ bool next(const AttnArgs& p, Segment* g) {
    if (left <= 0) return false;
    TileSpan t;
    while (true) {
      if (w < u) {
        t = unit_span(p, s, w);
        if (t.last > t.first) break;
        ++w;
        place += p.unit_cost;
      } else if (h + 1 < p.g.kv_heads && u > 0) {
        ++h, w = 0;
      } else {
        if (++b >= p.s.num_seqs) return false;
        h = 0, w = 0;
        s = seq_shape(p, b);
        u = units_of(p, s);
      }
    }
    g->b = b;
    g->h = h;
    g->w = w;
    g->s = s;
    g->i0 = w * p.unit_q;
    g->i1 = min(s.n, g->i0 + p.unit_q);
    g->t0 = t.first + at;
    g->t1 = min(t.last, g->t0 + left);
    g->place = place;
    g->unit_tiles = t.last - t.first;
    g->starts = at == 0;
    g->ends = g->t1 == t.last;
    left -= g->t1 - g->t0;
    place += g->t1 - g->t0 + p.unit_cost;
    at = 0;
    ++w;
    return true;
  }
};

// Slot of a segment that is not a whole unit: the run's first segment when it
// continues a unit, its last one when it begins a unit.
__device__ __forceinline__ int64_t part_slot(const AttnArgs& p, int run, bool starts) {
  return static_cast<int64_t>(2 * run + (starts ? 1 : 0)) * p.unit_rows;
}
// Notes the unit that a run's last segment begins and does not end (a run cuts
// no other one); called for every segment, over the zeros that the CTA begins with.
__device__ __forceinline__ void note_cut(const AttnArgs& p, const Segment& g, const RunCut& k, int run) {
  if (g.starts && !g.ends)
    p.cuts[run] = make_int4(g.s.row0 + g.i0, g.h * 512 + (g.i1 - g.i0) * p.group,
                            (g.b * p.g.kv_heads + g.h) * p.units_per_pair + g.w,
                            run_of(k, g.place + g.unit_tiles - 1));
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
constexpr int kMaxRuns = 320;      // decode kernel: up to two CTAs per SM
constexpr int kMaxTileRuns = 160;  // tile kernel: one

// What it costs to begin and end a unit, in tiles.  Decode, 64 sequences of 1 to 4014 keys: 23.3 us
// the call at 0, 16.9 at 2, 17.3 at 3, 17.7 at 4, 19.0 at 6.  Tiles, six prompts of 209 to 855
// tokens at head_dim 256: 110 us at 0, 66.0 at 3, 63.2 at 4, 66.4 at 5, 70.5 at 8; 16 sequences of
// 3 to 5 rows: 36.0, 30.6, 29.4, 29.5, 30.7.
constexpr int kDecodeUnitCost = 2, kTileUnitCost = 4;

// What cutting costs, in tiles: the second kernel, the parts and the search for the run.  Where the
// longest unit has at most as many tiles as that and a run of half-full units together, and all
// units run at the same time, they are better left whole.  Cut and whole, us: one sequence, 8 rows
// a head, of 500 keys 9.8 and 8.4, of 2000 keys 10.4 and 20.1; 64 of 1000 keys 19.3 and 14.3; eight,
// 40 rows, of 500 keys 15.7 and 11.4, of 2000 19.5 and 25.0; the last 256 of 1000 tokens, 32/4 heads,
// 36.2 and 23.5.
inline bool leave_whole(int64_t units, int64_t most, int runs, int unit_cost, int unit_rows, int head_dim) {
  const int cut = unit_rows == 256 ? 10 : unit_rows <= 16 && head_dim == 256 ? 4 : 6;
  return units <= runs && 2 * most * runs <= 2 * cut * runs + units * (most + 2 * unit_cost);
}

// Launchers (the result is cudaGetLastError's).
cudaError_t launch_kv_decode(const AttnArgs& a, int dtype, const CUtensorMap& tm, cudaStream_t s);
cudaError_t launch_kv_tiles(const AttnArgs& a, int dtype, const CUtensorMap& tm, const CUtensorMap& tm_v,
                            cudaStream_t s);
cudaError_t launch_kv_join(const AttnArgs& a, int dtype, cudaStream_t s);
// Rows of a unit of the decode kernel: 8 or 16.
constexpr int kDecodeMaxRows = 16;
// Most rows of a unit of the tile kernel (two query tiles of 128; one at head_dim 256).
constexpr int tile_rows(int head_dim) { return head_dim <= 128 ? 256 : 128; }
int kv_decode_runs(int sms, int head_dim, int rows);

}  // namespace rimuru
