// Host check of how attention's work is cut (run by test_kv_split.py, without a device): the tiles of
// a (sequence, head) in closed form against a count over its units and rows, in 64 bits.
#include <cstdio>
#include <cstdlib>
#include <limits>

#include "../paged_moe_shared_gb300/csrc/kv_attn.h"

using namespace rimuru;

static int64_t tiles_of(int64_t len, int64_t n, int64_t window, int64_t q, int64_t w) {
  const int64_t i0 = w * q, i1 = i0 + q < n ? i0 + q : n;
  const int64_t p0 = len - n + i0, p1 = len - n + i1;  // positions p0 .. p1 - 1
  if (p1 <= 0) return 0;
  const int64_t first = window > 0 && p0 - window + 1 > 0 ? p0 - window + 1 : 0;
  return (p1 - 1) / kTileTokens - first / kTileTokens + 1;
}

int main() {
  const int big = std::numeric_limits<int>::max();
  const int lens[] = {0, 1, 2, 127, 128, 129, 500, 1000, 5000, 1 << 24, (1 << 30) - 1, 1 << 30};
  const int rows[] = {1, 2, 16, 100, 129, 700, 5000};
  const int windows[] = {0, 1, 2, 100, 128, 129, 1000, 5000, 1 << 24, (1 << 30) - 1, 1 << 30, big - 1, big};
  const int units[] = {1, 2, 5, 16, 18, 32, 128, 256};
  long bad = 0, seen = 0;
  for (int len : lens)
    for (int n : rows)
      for (int window : windows)
        for (int q : units) {
          int32_t cu[2] = {0, n}, l = len;
          AttnArgs p{};
          p.window = window;
          p.max_q = n;
          p.s.cu = cu;
          p.s.lens = &l;
          p.s.table_stride = int64_t{1} << 31;
          p.s.num_seqs = 1;
          p.s.rows = n;
          p.s.max_len = 1 << 30;
          p.g.page_tokens = 16;
          p.unit_q = q;
          p.units_per_pair = (n + q - 1) / q;
          const SeqShape s = seq_shape(p, 0);
          if (!s.ok) { printf("len %d rows %d refused\n", len, n); ++bad; continue; }
          int64_t sum = 0;
          bool ok = units_of(p, s) == p.units_per_pair;
          for (int w = 0; w < p.units_per_pair; ++w) {
            if (w <= 40 || w > p.units_per_pair - 40) ok &= w == 0 || tiles_before(p, s, w) == sum;
            const int64_t t = tiles_of(len, n, window, q, w);
            const TileSpan span = unit_span(p, s, w);
            ok &= (span.last > span.first ? span.last - span.first : 0) == t;
            sum += t;
          }
          ++seen;
          if (sum < 2000000000) ok &= pair_tiles(p, s) == sum;
          else continue;  // refused on the host
          if (!ok && ++bad < 20)
            printf("len %d rows %d window %d unit %d: %d tiles, counted %lld\n", len, n, window, q, pair_tiles(p, s),
                   static_cast<long long>(sum));
        }
  printf("%ld combinations, %ld wrong\n", seen, bad);
  return bad != 0;
}
