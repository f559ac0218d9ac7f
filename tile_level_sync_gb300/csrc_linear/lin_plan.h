// Which kernel computes a product of a linear layer, and in which tiles: plain arithmetic on the host, from
// estimated times.
#pragma once
#include <algorithm>
#include <cstddef>
#include <cstdint>

#include "../csrc/geometry.h"

namespace cusync {
namespace lin {

// A product's kind: forward, the two gradients on clusters, both of them on pairs.
enum : int { FWD = 0, DX = 1, DW = 2, GRAD = 3 };

constexpr int kSmemPerSm = 227 * 1024;

// Products on clusters: most stages of the ring; a stage holds two blocks of 128 bytes of the reduction.
constexpr int kMaxStages = 8;
CUSYNC_HD constexpr int split_stage_bytes(int cols) { return 2 * (128 + cols) * 128; }
constexpr size_t split_smem(int cols, int stages, bool apart) {
  const size_t ring = (size_t)stages * split_stage_bytes(cols), sums = (size_t)cols * 128 * 4;
  return 1024 + (apart ? ring + sums : ring > sums ? ring : sums);
}

inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// How products are computed: on CTA pairs with tiles of 256 x `bn` (SwiGLU: bn / 2 columns of Y), or (bn = 0) on
// clusters of `splits` CTAs with tiles of 128 (64) columns x `cols` rows; and about how long it takes.  The
// times are fits to passes on one GB300 (us; bf16, no activation, weights in the L2 where they fit it):
//   rows x cols   reduction   pairs 256   pairs 128   clusters (cols, splits)
//   1777 x 1024        2048        13.7        10.5        14.6 (128, 1)  21.6 (64, 2)
//   4096 x 2048        4096        43.3        51.9        89.4 (128, 1)
//    333 x  776         512         7.5         5.6         5.7 (64, 2)    7.0 (128, 4)
//    333 x  776        4096        22.2        13.6        11.9 (64, 2)   11.1 (128, 4)
//    100 x 4096        2048        13.2         8.7         9.0 (64, 2)    9.3 (128, 4)
//    100 x 4096        4096        22.6        15.0        16.5 (64, 2)   12.7 (128, 4)
//     16 x 4096        4096        21.7        14.1        11.0 (16, 2)    8.7 (16, 4)
struct Plan {
  double us;
  int bn, cols, splits, stages;
  bool apart;  // clusters: room of their own for the sums
};
constexpr double kBytesPerUs = 6.5e6;  // of HBM

// A tile of 256 x bn with `blocks` blocks of 128 bytes of the reduction, on a pair.
inline double pair_tile(int bn, int64_t blocks) { return 0.5 + (bn == 256 ? 0.30 : 0.19) * (double)blocks; }
// n tiles that take a each, then m that take b, dealt out to `pairs` pairs in turn: the pair that ends last is
// the first one, or the first one with a tile less of the first kind.
inline double pair_time(int64_t n, double a, int64_t m, double b, int64_t pairs) {
  const int64_t rest = n % pairs;
  const double first = (double)div_up(n, pairs) * a + (double)(div_up(n + m, pairs) - div_up(n, pairs)) * b;
  const double other = (double)(n / pairs) * a + (double)(div_up(n + m - rest, pairs) - n / pairs) * b;
  return 4.2 + (rest ? std::max(first, other) : first);
}

inline Plan pair_plan(int64_t rows, int64_t cols, int64_t depth, int sms, int elems, bool gated) {
  Plan best = {1e30, 0, 0, 0, 0, false};
  if (sms < 2) return best;
  for (int bn = 128; bn <= 256; bn += 128) {
    const int64_t tiles = div_up(rows, 256) * div_up(cols, gated ? bn / 2 : bn);
    const double us = pair_time(tiles, pair_tile(bn, div_up(depth, elems)), 0, 0.0, sms / 2);
    if (us < best.us) best = {us, bn, 0, 0, 0, false};
  }
  return best;
}

template <int MODE, bool GATED>
Plan split_plan(int64_t rows, int64_t cols, int64_t depth, int sms, int elems) {
  Plan best = {1e30, 0, 0, 0, 0, false};
  int most = 16;  // rows of a tile that covers all rows, where one does
  while (most < 128 && most < rows) most *= 2;
  const int64_t blocks = div_up(depth, elems);
  for (int n = MODE == DW ? 64 : std::max(16, most / 2); n <= std::max(most, MODE == DW ? 64 : 16); n *= 2) {
    const int stage = split_stage_bytes(n);
    const int64_t tiles = div_up(rows, n) * div_up(cols, GATED ? 64 : 128);
    for (int splits = 1; splits <= 8; splits *= 2) {
      if (splits > 1 && splits > div_up(blocks, 2)) break;
      const int64_t ctas = tiles * splits;
      // two CTAs an SM where there are enough and two stages of both fit; clusters of four or eight leave some
      // SMs out (of 152: 144 and 120 take one CTA, 296 and 288 CTAs fit two an SM)
      const int64_t alone = std::max(1, splits == 8 ? sms * 15 / 19 : splits == 4 ? sms * 18 / 19 : sms);
      const int64_t both = std::max(1, splits == 8 ? sms * 36 / 19 : splits == 4 ? sms * 37 / 19 : 2 * sms);
      const bool two = ctas > alone && 2 * (2 * stage + 2048) <= kSmemPerSm;
      // an SM's CTAs share what it can load: 0.2 us a block (0.26 with 128 rows), one CTA or two
      const double stream = (double)(div_up(ctas, sms) * div_up(blocks, splits)) * (n <= 64 ? 0.2 : 0.26);
      // weights come at HBM's rate, a little less where SMs are left out
      const double weights = (double)(cols * (GATED ? 2 : 1) * depth) * (64.0 / elems) * 2.0 / kBytesPerUs /
                             std::min(1.0, 0.9 + 0.1 * (double)ctas / sms);
      const double us = 5.2 + 0.012 * n + 0.15 * (splits - 1) + 2.0 * (double)(div_up(ctas, two ? both : alone) - 1) +
                        std::max(stream, MODE == DW ? 0.0 : weights);
      if (us < best.us) {
        const int room = (two ? kSmemPerSm / 2 : kSmemPerSm) - 1024;  // static shared memory and the block's own
        best = {us, 0, n, splits, 0, false};
        best.stages = (int)std::min<int64_t>(std::min(kMaxStages, (room - 1024) / stage), div_up(div_up(blocks, 2), splits));
        best.apart = splits > 1 && split_smem(n, best.stages, true) <= (size_t)room;
      }
    }
  }
  return best;
}

}  // namespace lin
}  // namespace cusync
