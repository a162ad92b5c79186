// How the row tiles of a product grouped by expert go to the XCDs.  Host code.
#ifndef MRS_PRODUCT_RUNS_H_
#define MRS_PRODUCT_RUNS_H_

#include <stdint.h>

constexpr int kXcds = 8;

// Row tiles with a route on each XCD, for runs of 1 << run tiles dealt out in turn, where the
// first `live` of every `stride` tiles hold routes, for each of `experts` (the pattern of 64
// comes again).
struct XcdTiles {
  int64_t of[kXcds] = {};
  XcdTiles(int64_t experts, int64_t stride, int64_t live, int run) {
    for (int64_t e = 0; e < experts && e < 64; ++e) {
      const int64_t end = e * stride + live;
      for (int64_t t = e * stride; t < end;) {
        const int64_t next = ((t >> run) + 1) << run, upto = next < end ? next : end;
        of[(t >> run) % kXcds] += upto - t;
        t = upto;
      }
    }
  }
  int reached() const {
    int n = 0;
    for (int64_t t : of) n += t > 0;
    return n;
  }
  int64_t busiest() const {
    int64_t most = 0;
    for (int64_t t : of) most = t > most ? t : most;
    return most;
  }
};

// Tiles of bm rows: `live` of an expert with `average` routes, and all of its blocks.
inline int64_t live_tiles(int64_t average, int bm) { return (average + bm - 1) / bm; }
inline int64_t block_tiles(int64_t average, int bm, int block) { return (average + block - 1) / block * (block / bm); }

// The row tiles of a run, as a power of two: those that share an expert's weights, up to four
// (twice the average, for experts are uneven), or the tiles of a block, of which the first ones
// hold the routes.  Runs of 1, 2 and 4 (us): 64 tokens of 896 experts, top-16, K 3584, N 768,
// blocks of 16 441, 441, 457; 512 tokens of 64, top-8, blocks of 128 71, 71, 99; 2048 tokens of
// them, blocks of 64 227, 191, 180; 777 of 24, top-6, K 1000, N 397 18.7, 17.5, 17.1; runs of 1,
// 2, 4, 8, 16, 32: 8192 tokens of 896, top-16, blocks of 128 1333, 1285, 1261, 1272, 1285, 1258.
//
// Where that leaves an XCD without a tile: the run whose busiest XCD has the fewest, the nearest
// of them, if it is at most half as many.  us, kForward / kRows, so and without: 512 tokens of one
// expert, K 2048, N 2048 14.9 / 18.5 and 28.9 / 26.2; 400 of 8, top-2, K 2048, N 1280 16.2 / 21.6
// and 31.4 / 21.6; 256 of 8 in blocks of 1024, K 1024, N 768 9.1 / 9.7 and 24.2 / 18.2; 64 of 64,
// one row each, in blocks of 4096, K 40, N 2048 108 / 25 and 109 / 46.  By less than half it
// costs more than it gives, since XCDs that share an expert read its weights each: 512 of 5,
// top-2, K 2048, N 1024 19.6 / 18.5 by runs of 1 (busiest XCD 3), 14.8 / 14.0 by runs of 4 (4).
inline int run_of(int64_t experts, int64_t average, int bm, int block) {
  const int64_t live = live_tiles(average, bm), stride = block_tiles(average, bm, block), of_block = block / bm;
  int64_t want = live_tiles(2 * average, bm);
  want = want > 4 ? 4 : want;
  const int64_t padded = of_block < experts * live / 4 ? of_block : experts * live / 4;
  if (padded > want) want = padded > 8 ? 8 : padded;
  int log2 = 0;
  while (1 << log2 < want) ++log2;
  // an expert's tiles, or those of many without a run between them, reach every XCD
  if (live >= kXcds << log2 || (experts * live >= kXcds << 7 && of_block <= want)) return log2;
  const XcdTiles first(experts, stride, live, log2);
  if (first.reached() == kXcds) return log2;
  int best = log2;
  int64_t least = first.busiest() / 2 + 1;
  const auto consider = [&](int run) {
    const int64_t most = XcdTiles(experts, stride, live, run).busiest();
    if (most < least) best = run, least = most;
  };
  for (int run = log2 - 1; run >= 0; --run) consider(run);
  for (int run = log2 + 1; run < 24 && int64_t(1) << (run - 1) < of_block; ++run) consider(run);
  return best;
}

// Whether an XCD's tiles of `columns` column tiles each run at once, two to each of its 32 compute
// units, where experts get a sixteenth more than the average (they are uneven): a third one to a
// unit has to wait for one of the first to end.
inline bool at_once(int64_t experts, int64_t average, int bm, int block, int64_t columns) {
  const int64_t most = average + average / 16;
  const XcdTiles x(experts, block_tiles(most, bm, block), live_tiles(most, bm), run_of(experts, most, bm, block));
  return x.busiest() * columns <= 64;
}

#endif  // MRS_PRODUCT_RUNS_H_
