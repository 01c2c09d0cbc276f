// How int8 products and gradients are done, by their sizes: which kernel, which tile,
// how many workgroups share K. Host rules alone, in plain C++, so that a test can ask
// them without a GPU.
#pragma once

#include <stdint.h>

#include <algorithm>
#include <cmath>

namespace aqlm {

// A tile kernel's workgroup: RW x TW wavefronts of RT x NT 32 x 32 tiles, KW such sets that
// share K, STAGES steps of K in LDS.
template <int RT_, int NT_, int RW_, int TW_, int KW_, int STAGES_> struct I8Shape {
  static constexpr int RT = RT_, NT = NT_, RW = RW_, TW = TW_, KW = KW_, STAGES = STAGES_;
  static constexpr int kWaves = RW * TW, kThreads = 64 * kWaves;  // of one share of K
  static constexpr int kAcross = 32 * RT * RW, kToks = 32 * NT * TW;
  static constexpr int kSums = kAcross * kToks * 4;
};

constexpr int kLdsBytes = 160 * 1024;  // of a CU
constexpr int kCus = 256;

// Of a product (i8_tile.hip): a step is 128 inputs, a byte each on both sides.
template <int RT, int NT, int RW, int TW, int KW, int STAGES>
struct I8TileShape : I8Shape<RT, NT, RW, TW, KW, STAGES> {
  using Base = I8Shape<RT, NT, RW, TW, KW, STAGES>;
  static constexpr int kRows = Base::kAcross;  // GATED: half of them the gate's, half up's
  static constexpr int kWBytes = kRows * 128, kStage = kWBytes + Base::kToks * 128;
  static constexpr int kSlots = kCus * (kLdsBytes / (STAGES * KW * kStage));  // workgroups the chip holds
};

// Of a gradient (i8_grad.hip): a step is 64 rows of W, a byte each, and 64 terms of two
// halves.
template <int RT, int NT, int RW, int TW, int KW, int STAGES>
struct I8GradShape : I8Shape<RT, NT, RW, TW, KW, STAGES> {
  using Base = I8Shape<RT, NT, RW, TW, KW, STAGES>;
  static constexpr int kCols = Base::kAcross;
  static constexpr int kWBytes = 64 * kCols, kXBytes = Base::kToks * 128, kStage = kWBytes + 2 * kXBytes;
  // LDS bytes of a stage's array: the stage, the shares' sums in the first one, the
  // results in the second (and third: half of the wavefronts each)
  static constexpr int kStore = RT * 2048;  // a wavefront's results
  static constexpr int kArray =
      std::max({KW * kStage, KW > 1 ? Base::kSums : 0, Base::kWaves * kStore / (STAGES > 2 ? 2 : 1)});
  static constexpr int kSlots = kCus * (kLdsBytes / (STAGES * kArray));
};

// The choice of a tile kernel's call.
struct I8Plan {
  int shape, splits, steps_per_split;
  int64_t across, tok_tiles;  // tiles of W's rows (a gradient: of its columns), and of tokens
  int64_t sums;               // bytes of the split parts' sums in the workspace
  double us;                  // modelled duration
};

// Modelled durations. The grid runs in rounds of as many workgroups as the chip holds
// (`slots`); a round takes f us, and a + b * (its share of the slots) us for each step of a
// share of K, and c more where it fills more than half of them. That, the reading of W
// and the products at the rates of I8Rates are joined as a cube root of cubes; a split
// launches a second kernel and writes and reads its sums.
struct I8TileCost {
  int across, toks, kw, sums;  // sums: bytes of a workgroup's in the workspace
  int slots;
  double f, a, b, c;
};
struct I8Rates {
  double read, ops, sums;   // a us: bytes of W, operations where power holds the clock, bytes of sums
  double around, around_split;  // us beside them
  int split_grid;           // workgroups that a split grid has at most; 0: the shape's slots
};

template <class S> constexpr I8TileCost i8_cost_of(double f, double a, double b, double c = 0.0) {
  return {S::kAcross, S::kToks, S::KW, S::kSums, S::kSlots, f, a, b, c};
}

// The tile and split (into up to eight) of the shortest modelled time: `results` by
// `batch` results (`pair`: a tile's rows are two matrices'), `steps` of K, `bytes` of W.
template <int N>
I8Plan i8_choose(const I8TileCost (&costs)[N], const I8Rates &rates, int64_t results, bool pair, int64_t batch,
                 int steps, double bytes) {
  I8Plan best{};
  const double read = bytes / rates.read, power = 2.0 * bytes * (double)batch / rates.ops;
  const double bounds = read * read * read + power * power * power;
  for (int c = 0; c < N; ++c) {
    const I8TileCost &k = costs[c];
    I8Plan p{};
    p.shape = c;
    const int out = pair ? k.across / 2 : k.across;
    p.across = (results + out - 1) / out;
    p.tok_tiles = (batch + k.toks - 1) / k.toks;
    const int64_t tiles = p.across * p.tok_tiles;
    for (int s = 1; s <= 8; ++s) {
      p.steps_per_split = (steps + s - 1) / s;
      p.splits = (steps + p.steps_per_split - 1) / p.steps_per_split;
      if (p.splits != s || (s > 1 && tiles * s > (rates.split_grid ? rates.split_grid : k.slots))) break;
      const int64_t rounds = tiles * s < k.slots ? 0 : tiles * s / k.slots;  // (spares a division)
      const double whole = (double)rounds, rest = (double)(tiles * s - rounds * k.slots) / (double)k.slots;
      const double turns = (double)(k.kw == 1 ? p.steps_per_split : (p.steps_per_split + k.kw - 1) / k.kw);
      const double last = rest > 0 ? k.f + turns * (k.a + k.b * rest + (rest > 0.5 ? k.c : 0.0)) : 0.0;
      const double us = whole * (k.f + turns * (k.a + k.b + k.c)) + last;
      p.sums = s > 1 ? tiles * s * k.sums : 0;
      const double around = s > 1 ? rates.around_split + (double)p.sums * 2.0 / rates.sums : rates.around;
      if (best.splits != 0 && us + around >= best.us) continue;  // (spares the root)
      p.us = around + std::cbrt((float)(us * us * us + bounds));
      if (best.splits == 0 || p.us < best.us) best = p;
    }
  }
  return best;
}

// --- products ----------------------------------------------------------------
namespace i8_tile {
typedef I8TileShape<4, 2, 2, 4, 1, 2> Large;    // 256 rows x 256 tokens
typedef I8TileShape<2, 3, 4, 2, 1, 2> Wide;     // 256 x 192
typedef I8TileShape<2, 2, 4, 2, 1, 3> Middle;   // 256 x 128
typedef I8TileShape<2, 1, 4, 2, 1, 3> Half;     // 256 x 64
typedef I8TileShape<2, 2, 2, 1, 2, 3> Small;    // 128 x 64
typedef I8TileShape<2, 1, 2, 1, 2, 3> Slim;     // 128 x 32
typedef I8TileShape<2, 1, 1, 1, 2, 3> Least;    // 64 x 32, two workgroups to a CU

// Fitted to eight layers (1024 x 8192 to 22016 x 4096, 8192 x 28672) from 9 to 2048
// tokens, each shape and split measured at each, within 6 % at the median; the choice
// costs 2.5 % on average against the best one.
// (Each shape with its best splits, Large to Least: 64 x 8192 x 28672 60, 58, 49, 46,
// 47, 60 and 64 us, 301 x 11008 x 4096 43, 41, 31, 28, 40, 52, 51, 2048 x 4096 x 11008
// 116, 123, 91, 133, 195, 251, 245, 16 x 4096 x 4096 14, 13, 11, 10.5, 12, 9.7, 8.9.)
constexpr I8TileCost kCosts[] = {i8_cost_of<Large>(2.52, 1.276, 0.0),    i8_cost_of<Wide>(2.0, 1.171, 0.0),
                                 i8_cost_of<Middle>(2.41, 0.708, 0.151), i8_cost_of<Half>(2.14, 0.612, 0.09),
                                 i8_cost_of<Small>(3.2, 0.823, 0.171),   i8_cost_of<Slim>(2.22, 0.583, 0.093),
                                 i8_cost_of<Least>(2.05, 0.349, 0.366)};
constexpr I8Rates kRates = {5.3e6, 2.2e9, 5.9e6, 2.3, 4.0, 0};
}  // namespace i8_tile

inline I8Plan i8_tile_plan(int64_t rows, int64_t cols, bool gated, int64_t batch) {
  return i8_choose(i8_tile::kCosts, i8_tile::kRates, rows, gated, batch, (int)((cols + 127) / 128),
                   (double)rows * (gated ? 2 : 1) * (double)cols);
}

// Up to kI8RowTokens tokens of a gated block, and four of a layer, may go by whole rows of W
// (i8_rows.hip).
constexpr int kI8RowTokens = 8;
constexpr int kI8RowThreads = 512;

// Where whole-row wavefronts are the faster: up to four tokens, and up to eight for a
// gated block, which gives them twice the rows, of at most 4096 (with the tokens'
// quantisation, four tokens of 4096 x 4096 8.3 us against 9.8 of the better of the
// others, of 28672 x 8192 gated 82 and 94; eight of 1376 x 4096 gated 10.6 and 12.1,
// but of 4096 x 4096 11.7 and 10.0, of 11008 x 4096 gated 26.6 and 23.7).
inline bool i8_rows_pay(int64_t rows, bool gated, int64_t batch) {
  return batch <= 4 || (gated && batch <= kI8RowTokens && rows <= 4096);
}

// Whether they can quantise x on its way: a thread holds `most` octets of a token.
inline bool i8_rows_quantize(int64_t cols, int64_t batch) {
  const int64_t most = batch == 1 ? 8 : batch == 2 ? 4 : 1;
  return batch <= 4 && cols / 8 <= most * kI8RowThreads;
}

// Whether they do, every workgroup again, rather than a launch of its
// own: one or two tokens (one of 4096 x 4096 5.2 us against 8.7, of 11008 x 4096 gated
// 16.5 and 19.3, of 8192 x 28672 39 and 43, two of 4096 x 11008 12.6 and 15.3), and four
// where the rows are few (4096 x 4096 8.3 and 10.1, 1376 x 4096 gated 7.8 and 8.9, but
// 11008 x 4096 gated 26 and 22).
inline bool i8_quant_pays(int64_t rows, int64_t cols, bool gated, int64_t batch) {
  return i8_rows_pay(rows, gated, batch) && i8_rows_quantize(cols, batch) &&
         (batch <= 2 || rows * (gated ? 2 : 1) <= 8192);
}

// Modelled duration of the skinny kernel (i8_gemm.hip) in us: 0.95 us and 0.054 us a token
// for each turn of its wavefronts, or, with many rows, 1.6 us and 0.062 us a token for a turn of
// 256 workgroups (fitted as the tiles: 16 x 4096 x 4096 7.2 us against their 9.5, 16 x
// 11008 x 4096 15.8 and 13.3, 32 x 1024 x 8192 13.3 and 8.5).
constexpr int64_t kI8MostSkinny = 64;  // tokens
inline double i8_skinny_us(int64_t rows, int64_t cols, bool gated, int64_t batch) {
  const double turns = (double)((cols + 2047) / 2048), tok_tiles = (double)((batch + 31) / 32);
  const double tiles = (double)((rows + 15) / 16) * (gated ? 2 : 1) * tok_tiles;
  const double b = (double)std::min<int64_t>(batch, 32);
  const double alone = turns * (0.95 + 0.054 * b), full = tiles * turns / 256.0 * (1.6 + 0.062 * b);
  return 2.6 + std::cbrt((float)(alone * alone * alone + full * full * full));
}

// Workspace of quantised activations: scales, then codes, from multiples of 256 bytes on.
inline int64_t i8_codes_at(int64_t batch) { return (batch * 4 + 255) / 256 * 256; }
inline int64_t i8_product_at(int64_t cols, int64_t batch) { return i8_codes_at(batch) + (batch * cols + 255) / 256 * 256; }

// The kernels of a product (`quant`: x is halves), by its sizes: chosen once a call,
// since a choice takes the host a microsecond.
struct I8Route {
  enum Kind { kRows, kSkinny, kTiles } kind;
  bool inside;  // the product's own workgroups quantise x
  I8Plan plan;  // kTiles
  int64_t ws_bytes;
};
inline I8Route i8_route(int64_t rows, int64_t cols, bool gated, int64_t batch, bool quant) {
  I8Route r = {I8Route::kRows, quant && i8_quant_pays(rows, cols, gated, batch), {}, 0};
  if (r.inside) return r;
  if (!i8_rows_pay(rows, gated, batch)) {
    r.plan = i8_tile_plan(rows, cols, gated, batch);
    const bool tiles = batch > kI8MostSkinny || r.plan.us < i8_skinny_us(rows, cols, gated, batch);
    r.kind = tiles ? I8Route::kTiles : I8Route::kSkinny;
  }
  r.ws_bytes = (quant ? i8_product_at(cols, batch) : 0) + (r.kind == I8Route::kTiles ? r.plan.sums : 0);
  return r;
}

// --- gradients -----------------------------------------------------------------
namespace i8_grad {
typedef I8GradShape<2, 2, 4, 2, 1, 3> Large;   // 256 columns x 128 tokens
typedef I8GradShape<2, 1, 4, 2, 1, 2> Half;    // 256 x 64, two workgroups to a CU
typedef I8GradShape<2, 1, 2, 1, 2, 2> Small;   // 128 x 32, two
typedef I8GradShape<2, 1, 2, 1, 2, 3> Deep;    // 128 x 32, one, with a step more under way

// Fitted to eight layers from 1 to 2048 tokens, each shape and 1, 2, 4 and 8 splits
// measured at each, within 5 % at the median; the choice costs 0.3 % on average against
// the best one.
// (Each shape with its best splits, terms' launch included, Large to Deep: 301 x 4096 x
// 11008 94, 72, 95 and 121 us, 2048 x 11008 x 4096 348, 374, 486, 587, 1 x 28672 x 8192 92,
// 70, 58, 60, 9 x 11008 x 4096 41, 32, 24, 22. Tiles of 128 x 64, by two or four
// wavefronts, 256 x 64 by four and 256 x 128 by four would spare 0.1 % of the choice's time
// at most.)
constexpr I8TileCost kCosts[] = {i8_cost_of<Large>(1.07, 1.309, 0.0, 0.0), i8_cost_of<Half>(1.42, 0.836, 0.261, 0.514),
                                 i8_cost_of<Small>(2.12, 0.73, 0.462, 0.189), i8_cost_of<Deep>(2.12, 0.719, 0.122, 0.0)};
constexpr I8Rates kRates = {5.3e6, 0.7e9, 4.7e6, 0.0, 2.2, 512};
}  // namespace i8_grad

inline I8Plan i8_grad_plan(int64_t rows, int64_t cols, bool gated, int64_t batch) {
  return i8_choose(i8_grad::kCosts, i8_grad::kRates, cols, false, batch, (int)((rows + 63) / 64) * (gated ? 2 : 1),
                   (double)rows * (gated ? 2 : 1) * (double)cols);
}

// Rows of one matrix among the terms: whole steps.
inline int64_t i8_term_rows(int64_t rows) { return (rows + 63) / 64 * 64; }
// Workspace: the powers, the terms (two halves each) and the split sums, from multiples of
// 256 bytes on.
inline int64_t i8_terms_at(int64_t batch) { return (batch * 4 + 255) / 256 * 256; }
inline int64_t i8_grad_sums_at(int64_t rows, bool gated, int64_t batch) {
  return i8_terms_at(batch) + (batch * i8_term_rows(rows) * (gated ? 2 : 1) * 4 + 255) / 256 * 256;
}
inline int64_t i8_grad_ws_bytes(int64_t rows, bool gated, int64_t batch, const I8Plan &plan) {
  return i8_grad_sums_at(rows, gated, batch) + plan.sums;
}

}  // namespace aqlm
