// zero_hidden_api.cpp -- host side of the operators on the hidden matrices:
// argument checks, launch shapes and the extern "C" entry points declared in
// include/zero.h.  As in zero_api.cpp, nothing allocates device memory and every
// table travels in the kernel arguments.
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <cmath>
#include <vector>

#include "zero.h"
#include "zero_hidden.h"
#include "zero_host.h"

using namespace zk::host;
using namespace zk::hidden;

namespace {

constexpr int64_t kMaxWide = int64_t(1) << 21;    // of a row that is staged: 256 rows stay within 2^31 bytes
constexpr int64_t kMaxLong = int64_t(1) << 30;
constexpr int64_t kMaxSide = int64_t(1) << 20;    // of a matrix to orthogonalise
constexpr int kStage = 64;                        // depth of a stage of the products

int64_t round_up(int64_t n, int64_t to) { return ceil_div(n, to) * to; }

// ---------------------------------------------------------------------------
// Launch shapes
// ---------------------------------------------------------------------------

// Time of a product's launch in us, from what a stage takes on one CU: `alone`
// with one workgroup there, `full` for each of `slots` that share it,
// and `start` for a tile's first loads and its epilogue.  Fitted to 600 timed
// launches (19 shapes, the three products, every tile and 1 to 32 pieces), whose
// best choice it misses by 2% on average.
struct TileCost { double alone, full, start; int slots; };
constexpr TileCost kCost[kTiles] = {{1.35, 1.08, 9.7, 1}, {0.61, 0.50, 4.1, 2}, {0.23, 0.19, 3.0, 3}};
constexpr int kCus = 256;
constexpr double kJoinStart = 3.2;       // us: a launch that joins pieces of k
constexpr double kPartRate = 4.5e6;      // bytes a us, written and read again

double cost_of(int tile, int64_t tiles, int64_t stages) {
  const TileCost& c = kCost[tile];
  const int64_t per_cu = ceil_div(tiles, kCus), rounds = per_cu / c.slots, rest = per_cu % c.slots;
  const double last = rest ? std::max(c.alone, rest * c.full) : 0.0;
  return (double)stages * ((double)rounds * c.slots * c.full + last) + c.start * (double)(rounds + (rest ? 1 : 0));
}

// How a product is cut into workgroups: `whole` tiles in one piece, the others in
// `splits` pieces of k.
struct Pick {
  int tile;
  int64_t whole, cut;
  int splits;
  double us;
};

int64_t part_bytes(const Pick& c) { return c.splits > 1 ? c.cut * c.splits * kTileSize[c.tile] * kTileSize[c.tile] * 4 : 0; }

double join_cost(int tile, int64_t tiles, int64_t splits) {
  return kJoinStart + (double)(tiles * kTileSize[tile]) * kTileSize[tile] * 4.0 * (double)(splits + 1) / kPartRate;
}

// For `batch` products of m x n x k.  With splits > 0 every tile is cut into so many
// pieces.  Otherwise all tiles are cut alike, or only those of a last round that
// would leave most CUs idle.  Tiles too small for one launch to hold them all are left
// out (2^30 rows into one column are 2^32 work items of the 64-row tile).
Pick pick(int64_t m, int64_t n, int64_t k, int64_t batch, int splits, bool upper = false) {
  const int64_t stages = std::max<int64_t>(1, ceil_div(k, kStage));
  Pick best = {kTile256, batch * ceil_div(m, kTileSize[kTile256]) * ceil_div(n, kTileSize[kTile256]), 0, 1, 1e300};
  for (int tile = 0; tile < kTiles; ++tile) {
    const int64_t tm = ceil_div(m, kTileSize[tile]), tn = ceil_div(n, kTileSize[tile]);
    const int64_t tiles = batch * (upper ? tm * (tm + 1) / 2 : tm * tn);
    for (int64_t s = splits ? splits : 1; s <= (splits ? splits : 64); s *= 2) {
      if (!splits && s > 1 && stages / s < 4) break;    // a piece has four stages or more
      const int64_t per = ceil_div(stages, s), now = ceil_div(stages, per);
      if (tiles * now > most_blocks(kTileThreads[tile])) continue;
      double us = cost_of(tile, tiles * now, per);
      if (now > 1) us += join_cost(tile, tiles, now);
      if (us < best.us) best = now > 1 ? Pick{tile, 0, tiles, (int)now, us} : Pick{tile, tiles, 0, 1, us};
    }
    const int64_t slots = (int64_t)kCus * kCost[tile].slots, whole = tiles / slots * slots, rest = tiles - whole;
    if (splits || whole == 0 || rest == 0 || tiles > most_blocks(kTileThreads[tile]) - slots) continue;
    const int64_t s = std::min(slots / rest, stages / 4);
    if (s < 2) continue;
    const int64_t per = ceil_div(stages, s), now = ceil_div(stages, per);
    const double us = cost_of(tile, whole, stages) + cost_of(tile, rest * now, per) + join_cost(tile, rest, now);
    if (now > 1 && us < best.us) best = {tile, whole, rest, (int)now, us};
  }
  return best;
}

void lay_out(Product& p, int64_t m, int64_t n, int64_t k, const Pick& c, void* part, bool upper = false) {
  const int64_t stages = std::max<int64_t>(1, ceil_div(k, kStage)), per = ceil_div(stages, c.splits);
  p.m = (int32_t)m;
  p.n = (int32_t)n;
  p.k = (int32_t)k;
  p.size = kTileSize[c.tile];
  p.tm = (int32_t)ceil_div(m, p.size);
  p.tn = (int32_t)ceil_div(n, p.size);
  p.tiles = (int32_t)std::min<int64_t>(INT32_MAX, upper ? (int64_t)p.tm * (p.tm + 1) / 2 : (int64_t)p.tm * p.tn);
  p.whole = (int32_t)std::min<int64_t>(INT32_MAX, c.whole);
  p.cut = (int32_t)std::min<int64_t>(INT32_MAX, c.cut);
  p.splits = c.splits;
  p.k_piece = (int32_t)(per * kStage);
  p.part = (float*)part;
}

int64_t blocks_of(const Pick& c) { return c.whole + c.cut * c.splits; }
int64_t joins_of(const Pick& c) {
  return c.splits > 1 ? ceil_div(c.cut * kTileSize[c.tile] * (kTileSize[c.tile] / 4), kJoinThreads) : 0;
}

zero_status check_grid(int64_t blocks, int threads) {
  if (blocks > most_blocks(threads))
    return fail(ZERO_EUNSUPPORTED, "the call needs %lld workgroups of %d, one launch takes %lld", (long long)blocks, threads,
                (long long)most_blocks(threads));
  return ok();
}

// An operand's rows can be loaded straight into LDS, which takes addresses that are
// multiples of 4, and whole words: form M's last row must not end inside one.
bool direct_k(const void* p, int64_t ld) { return aligned(p, 4) && ld % 2 == 0; }
bool direct_m(const void* p, int64_t ld, int64_t width) { return direct_k(p, ld) && width % 2 == 0; }

// Odd rows cannot be loaded straight into LDS; the products then run at 0.8 of
// their rate in large tiles and half of it in small ones.  Where a quarter of the
// product's time is more than copying the odd operands takes, they are copied into
// the workspace first, with rows of whole eights (12527 x 33 x 12736 backward pass: 325 -> 276 us).
struct Copies {
  bool a, b;
  int64_t lda, ldb, a_bytes, b_bytes;
};

constexpr double kCopyStart = 4.0;       // us
constexpr double kCopyRate = 4.5e6;      // bytes a us, read and written

Copies copies_of(const Pick& c, bool odd_a, int64_t rows_a, int64_t width_a, bool odd_b, int64_t rows_b, int64_t width_b) {
  Copies p = {odd_a, odd_b, round_up(width_a, 8), round_up(width_b, 8), 0, 0};
  if (odd_a) p.a_bytes = round_up(rows_a * p.lda * 2, 256);
  if (odd_b) p.b_bytes = round_up(rows_b * p.ldb * 2, 256);
  const double us = kCopyStart * (odd_a + odd_b) + 2.0 * (double)(p.a_bytes + p.b_bytes) / kCopyRate;
  if (!(us < 0.25 * c.us)) p = {false, false, 0, 0, 0, 0};
  return p;
}

zero_status copy_rows(const void* src, int64_t rows, int64_t width, int64_t ld_src, void* dst, int64_t ld_dst, void* stream) {
  const int64_t units = ld_dst / 8, part = most_blocks(kCopyThreads) * kCopyThreads / units;      // rows a launch
  for (int64_t row = 0; row < rows; row += part) {
    const int64_t now = std::min(part, rows - row);
    const CopyRowsArgs a = {(const char*)src + row * ld_src * 2, (char*)dst + row * ld_dst * 2, now, ld_src, ld_dst, (int32_t)width,
                            (int32_t)units};
    if (const int err = launch_copy_rows(a, ceil_div(now * units, kCopyThreads), stream)) return hip_fail(err);
  }
  return ok();
}

// Puts the operands that are to be copied in their places behind `at` bytes of the
// workspace.
zero_status make_copies(Product& p, const Copies& c, int64_t rows_a, int64_t width_a, int64_t rows_b, int64_t width_b, void* ws,
                        int64_t at, void* stream) {
  if (c.a) {
    char* d = (char*)ws + at;
    if (zero_status st = copy_rows(p.a, rows_a, width_a, p.lda, d, c.lda, stream)) return st;
    p.a = d;
    p.lda = c.lda;
  }
  if (c.b) {
    char* d = (char*)ws + at + c.a_bytes;
    if (zero_status st = copy_rows(p.b, rows_b, width_b, p.ldb, d, c.ldb, stream)) return st;
    p.b = d;
    p.ldb = c.ldb;
  }
  return ok();
}

// ---------------------------------------------------------------------------
// Arguments
// ---------------------------------------------------------------------------

// The weight: a tensor of the plan seen as rows of in_features elements.
zero_status weight_of(zero_plan_t p, int32_t tensor, int64_t in_features, int64_t& out_features) {
  if (check_plan(p)) return ZERO_EINVAL;
  if (tensor < 0 || tensor >= (int32_t)p->t_numel.size()) return fail(ZERO_EINVAL, "weight tensor %d out of range", tensor);
  if (in_features < 1) return fail(ZERO_EINVAL, "in_features must be >= 1 (got %lld)", (long long)in_features);
  if (p->t_numel[tensor] % in_features)
    return fail(ZERO_EINVAL, "tensor %d holds %lld elements, no multiple of in_features = %lld", tensor,
                (long long)p->t_numel[tensor], (long long)in_features);
  out_features = p->t_numel[tensor] / in_features;
  if (in_features > kMaxWide)
    return fail(ZERO_EUNSUPPORTED, "in_features %lld exceeds %lld", (long long)in_features, (long long)kMaxWide);
  if (out_features > kMaxLong)
    return fail(ZERO_EUNSUPPORTED, "%lld output features exceed %lld", (long long)out_features, (long long)kMaxLong);
  return ok();
}

zero_status bias_of(zero_plan_t p, int32_t bias, int64_t out_features) {
  if (bias < 0) return ok();
  if (bias >= (int32_t)p->t_numel.size()) return fail(ZERO_EINVAL, "bias tensor %d out of range", bias);
  if (p->t_numel[bias] != out_features)
    return fail(ZERO_EINVAL, "bias tensor %d holds %lld elements, the layer has %lld outputs", bias,
                (long long)p->t_numel[bias], (long long)out_features);
  return ok();
}

zero_status check_n(int64_t n) {
  if (n < 0) return fail(ZERO_EINVAL, "n must be >= 0 (got %lld)", (long long)n);
  if (n > kMaxLong) return fail(ZERO_EUNSUPPORTED, "n = %lld exceeds %lld", (long long)n, (long long)kMaxLong);
  return ok();
}

zero_status check_16(int dt, const char* what) {
  if (!valid_dt(dt)) return fail(ZERO_EINVAL, "unknown dtype %d", dt);
  if (!is16(dt)) return fail(ZERO_EUNSUPPORTED, "%s are 16-bit, not fp32", what);
  return ok();
}

zero_status check_act(int act) {
  if (act < ZERO_ACT_NONE || act > ZERO_ACT_SILU) return fail(ZERO_EINVAL, "unknown activation %d", act);
  return ok();
}

// n rows of `width` 16-bit elements; a staged operand's stride is bounded.
zero_status check_rows(const void* p, int64_t n, int64_t width, int64_t stride, bool staged, const char* what, Range& r) {
  if (stride < width)
    return fail(ZERO_EINVAL, "the stride %lld of %s is shorter than a row of %lld", (long long)stride, what, (long long)width);
  if (staged && stride > kMaxWide)
    return fail(ZERO_EUNSUPPORTED, "the stride %lld of %s exceeds %lld", (long long)stride, what, (long long)kMaxWide);
  const int64_t span = span_of(n, stride, width);
  if (span < 0) return fail(ZERO_EINVAL, "the extent of %s overflows", what);
  if (zero_status st = check_buffer(p, span, 2, what)) return st;
  r = range_of(p, span, 2, what);
  return ok();
}

bool same_place(const Range& a, const Range& b) { return a.lo == b.lo && a.hi == b.hi; }

// The part of a tensor that rank's slice holds (all of it for rank < 0), and
// where that part starts in dst.
void part_of_tensor(const zero_plan_s& p, int32_t tensor, int32_t rank, int64_t& lo, int64_t& hi, int64_t& at) {
  const int64_t off = p.t_off[tensor], numel = p.t_numel[tensor];
  lo = 0;
  hi = numel;
  at = off;
  if (rank >= 0) {
    const auto& b = p.buckets[p.t_bucket[tensor]];
    const int64_t own = b.flat_off + (int64_t)rank * b.shard_numel;
    lo = std::max<int64_t>(0, own - off);
    hi = std::min<int64_t>(numel, own + b.shard_numel - off);
    at = b.shard_off + (off + lo - own);
  }
}

// Rows of dz whose sums one bias workgroup takes, from n and the outputs alone: as
// many as leave about 1024 workgroups, 64 to 512 (12736 columns of 12527 rows beside
// their weight: 326 -> 237 us against 256 workgroups).
int64_t bias_chunk(int64_t n, int64_t out_features) {
  const int64_t want = ceil_div(n, std::max<int64_t>(1, 1024 / ceil_div(out_features, kBiasCols)));
  return std::min<int64_t>(512, std::max<int64_t>(64, round_up(want, 32)));
}

// Pieces of k where every tile is to have the same, for the whole result and a
// share of its rows.
int alike(int64_t m, int64_t n, int64_t k, int64_t shares) {
  const int64_t stages = std::max<int64_t>(1, ceil_div(k, kStage));
  double us = 1e300;
  int best = 1;
  for (int64_t s = 1; s <= 64 && (s == 1 || stages / s >= 4); s *= 2) {
    const Pick c = pick(m, n, k, 1, (int)s);
    const double both = shares > 1 ? c.us + pick(ceil_div(m, shares), n, k, 1, (int)s).us : c.us;
    if (both < us) {
      us = both;
      best = c.splits;
    }
  }
  return best;
}

struct WeightShape {
  int64_t lo, hi, at;       // elements of the weight, and their place in dst
  int64_t row0, rows;
  int splits;
  Pick c;
  Copies copies;
  int64_t part, bias_part, bytes;  // of the workspace
};

WeightShape weight_shape(const zero_plan_s& p, int32_t weight, int64_t in_features, int64_t out_features, int64_t n, int32_t rank) {
  WeightShape s;
  part_of_tensor(p, weight, rank, s.lo, s.hi, s.at);
  s.row0 = s.rows = 0;
  if (s.lo < s.hi) {      // in whole eights where there are, for their loads' sake
    s.row0 = s.lo / in_features / 8 * 8;
    s.rows = std::min(round_up((s.hi - 1) / in_features + 1, 8), out_features) - s.row0;
  }
  // The pieces of k follow from the whole weight, and every tile has the same, so that
  // a slice's sums are those of the full buffer.
  s.splits = alike(out_features, in_features, n, p.n_d);
  s.c = s.rows > 0 ? pick(s.rows, in_features, n, 1, s.splits) : Pick{kTile64, 0, 0, 1, 0.0};
  s.copies = copies_of(s.c, n > 1 && out_features % 2, n, s.rows, n > 1 && in_features % 2, n, in_features);
  s.part = round_up(part_bytes(s.c), 256);
  s.bias_part = round_up(ceil_div(n, bias_chunk(n, out_features)) * out_features * 4, 256);
  s.bytes = s.part + s.bias_part + s.copies.a_bytes + s.copies.b_bytes;
  return s;
}

// What zero_linear and zero_linear_input_grad run: n rows into `out` columns over
// `inner` terms.  The operands that may be copied follow from the shapes and the plan.
struct LinearShape {
  Pick c;
  Copies copies;
  int64_t part, bytes;      // of the workspace
};

LinearShape linear_shape(const zero_plan_s& p, int32_t weight, int64_t in_features, int64_t out_features, int64_t n, bool grad) {
  LinearShape s;
  const int64_t cols = grad ? in_features : out_features, inner = grad ? out_features : in_features;
  s.c = pick(n, cols, inner, 1, 0);
  s.copies = copies_of(s.c, n > 1 && inner % 2, n, inner, in_features % 2 || p.t_off[weight] % 2, out_features, in_features);
  s.part = round_up(part_bytes(s.c), 256);
  s.bytes = s.part + s.copies.a_bytes + s.copies.b_bytes;
  return s;
}

zero_status run_linear(LinearArgs& a, int epi, int dt, const Pick& c, bool direct, void* stream) {
  const int64_t joins = joins_of(c);
  if (zero_status st = check_grid(blocks_of(c), kTileThreads[c.tile])) return st;
  if (zero_status st = check_grid(joins, kJoinThreads)) return st;
  if (const int err = launch_linear(a, epi, dt, c.tile, direct, stream)) return hip_fail(err);
  if (joins == 0) return ok();
  return launched(launch_linear_join(a, epi, dt, joins, stream));
}

// ---------------------------------------------------------------------------
// Orthogonalisation: groups of matrices of one shape
// ---------------------------------------------------------------------------

constexpr int kDefaultSteps = 5;
const zero_newton_schulz kDefaultPoly = {kDefaultSteps, 3.4445, -4.7750, 2.0315, 1e-7};
// From this step on A - I / 2 is stored in place of A.
constexpr int kShiftFrom = 3;
constexpr float kShift = 0.5f;

struct Group {
  int64_t rows, cols;
  std::vector<int64_t> off;       // element of the flat buffer
  std::vector<float> scale;
};

// Workspace of a batch of `batch` matrices, in bytes from its start.
struct OrthoSpace {
  int64_t ldx, ldn, rows_pad, side;   // padded columns of X, of A; padded rows of X
  int64_t zx, zn;                     // elements of X and of A
  int64_t pitch, again;               // of X: elements between rows, and to its second copy (0: none)
  int64_t sums, factor, x0, x1, low, poly, part, total;    // A lies where the next X goes
  Pick c[3];                          // of the three products
};

OrthoSpace ortho_space(int64_t rows, int64_t cols, int64_t batch) {
  OrthoSpace s;
  s.ldx = round_up(cols, 8);
  s.rows_pad = round_up(rows, 8);
  s.side = std::min(s.rows_pad, s.ldx);
  s.ldn = s.side;
  const int64_t wide = std::max(s.rows_pad, s.ldx);
  s.zx = s.rows_pad * s.ldx;
  s.zn = s.side * s.ldn;
  s.pitch = s.ldx;
  s.again = 0;
  s.c[kGram] = pick(s.side, s.side, wide, batch, 0, true);
  s.c[kPoly] = pick(s.side, s.side, s.side, batch, 0, true);
  s.c[kNext] = pick(s.rows_pad, s.ldx, s.side, batch, 0);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += round_up(bytes, 256);
    return here;
  };
  s.sums = take(batch * kNormBlocks * 8);
  s.factor = take(batch * 8);
  s.x0 = take(batch * s.zx * 2);
  s.x1 = take(batch * s.zx * 2);
  s.low = take(batch * s.zx * 2);
  s.poly = take(batch * s.zn * 2);
  s.part = take(std::max({part_bytes(s.c[kGram]), part_bytes(s.c[kPoly]), part_bytes(s.c[kNext])}));
  s.total = at;
  return s;
}

// The same for matrices with a short side (zn is P's): X twice along k, pieces of A.
OrthoSpace thin_space(int64_t rows, int64_t cols, int64_t batch) {
  OrthoSpace s;
  memset(&s, 0, sizeof s);
  const bool tall = rows > cols;
  s.ldx = round_up(cols, 8);
  s.rows_pad = round_up(rows, 8);
  s.side = std::min(s.rows_pad, s.ldx);
  s.ldn = 2 * s.side;
  s.zx = 2 * s.rows_pad * s.ldx;
  s.zn = s.side * s.ldn;
  s.pitch = tall ? 2 * s.ldx : s.ldx;
  s.again = tall ? s.ldx : s.rows_pad * s.ldx;
  // Pieces of A: two workgroups a CU, of four stages or more.
  const int64_t stages = ceil_div(std::max(s.rows_pad, s.ldx), kStage);
  const int64_t want = std::max<int64_t>(1, std::min({ceil_div(2 * kCus, batch), stages / 4, int64_t(32)}));
  s.c[kGram] = {kTile64, 0, batch, (int)ceil_div(stages, ceil_div(stages, want)), 0.0};
  s.c[kNext] = pick(s.rows_pad, s.ldx, 2 * s.side, batch, 0);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += round_up(bytes, 256);
    return here;
  };
  s.sums = take(batch * kNormBlocks * 8);
  s.factor = take(batch * 8);
  s.x0 = take(batch * s.zx * 2);
  s.poly = take(batch * s.zn * 2);
  s.part = take(std::max(batch * s.c[kGram].splits * kThinSide * kThinSide * 4, part_bytes(s.c[kNext])));
  s.total = at;
  return s;
}

bool is_thin(int64_t rows, int64_t cols) { return std::min(rows, cols) <= kThinSide; }

// Whether P may stand for the steps.  What rounding leaves of A in directions that X
// lacks (equal rows, say) grows by a^2 in each step, and P by a: 64 x 128 of three strong
// directions over 10^-5 of noise ends 0.0002 off with 10 steps of a = 1.875, which grow by 537, and 0.03
// with 14, which grow by 6638 (its number formats emulated).
bool may_be_thin(const zero_newton_schulz& q) { return std::pow(std::fabs(q.a), q.steps) <= 1000.0; }

OrthoSpace space_of(bool thin, int64_t rows, int64_t cols, int64_t batch) {
  return thin ? thin_space(rows, cols, batch) : ortho_space(rows, cols, batch);
}

// As many matrices as one batch takes: all of them where X, A and B stay within
// 1 GiB, as launches of many tiles waste the least (48 matrices of 768 x 768 in one
// batch, two and four: 870, 875 and 1160 us; 24 of 1024 x 4096 in one and two: 2370
// and 2520), or a few batches more where those fill their rounds better.  With padded
// sides, norms and pieces of sums the workspace stays within an eighth more (32 of
// 2048 x 2048, which are 1 GiB by themselves, in one batch and two: 6335 and 7047 us).
int64_t batch_of(bool thin, int64_t rows, int64_t cols, int64_t count) {
  constexpr int64_t bulk = int64_t(1) << 30, limit = bulk + bulk / 8;
  const int64_t n = std::min(rows, cols), bytes = rows * cols * 6 + n * n * 2;
  int64_t most = std::min<int64_t>({count, kMaxBatch, std::max<int64_t>(1, bulk / bytes)});
  while (most > 1) {
    const int64_t total = space_of(thin, rows, cols, most).total;
    if (total <= limit) break;
    most = std::max<int64_t>(1, std::min(most - 1, (int64_t)((double)most * (double)limit / (double)total)));
  }
  const int64_t fewest = ceil_div(count, most);
  int64_t best = 0;
  double us = 1e300;
  for (int64_t parts = fewest; parts <= count && (parts <= fewest + 3 || best == 0); ++parts) {
    const int64_t batch = ceil_div(count, parts);
    const OrthoSpace s = space_of(thin, rows, cols, batch);
    if (s.total > limit && batch > 1) continue;       // fewer matrices may be cut into more pieces
    const double now = (double)ceil_div(count, batch) * (s.c[kGram].us + s.c[kPoly].us + s.c[kNext].us);
    if (now < us) us = now, best = batch;
  }
  return best;
}

zero_status collect(zero_plan_t p, const zero_matrix* ms, int32_t n, std::vector<Group>& groups) {
  if (check_plan(p)) return ZERO_EINVAL;
  if (n < 0) return fail(ZERO_EINVAL, "n_matrices must be >= 0 (got %d)", n);
  if (n > 0 && !ms) return fail(ZERO_EINVAL, "matrices is NULL");
  std::vector<char> seen(p->t_numel.size(), 0);
  for (int32_t i = 0; i < n; ++i) {
    const zero_matrix& m = ms[i];
    if (m.tensor < 0 || m.tensor >= (int32_t)p->t_numel.size())
      return fail(ZERO_EINVAL, "matrix %d: tensor %d out of range", i, m.tensor);
    if (seen[m.tensor]) return fail(ZERO_EINVAL, "matrix %d: tensor %d is listed twice", i, m.tensor);
    seen[m.tensor] = 1;
    if (m.rows < 1 || m.cols < 1)
      return fail(ZERO_EINVAL, "matrix %d: rows and cols must be >= 1 (got %lld, %lld)", i, (long long)m.rows, (long long)m.cols);
    if (m.rows > kMaxSide || m.cols > kMaxSide)
      return fail(ZERO_EUNSUPPORTED, "matrix %d: %lld x %lld exceeds a side of %lld", i, (long long)m.rows, (long long)m.cols,
                  (long long)kMaxSide);
    const int64_t numel = p->t_numel[m.tensor], size = m.rows * m.cols;
    if (numel % size)
      return fail(ZERO_EINVAL, "matrix %d: tensor %d holds %lld elements, no multiple of %lld x %lld", i, m.tensor,
                  (long long)numel, (long long)m.rows, (long long)m.cols);
    if (!std::isfinite((float)m.scale)) return fail(ZERO_EINVAL, "matrix %d: scale %g is beyond fp32", i, m.scale);
    auto g = std::find_if(groups.begin(), groups.end(), [&](const Group& x) { return x.rows == m.rows && x.cols == m.cols; });
    if (g == groups.end()) {
      groups.push_back({m.rows, m.cols, {}, {}});
      g = groups.end() - 1;
    }
    for (int64_t k = 0; k < numel / size; ++k) {
      g->off.push_back(p->t_off[m.tensor] + k * size);
      g->scale.push_back((float)m.scale);
    }
  }
  return ok();
}

// Whether the matrices between the products stay within fp16: the largest singular
// values of X, A and b A + c A A over the steps, by points a 256th of the range apart.
// And how far directions that the matrix hardly has are brought up, by a in each step: what
// fp16 rounds off A and B couples them to the strong ones, which at the limit is 0.01 to
// 0.02 of the result.
zero_status check_growth(const zero_newton_schulz& q) {
  constexpr double most = 30000.0, grown = 10000.0;
  if (std::pow(std::fabs(q.a), q.steps) > grown)
    return fail(ZERO_EUNSUPPORTED, "%d steps of a = %g bring rounding up by more than %g", q.steps, q.a, grown);
  double hi = 1.0;
  for (int step = 0; step < q.steps; ++step) {
    double next = 0.0, b = hi * hi;
    for (int i = 1; i <= 256; ++i) {
      const double s = hi * i / 256.0, s2 = s * s, t = (q.b + q.c * s2) * s2;
      b = std::max(b, std::fabs(t));
      next = std::max(next, std::fabs(s * (q.a + t)));
    }
    if (b > most || next > most)
      return fail(ZERO_EUNSUPPORTED, "step %d of the polynomial reaches singular values of %g, beyond %g", step + 1, std::max(b, next), most);
    hi = next;
  }
  return ok();
}

// Matrices that one workgroup orthogonalises in its LDS: 16384 elements with the
// sides rounded up to 32.
bool is_small(int64_t rows, int64_t cols) {
  return rows <= kSmallElems && cols <= kSmallElems && round_up(rows, 32) * round_up(cols, 32) <= kSmallElems;
}

int64_t ortho_bytes(const std::vector<Group>& groups) {
  int64_t most = 0;
  for (const Group& g : groups) {
    if (g.off.empty() || is_small(g.rows, g.cols)) continue;
    for (int thin = is_thin(g.rows, g.cols); thin >= 0; --thin)      // either way may be taken, by the polynomial
      most = std::max(most, space_of(thin, g.rows, g.cols, batch_of(thin, g.rows, g.cols, (int64_t)g.off.size())).total);
  }
  return most;
}

// One product of a step over the batch.  A last batch of fewer matrices is laid out
// as the others are, with as many tiles whole as it has.
zero_status run_ortho(OrthoArgs& a, int64_t m, int64_t n, int64_t k, const Pick& c, void* part, void* stream) {
  lay_out(a.p, m, n, k, c, part, a.epi != kNext);
  Pick now = c;
  const int64_t tiles = (int64_t)a.batch * a.p.tiles;
  now.whole = std::min(c.whole, tiles);
  now.cut = tiles - now.whole;
  a.p.whole = (int32_t)now.whole;
  a.p.cut = (int32_t)now.cut;
  const int64_t joins = joins_of(now);
  if (zero_status st = check_grid(blocks_of(now), kTileThreads[c.tile])) return st;
  if (zero_status st = check_grid(joins, kJoinThreads)) return st;
  if (const int err = launch_ortho(a, c.tile, blocks_of(now), stream)) return hip_fail(err);
  if (joins == 0) return ok();
  return launched(launch_ortho_join(a, joins, stream));
}

zero_status ortho_small(const Group& g, int64_t first, int64_t batch, const zero_newton_schulz& poly, const void* src, int src_dt,
                        void* dst, int dst_dt, void* stream) {
  OrthoSmallArgs a;
  memset(&a, 0, sizeof a);
  a.src = src;
  a.dst = dst;
  a.eps = poly.eps;
  a.a = (float)poly.a;
  a.b = (float)poly.b;
  a.c = (float)poly.c;
  a.shift = kShift;
  a.shift_from = kShiftFrom;
  a.steps = poly.steps;
  a.rows = (int32_t)g.rows;
  a.cols = (int32_t)g.cols;
  a.rp = (int32_t)round_up(g.rows, 32);
  a.cp = (int32_t)round_up(g.cols, 32);
  a.src_dt = src_dt;
  a.dst_dt = dst_dt;
  a.is_short = std::min(g.rows, g.cols) <= kShortSide && may_be_thin(poly);
  for (int64_t i = 0; i < batch; ++i) {
    a.scale[i] = g.scale[first + i];
    a.off[i] = g.off[first + i];
  }
  return launched(launch_ortho_small(a, batch, stream));
}

// The norms and the first X of a batch.
zero_status ortho_load(const Group& g, const OrthoSpace& s, int64_t first, int64_t batch, const zero_newton_schulz& poly, const void* src,
                       int src_dt, char* ws, void* stream) {
  OrthoLoadArgs l;
  memset(&l, 0, sizeof l);
  l.src = src;
  l.x = ws + s.x0;
  l.sums = (double*)(ws + s.sums);
  l.factor = (float*)(ws + s.factor);
  l.eps = poly.eps;
  l.numel = g.rows * g.cols;
  l.zx = s.zx;
  l.pitch = s.pitch;
  l.again = s.again;
  l.rows = (int32_t)g.rows;
  l.cols = (int32_t)g.cols;
  l.ld = (int32_t)s.ldx;
  l.rows_pad = (int32_t)s.rows_pad;
  l.batch = (int32_t)batch;
  // A piece of a norm is 16 Ki elements or more (8192 x 8192: 37 us in 1024 pieces, 282 in 64).
  l.norm_blocks = (int32_t)std::max<int64_t>(1, std::min<int64_t>(kNormBlocks, l.numel / 16384));
  for (int64_t i = 0; i < batch; ++i) l.src_off[i] = g.off[first + i];
  const int64_t load_blocks = batch * ceil_div(s.rows_pad * (s.ldx / 8), kLoadThreads * kLoadUnits);
  if (zero_status st = check_grid(load_blocks, kLoadThreads)) return st;
  if (const int err = launch_ortho_norm(l, src_dt, stream)) return hip_fail(err);
  return launched(launch_ortho_load(l, src_dt, load_blocks, stream));
}

// What the products of a batch share.
void ortho_args(OrthoArgs& a, const Group& g, const OrthoSpace& s, int64_t first, int64_t batch, void* dst, int dst_dt, char* ws) {
  memset(&a, 0, sizeof a);
  a.factor = (const float*)(ws + s.factor);
  a.batch = (int32_t)batch;
  a.tall = g.rows > g.cols;
  a.rows = (int32_t)g.rows;
  a.cols = (int32_t)g.cols;
  a.dst = dst;
  a.dst_dt = dst_dt;
  for (int64_t i = 0; i < batch; ++i) {
    a.scale[i] = g.scale[first + i];
    a.dst_off[i] = g.off[first + i];
  }
}

zero_status ortho_batch(const Group& g, const OrthoSpace& s, int64_t first, int64_t batch, const zero_newton_schulz& poly, const void* src, int src_dt,
                        void* dst, int dst_dt, char* ws, void* stream) {
  const bool tall = g.rows > g.cols;
  if (zero_status st = ortho_load(g, s, first, batch, poly, src, src_dt, ws, stream)) return st;
  OrthoArgs a;
  ortho_args(a, g, s, first, batch, dst, dst_dt, ws);
  a.a = (float)poly.a;
  a.b = (float)poly.b;
  a.c = (float)poly.c;
  char* x = ws + s.x0;
  char* next = ws + s.x1;
  const int64_t wide = std::max(s.rows_pad, s.ldx);
  for (int step = 0; step < poly.steps; ++step) {
    a.first = step == 0;
    a.shift = step >= kShiftFrom ? kShift : 0.0f;
    // A - d I
    a.epi = kGram;
    a.last = 0;
    a.p.a = a.p.b = x;
    a.p.lda = a.p.ldb = s.ldx;
    a.za = a.zb = s.zx;
    a.out = next;
    a.ldo = s.ldn;
    a.zout = s.zn;
    if (zero_status st = run_ortho(a, s.side, s.side, wide, s.c[kGram], ws + s.part, stream)) return st;
    // B
    a.epi = kPoly;
    a.p.a = a.p.b = next;
    a.p.lda = a.p.ldb = s.ldn;
    a.za = a.zb = s.zn;
    a.add = next;
    a.ldadd = s.ldn;
    a.zadd = s.zn;
    a.out = ws + s.poly;
    if (zero_status st = run_ortho(a, s.side, s.side, s.side, s.c[kPoly], ws + s.part, stream)) return st;
    // a X + B X, or a X + X B
    a.epi = kNext;
    a.last = step + 1 == poly.steps;
    a.p.a = tall ? x : ws + s.poly;
    a.p.b = tall ? ws + s.poly : x;
    a.p.lda = tall ? s.ldx : s.ldn;
    a.p.ldb = tall ? s.ldn : s.ldx;
    a.za = tall ? s.zx : s.zn;
    a.zb = tall ? s.zn : s.zx;
    a.add = x;
    a.ldadd = s.ldx;
    a.zadd = s.zx;
    a.low = ws + s.low;
    a.out = next;
    a.ldo = s.ldx;
    a.zout = s.zx;
    if (zero_status st = run_ortho(a, s.rows_pad, s.ldx, s.side, s.c[kNext], ws + s.part, stream)) return st;
    std::swap(x, next);
  }
  return ok();
}

// Matrices with a short side: A's pieces, P from them, P X.
zero_status ortho_thin(const Group& g, const OrthoSpace& s, int64_t first, int64_t batch, const zero_newton_schulz& poly, const void* src, int src_dt,
                       void* dst, int dst_dt, char* ws, void* stream) {
  const bool tall = g.rows > g.cols;
  if (zero_status st = ortho_load(g, s, first, batch, poly, src, src_dt, ws, stream)) return st;
  OrthoArgs a;
  ortho_args(a, g, s, first, batch, dst, dst_dt, ws);
  Pick c = s.c[kGram];
  c.cut = batch;
  a.epi = kGram;
  a.p.a = a.p.b = ws + s.x0;
  a.p.lda = a.p.ldb = s.pitch;
  a.za = a.zb = s.zx;
  lay_out(a.p, s.side, s.side, std::max(s.rows_pad, s.ldx), c, ws + s.part, true);
  if (zero_status st = check_grid(blocks_of(c), kTileThreads[c.tile])) return st;
  if (const int err = launch_ortho(a, c.tile, blocks_of(c), stream)) return hip_fail(err);

  OrthoThinArgs t;
  memset(&t, 0, sizeof t);
  t.part = (const float*)(ws + s.part);
  t.factor = (float*)(ws + s.factor);
  t.p = ws + s.poly;
  t.a = (float)poly.a;
  t.b = (float)poly.b;
  t.c = (float)poly.c;
  t.steps = poly.steps;
  t.splits = a.p.splits;
  t.n = (int32_t)std::min(g.rows, g.cols);
  t.side = (int32_t)s.side;
  if (const int err = launch_ortho_thin(t, batch, stream)) return hip_fail(err);

  a.epi = kNext;              // with a = b = c = 0, so that X itself adds nothing
  a.first = a.last = 1;
  a.p.a = tall ? ws + s.x0 : ws + s.poly;
  a.p.b = tall ? ws + s.poly : ws + s.x0;
  a.p.lda = tall ? s.pitch : s.ldn;
  a.p.ldb = tall ? s.ldn : s.pitch;
  a.za = tall ? s.zx : s.zn;
  a.zb = tall ? s.zn : s.zx;
  a.add = ws + s.x0;
  a.ldadd = s.pitch;
  a.zadd = s.zx;
  return run_ortho(a, s.rows_pad, s.ldx, 2 * s.side, s.c[kNext], ws + s.part, stream);
}

}  // namespace

extern "C" {

size_t zero_linear_workspace_bytes(zero_plan_t p, int32_t weight, int64_t in_features, int64_t n) {
  int64_t out;
  if (weight_of(p, weight, in_features, out) || check_n(n) || n == 0 || out == 0) return 0;
  return (size_t)linear_shape(*p, weight, in_features, out, n, false).bytes;
}

zero_status zero_linear(zero_plan_t p, int32_t weight, int32_t bias, int64_t in_features, const void* params, zero_dtype dt,
                        const void* x, int64_t n, int64_t x_stride, zero_act act, const void* residual,
                        int64_t residual_stride, void* pre, int64_t pre_stride, void* y, int64_t y_stride, void* workspace,
                        size_t ws_bytes, void* stream) {
  return guarded("zero_linear", [&]() -> zero_status {
    int64_t out = 0;
    if (zero_status st = weight_of(p, weight, in_features, out)) return st;
    if (zero_status st = bias_of(p, bias, out)) return st;
    if (zero_status st = check_16(dt, "the products")) return st;
    if (zero_status st = check_act(act)) return st;
    if (zero_status st = check_n(n)) return st;
    if (zero_status st = check_buffer(params, p->psi_pad, 2, "params")) return st;
    Range rx, ry, rr = {0, 0, "residual"}, rp = {0, 0, "pre"};
    if (zero_status st = check_rows(x, n, in_features, x_stride, true, "x", rx)) return st;
    if (zero_status st = check_rows(y, n, out, y_stride, false, "y", ry)) return st;
    if (residual)
      if (zero_status st = check_rows(residual, n, out, residual_stride, false, "residual", rr)) return st;
    if (pre)
      if (zero_status st = check_rows(pre, n, out, pre_stride, false, "pre", rp)) return st;
    const bool some = n > 0 && out > 0;
    const LinearShape s = some ? linear_shape(*p, weight, in_features, out, n, false) : LinearShape{};
    const Pick& c = s.c;
    const size_t need = (size_t)s.bytes;
    if (zero_status st = check_workspace(workspace, ws_bytes, need)) return st;
    std::vector<Range> reads = {range_of(params, p->psi_pad, 2, "params"), rx};
    std::vector<Range> writes = {ry, rp, range_of(workspace, (int64_t)need, 1, "workspace")};
    if (zero_status st = check_disjoint(writes, reads)) return st;
    const bool in_place = residual && same_place(ry, rr) && residual_stride == y_stride;
    if (in_place) writes.erase(writes.begin());
    if (zero_status st = check_disjoint(writes, {rr})) return st;
    if (n == 0 || out == 0) return ok();
    LinearArgs a;
    memset(&a, 0, sizeof a);
    a.p.a = x;
    a.p.b = (const char*)params + p->t_off[weight] * 2;
    a.p.lda = n > 1 ? x_stride : round_up(in_features, 2);     // a single row has no neighbour
    a.p.ldb = in_features;
    lay_out(a.p, n, out, in_features, c, workspace);
    a.out = y;
    a.pre_out = pre;
    a.add = residual;
    a.bias = bias >= 0 ? (const char*)params + p->t_off[bias] * 2 : nullptr;
    a.ldo = y_stride;
    a.ldpre = pre_stride;
    a.ldadd = residual_stride;
    a.act = act;
    if (zero_status st = make_copies(a.p, s.copies, n, in_features, out, in_features, workspace, s.part, stream)) return st;
    const bool direct = direct_k(a.p.a, a.p.lda) && direct_k(a.p.b, a.p.ldb);
    return run_linear(a, 0, dt, c, direct, stream);
  });
}

size_t zero_linear_input_grad_workspace_bytes(zero_plan_t p, int32_t weight, int64_t in_features, int64_t n) {
  int64_t out;
  if (weight_of(p, weight, in_features, out) || check_n(n) || n == 0) return 0;
  return (size_t)linear_shape(*p, weight, in_features, out, n, true).bytes;
}

zero_status zero_linear_input_grad(zero_plan_t p, int32_t weight, int64_t in_features, const void* params, zero_dtype dt,
                                   const void* dz, int64_t n, int64_t dz_stride, zero_act act, const void* pre,
                                   int64_t pre_stride, const void* addend, int64_t addend_stride, void* dx,
                                   int64_t dx_stride, void* workspace, size_t ws_bytes, void* stream) {
  return guarded("zero_linear_input_grad", [&]() -> zero_status {
    int64_t out = 0;
    if (zero_status st = weight_of(p, weight, in_features, out)) return st;
    if (out > kMaxWide) return fail(ZERO_EUNSUPPORTED, "%lld output features exceed %lld", (long long)out, (long long)kMaxWide);
    if (zero_status st = check_16(dt, "the products")) return st;
    if (zero_status st = check_act(act)) return st;
    if (zero_status st = check_n(n)) return st;
    if (zero_status st = check_buffer(params, p->psi_pad, 2, "params")) return st;
    if (n > 0 && (act != ZERO_ACT_NONE) != (pre != nullptr))
      return fail(ZERO_EINVAL, act == ZERO_ACT_NONE ? "pre is given without an activation" : "pre is NULL");
    Range rz, rx, ra = {0, 0, "addend"}, rp = {0, 0, "pre"};
    if (zero_status st = check_rows(dz, n, out, dz_stride, true, "dz", rz)) return st;
    if (zero_status st = check_rows(dx, n, in_features, dx_stride, false, "dx", rx)) return st;
    if (addend)
      if (zero_status st = check_rows(addend, n, in_features, addend_stride, false, "addend", ra)) return st;
    if (pre)
      if (zero_status st = check_rows(pre, n, in_features, pre_stride, false, "pre", rp)) return st;
    const LinearShape s = n > 0 ? linear_shape(*p, weight, in_features, out, n, true) : LinearShape{};
    const Pick& c = s.c;
    const size_t need = (size_t)s.bytes;
    if (zero_status st = check_workspace(workspace, ws_bytes, need)) return st;
    std::vector<Range> writes = {rx, range_of(workspace, (int64_t)need, 1, "workspace")};
    if (zero_status st = check_disjoint(writes, {range_of(params, p->psi_pad, 2, "params"), rz, rp})) return st;
    const bool in_place = addend && same_place(rx, ra) && addend_stride == dx_stride;
    if (in_place) writes.erase(writes.begin());
    if (zero_status st = check_disjoint(writes, {ra})) return st;
    if (n == 0) return ok();
    LinearArgs a;
    memset(&a, 0, sizeof a);
    a.p.a = dz;
    a.p.b = (const char*)params + p->t_off[weight] * 2;
    a.p.lda = n > 1 ? dz_stride : round_up(std::max<int64_t>(out, 1), 2);
    a.p.ldb = in_features;
    lay_out(a.p, n, in_features, out, c, workspace);
    a.out = dx;
    a.pre_in = pre;
    a.add = addend;
    a.ldo = dx_stride;
    a.ldpre = pre_stride;
    a.ldadd = addend_stride;
    a.act = act;
    if (zero_status st = make_copies(a.p, s.copies, n, out, out, in_features, workspace, s.part, stream)) return st;
    const bool direct = direct_k(a.p.a, a.p.lda) && direct_m(a.p.b, a.p.ldb, s.copies.b ? s.copies.ldb : in_features);
    return run_linear(a, 1, dt, c, direct, stream);
  });
}

size_t zero_linear_weight_grad_workspace_bytes(zero_plan_t p, int32_t weight, int64_t in_features, int64_t n, int32_t rank) {
  int64_t out;
  if (weight_of(p, weight, in_features, out) || check_n(n) || n == 0 || out == 0 || rank >= p->n_d) return 0;
  return (size_t)weight_shape(*p, weight, in_features, out, n, rank).bytes;
}

zero_status zero_linear_weight_grad(zero_plan_t p, int32_t weight, int32_t bias, int64_t in_features, const void* dz,
                                    int64_t dz_stride, const void* x, int64_t x_stride, zero_dtype dt, int64_t n,
                                    double scale, void* dst, zero_dtype dst_dt, int32_t rank, int32_t accumulate,
                                    void* workspace, size_t ws_bytes, void* stream) {
  return guarded("zero_linear_weight_grad", [&]() -> zero_status {
    int64_t out = 0;
    if (zero_status st = weight_of(p, weight, in_features, out)) return st;
    if (zero_status st = bias_of(p, bias, out)) return st;
    if (bias == weight) return fail(ZERO_EINVAL, "weight and bias are the same tensor");
    if (out > kMaxWide) return fail(ZERO_EUNSUPPORTED, "%lld output features exceed %lld", (long long)out, (long long)kMaxWide);
    if (zero_status st = check_16(dt, "the products")) return st;
    if (!valid_dt(dst_dt)) return fail(ZERO_EINVAL, "unknown dtype %d", (int)dst_dt);
    if (zero_status st = check_n(n)) return st;
    if (rank >= p->n_d) return fail(ZERO_EINVAL, "rank %d outside [0, %d)", rank, p->n_d);
    if (accumulate != 0 && accumulate != 1) return fail(ZERO_EINVAL, "accumulate must be 0 or 1 (got %d)", accumulate);
    if (!std::isfinite((float)scale)) return fail(ZERO_EINVAL, "scale %g is beyond fp32", scale);
    Range rz, rx;
    if (zero_status st = check_rows(dz, n, out, dz_stride, true, "dz", rz)) return st;
    if (zero_status st = check_rows(x, n, in_features, x_stride, true, "x", rx)) return st;
    const int64_t dst_elems = rank < 0 ? p->psi_pad : p->shard_total;
    if (zero_status st = check_buffer(dst, dst_elems, esize(dst_dt), "dst")) return st;
    const size_t need = zero_linear_weight_grad_workspace_bytes(p, weight, in_features, n, rank);
    if (zero_status st = check_workspace(workspace, ws_bytes, need)) return st;
    if (zero_status st = check_disjoint({range_of(dst, dst_elems, esize(dst_dt), "dst"),
                                         range_of(workspace, (int64_t)need, 1, "workspace")}, {rz, rx}))
      return st;
    if (out == 0 || (accumulate && n == 0)) return ok();

    const WeightShape s = weight_shape(*p, weight, in_features, out, n, rank);
    WeightGradArgs a;
    memset(&a, 0, sizeof a);
    const Pick& c = s.c;
    a.dst_dt = dst_dt;
    a.accumulate = accumulate;
    a.scale = (float)scale;
    a.row0 = (int32_t)s.row0;
    a.lo = s.lo;
    a.hi = s.hi;
    if (s.rows > 0) a.dst = (char*)dst + s.at * esize(dst_dt);
    a.p.a = (const char*)dz + s.row0 * 2;
    a.p.b = x;
    a.p.lda = n > 1 ? dz_stride : round_up(out, 2);
    a.p.ldb = n > 1 ? x_stride : round_up(in_features, 2);
    lay_out(a.p, s.rows, in_features, n, c, workspace);
    if (bias >= 0) {
      int64_t lo, hi, at;
      part_of_tensor(*p, bias, rank, lo, hi, at);
      if (lo < hi) {
        a.bias_dst = (char*)dst + at * esize(dst_dt);
        a.bias_part = (float*)((char*)workspace + s.part);
        a.b_lo = (int32_t)lo;
        a.b_hi = (int32_t)hi;
        const int64_t chunk = bias_chunk(n, out);
        a.chunk_rows = (int32_t)chunk;
        a.chunks = (int32_t)std::max<int64_t>(1, ceil_div(n, chunk));
        a.col_blocks = (int32_t)ceil_div(hi - lo, kBiasCols);
        const int64_t bias_blocks = (int64_t)a.chunks * a.col_blocks;
        if (zero_status st = check_grid(bias_blocks, kTileThreads[c.tile])) return st;
        a.bias_blocks = (int32_t)bias_blocks;
      }
    }
    const int64_t blocks = a.bias_blocks + blocks_of(c);
    if (blocks == 0) return ok();
    a.join_blocks = (int32_t)std::min<int64_t>(INT32_MAX, joins_of(c));
    const int64_t joins = a.join_blocks + (a.bias_blocks && a.chunks > 1 ? ceil_div(a.b_hi - a.b_lo, kJoinThreads) : 0);
    if (zero_status st = check_grid(blocks, kTileThreads[c.tile])) return st;
    if (zero_status st = check_grid(joins, kJoinThreads)) return st;
    // The bias is summed from dz itself.
    a.dz = a.p.a;
    a.dz_stride = a.p.lda;
    if (zero_status st = make_copies(a.p, s.copies, n, s.rows, n, in_features, workspace, s.part + s.bias_part, stream)) return st;
    const bool direct = direct_m(a.p.a, a.p.lda, s.copies.a ? s.copies.lda : s.rows) && direct_m(a.p.b, a.p.ldb, s.copies.b ? s.copies.ldb : in_features);
    if (const int err = launch_weight_grad(a, dt, c.tile, direct, blocks, stream)) return hip_fail(err);
    if (joins == 0) return ok();
    return launched(launch_weight_grad_join(a, joins, stream));
  });
}

zero_status zero_activation_grad(const void* dy, const void* pre, void* dz, int64_t n, zero_dtype dt, zero_act act, void* stream) {
  return guarded("zero_activation_grad", [&]() -> zero_status {
    if (zero_status st = check_16(dt, "the elements")) return st;
    if (zero_status st = check_act(act)) return st;
    if (n < 0 || n > kMaxElems) return fail(ZERO_EINVAL, "n = %lld is out of range", (long long)n);
    if (zero_status st = check_buffer(dy, n, 2, "dy")) return st;
    if (zero_status st = check_buffer(pre, n, 2, "pre")) return st;
    if (zero_status st = check_buffer(dz, n, 2, "dz")) return st;
    const Range rz = range_of(dz, n, 2, "dz");
    std::vector<Range> reads = {range_of(pre, n, 2, "pre")};
    if (dz != dy) reads.push_back(range_of(dy, n, 2, "dy"));
    if (zero_status st = check_disjoint({rz}, reads)) return st;
    const int64_t per = (int64_t)kActThreads * kActVec, part = most_blocks(kActThreads) * per;
    for (int64_t i = 0; i < n; i += part) {
      ActGradArgs a;
      memset(&a, 0, sizeof a);
      a.dy = (const char*)dy + i * 2;
      a.pre = (const char*)pre + i * 2;
      a.dz = (char*)dz + i * 2;
      a.n = std::min(part, n - i);
      a.act = act;
      if (const int err = launch_act_grad(a, dt, ceil_div(a.n, per), stream)) return hip_fail(err);
    }
    return ok();
  });
}

size_t zero_orthogonalize_workspace_bytes(zero_plan_t p, const zero_matrix* matrices, int32_t n_matrices) {
  size_t need = 0;
  guarded("zero_orthogonalize_workspace_bytes", [&]() -> zero_status {
    std::vector<Group> groups;
    if (zero_status st = collect(p, matrices, n_matrices, groups)) return st;
    need = (size_t)ortho_bytes(groups);
    return ok();
  });
  return need;
}

zero_status zero_orthogonalize(zero_plan_t p, const zero_matrix* matrices, int32_t n_matrices, const zero_newton_schulz* poly,
                               const void* src, zero_dtype src_dt, void* dst, zero_dtype dst_dt, void* workspace,
                               size_t ws_bytes, void* stream) {
  return guarded("zero_orthogonalize", [&]() -> zero_status {
    std::vector<Group> groups;
    if (zero_status st = collect(p, matrices, n_matrices, groups)) return st;
    const zero_newton_schulz q = poly ? *poly : kDefaultPoly;
    if (q.steps < 1 || q.steps > 32) return fail(ZERO_EINVAL, "steps must lie in [1, 32] (got %d)", q.steps);
    for (double v : {q.a, q.b, q.c})
      if (!(std::fabs(v) <= 1000.0)) return fail(ZERO_EINVAL, "coefficient %g exceeds 1000", v);
    if (!(q.eps > 0.0 && q.eps <= 1e30)) return fail(ZERO_EINVAL, "eps must lie in (0, 1e30] (got %g)", q.eps);
    if (poly)
      if (zero_status st = check_growth(q)) return st;
    if (zero_status st = check_16(src_dt, "the matrices")) return st;
    if (zero_status st = check_16(dst_dt, "the results")) return st;
    if (zero_status st = check_buffer(src, p->psi_pad, 2, "src")) return st;
    if (zero_status st = check_buffer(dst, p->psi_pad, 2, "dst")) return st;
    const size_t need = (size_t)ortho_bytes(groups);
    if (zero_status st = check_workspace(workspace, ws_bytes, need)) return st;
    if (need && !aligned(workspace, 256)) return fail(ZERO_EINVAL, "workspace is not 256-byte aligned");
    std::vector<Range> writes = {range_of(workspace, (int64_t)need, 1, "workspace")};
    if (dst == src && dst_dt != src_dt) return fail(ZERO_EINVAL, "dst is src with another type");
    if (dst != src) writes.push_back(range_of(dst, p->psi_pad, 2, "dst"));
    if (zero_status st = check_disjoint(writes, {range_of(src, p->psi_pad, 2, "src")})) return st;
    for (const Group& g : groups) {
      const int64_t count = (int64_t)g.off.size();
      if (count == 0) continue;
      if (is_small(g.rows, g.cols)) {
        for (int64_t i = 0; i < count; i += kMaxBatch)
          if (zero_status st = ortho_small(g, i, std::min<int64_t>(kMaxBatch, count - i), q, src, src_dt, dst, dst_dt, stream)) return st;
        continue;
      }
      const bool thin = is_thin(g.rows, g.cols) && may_be_thin(q);
      const int64_t batch = batch_of(thin, g.rows, g.cols, count);
      const OrthoSpace s = space_of(thin, g.rows, g.cols, batch);      // a smaller last batch takes the same shapes
      const auto run = thin ? ortho_thin : ortho_batch;
      for (int64_t i = 0; i < count; i += batch)
        if (zero_status st = run(g, s, i, std::min(batch, count - i), q, src, src_dt, dst, dst_dt, (char*)workspace, stream))
          return st;
    }
    return ok();
  });
}

}  // extern "C"
