// zero_ops_api.cpp -- host side of the vocabulary operators: argument checks,
// launch shapes and the extern "C" entry points declared in include/zero.h.
// As in zero_api.cpp, nothing allocates device memory and every table travels
// in the kernel arguments.
#include <limits.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "zero.h"
#include "zero_host.h"
#include "zero_internal.h"
#include "zero_ops.h"

using namespace zk::host;
using namespace zk::ops;

namespace {

constexpr int64_t kMaxRows = INT32_MAX - 1;
constexpr int64_t kMaxHidden = int64_t(1) << 24;
constexpr int64_t kMaxTokens = int64_t(1) << 30;
constexpr int64_t kMaxVocab = int64_t(1) << 30;
constexpr int64_t kInfinityCache = int64_t(256) << 20;   // memory-side cache of MI355X
constexpr int64_t kMaxElems = int64_t(1) << 59;   // of one buffer: byte offsets stay in int64

bool valid_it(int it) { return it == ZERO_I32 || it == ZERO_I64; }
int isize(int it) { return it == ZERO_I64 ? 8 : 4; }

uint64_t mix64(uint64_t z) {
  z = (z ^ (z >> 30)) * kMix1;
  z = (z ^ (z >> 27)) * kMix2;
  return z ^ (z >> 31);
}

// Elements spanned by n rows of `width`, `stride` apart; -1 if too many.
int64_t span_of(int64_t n, int64_t stride, int64_t width) {
  if (n == 0 || width == 0) return 0;
  int64_t s;
  if (__builtin_mul_overflow(n - 1, stride, &s) || s > kMaxElems || width > kMaxElems - s) return -1;
  return s + width;
}

zero_status check_buffer(const void* p, int64_t elems, int es, const char* what) {
  if (!p && elems > 0) return fail(ZERO_EINVAL, "%s is NULL", what);
  if (!aligned(p, es)) return fail(ZERO_EINVAL, "%s is not element aligned", what);
  return ok();
}

zero_status check_workspace(const void* ws, size_t bytes, size_t need) {
  if (need == 0) return ok();
  if (!ws) return fail(ZERO_EINVAL, "workspace is NULL, %zu bytes are needed", need);
  if (bytes < need) return fail(ZERO_EINVAL, "workspace holds %zu bytes, %zu are needed", bytes, need);
  if (!aligned(ws, 16)) return fail(ZERO_EINVAL, "workspace is not 16-byte aligned");
  return ok();
}

// No written range may overlap another written one or a read one.
zero_status check_disjoint(const std::vector<Range>& writes, const std::vector<Range>& reads) {
  for (size_t i = 0; i < writes.size(); ++i) {
    for (size_t j = i + 1; j < writes.size(); ++j)
      if (overlap(writes[i], writes[j])) return fail(ZERO_EINVAL, "%s overlaps %s", writes[i].what, writes[j].what);
    for (const Range& r : reads)
      if (overlap(writes[i], r)) return fail(ZERO_EINVAL, "%s overlaps %s", writes[i].what, r.what);
  }
  return ok();
}

// A dropout's kernel arguments and the factor of the elements it keeps.
zero_status make_drop(const zero_drop* d, int64_t elems, DropArgs& out, double& keep) {
  memset(&out, 0, sizeof out);
  keep = 1.0;
  if (!d) return ok();
  if (!(d->p >= 0.0 && d->p <= 1.0)) return fail(ZERO_EINVAL, "dropout p must lie in [0, 1] (got %g)", d->p);
  if (d->first < 0 || d->first > INT64_MAX / 2 - elems)
    return fail(ZERO_EINVAL, "dropout position %lld is out of range", (long long)d->first);
  if (!aligned(d->step_dev, 8)) return fail(ZERO_EINVAL, "step_dev is not 8-byte aligned");
  out.cut = (uint32_t)std::nearbyint(d->p * 65536.0);
  out.first = d->first;
  out.step_dev = d->step_dev;
  out.site_key = mix64((d->seed ^ d->site) + kGamma);
  out.key = mix64((out.site_key ^ d->step) + kGamma);
  keep = out.cut < 65536 ? 65536.0 / (65536.0 - out.cut) : 0.0;
  return ok();
}

// The table: a tensor of the plan seen as rows of `hidden` elements.
zero_status table_of(zero_plan_t p, int32_t tensor, int64_t hidden, int64_t& rows) {
  if (check_plan(p)) return ZERO_EINVAL;
  if (tensor < 0 || tensor >= (int32_t)p->t_numel.size())
    return fail(ZERO_EINVAL, "tensor %d out of range", tensor);
  if (hidden < 1) return fail(ZERO_EINVAL, "hidden must be >= 1 (got %lld)", (long long)hidden);
  if (hidden > kMaxHidden) return fail(ZERO_EUNSUPPORTED, "hidden %lld exceeds %lld", (long long)hidden, (long long)kMaxHidden);
  if (p->t_numel[tensor] % hidden)
    return fail(ZERO_EINVAL, "tensor %d holds %lld elements, no multiple of hidden = %lld", tensor,
                (long long)p->t_numel[tensor], (long long)hidden);
  rows = p->t_numel[tensor] / hidden;
  if (rows > kMaxRows) return fail(ZERO_EUNSUPPORTED, "%lld rows exceed %lld", (long long)rows, (long long)kMaxRows);
  return ok();
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

zero_status check_blocks(int64_t blocks, int threads) {
  if (blocks > most_blocks(threads))
    return fail(ZERO_EUNSUPPORTED, "the call needs %lld workgroups of %d, one launch takes %lld", (long long)blocks, threads,
                (long long)most_blocks(threads));
  return ok();
}

// Size of the equal parts of n > 0 things of which one launch takes `most`.
int64_t part_of(int64_t n, int64_t most) { return ceil_div(n, ceil_div(n, most)); }

// ---------------------------------------------------------------------------
// Launch shapes
// ---------------------------------------------------------------------------

struct SortShape {
  bool small;           // ranked by counting
  int passes, bits;
  int64_t tile, blocks, tiles_per_block;
  size_t bytes;
};

SortShape sort_shape(int64_t n, int64_t rows) {
  SortShape s;
  memset(&s, 0, sizeof s);
  s.small = n <= kSmallSort && rows < (int64_t(1) << (32 - kSmallSortPosBits)) - 1;
  if (s.small || n == 0) return s;
  int key_bits = 1;
  while ((rows >> key_bits) != 0) ++key_bits;   // tokens are 0..rows
  s.passes = (int)ceil_div(key_bits, kDigitBits);
  s.bits = (int)ceil_div(key_bits, s.passes);
  s.tile = kSortThreads * (n <= kSortFew ? kSortKeysFew : kSortKeysMany);
  const int64_t tiles = ceil_div(n, s.tile);
  s.tiles_per_block = ceil_div(tiles, std::min<int64_t>(tiles, kSortBlocks));
  s.blocks = ceil_div(tiles, s.tiles_per_block);
  s.bytes = (size_t)s.blocks * kBins * 4 + (s.passes > 1 ? (size_t)n * 8 : 0);
  return s;
}

// Positions per chunk, from n and hidden alone: a run is summed chunk by chunk,
// so that an owner's slice holds the bits of the whole buffer only if it is cut
// alike.  As many as leave the GPU about 4096 waves, from 4 to 32, and 64 where
// that still leaves 32768 waves.  Longer chunks write fewer partial rows (the
// whole buffer of 32768 x 768: 47 us at 24, 54 at 8; of 2^20 x 768: 410 at 64,
// 427 at 32), shorter ones have fewer rows in a row in one wave (an eighth of
// 65536 x 2048: 59 us at 64, 48 at 32; the whole: 127 and 131).
int64_t grad_chunk(int64_t n, int64_t hidden) {
  const double tiles = (double)ceil_div(hidden, 256);
  const int64_t want = (int64_t)((double)n * tiles / 4096.0 + 3.0) / 4 * 4;
  return want >= 512 ? 64 : std::min<int64_t>(32, std::max<int64_t>(4, want));
}

// Waves that share a chunk's runs, where a slice leaves the GPU few: none with
// fewer than 8 positions.  An eighth of 65536 x 2048 in 47.8, 44.5 and 49.5 us
// at 1, 2 and 4, of 8192 x 8192 in 41.7, 37.3 and 40.2; a 64th of 65536 x 768 in
// 39.9, 35.1 and 32.9; half of 65536 x 2048 in 75, 81 and 86.
int32_t grad_parts(int64_t n, int64_t hidden, int64_t chunk, double share) {
  const double waves = (double)n * share * (double)ceil_div(hidden, 256) / (double)chunk;
  const int64_t parts = waves > 2048 ? 1 : waves > 256 ? 2 : 4;
  return (int32_t)std::max<int64_t>(1, std::min(parts, chunk / 8));
}

// Workgroups per row: one where the rows fill the GPU, else enough for about
// 1024, each with 16384 elements or more (two rows of 131072 in 7.2 us; 7.9 at
// 8192, 10.2 at 4096, for the pieces that the join then reads).
int64_t logp_splits(int64_t n, int64_t vocab) {
  if (n <= 0 || n >= 1024) return 1;
  return std::max<int64_t>(1, std::min<int64_t>(ceil_div(1024, n), vocab / 16384));
}

int64_t dlogits_splits(int64_t vocab) { return std::max<int64_t>(1, ceil_div(vocab, kDlogitsPiece)); }

zero_status check_logits(const void* logits, zero_dtype dt, int64_t n, int64_t vocab, int64_t stride,
                         const void* labels, zero_itype label_it, int64_t& span) {
  if (!valid_dt(dt)) return fail(ZERO_EINVAL, "unknown dtype %d", (int)dt);
  if (!valid_it(label_it)) return fail(ZERO_EINVAL, "unknown label type %d", (int)label_it);
  if (n < 0) return fail(ZERO_EINVAL, "n must be >= 0 (got %lld)", (long long)n);
  if (vocab < 1) return fail(ZERO_EINVAL, "vocab must be >= 1 (got %lld)", (long long)vocab);
  if (n > INT32_MAX) return fail(ZERO_EUNSUPPORTED, "n = %lld exceeds %d", (long long)n, INT32_MAX);
  if (vocab > kMaxVocab) return fail(ZERO_EUNSUPPORTED, "vocab %lld exceeds %lld", (long long)vocab, (long long)kMaxVocab);
  if (stride < vocab) return fail(ZERO_EINVAL, "stride %lld is shorter than a row of %lld", (long long)stride, (long long)vocab);
  span = span_of(n, stride, vocab);
  if (span < 0) return fail(ZERO_EINVAL, "the logits' extent overflows");
  if (zero_status st = check_buffer(logits, span, esize(dt), "logits")) return st;
  return check_buffer(labels, n, isize(label_it), "labels");
}

template <typename F>
zero_status guarded(const char* name, F f) {
  try {
    return f();
  } catch (const std::bad_alloc&) {
    return fail(ZERO_ENOMEM, "host allocation failed");
  } catch (...) {
    return fail(ZERO_EINVAL, "unexpected failure in %s", name);
  }
}

zero_status launched(int err) { return err ? hip_fail(err) : ok(); }

}  // namespace

extern "C" {

zero_status zero_embed(zero_plan_t p, int32_t tensor, int64_t hidden, const void* params, zero_dtype param_dt,
                       const void* tokens, zero_itype token_it, int64_t n, double scale, const zero_drop* drop,
                       void* out, zero_dtype out_dt, int64_t out_stride, void* stream) {
  return guarded("zero_embed", [&]() -> zero_status {
    int64_t rows = 0;
    if (zero_status st = table_of(p, tensor, hidden, rows)) return st;
    if (!valid_dt(param_dt)) return fail(ZERO_EINVAL, "unknown dtype %d", (int)param_dt);
    if (!valid_dt(out_dt)) return fail(ZERO_EINVAL, "unknown dtype %d", (int)out_dt);
    if (!valid_it(token_it)) return fail(ZERO_EINVAL, "unknown token type %d", (int)token_it);
    if (n < 0) return fail(ZERO_EINVAL, "n must be >= 0 (got %lld)", (long long)n);
    if (out_stride < hidden)
      return fail(ZERO_EINVAL, "out_stride %lld is shorter than a row of %lld", (long long)out_stride, (long long)hidden);
    const int64_t span = span_of(n, out_stride, hidden);
    if (span < 0) return fail(ZERO_EINVAL, "the output's extent overflows");
    if (zero_status st = check_buffer(params, p->psi_pad, esize(param_dt), "params")) return st;
    if (zero_status st = check_buffer(tokens, n, isize(token_it), "tokens")) return st;
    if (zero_status st = check_buffer(out, span, esize(out_dt), "out")) return st;
    EmbedArgs a;
    memset(&a, 0, sizeof a);
    double keep;
    if (zero_status st = make_drop(drop, span, a.drop, keep)) return st;
    if (!std::isfinite((float)(scale * keep))) return fail(ZERO_EINVAL, "scale %g is beyond fp32", scale);
    if (zero_status st = check_disjoint({range_of(out, span, esize(out_dt), "out")},
                                        {range_of(params, p->psi_pad, esize(param_dt), "params"),
                                         range_of(tokens, n, isize(token_it), "tokens")}))
      return st;
    if (n == 0) return ok();
    const int vec = vec_of(param_dt, out_dt);
    const bool wide = hidden >= vec;
    a.table = (const char*)params + p->t_off[tensor] * esize(param_dt);
    a.out_stride = out_stride;
    a.rows = (int32_t)rows;
    a.hidden = (int32_t)hidden;
    a.upr = (int32_t)(wide ? ceil_div(hidden, vec) : hidden);
    a.magic = a.upr > 1 ? (uint32_t)((uint64_t(1) << 32) / a.upr + 1) : 0;
    a.tok64 = token_it == ZERO_I64;
    a.f = (float)(scale * keep);
    const int64_t units = (int64_t)kEmbedThreads * kEmbedUnroll, part = part_of(n, most_blocks(kEmbedThreads) * units / a.upr);
    const int64_t first = a.drop.first;
    for (int64_t r = 0; r < n; r += part) {
      a.n = std::min(part, n - r);
      a.tokens = (const char*)tokens + r * isize(token_it);
      a.out = (char*)out + r * out_stride * esize(out_dt);
      a.drop.first = first + r * hidden;
      if (const int err = launch_embed(a, param_dt, out_dt, wide, ceil_div(a.n * a.upr, units), stream)) return hip_fail(err);
    }
    return ok();
  });
}

size_t zero_token_order_workspace_bytes(int64_t n, int64_t rows) {
  if (n < 0 || n > kMaxTokens || rows < 0 || rows > kMaxRows) return 0;
  return sort_shape(n, rows).bytes;
}

zero_status zero_token_order(const void* tokens, zero_itype token_it, int64_t n, int64_t rows, int32_t* sorted,
                             int32_t* order, void* workspace, size_t ws_bytes, void* stream) {
  return guarded("zero_token_order", [&]() -> zero_status {
    if (!valid_it(token_it)) return fail(ZERO_EINVAL, "unknown token type %d", (int)token_it);
    if (n < 0) return fail(ZERO_EINVAL, "n must be >= 0 (got %lld)", (long long)n);
    if (rows < 0) return fail(ZERO_EINVAL, "rows must be >= 0 (got %lld)", (long long)rows);
    if (n > kMaxTokens) return fail(ZERO_EUNSUPPORTED, "n = %lld exceeds %lld", (long long)n, (long long)kMaxTokens);
    if (rows > kMaxRows) return fail(ZERO_EUNSUPPORTED, "%lld rows exceed %lld", (long long)rows, (long long)kMaxRows);
    if (zero_status st = check_buffer(tokens, n, isize(token_it), "tokens")) return st;
    if (zero_status st = check_buffer(sorted, n, 4, "sorted")) return st;
    if (zero_status st = check_buffer(order, n, 4, "order")) return st;
    const SortShape s = sort_shape(n, rows);
    if (zero_status st = check_workspace(workspace, ws_bytes, s.bytes)) return st;
    if (zero_status st = check_disjoint({range_of(sorted, n, 4, "sorted"), range_of(order, n, 4, "order"),
                                         range_of(workspace, (int64_t)s.bytes, 1, "workspace")},
                                        {range_of(tokens, n, isize(token_it), "tokens")}))
      return st;
    if (n == 0) return ok();
    if (s.small) {
      RankArgs a{tokens, sorted, order, (int32_t)n, (int32_t)rows, token_it == ZERO_I64};
      return launched(launch_rank(a, ceil_div(n, kRankItems), stream));
    }
    uint32_t* hist = (uint32_t*)workspace;
    int32_t* ws_key = (int32_t*)((char*)workspace + (size_t)s.blocks * kBins * 4);
    int32_t* ws_pos = ws_key + n;
    RadixArgs a;
    memset(&a, 0, sizeof a);
    a.tokens = tokens;
    a.hist = hist;
    a.n = n;
    a.rows = (int32_t)rows;
    a.tok64 = token_it == ZERO_I64;
    a.bits = s.bits;
    a.n_blocks = (int32_t)s.blocks;
    a.tile = (int32_t)s.tile;
    a.tiles_per_block = s.tiles_per_block;
    for (int pass = 0; pass < s.passes; ++pass) {   // the last pass writes the outputs
      const bool to_out = (s.passes - 1 - pass) % 2 == 0;
      a.first = pass == 0;
      a.shift = pass * s.bits;
      a.key_in = to_out ? ws_key : sorted;
      a.pos_in = to_out ? ws_pos : order;
      a.key_out = to_out ? sorted : ws_key;
      a.pos_out = to_out ? order : ws_pos;
      if (const int err = launch_radix(a, stream)) return hip_fail(err);
    }
    return ok();
  });
}

size_t zero_embed_grad_workspace_bytes(int64_t n, int64_t hidden) {
  if (n <= 0 || n > kMaxTokens || hidden < 1 || hidden > kMaxHidden) return 0;
  return (size_t)(2 * ceil_div(n, grad_chunk(n, hidden))) * (size_t)hidden * 4;
}

zero_status zero_embed_grad(zero_plan_t p, int32_t tensor, int64_t hidden, const int32_t* sorted,
                            const int32_t* order, int64_t n, const void* dy, zero_dtype dy_dt, int64_t dy_stride,
                            double scale, const zero_drop* drop, void* dst, zero_dtype dst_dt, int32_t rank,
                            int32_t accumulate, void* workspace, size_t ws_bytes, void* stream) {
  return guarded("zero_embed_grad", [&]() -> zero_status {
    int64_t rows = 0;
    if (zero_status st = table_of(p, tensor, hidden, rows)) return st;
    if (!valid_dt(dy_dt)) return fail(ZERO_EINVAL, "unknown dtype %d", (int)dy_dt);
    if (!valid_dt(dst_dt)) return fail(ZERO_EINVAL, "unknown dtype %d", (int)dst_dt);
    if (n < 0) return fail(ZERO_EINVAL, "n must be >= 0 (got %lld)", (long long)n);
    if (n > kMaxTokens) return fail(ZERO_EUNSUPPORTED, "n = %lld exceeds %lld", (long long)n, (long long)kMaxTokens);
    if (rank >= p->n_d) return fail(ZERO_EINVAL, "rank %d outside [0, %d)", rank, p->n_d);
    if (accumulate != 0 && accumulate != 1) return fail(ZERO_EINVAL, "accumulate must be 0 or 1 (got %d)", accumulate);
    if (dy_stride < hidden)
      return fail(ZERO_EINVAL, "dy_stride %lld is shorter than a row of %lld", (long long)dy_stride, (long long)hidden);
    const int64_t span = span_of(n, dy_stride, hidden);
    if (span < 0) return fail(ZERO_EINVAL, "the extent of dy overflows");
    const int64_t dst_elems = rank < 0 ? p->psi_pad : p->shard_total;
    if (zero_status st = check_buffer(sorted, n, 4, "sorted")) return st;
    if (zero_status st = check_buffer(order, n, 4, "order")) return st;
    if (zero_status st = check_buffer(dy, span, esize(dy_dt), "dy")) return st;
    if (zero_status st = check_buffer(dst, dst_elems, esize(dst_dt), "dst")) return st;
    const size_t need = zero_embed_grad_workspace_bytes(n, hidden);
    if (zero_status st = check_workspace(workspace, ws_bytes, need)) return st;
    GradArgs a;
    memset(&a, 0, sizeof a);
    double keep;
    if (zero_status st = make_drop(drop, span, a.drop, keep)) return st;
    if (!std::isfinite((float)(scale * keep))) return fail(ZERO_EINVAL, "scale %g is beyond fp32", scale);
    if (zero_status st = check_disjoint({range_of(dst, dst_elems, esize(dst_dt), "dst"),
                                         range_of(workspace, (int64_t)need, 1, "workspace")},
                                        {range_of(sorted, n, 4, "sorted"), range_of(order, n, 4, "order"),
                                         range_of(dy, span, esize(dy_dt), "dy")}))
      return st;

    // The part of the tensor that is written, and where it stands in dst.
    const int64_t off = p->t_off[tensor], numel = p->t_numel[tensor];
    int64_t dst_off = off;
    a.hi = numel;
    if (rank >= 0) {
      const auto& b = p->buckets[p->t_bucket[tensor]];
      const int64_t own = b.flat_off + (int64_t)rank * b.shard_numel;
      a.lo = std::max<int64_t>(0, own - off);
      a.hi = std::min<int64_t>(numel, own + b.shard_numel - off);
      dst_off = b.shard_off + (off + a.lo - own);
    }
    if (a.lo >= a.hi || (accumulate && n == 0)) return ok();
    a.sorted = sorted;
    a.order = order;
    a.dy = dy;
    a.dst = (char*)dst + dst_off * esize(dst_dt);
    a.part = (float*)workspace;
    a.n = n;
    a.dy_stride = dy_stride;
    a.row_lo = (int32_t)(a.lo / hidden);
    a.row_hi = (int32_t)((a.hi - 1) / hidden + 1);
    a.rows = (int32_t)rows;
    a.hidden = (int32_t)hidden;
    a.accumulate = accumulate;
    a.f = (float)(scale * keep);
    // Eight columns a lane, unless four leave fewer lanes of the last tile idle
    // (calls of 2^20 x 768: 408 us with four, 428 with eight; of 65536 x 8192: 403
    // with eight, 430 with four).
    int vec = hidden < 4 ? 1 : 4;
    if (vec_of(dy_dt, dst_dt) == 8 && hidden >= 8 && ceil_div(hidden, 512) * 2 == ceil_div(hidden, 256)) vec = 8;
    a.chunk = (int32_t)grad_chunk(n, hidden);
    a.n_chunks = (int32_t)ceil_div(n, a.chunk);
    a.parts = grad_parts(n, hidden, a.chunk, (double)(a.hi - a.lo) / (double)numel);
    a.tiles = (int32_t)ceil_div(hidden, 64 * vec) * a.parts;
    // Zero rows: 128 KiB a workgroup, down to 8 KiB where that leaves fewer than
    // about 2048 workgroups.
    const int64_t row_bytes = hidden * esize(dst_dt);
    const int64_t fill_bytes = std::max<int64_t>(8192, std::min<int64_t>(131072, (a.row_hi - a.row_lo) * row_bytes / 2048));
    a.fill_rows = (int32_t)std::max<int64_t>(1, std::min<int64_t>(1024, fill_bytes / row_bytes));
    a.chunk_blocks = ceil_div(a.n_chunks, kGradChunks) * a.tiles;
    a.stream_dy = n * hidden * esize(dy_dt) > kInfinityCache;
    const int64_t blocks = a.chunk_blocks + (accumulate ? 0 : ceil_div(a.row_hi - a.row_lo, a.fill_rows));
    a.join_tiles = (int32_t)ceil_div(hidden, hidden >= 4 ? 256 : 64);
    const int64_t joins = ceil_div(a.n_chunks, kJoinChunks) * a.join_tiles;
    if (zero_status st = check_blocks(blocks, kGradThreads)) return st;
    if (zero_status st = check_blocks(joins, kJoinThreads)) return st;
    if (const int err = launch_grad(a, dy_dt, dst_dt, vec, blocks, stream)) return hip_fail(err);
    if (a.n_chunks < 2) return ok();   // no run crosses a boundary
    return launched(launch_grad_join(a, dst_dt, hidden >= 4, joins, stream));
  });
}

zero_status zero_dropout(const void* x, const void* residual, void* out, int64_t n, zero_dtype dt,
                         const zero_drop* drop, void* stream) {
  return guarded("zero_dropout", [&]() -> zero_status {
    if (!valid_dt(dt)) return fail(ZERO_EINVAL, "unknown dtype %d", (int)dt);
    if (!drop) return fail(ZERO_EINVAL, "drop is NULL");
    if (n < 0 || n > kMaxElems) return fail(ZERO_EINVAL, "n = %lld is out of range", (long long)n);
    if (zero_status st = check_buffer(x, n, esize(dt), "x")) return st;
    if (zero_status st = check_buffer(residual, 0, esize(dt), "residual")) return st;
    if (zero_status st = check_buffer(out, n, esize(dt), "out")) return st;
    DropoutArgs a;
    memset(&a, 0, sizeof a);
    double keep;
    if (zero_status st = make_drop(drop, n, a.drop, keep)) return st;
    const Range w = range_of(out, n, esize(dt), "out");
    if (out != x && overlap(w, range_of(x, n, esize(dt), "x"))) return fail(ZERO_EINVAL, "out overlaps x without being it");
    if (residual && out != residual && overlap(w, range_of(residual, n, esize(dt), "residual")))
      return fail(ZERO_EINVAL, "out overlaps the residual without being it");
    if (n == 0) return ok();
    a.f = (float)keep;
    const int64_t per = (int64_t)kDropoutThreads * vec_of(dt, dt), part = most_blocks(kDropoutThreads) * per;
    const int64_t first = a.drop.first;
    for (int64_t e = 0; e < n; e += part) {   // parts of whole workgroups keep the accesses' alignment
      a.n = std::min(part, n - e);
      a.x = (const char*)x + e * esize(dt);
      a.residual = residual ? (const char*)residual + e * esize(dt) : nullptr;
      a.out = (char*)out + e * esize(dt);
      a.drop.first = first + e;
      if (const int err = launch_dropout(a, dt, ceil_div(a.n, per), stream)) return hip_fail(err);
    }
    return ok();
  });
}

size_t zero_token_logp_workspace_bytes(int64_t n, int64_t vocab) {
  const int64_t splits = logp_splits(n, vocab);
  return splits > 1 ? (size_t)(n * splits) * 8 : 0;
}

zero_status zero_token_logp(const void* logits, zero_dtype dt, int64_t n, int64_t vocab, int64_t stride,
                            const void* labels, zero_itype label_it, float* logp, float* stats, void* workspace,
                            size_t ws_bytes, void* stream) {
  return guarded("zero_token_logp", [&]() -> zero_status {
    int64_t span = 0;
    if (zero_status st = check_logits(logits, dt, n, vocab, stride, labels, label_it, span)) return st;
    if (zero_status st = check_buffer(logp, n, 4, "logp")) return st;
    if (zero_status st = check_buffer(stats, 2 * n, 4, "stats")) return st;
    const size_t need = zero_token_logp_workspace_bytes(n, vocab);
    if (zero_status st = check_workspace(workspace, ws_bytes, need)) return st;
    if (zero_status st = check_disjoint({range_of(logp, n, 4, "logp"), range_of(stats, 2 * n, 4, "stats"),
                                         range_of(workspace, (int64_t)need, 1, "workspace")},
                                        {range_of(logits, span, esize(dt), "logits"),
                                         range_of(labels, n, isize(label_it), "labels")}))
      return st;
    if (n == 0) return ok();
    LogpArgs a;
    memset(&a, 0, sizeof a);
    a.part = (float*)workspace;
    a.stride = stride;
    a.vocab = (int32_t)vocab;
    a.lab64 = label_it == ZERO_I64;
    a.splits = (int32_t)logp_splits(n, vocab);   // 1 wherever the rows take several launches
    const int64_t cached_from = n - kCachedBytes / (vocab * esize(dt));
    const int64_t part = part_of(n, most_blocks(logp_threads(n, vocab)) / a.splits);
    for (int64_t r = 0; r < n; r += part) {
      a.n = std::min(part, n - r);
      a.logits = (const char*)logits + r * stride * esize(dt);
      a.labels = (const char*)labels + r * isize(label_it);
      a.logp = logp + r;
      a.stats = stats + 2 * r;
      a.cached_from = (int32_t)std::max<int64_t>(0, std::min(a.n, cached_from - r));
      if (const int err = launch_logp(a, dt, stream)) return hip_fail(err);
    }
    return a.splits > 1 ? launched(launch_logp_join(a, dt, stream)) : ok();
  });
}

zero_status zero_preference_loss(int64_t n_pairs, const void* offsets, zero_itype offset_it, int64_t n,
                                 const void* labels, zero_itype label_it, int64_t vocab, const float* logp,
                                 const float* ref_logp, double beta, double smoothing, double grad_scale,
                                 float* loss, float* pair_loss, float* rewards, float* coef, void* stream) {
  return guarded("zero_preference_loss", [&]() -> zero_status {
    if (!valid_it(offset_it)) return fail(ZERO_EINVAL, "unknown offset type %d", (int)offset_it);
    if (!valid_it(label_it)) return fail(ZERO_EINVAL, "unknown label type %d", (int)label_it);
    if (n_pairs < 0) return fail(ZERO_EINVAL, "n_pairs must be >= 0 (got %lld)", (long long)n_pairs);
    if (n < 0) return fail(ZERO_EINVAL, "n must be >= 0 (got %lld)", (long long)n);
    if (labels && vocab < 1) return fail(ZERO_EINVAL, "vocab must be >= 1 (got %lld)", (long long)vocab);
    if (!(smoothing >= 0.0 && smoothing <= 1.0)) return fail(ZERO_EINVAL, "smoothing must lie in [0, 1] (got %g)", smoothing);
    if (!std::isfinite(beta)) return fail(ZERO_EINVAL, "beta is not finite");
    if (!std::isfinite(grad_scale)) return fail(ZERO_EINVAL, "grad_scale is not finite");
    const double slope = n_pairs > 0 ? beta * grad_scale / (double)n_pairs : 0.0;
    if (!std::isfinite((float)slope)) return fail(ZERO_EINVAL, "beta * grad_scale / n_pairs = %g is beyond fp32", slope);
    if (n_pairs > (int64_t(1) << 29)) return fail(ZERO_EUNSUPPORTED, "n_pairs = %lld exceeds 2^29", (long long)n_pairs);
    if (n > INT32_MAX) return fail(ZERO_EUNSUPPORTED, "n = %lld exceeds %d", (long long)n, INT32_MAX);
    const int64_t n_off = n_pairs ? 2 * n_pairs + 1 : 0;
    if (zero_status st = check_buffer(offsets, n_off, isize(offset_it), "offsets")) return st;
    if (zero_status st = check_buffer(labels, 0, isize(label_it), "labels")) return st;
    if (zero_status st = check_buffer(logp, n, 4, "logp")) return st;
    if (zero_status st = check_buffer(ref_logp, 0, 4, "ref_logp")) return st;
    if (zero_status st = check_buffer(loss, 1, 4, "loss")) return st;
    if (zero_status st = check_buffer(pair_loss, n_pairs, 4, "pair_loss")) return st;
    if (zero_status st = check_buffer(rewards, 2 * n_pairs, 4, "rewards")) return st;
    if (zero_status st = check_buffer(coef, n, 4, "coef")) return st;
    std::vector<Range> reads = {range_of(offsets, n_off, isize(offset_it), "offsets"), range_of(logp, n, 4, "logp")};
    if (labels) reads.push_back(range_of(labels, n, isize(label_it), "labels"));
    if (ref_logp) reads.push_back(range_of(ref_logp, n, 4, "ref_logp"));
    if (zero_status st = check_disjoint({range_of(loss, 1, 4, "loss"), range_of(pair_loss, n_pairs, 4, "pair_loss"),
                                         range_of(rewards, 2 * n_pairs, 4, "rewards"), range_of(coef, n, 4, "coef")},
                                        reads))
      return st;
    PrefArgs a;
    memset(&a, 0, sizeof a);
    a.offsets = offsets;
    a.labels = labels;
    a.logp = logp;
    a.ref = ref_logp;
    a.loss = loss;
    a.pair_loss = pair_loss;
    a.rewards = rewards;
    a.coef = coef;
    a.n = n;
    a.n_pairs = n_pairs;
    a.vocab = vocab;
    a.beta = beta;
    a.smoothing = smoothing;
    a.slope = slope;
    a.off64 = offset_it == ZERO_I64;
    a.lab64 = label_it == ZERO_I64;
    // The launch of the last pairs also takes the rows in no sequence, and the mean.
    const int64_t most = most_blocks(kPrefThreads) - 1;
    do {
      a.pair_count = std::min(most, n_pairs - a.pair0);
      if (const int err = launch_preference(a, stream)) return hip_fail(err);
      a.pair0 += a.pair_count;
    } while (a.pair0 < n_pairs);
    return ok();
  });
}

zero_status zero_token_logp_grad(const void* logits, zero_dtype dt, int64_t n, int64_t vocab, int64_t stride,
                                 const void* labels, zero_itype label_it, const float* stats, const float* coef,
                                 void* dlogits, int64_t dl_stride, void* stream) {
  return guarded("zero_token_logp_grad", [&]() -> zero_status {
    int64_t span = 0;
    if (zero_status st = check_logits(logits, dt, n, vocab, stride, labels, label_it, span)) return st;
    if (dl_stride < vocab)
      return fail(ZERO_EINVAL, "dl_stride %lld is shorter than a row of %lld", (long long)dl_stride, (long long)vocab);
    const int64_t dspan = span_of(n, dl_stride, vocab);
    if (dspan < 0) return fail(ZERO_EINVAL, "the gradient's extent overflows");
    if (zero_status st = check_buffer(stats, 2 * n, 4, "stats")) return st;
    if (zero_status st = check_buffer(coef, n, 4, "coef")) return st;
    if (zero_status st = check_buffer(dlogits, dspan, esize(dt), "dlogits")) return st;
    std::vector<Range> reads = {range_of(labels, n, isize(label_it), "labels"), range_of(stats, 2 * n, 4, "stats"),
                                range_of(coef, n, 4, "coef")};
    if (dlogits != logits || dl_stride != stride) reads.push_back(range_of(logits, span, esize(dt), "logits"));
    if (zero_status st = check_disjoint({range_of(dlogits, dspan, esize(dt), "dlogits")}, reads)) return st;
    if (n == 0) return ok();
    LogpArgs a;
    memset(&a, 0, sizeof a);
    a.stride = stride;
    a.dl_stride = dl_stride;
    a.vocab = (int32_t)vocab;
    a.lab64 = label_it == ZERO_I64;
    a.splits = (int32_t)dlogits_splits(vocab);
    const int64_t part = part_of(n, most_blocks(kDlogitsThreads) / a.splits);
    for (int64_t end = n; end > 0; end -= part) {   // the last rows first, as in each launch
      const int64_t r = std::max<int64_t>(0, end - part);
      a.n = end - r;
      a.logits = (const char*)logits + r * stride * esize(dt);
      a.labels = (const char*)labels + r * isize(label_it);
      a.stats = const_cast<float*>(stats) + 2 * r;
      a.coef = coef + r;
      a.dlogits = (char*)dlogits + r * dl_stride * esize(dt);
      if (const int err = launch_dlogits(a, dt, stream)) return hip_fail(err);
    }
    return ok();
  });
}

}  // extern "C"
