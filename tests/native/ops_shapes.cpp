// Launch shapes of the vocabulary operators, checked on the CPU.
//
// zero_ops_api.cpp is compiled together with this file, which stands in for
// the kernel launchers: instead of launching, it checks that each launch
// covers its work and that every index the kernels form from its arguments
// lies inside the buffers and the workspace of the call.  Built with g++ under
// AddressSanitizer and UndefinedBehaviorSanitizer; no GPU is involved.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <cmath>
#include <random>
#include <vector>

#include "zero.h"
#include "zero_internal.h"
#include "zero_ops.h"

namespace {

int g_fail = 0;
#define EXPECT(c, ...)                         \
  do {                                         \
    if (!(c)) {                                \
      if (g_fail < 20) {                       \
        fprintf(stderr, "FAIL: " __VA_ARGS__); \
        fprintf(stderr, "\n");                 \
      }                                        \
      ++g_fail;                                \
    }                                          \
  } while (0)

constexpr uint64_t kSpan = 1ull << 57;
void* fake(int id) { return (void*)(uintptr_t)((uint64_t)(id + 1) * kSpan); }

// What the running call passed.
int64_t g_n, g_rows, g_hidden, g_ws;
int g_passes, g_launches;
const void *g_sorted, *g_order;

bool in_ws(const void* p, int64_t bytes) {
  const uint64_t lo = (uint64_t)(uintptr_t)fake(9), a = (uint64_t)(uintptr_t)p;
  return a >= lo && a + bytes <= lo + g_ws;
}

}  // namespace

namespace zk {
const char* hip_error_string(int) { return "stub"; }
int launch_step(const StepArgs&, int, int, int, int, bool, int, void*) { return 0; }
int launch_copy(const CopyArgs&, int, int, void*) { return 0; }
int launch_warm(const WarmArgs&, int, void*) { return 0; }
int resident_blocks(int, int, int, int, bool) { return 0; }
double wall_clock_hz() { return 0; }
double hbm_peak_bps() { return 0; }

namespace ops {

int launch_embed(const EmbedArgs& a, int tdt, int odt, bool vec, int64_t blocks, void*) {
  ++g_launches;
  const int n = vec ? vec_of(tdt, odt) : 1;
  EXPECT((int64_t)a.upr * n >= a.hidden && (int64_t)(a.upr - 1) * n < a.hidden, "upr %d of hidden %d", a.upr, a.hidden);
  EXPECT(a.hidden >= n, "access wider than a row");
  EXPECT(blocks * kEmbedThreads * kEmbedUnroll >= a.n * a.upr, "units not covered");
  // The division every thread makes, over its whole range.
  const uint32_t upr = (uint32_t)a.upr, top = upr + kEmbedThreads * kEmbedUnroll;
  for (uint32_t t = 0; t < top; t += top > 100000 ? 97 : 1) {
    const uint32_t r = upr > kEmbedThreads * kEmbedUnroll ? (t >= upr) : a.magic ? (uint32_t)(((uint64_t)t * a.magic) >> 32) : t;
    EXPECT(r == t / upr, "t %u upr %u: %u", t, upr, r);
  }
  return 0;
}

int launch_rank(const RankArgs& a, int64_t blocks, void*) {
  ++g_launches;
  EXPECT(a.n <= kSmallSort && blocks * kRankItems >= a.n, "rank: %d positions", a.n);
  EXPECT(((uint64_t)a.rows << kSmallSortPosBits | (kSmallSort - 1)) <= 0xffffffffull, "word overflows: rows %d", a.rows);
  return 0;
}

int launch_radix(const RadixArgs& a, void*) {
  ++g_launches;
  const int64_t per = a.tiles_per_block * a.tile;
  EXPECT(a.bits >= 1 && a.bits <= kDigitBits, "bits %d", a.bits);
  EXPECT(a.tile == kSortThreads * kSortKeysFew || a.tile == kSortThreads * kSortKeysMany, "tile %d", a.tile);
  EXPECT(a.n_blocks >= 1 && a.n_blocks <= kSortBlocks && a.n_blocks * per >= a.n && (a.n_blocks - 1) * per < a.n, "blocks");
  EXPECT(in_ws(a.hist, (int64_t)a.n_blocks * kBins * 4), "histogram outside the workspace");
  EXPECT(a.first == (g_passes == 0) && a.shift == g_passes * a.bits, "pass %d", g_passes);
  if (!a.first) EXPECT(a.key_in != a.key_out && a.pos_in != a.pos_out, "pass in place");
  for (const int32_t* p : {a.key_out, a.pos_out})
    EXPECT(p == g_sorted || p == g_order || in_ws(p, g_n * 4), "output of a pass");
  if (a.key_out != g_sorted) {
    EXPECT(in_ws(a.key_out, g_n * 4) && (const char*)a.key_out >= (const char*)a.hist + (int64_t)a.n_blocks * kBins * 4 &&
               (const char*)a.pos_out == (const char*)a.key_out + g_n * 4, "workspace layout");
  }
  ++g_passes;
  if (((int64_t)g_rows >> std::min(62, g_passes * a.bits)) == 0)
    EXPECT(a.key_out == g_sorted && a.pos_out == g_order, "the last pass writes the outputs");
  return 0;
}

int launch_grad(const GradArgs& a, int ydt, int gdt, int vec, int64_t blocks, void*) {
  ++g_launches;
  EXPECT(a.chunk >= 1 && a.chunk <= 64, "chunk %d", a.chunk);
  EXPECT((int64_t)a.n_chunks * a.chunk >= a.n && (a.n == 0 || (int64_t)(a.n_chunks - 1) * a.chunk < a.n), "chunks");
  EXPECT(a.n == 0 || in_ws(a.part, 2 * (int64_t)a.n_chunks * a.hidden * 4), "partial rows outside the workspace");
  EXPECT(vec == 1 || (vec == 4 && a.hidden >= 4) || (vec == 8 && a.hidden >= 8 && vec_of(ydt, gdt) == 8), "vec %d", vec);
  EXPECT((int64_t)a.tiles * 64 * vec >= a.hidden, "tiles");
  EXPECT(a.chunk_blocks == (a.n_chunks + kGradChunks - 1) / kGradChunks * (int64_t)a.tiles, "chunk blocks");
  EXPECT(a.fill_rows >= 1 && a.fill_rows <= 1024, "fill rows %d", a.fill_rows);
  EXPECT((int64_t)a.fill_rows * a.hidden < (int64_t(1) << 31), "fill units");
  EXPECT(a.lo >= 0 && a.lo < a.hi && a.hi <= g_rows * g_hidden, "range");
  EXPECT(a.row_lo == a.lo / a.hidden && a.row_hi == (a.hi + a.hidden - 1) / a.hidden && a.row_hi <= a.rows, "rows");
  const int64_t fill = blocks - a.chunk_blocks;
  EXPECT(a.accumulate ? fill == 0 : fill * a.fill_rows >= a.row_hi - a.row_lo, "zero rows not covered");
  return 0;
}

int launch_grad_join(const GradArgs& a, int, bool vec, int64_t blocks, void*) {
  ++g_launches;
  EXPECT((int64_t)a.join_tiles * (vec ? 256 : 64) >= a.hidden, "join tiles");
  EXPECT(blocks == (a.n_chunks + kJoinChunks - 1) / kJoinChunks * (int64_t)a.join_tiles, "join workgroups");
  EXPECT(a.n_chunks >= 2 && vec == (a.hidden >= 4), "join");
  return 0;
}

int launch_dropout(const DropoutArgs& a, int dt, int64_t blocks, void*) {
  ++g_launches;
  EXPECT(blocks * kDropoutThreads * vec_of(dt, dt) >= a.n, "dropout not covered");
  return 0;
}

int launch_logp(const LogpArgs& a, int, void*) {
  ++g_launches;
  EXPECT(a.splits >= 1 && (a.splits == 1 || in_ws(a.part, a.n * a.splits * 8)), "pieces outside the workspace");
  EXPECT(a.cached_from >= 0 && a.cached_from <= a.n, "cached_from");
  return 0;
}
int launch_logp_join(const LogpArgs& a, int, void*) {
  EXPECT(a.splits > 1, "join of one piece");
  return 0;
}
int launch_dlogits(const LogpArgs& a, int, void*) {
  ++g_launches;
  EXPECT((int64_t)a.splits * kDlogitsPiece >= a.vocab, "pieces");
  return 0;
}
int launch_preference(const PrefArgs&, void*) {
  ++g_launches;
  return 0;
}

}  // namespace ops
}  // namespace zk

int main() {
  std::mt19937_64 rng(7);
  auto log_size = [&](int64_t hi) {
    return (int64_t)std::exp(std::uniform_real_distribution<double>(0, std::log((double)hi + 1))(rng));
  };
  for (int trial = 0; trial < 4000; ++trial) {
    g_hidden = std::max<int64_t>(1, log_size(trial % 7 ? 20000 : 1 << 24));
    g_rows = std::min<int64_t>(log_size(3000000), (int64_t(1) << 36) / g_hidden);
    g_n = trial % 11 == 0 ? 0 : log_size(trial % 5 ? 300000 : int64_t(1) << 30);
    const int64_t before = trial % 3 ? (int64_t)(rng() % 5000) : 0;
    const int nd = 1 + (int)(rng() % 9), rank = (int)(rng() % (nd + 1)) - 1;
    const int64_t sizes[2] = {before, g_rows * g_hidden};
    zero_plan_t plan;
    if (zero_plan(sizes[0] + sizes[1], nd, sizes, 2, 0, 1 + (int)(rng() % 64), &plan) != ZERO_OK) return 2;
    const auto dt = [&]() { return (zero_dtype)(rng() % 3); };
    const zero_drop drop = {0.1, 1, 2, 3, nullptr, (int64_t)(rng() % 5)};
    const zero_drop* d = rng() % 2 ? &drop : nullptr;
    zero_status st = zero_embed(plan, 1, g_hidden, fake(0), dt(), fake(1), ZERO_I64, std::min<int64_t>(g_n, 1 << 20), 1.0, d,
                                fake(2), dt(), g_hidden + (int64_t)(rng() % 3), nullptr);
    EXPECT(st == ZERO_OK || st == ZERO_EUNSUPPORTED, "embed: %s", zero_last_error());
    g_ws = (int64_t)zero_token_order_workspace_bytes(g_n, g_rows);
    g_passes = 0;
    g_sorted = fake(3);
    g_order = fake(4);
    st = zero_token_order(fake(1), ZERO_I32, g_n, g_rows, (int32_t*)fake(3), (int32_t*)fake(4), fake(9), g_ws, nullptr);
    EXPECT(st == ZERO_OK, "order: %s", zero_last_error());
    g_ws = (int64_t)zero_embed_grad_workspace_bytes(g_n, g_hidden);
    st = zero_embed_grad(plan, 1, g_hidden, (int32_t*)fake(3), (int32_t*)fake(4), g_n, fake(5), dt(), g_hidden, 1.0, d,
                         fake(6), dt(), rank, (int)(rng() % 2), fake(9), g_ws, nullptr);
    EXPECT(st == ZERO_OK || st == ZERO_EUNSUPPORTED, "grad: %s", zero_last_error());
    if (g_n > 0 && g_ws > 16) {
      st = zero_embed_grad(plan, 1, g_hidden, (int32_t*)fake(3), (int32_t*)fake(4), g_n, fake(5), dt(), g_hidden, 1.0, d,
                           fake(6), dt(), -1, 0, fake(9), g_ws - 1, nullptr);
      EXPECT(st == ZERO_EINVAL, "a short workspace passed");
    }
    zero_plan_destroy(plan);
    const int64_t vocab = std::max<int64_t>(1, log_size(300000)), n = std::min<int64_t>(g_n, 100000);
    g_ws = (int64_t)zero_token_logp_workspace_bytes(n, vocab);
    const zero_dtype t = dt();
    st = zero_token_logp(fake(0), t, n, vocab, vocab, fake(1), ZERO_I64, (float*)fake(2), (float*)fake(3), fake(9), g_ws, nullptr);
    EXPECT(st == ZERO_OK, "logp: %s", zero_last_error());
    st = zero_token_logp_grad(fake(0), t, n, vocab, vocab, fake(1), ZERO_I64, (float*)fake(3), (float*)fake(4), fake(5),
                              vocab + 1, nullptr);
    EXPECT(st == ZERO_OK, "dlogits: %s", zero_last_error());
    st = zero_dropout(fake(0), nullptr, fake(1), g_n, t, &drop, nullptr);
    EXPECT(st == ZERO_OK, "dropout: %s", zero_last_error());
  }
  printf("%d launches, %d failures\n", g_launches, g_fail);
  return g_fail != 0;
}
