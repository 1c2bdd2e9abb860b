// Launches of the vocabulary operators at the limits of the documented sizes,
// checked on the CPU.
//
// As in ops_shapes.cpp, this file stands in for the kernel launchers.  A
// launch may have fewer than 2^32 work items, so a call whose work is more has
// to be cut into launches that cover it once, in its own order, each with the
// pointers and the mask position of its part.
#include <stdint.h>
#include <stdio.h>

#include <vector>

#include "zero.h"
#include "zero_internal.h"
#include "zero_ops.h"

namespace {

int g_fail = 0;
#define EXPECT(c, ...)                       \
  do {                                       \
    if (!(c)) {                              \
      if (g_fail < 20) {                     \
        fprintf(stderr, "FAIL: " __VA_ARGS__); \
        fprintf(stderr, "\n");               \
      }                                      \
      ++g_fail;                              \
    }                                        \
  } while (0)

constexpr uint64_t kSpan = 1ull << 57;
constexpr int kBuffers = 10;
void* fake(int id) { return (void*)(uintptr_t)((uint64_t)(id + 1) * kSpan); }
int64_t past(const void* p, int id, int64_t bytes) {   // index in buffer id
  const int64_t d = (int64_t)((uint64_t)(uintptr_t)p - (uint64_t)(uintptr_t)fake(id));
  EXPECT(d % bytes == 0, "address inside an element");
  return d / bytes;
}

int64_t g_done;       // rows, elements or pairs covered so far
int64_t g_left;       // backwards: what is still to come
int g_launches, g_means;
int64_t g_hidden, g_stride, g_first;

void grid(int64_t blocks, int threads, const char* what) {
  ++g_launches;
  EXPECT(blocks >= 1 && blocks * threads < (int64_t(1) << 32), "%s: %lld x %d work items", what, (long long)blocks, threads);
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

int launch_embed(const EmbedArgs& a, int, int, bool, int64_t blocks, void*) {
  grid(blocks, kEmbedThreads, "embed");
  EXPECT(past(a.tokens, 1, 4) == g_done && past(a.out, 2, 2) == g_done * g_stride, "embed's rows");
  EXPECT(a.drop.first == g_first + g_done * g_hidden, "embed's mask");
  EXPECT(blocks * kEmbedThreads * kEmbedUnroll >= a.n * a.upr, "units not covered");
  g_done += a.n;
  return 0;
}
int launch_rank(const RankArgs&, int64_t blocks, void*) {
  grid(blocks, kRankThreads, "rank");
  return 0;
}
int launch_radix(const RadixArgs& a, void*) {
  grid(a.n_blocks, kSortThreads, "radix");
  return 0;
}
int launch_grad(const GradArgs&, int, int, int, int64_t blocks, void*) {
  grid(blocks, kGradThreads, "grad");
  return 0;
}
int launch_grad_join(const GradArgs&, int, bool, int64_t blocks, void*) {
  grid(blocks, kJoinThreads, "join");
  return 0;
}
int launch_dropout(const DropoutArgs& a, int dt, int64_t blocks, void*) {
  grid(blocks, kDropoutThreads, "dropout");
  const int es = dt == ZERO_F32 ? 4 : 2;
  EXPECT(past(a.x, 0, es) == g_done && past(a.residual, 1, es) == g_done && past(a.out, 2, es) == g_done, "dropout's elements");
  EXPECT(a.drop.first == g_first + g_done, "dropout's mask");
  EXPECT(blocks * kDropoutThreads * vec_of(dt, dt) >= a.n, "dropout not covered");
  g_done += a.n;
  return 0;
}
int launch_logp(const LogpArgs& a, int, void*) {
  grid(a.n * a.splits, logp_threads(a.n, a.vocab), "logp");
  EXPECT(past(a.logits, 0, 2) == g_done * g_stride && past(a.labels, 1, 4) == g_done && past(a.logp, 2, 4) == g_done &&
             past(a.stats, 3, 4) == 2 * g_done, "logp's rows");
  EXPECT(a.cached_from >= 0 && a.cached_from <= a.n, "cached_from");
  g_done += a.n;
  return 0;
}
int launch_logp_join(const LogpArgs& a, int, void*) {
  grid((a.n + 63) / 64, 64, "logp join");
  return 0;
}
int launch_dlogits(const LogpArgs& a, int, void*) {
  grid(a.n * a.splits, kDlogitsThreads, "dlogits");
  g_left -= a.n;   // the last rows first
  EXPECT(past(a.logits, 0, 2) == g_left * g_stride && past(a.labels, 1, 4) == g_left && past(a.stats, 3, 4) == 2 * g_left &&
             past(a.coef, 4, 4) == g_left && past(a.dlogits, 5, 2) == g_left * (g_stride + 1), "dlogits' rows");
  return 0;
}
int launch_preference(const PrefArgs& a, void*) {
  const bool small = a.n_pairs <= kPrefSmallPairs && a.n <= kPrefSmallRows;
  EXPECT(a.pair0 == g_done, "pairs");
  g_done += a.pair_count;
  const bool last = g_done == a.n_pairs;
  grid(small ? 1 : a.pair_count + last, kPrefThreads, "preference");
  g_means += last;
  return 0;
}

}  // namespace ops
}  // namespace zk

using namespace zk::ops;

int main() {
  const int64_t big = int64_t(1) << 32;
  // Elements of one launch of each kind, and sizes around it and far beyond.
  for (const int64_t n : {int64_t(1), big * 8 - 4096 * 2, big * 8 - 4096, big * 8 - 4095, big * 8, big * 8 + 1, big * 40 + 7}) {
    for (const zero_dtype dt : {ZERO_BF16, ZERO_F32}) {
      const zero_drop d = {0.5, 1, 2, 3, nullptr, 5};
      g_done = 0, g_first = 5;
      EXPECT(zero_dropout(fake(0), fake(1), fake(2), n, dt, &d, nullptr) == ZERO_OK, "dropout: %s", zero_last_error());
      EXPECT(g_done == n, "dropout of %lld: %lld", (long long)n, (long long)g_done);
    }
  }
  for (const int64_t hidden : {int64_t(1), int64_t(7), int64_t(8), int64_t(8192), int64_t(1) << 24}) {
    const int64_t upr = hidden < 8 ? hidden : hidden / 8, most = ((big - 1) / kEmbedThreads * kEmbedThreads * kEmbedUnroll) / upr;
    const int64_t sizes[2] = {3, 5 * hidden};
    zero_plan_t plan;
    if (zero_plan(3 + 5 * hidden, 1, sizes, 2, 0, 1, &plan) != ZERO_OK) return 2;
    const zero_drop d = {0.5, 1, 2, 3, nullptr, 3};
    for (const int64_t n : {int64_t(1), most - 1, most, most + 1, 5 * most + 3}) {
      g_done = 0, g_first = 3, g_hidden = hidden, g_stride = hidden + 2;
      EXPECT(zero_embed(plan, 1, hidden, fake(0), ZERO_BF16, fake(1), ZERO_I32, n, 1.0, &d, fake(2), ZERO_BF16, g_stride,
                        nullptr) == ZERO_OK, "embed: %s", zero_last_error());
      EXPECT(g_done == n, "embed of %lld: %lld", (long long)n, (long long)g_done);
    }
    zero_plan_destroy(plan);
  }
  const int64_t rows = INT32_MAX;
  for (const int64_t vocab : {int64_t(2), int64_t(2049), int64_t(8191), int64_t(8192), int64_t(32767), int64_t(32768), int64_t(131072), int64_t(1) << 30}) {
    for (const int64_t n : {int64_t(1), int64_t(1023), int64_t(1024), int64_t(4095), big / 512 - 1, big / 512, big / 128, big / 64 - 1, big / 64,
                            big / 64 + 1, rows}) {
      if (n > (int64_t(1) << 55) / vocab) continue;   // the stand-in buffers end
      g_done = 0, g_left = n, g_stride = vocab;
      const size_t ws = zero_token_logp_workspace_bytes(n, vocab);
      zero_status st = zero_token_logp(fake(0), ZERO_BF16, n, vocab, vocab, fake(1), ZERO_I32, (float*)fake(2), (float*)fake(3),
                                       fake(9), ws, nullptr);
      EXPECT(st == ZERO_OK && g_done == n, "logp of %lld x %lld: %s", (long long)n, (long long)vocab, zero_last_error());
      st = zero_token_logp_grad(fake(0), ZERO_BF16, n, vocab, vocab, fake(1), ZERO_I32, (float*)fake(3), (float*)fake(4), fake(5),
                                vocab + 1, nullptr);
      EXPECT(st == ZERO_OK && g_left == 0, "dlogits of %lld x %lld: %s", (long long)n, (long long)vocab, zero_last_error());
    }
  }
  for (const int64_t pairs : {int64_t(0), int64_t(1), int64_t(17), big / 1024 - 2, big / 1024 - 1, big / 1024, int64_t(1) << 29}) {
    for (const int64_t n : {int64_t(0), int64_t(1025), rows}) {
      g_done = 0, g_means = 0;
      const zero_status st = zero_preference_loss(pairs, fake(0), ZERO_I32, n, nullptr, ZERO_I32, 1, (float*)fake(1), nullptr, 0.1, 0, 1,
                                                  (float*)fake(2), (float*)fake(3), (float*)fake(4), (float*)fake(5), nullptr);
      EXPECT(st == ZERO_OK && g_done == pairs && g_means == 1, "preference of %lld: %s", (long long)pairs, zero_last_error());
    }
  }
  // Positions and activations that one launch takes, and more than it takes
  // (of a size that no memory holds), which is refused.
  struct {
    int64_t hidden, tiles;
  } const wide[] = {{1, 1}, {513, 3}, {8192, 16}, {1 << 20, 2048}, {1 << 24, 32768}};
  for (const auto [hidden, tiles] : wide) {
    const int64_t sizes[1] = {3 * hidden}, n = int64_t(1) << 30;
    zero_plan_t plan;
    if (zero_plan(3 * hidden, 1, sizes, 1, 0, 1, &plan) != ZERO_OK) return 2;
    const zero_status st = zero_embed_grad(plan, 0, hidden, (int32_t*)fake(3), (int32_t*)fake(4), n, fake(5), ZERO_BF16, hidden, 1.0,
                                           nullptr, fake(6), ZERO_BF16, -1, 0, fake(8), zero_embed_grad_workspace_bytes(n, hidden), nullptr);
    EXPECT(st == (n / 256 * tiles * kGradThreads < big ? ZERO_OK : ZERO_EUNSUPPORTED), "grad of %lld: %d %s", (long long)hidden, (int)st,
           zero_last_error());
    zero_plan_destroy(plan);
  }
  printf("%d launches, %d failures\n", g_launches, g_fail);
  return g_fail != 0;
}
