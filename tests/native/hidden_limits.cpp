// Calls of the operators on the hidden matrices at the ends of what the header
// allows, checked on the CPU.
//
// zero_hidden_api.cpp is compiled together with this file, which stands in for
// the kernel launchers: each launch has to have work and stay within 2^32 work
// items, and a call within the limits has to succeed.  Built with g++ under
// AddressSanitizer and UndefinedBehaviorSanitizer; no GPU is involved.
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <random>
#include <vector>

#include "zero.h"
#include "zero_hidden.h"
#include "zero_internal.h"

namespace {

int g_fail = 0, g_calls = 0;
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

void* fake(int id) { return (void*)(uintptr_t)((uint64_t)(id + 1) << 52); }

int grid(const char* what, int64_t blocks, int threads) {
  EXPECT(blocks >= 1 && blocks * threads < (int64_t(1) << 32), "%s: %lld workgroups of %d", what, (long long)blocks, threads);
  return 0;
}

std::vector<zk::hidden::CopyRowsArgs> g_copies;      // of the running call, launches that go on from one another joined

}  // namespace

namespace zk {
const char* hip_error_string(int) { return "stub"; }
int64_t g_elems;      // of the running call's launches
int launch_step(const StepArgs& a, int, int, int, int, bool vec, int blocks, void*) {
  for (int i = 0; i < a.n_seg; ++i) g_elems += a.seg[i].len;
  return grid("step over the shard", blocks, vec ? kStepThreads : kThreads);
}
int launch_copy(const CopyArgs&, int, int, void*) { return 0; }
int launch_warm(const WarmArgs&, int, void*) { return 0; }
int resident_blocks(int, int, int, int, bool) { return 0; }
double wall_clock_hz() { return 0; }
double hbm_peak_bps() { return 0; }

namespace hidden {
int launch_linear(const LinearArgs& a, int, int, int tile, bool, void*) {
  return grid("product", a.p.whole + (int64_t)a.p.cut * a.p.splits, kTileThreads[tile]);
}
int launch_linear_join(const LinearArgs&, int, int, int64_t blocks, void*) { return grid("join", blocks, kJoinThreads); }
int launch_weight_grad(const WeightGradArgs&, int, int tile, bool, int64_t blocks, void*) { return grid("weight gradient", blocks, kTileThreads[tile]); }
int launch_weight_grad_join(const WeightGradArgs&, int64_t blocks, void*) { return grid("weight gradient's join", blocks, kJoinThreads); }
int launch_copy_rows(const CopyRowsArgs& a, int64_t blocks, void*) {
  EXPECT(blocks * kCopyThreads >= a.rows * a.units, "copy: units");
  CopyRowsArgs* l = g_copies.empty() ? nullptr : &g_copies.back();
  if (l && (const char*)a.src == (const char*)l->src + l->rows * l->ld_src * 2 && (char*)a.dst == (char*)l->dst + l->rows * l->ld_dst * 2 &&
      a.ld_src == l->ld_src && a.ld_dst == l->ld_dst && a.width == l->width)
    l->rows += a.rows;
  else
    g_copies.push_back(a);
  return grid("copy", blocks, kCopyThreads);
}
int launch_act_grad(const ActGradArgs&, int, int64_t blocks, void*) { return grid("activation gradient", blocks, kActThreads); }
int launch_ortho_small(const OrthoSmallArgs&, int64_t batch, void*) { return grid("small matrices", batch, kSmallThreads); }
int launch_ortho_norm(const OrthoLoadArgs& a, int, void*) { return grid("norms", (int64_t)a.batch * a.norm_blocks, kLoadThreads); }
int launch_ortho_load(const OrthoLoadArgs&, int, int64_t blocks, void*) { return grid("first X", blocks, kLoadThreads); }
int launch_ortho(const OrthoArgs&, int tile, int64_t blocks, void*) { return grid("step", blocks, kTileThreads[tile]); }
int launch_ortho_thin(const OrthoThinArgs&, int64_t batch, void*) { return grid("polynomials", batch, kThinThreads); }
int launch_ortho_join(const OrthoArgs&, int64_t blocks, void*) { return grid("step's join", blocks, kJoinThreads); }
}  // namespace hidden
}  // namespace zk

namespace {

constexpr int64_t kMemory = int64_t(288) << 30;

// Whole operands have been copied: two at most, of n or `out` rows.
void copied(int64_t n, int64_t out) {
  EXPECT(g_copies.size() <= 2, "%zu copies", g_copies.size());
  for (const auto& c : g_copies) EXPECT(c.rows == n || c.rows == out, "%lld rows copied of %lld or %lld", (long long)c.rows, (long long)n, (long long)out);
  g_copies.clear();
}

// The three products of a layer, where their operands fit a GPU's memory.
void layer(int64_t n, int64_t in, int64_t out, int nd, int64_t odd, int64_t before) {
  const int64_t xs = in + odd, ys = out + odd;
  const int64_t numel[3] = {before, in * out, out};
  zero_plan_t plan;
  if (zero_plan(before + in * out + out, nd, numel, 3, 0, 1, &plan)) {
    EXPECT(false, "plan");
    return;
  }
  int64_t pad, shard;
  int32_t nb, nd2;
  zero_plan_info(plan, &pad, &shard, &nb, &nd2);
  const int64_t bytes = 2 * (pad + n * (xs + ys));
  int64_t ws = (int64_t)zero_linear_workspace_bytes(plan, 1, in, n);
  if (bytes + ws <= kMemory && xs <= 1 << 21) {
    const int st = zero_linear(plan, 1, 2, in, fake(0), ZERO_BF16, fake(1), n, xs, ZERO_ACT_GELU, nullptr, 0, nullptr, 0, fake(2), ys, fake(3), ws, nullptr);
    EXPECT(st == ZERO_OK, "linear %lld x %lld -> %lld: %s", (long long)n, (long long)in, (long long)out, zero_last_error());
    ++g_calls;
    copied(n, out);
  }
  ws = (int64_t)zero_linear_input_grad_workspace_bytes(plan, 1, in, n);
  if (bytes + ws <= kMemory && ys <= 1 << 21) {
    const int st = zero_linear_input_grad(plan, 1, in, fake(0), ZERO_BF16, fake(1), n, ys, ZERO_ACT_NONE, nullptr, 0, nullptr, 0, fake(2), xs, fake(3), ws, nullptr);
    EXPECT(st == ZERO_OK, "input gradient %lld x %lld -> %lld: %s", (long long)n, (long long)in, (long long)out, zero_last_error());
    ++g_calls;
    copied(n, out);
  }
  ws = (int64_t)zero_linear_weight_grad_workspace_bytes(plan, 1, in, n, nd - 1);
  if (bytes + 2 * (shard - pad) + ws <= kMemory && std::max(xs, ys) <= 1 << 21) {
    const int st = zero_linear_weight_grad(plan, 1, 2, in, fake(0), ys, fake(1), xs, ZERO_F16, n, 1.0, fake(2), ZERO_F16, nd - 1, 0, fake(3), ws, nullptr);
    EXPECT(st == ZERO_OK, "weight gradient %lld x %lld -> %lld: %s", (long long)n, (long long)in, (long long)out, zero_last_error());
    ++g_calls;
    copied(n, out);
  }
  zero_plan_destroy(plan);
}

// `count` matrices of a shape: the workspace stays within 1.125 GiB, or what one of them
// takes, and the call succeeds.
void matrices(int64_t rows, int64_t cols, int64_t count) {
  const int64_t numel[2] = {rows * cols * count, rows * cols};
  zero_plan_t plan;
  if (zero_plan(numel[0] + numel[1], 1, numel, 2, 0, 1, &plan)) {
    EXPECT(false, "plan");
    return;
  }
  const zero_matrix all = {0, rows, cols, 1.0}, one = {1, rows, cols, 1.0};
  const int64_t ws = (int64_t)zero_orthogonalize_workspace_bytes(plan, &all, 1), single = (int64_t)zero_orthogonalize_workspace_bytes(plan, &one, 1);
  EXPECT(ws <= std::max(int64_t(9) << 27, single), "%lld of %lld x %lld take %lld bytes, one %lld", (long long)count, (long long)rows, (long long)cols,
         (long long)ws, (long long)single);
  const zero_newton_schulz fast = {7, 3.4445, -4.7750, 2.0315, 1e-7};      // beyond what short sides take a way of their own for
  for (const zero_newton_schulz* q : {(const zero_newton_schulz*)nullptr, &fast}) {
    const int st = zero_orthogonalize(plan, &all, 1, q, fake(0), ZERO_BF16, fake(1), ZERO_F16, fake(3), ws, nullptr);
    EXPECT(st == ZERO_OK, "%lld of %lld x %lld: %s", (long long)count, (long long)rows, (long long)cols, zero_last_error());
    ++g_calls;
  }
  zero_plan_destroy(plan);
}

// The two halves of the step on buffers `off` bytes off their alignment.
void step(int64_t n, int off) {
  zero_plan_t plan;
  if (zero_plan(n, 1, &n, 1, 0, 1, &plan)) {
    EXPECT(false, "plan");
    return;
  }
  const zero_muon_hyper hp = {0.02, 0.95, 0.1, 1.0, 1};
  auto at = [&](int id, int es) { return (char*)fake(id) + off / 4 * es; };
  const void* slices[1] = {at(0, 2)};
  const zero_grad_src src = {ZERO_BF16, 1, slices, nullptr};
  zk::g_elems = 0;
  int st = zero_muon_momentum(plan, 0, &hp, &src, nullptr, (float*)at(1, 4), at(2, 2), ZERO_BF16, 1, nullptr);
  EXPECT(st == ZERO_OK && zk::g_elems == n, "momentum of %lld: %s, %lld elements", (long long)n, zero_last_error(), (long long)zk::g_elems);
  zk::g_elems = 0;
  st = zero_muon_apply(plan, 0, &hp, at(0, 2), ZERO_BF16, 1, (float*)at(1, 4), at(2, 2), ZERO_F16, 1, nullptr);
  EXPECT(st == ZERO_OK && zk::g_elems == n, "apply of %lld: %s, %lld elements", (long long)n, zero_last_error(), (long long)zk::g_elems);
  g_calls += 2;
  zero_plan_destroy(plan);
}

}  // namespace

int main() {
  std::mt19937_64 rng(11);
  auto pick = [&](int64_t lo, int64_t hi) { return lo + (int64_t)(rng() % (uint64_t)(hi - lo + 1)); };
  auto log_pick = [&](double hi) { return std::max<int64_t>(1, (int64_t)exp2(log2(hi) * (double)(rng() % 4097) / 4096.0)); };
  const int64_t most = int64_t(1) << 30, wide = int64_t(1) << 21;
  // The longest sides, alone and with others that fill the memory.
  for (int64_t one : {1, 2, 33, 63, 64, 128, 2049})
    for (int64_t other : {1, 2, 31, 64, 100}) {
      layer(most, one, other, 1, 0, 0);
      layer(most, other, one, 1, 0, 0);
      layer(one, other, most, 1, 0, 0);
      layer(most / 64, one, other * 33, 8, 1, 3);
      layer(one, wide, other, 1, 0, 0);
      layer(one, other, wide, 1, 0, 0);
    }
  // A layer without outputs: its input's gradient is the addend.
  for (int64_t n : {int64_t(1), int64_t(100), int64_t(1) << 20, int64_t(1) << 24})
    for (int64_t in : {1, 8, 33, 4097}) layer(n, in, 0, 2, 0, 1);
  for (int it = 0; it < 30000; ++it) {
    const int64_t n = log_pick((double)most), in = log_pick((double)wide), out = log_pick(pick(0, 3) ? (double)wide : (double)most);
    if ((double)n * (double)(in + out) + (double)in * (double)out > 3e11) continue;
    layer(n, in, out, (int)pick(1, 4), pick(0, 2) ? 0 : 1, pick(0, 1));
  }
  for (int64_t side : {1, 2, 3, 7, 8, 17, 33, 64, 65, 72, 200})
    for (int64_t length : {16385, 70000, 1 << 18, 1 << 20})
      for (int64_t count : {1, 2, 17, 128, 129, 500}) {
        matrices(side, length, count);
        matrices(length, side, count);
      }
  for (int it = 0; it < 3000; ++it) {
    const int64_t rows = log_pick(1 << 20), cols = log_pick(1 << 20);
    if (rows * cols > int64_t(1) << 31) continue;
    matrices(rows, cols, std::max<int64_t>(1, std::min<int64_t>(log_pick(700), (int64_t(1) << 36) / (rows * cols))));
  }
  for (int off : {0, 4})
    for (int64_t n : {int64_t(1), int64_t(1001), int64_t(1) << 28, (int64_t(1) << 32) - 3, int64_t(1) << 32, (int64_t(1) << 34) + 5}) step(n, off);
  printf("%d calls, %d failures\n", g_calls, g_fail);
  return g_fail != 0;
}
