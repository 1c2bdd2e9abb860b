// The order of the table gradient's sums, checked on the CPU.
//
// A run of equal tokens is summed chunk by chunk.  As in ops_shapes.cpp the
// launchers are stand-ins: every owner's slice of a table has to be cut into
// the chunks that the whole buffer is cut into, and where several waves share
// a chunk, each of its runs has to be whole and in one of them.
#include <stdint.h>
#include <stdio.h>

#include <random>

#include "zero.h"
#include "zero_internal.h"
#include "zero_ops.h"

namespace {
int g_fail = 0, g_checks = 0;
int32_t g_chunk, g_parts;
void expect(bool c, const char* what, long long a, long long b) {
  ++g_checks;
  if (!c && g_fail++ < 20) fprintf(stderr, "FAIL: %s (%lld, %lld)\n", what, a, b);
}
void* fake(int id) { return (void*)(uintptr_t)((uint64_t)(id + 1) << 57); }
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
int launch_embed(const EmbedArgs&, int, int, bool, int64_t, void*) { return 0; }
int launch_rank(const RankArgs&, int64_t, void*) { return 0; }
int launch_radix(const RadixArgs&, void*) { return 0; }
int launch_grad(const GradArgs& a, int, int, int, int64_t, void*) {
  g_chunk = a.chunk;
  g_parts = a.parts;
  return 0;
}
int launch_grad_join(const GradArgs&, int, bool, int64_t, void*) { return 0; }
int launch_dropout(const DropoutArgs&, int, int64_t, void*) { return 0; }
int launch_logp(const LogpArgs&, int, void*) { return 0; }
int launch_logp_join(const LogpArgs&, int, void*) { return 0; }
int launch_dlogits(const LogpArgs&, int, void*) { return 0; }
int launch_preference(const PrefArgs&, void*) { return 0; }
}  // namespace ops
}  // namespace zk

int main() {
  for (const int64_t hidden : {1, 64, 65, 768, 1601, 2048, 8192, 20000}) {
    for (int64_t n = 1; n <= (1 << 22); n = n * 3 + 1) {
      for (const int nd : {1, 2, 8, 64}) {
        const int64_t sizes[1] = {1000 * hidden};
        zero_plan_t plan;
        if (zero_plan(sizes[0], nd, sizes, 1, 0, 1, &plan) != ZERO_OK) return 2;
        int32_t whole = 0;
        for (int rank = -1; rank < nd; ++rank) {
          for (int acc = 0; acc < 2; ++acc) {
            const zero_status st = zero_embed_grad(plan, 0, hidden, (int32_t*)fake(3), (int32_t*)fake(4), n, fake(5), rank % 2 ? ZERO_BF16 : ZERO_F32,
                                                   hidden, 1.0, nullptr, fake(6), acc ? ZERO_F32 : ZERO_F16, rank, acc, fake(8),
                                                   zero_embed_grad_workspace_bytes(n, hidden), nullptr);
            expect(st == ZERO_OK, "call refused", n, hidden);
            if (rank < 0 && !acc) whole = g_chunk;
            expect(g_chunk == whole, "a slice is cut into other chunks than the whole", g_chunk, whole);
            expect(g_parts >= 1 && g_parts <= 4 && g_chunk % 4 == 0 && g_chunk <= 64, "parts", g_parts, g_chunk);
          }
        }
        zero_plan_destroy(plan);
      }
    }
  }
  // Chunks of random runs, cut at both ends by what the slice holds.
  std::mt19937_64 rng(3);
  for (int trial = 0; trial < 200000; ++trial) {
    const int chunk = 4 * (1 + (int)(rng() % 16)), parts = 1 + (int)(rng() % 4), len = trial % 4 ? chunk : 1 + (int)(rng() % chunk);
    uint64_t starts = rng();
    for (int k = (int)(rng() % 4); k > 0; --k) starts &= rng();
    starts &= (len < 64 ? (uint64_t(1) << len) - 1 : ~uint64_t(0)) & ~uint64_t(1);
    // The slice begins and ends with runs.
    int p0 = (int)(rng() % len), p1 = p0 + 1 + (int)(rng() % (len - p0));
    if (trial % 3) p0 = 0, p1 = len;
    while (p0 > 0 && !(starts >> p0 & 1)) --p0;
    while (p1 < len && !(starts >> p1 & 1)) ++p1;
    int at = p0;
    for (int part = 0; part < parts; ++part) {
      const zk::ops::Span s = zk::ops::runs_of_part(starts, p0, p1, chunk, parts, part);
      if (s.lo >= s.hi) continue;
      expect(s.lo == at, "positions left out or taken twice", s.lo, at);
      expect(s.hi == p1 || (starts >> s.hi & 1), "a run is cut", s.hi, part);
      const int each = chunk / parts;
      expect(s.lo == p0 || s.lo >= part * each, "a run of an earlier part", s.lo, part);
      at = s.hi;
    }
    expect(at == p1, "positions left out", at, p1);
  }
  printf("%d checks, %d failures\n", g_checks, g_fail);
  return g_fail != 0;
}
