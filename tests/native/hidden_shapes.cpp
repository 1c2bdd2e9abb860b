// Launch shapes of the operators on the hidden matrices, checked on the CPU.
//
// zero_hidden_api.cpp is compiled together with this file, which stands in for
// the kernel launchers: instead of launching, it checks that each launch covers
// its work once and that what its kernels read and write lies inside the buffers
// and the workspace of the call, apart where it has to be.  Built with g++ under
// AddressSanitizer and UndefinedBehaviorSanitizer; no GPU is involved.
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

constexpr uint64_t kSpan = 1ull << 50;
enum { kParams, kX, kOut, kPre, kAdd, kWs, kBuffers };
int64_t g_bytes[kBuffers];      // of the running call's buffers
void* fake(int id) { return (void*)(uintptr_t)((uint64_t)(id + 1) * kSpan); }

struct Span { uint64_t lo, hi; };
Span span(const void* p, int64_t bytes) { return {(uint64_t)(uintptr_t)p, (uint64_t)(uintptr_t)p + (uint64_t)std::max<int64_t>(0, bytes)}; }
bool inside(Span s) {
  if (s.lo == s.hi) return true;
  const int id = (int)(s.lo / kSpan) - 1;
  if (id < 0 || id >= kBuffers) return false;
  const uint64_t lo = (uint64_t)(id + 1) * kSpan;
  return s.hi <= lo + (uint64_t)g_bytes[id];
}
bool apart(Span a, Span b) { return a.hi <= b.lo || b.hi <= a.lo; }
bool in_ws(Span s) { return s.lo == s.hi || (inside(s) && (int)(s.lo / kSpan) - 1 == kWs); }

using namespace zk::hidden;

// Rows of an operand that a product reads: 16-bit, `rows` memory rows of `width`.
Span operand(const void* p, int64_t ld, int64_t rows, int64_t width) { return span(p, ((rows - 1) * ld + width) * 2); }

struct Sums { Span part; };
Sums product(const char* what, const Product& p, int64_t tiles_all, bool m_a, bool m_b, bool direct, int64_t batch, int64_t za, int64_t zb) {
  EXPECT(p.size == 256 || p.size == 128 || p.size == 64, "%s: tile %d", what, p.size);
  EXPECT((int64_t)p.tm * p.size >= p.m && (int64_t)(p.tm - 1) * p.size < std::max(p.m, 1), "%s: rows of tiles", what);
  EXPECT((int64_t)p.tn * p.size >= p.n && (int64_t)(p.tn - 1) * p.size < std::max(p.n, 1), "%s: columns of tiles", what);
  EXPECT((int64_t)p.whole + p.cut == tiles_all, "%s: %d + %d tiles of %lld", what, p.whole, p.cut, (long long)tiles_all);
  EXPECT(p.splits >= 1 && p.k_piece % 64 == 0, "%s: pieces", what);
  if (p.cut) {
    EXPECT((int64_t)p.splits * p.k_piece >= p.k, "%s: %d pieces of %d do not cover %d", what, p.splits, p.k_piece, p.k);
    EXPECT(p.splits == 1 || (int64_t)(p.splits - 1) * p.k_piece < p.k, "%s: an empty piece", what);
  }
  const Span a = operand(p.a, p.lda, m_a ? p.k : p.m, m_a ? p.m : p.k), b = operand(p.b, p.ldb, m_b ? p.k : p.n, m_b ? p.n : p.k);
  if (p.m > 0 && p.n > 0 && p.k > 0) {
    EXPECT(inside({a.lo, a.hi + (uint64_t)((batch - 1) * za * 2)}), "%s: a leaves its buffer", what);
    EXPECT(inside({b.lo, b.hi + (uint64_t)((batch - 1) * zb * 2)}), "%s: b leaves its buffer", what);
  }
  if (direct) {
    EXPECT(a.lo % 4 == 0 && p.lda % 2 == 0 && b.lo % 4 == 0 && p.ldb % 2 == 0, "%s: direct loads at odd places", what);
    EXPECT((!m_a || p.m % 2 == 0 || p.lda > p.m) && (!m_b || p.n % 2 == 0 || p.ldb > p.n), "%s: a word behind the last row", what);
  }
  EXPECT((int64_t)(256 - 1) * std::max(p.lda, p.ldb) * 2 < (int64_t(1) << 31), "%s: a tile's rows pass 31 bits", what);
  const Span part = span(p.part, p.splits > 1 || p.cut ? (int64_t)p.cut * p.splits * p.size * p.size * 4 : 0);
  EXPECT(in_ws(part) && part.lo % 16 == 0, "%s: partial sums outside the workspace", what);
  EXPECT(apart(part, a) && apart(part, b), "%s: partial sums over an operand", what);
  return {part};
}

int g_launches;
Span g_copies[4];
int g_n_copies;

}  // namespace

namespace zk {
const char* hip_error_string(int) { return "stub"; }
int launch_step(const StepArgs&, int, int, int, int, bool, int, void*) { return 0; }
int launch_copy(const CopyArgs&, int, int, void*) { return 0; }
int launch_warm(const WarmArgs&, int, void*) { return 0; }
int resident_blocks(int, int, int, int, bool) { return 0; }
double wall_clock_hz() { return 0; }
double hbm_peak_bps() { return 0; }

namespace hidden {

int launch_linear(const LinearArgs& a, int epi, int, int tile, bool direct, void*) {
  ++g_launches;
  EXPECT(a.p.size == kTileSize[tile], "the tile's size");
  const Sums s = product("linear", a.p, (int64_t)a.p.tm * a.p.tn, false, epi == 1, direct, 1, 0, 0);
  EXPECT(inside(span(a.out, ((a.p.m - 1) * a.ldo + a.p.n) * 2)), "linear: y");
  if (a.add) EXPECT(inside(span(a.add, ((a.p.m - 1) * a.ldadd + a.p.n) * 2)), "linear: residual");
  if (a.pre_out) EXPECT(inside(span(a.pre_out, ((a.p.m - 1) * a.ldpre + a.p.n) * 2)), "linear: pre");
  if (a.pre_in) EXPECT(inside(span(a.pre_in, ((a.p.m - 1) * a.ldpre + a.p.n) * 2)), "input grad: pre");
  if (a.bias) EXPECT(inside(span(a.bias, (int64_t)a.p.n * 2)), "linear: bias");
  for (int i = 0; i < g_n_copies; ++i) EXPECT(apart(s.part, g_copies[i]), "linear: partial sums over a copy");
  return 0;
}
int launch_linear_join(const LinearArgs& a, int, int, int64_t blocks, void*) {
  EXPECT(blocks * kJoinThreads * 4 >= (int64_t)a.p.cut * a.p.size * a.p.size, "linear: a join too small");
  return 0;
}

int launch_weight_grad(const WeightGradArgs& a, int, int tile, bool direct, int64_t blocks, void*) {
  ++g_launches;
  EXPECT(a.p.m == 0 || a.p.size == kTileSize[tile], "the tile's size");
  EXPECT(blocks == a.bias_blocks + (int64_t)a.p.whole + (int64_t)a.p.cut * a.p.splits, "weight grad: workgroups");
  Span part = {0, 0};
  if (a.p.m > 0) {
    part = product("weight grad", a.p, (int64_t)a.p.tm * a.p.tn, true, true, direct, 1, 0, 0).part;
    const int es = a.dst_dt == ZERO_F32 ? 4 : 2;
    EXPECT(inside(span(a.dst, (a.hi - a.lo) * es)), "weight grad: dst");
    EXPECT(a.lo >= (int64_t)a.row0 * a.p.n && a.hi <= ((int64_t)a.row0 + a.p.m) * a.p.n, "weight grad: rows do not hold the slice");
  }
  if (a.bias_blocks) {
    const int64_t cols = a.b_hi - a.b_lo;
    EXPECT((int64_t)a.chunks * a.chunk_rows >= a.p.k && (a.chunks == 1 || (int64_t)(a.chunks - 1) * a.chunk_rows < a.p.k), "bias: chunks");
    EXPECT((int64_t)a.col_blocks * kBiasCols >= cols, "bias: columns");
    if (a.p.k > 0) EXPECT(inside(span((const char*)a.dz + (a.b_lo - a.row0) * 2, ((a.p.k - 1) * a.dz_stride + cols) * 2)), "bias: dz");
    EXPECT(inside(span(a.bias_dst, cols * (a.dst_dt == ZERO_F32 ? 4 : 2))), "bias: dst");
    if (a.chunks > 1) {
      const Span b = span(a.bias_part, a.chunks * cols * 4);
      EXPECT(in_ws(b) && apart(b, part), "bias: partial sums");
      for (int i = 0; i < g_n_copies; ++i) EXPECT(apart(b, g_copies[i]) && apart(part, g_copies[i]), "weight grad: sums over a copy");
    }
  }
  return 0;
}
int launch_weight_grad_join(const WeightGradArgs& a, int64_t blocks, void*) {
  const int64_t cols = a.bias_blocks && a.chunks > 1 ? a.b_hi - a.b_lo : 0;
  EXPECT((int64_t)a.join_blocks * kJoinThreads * 4 >= (a.p.splits > 1 ? (int64_t)a.p.cut * a.p.size * a.p.size : 0), "weight grad: a join too small");
  EXPECT((blocks - a.join_blocks) * kJoinThreads >= cols, "bias: a join too small");
  return 0;
}

int launch_copy_rows(const CopyRowsArgs& a, int64_t blocks, void*) {
  EXPECT(blocks * kCopyThreads >= a.rows * a.units && a.units * 8 >= a.width && a.ld_dst == a.units * 8, "copy: units");
  EXPECT(inside(operand(a.src, a.ld_src, a.rows, a.width)), "copy: source");
  const Span d = span(a.dst, a.rows * a.ld_dst * 2);
  EXPECT(in_ws(d) && d.lo % 16 == 0, "copy: destination");
  for (int i = 0; i < g_n_copies; ++i) EXPECT(apart(d, g_copies[i]), "copies overlap");
  if (g_n_copies < 4) g_copies[g_n_copies++] = d;
  return 0;
}

int launch_act_grad(const ActGradArgs&, int, int64_t, void*) { return 0; }

int64_t g_matrices, g_last;
int launch_ortho_small(const OrthoSmallArgs& a, int64_t batch, void*) {
  ++g_launches;
  const int side = std::min(a.rp, a.cp);
  EXPECT(a.rp >= a.rows && a.cp >= a.cols && a.rp % 32 == 0 && a.cp % 32 == 0, "small: sides");
  EXPECT(a.rp * (a.cp * 2 + 16) + 2 * side * (side * 2 + 16) <= 160 * 1024, "small: LDS");
  EXPECT((a.rp / 16) * (a.cp / 16) <= 8 * (kSmallThreads / 64), "small: tiles a wave");
  EXPECT(batch >= 1 && batch <= kMaxBatch, "small: batch");
  for (int64_t i = 0; i < batch; ++i) EXPECT(inside(span((const char*)a.dst + a.off[i] * 2, (int64_t)a.rows * a.cols * 2)), "small: dst");
  g_matrices += batch;
  return 0;
}
Span g_sums, g_factor, g_x;
int launch_ortho_norm(const OrthoLoadArgs& a, int, void*) {
  EXPECT(a.norm_blocks >= 1 && a.norm_blocks <= kNormBlocks && a.batch >= 1 && a.batch <= kMaxBatch, "norm: pieces");
  g_sums = span(a.sums, (int64_t)a.batch * a.norm_blocks * 8);
  g_factor = span(a.factor, (int64_t)a.batch * 8);
  EXPECT(in_ws(g_sums) && in_ws(g_factor) && apart(g_sums, g_factor) && g_sums.lo % 8 == 0, "norm: sums");
  for (int i = 0; i < a.batch; ++i) EXPECT(inside(span((const char*)a.src + a.src_off[i] * 2, a.numel * 2)), "norm: source");
  g_matrices += a.batch;
  return 0;
}
int launch_ortho_load(const OrthoLoadArgs& a, int, int64_t blocks, void*) {
  const int64_t per = (int64_t)a.rows_pad * (a.ld / 8), of = kLoadThreads * kLoadUnits;
  EXPECT(blocks == a.batch * ((per + of - 1) / of), "load: workgroups");
  EXPECT(a.ld % 8 == 0 && a.ld >= a.cols && a.rows_pad >= a.rows && a.pitch % 8 == 0 && a.again % 8 == 0, "load: rows");
  EXPECT(a.again == 0 || a.again >= (a.pitch > a.ld ? a.ld : a.rows_pad * a.pitch), "load: the copies overlap");
  const int64_t most = (a.rows_pad - 1) * a.pitch + a.ld + a.again;
  EXPECT(most <= a.zx, "load: a matrix passes into the next");
  g_x = span(a.x, ((a.batch - 1) * a.zx + most) * 2);
  EXPECT(in_ws(g_x) && apart(g_x, g_sums) && apart(g_x, g_factor) && g_x.lo % 16 == 0, "load: X");
  return 0;
}
int launch_ortho(const OrthoArgs& a, int tile, int64_t blocks, void*) {
  ++g_launches;
  EXPECT(a.p.size == kTileSize[tile], "the tile's size");
  const bool sym = a.epi != kNext;
  const int64_t tiles = (sym ? (int64_t)a.p.tm * (a.p.tm + 1) / 2 : (int64_t)a.p.tm * a.p.tn) * a.batch;
  EXPECT(blocks == (int64_t)a.p.whole + (int64_t)a.p.cut * a.p.splits, "ortho: workgroups");
  const bool m_a = a.epi == kGram && a.tall, m_b = (a.epi == kGram && a.tall) || (a.epi == kNext && !a.tall);
  const Span part = product("ortho", a.p, tiles, m_a, m_b, true, a.batch, a.za, a.zb).part;
  const Span pa = {span(a.p.a, 0).lo, operand(a.p.a, a.p.lda, m_a ? a.p.k : a.p.m, m_a ? a.p.m : a.p.k).hi + (uint64_t)((a.batch - 1) * a.za * 2)};
  const Span pb = {span(a.p.b, 0).lo, operand(a.p.b, a.p.ldb, m_b ? a.p.k : a.p.n, m_b ? a.p.n : a.p.k).hi + (uint64_t)((a.batch - 1) * a.zb * 2)};
  EXPECT(in_ws(pa) && in_ws(pb), "ortho: operands");
  EXPECT(apart(part, g_factor) && apart(part, pa) && apart(part, pb), "ortho: partial sums");
  if (a.p.whole == 0 && a.out == nullptr) return 0;      // pieces of A alone
  Span out = {0, 0}, low = {0, 0}, add = {0, 0};
  const int64_t rows = ((a.p.m - 1) * a.ldo + a.p.n), of_add = ((a.p.m - 1) * a.ldadd + a.p.n);
  if (a.epi != kGram) {
    add = span(a.add, ((a.batch - 1) * a.zadd + of_add) * 2);
    EXPECT(in_ws(add) && add.lo % 16 == 0 && a.ldadd % 8 == 0, "ortho: what is added");
  }
  if (!a.last) {
    EXPECT(rows <= a.zout, "ortho: a result passes into the next");
    out = span(a.out, ((a.batch - 1) * a.zout + rows) * 2);
    EXPECT(in_ws(out) && apart(out, pa) && apart(out, pb) && apart(out, part) && apart(out, add) && apart(out, g_factor) && apart(out, g_sums),
           "ortho: the result");
    if (a.epi == kNext) {
      low = span(a.low, ((a.batch - 1) * a.zadd + of_add) * 2);
      EXPECT(in_ws(low) && apart(low, pa) && apart(low, pb) && apart(low, part) && apart(low, out) && apart(low, g_factor), "ortho: X's rest");
    }
  } else {
    for (int i = 0; i < a.batch; ++i)
      EXPECT(inside(span((const char*)a.dst + a.dst_off[i] * 2, (int64_t)a.rows * a.cols * 2)), "ortho: dst");
    EXPECT(a.rows <= a.p.m && a.cols <= a.p.n, "ortho: not all of the result is computed");
    g_last += a.batch;
  }
  return 0;
}
int launch_ortho_thin(const OrthoThinArgs& a, int64_t batch, void*) {
  ++g_launches;
  EXPECT(a.side % 8 == 0 && a.side >= a.n && a.n >= 1 && a.side <= kThinSide && a.splits >= 1, "thin: side");
  const Span part = span(a.part, batch * a.splits * kThinSide * kThinSide * 4), p = span(a.p, batch * a.side * a.side * 4);
  EXPECT(in_ws(part) && in_ws(p) && apart(part, p) && apart(p, g_x) && apart(part, g_x) && apart(p, g_factor), "thin: buffers");
  EXPECT(g_factor.lo == span(a.factor, 0).lo, "thin: factor");
  return 0;
}
int launch_ortho_join(const OrthoArgs& a, int64_t blocks, void*) {
  EXPECT(blocks * kJoinThreads * 4 >= (int64_t)a.p.cut * a.p.size * a.p.size, "ortho: a join too small");
  return 0;
}

}  // namespace hidden
}  // namespace zk

int main() {
  std::mt19937_64 rng(7);
  auto pick = [&](int64_t lo, int64_t hi) { return lo + (int64_t)(rng() % (uint64_t)(hi - lo + 1)); };
  auto log_pick = [&](int64_t hi) { return std::min<int64_t>(hi, pick(1, int64_t(1) << pick(0, 63 - __builtin_clzll((uint64_t)hi)))); };
  int calls = 0;
  for (int it = 0; it < 20000; ++it) {
    const int64_t in = log_pick(20000), out = log_pick(20000), n = log_pick(40000);
    const int nd = (int)pick(1, 9);
    const int64_t numel[4] = {pick(0, 40), in * out, pick(0, 9), out};
    zero_plan_t plan;
    if (zero_plan(numel[0] + numel[1] + numel[2] + numel[3], nd, numel, 4, 0, pick(0, 1) ? 1 : 64, &plan)) return 2;
    int64_t psi_pad, shard;
    int32_t nb, nd2;
    zero_plan_info(plan, &psi_pad, &shard, &nb, &nd2);
    const int64_t xs = in + pick(0, 1) * pick(0, 7), ys = out + pick(0, 1) * pick(0, 7);
    const int off = (int)pick(0, 3) * 2;      // bytes off 16-byte alignment
    auto at = [&](int id) { return (void*)((char*)fake(id) + off); };
    auto sizes = [&](int64_t x, int64_t o, int64_t pre, int64_t add, int64_t ws) {
      g_bytes[kParams] = psi_pad * 2;
      g_bytes[kX] = x + off;
      g_bytes[kOut] = o + off;
      g_bytes[kPre] = pre + off;
      g_bytes[kAdd] = add + off;
      g_bytes[kWs] = ws;
      g_n_copies = g_launches = 0;
    };
    auto rows = [&](int64_t stride, int64_t width) { return ((n - 1) * stride + width) * 2; };
    const zero_dtype dt = pick(0, 1) ? ZERO_BF16 : ZERO_F16;
    int64_t ws = (int64_t)zero_linear_workspace_bytes(plan, 1, in, n);
    sizes(rows(xs, in), rows(ys, out), rows(out, out), rows(ys, out), ws);
    int st = zero_linear(plan, 1, pick(0, 1) ? 3 : -1, in, fake(kParams), dt, at(kX), n, xs, ZERO_ACT_GELU, at(kAdd), ys, at(kPre), out, at(kOut), ys,
                         fake(kWs), ws, nullptr);
    EXPECT(st == ZERO_OK && g_launches == 1, "zero_linear: %d, %s", st, zero_last_error());
    ws = (int64_t)zero_linear_input_grad_workspace_bytes(plan, 1, in, n);
    sizes(rows(ys, out), rows(xs, in), rows(in, in), rows(xs, in), ws);
    st = zero_linear_input_grad(plan, 1, in, fake(kParams), dt, at(kX), n, ys, ZERO_ACT_SILU, at(kPre), in, at(kAdd), xs, at(kOut), xs, fake(kWs), ws, nullptr);
    EXPECT(st == ZERO_OK && g_launches == 1, "zero_linear_input_grad: %d, %s", st, zero_last_error());
    const int rank = (int)pick(-1, nd - 1);
    const zero_dtype ddt = pick(0, 2) ? dt : ZERO_F32;
    ws = (int64_t)zero_linear_weight_grad_workspace_bytes(plan, 1, in, n, rank);
    sizes(rows(ys, out), (rank < 0 ? psi_pad : shard) * (ddt == ZERO_F32 ? 4 : 2), 0, rows(xs, in), ws);
    st = zero_linear_weight_grad(plan, 1, pick(0, 1) ? 3 : -1, in, at(kX), ys, at(kAdd), xs, dt, n, 1.0, fake(kOut), ddt, rank, (int)pick(0, 1), fake(kWs), ws,
                                 nullptr);
    EXPECT(st == ZERO_OK && g_launches <= 1, "zero_linear_weight_grad: %d, %s", st, zero_last_error());
    calls += 3;
    zero_plan_destroy(plan);
  }
  for (int it = 0; it < 20000; ++it) {
    const int kinds = (int)pick(1, 3);
    std::vector<int64_t> numel;
    std::vector<zero_matrix> ms;
    int64_t want = 0;
    for (int k = 0; k < kinds; ++k) {
      const int64_t top = pick(0, 3) ? 4000 : 20000, r = log_pick(top), c = pick(0, 3) ? log_pick(top) : r;
      const int64_t stack = pick(0, 5) ? 1 : pick(2, 5), tensors = std::min<int64_t>(log_pick(300), std::max<int64_t>(1, (int64_t(3) << 27) / (r * c * stack)));
      for (int64_t t = 0; t < tensors; ++t) {
        ms.push_back({(int32_t)numel.size(), r, c, 1.0});
        numel.push_back(r * c * stack);
        want += stack;
      }
    }
    std::shuffle(ms.begin(), ms.end(), rng);
    int64_t psi = 0;
    for (int64_t v : numel) psi += v;
    zero_plan_t plan;
    if (zero_plan(psi, 1, numel.data(), (int32_t)numel.size(), 0, pick(0, 1) ? 1 : 64, &plan)) return 2;
    int64_t psi_pad, shard;
    int32_t nb, nd;
    zero_plan_info(plan, &psi_pad, &shard, &nb, &nd);
    const int64_t ws = (int64_t)zero_orthogonalize_workspace_bytes(plan, ms.data(), (int32_t)ms.size());
    memset(g_bytes, 0, sizeof g_bytes);
    g_bytes[kX] = g_bytes[kOut] = psi_pad * 2;
    g_bytes[kWs] = ws;
    zk::hidden::g_matrices = zk::hidden::g_last = 0;
    const zero_newton_schulz poly = {(int32_t)pick(1, 14), 1.875, -1.25, 0.375, 1e-7};
    const int st = zero_orthogonalize(plan, ms.data(), (int32_t)ms.size(), pick(0, 1) ? &poly : nullptr, fake(kX), ZERO_BF16, fake(kOut), ZERO_F16, fake(kWs), ws,
                                      nullptr);
    EXPECT(st == ZERO_OK, "zero_orthogonalize: %d, %s", st, zero_last_error());
    EXPECT(zk::hidden::g_matrices == want, "%lld matrices of %lld", (long long)zk::hidden::g_matrices, (long long)want);
    ++calls;
    zero_plan_destroy(plan);
  }
  printf("%d calls, %d failures\n", calls, g_fail);
  return g_fail != 0;
}
