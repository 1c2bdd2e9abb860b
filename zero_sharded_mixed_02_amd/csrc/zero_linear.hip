// zero_linear.hip -- gfx950 kernels of the hidden matrices' products: the linear
// layer with bias, activation and residual in the product's epilogue, the
// gradient of its input, and the gradient of its weight and bias.
#include "zero_gemm.h"
#include "zero_act.h"
#include "zero_hidden_dev.h"

#pragma clang fp contract(off)

namespace zk {
namespace hidden {
namespace {

using namespace zk::gemm;

// What the epilogue of V sums of row `row` from column `col` on reads (the bias, of
// the same columns for all of a lane's rows, comes from outside), and the epilogue.
// One rounding to 16 bits, of the finished value.
template <typename T, int EPI, int V>
struct Epilogue {
  Row<T, V> pre[EPI];       // the activation's argument
  Row<T, V> add;            // the residual or addend

  __device__ __forceinline__ void load(const LinearArgs& a, int64_t row, int col) {
    const int have = a.p.n - col;
    if constexpr (EPI == 1) {
      if (a.pre_in) pre[0].load(a.pre_in, row * a.ldpre + col, have);
    }
    if (a.add) add.load(a.add, row * a.ldadd + col, have);
  }

  __device__ __forceinline__ void finish(const LinearArgs& a, int64_t row, int col, const float (&acc)[V], const Row<T, V>& bias) const {
    const int have = a.p.n - col;
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = acc[i];
    if constexpr (EPI == 0) {
      if (a.bias) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] += (float)bias.v[i];
      }
      if (a.pre_out) store_row<T, V>(a.pre_out, row * a.ldpre + col, have, v);
      if (a.act != ZERO_ACT_NONE) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = act::forward(a.act, v[i]);
      }
    } else {
      if (a.pre_in) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= act::slope(a.act, (float)pre[0].v[i]);
      }
    }
    if (a.add) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] += (float)add.v[i];
    }
    store_row<T, V>(a.out, row * a.ldo + col, have, v);
  }
};

// A workgroup a tile.  EPI 0: forms K and K; EPI 1: K and M.  Large products are bound
// by the power limit (4096 x 8192 -> 32768 bf16, gelu, z kept: 1755 us, 1253 TFLOP/s,
// the matrix units busy 63% of the time at 1.9 GHz; dx of 8192 x 8192 x 8192: 852 us),
// short sums by a tile's first loads and its epilogue (2048 x 768 -> 50257: 214 us),
// few rows by latency (one row of 768 x 768: 12 workgroups, about 4 us).
template <typename T, int EPI, int TILE, bool DIRECT>
__global__ void __launch_bounds__(kTileThreads[TILE]) linear_kernel(const LinearArgs a) {
  typedef CoreOf<T, kFormK, EPI == 0 ? kFormK : kFormM, TILE, DIRECT> C;
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  C core;
  int z, m0, n0;
  if (!run_tile<false>(core, (ZK_LDS char*)smem, a.p, blockIdx.x, 0, 0, z, m0, n0)) return;
  typedef Epilogue<T, EPI, 8> E;
  Row<T, 8> bias;
  if (EPI == 0 && a.bias) bias.load(a.bias, C::column(n0), a.p.n - C::column(n0));
  core.template each<E>((ZK_LDS char*)smem, m0, n0, false,
                        [&](int row, int col, E& e) { if (row < a.p.m && col < a.p.n) e.load(a, row, col); },
                        [&](int row, int col, const float (&v)[8], const E& e) {
                          if (row < a.p.m && col < a.p.n) e.finish(a, row, col, v, bias);
                        }, 0);
}

template <typename T, int EPI>
__global__ void __launch_bounds__(kJoinThreads) linear_join_kernel(const LinearArgs a) {
  int z, row, col;
  bool twice;
  float v[4];
  if (join4<false>(a.p, (int64_t)blockIdx.x * kJoinThreads + threadIdx.x, z, row, col, v, twice)) {
    Epilogue<T, EPI, 4> e;
    Row<T, 4> bias;
    if (EPI == 0 && a.bias) bias.load(a.bias, col, a.p.n - col);
    e.load(a, row, col);
    e.finish(a, row, col, v, bias);
  }
}

// ---------------------------------------------------------------------------
// Gradient of the weight and the bias
// ---------------------------------------------------------------------------

__device__ __forceinline__ float load_dst(const void* dst, int dt, int64_t e) {
  if (dt == ZERO_F32) return ((const AS1 float*)dst)[e];
  if (dt == ZERO_BF16) return (float)((const AS1 __bf16*)dst)[e];
  return (float)((const AS1 _Float16*)dst)[e];
}
__device__ __forceinline__ void store_dst(void* dst, int dt, int64_t e, float v) {
  if (dt == ZERO_F32) ((AS1 float*)dst)[e] = v;
  else if (dt == ZERO_BF16) ((AS1 __bf16*)dst)[e] = (__bf16)v;
  else ((AS1 _Float16*)dst)[e] = (_Float16)v;
}

// Whole vectors of 16-bit results go out at once; fp32 ones, and the ends of a slice, element by
// element (8192 x 8192 x 8192 into bf16 809 us, added 845; into fp32 947, added 1261).
template <int V>
__device__ __forceinline__ void finish_weight(const WeightGradArgs& a, int row, int col, const float (&acc)[V]) {
  const int have = a.p.n - col;
  const int64_t e = (int64_t)(row + a.row0) * a.p.n + col;       // element of the weight
  float v[V], x[V];
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = acc[i] * a.scale;
  if (have >= V && e >= a.lo && e + V <= a.hi && a.dst_dt != ZERO_F32) {
    if (a.dst_dt == ZERO_BF16) {
      if (a.accumulate) {
        load_row<__bf16, V>(a.dst, e - a.lo, V, x);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] += x[i];
      }
      store_row<__bf16, V>(a.dst, e - a.lo, V, v);
    } else {
      if (a.accumulate) {
        load_row<_Float16, V>(a.dst, e - a.lo, V, x);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] += x[i];
      }
      store_row<_Float16, V>(a.dst, e - a.lo, V, v);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (i < have && e + i >= a.lo && e + i < a.hi) {
      const int64_t d = e + i - a.lo;
      store_dst(a.dst, a.dst_dt, d, a.accumulate ? load_dst(a.dst, a.dst_dt, d) + v[i] : v[i]);
    }
  }
}

__device__ __forceinline__ void finish_bias(const WeightGradArgs& a, int col, float s) {
  const float v = s * a.scale;
  const int64_t d = col - a.b_lo;
  store_dst(a.bias_dst, a.dst_dt, d, a.accumulate ? load_dst(a.bias_dst, a.dst_dt, d) + v : v);
}

// Sums of 256 columns of dz over a chunk of rows: 32 lanes of eight columns, the
// workgroup's other lanes on other rows; joined in LDS in the lanes' order.
template <typename T, int NT>
__device__ void bias_block(const WeightGradArgs& a, ZK_LDS float* lds, int b) {
  constexpr int V = 8, RL = 8;      // whatever NT is: the tile leaves the order of the sums alone
  const int chunk = b / a.col_blocks, col0 = a.b_lo + (b % a.col_blocks) * kBiasCols;
  const int lane = threadIdx.x & 31, rl = threadIdx.x >> 5, col = col0 + lane * V;
  const int have = a.b_hi - col;
  const int r0 = chunk * a.chunk_rows, r1 = a.p.k - r0 < a.chunk_rows ? a.p.k : r0 + a.chunk_rows;
  float s[V], x[V];
#pragma unroll
  for (int i = 0; i < V; ++i) s[i] = 0.0f;
  if (have > 0 && rl < RL) {
#pragma unroll 4
    for (int r = r0 + rl; r < r1; r += RL) {
      load_row<T, V>(a.dz, (int64_t)r * a.dz_stride + (col - a.row0), have, x);
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] += x[i];
    }
  }
  if (rl < RL) {
#pragma unroll
    for (int i = 0; i < V; ++i) lds[rl * kBiasCols + lane * V + i] = s[i];
  }
  __syncthreads();
  for (int j = threadIdx.x; j < kBiasCols; j += NT) {
    if (col0 + j >= a.b_hi) continue;
    float t = lds[j];
    for (int q = 1; q < RL; ++q) t += lds[q * kBiasCols + j];
    if (a.chunks > 1) a.bias_part[(int64_t)chunk * (a.b_hi - a.b_lo) + (col0 + j - a.b_lo)] = t;
    else finish_bias(a, col0 + j, t);
  }
}

// The bias's workgroups first, whose reads of dz run beside the first tiles, then a
// workgroup a tile or a piece of k of it.  8192 x 8192 x 8192 bf16: 820 us, 1341
// TFLOP/s, at the power limit; an eighth of 768 x 768 over 8191 rows: 7.9 us and the
// join 4.2, latencies in a row.
template <typename T, int TILE, bool DIRECT>
__global__ void __launch_bounds__(kTileThreads[TILE]) weight_grad_kernel(const WeightGradArgs a) {
  typedef CoreOf<T, kFormM, kFormM, TILE, DIRECT> C;
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  const int b = (int)blockIdx.x - a.bias_blocks;
  if (b < 0) {
    bias_block<T, kTileThreads[TILE]>(a, (ZK_LDS float*)smem, blockIdx.x);
    return;
  }
  C core;
  int z, m0, n0;
  if (!run_tile<false>(core, (ZK_LDS char*)smem, a.p, b, 0, 0, z, m0, n0)) return;
  core.template each<int>((ZK_LDS char*)smem, m0, n0, false, [](int, int, int&) {},
                          [&](int row, int col, const float (&v)[8], int) {
                            if (row < a.p.m && col < a.p.n) finish_weight<8>(a, row, col, v);
                          }, 0);
}

__global__ void __launch_bounds__(kJoinThreads) weight_grad_join_kernel(const WeightGradArgs a) {
  if ((int)blockIdx.x < a.join_blocks) {
    int z, row, col;
    bool twice;
    float v[4];
    if (join4<false>(a.p, (int64_t)blockIdx.x * kJoinThreads + threadIdx.x, z, row, col, v, twice)) finish_weight<4>(a, row, col, v);
    return;
  }
  const int cols = a.b_hi - a.b_lo;
  const int j = ((int)blockIdx.x - a.join_blocks) * kJoinThreads + threadIdx.x;
  if (j >= cols) return;
  float t = a.bias_part[j];
#pragma unroll 8
  for (int c = 1; c < a.chunks; ++c) t += a.bias_part[(int64_t)c * cols + j];
  finish_bias(a, a.b_lo + j, t);
}

// ---------------------------------------------------------------------------
// Gradient through an activation alone
// ---------------------------------------------------------------------------

// Eight elements a thread; bound by memory (268 M elements through gelu's slope: 271 us, 5.9 TB/s).
template <typename T>
__global__ void __launch_bounds__(kActThreads) act_grad_kernel(const ActGradArgs a) {
  const int64_t e = ((int64_t)blockIdx.x * kActThreads + threadIdx.x) * kActVec;
  if (e >= a.n) return;
  const int have = a.n - e < kActVec ? (int)(a.n - e) : kActVec;
  float dy[kActVec], z[kActVec];
  load_row<T, kActVec>(a.dy, e, have, dy);
  load_row<T, kActVec>(a.pre, e, have, z);
#pragma unroll
  for (int i = 0; i < kActVec; ++i) dy[i] *= act::slope(a.act, z[i]);
  store_row<T, kActVec>(a.dz, e, have, dy);
}

// Rows at any alignment into rows of whole eights, a unit of eight a thread.
__global__ void __launch_bounds__(kCopyThreads) copy_rows_kernel(const CopyRowsArgs a) {
  const int64_t u = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x;
  const int64_t row = u / a.units;
  if (row >= a.rows) return;
  const int col = (int)(u - row * a.units) * 8;
  Row<_Float16, 8> x;       // bits, whichever type
  x.load(a.src, row * a.ld_src + col, a.width - col);
  *(AS1 Row<_Float16, 8>::tv*)((AS1 _Float16*)a.dst + row * a.ld_dst + col) = x.v;
}

// ---------------------------------------------------------------------------
// Dispatch
// ---------------------------------------------------------------------------

template <typename T, int EPI, int TILE, bool DIRECT>
int go_linear(const LinearArgs& a, void* stream) {
  return launch(&linear_kernel<T, EPI, TILE, DIRECT>, a, a.p.whole + (int64_t)a.p.cut * a.p.splits, kTileThreads[TILE],
                CoreOf<T, kFormK, EPI == 0 ? kFormK : kFormM, TILE, DIRECT>::kLds, stream);
}
template <typename T, int EPI, int TILE>
int go_linear(const LinearArgs& a, bool direct, void* stream) {
  return direct ? go_linear<T, EPI, TILE, true>(a, stream) : go_linear<T, EPI, TILE, false>(a, stream);
}
template <typename T, int EPI>
int go_linear(const LinearArgs& a, int tile, bool direct, void* stream) {
  if (tile == kTile256) return go_linear<T, EPI, kTile256>(a, direct, stream);
  if (tile == kTile128) return go_linear<T, EPI, kTile128>(a, direct, stream);
  return go_linear<T, EPI, kTile64>(a, direct, stream);
}

template <typename T, int TILE, bool DIRECT>
int go_weight(const WeightGradArgs& a, int64_t blocks, void* stream) {
  constexpr int bias = 8 * kBiasCols * 4;
  constexpr int lds = CoreOf<T, kFormM, kFormM, TILE, DIRECT>::kLds;
  return launch(&weight_grad_kernel<T, TILE, DIRECT>, a, blocks, kTileThreads[TILE], lds > bias ? lds : bias, stream);
}
template <typename T, int TILE>
int go_weight(const WeightGradArgs& a, bool direct, int64_t blocks, void* stream) {
  return direct ? go_weight<T, TILE, true>(a, blocks, stream) : go_weight<T, TILE, false>(a, blocks, stream);
}
template <typename T>
int go_weight(const WeightGradArgs& a, int tile, bool direct, int64_t blocks, void* stream) {
  if (tile == kTile256) return go_weight<T, kTile256>(a, direct, blocks, stream);
  if (tile == kTile128) return go_weight<T, kTile128>(a, direct, blocks, stream);
  return go_weight<T, kTile64>(a, direct, blocks, stream);
}

}  // namespace

int launch_linear(const LinearArgs& a, int epi, int dt, int tile, bool direct, void* stream) {
  if (dt == ZERO_BF16)
    return epi == 0 ? go_linear<__bf16, 0>(a, tile, direct, stream) : go_linear<__bf16, 1>(a, tile, direct, stream);
  return epi == 0 ? go_linear<_Float16, 0>(a, tile, direct, stream) : go_linear<_Float16, 1>(a, tile, direct, stream);
}

int launch_linear_join(const LinearArgs& a, int epi, int dt, int64_t blocks, void* stream) {
  if (dt == ZERO_BF16)
    return epi == 0 ? launch(&linear_join_kernel<__bf16, 0>, a, blocks, kJoinThreads, 0, stream)
                    : launch(&linear_join_kernel<__bf16, 1>, a, blocks, kJoinThreads, 0, stream);
  return epi == 0 ? launch(&linear_join_kernel<_Float16, 0>, a, blocks, kJoinThreads, 0, stream)
                  : launch(&linear_join_kernel<_Float16, 1>, a, blocks, kJoinThreads, 0, stream);
}

int launch_weight_grad(const WeightGradArgs& a, int dt, int tile, bool direct, int64_t blocks, void* stream) {
  return dt == ZERO_BF16 ? go_weight<__bf16>(a, tile, direct, blocks, stream)
                         : go_weight<_Float16>(a, tile, direct, blocks, stream);
}

int launch_weight_grad_join(const WeightGradArgs& a, int64_t blocks, void* stream) {
  return launch(&weight_grad_join_kernel, a, blocks, kJoinThreads, 0, stream);
}

int launch_copy_rows(const CopyRowsArgs& a, int64_t blocks, void* stream) {
  return launch(&copy_rows_kernel, a, blocks, kCopyThreads, 0, stream);
}

int launch_act_grad(const ActGradArgs& a, int dt, int64_t blocks, void* stream) {
  return dt == ZERO_BF16 ? launch(&act_grad_kernel<__bf16>, a, blocks, kActThreads, 0, stream)
                         : launch(&act_grad_kernel<_Float16>, a, blocks, kActThreads, 0, stream);
}

}  // namespace hidden
}  // namespace zk
