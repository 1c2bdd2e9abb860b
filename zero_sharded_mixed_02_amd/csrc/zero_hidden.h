// zero_hidden.h -- structures shared by the host entries (zero_hidden_api.cpp)
// and the gfx950 kernels (zero_linear.hip, zero_muon.hip) of the operators on a
// model's hidden matrices.
#pragma once

#include <stdint.h>

#include "zero.h"

namespace zk {
namespace hidden {

constexpr int64_t kLaunchItems = int64_t(1) << 32;   // work items of a launch, exclusive
inline int64_t most_blocks(int threads) { return (kLaunchItems - 1) / threads; }

// Tiles of a product: rows x columns of the result per workgroup.
enum Tile : int { kTile256 = 0, kTile128 = 1, kTile64 = 2, kTiles = 3 };
constexpr int kTileSize[kTiles] = {256, 128, 64};
constexpr int kTileThreads[kTiles] = {512, 256, 256};

// What one product reads and how its tiles are laid out.
struct Product {
  const void* a;
  const void* b;
  int64_t lda, ldb;       // elements between memory rows
  int32_t m, n, k;
  int32_t tm, tn, tiles;  // of one result: rows, columns, how many are computed
  int32_t size;           // rows and columns of a tile
  int32_t whole;          // tiles (over all results) summed in one piece; the others ("cut") in
  int32_t cut;            //   `splits` pieces of k,
  int32_t splits;
  int32_t k_piece;        //   of so many elements, a multiple of the stage depth
  int32_t pad_;
  float* part;            // fp32[cut][splits][size][size]: partial sums
};

// zero_linear (EPI 0) and zero_linear_input_grad (EPI 1).
struct LinearArgs {
  Product p;
  void* out;
  void* pre_out;          // EPI 0: the sum before act, or NULL
  const void* pre_in;     // EPI 1: where act' is taken, or NULL
  const void* add;        // residual or addend, or NULL
  const void* bias;       // EPI 0, or NULL
  int64_t ldo, ldpre, ldadd;
  int32_t act;
  int32_t pad_;
};

// zero_linear_weight_grad: m rows of the weight from row0 on, n columns.
struct WeightGradArgs {
  Product p;
  void* dst;              // the element lo of the weight
  int64_t lo, hi;         // elements of the weight that are written
  int32_t row0;
  int32_t dst_dt;
  int32_t accumulate;
  float scale;
  // The bias: columns [b_lo, b_hi) of dz are summed (dz: column row0 of its first row).
  const void* dz;
  int64_t dz_stride;
  void* bias_dst;         // the element b_lo of the bias
  float* bias_part;       // fp32[chunks][columns]
  int32_t b_lo, b_hi;
  int32_t chunk_rows, chunks, col_blocks, bias_blocks;
  int32_t join_blocks, pad_;
};

// Rows of `width` 16-bit elements into rows of whole eights, padded with zeros.
struct CopyRowsArgs {
  const void* src;
  void* dst;
  int64_t rows, ld_src, ld_dst;
  int32_t width, units;     // units of eight in a row of dst
};
constexpr int kCopyThreads = 256;

struct ActGradArgs {
  const void* dy;
  const void* pre;
  void* dz;
  int64_t n;
  int32_t act;
  int32_t pad_;
};

// zero_orthogonalize: one launch over `batch` matrices of one shape, which lie
// `z*` elements apart in the workspace.
constexpr int kMaxBatch = 128;
enum OrthoEpi : int { kGram = 0, kPoly = 1, kNext = 2 };

struct OrthoArgs {
  Product p;              // of one matrix
  int64_t za, zb, zout, zadd;
  const float* factor;    // fp32[batch][2]: what the first X is to be multiplied by, and whether to shift
  void* out;              // 16-bit result in the workspace, rows of ldo
  void* low;              // kNext: what X's rounding left, bf16, read (not at first) and written
  const void* add;        // kPoly: A - shift I; kNext: X
  int64_t ldo, ldadd;
  int32_t batch, epi;
  int32_t tall;           // rows > cols: A = X^T X, and X A
  int32_t first;          // X as loaded: the factor applies, and add is 16-bit
  int32_t last, dst_dt;   // the result goes to dst
  float a, b, c, shift;   // d = shift or 0: kGram: factor^2 sum - d I; kPoly: (b + 2 c d) add + c sum;
                          // kNext: factor ((a + b d + c d^2) add + sum)
  int32_t rows, cols;     // of dst
  void* dst;              // flat buffer
  float scale[kMaxBatch];
  int64_t dst_off[kMaxBatch];
};

// Norms and the first X of a batch.
struct OrthoLoadArgs {
  const void* src;
  void* x;                // fp16, rows `pitch` apart of ld elements, padded with zeros
  double* sums;           // fp64[batch][kNormBlocks]
  float* factor;
  double eps;
  int64_t numel, zx;
  int64_t pitch, again;   // a second copy lies `again` elements behind the first (0: none)
  int32_t rows, cols, ld, rows_pad, batch, norm_blocks;
  int64_t src_off[kMaxBatch];
};
// The polynomials of a batch of matrices whose shorter side is at most kThinSide.
constexpr int kThinSide = 64;
constexpr int kThinThreads = 512;
struct OrthoThinArgs {
  const float* part;      // fp32[batch][splits][64][64]: pieces of X X^T
  float* factor;          // as above; takes the power of two that is left out of p
  void* p;                // fp16[batch][side][2 side]: P, and what its rounding left
  float a, b, c;
  int32_t steps, splits;
  int32_t n, side;        // the shorter side, and rounded up to 8
};

// A batch of matrices of one shape that a workgroup each orthogonalises in LDS.
constexpr int kSmallElems = 16384;
constexpr int kSmallThreads = 512;
constexpr int kShortSide = 16;
struct OrthoSmallArgs {
  const void* src;
  void* dst;
  double eps;
  float a, b, c, shift;
  int32_t shift_from, steps;
  int32_t rows, cols, rp, cp;       // sides, and rounded up to 32
  int32_t src_dt, dst_dt;
  int32_t is_short, pad_;           // a side of at most kShortSide, and P may stand for the steps
  float scale[kMaxBatch];
  int64_t off[kMaxBatch];
};

constexpr int kNormBlocks = 1024;    // most pieces of a matrix's norm
constexpr int kLoadThreads = 256;
constexpr int kLoadUnits = 4;        // of eight elements, a thread

constexpr int kBiasCols = 256;     // columns of a bias workgroup
constexpr int kJoinThreads = 256;
constexpr int kActThreads = 256;
constexpr int kActVec = 8;

// Launchers.  Return a hipError_t as int.
int launch_linear(const LinearArgs& a, int epi, int dt, int tile, bool direct, void* stream);
int launch_linear_join(const LinearArgs& a, int epi, int dt, int64_t blocks, void* stream);
int launch_weight_grad(const WeightGradArgs& a, int dt, int tile, bool direct, int64_t blocks, void* stream);
int launch_weight_grad_join(const WeightGradArgs& a, int64_t blocks, void* stream);
int launch_ortho_small(const OrthoSmallArgs& a, int64_t batch, void* stream);
int launch_ortho_thin(const OrthoThinArgs& a, int64_t batch, void* stream);
int launch_ortho_norm(const OrthoLoadArgs& a, int dt, void* stream);
int launch_ortho_load(const OrthoLoadArgs& a, int dt, int64_t blocks, void* stream);
int launch_ortho(const OrthoArgs& a, int tile, int64_t blocks, void* stream);
int launch_ortho_join(const OrthoArgs& a, int64_t blocks, void* stream);
int launch_copy_rows(const CopyRowsArgs& a, int64_t blocks, void* stream);
int launch_act_grad(const ActGradArgs& a, int dt, int64_t blocks, void* stream);

}  // namespace hidden
}  // namespace zk
