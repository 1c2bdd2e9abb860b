// zero_ops.h -- structures shared by the host entries (zero_ops_api.cpp) and
// the gfx950 kernels (zero_ops.hip) of the vocabulary operators.
#pragma once

#include <stdint.h>

#include "zero.h"

namespace zk {
namespace ops {

// SplitMix64's increment and output function (Steele, Lea & Flood, OOPSLA 2014).
constexpr uint64_t kGamma = 0x9E3779B97F4A7C15ull;
constexpr uint64_t kMix1 = 0xBF58476D1CE4E5B9ull;
constexpr uint64_t kMix2 = 0x94D049BB133111EBull;

// A dropout as the kernels take it.
struct DropArgs {
  uint64_t key;               // of the mask, when step_dev is NULL
  uint64_t site_key;          // key before the step is mixed in
  const uint64_t* step_dev;   // step read on the device, or NULL
  int64_t first;              // mask position of the call's first element
  uint32_t cut;               // 16-bit draws below it are dropped; 0: keep all
  uint32_t pad_;
};

struct EmbedArgs {
  const void* table;
  const void* tokens;
  void* out;
  int64_t n;
  int64_t out_stride;
  int32_t rows;
  int32_t hidden;
  int32_t upr;       // units of one access per row
  int32_t tok64;     // tokens are int64
  float f;
  uint32_t magic;    // floor(2^32 / upr) + 1, 0 for upr = 1
  DropArgs drop;
};

// Sorting tokens: positions are ranked by counting when there are few, and by
// radix passes of at most kDigitBits bits otherwise.
// Most positions ranked by counting: what 13 bits beside a token's 19 and 32 KiB
// of LDS hold.  There it takes 7.8 us and the radix passes 17.4; n^2 would meet
// them at about 12000.
constexpr int kSmallSort = 8192;
constexpr int kSmallSortPosBits = 13;
constexpr int kRankThreads = 1024;
constexpr int kRankItems = 32;           // positions ranked per workgroup
constexpr int kDigitBits = 9;
constexpr int kBins = 1 << kDigitBits;
constexpr int kSortThreads = 512;        // also one thread per bin
// Keys per thread and tile: two up to kSortFew positions, where four leave CUs
// without a tile (65536: 17.9 us against 19.9), four beyond, where two make
// more workgroups than their counts are worth (262144: 28 us against 33).
constexpr int kSortKeysFew = 2;
constexpr int kSortKeysMany = 4;
constexpr int kSortFew = 131072;
constexpr int kSortBlocks = 256;         // most workgroups of a pass

struct RankArgs {
  const void* tokens;
  int32_t* sorted;
  int32_t* order;
  int32_t n;
  int32_t rows;
  int32_t tok64;
};

struct RadixArgs {
  const void* tokens;       // first pass: ids
  const int32_t* key_in;    // later passes
  const int32_t* pos_in;
  int32_t* key_out;
  int32_t* pos_out;
  uint32_t* hist;           // [n_blocks][kBins]
  int64_t n;
  int32_t rows;
  int32_t tok64;
  int32_t first;            // reads tokens
  int32_t shift;
  int32_t bits;
  int32_t n_blocks;
  int32_t tile;             // positions of a tile
  int64_t tiles_per_block;
};

// Gradient of the table: positions in token order are cut into chunks of
// `chunk`; see zero_ops.hip.
constexpr int kGradThreads = 256;
constexpr int kGradChunks = kGradThreads / 64;   // neighbouring chunks of a workgroup, one a wave
constexpr int kJoinThreads = 512;
constexpr int kJoinChunks = 16;          // chunks it looks after
constexpr int kJoinLong = 64;            // chunks from which a run is cut into pieces

// A search for the first index in [lo, hi) whose key is not below the wanted
// one, by 64 lanes that look at an index each.
struct LowerBound {
  int64_t lo, hi;
  constexpr bool open() const { return hi > lo; }
  // At least 1, so that a search which has ended (beside another that goes on)
  // has all lanes at hi or beyond.
  constexpr int64_t step() const { return hi - lo > 64 ? (hi - lo + 63) / 64 : 1; }
  constexpr int64_t probe(int lane) const { return lo + (lane + 1) * step() - 1; }   // nothing to look at from hi on
  constexpr void narrow(int below) {   // that many lanes saw a key below
    const int64_t s = step();
    lo += below * s;
    if (lo > hi) lo = hi;
    if (lo + s - 1 < hi) hi = lo + s - 1;
  }
};

// Positions [lo, hi) of a chunk.
struct Span {
  int lo, hi;
};

// What one of `parts` waves takes of the positions [p0, p1) of a chunk: the
// runs that begin in its part, whole, the first one beginning at p0.  `starts`
// has a bit for each position where a token differs from the one before.
constexpr Span runs_of_part(uint64_t starts, int p0, int p1, int chunk, int parts, int part) {
  const uint64_t begins = (starts | (uint64_t(1) << p0)) >> p0 << p0;
  const int each = chunk / parts, q0 = part * each, q1 = part + 1 < parts ? q0 + each : 64;
  const uint64_t from0 = begins >> q0 << q0, from1 = q1 < 64 ? begins >> q1 << q1 : 0;
  const int lo = from0 ? __builtin_ctzll(from0) : p1, hi = from1 ? __builtin_ctzll(from1) : p1;
  return Span{lo < p1 ? lo : p1, hi < p1 ? hi : p1};
}

struct GradArgs {
  const int32_t* sorted;
  const int32_t* order;
  const void* dy;
  void* dst;               // element lo of the tensor
  float* part;             // [2 * n_chunks][hidden]
  int64_t n;
  int64_t dy_stride;
  int64_t lo, hi;          // elements of the tensor that are written
  int32_t row_lo, row_hi;  // rows they lie in
  int32_t rows;
  int32_t hidden;
  int32_t chunk;
  int32_t n_chunks;
  int32_t tiles;           // workgroups of a group of chunks: column tiles times parts
  int32_t fill_rows;       // rows of one zero-fill workgroup
  int32_t accumulate;
  float f;
  int64_t chunk_blocks;    // workgroups before those that write zero rows
  int32_t stream_dy;       // dy is read past the caches
  int32_t join_tiles;      // column tiles of the join
  int32_t parts;           // waves that share a chunk's runs
  DropArgs drop;
};

struct DropoutArgs {
  const void* x;
  const void* residual;
  void* out;
  int64_t n;
  float f;
  int32_t pad_;
  DropArgs drop;
};

constexpr int kLogpThreads = 512;
// Rows shorter than this take one wave instead of eight, and rows four times
// as long where there are waves for all CUs anyway: 8192 rows of 2000 bf16 in
// 16 us against 38, of 16000 in 68 against 83.
constexpr int kLogpShortRow = 8192;
constexpr int kLogpManyRows = 4096;
constexpr int kDlogitsThreads = 128;
constexpr int kDlogitsUnroll = 2;
constexpr int kDlogitsPiece = 2048;      // elements of a row per workgroup
// The forward pass reads its last rows through the caches, and the gradient
// starts with them.  Of the 256 MB Infinity Cache, 128 MiB cost nothing: a
// forward pass alone over 823 MB of logits takes 107 us and 109 without, with the
// gradient over 412 MB 185 either way; 192 MiB make that 183 but the first 112.
constexpr int64_t kCachedBytes = int64_t(128) << 20;

struct LogpArgs {
  const void* logits;
  const void* labels;
  float* logp;
  float* stats;
  float* part;        // [n][splits][2] when splits > 1
  const float* coef;  // gradient
  void* dlogits;
  int64_t n;
  int64_t stride;
  int64_t dl_stride;
  int32_t vocab;
  int32_t lab64;
  int32_t splits;     // workgroups per row
  int32_t cached_from;   // first row that is read through the caches
};

constexpr int kPrefThreads = 1024;
// Largest loss that one workgroup computes in one launch: one pair of 24 rows
// each in 4.8 us against 5.9 for two launches, of 512 in 6.3 against 6.7, of
// 2048 in 15.9 against 7.6.
constexpr int kPrefSmallPairs = 16;
constexpr int kPrefSmallRows = 1024;

struct PrefArgs {
  const void* offsets;
  const void* labels;      // or NULL
  const float* logp;
  const float* ref;        // or NULL
  float* loss;
  float* pair_loss;
  float* rewards;
  float* coef;
  int64_t n;
  int64_t n_pairs;
  int64_t vocab;
  double beta, smoothing, slope;   // slope = beta * grad_scale / n_pairs
  int64_t pair0, pair_count;       // pairs of this launch
  int32_t off64;
  int32_t lab64;
};

// A launch has fewer than 2^32 work items in each dimension (HIP's limit on
// grid times workgroup).  A call with more work takes several launches, each
// over a part of the rows, elements or pairs.
constexpr int64_t kLaunchItems = (int64_t(1) << 32) - 1;
constexpr int64_t most_blocks(int threads) { return kLaunchItems / threads; }

// Threads per row, or per piece of one (see kLogpShortRow).
constexpr int logp_threads(int64_t n, int64_t vocab) {
  return vocab < (n < kLogpManyRows ? kLogpShortRow : 4 * kLogpShortRow) ? 64 : kLogpThreads;
}

// Launchers (zero_ops.hip).  Return a hipError_t as int.
int launch_embed(const EmbedArgs& a, int tdt, int odt, bool vec, int64_t blocks, void* stream);
int launch_rank(const RankArgs& a, int64_t blocks, void* stream);
int launch_radix(const RadixArgs& a, void* stream);
int launch_grad(const GradArgs& a, int ydt, int gdt, int vec, int64_t blocks, void* stream);
int launch_grad_join(const GradArgs& a, int gdt, bool vec, int64_t blocks, void* stream);
int launch_dropout(const DropoutArgs& a, int dt, int64_t blocks, void* stream);
int launch_logp(const LogpArgs& a, int dt, void* stream);
int launch_logp_join(const LogpArgs& a, int dt, void* stream);
int launch_dlogits(const LogpArgs& a, int dt, void* stream);
int launch_preference(const PrefArgs& a, void* stream);

// Elements of one access of the embedding kernels: 16 bytes of a 16-bit
// buffer, or four elements where an fp32 buffer takes part.
constexpr int vec_of(int a, int b) { return a == ZERO_F32 || b == ZERO_F32 ? 4 : 8; }
constexpr int kEmbedUnroll = 4;     // accesses per thread
constexpr int kEmbedThreads = 256;
constexpr int kDropoutThreads = 512;

}  // namespace ops
}  // namespace zk
