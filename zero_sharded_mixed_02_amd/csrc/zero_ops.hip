// zero_ops.hip -- gfx950 kernels of the vocabulary operators: embedding lookup
// and its gradient, dropout, token log-probabilities and the paired preference
// loss.
//
// None of them is a contraction: each reads its inputs once, does a few fp32
// operations per element and writes its outputs once, so HBM bounds the large
// calls and launch latency the small ones.  Rows start at any element offset
// (a table behind an odd-sized tensor, a vocabulary of odd size), so accesses
// are 16 bytes wide at element alignment, which gfx950 takes from global
// memory at any address; where a row's length is no multiple of an access, its
// last access is moved back to end with the row.
//
// Times below are on one MI355X, where a large copy moves 6.0 TB/s (read and
// written together) and a large read 7.1 TB/s: of single launches, after some
// tens of the same, or of whole calls where they say so.
//
// Floating point: compiled with -ffp-contract=off; fused multiply-adds are
// written out where they are meant.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "zero_internal.h"
#include "zero_ops.h"

#pragma clang fp contract(off)

namespace zk {
namespace ops {
namespace {

#define AS1 __attribute__((address_space(1)))

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
// The same at element alignment.
typedef uint32_t u32x4h __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2h __attribute__((ext_vector_type(2), aligned(2)));

constexpr float kLog2eHi = 1.44269504f;                                   // fp32(log2 e)
constexpr float kLog2eLo = (float)(1.4426950408889634 - (double)kLog2eHi);

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// ---------------------------------------------------------------------------
// Elements
// ---------------------------------------------------------------------------

template <int DT>
constexpr int es_of = DT == ZERO_F32 ? 4 : 2;

template <int DT>
__device__ __forceinline__ float widen(uint32_t h) {
  if constexpr (DT == ZERO_F32) return __uint_as_float(h);
  else if constexpr (DT == ZERO_BF16) return __uint_as_float(h << 16);
  else return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
}

// fp32 -> element, round to nearest even (the one rounding of every operator).
template <int DT>
__device__ __forceinline__ uint32_t narrow(float x) {
  if constexpr (DT == ZERO_F32) return __float_as_uint(x);
  else if constexpr (DT == ZERO_BF16) return __builtin_bit_cast(uint16_t, (__bf16)x);
  else return __builtin_bit_cast(uint16_t, (_Float16)x);
}

// N consecutive elements as they lie in memory.
template <int DT, int N>
struct Raw {
  static constexpr int kWords = N * es_of<DT> >= 4 ? N * es_of<DT> / 4 : 1;
  uint32_t w[kWords];
};

template <int DT, int N>
__device__ __forceinline__ uint64_t at(const void* base, int64_t e) {
  return (uint64_t)(uintptr_t)base + (uint64_t)(e * es_of<DT>);
}

template <int DT, int N, bool NT = false>
__device__ __forceinline__ Raw<DT, N> load(const void* base, int64_t e) {
  Raw<DT, N> r;
  const uint64_t p = at<DT, N>(base, e);
  constexpr int bytes = N * es_of<DT>;
  if constexpr (bytes == 2) {
    r.w[0] = *(const AS1 uint16_t*)p;
  } else if constexpr (bytes == 4) {
    r.w[0] = *(const AS1 uint32_t*)p;
  } else if constexpr (bytes == 8) {
    const u32x2 v = NT ? __builtin_nontemporal_load((const AS1 u32x2h*)p) : *(const AS1 u32x2h*)p;
    r.w[0] = v[0];
    r.w[1] = v[1];
  } else {
    static_assert(bytes == 16, "access size");
    const u32x4 v = NT ? __builtin_nontemporal_load((const AS1 u32x4h*)p) : *(const AS1 u32x4h*)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = v[i];
  }
  return r;
}

template <int DT, int N, bool NT = false>
__device__ __forceinline__ void store(void* base, int64_t e, const Raw<DT, N>& r) {
  const uint64_t p = at<DT, N>(base, e);
  constexpr int bytes = N * es_of<DT>;
  if constexpr (bytes == 2) {
    *(AS1 uint16_t*)p = (uint16_t)r.w[0];
  } else if constexpr (bytes == 4) {
    *(AS1 uint32_t*)p = r.w[0];
  } else if constexpr (bytes == 8) {
    const u32x2 v = {r.w[0], r.w[1]};
    if (NT) __builtin_nontemporal_store(v, (AS1 u32x2h*)p);
    else *(AS1 u32x2h*)p = v;
  } else {
    static_assert(bytes == 16, "access size");
    const u32x4 v = {r.w[0], r.w[1], r.w[2], r.w[3]};
    if (NT) __builtin_nontemporal_store(v, (AS1 u32x4h*)p);
    else *(AS1 u32x4h*)p = v;
  }
}

template <int DT, int N>
__device__ __forceinline__ void to_float(const Raw<DT, N>& r, float (&x)[N]) {
  if constexpr (DT == ZERO_F32 || N == 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = widen<DT>(r.w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      x[2 * i] = DT == ZERO_BF16 ? widen<DT>(r.w[i]) : widen<DT>(r.w[i] & 0xffffu);
      x[2 * i + 1] = DT == ZERO_BF16 ? __uint_as_float(r.w[i] & 0xffff0000u) : widen<DT>(r.w[i] >> 16);
    }
  }
}

template <int DT, int N>
__device__ __forceinline__ Raw<DT, N> from_float(const float (&x)[N]) {
  Raw<DT, N> r;
  if constexpr (DT == ZERO_F32 || N == 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) r.w[i] = narrow<DT>(x[i]);
  } else if constexpr (DT == ZERO_F16) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < N / 2; ++i)   // one conversion for both halves
      r.w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x[2 * i], x[2 * i + 1]}, f16x2));
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) r.w[i] = narrow<DT>(x[2 * i]) | (narrow<DT>(x[2 * i + 1]) << 16);
  }
  return r;
}

// Keeps the compiler from widening a row ahead of its use: all rows of a batch
// widened at once would take twice the registers.
template <int DT, int N>
__device__ __forceinline__ void pin(Raw<DT, N>& r) {
#pragma unroll
  for (int i = 0; i < Raw<DT, N>::kWords; ++i) asm volatile("" : "+v"(r.w[i]));
}

__device__ __forceinline__ int64_t load_id(const void* p, int64_t i, int wide) {
  return wide ? ((const AS1 int64_t*)(uintptr_t)p)[i] : (int64_t)((const AS1 int32_t*)(uintptr_t)p)[i];
}

// K ids at once: the loads are issued together, whichever their type.
template <int K>
__device__ __forceinline__ void load_ids(const void* p, const int64_t (&i)[K], int wide, int64_t (&id)[K]) {
  if (wide) {
#pragma unroll
    for (int k = 0; k < K; ++k) id[k] = ((const AS1 int64_t*)(uintptr_t)p)[i[k]];
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k) id[k] = ((const AS1 int32_t*)(uintptr_t)p)[i[k]];
  }
}

// The table row an id names, or `rows` for a padding id.
__device__ __forceinline__ int32_t row_of(int64_t id, int32_t rows) {
  return (uint64_t)id < (uint64_t)rows ? (int32_t)id : rows;
}

// ---------------------------------------------------------------------------
// Dropout's mask
// ---------------------------------------------------------------------------

// z ^ (z >> K) for K < 32, in 32-bit halves: gfx950 shifts 64 bits at a
// fraction of the rate.
template <int K>
__device__ __forceinline__ uint64_t xorshift(uint64_t z) {
  const uint32_t lo = (uint32_t)z, hi = (uint32_t)(z >> 32);
  const uint32_t l = lo ^ __builtin_amdgcn_alignbit(hi, lo, K), h = hi ^ (hi >> K);
  return ((uint64_t)h << 32) | l;
}

__device__ __forceinline__ uint64_t mix64(uint64_t z) {
  z = xorshift<30>(z) * kMix1;
  z = xorshift<27>(z) * kMix2;
  return xorshift<31>(z);
}

__device__ __forceinline__ uint64_t mask_key(const DropArgs& d) {
  return d.step_dev ? mix64((d.site_key ^ *(const AS1 uint64_t*)(uintptr_t)d.step_dev) + kGamma) : d.key;
}

// A mask from a position that the whole wave (or workgroup) shares: its word
// is found on the scalar unit, and the lanes add to it.
struct MaskBase {
  uint64_t z;        // state of the word that holds the shared position
  uint32_t sub;      // the position's place in that word, 0..3
};

__device__ __forceinline__ MaskBase mask_base(uint64_t key, int64_t position) {
  return MaskBase{key + (uint64_t)((position >> 2) + 1) * kGamma, (uint32_t)position & 3u};
}

// Zeroes the dropped ones among N elements, as they lie in memory, whose first
// stands `local` behind the shared position: before any arithmetic, so that
// what is dropped may hold anything.  One mix64 gives four elements 16 bits
// each, so a group that starts inside a word takes one word more and shifts.
// 16 bits an element and not 32 halve the generator's work, which is what
// dropout costs (a lookup of 65536 x 8192 fp16 takes 250 us without and 270
// with it); p is a multiple of 2^-16 for it.  Two draws are compared at once,
// beside the two 16-bit elements they decide on: draw - (cut - 1), held at 0
// below, is 0 for a dropped one, and at most 1 it is the factor of the
// element's bits (0 < cut < 65536; p = 1 drops everything without draws).
// ALIGNED: every group starts a word (the positions are multiples of 4).
template <int DT, int N, bool ALIGNED = false>
__device__ __forceinline__ void drop(Raw<DT, N>& r, const MaskBase& b, uint32_t local, uint32_t cut) {
  if (cut > 0xffffu) {
    r = Raw<DT, N>{};
    return;
  }
  const uint32_t p = b.sub + local;
  const uint64_t z = b.z + (uint64_t)(p >> 2) * kGamma;
  const uint32_t off = (p & 3u) * 16u;
  constexpr int W = (N + 3) / 4;
  uint64_t w[W];
#pragma unroll
  for (int i = 0; i < W; ++i) w[i] = mix64(z + (uint64_t)i * kGamma);
  if (!ALIGNED && off) {
    if constexpr (N > 1) {
      const uint64_t last = mix64(z + (uint64_t)W * kGamma);
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = (w[i] >> off) | ((i + 1 < W ? w[i + 1] : last) << (64 - off));
    } else {
      w[0] >>= off;
    }
  }
  if constexpr (DT != ZERO_F32 && N > 1) {
    const uint32_t below = (cut - 1) * 0x10001u;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const uint32_t draw = (uint32_t)(w[i / 2] >> (32 * (i % 2)));
      uint32_t keep;   // as instructions, since the compiler makes two compares and two selects of it
      asm("v_pk_sub_u16 %0, %1, %2 clamp" : "=v"(keep) : "v"(draw), "s"(below));
      asm("v_pk_min_u16 %0, %1, %2" : "=v"(keep) : "v"(keep), "s"(0x10001u));
      asm("v_pk_mul_lo_u16 %0, %1, %2" : "=v"(r.w[i]) : "v"(r.w[i]), "v"(keep));
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t half = (uint32_t)(w[i / 4] >> (32 * (i / 2 % 2)));
      const bool keep = i % 2 ? half >= (cut << 16) : (uint16_t)half >= (uint16_t)cut;
      r.w[i] = keep ? r.w[i] : 0;
    }
  }
}

// ---------------------------------------------------------------------------
// Embedding lookup
// ---------------------------------------------------------------------------

// t / upr for t < upr + kEmbedThreads * kEmbedUnroll: at most 1 where upr is that
// long, else by the reciprocal floor(2^32 / upr) + 1, exact since
// t * upr < 2^32 (0 stands for upr = 1).
__device__ __forceinline__ uint32_t row_in(uint32_t t, uint32_t upr, uint32_t magic) {
  if (upr > kEmbedThreads * kEmbedUnroll) return t >= upr;
  return magic ? __umulhi(t, magic) : t;
}

// y[i, :] = keep(i, :) * f * table[token[i], :].  A thread owns kEmbedUnroll
// accesses of N elements, kEmbedThreads accesses apart, numbered row by row
// through the output, so that every lane has work at any row length; their ids
// are loaded together, then their rows.  Bound by the output's stores beside
// row reads that the caches serve in part: 65536 rows of 8192 fp16 of skewed
// ids in 250 us, 1.07 GB written and 0.27 GB of different rows (5.4 TB/s; 270 us
// with dropout, and up to 350 some fifteen calls after a pause, while the clock
// dips).  Stores are non-temporal (8% there); one, two or eight
// accesses a thread take 343, 291 and 266 us, and walking the table in column
// tiles, for more hits in the L2, 268 us and more.
// DROP: 0 no dropout, 1 rows of whole accesses, so that the mask runs on with
// the accesses, each starting a word of it, 2 any.
template <int TDT, int ODT, int N, int DROP>
__global__ __launch_bounds__(kEmbedThreads) void embed_kernel(const EmbedArgs a) {
  const int64_t u0 = (int64_t)blockIdx.x * (kEmbedThreads * kEmbedUnroll);
  const int64_t row0 = u0 / a.upr;
  const uint32_t rem0 = (uint32_t)(u0 - row0 * a.upr);
  const int64_t left = a.n - row0;   // rows from here on
  MaskBase mask{};
  if constexpr (DROP == 1) {
    mask = mask_base(mask_key(a.drop), a.drop.first + u0 * N);
    mask.z += (uint64_t)(threadIdx.x * (N / 4)) * kGamma;
  } else if constexpr (DROP == 2) {
    mask = mask_base(mask_key(a.drop), a.drop.first + row0 * a.hidden);
  }
  void* const out = (char*)a.out + row0 * a.out_stride * es_of<ODT>;
  uint32_t row[kEmbedUnroll];             // behind row0
  int32_t col[kEmbedUnroll], id[kEmbedUnroll];
  int64_t where[kEmbedUnroll], token[kEmbedUnroll];
#pragma unroll
  for (int j = 0; j < kEmbedUnroll; ++j) {
    const uint32_t t = rem0 + j * kEmbedThreads + threadIdx.x;
    row[j] = row_in(t, (uint32_t)a.upr, a.magic);
    const int32_t c = (int32_t)(t - row[j] * (uint32_t)a.upr) * N;
    col[j] = c < a.hidden - N ? c : a.hidden - N;   // the last access ends with the row
    where[j] = row0 + (row[j] < left ? row[j] : 0);
  }
  load_ids(a.tokens, where, a.tok64, token);
#pragma unroll
  for (int j = 0; j < kEmbedUnroll; ++j) id[j] = row_of(token[j], a.rows);
  Raw<TDT, N> raw[kEmbedUnroll];
  if (a.rows > 0) {
#pragma unroll
    for (int j = 0; j < kEmbedUnroll; ++j)
      raw[j] = load<TDT, N>(a.table, (int64_t)((uint64_t)(uint32_t)(id[j] < a.rows ? id[j] : 0) * (uint32_t)a.hidden) + col[j]);
  } else {
#pragma unroll
    for (int j = 0; j < kEmbedUnroll; ++j) raw[j] = Raw<TDT, N>{};
  }
#pragma unroll
  for (int j = 0; j < kEmbedUnroll; ++j) {
    if (row[j] >= left) continue;
    if (id[j] >= a.rows) raw[j] = Raw<TDT, N>{};   // a padding id
    if constexpr (DROP == 1) {
      drop<TDT, N, true>(raw[j], MaskBase{mask.z + (uint64_t)(j * kEmbedThreads * (N / 4)) * kGamma, 0}, 0, a.drop.cut);
    } else if constexpr (DROP == 2) {
      if (a.drop.cut) drop<TDT, N>(raw[j], mask, row[j] * (uint32_t)a.hidden + col[j], a.drop.cut);
    }
    float x[N];
    to_float<TDT, N>(raw[j], x);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = x[i] * a.f;
    store<ODT, N, (N > 1)>(out, (int64_t)row[j] * a.out_stride + col[j], from_float<ODT, N>(x));
  }
}

// ---------------------------------------------------------------------------
// Token order
// ---------------------------------------------------------------------------

// Few positions: the place of position i is the number of positions whose
// (token, position) is smaller, counted outright: n^2 comparisons of one word
// that holds both, all over the chip, in one launch.  Bound by the comparisons
// (two instructions each): 2.8 us for 37 positions, 7.8 for 8192, where the
// radix passes below take 17.4; at twice as many it would lose.
__global__ __launch_bounds__(kRankThreads) void rank_kernel(const RankArgs a) {
  __shared__ uint4 word4[kSmallSort / 4];
  __shared__ int count[kRankItems];
  uint32_t* word = (uint32_t*)word4;
  constexpr int kSegs = kRankThreads / kRankItems;
  const int padded = (a.n + 4 * kSegs - 1) / (4 * kSegs) * (4 * kSegs);
  int64_t where[kSmallSort / kRankThreads], token[kSmallSort / kRankThreads];
#pragma unroll
  for (int k = 0; k < kSmallSort / kRankThreads; ++k) {
    const int i = k * kRankThreads + threadIdx.x;
    where[k] = i < a.n ? i : a.n - 1;
  }
  load_ids(a.tokens, where, a.tok64, token);
#pragma unroll
  for (int k = 0; k < kSmallSort / kRankThreads; ++k) {
    const int i = k * kRankThreads + threadIdx.x;
    if (i < padded)
      word[i] = i < a.n ? ((uint32_t)row_of(token[k], a.rows) << kSmallSortPosBits) | (uint32_t)i : 0xffffffffu;
  }
  if (threadIdx.x < kRankItems) count[threadIdx.x] = 0;
  __syncthreads();
  const int item = threadIdx.x % kRankItems, seg = threadIdx.x / kRankItems;
  const int i = blockIdx.x * kRankItems + item;
  const uint32_t mine = i < a.n ? word[i] : 0;
  const int len = padded / kSegs / 4;
  const uint4* w = word4 + seg * len;
  int c = 0;
#pragma unroll 4
  for (int j = 0; j < len; ++j) {
    const uint4 v = w[j];
    c += (v.x < mine) + (v.y < mine) + (v.z < mine) + (v.w < mine);
  }
  atomicAdd(&count[item], c);
  __syncthreads();
  if (threadIdx.x < kRankItems && i < a.n) {
    const int place = count[item];
    a.sorted[place] = (int32_t)(mine >> kSmallSortPosBits);
    a.order[place] = i;
  }
}

// K positions of a pass and their tokens, from index i on, 64 or more apart;
// past the end the last one.
template <int K>
__device__ __forceinline__ void radix_read(const RadixArgs& a, int64_t i, int step, int32_t (&key)[K], int32_t (&pos)[K]) {
  int64_t where[K];
#pragma unroll
  for (int k = 0; k < K; ++k) where[k] = i + k * step < a.n ? i + k * step : a.n - 1;
  if (a.first) {
    int64_t token[K];
    load_ids(a.tokens, where, a.tok64, token);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      key[k] = row_of(token[k], a.rows);
      pos[k] = (int32_t)where[k];
    }
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      key[k] = a.key_in[where[k]];
      pos[k] = a.pos_in[where[k]];
    }
  }
}

// One stable pass by `bits` bits of the token.  Each workgroup owns a run of
// tiles; this counts its digits.  A pass is bound by latency: 50257 tokens take
// two, 18 us for 65536 positions and 54 for 2^20.
__global__ __launch_bounds__(kSortThreads) void radix_count_kernel(const RadixArgs a) {
  __shared__ uint32_t bin[kBins];
  bin[threadIdx.x] = 0;
  __syncthreads();
  const uint32_t mask = (1u << a.bits) - 1;
  const int64_t lo = (int64_t)blockIdx.x * a.tiles_per_block * a.tile;
  int64_t hi = lo + a.tiles_per_block * a.tile;
  if (hi > a.n) hi = a.n;
  constexpr int K = 2;
  for (int64_t i = lo + threadIdx.x; i < hi; i += K * kSortThreads) {
    int32_t key[K], pos[K];
    radix_read(a, i, kSortThreads, key, pos);
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (i + k * kSortThreads < hi) atomicAdd(&bin[((uint32_t)key[k] >> a.shift) & mask], 1u);
  }
  __syncthreads();
  a.hist[(int64_t)blockIdx.x * kBins + threadIdx.x] = bin[threadIdx.x];
}

// ... and this moves its positions.  A digit's place is the count of smaller
// digits, plus the same digit in earlier workgroups, plus its rank in this
// one.  In a tile each wave owns 64 * KEYS consecutive positions and takes
// them 64 at a time: lanes of the same digit find each other with one ballot
// per bit, and rank themselves by lane, so equal tokens keep their order.
template <int KEYS>
__global__ __launch_bounds__(kSortThreads) void radix_move_kernel(const RadixArgs a) {
  constexpr int kWaves = kSortThreads / 64;
  __shared__ uint32_t base[kBins];               // next place of each digit
  __shared__ uint32_t scan[kWaves];
  __shared__ uint32_t cnt[kWaves][kBins];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  {
    uint32_t before = 0, total = 0;
#pragma unroll 32   // one latency for many workgroups' counts
    for (int b = 0; b < a.n_blocks; ++b) {
      const uint32_t h = a.hist[(int64_t)b * kBins + threadIdx.x];
      before += b < (int)blockIdx.x ? h : 0;
      total += h;
    }
    uint32_t inc = total;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t v = __shfl_up(inc, d);
      if (lane >= d) inc += v;
    }
    if (lane == 63) scan[wave] = inc;
    __syncthreads();
    uint32_t prev = 0;
    for (int w = 0; w < wave; ++w) prev += scan[w];
    base[threadIdx.x] = prev + inc - total + before;
  }
  const uint32_t mask = (1u << a.bits) - 1;
  const int64_t tile0 = (int64_t)blockIdx.x * a.tiles_per_block;
  for (int64_t t = 0; t < a.tiles_per_block; ++t) {
    const int64_t lo = (tile0 + t) * (kSortThreads * KEYS);
    if (lo >= a.n) break;   // uniform
#pragma unroll
    for (int w = 0; w < kWaves; ++w) cnt[w][threadIdx.x] = 0;
    __syncthreads();
    int32_t key[KEYS], pos[KEYS];
    uint32_t rank[KEYS];
    const int64_t first = lo + wave * (64 * KEYS) + lane;
    radix_read(a, first, 64, key, pos);
#pragma unroll
    for (int k = 0; k < KEYS; ++k) {
      const bool in = first + k * 64 < a.n;
      const uint32_t d = ((uint32_t)key[k] >> a.shift) & mask;
      uint64_t same = __ballot(in);
      for (int b = 0; b < a.bits; ++b) {
        const bool bit = (d >> b) & 1u;
        const uint64_t set = __ballot(bit);
        same &= bit ? set : ~set;
      }
      const uint32_t below = __popcll(same & ((1ull << lane) - 1));
      const uint32_t old = cnt[wave][d];
      rank[k] = old + below;
      __builtin_amdgcn_wave_barrier();
      __threadfence_block();
      if (in && below == 0) cnt[wave][d] = old + __popcll(same);
      __threadfence_block();
      __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    uint32_t run = base[threadIdx.x];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const uint32_t c = cnt[w][threadIdx.x];
      cnt[w][threadIdx.x] = run;
      run += c;
    }
    base[threadIdx.x] = run;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < KEYS; ++k) {
      if (first + k * 64 >= a.n) continue;
      const uint32_t d = ((uint32_t)key[k] >> a.shift) & mask;
      const int64_t place = (int64_t)cnt[wave][d] + rank[k];
      if (place < a.n) {
        a.key_out[place] = key[k];
        a.pos_out[place] = pos[k];
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Gradient of the table
// ---------------------------------------------------------------------------
//
// The positions in token order are cut into chunks of equal length, whatever
// their tokens, so that frequent tokens spread over as many waves as rare ones.
// A wave owns one chunk and one tile of columns and sums its runs of equal
// tokens in fp32 registers; for a slice with few chunks, up to four waves share
// the runs of one.  A run inside a chunk is finished there.  One that
// crosses a boundary leaves a partial row (fp32, in the workspace) in each
// chunk it touches: slot 2c of chunk c if it came in from the chunk before,
// slot 2c + 1 if it begins in c and goes on.  A workgroup's waves own
// neighbouring chunks: where one run passes through all of them, they add up
// their rows first, and slot 2c of the first holds the sum.  The join kernel
// adds the partial rows in order.  Further workgroups of the same launch write
// zeros to the rows that no token names.
//
// Bound by HBM at the large end: 65536 x 8192 bf16 with dropout into 50257 rows
// takes 369 us for 1.07 GB read and 0.85 GB written (5.2 TB/s) and 15 us for the
// join.  How often a token repeats hardly matters: 2^20 positions of 768 take
// 333 + 23 us evenly spread and 280 + 83 us all of one token.  At GPT-2-small's
// size (8192 x 768, 20 + 6 us) 77 MB of mostly zero rows and the latencies of search,
// gather and join count.

// First indices in [0, n) whose sorted token is >= key0 and >= key1 (n if
// none), found by a whole wave: both at once, 64 probes each at a time.
__device__ __forceinline__ void wave_lower_bounds(const int32_t* sorted, int64_t n, int64_t key0, int64_t key1,
                                                  int64_t& at0, int64_t& at1) {
  const int lane = threadIdx.x & 63;
  LowerBound search[2] = {{0, n}, {0, n}};
  const int64_t key[2] = {key0, key1};
  while (search[0].open() || search[1].open()) {
    int32_t probe[2];
    bool in[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int64_t i = search[k].probe(lane);
      in[k] = i < search[k].hi;
      probe[k] = sorted[in[k] ? i : 0];
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) search[k].narrow(__popcll(__ballot(in[k] && (int64_t)probe[k] < key[k])));
  }
  at0 = search[0].lo;
  at1 = search[1].lo;
}

__device__ __forceinline__ int64_t wave_lower_bound(const int32_t* sorted, int64_t n, int64_t key) {
  int64_t a, b;
  wave_lower_bounds(sorted, n, key, key, a, b);
  return a;
}

// Writes N columns of a finished row; `begin` is the first column that this
// lane owns (col < begin where its access was moved back: written twice with
// the same value, but added to dst once).
template <int GDT, int N>
__device__ __forceinline__ void write_row(const GradArgs& a, int32_t row, int32_t col, int32_t begin,
                                          const float (&sum)[N]) {
  const int64_t row_e = (int64_t)row * a.hidden, e = row_e + col;
  void* const dst = (char*)a.dst + (row_e - a.lo) * es_of<GDT>;   // of the row's first column
  if (e >= a.lo && e + N <= a.hi && (begin == col || !a.accumulate)) {
    float x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = sum[i] * a.f;
    if (a.accumulate) {
      float old[N];
      to_float<GDT, N>(load<GDT, N>(dst, col), old);
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = old[i] + x[i];
    }
    store<GDT, N, (N > 1)>(dst, col, from_float<GDT, N>(x));
    return;
  }
  bool mine[N];
  float old[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    mine[i] = col + i >= begin && e + i >= a.lo && e + i < a.hi;
    old[i] = 0.0f;
    if (mine[i] && a.accumulate) {
      float v[1];
      to_float<GDT, 1>(load<GDT, 1>(dst, col + i), v);
      old[i] = v[0];
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float x[1] = {a.accumulate ? old[i] + sum[i] * a.f : sum[i] * a.f};
    if (mine[i]) store<GDT, 1>(dst, col + i, from_float<GDT, 1>(x));
  }
}

template <int N>
__device__ __forceinline__ void write_part(const GradArgs& a, int64_t slot, int32_t col, const float (&sum)[N]) {
  const int64_t e = slot * a.hidden + col;
  if constexpr (N == 1) {
    store<ZERO_F32, 1>(a.part, e, from_float<ZERO_F32, 1>(sum));
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float x[4] = {sum[i], sum[i + 1], sum[i + 2], sum[i + 3]};
      store<ZERO_F32, 4>(a.part, e + i, from_float<ZERO_F32, 4>(x));
    }
  }
}

// Zero rows of one workgroup, behind the chunks in the grid: before them, or
// mixed with them, the whole is 4-12% slower (65536 x 8192).
template <int GDT>
__device__ void fill_rows(const GradArgs& a, int64_t block) {
  __shared__ uint8_t named[1024];
  constexpr int N = 16 / es_of<GDT>;
  const int64_t r0 = a.row_lo + block * a.fill_rows;
  int64_t r1 = r0 + a.fill_rows;
  if (r1 > a.row_hi) r1 = a.row_hi;
  int64_t from, to;
  wave_lower_bounds(a.sorted, a.n, r0, r1, from, to);
  if (to - from <= 2 * kGradThreads) {   // few positions: each marks its row
    for (int r = threadIdx.x; r < a.fill_rows; r += kGradThreads) named[r] = 0;
    __syncthreads();
    for (int64_t i = from + threadIdx.x; i < to; i += kGradThreads) {
      const int64_t r = a.sorted[i] - r0;
      if ((uint64_t)r < (uint64_t)a.fill_rows) named[r] = 1;
    }
  } else {                               // many, as where a token repeats: each row looks for one
    for (int64_t r = r0 + threadIdx.x; r < r1; r += kGradThreads) {
      int64_t lo = from, hi = to;
      while (lo < hi) {
        const int64_t mid = lo + (hi - lo) / 2;
        if (a.sorted[mid] < r) lo = mid + 1;
        else hi = mid;
      }
      named[r - r0] = lo < a.n && a.sorted[lo] == r;
    }
  }
  __syncthreads();
  const uint32_t upr = (uint32_t)(a.hidden + N - 1) / N;
  const uint32_t units = (uint32_t)(r1 - r0) * upr;   // fill_rows keeps this small
  for (uint32_t u = threadIdx.x; u < units; u += kGradThreads) {
    const uint32_t r = u / upr;
    if (named[r]) continue;
    const int64_t row_e = (r0 + r) * a.hidden;
    const int64_t e = row_e + (int64_t)(u - r * upr) * N;
    const int64_t end = row_e + a.hidden < e + N ? row_e + a.hidden : e + N;
    if (e + N <= end && e >= a.lo && e + N <= a.hi) {
      store<GDT, N, true>(a.dst, e - a.lo, Raw<GDT, N>{});
    } else {
      for (int64_t i = e; i < end; ++i)
        if (i >= a.lo && i < a.hi) store<GDT, 1>(a.dst, i - a.lo, Raw<GDT, 1>{});
    }
  }
}

// DROP: 0 no dropout, 1 every access starts a word of the mask, 2 any.
// NT: dy is read past the caches, which is faster where it exceeds the Infinity
// Cache (calls of 2^20 x 768: 408 us against 440, of 65536 x 8192: 403 against
// 415) and slower where it may sit there (32768 x 768: 55 against 48), as it does when the backward pass just wrote it.
template <int YDT, int GDT, int N, int DROP, bool NT>
__global__ __launch_bounds__(kGradThreads) void grad_kernel(const GradArgs a) {
  if ((int64_t)blockIdx.x >= a.chunk_blocks) {
    fill_rows<GDT>(a, (int64_t)blockIdx.x - a.chunk_blocks);
    return;
  }
  __shared__ float bounce[kGradChunks][64 * N];
  __shared__ int through[kGradChunks];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int64_t group = blockIdx.x / (uint32_t)a.tiles;
  const int64_t c = group * kGradChunks + wave;
  const uint32_t piece = (uint32_t)(blockIdx.x - group * a.tiles);
  const int32_t tile = (int32_t)(piece / (uint32_t)a.parts) * 64 * N;
  // Consecutive workgroups go to the XCDs in turn: the part changes with the
  // group, so that no XCD gets the parts where long runs begin alone.
  const int part = (int)((piece + (uint32_t)group) % (uint32_t)a.parts);
  const int32_t begin = tile + lane * N;
  const bool on = begin < a.hidden;
  const int32_t col = begin < a.hidden - N ? begin : a.hidden - N;
  float acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.0f;

  // Sums the wave's chunk; true if all of it belongs to a run that came in and
  // goes on, whose sum is then left in acc.
  auto sum_chunk = [&]() -> bool {
    // The chunk's tokens and positions, one a lane (a chunk has at most 64).
    const int64_t s = c * a.chunk;
    const int len = (int)(s + a.chunk < a.n ? a.chunk : a.n - s);
    const int64_t at = s + (lane < len ? lane : len - 1);
    const int32_t rows = a.sorted[at], from = a.order[at];
    const int32_t before = a.sorted[s > 0 ? s - 1 : 0], after = a.sorted[s + len < a.n ? s + len : 0];
    const int32_t poss = (uint32_t)from < (uint64_t)a.n ? from : -1;
    const uint64_t here = __ballot(lane < len && rows >= a.row_lo && rows < a.row_hi);
    if (!here) return false;
    int p0 = __builtin_ctzll(here), p1 = 64 - __builtin_clzll(here);   // what is written, in sorted rows
    const int32_t left_of = __shfl_up(rows, 1);   // by all lanes: a lane reads only from active ones
    const uint64_t starts = __ballot(lane > 0 && lane < len && rows != left_of);
    if (a.parts > 1) {
      const Span mine = runs_of_part(starts, p0, p1, a.chunk, a.parts, part);
      p0 = mine.lo;
      p1 = mine.hi;
      if (p0 >= p1) return false;
    }
    bool head = p0 == 0 && s > 0 && before == __builtin_amdgcn_readlane(rows, 0);   // came in from the chunk before
    const bool goes_on = p1 == len && s + len < a.n && after == __builtin_amdgcn_readlane(rows, len - 1);
    const bool whole_run = head && goes_on && !starts;
    const uint64_t key = DROP ? mask_key(a.drop) : 0;

    // Rows in a batch.  Eight gain under 1% where dy comes from HBM (2^20 x 768)
    // and lose 4% where it sits in the Infinity Cache (32768 x 768).
    constexpr int U = 4;
    auto fetch = [&](int q, Raw<YDT, N>& raw) {
      const int32_t pos = __builtin_amdgcn_readlane(poss, q < p1 ? q : p1 - 1);
      raw = load<YDT, N, NT>((const char*)a.dy + (int64_t)(pos < 0 ? 0 : pos) * a.dy_stride * es_of<YDT>, col);
    };
    Raw<YDT, N> cur[U], next[U];
#pragma unroll
    for (int u = 0; u < U; ++u) fetch(p0 + u, cur[u]);
    for (int b = p0; b < p1; b += U) {
      // The next positions' rows are on their way while these are summed.
      if (b + U < p1) {
#pragma unroll
        for (int u = 0; u < U; ++u) fetch(b + U + u, next[u]);
      }
      const int n = p1 - b < U ? p1 - b : U;
      int u0 = 0;
      while (u0 < n) {
        // The run of position b + u0 ends before `end`, in this batch or later.
        const uint64_t later = b + u0 < 63 ? starts >> (b + u0 + 1) << (b + u0 + 1) : 0;
        int end = later ? __builtin_ctzll(later) : p1;
        if (end > p1) end = p1;
        const int u1 = end - b < n ? end - b : n;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (u < u0 || u >= u1) continue;
          const int32_t pos = __builtin_amdgcn_readlane(poss, b + u);
          if (pos < 0) continue;
          float x[N];
          pin(cur[u]);
          if constexpr (DROP != 0)
            drop<YDT, N, DROP == 1>(cur[u], mask_base(key, a.drop.first + (int64_t)pos * a.hidden), (uint32_t)col,
                                    a.drop.cut);
          to_float<YDT, N>(cur[u], x);
#pragma unroll
          for (int i = 0; i < N; ++i) acc[i] += x[i];
        }
        u0 = u1;
        if (end - b > n) break;   // it goes on in the next batch
        if (whole_run) return true;
        const int32_t row = __builtin_amdgcn_readlane(rows, end - 1);
        const bool tail = end == p1 && goes_on;
        if (row >= a.row_lo && row < a.row_hi) {
          if (!on) {
          } else if (!head && !tail) {
            write_row<GDT, N>(a, row, col, begin, acc);
          } else {
            write_part<N>(a, 2 * c + (head ? 0 : 1), col, acc);
          }
        }
        head = false;
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = 0.0f;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) cur[u] = next[u];
    }
    return false;
  };
  const bool pass = c < a.n_chunks && sum_chunk();
  if (lane == 0) through[wave] = pass;
  __syncthreads();
  bool all = true;
#pragma unroll
  for (int w = 0; w < kGradChunks; ++w) all &= through[w] != 0;
  if (!all) {
    if (pass && on) write_part<N>(a, 2 * c, col, acc);
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) bounce[wave][lane * N + i] = acc[i];
  __syncthreads();
  if (wave == 0 && on) {
#pragma unroll
    for (int w = 1; w < kGradChunks; ++w)
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] += bounce[w][lane * N + i];
    write_part<N>(a, 2 * c, col, acc);
  }
}

// Joins runs that cross chunk boundaries: their partial rows in chunk order.
// A workgroup looks after the runs that begin in kJoinChunks chunks, for one
// tile of columns.  A lane each finds out which chunks have one; short runs go
// to a wave each, and long ones (64 chunks and more) are cut into one piece a
// wave, joined in order in shared memory.  Bound by latency: 6 us after 8192 x
// 768, 15 after 65536 x 8192.
template <int GDT, int N>
__global__ __launch_bounds__(kJoinThreads) void grad_join_kernel(const GradArgs a) {
  constexpr int kWaves = kJoinThreads / 64;
  __shared__ float piece[kWaves][64 * N];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int64_t group = blockIdx.x / (uint32_t)a.join_tiles;
  const int32_t begin = ((int32_t)(blockIdx.x - group * a.join_tiles) * 64 + lane) * N;
  const bool on = begin < a.hidden;
  const int32_t col = begin < a.hidden - N ? begin : a.hidden - N;

  const int64_t c0 = group * kJoinChunks;
  const int64_t mine = c0 + lane, s = mine * a.chunk, e = s + a.chunk;
  const int64_t next = e + a.chunk, far = e + (int64_t)kJoinLong * a.chunk;
  const int64_t end = a.n - 1;
  const bool look = lane < kJoinChunks && e < a.n;
  // One latency for all five.
  const int32_t before = a.sorted[look && s > 0 ? s - 1 : 0], row = a.sorted[look ? e - 1 : 0],
                after = a.sorted[look ? e : 0], third = a.sorted[look && next < a.n ? next : end],
                last = a.sorted[look && far < a.n ? far : end];
  const bool has = look && after == row && row >= a.row_lo && row < a.row_hi && !(s > 0 && before == row);
  const bool more = has && next < a.n && third == row;   // it comes into a third chunk
  const bool lots = has && far < a.n && last == row;
  const uint64_t runs = __ballot(has), many = __ballot(more), longs = __ballot(lots);

  // The partial rows of the run from chunk c to chunk l: the one of c, single
  // chunks up to a group that it passes through, such groups, single chunks.
  struct Run {
    int64_t c, first, groups, group0, rest0, count;
  };
  auto run_of = [&](int64_t c, int64_t l) {
    const int64_t g0 = (c + kGradChunks) / kGradChunks, g1 = l / kGradChunks;   // groups [g0, g1)
    Run r;
    r.c = c;
    r.groups = g1 > g0 ? g1 - g0 : 0;
    r.first = r.groups ? g0 * kGradChunks - (c + 1) : l - c;
    r.group0 = g0 * kGradChunks;
    r.rest0 = g1 * kGradChunks;
    r.count = 1 + r.first + r.groups + (r.groups ? l - r.rest0 + 1 : 0);
    return r;
  };
  // Sums its partial rows [j0, j1).
  auto sum = [&](const Run& run, int64_t j0, int64_t j1, float (&acc)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.0f;
    if (!on) return;
#pragma unroll 8
    for (int64_t j = j0; j < j1; ++j) {
      const int64_t k = j - 1 - run.first;
      const int64_t chunk = k < 0 ? run.c + j : k < run.groups ? run.group0 + k * kGradChunks : run.rest0 + (k - run.groups);
      const int64_t slot = 2 * chunk + (j == 0);
      float x[N];
      to_float<ZERO_F32, N>(load<ZERO_F32, N>(a.part, slot * a.hidden + col), x);
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] += x[i];
    }
  };
  auto last_chunk = [&](int64_t c, int32_t r) {   // of the run of row r
    const int64_t l = (wave_lower_bound(a.sorted, a.n, (int64_t)r + 1) - 1) / a.chunk;
    return l > c ? l : c;
  };
  int k = 0;
  for (uint64_t left = runs & ~longs; left; left &= left - 1, ++k) {
    if (k % kWaves != wave) continue;
    const int l = __builtin_ctzll(left);
    const int64_t c = c0 + l;
    const int32_t r = __builtin_amdgcn_readlane(row, l);
    const Run run = run_of(c, (many >> l) & 1 ? last_chunk(c, r) : c + 1);
    float acc[N];
    sum(run, 0, run.count, acc);
    if (on) write_row<GDT, N>(a, r, col, begin, acc);
  }
  for (uint64_t left = longs; left; left &= left - 1) {   // the same in every wave
    const int l = __builtin_ctzll(left);
    const int64_t c = c0 + l;
    const int32_t r = __builtin_amdgcn_readlane(row, l);
    const Run run = run_of(c, last_chunk(c, r));
    const int64_t per = (run.count + kWaves - 1) / kWaves, j0 = wave * per;
    float acc[N];
    sum(run, j0, j0 + per < run.count ? j0 + per : run.count, acc);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) piece[wave][lane * N + i] = acc[i];
    __syncthreads();
    if (wave == 0) {
      for (int v = 1; v < kWaves; ++v)
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] += piece[v][lane * N + i];
      if (on) write_row<GDT, N>(a, r, col, begin, acc);
    }
  }
}

// ---------------------------------------------------------------------------
// Dropout
// ---------------------------------------------------------------------------

template <int DT, int N>
__device__ __forceinline__ void dropout_one(const DropoutArgs& a, const MaskBase& mask, int64_t e0, uint32_t local,
                                            Raw<DT, N> xr, const Raw<DT, N>& rr) {
  const int64_t e = e0 + local;
  if (a.drop.cut) drop<DT, N>(xr, mask, local, a.drop.cut);
  float x[N];
  to_float<DT, N>(xr, x);
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = x[i] * a.f;   // 1 where nothing is dropped
  if (a.residual) {
    float r[N];
    to_float<DT, N>(rr, r);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = r[i] + x[i];
  }
  store<DT, N, (N > 1)>(a.out, e, from_float<DT, N>(x));
}

// out = residual + keep * f * x, one access a thread: short workgroups keep
// loads and stores flowing side by side.  Bound by HBM: 2^26 bf16 elements with a
// residual in 62 us (6.5 TB/s); 65 at two accesses a thread, 69 at four, 75
// with cached accesses.
template <int DT, int N>
__global__ __launch_bounds__(kDropoutThreads) void dropout_kernel(const DropoutArgs a) {
  const int64_t e0 = (int64_t)blockIdx.x * (kDropoutThreads * N);   // first element of the workgroup
  const MaskBase mask = a.drop.cut ? mask_base(mask_key(a.drop), a.drop.first + e0) : MaskBase{};
  const int64_t left = a.n - e0;
  const uint32_t e = threadIdx.x * N;
  if ((int64_t)e + N <= left) {
    dropout_one<DT, N>(a, mask, e0, e, load<DT, N, true>(a.x, e0 + e),
                       a.residual ? load<DT, N, true>(a.residual, e0 + e) : Raw<DT, N>{});
    return;
  }
  for (uint32_t i = e; i < left; ++i)   // fewer than N, in one thread
    dropout_one<DT, 1>(a, mask, e0, i, load<DT, 1>(a.x, e0 + i),
                       a.residual ? load<DT, 1>(a.residual, e0 + i) : Raw<DT, 1>{});
}

// ---------------------------------------------------------------------------
// Token log-probabilities
// ---------------------------------------------------------------------------

// exp(z) for z <= 0 as 2^(z log2 e), log2 e in two parts: with the leading
// part alone every term of a sum over the vocabulary would be off the same
// way, by 1.3e-8 |z|.
__device__ __forceinline__ float exp_of(float z) {
  return __builtin_amdgcn_exp2f(__builtin_fmaf(z, kLog2eHi, z * kLog2eLo));
}

// A running maximum and the sum of exp(x - max), extended by K values.  The
// maximum of nothing is -inf; it is not subtracted while it is (-inf - -inf).
template <int K>
__device__ __forceinline__ void absorb(const float (&x)[K], float& m, float& s) {
  float top = x[0];
#pragma unroll
  for (int i = 1; i < K; ++i) top = __builtin_fmaxf(top, x[i]);
  if (top > m) {
    s = s * exp_of(m - top);
    m = top;
  }
  const float base = m == neg_inf() ? 0.0f : m;
  float part = 0.0f;
#pragma unroll
  for (int i = 0; i < K; ++i) part += exp_of(x[i] - base);
  s += part;
}

// s of maximum m, as a share of the sum over the maximum top >= m.
__device__ __forceinline__ float rebase(float m, float s, float top) {
  return m == top || m == neg_inf() ? s : s * exp_of(m - top);
}

// Reduces (m, s) over the workgroup, in a fixed order; valid in thread 0.
template <int THREADS>
__device__ __forceinline__ void reduce_stats(float& m, float& s) {
  constexpr int kWaves = THREADS / 64;
  __shared__ float sm[kWaves], ss[kWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float top = m;
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, d));
  s = rebase(m, s, top);
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
  if (lane == 0) {
    sm[wave] = top;
    ss[wave] = s;
  }
  __syncthreads();
  m = sm[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) m = __builtin_fmaxf(m, sm[w]);
  s = 0.0f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) s += rebase(sm[w], ss[w], m);
}

// exp(z) for z <= 0 to 3 * 2^-24 of itself, however far down: fp32's
// exponential takes the fraction of z log2 e, and a double its whole part.
__device__ __forceinline__ double far_exp(double z) {
  if (z < -10000.0) return 0.0;
  const double t = z * 1.4426950408889634, k = rint(t);
  return ldexp((double)__builtin_amdgcn_exp2f((float)(t - k)), (int)k);
}

// Statistics and log-probability of a row from its label's logit y and from
// the maximum m and the sum s of exp(x - m) over the other logits.  Kept apart,
// since a likely label's term would drown them: with y at the top, the log of
// the sum is log(1 + rest), right in its last bits however small the rest.
template <int DT>
__device__ __forceinline__ void write_stats(const LogpArgs& a, int64_t t, const Raw<DT, 1>& logit, float m, float s) {
  const float y = widen<DT>(logit.w[0]), top = __builtin_fmaxf(m, y);
  const double gap = (double)y - (double)m, small = m == y ? 1.0 : far_exp(gap > 0 ? -gap : gap);
  const bool first = y >= m;
  const double rest = first ? (double)s * small : (double)s + small - 1.0;
  double ls = log(top == neg_inf() ? (double)s : 1.0 + rest);
  if (first && rest < 0x1p-20) ls = top == neg_inf() ? ls : rest - 0.5 * rest * rest;
  ls += first && top != neg_inf() ? (double)y - (double)top : 0.0;   // 0, or NaN where y is infinite
  a.stats[2 * t] = top;
  a.stats[2 * t + 1] = (float)ls;
  a.logp[t] = (float)(((double)y - (double)top) - ls);
}

// log softmax at the label, in one pass over the logits with a running maximum
// and sum in every thread.  One row, or one of `splits` pieces of a row, per
// workgroup.  Loads are aligned: the elements before the first 16-byte boundary
// of the row and behind the last one are taken singly.  Bound by HBM: 12288 scored
// rows of 131072 bf16 in 467 us (6.9 TB/s), 6144 of 50257 in 97 us (6.4 TB/s).
// Loads past the caches gain 10% at the large end; the last kCachedBytes of
// rows go through them, for the gradient that may follow.
template <int DT, int THREADS>
__global__ __launch_bounds__(THREADS) void logp_kernel(const LogpArgs a) {
  constexpr int N = 16 / es_of<DT>;
  constexpr int U = 2;
  const int64_t t = blockIdx.x / (uint32_t)a.splits;
  const int part = (int)(blockIdx.x - (uint32_t)t * (uint32_t)a.splits);
  const int64_t label = load_id(a.labels, t, a.lab64);
  if ((uint64_t)label >= (uint64_t)a.vocab) {
    if (part == 0 && threadIdx.x == 0) {
      a.stats[2 * t] = a.stats[2 * t + 1] = 0.0f;
      a.logp[t] = 0.0f;
    }
    return;
  }
  const int64_t row = t * a.stride;
  const uint32_t skew = (uint32_t)(at<DT, 1>(a.logits, row) & 15u);
  int head = skew ? (int)(16 - skew) / es_of<DT> : 0;
  if (head > a.vocab) head = a.vocab;
  const int vecs = (a.vocab - head) / N;
  const int tail = a.vocab - head - vecs * N;
  const int per = (vecs + a.splits - 1) / a.splits;
  const int v0 = part * per;
  const int v1 = v0 + per < vecs ? v0 + per : vecs;
  float m = neg_inf(), s = 0.0f;   // of all but the label: see write_stats
  const int tid = threadIdx.x;
  const Raw<DT, 1> logit = load<DT, 1>(a.logits, row + label);   // on its way while the rest is read
  const int lab = (int)label - head, lab_vec = lab >= 0 ? lab / N : -1, lab_in = lab % N;   // its access, its place there
  auto without_label = [&](float* x) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = i == lab_in ? neg_inf() : x[i];
  };
  // The step of the workgroup's accesses that meets it.
  const int lab_step = lab_vec < v0 ? -1 : v0 + (lab_vec - v0) / (U * THREADS) * (U * THREADS);
  int v = v0;
  auto stream = [&](auto nt) {
    for (; v + U * THREADS <= v1; v += U * THREADS) {
      float x[U * N];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        float y[N];
        to_float<DT, N>(load<DT, N, decltype(nt)::value>(a.logits, row + head + (int64_t)(v + j * THREADS + tid) * N), y);
#pragma unroll
        for (int i = 0; i < N; ++i) x[j * N + i] = y[i];
      }
      if (v == lab_step) {   // uniform
#pragma unroll
        for (int j = 0; j < U; ++j)
          if (v + j * THREADS + tid == lab_vec) without_label(x + j * N);
      }
      absorb<U * N>(x, m, s);
    }
  };
  if (t < a.cached_from) stream(std::true_type{});
  else stream(std::false_type{});
  for (v += tid; v < v1; v += THREADS) {
    float x[N];
    to_float<DT, N>(load<DT, N>(a.logits, row + head + (int64_t)v * N), x);
    if (v == lab_vec) without_label(x);
    absorb<N>(x, m, s);
  }
  if (part == 0 && tid < head && tid != (int)label) {
    float x[1];
    to_float<DT, 1>(load<DT, 1>(a.logits, row + tid), x);
    absorb<1>(x, m, s);
  }
  if (part == a.splits - 1 && tid < tail && a.vocab - tail + tid != (int)label) {
    float x[1];
    to_float<DT, 1>(load<DT, 1>(a.logits, row + a.vocab - tail + tid), x);
    absorb<1>(x, m, s);
  }
  reduce_stats<THREADS>(m, s);
  if (tid != 0) return;
  if (a.splits > 1) {
    a.part[2 * (int64_t)blockIdx.x] = m;
    a.part[2 * (int64_t)blockIdx.x + 1] = s;
  } else {
    write_stats<DT>(a, t, logit, m, s);
  }
}

// Joins the pieces of each row: one thread per row.
template <int DT>
__global__ __launch_bounds__(64) void logp_join_kernel(const LogpArgs a) {
  const int64_t t = (int64_t)blockIdx.x * 64 + threadIdx.x;
  if (t >= a.n) return;
  const int64_t label = load_id(a.labels, t, a.lab64);
  if ((uint64_t)label >= (uint64_t)a.vocab) return;   // written by logp_kernel
  const float* p = a.part + 2 * t * a.splits;
  const Raw<DT, 1> logit = load<DT, 1>(a.logits, t * a.stride + label);
  float m = neg_inf();
  for (int k = 0; k < a.splits; ++k) m = __builtin_fmaxf(m, p[2 * k]);
  float s = 0.0f;
  for (int k = 0; k < a.splits; ++k) s += rebase(p[2 * k], p[2 * k + 1], m);
  write_stats<DT>(a, t, logit, m, s);
}

// Gradient of the logits, coef (onehot - softmax): one piece of a row per
// workgroup, the last rows first.  Bound by HBM: 16384 rows of 131072 bf16, 12288 of
// them scored, in 1162 us for 7.5 GB (6.5 TB/s).  Short workgroups do best: with
// the forward pass 1636 us at 128 threads of two accesses, 1689 at 256, 1748 at
// four accesses, 1898 at one; cached stores cost another 3%.
template <int DT>
__global__ __launch_bounds__(kDlogitsThreads) void dlogits_kernel(const LogpArgs a) {
  constexpr int N = 16 / es_of<DT>;
  constexpr int U = kDlogitsUnroll;
  const uint32_t back = blockIdx.x / (uint32_t)a.splits;
  const int64_t t = a.n - 1 - back;   // last rows first: see kCachedBytes
  const int part = (int)(blockIdx.x - back * (uint32_t)a.splits);
  const int64_t label = load_id(a.labels, t, a.lab64);
  const float c = a.coef[t], m = a.stats[2 * t], ls = a.stats[2 * t + 1];
  const float coef = (uint64_t)label < (uint64_t)a.vocab ? c : 0.0f;
  const bool zero = coef == 0.0f;   // uniform over the workgroup
  const int64_t row = t * a.stride, drow = t * a.dl_stride;
  const uint32_t skew = (uint32_t)(at<DT, 1>(a.logits, row) & 15u);
  int head = skew ? (int)(16 - skew) / es_of<DT> : 0;
  if (head > a.vocab) head = a.vocab;
  const int vecs = (a.vocab - head) / N;
  const int tail = a.vocab - head - vecs * N;
  const int per = (vecs + a.splits - 1) / a.splits;
  const int v0 = part * per;
  const int v1 = v0 + per < vecs ? v0 + per : vecs;
  const int tid = threadIdx.x;
  const int lab = zero ? -1 : (int)label;
  auto grad = [&](float x) { return zero ? 0.0f : -coef * exp_of((x - m) - ls); };
  // 1 - p of the label, which keeps its bits where p is close to 1.
  auto label_grad = [&](float x) { return coef * -expm1f((x - m) - ls); };
  auto one = [&](int j) {
    float x[1] = {0.0f};
    if (!zero) to_float<DT, 1>(load<DT, 1>(a.logits, row + j), x);
    x[0] = j == lab ? label_grad(x[0]) : grad(x[0]);
    store<DT, 1>(a.dlogits, drow + j, from_float<DT, 1>(x));
  };
  for (int v = v0 + tid; v < v1; v += U * kDlogitsThreads) {
    Raw<DT, N> raw[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      raw[j] = Raw<DT, N>{};
      const int u = v + j * kDlogitsThreads;
      if (!zero) raw[j] = load<DT, N, true>(a.logits, row + head + (int64_t)(u < v1 ? u : v) * N);
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int u = v + j * kDlogitsThreads;
      if (u >= v1) continue;
      float x[N];
      to_float<DT, N>(raw[j], x);
      const int at0 = head + u * N;
      const bool has = (uint32_t)(lab - at0) < (uint32_t)N;
      float hot = 0.0f;
      if (has) {
#pragma unroll
        for (int i = 0; i < N; ++i) hot = at0 + i == lab ? x[i] : hot;
        hot = label_grad(hot);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = has && at0 + i == lab ? hot : grad(x[i]);
      store<DT, N, true>(a.dlogits, drow + at0, from_float<DT, N>(x));
    }
  }
  if (part == 0 && tid < head) one(tid);
  if (part == a.splits - 1 && tid < tail) one(a.vocab - tail + tid);
}

// ---------------------------------------------------------------------------
// Paired preference loss
// ---------------------------------------------------------------------------

__device__ __forceinline__ int64_t row_limit(const PrefArgs& a, int64_t i, int64_t floor_) {
  int64_t v = load_id(a.offsets, i, a.off64);
  if (v > a.n) v = a.n;
  return v < floor_ ? floor_ : v;
}

__device__ __forceinline__ bool counts(const PrefArgs& a, int64_t t) {
  return !a.labels || (uint64_t)load_id(a.labels, t, a.lab64) < (uint64_t)a.vocab;
}

// Lane's share of the sum over a sequence's scored rows, fp64.  What a row
// holds is loaded before it is known to count, so that the loads of U rows
// share one latency.
template <int THREADS>
__device__ __forceinline__ double sum_rows(const PrefArgs& a, int64_t lo, int64_t hi, int tid) {
  constexpr int U = THREADS == 64 ? 8 : 2;
  double s = 0.0;
  for (int64_t t0 = lo + tid; t0 < hi; t0 += U * THREADS) {
    float lp[U], ref[U];
    bool in[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + u * THREADS, at = t < hi ? t : t0;
      lp[u] = a.logp[at];
      ref[u] = a.ref ? a.ref[at] : 0.0f;
      in[u] = counts(a, at) && t < hi;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) s += in[u] ? (double)lp[u] - (double)ref[u] : 0.0;
  }
  return s;
}

__device__ __forceinline__ double wave_sum(double s) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
  return s;
}

// Loss and slope of a pair with difference h; one exponential serves both:
// with t = exp(-|h|), sigmoid is 1 / (1 + t) on one side and t / (1 + t) on
// the other, and -log sigmoid(h) = log(1 + t) + max(-h, 0).
struct Pair {
  double loss;
  float coef;
};

__device__ __forceinline__ Pair pair_of(const PrefArgs& a, double h) {
  const double t = exp(-fabs(h)), soft = log1p(t);
  const double big = 1.0 / (1.0 + t), small = t / (1.0 + t);
  const double sig = h >= 0 ? big : small, sig_neg = h >= 0 ? small : big;
  const double up = soft + (h < 0 ? -h : 0.0), down = soft + (h > 0 ? h : 0.0);
  Pair p;
  p.loss = (a.smoothing < 1 ? (1.0 - a.smoothing) * up : 0.0) + (a.smoothing > 0 ? a.smoothing * down : 0.0);
  p.coef = (float)(a.slope * (a.smoothing * sig - (1.0 - a.smoothing) * sig_neg));
  return p;
}

template <int THREADS>
__device__ __forceinline__ void write_coef(const PrefArgs& a, int64_t lo, int64_t hi, int tid, float coef) {
#pragma unroll 4
  for (int64_t t = lo + tid; t < hi; t += THREADS) a.coef[t] = counts(a, t) ? coef : 0.0f;
}

// Rows in no sequence.
template <int THREADS>
__device__ __forceinline__ void write_outside(const PrefArgs& a, int tid) {
  const int64_t lo = a.n_pairs ? row_limit(a, 0, 0) : a.n;
  const int64_t hi = a.n_pairs ? row_limit(a, 2 * a.n_pairs, lo) : a.n;
  for (int64_t t = tid; t < lo; t += THREADS) a.coef[t] = 0.0f;
  for (int64_t t = hi + tid; t < a.n; t += THREADS) a.coef[t] = 0.0f;
}

// A pair per workgroup, half of it for each sequence; one more workgroup, in
// the launch of the last pairs, writes the rows in no sequence.
__global__ __launch_bounds__(kPrefThreads) void preference_kernel(const PrefArgs a) {
  constexpr int kHalf = kPrefThreads / 2;
  __shared__ double part[kPrefThreads / 64];
  const int64_t i = a.pair0 + blockIdx.x;
  const int tid = threadIdx.x;
  if (i == a.n_pairs) {
    write_outside<kPrefThreads>(a, tid);
    return;
  }
  const int side = tid / kHalf;   // 0 chosen, 1 rejected
  const int64_t seq = i + side * a.n_pairs;
  const int64_t lo = row_limit(a, seq, 0), hi = row_limit(a, seq + 1, lo);
  const double s = wave_sum(sum_rows<kHalf>(a, lo, hi, tid % kHalf));
  if (tid % 64 == 0) part[tid / 64] = s;
  __syncthreads();
  double chosen = 0.0, rejected = 0.0;
#pragma unroll
  for (int w = 0; w < kHalf / 64; ++w) {
    chosen += part[w];
    rejected += part[kHalf / 64 + w];
  }
  chosen *= a.beta;
  rejected *= a.beta;
  const Pair p = pair_of(a, chosen - rejected);
  if (tid == 0) {
    a.rewards[i] = (float)chosen;
    a.rewards[a.n_pairs + i] = (float)rejected;
    a.pair_loss[i] = (float)p.loss;
  }
  write_coef<kHalf>(a, lo, hi, tid % kHalf, side ? -p.coef : p.coef);
}

__global__ __launch_bounds__(64) void mean_kernel(const PrefArgs a) {
  double s = 0.0;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < a.n_pairs; i += 64) s += (double)a.pair_loss[i];
  s = wave_sum(s);
  if (threadIdx.x == 0) a.loss[0] = a.n_pairs ? (float)(s / (double)a.n_pairs) : 0.0f;
}

// Few pairs of few rows: all of it in one workgroup and one launch, a wave per
// sequence (see kPrefSmallRows).
__global__ __launch_bounds__(kPrefThreads) void preference_small_kernel(const PrefArgs a) {
  __shared__ double reward[2 * kPrefSmallPairs];
  __shared__ float coef[kPrefSmallPairs], loss[kPrefSmallPairs];
  constexpr int kWaves = kPrefThreads / 64;
  const int wave = threadIdx.x / 64, lane = threadIdx.x % 64, tid = threadIdx.x;
  const int pairs = (int)a.n_pairs;
  for (int seq = wave; seq < 2 * pairs; seq += kWaves) {
    const int64_t lo = row_limit(a, seq, 0), hi = row_limit(a, seq + 1, lo);
    const double s = a.beta * wave_sum(sum_rows<64>(a, lo, hi, lane));
    if (lane == 0) {
      reward[seq] = s;
      a.rewards[seq] = (float)s;
    }
  }
  __syncthreads();
  if (tid < pairs) {
    const Pair p = pair_of(a, reward[tid] - reward[pairs + tid]);
    coef[tid] = p.coef;
    loss[tid] = (float)p.loss;
    a.pair_loss[tid] = (float)p.loss;
  }
  __syncthreads();
  for (int seq = wave; seq < 2 * pairs; seq += kWaves) {
    const int64_t lo = row_limit(a, seq, 0), hi = row_limit(a, seq + 1, lo);
    write_coef<64>(a, lo, hi, lane, seq < pairs ? coef[seq] : -coef[seq - pairs]);
  }
  write_outside<kPrefThreads>(a, tid);
  if (tid == 0) {
    double s = 0.0;
    for (int i = 0; i < pairs; ++i) s += (double)loss[i];
    a.loss[0] = pairs ? (float)(s / (double)pairs) : 0.0f;
  }
}

// ---------------------------------------------------------------------------
// Launch
// ---------------------------------------------------------------------------

template <typename F>
int by_type(int dt, F f) {
  switch (dt) {
    case ZERO_F32: return f(std::integral_constant<int, ZERO_F32>{});
    case ZERO_F16: return f(std::integral_constant<int, ZERO_F16>{});
    default: return f(std::integral_constant<int, ZERO_BF16>{});
  }
}

// The launch's own error, and none that an earlier call of the program left.
template <typename Args>
int launch(void (*kernel)(Args), int64_t blocks, int threads, const Args& a, void* stream) {
  void* args[] = {const_cast<void*>((const void*)&a)};
  return (int)hipLaunchKernel((const void*)kernel, dim3((uint32_t)blocks), dim3((uint32_t)threads), args, 0,
                              (hipStream_t)stream);
}

}  // namespace

int launch_embed(const EmbedArgs& a, int tdt, int odt, bool vec, int64_t blocks, void* stream) {
  return by_type(tdt, [&](auto T) {
    return by_type(odt, [&](auto O) {
      constexpr int t = decltype(T)::value, o = decltype(O)::value, n = vec_of(t, o);
      auto kernel = embed_kernel<t, o, n, 2>;
      if (!vec) kernel = embed_kernel<t, o, 1, 2>;   // p = 0 keeps all
      else if (!a.drop.cut) kernel = embed_kernel<t, o, n, 0>;
      else if (a.hidden % n == 0 && a.drop.first % 4 == 0) kernel = embed_kernel<t, o, n, 1>;
      return launch(kernel, blocks, kEmbedThreads, a, stream);
    });
  });
}

int launch_rank(const RankArgs& a, int64_t blocks, void* stream) {
  return launch(rank_kernel, blocks, kRankThreads, a, stream);
}

int launch_radix(const RadixArgs& a, void* stream) {
  if (const int err = launch(radix_count_kernel, a.n_blocks, kSortThreads, a, stream)) return err;
  return launch(a.tile == kSortThreads * kSortKeysFew ? radix_move_kernel<kSortKeysFew> : radix_move_kernel<kSortKeysMany>,
                a.n_blocks, kSortThreads, a, stream);
}

int launch_grad(const GradArgs& a, int ydt, int gdt, int vec, int64_t blocks, void* stream) {
  return by_type(ydt, [&](auto Y) {
    return by_type(gdt, [&](auto G) {
      constexpr int y = decltype(Y)::value, g = decltype(G)::value;
      auto go = [&](auto N, auto NT) {
        constexpr int n = decltype(N)::value;
        constexpr bool nt = decltype(NT)::value;
        auto kernel = grad_kernel<y, g, n, 2, nt>;
        constexpr int whole_words = n > 1 ? 1 : 2;
        if (!a.drop.cut) kernel = grad_kernel<y, g, n, 0, nt>;
        else if (a.hidden % 4 == 0 && a.drop.first % 4 == 0) kernel = grad_kernel<y, g, n, whole_words, nt>;
        return launch(kernel, blocks, kGradThreads, a, stream);
      };
      auto wide = [&](auto N) { return a.stream_dy ? go(N, std::true_type{}) : go(N, std::false_type{}); };
      if (vec == 1) return go(std::integral_constant<int, 1>{}, std::false_type{});
      if constexpr (vec_of(y, g) == 8)
        if (vec == 8) return wide(std::integral_constant<int, 8>{});
      return wide(std::integral_constant<int, 4>{});
    });
  });
}

int launch_grad_join(const GradArgs& a, int gdt, bool vec, int64_t blocks, void* stream) {
  return by_type(gdt, [&](auto G) {
    constexpr int g = decltype(G)::value;
    return launch(vec ? grad_join_kernel<g, 4> : grad_join_kernel<g, 1>, blocks, kJoinThreads, a, stream);
  });
}

int launch_dropout(const DropoutArgs& a, int dt, int64_t blocks, void* stream) {
  return by_type(dt, [&](auto D) {
    constexpr int d = decltype(D)::value;
    return launch(dropout_kernel<d, vec_of(d, d)>, blocks, kDropoutThreads, a, stream);
  });
}

int launch_logp(const LogpArgs& a, int dt, void* stream) {
  return by_type(dt, [&](auto D) {
    constexpr int d = decltype(D)::value;
    return logp_threads(a.n, a.vocab) == 64 ? launch(logp_kernel<d, 64>, a.n * a.splits, 64, a, stream)
                                            : launch(logp_kernel<d, kLogpThreads>, a.n * a.splits, kLogpThreads, a, stream);
  });
}

int launch_logp_join(const LogpArgs& a, int dt, void* stream) {
  return by_type(dt, [&](auto D) {
    return launch(logp_join_kernel<decltype(D)::value>, (a.n + 63) / 64, 64, a, stream);
  });
}

int launch_dlogits(const LogpArgs& a, int dt, void* stream) {
  return by_type(dt, [&](auto D) {
    return launch(dlogits_kernel<decltype(D)::value>, a.n * a.splits, kDlogitsThreads, a, stream);
  });
}

int launch_preference(const PrefArgs& a, void* stream) {
  if (a.n_pairs <= kPrefSmallPairs && a.n <= kPrefSmallRows)
    return launch(preference_small_kernel, 1, kPrefThreads, a, stream);
  const bool last = a.pair0 + a.pair_count == a.n_pairs;
  if (const int err = launch(preference_kernel, a.pair_count + last, kPrefThreads, a, stream)) return err;
  return last ? launch(mean_kernel, 1, 64, a, stream) : 0;
}

}  // namespace ops
}  // namespace zk
