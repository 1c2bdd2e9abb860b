// zero_gemm.h -- the matrix-product core of the hidden-matrix operators:
// device templates, included by the .hip files that instantiate them.
//
// C[m, n] = sum_k A(m, k) B(n, k), A and B of 16-bit elements in one of two
// forms, sums in fp32 on the matrix units:
//   form K   the operand's memory rows run along k  (x and W of x W^T)
//   form M   the operand's memory rows run along m (or n), one row per k
//            (W of dz W; both operands of dz^T x)
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zero.h"

#pragma clang fp contract(off)

namespace zk {
namespace gemm {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

#define ZK_LDS __attribute__((address_space(3)))

enum Form : int { kFormK = 0, kFormM = 1 };

constexpr int kBK = 64;          // depth of a stage, elements

template <typename T>
__device__ __forceinline__ f32x4 mfma(s16x8 a, s16x8 b, f32x4 c);
template <>
__device__ __forceinline__ f32x4 mfma<_Float16>(s16x8 a, s16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
template <>
__device__ __forceinline__ f32x4 mfma<__bf16>(s16x8 a, s16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// XOR of a row's 16-byte units in LDS.  Form K: rows of 128 bytes; a fragment reads
// 16 consecutive rows at one unit, which with 64 banks then covers each bank once.
__device__ __forceinline__ int swz_k(int row) { return (row >> 1) & 7; }
// Form M: rows of W elements, one per k; a transposing read takes 32 bytes of
// each of four rows k .. k + 3 per 16 lanes, and of four rows 8 further on in the
// next 16.
template <int W>
__device__ __forceinline__ int swz_m(int k) {
  if constexpr (W >= 128) return ((k & 3) | (((k >> 3) & 1) << 2)) << 1;
  else return (((k >> 1) & 1) | (((k >> 3) & 1) << 1)) << 1;
}

// One operand's panel of W rows (of the product) and its staging.
template <int FORM, int W, int NT>
struct Panel {
  static constexpr int kBytes = W * kBK * 2;
  static constexpr int kLoads = W * 8 / NT;       // 16-byte units a thread
  static_assert(W * 8 % NT == 0, "the panel is a whole number of units a thread");

  const char* base;       // first element of the panel at the current k
  int64_t step;           // bytes from one stage to the next
  int64_t span;           // bytes of the panel from base on (form K), or of a row (form M)
  uint32_t ld;            // bytes between memory rows
  int rows;               // rows of the product left in this panel (may exceed W)
  int before;             // elements of a memory row before the panel
  uint32_t voff[kLoads];

  __device__ __forceinline__ void init(const void* p, int64_t lde, int row0, int rows_total, int k0, int k_end, int tid) {
    ld = (uint32_t)lde * 2u;
    rows = rows_total - row0;
    if constexpr (FORM == kFormK) {
      base = (const char*)p + (int64_t)row0 * lde * 2 + (int64_t)k0 * 2;
      step = kBK * 2;
      before = k0;
      const int last = (rows < W ? rows : W) - 1;
      span = (int64_t)last * lde * 2 + (int64_t)(k_end - k0) * 2;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int g = i * NT + tid, row = g >> 3, unit = (g & 7) ^ swz_k(row);
        voff[i] = (uint32_t)(row < last ? row : last) * ld + unit * 16u;
      }
    } else {
      base = (const char*)p + (int64_t)k0 * lde * 2 + (int64_t)row0 * 2;
      step = (int64_t)kBK * lde * 2;
      span = (int64_t)(rows + (rows & 1)) * 2;      // whole words: the row is even, or padded
      before = row0;
      constexpr int U = W / 8;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int g = i * NT + tid, k = g / U, unit = (g % U) ^ swz_m<W>(k);
        voff[i] = (uint32_t)k * ld + unit * 16u;
      }
    }
  }

  // Bytes of this stage that may be read: what lies behind reads as zero.
  __device__ __forceinline__ uint32_t records(int k_left) const {
    if (k_left <= 0) return 0;
    if constexpr (FORM == kFormK) return (uint32_t)span;
    const int kr = k_left < kBK ? k_left : kBK;
    return (uint32_t)(kr - 1) * ld + (uint32_t)span;
  }

  __device__ __forceinline__ void advance() {
    base += step;
    if constexpr (FORM == kFormK) span -= step;
  }

  // Starts load i of a stage straight into LDS (rows 4-byte aligned; in form K a
  // whole number of 16-byte units).  Behind the last k it reads nothing and writes
  // zeros; in form M what lies behind a row's end reaches only sums that are
  // dropped.
  __device__ __forceinline__ u32x4 source(int k_left) const {
    const uint64_t p = (uint64_t)(uintptr_t)base;
    return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)p), (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(p >> 32)),
                 (uint32_t)__builtin_amdgcn_readfirstlane(records(k_left)), 0x00020000u};
  }
  __device__ __forceinline__ void load_one(u32x4 rs, uint32_t lds, int i, int wave, int tid, int k_left) const {
    uint32_t off = voff[i];
    if (FORM == kFormK && k_left < kBK) {   // units behind the last k would hold the next row's
      const int g = i * NT + tid, unit = (g & 7) ^ swz_k(g >> 3);
      if (unit * 8 >= k_left) off = 0x7ffffff0u;
    }
    // In assembly, since the compiler would have every later read of LDS wait for it.
    // It has no result in registers; arrive() waits for what it puts into LDS.
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 ::"s"(lds + (uint32_t)(i * NT + wave * 64) * 16u), "v"(off), "s"(rs));
  }

  // Any alignment: through registers, a stage of which every unit exists (rows behind
  // the last are the last's again).
  __device__ __forceinline__ void load_whole(u32x4 (&r)[kLoads]) const {
    typedef u32x4 __attribute__((aligned(2))) u32x4_2;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) r[i] = *(const __attribute__((address_space(1))) u32x4_2*)(base + voff[i]);
  }
  __device__ __forceinline__ bool whole() const { return FORM == kFormK || rows >= W; }

  // The same where units may be missing.  A unit that ends behind its row is loaded so
  // that it ends with the row, and shifted down.
  __device__ __forceinline__ void load_regs(u32x4 (&r)[kLoads], int tid, int k_left) const {
    typedef u32x4 __attribute__((aligned(2))) u32x4_2;
    typedef const __attribute__((address_space(1))) u32x4_2* Units;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int g = i * NT + tid;
      int have, unit;       // elements of the unit that exist
      bool row_ok;
      if constexpr (FORM == kFormK) {
        unit = (g & 7) ^ swz_k(g >> 3);
        row_ok = true;
        have = k_left - unit * 8;
      } else {
        constexpr int U = W / 8;
        const int k = g / U;
        unit = (g % U) ^ swz_m<W>(k);
        row_ok = k < k_left;
        have = rows - unit * 8;
      }
      u32x4 v = {0u, 0u, 0u, 0u};
      if (row_ok && have > 0) {
        const char* p = base + voff[i];
        const int d = have < 8 ? 8 - have : 0;
        if (d <= before + unit * 8) {
          const u32x4 t = *(Units)(p - 2 * d);
          uint64_t lo = t[0] | ((uint64_t)t[1] << 32), hi = t[2] | ((uint64_t)t[3] << 32);
          if (d >= 4) {
            lo = hi >> (16 * (d - 4));
            hi = 0;
          } else if (d > 0) {
            lo = (lo >> (16 * d)) | (hi << (64 - 16 * d));
            hi >>= 16 * d;
          }
          v = u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
        } else {            // the row is shorter than a unit
          uint32_t e[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) e[j] = j < have ? ((const __attribute__((address_space(1))) uint16_t*)p)[j] : 0u;
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = e[2 * j] | (e[2 * j + 1] << 16);
        }
      }
      r[i] = v;
    }
  }
  __device__ __forceinline__ void store_regs(ZK_LDS char* lds, int tid, const u32x4 (&r)[kLoads]) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) *(ZK_LDS u32x4*)(lds + (i * NT + tid) * 16) = r[i];
  }
};

// Reads fragments of 16 rows by 32 k out of a staged panel.
template <int FORM, int W>
struct Frag {
  // Form K: byte address of (row, unit 0) and the row's XOR; form M: of the
  // lane's piece at k = 0.
  __device__ static __forceinline__ s16x8 read(const ZK_LDS char* lds, int row0, int t, int s, int lane) {
    const int c = lane & 15, q = lane >> 4;
    if constexpr (FORM == kFormK) {
      const int row = row0 + t * 16 + c;
      const int unit = (s * 4 + q) ^ swz_k(row);
      return *(const ZK_LDS s16x8*)(lds + row * 128 + unit * 16);
    } else {
      const int p = c & 3, kr = c >> 2;
      const int mb = (row0 + t * 16 + p * 4) * 2;   // byte within the row
      const int k = s * 32 + q * 8 + kr;
      const ZK_LDS char* a0 = lds + k * (W * 2) + (mb ^ (swz_m<W>(k) * 16));
      const int k1 = k + 4;
      const ZK_LDS char* a1 = lds + k1 * (W * 2) + (mb ^ (swz_m<W>(k1) * 16));
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZK_LDS s16x4*)a0);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZK_LDS s16x4*)a1);
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
};

// Order of the workgroups.  They go to the eight dies in turn; each die gets a
// run of consecutive pieces of work, so that its L2 holds the panels that its
// workgroups share.
__device__ __forceinline__ int die_order(int b, int n_blocks) {
  const int per = n_blocks >> 3, more = n_blocks & 7, die = b & 7;
  return die * per + (die < more ? die : more) + (b >> 3);
}

// Tile t of tm x tn: down eight rows of tiles at a time.
__device__ __forceinline__ void place(int t, int tm, int tn, int& im, int& in) {
  constexpr int G = 8;
  const int group = G * tn, g = t / group, first = g * G;
  const int gm = tm - first < G ? tm - first : G, r = t - g * group;
  im = first + r % gm;
  in = r / gm;
}

// Tile t of the tm (tm + 1) / 2 on and above the diagonal, column by column.
__device__ __forceinline__ void place_upper(int t, int& im, int& in) {
  int j = (int)((__builtin_sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
  while (j > 0 && j * (j + 1) / 2 > t) --j;
  while ((j + 1) * (j + 2) / 2 <= t) ++j;
  im = t - j * (j + 1) / 2;
  in = j;
}

template <typename T, int AF, int BF, int BM, int BN, int WM, int WN, bool DIRECT>
struct Core {
  static constexpr int NT = 64 * WM * WN;
  static constexpr int TM = BM / WM / 16, TN = BN / WN / 16;
  typedef Panel<AF, BM, NT> PA;
  typedef Panel<BF, BN, NT> PB;
  static constexpr int kStage = PA::kBytes + PB::kBytes;
  // Stages in LDS: three of the small tile, whose few products do not cover a load's
  // latency (16 x 4096 x 4096: 10.4 us with three, 12.6 with two; with four, which
  // leave a CU two workgroups, 2048 x 2048 x 4096 takes 42 us in place of 38).
  static constexpr int kRing = DIRECT && kStage <= 16384 ? 3 : 2;
  static constexpr int kLds = kRing * kStage;

  f32x4 acc[TM][TN];

  struct Frags { s16x8 a[TM], b[TN]; };

  __device__ __forceinline__ static void read(Frags& f, const ZK_LDS char* lds, int s, int wm, int wn, int lane) {
#pragma unroll
    for (int j = 0; j < TN; ++j) f.b[j] = Frag<BF, BN>::read(lds + PA::kBytes, wn * TN * 16, j, s, lane);
#pragma unroll
    for (int i = 0; i < TM; ++i) f.a[i] = Frag<AF, BM>::read(lds, wm * TM * 16, i, s, lane);
  }
  __device__ __forceinline__ void multiply(const Frags& f) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = mfma<T>(f.b[j], f.a[i], acc[i][j]);
  }

  static constexpr int kL = PA::kLoads + PB::kLoads, kF = TM + TN;

  __device__ __forceinline__ static void read_one(Frags& f, const ZK_LDS char* lds, int i, int s, int wm, int wn, int lane) {
    if (i < TN) f.b[i] = Frag<BF, BN>::read(lds + PA::kBytes, wn * TN * 16, i, s, lane);
    else f.a[i - TN] = Frag<AF, BM>::read(lds, wm * TM * 16, i - TN, s, lane);
  }

  // The products of `now`; between their rows the reads of `next`, and, with LOAD,
  // the loads of a stage.
  template <bool LOAD>
  __device__ __forceinline__ void step(const Frags& now, Frags& next, const ZK_LDS char* from, int s, const PA& pa, const PB& pb,
                                       uint32_t to, int wave, int tid, int left, int wm, int wn, int lane) {
    const u32x4 ra = pa.source(left), rb = pb.source(left);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      if constexpr (LOAD) {
#pragma unroll
        for (int k = 0; k < kL; ++k) {
          if (k < i * kL / TM || k >= (i + 1) * kL / TM) continue;
          if (k < PA::kLoads) pa.load_one(ra, to, k, wave, tid, left);
          else pb.load_one(rb, to + PA::kBytes, k - PA::kLoads, wave, tid, left);
        }
      }
#pragma unroll
      for (int k = 0; k < kF; ++k)
        if (k >= i * kF / TM && k < (i + 1) * kF / TM) read_one(next, from, k, s, wm, wn, lane);
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = mfma<T>(now.b[j], now.a[i], acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  __device__ __forceinline__ static void load(const PA& pa, const PB& pb, uint32_t lds, int wave, int tid, int left) {
    const u32x4 ra = pa.source(left), rb = pb.source(left);
#pragma unroll
    for (int i = 0; i < PA::kLoads; ++i) pa.load_one(ra, lds, i, wave, tid, left);
#pragma unroll
    for (int i = 0; i < PB::kLoads; ++i) pb.load_one(rb, lds + PA::kBytes, i, wave, tid, left);
  }

  // All but the youngest kKeep of this wave's loads have arrived and its reads of LDS
  // are done; then all waves' have.
  template <int kKeep = 0>
  __device__ __forceinline__ static void arrive() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kKeep) : "memory");
    __builtin_amdgcn_sched_barrier(0);
  }

  // Sums k0 .. k_end of the tile whose first rows are m0 and n0.
  __device__ __forceinline__ void run(ZK_LDS char* lds, const void* a, int64_t lda, int m, const void* b, int64_t ldb, int n,
                                      int m0, int n0, int k0, int k_end) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    PA pa;
    PB pb;
    pa.init(a, lda, m0, m, k0, k_end, tid);
    pb.init(b, ldb, n0, n, k0, k_end, tid);
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    int left = k_end - k0;
    if (left <= 0) return;
    // A last stage that is not whole goes through registers, or, loaded directly, one
    // that ends inside a unit of form K.
    const int ragged = !DIRECT || ((AF == kFormK || BF == kFormK) && left % 8) ? left % kBK : 0;
    left -= ragged;
    if constexpr (DIRECT) {
      // A ring of stages in LDS.  While the products of one half of a stage run, the
      // fragments of the next half are read; in the middle of a stage every wave has
      // read all of it and the next has arrived, so that one barrier a stage is enough
      // and the matrix units have work on both sides of it.
      Frags f0, f1;
      const uint32_t at = (uint32_t)(uintptr_t)lds;      // LDS address
      if (left > 0) {
#pragma unroll
        for (int i = 0; i < kRing; ++i) {
          load(pa, pb, at + i * kStage, wave, tid, left - i * kBK);
          pa.advance();
          pb.advance();
        }
        arrive<kL * (kRing - 1)>();
        read(f0, lds, 0, wm, wn, lane);
        int cur = 0;
        for (; left > kBK; left -= kBK) {
          const int here = cur * kStage;
          cur = cur + 1 == kRing ? 0 : cur + 1;
          step<false>(f0, f1, lds + here, 1, pa, pb, 0, wave, tid, 0, wm, wn, lane);
          arrive<kL * (kRing - 2)>();
          step<true>(f1, f0, lds + cur * kStage, 0, pa, pb, at + here, wave, tid, left - kRing * kBK, wm, wn, lane);
          pa.advance();
          pb.advance();
        }
        read(f1, lds + cur * kStage, 1, wm, wn, lane);
        multiply(f0);
        multiply(f1);
      }
    } else {
      // Through registers: a stage is loaded while the one before it is multiplied.
      if (pa.whole() && pb.whole()) {
        reg_loop(lds, pa, pb, left, wm, wn, lane, tid, [&](u32x4 (&ra)[PA::kLoads], u32x4 (&rb)[PB::kLoads]) {
          pa.load_whole(ra);
          pb.load_whole(rb);
        });
      } else {
        reg_loop(lds, pa, pb, left, wm, wn, lane, tid, [&](u32x4 (&ra)[PA::kLoads], u32x4 (&rb)[PB::kLoads]) {
          pa.load_regs(ra, tid, kBK);
          pb.load_regs(rb, tid, kBK);
        });
      }
    }
    if (ragged) {
      Frags f;
      PA ta;
      PB tb;
      ta.init(a, lda, m0, m, k_end - ragged, k_end, tid);
      tb.init(b, ldb, n0, n, k_end - ragged, k_end, tid);
      u32x4 ra[PA::kLoads], rb[PB::kLoads];
      ta.load_regs(ra, tid, ragged);
      tb.load_regs(rb, tid, ragged);
      arrive();           // no load is under way into this stage, and nobody reads it
      ta.store_regs(lds, tid, ra);
      tb.store_regs(lds + PA::kBytes, tid, rb);
      __syncthreads();
#pragma unroll
      for (int s = 0; s < kBK / 32; ++s) {
        read(f, lds, s, wm, wn, lane);
        multiply(f);
      }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }

  template <typename L>
  __device__ __forceinline__ void reg_loop(ZK_LDS char* lds, PA& pa, PB& pb, int left, int wm, int wn, int lane, int tid, L fetch) {
    if (left <= 0) return;
    u32x4 ra[PA::kLoads], rb[PB::kLoads];
    Frags f;
    fetch(ra, rb);
    int cur = 0;
    for (; left > 0; left -= kBK) {
      ZK_LDS char* here = lds + cur * kStage;
      pa.store_regs(here, tid, ra);
      pb.store_regs(here + PA::kBytes, tid, rb);
      __syncthreads();
      if (left > kBK) {
        pa.advance();
        pb.advance();
        fetch(ra, rb);
      }
#pragma unroll
      for (int s = 0; s < kBK / 32; ++s) {
        read(f, here, s, wm, wn, lane);
        multiply(f);
      }
      cur ^= 1;
    }
  }

  // The tile's values on their way out, eight consecutive n of a row at a time, so
  // that eight lanes write whole lines.  The sums go through LDS 32 rows of a wave at
  // a time, in a loop: unrolled, the epilogue of a tile was 40 to 70 KB of code that
  // each launch fetched anew.  before(row, first n, p) starts what the epilogue
  // reads, 32 rows ahead; after(row, first n, values, p) ends it and leaves the
  // finished values, which with `twice` mirror(row, first n, values) takes to the
  // transposed place.
  // The first of a lane's eight columns, the same in all its pieces.
  __device__ __forceinline__ static int column(int n0) {
    return n0 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % WN * TN * 16 + (threadIdx.x & 63) % (TN * 2) * 8;
  }
  static constexpr int kPitch = TN * 64 + 16;      // bytes between rows: 16 rows' 16 bytes lie in different banks
  static constexpr int kWaveBytes = 32 * kPitch;
  static_assert(kWaveBytes * WM * WN <= kLds, "the waves' parts fit");
  template <typename P, typename F, typename G, typename H>
  __device__ __forceinline__ void each(ZK_LDS char* lds, int m0, int n0, bool twice, F before, G after, H mirror) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    constexpr int kRow = TN * 2, kN = 32 * kRow / 64;      // pieces of a row, and of a lane in 32 rows
    ZK_LDS char* mine = lds + wave * kWaveBytes;
    const int col = column(n0);
    m0 += wm * TM * 16 + lane / kRow;
    n0 += wn * TN * 16;
    P p[kN];
#pragma unroll
    for (int b = 0; b < kN; ++b) before(m0 + b * (64 / kRow), col, p[b]);
    arrive();               // nobody reads a stage any more
#pragma unroll 1
    for (int i = 0; i < TM; i += 2, m0 += 32) {
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          *(ZK_LDS f32x4*)(mine + (x * 16 + (lane & 15)) * kPitch + j * 64 + (lane >> 4) * 16) = acc[x][j];
#pragma unroll
      for (int x = 2; x < TM; ++x)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[x - 2][j] = acc[x][j];
      P q[kN];
      if (i + 2 < TM) {
#pragma unroll
        for (int b = 0; b < kN; ++b) before(m0 + 32 + b * (64 / kRow), col, q[b]);
      }
      ZK_LDS char* at = mine + lane / kRow * kPitch + lane % kRow * 32;
#pragma unroll 1
      for (int b = 0; b < kN; ++b) {
        const f32x4 lo = *(ZK_LDS f32x4*)at, hi = *(ZK_LDS f32x4*)(at + 16);
        float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        after(m0 + b * (64 / kRow), col, v, p[0]);
        if constexpr (!__is_same(H, int)) {
          if (twice) {
            *(ZK_LDS f32x4*)at = f32x4{v[0], v[1], v[2], v[3]};
            *(ZK_LDS f32x4*)(at + 16) = f32x4{v[4], v[5], v[6], v[7]};
          }
        }
        at += 64 / kRow * kPitch;
#pragma unroll
        for (int x = 1; x < kN; ++x) p[x - 1] = p[x];
      }
#pragma unroll
      for (int b = 0; b < kN; ++b) p[b] = q[b];
      if constexpr (!__is_same(H, int)) {
        if (twice) {
          const int first = m0 - lane / kRow + lane % 4 * 8;
#pragma unroll 2
          for (int n = lane / 4; n < TN * 16; n += 16) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = *(const ZK_LDS float*)(mine + (lane % 4 * 8 + k) * kPitch + n * 4);
            mirror(n0 + n, first, v);
          }
        }
      }
    }
  }
};

}  // namespace gemm
}  // namespace zk
