// zero_muon.hip -- gfx950 kernels that orthogonalise matrices by Newton-Schulz
// products.
//
// X <- a X + (b A + c A A) X with A = X X^T drives every singular value of X
// towards 1.  With n the shorter side a step is three products, two of which
// have symmetric results of which only the tiles on and above the diagonal are
// computed and the others mirrored.  A tall matrix takes A = X^T X and X A, so
// that nothing is transposed in memory.
//
// Numbers between the products.  X is held in two numbers of 16 bits for the term a X, and its
// fp16 rounding is the products' operand: directions that the gradient hardly holds
// are scaled up by a in each step, and X rounded to 16 bits would carry its rounding
// up with them (a matrix of exponentially falling singular values ends 1.3% off its
// 64-bit result; with two numbers 0.04%).  They are the
// fp16 rounding and what it left as bf16: 20 significant bits and more, 8 where
// fp16 has nothing left (X below 2^-25), for two bytes less to write than an fp32
// beside the operand.  A and B = b A + c A A are held in fp16:
// their entries are of order one and below, where fp16 has three bits more than
// bf16 (1.0% of error against 0.14%).  Rounding X, A and B for the products is what the result is
// off by: 0.0015 as a rule, up to 0.02 where few entries count and it does not average out.  From the fourth step on A's eigenvalues
// lie around 1, and A - I/2 is stored in place of A, which halves its largest
// entries and their rounding; the polynomial is rewritten for it:
//   b A + c A^2 = (b d + c d^2) I + (b + 2 c d) D + c D^2,  D = A - d I,
// and the multiple of I joins a.  (Where |G| is below eps, X stays small for more
// steps, and fp16 may lose it: there d is 0, so that B X stays small beside a X.)
// The first X is the gradient times a power of two, which rounds nothing that
// fp16 holds; the rest of 1 / (|G| + eps) enters as a factor of the first step's
// results.
#include "zero_hidden_dev.h"

#pragma clang fp contract(off)

namespace zk {
namespace hidden {
namespace {

// Sum of squares of a piece of a matrix, in fp64 (exact products of 16-bit
// values, no overflow).  8192 x 8192: 38.6 us, 3.5 TB/s; the fp64 sums keep it from
// the memory's rate.
template <typename T>
__global__ void __launch_bounds__(kLoadThreads) ortho_norm_kernel(const OrthoLoadArgs a) {
  const int z = blockIdx.x / a.norm_blocks, piece = blockIdx.x % a.norm_blocks;
  const int64_t units = (a.numel + 7) / 8, per = (units + a.norm_blocks - 1) / a.norm_blocks;
  const int64_t u1 = (piece + 1) * per < units ? (piece + 1) * per : units;
  double s = 0.0;
#pragma unroll 4
  for (int64_t u = piece * per + threadIdx.x; u < u1; u += kLoadThreads) {
    float x[8];
    const int64_t e = u * 8;
    load_row<T, 8>(a.src, a.src_off[z] + e, a.numel - e < 8 ? (int)(a.numel - e) : 8, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) s += (double)x[i] * (double)x[i];
  }
  __shared__ double w[kLoadThreads];
  w[threadIdx.x] = s;
  __syncthreads();
  for (int k = kLoadThreads / 2; k > 0; k >>= 1) {
    if ((int)threadIdx.x < k) w[threadIdx.x] += w[threadIdx.x + k];
    __syncthreads();
  }
  if (threadIdx.x == 0) a.sums[(int64_t)z * a.norm_blocks + piece] = w[0];
}

// What is left of 1 / (|G| + eps) beside 2^e, at most 1/32.  A matrix of zeros takes 1:
// 1 / eps or its square may be beyond fp32, and zeros times infinity are no zeros.
__device__ __forceinline__ float factor_left(bool good, double norm, double den, int e) {
  return !good ? __builtin_nanf("") : norm > 0.0 ? (float)(1.0 / ldexp(den, e)) : 1.0f;
}

// X = G * 2^k in fp16 with |X| in [32, 64), padded with zeros to multiples of 8,
// and the factor that is left of 1 / (|G| + eps).  A workgroup joins the norm's
// pieces once for kLoadUnits pieces of eight a thread (8192 x 8192: 51 us, 5.2 TB/s).
template <typename T>
__global__ void __launch_bounds__(kLoadThreads) ortho_load_kernel(const OrthoLoadArgs a) {
  const int upr = a.ld >> 3;
  const int64_t per = (int64_t)a.rows_pad * upr, span = kLoadThreads * kLoadUnits, blocks = (per + span - 1) / span;
  const int z = (int)(blockIdx.x / blocks);
  const int64_t u0 = (blockIdx.x - z * blocks) * span + threadIdx.x;
  Row<T, 8> x[kLoadUnits];
#pragma unroll
  for (int i = 0; i < kLoadUnits; ++i) {
    const int64_t u = u0 + i * kLoadThreads;
    const int row = (int)(u / upr), col = (int)(u - (int64_t)row * upr) * 8;
    const int have = u < per && row < a.rows ? a.cols - col : 0;
    if (have > 0) x[i].load(a.src, a.src_off[z] + (int64_t)row * a.cols + col, have);
    else x[i].v = {};
  }
  __shared__ double w[kLoadThreads / 64];
  double s = 0.0;
  for (int i = threadIdx.x; i < a.norm_blocks; i += kLoadThreads) s += a.sums[(int64_t)z * a.norm_blocks + i];
#pragma unroll
  for (int k = 32; k > 0; k >>= 1) s += __shfl_xor(s, k);
  if ((threadIdx.x & 63) == 0) w[threadIdx.x >> 6] = s;
  __syncthreads();
  s = 0.0;
#pragma unroll
  for (int k = 0; k < kLoadThreads / 64; ++k) s += w[k];
  const double norm = __builtin_sqrt(s), d = norm + a.eps;
  const bool good = d < __builtin_inf();                          // not NaN either
  const int e = good && norm > 0.0 ? 5 - ilogb(norm) : 0;        // |G| 2^e in [32, 64)
  if (u0 == 0) {
    a.factor[2 * z] = factor_left(good, norm, d, e);
    a.factor[2 * z + 1] = norm > a.eps ? 1.0f : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < kLoadUnits; ++i) {
    const int64_t u = u0 + i * kLoadThreads;
    if (u >= per) break;
    f16x8 h;
#pragma unroll
    for (int k = 0; k < 8; ++k) h[k] = good ? (_Float16)ldexpf((float)x[i].v[k], e) : (_Float16)0.0f;
    const int row = (int)(u / upr), col = (int)(u - (int64_t)row * upr) * 8;
    AS1 _Float16* x16 = (AS1 _Float16*)a.x + z * a.zx + row * a.pitch + col;
    *(AS1 f16x8*)x16 = h;
    if (a.again) *(AS1 f16x8*)(x16 + a.again) = h;
  }
}

__device__ __forceinline__ float factor_of(const OrthoArgs& a, int z) { return a.first ? a.factor[2 * z] : 1.0f; }
__device__ __forceinline__ float shift_of(const OrthoArgs& a, int z) { return a.shift * a.factor[2 * z + 1]; }

template <int V>
__device__ __forceinline__ void store_half(void* base, int64_t e, const float (&v)[V]) {
  typename Row<_Float16, V>::tv h;
#pragma unroll
  for (int i = 0; i < V; ++i) h[i] = (_Float16)v[i];
  *(AS1 typename Row<_Float16, V>::tv*)((AS1 _Float16*)base + e) = h;
}

// What the epilogue of V sums of a row reads, and the epilogue, which leaves the
// finished values in place of the sums.  Rows in the workspace are whole eights and
// 16-byte aligned.
template <int EPI, int V>
struct Epilogue {
  typedef typename Row<_Float16, V>::tv Half;
  typedef typename Row<__bf16, V>::tv Low;
  Half x;               // kPoly: A - d I; kNext: X,
  Low low;              // and what its rounding left

  __device__ __forceinline__ void load(const OrthoArgs& a, int z, int row, int col) {
    if constexpr (EPI == kGram) return;
    const int64_t e = z * a.zadd + (int64_t)row * a.ldadd + col;
    x = *(const AS1 Half*)((const AS1 _Float16*)a.add + e);
    if (EPI == kNext && !a.first) low = *(const AS1 Low*)((const AS1 __bf16*)a.low + e);
    else low = Low{};
  }
  __device__ __forceinline__ float value(int i) const { return (float)x[i] + (float)low[i]; }

  __device__ __forceinline__ void finish(const OrthoArgs& a, int z, int row, int col, float (&v)[V]) const {
    if constexpr (EPI == kGram) {
      const float f = factor_of(a, z), f2 = f * f, d = shift_of(a, z);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = __builtin_fmaf(f2, v[i], row == col + i ? -d : 0.0f);
    } else if constexpr (EPI == kPoly) {
      const float b = __builtin_fmaf(2.0f * a.c, shift_of(a, z), a.b);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = __builtin_fmaf(a.c, v[i], b * (float)x[i]);
    } else {
      const float f = factor_of(a, z), d = shift_of(a, z);
      const float c0 = __builtin_fmaf(__builtin_fmaf(a.c, d, a.b), d, a.a);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = f * __builtin_fmaf(c0, value(i), v[i]);
      if (a.last) {
        if (row < a.rows && col < a.cols) {
          const float s = a.scale[z];
#pragma unroll
          for (int i = 0; i < V; ++i) v[i] *= s;
          const int64_t d = a.dst_off[z] + (int64_t)row * a.cols + col;
          if (a.dst_dt == ZERO_BF16) store_row<__bf16, V>(a.dst, d, a.cols - col, v);
          else store_row<_Float16, V>(a.dst, d, a.cols - col, v);
        }
        return;
      }
      Low left;
#pragma unroll
      for (int i = 0; i < V; ++i) left[i] = (__bf16)(v[i] - (float)(_Float16)v[i]);
      *(AS1 Low*)((AS1 __bf16*)a.low + z * a.zadd + (int64_t)row * a.ldadd + col) = left;
    }
    store_half<V>(a.out, z * a.zout + (int64_t)row * a.ldo + col, v);
  }
};

// A workgroup a tile of one of the batch's matrices.  8192 x 8192: 466, 457 and 880 us
// for A, B and the next X, at the power limit; 48 x 768 x 768: 41, 42 and 78 us, where
// 12 stages a tile do not cover the epilogue's bytes (X's two halves read and written:
// 0.2 GB).
template <int EPI, int AF, int BF, int TILE>
__global__ void __launch_bounds__(kTileThreads[TILE]) ortho_kernel(const OrthoArgs a) {
  typedef CoreOf<_Float16, AF, BF, TILE, true> C;
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  C core;
  int z, m0, n0;
  if (!run_tile<EPI != kNext>(core, (ZK_LDS char*)smem, a.p, blockIdx.x, a.za, a.zb, z, m0, n0)) return;
  typedef Epilogue<EPI, 8> E;
  const auto before = [&](int row, int col, E& e) { if (row < a.p.m && col < a.p.n) e.load(a, z, row, col); };
  const auto after = [&](int row, int col, float (&v)[8], const E& e) {
    if (row < a.p.m && col < a.p.n) e.finish(a, z, row, col, v);
  };
  if constexpr (EPI == kNext) {
    core.template each<E>((ZK_LDS char*)smem, m0, n0, false, before, after, 0);
  } else {
    // A tile above the diagonal stands for its mirror image too.
    core.template each<E>((ZK_LDS char*)smem, m0, n0, m0 != n0, before, after,
                          [&](int row, int col, const float (&v)[8]) {
                            if (row < a.p.m && col < a.p.n) store_half<8>(a.out, z * a.zout + (int64_t)row * a.ldo + col, v);
                          });
  }
}

template <int EPI>
__global__ void __launch_bounds__(kJoinThreads) ortho_join_kernel(const OrthoArgs a) {
  int z, row, col;
  bool twice;
  float v[4];
  if (join4<EPI != kNext>(a.p, (int64_t)blockIdx.x * kJoinThreads + threadIdx.x, z, row, col, v, twice)) {
    Epilogue<EPI, 4> e;
    e.load(a, z, row, col);
    e.finish(a, z, row, col, v);
    if (EPI != kNext && twice) {
#pragma unroll
      for (int i = 0; i < 4; ++i) ((AS1 _Float16*)a.out)[z * a.zout + (int64_t)(col + i) * a.ldo + row] = (_Float16)v[i];
    }
  }
}

// ---------------------------------------------------------------------------
// Matrices with a short side
// ---------------------------------------------------------------------------

// With n = the shorter side up to 64 the steps need X only once: each multiplies X by
// Q = a I + b A + c A^2, and the next A is Q A Q.  One workgroup forms P, the product
// of the Q, in fp32 from A = X X^T, whose pieces a launch of products has summed from
// the gradient's own bits; a last product takes X to P X, with P as two fp16 numbers
// along k.  In fp32 A's rounding shows in P as 0.0005 of the result at most (falling
// singular values, where rounding A to fp16 would leave nothing).  Five launches in
// the place of 17 (43 matrices of 33 x 7489: 271 -> 86 us); this one is a chain of 18
// products in LDS at the fp32 matrix rate of one CU (a side of 64: 29 us, 16: 9).
template <int NT>      // tiles of 16 along a side
__global__ void __launch_bounds__(kThinThreads) ortho_thin_kernel(const OrthoThinArgs a) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  __shared__ float most[kThinThreads / 64];
  constexpr int kPitch = kThinSide + 4;      // floats: 16 rows' 16 bytes lie in different banks
  ZK_LDS float* const A = (ZK_LDS float*)(ZK_LDS char*)smem;
  ZK_LDS float* const Q = A + kThinSide * kPitch;
  ZK_LDS float* const P = Q + kThinSide * kPitch;
  ZK_LDS float* const T = P + kThinSide * kPitch;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), z = blockIdx.x;
  const float f = a.factor[2 * z];

  const AS1 float* part = (const AS1 float*)a.part + (int64_t)z * a.splits * kThinSide * kThinSide;
  for (int u = threadIdx.x; u < kThinSide * kThinSide / 4; u += kThinThreads) {
    const int row = u / (kThinSide / 4), col = u % (kThinSide / 4) * 4;
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    if (row < a.side && col < a.side) {
#pragma unroll 4
      for (int i = 0; i < a.splits; ++i) {
        const f32x4 v = *(const AS1 f32x4*)(part + (int64_t)i * kThinSide * kThinSide + u * 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) s[k] += (double)v[k];
      }
    }
    f32x4 v, one;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = (float)(s[k] * (double)f * (double)f);
      one[k] = row == col + k && row < a.n ? 1.0f : 0.0f;
    }
    *(ZK_LDS f32x4*)(A + row * kPitch + col) = v;
    *(ZK_LDS f32x4*)(P + row * kPitch + col) = one;
  }
  __syncthreads();

  // A wave's tiles of 16 x 16, two at most; a lane has four columns of a row.
  constexpr int kMine = (NT * NT + 7) / 8;
  const auto place16 = [&](int i, int& row, int& col) {
    const int t = wave * kMine + i;
    row = t / NT * 16 + (lane & 15);
    col = t % NT * 16 + (lane >> 4) * 4;
    return t < NT * NT;
  };
  // l r for symmetric r.
  const auto product = [&](const ZK_LDS float* l, const ZK_LDS float* r, f32x4 (&acc)[kMine]) {
    f32x4 x[kMine][NT], y[kMine][NT];
#pragma unroll
    for (int k = 0; k < NT; ++k) {
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int t = wave * kMine + i, tile = t < NT * NT ? t : 0;      // a wave too many does the first again
        x[i][k] = *(const ZK_LDS f32x4*)(l + (tile / NT * 16 + (lane & 15)) * kPitch + (lane >> 4) * 4 + k * 16);
        y[i][k] = *(const ZK_LDS f32x4*)(r + (tile % NT * 16 + (lane & 15)) * kPitch + (lane >> 4) * 4 + k * 16);
      }
    }
#pragma unroll
    for (int i = 0; i < kMine; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < NT * 4; ++k)
#pragma unroll
      for (int i = 0; i < kMine; ++i)
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(y[i][k / 4][k % 4], x[i][k / 4][k % 4], acc[i], 0, 0, 0);
  };
  int row, col;
  f32x4 s[kMine], t[kMine];
#pragma unroll 1
  for (int step = 0; step < a.steps; ++step) {
    product(A, A, s);
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      if (!place16(i, row, col)) continue;
      const f32x4 x = *(const ZK_LDS f32x4*)(A + row * kPitch + col);
      f32x4 q;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        q[k] = __builtin_fmaf(a.c, s[i][k], __builtin_fmaf(a.b, x[k], row == col + k && row < a.n ? a.a : 0.0f));
      *(ZK_LDS f32x4*)(Q + row * kPitch + col) = q;
    }
    __syncthreads();
    const bool last = step + 1 == a.steps;
    product(Q, P, s);
    if (!last) product(Q, A, t);
    __syncthreads();        // nobody reads P and A any more
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      if (!place16(i, row, col)) continue;
      *(ZK_LDS f32x4*)(P + row * kPitch + col) = s[i];
      if (!last) *(ZK_LDS f32x4*)(T + row * kPitch + col) = t[i];
    }
    __syncthreads();
    if (last) break;
    product(T, Q, s);
#pragma unroll
    for (int i = 0; i < kMine; ++i)
      if (place16(i, row, col)) *(ZK_LDS f32x4*)(A + row * kPitch + col) = s[i];
    __syncthreads();
  }

  // P times a power of two that brings its largest entry to 2^12.
  float m = 0.0f;
  for (int u = threadIdx.x; u < a.side * a.side; u += kThinThreads) {
    const float x = __builtin_fabsf(P[u / a.side * kPitch + u % a.side]);
    m = x > m ? x : m;
  }
#pragma unroll
  for (int k = 32; k > 0; k >>= 1) {
    const float x = __shfl_xor(m, k);
    m = x > m ? x : m;
  }
  if (lane == 0) most[wave] = m;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kThinThreads / 64; ++k) m = most[k] > m ? most[k] : m;
  const int e = m > 0.0f && m < __builtin_inff() ? ilogbf(m) - 12 : 0;
  if (threadIdx.x == 0) a.factor[2 * z] = ldexpf(f, e);
  AS1 _Float16* const out = (AS1 _Float16*)a.p + (int64_t)z * a.side * 2 * a.side;
  for (int u = threadIdx.x; u < a.side * a.side; u += kThinThreads) {
    const int r = u / a.side, c = u % a.side;
    const float x = ldexpf(P[r * kPitch + c], -e);
    const _Float16 hi = (_Float16)x;
    out[r * 2 * a.side + c] = hi;
    out[r * 2 * a.side + a.side + c] = (_Float16)(x - (float)hi);
  }
}

// ---------------------------------------------------------------------------
// Small matrices
// ---------------------------------------------------------------------------

// A whole matrix of up to 16384 elements by one workgroup: X, A and B in LDS in fp16,
// X also in fp32 in the registers of the wave whose tiles of 16 x 16 it is, eight at
// most.  One launch in the place of 17, each of which is latency alone (65 x 33: 13.1 us,
// 67 with them; 26.7 while a wave's tiles were divided out in every product and its
// fragments were not under way ahead).  Rows are 16 bytes apart beyond their length, so that a fragment's 16
// rows lie in different banks.
struct Small {
  ZK_LDS char* p;
  int pitch;            // bytes
  __device__ __forceinline__ s16x8 along(int row0, int k0, int lane) const {     // 16 rows, 32 k along them
    return *(const ZK_LDS s16x8*)(p + (row0 + (lane & 15)) * pitch + (k0 + (lane >> 4) * 8) * 2);
  }
  __device__ __forceinline__ s16x8 across(int col0, int k0, int lane) const {    // 16 columns, k down the rows
    const int c = lane & 15;
    const ZK_LDS char* a = p + (k0 + (lane >> 4) * 8 + (c >> 2)) * pitch + (col0 + (c & 3) * 4) * 2;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZK_LDS s16x4*)a);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZK_LDS s16x4*)(a + 4 * pitch));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  typedef _Float16 half4 __attribute__((ext_vector_type(4)));
  __device__ __forceinline__ ZK_LDS half4* at(int row, int col) const { return (ZK_LDS half4*)(p + row * pitch + col * 2); }
};

// The matrix as it is into LDS in rows of X's length, its norm in fp64, then X = G 2^k in
// fp16.  Returns what is left of 1 / (|G| + eps); may_shift: whether |G| is above eps.
template <typename T, int NT>
__device__ __forceinline__ float small_load(const OrthoSmallArgs& a, const Small& X, int rp, int cp, double* sums, bool& may_shift) {
  const int upr = cp / 8, units = rp * upr, z = blockIdx.x;
  double s = 0.0;
  for (int u = threadIdx.x; u < units; u += NT) {
    const int row = u / upr, col = u % upr * 8, have = row < a.rows ? a.cols - col : 0;
    Row<T, 8> x;
    if (have > 0) x.load(a.src, a.off[z] + (int64_t)row * a.cols + col, have);
    else x.v = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) s += (double)(float)x.v[i] * (double)(float)x.v[i];
    *(ZK_LDS typename Row<T, 8>::tv*)X.at(row, col) = x.v;
  }
#pragma unroll
  for (int k = 32; k > 0; k >>= 1) s += __shfl_xor(s, k);
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = s;
  __syncthreads();
  s = 0.0;
#pragma unroll
  for (int k = 0; k < NT / 64; ++k) s += sums[k];
  const double norm = __builtin_sqrt(s), den = norm + a.eps;
  const bool good = den < __builtin_inf();
  const int e = good && norm > 0.0 ? 5 - ilogb(norm) : 0;
  for (int u = threadIdx.x; u < units; u += NT) {
    ZK_LDS char* at = (ZK_LDS char*)X.at(u / upr, u % upr * 8);
    const typename Row<T, 8>::tv x = *(ZK_LDS typename Row<T, 8>::tv*)at;
    f16x8 h;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = good ? (_Float16)ldexpf((float)x[i], e) : (_Float16)0.0f;
    *(ZK_LDS f16x8*)at = h;
  }
  __syncthreads();
  may_shift = norm > a.eps;
  return factor_left(good, norm, den, e);
}

// The result's four values of a row, on their way out.
__device__ __forceinline__ void small_store(const OrthoSmallArgs& a, int row, int col, float (&v)[4]) {
  if (row >= a.rows || col >= a.cols) return;
  const int z = blockIdx.x;
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] *= a.scale[z];
  const int64_t o = a.off[z] + (int64_t)row * a.cols + col;
  if (a.dst_dt == ZERO_BF16) store_row<__bf16, 4>(a.dst, o, a.cols - col, v);
  else store_row<_Float16, 4>(a.dst, o, a.cols - col, v);
}

// A wave's tiles of 16 x 16, with the divisions done once.  Beyond the last tile it
// does the first again and keeps nothing, so that no product has a branch.
template <int N>
struct SmallTiles {
  int count, row[N], col[N];
  __device__ __forceinline__ SmallTiles(int wave, int down, int across) : count(0) {
    const int each = (down * across + kSmallThreads / 64 - 1) / (kSmallThreads / 64);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int t = wave * each + i;
      const bool mine = i < each && t < down * across;
      row[i] = mine ? t / across * 16 : 0;
      col[i] = mine ? t % across * 16 : 0;
      if (mine) count = i + 1;
    }
  }
};

// Whether the next fragments are loaded while a product's run, where the registers hold
// them: with eight tiles 175 went to scratch (128 x 128: 66 us, 128 of them 100; without
// them ahead 50 and 52), with five of both 13 (96 x 128: 39 us, 33 without); 32 x 320, five
// tiles and one, takes 13.7 us with them ahead and 14.4 without.
constexpr bool small_ahead(int mx, int mn) { return mx <= 3 || (mx <= 5 && mn <= 2); }

template <typename T, int MX, int MN>      // tiles a wave of X, and of the n x n results, at most
__global__ void __launch_bounds__(kSmallThreads) ortho_small_kernel(const OrthoSmallArgs a) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  __shared__ double sums[kSmallThreads / 64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool tall = a.rows > a.cols;
  const int side = a.rp < a.cp ? a.rp : a.cp, wide = a.rp < a.cp ? a.cp : a.rp;
  const Small X = {(ZK_LDS char*)smem, a.cp * 2 + 16};
  const Small A = {X.p + a.rp * X.pitch, side * 2 + 16};
  const Small B = {A.p + side * A.pitch, A.pitch};

  bool shifts;
  float f = small_load<T, kSmallThreads>(a, X, a.rp, a.cp, sums, shifts);
  const float may_shift = shifts ? a.shift : 0.0f;

  // The wave's tiles of X and of the n x n results.
  const int q = lane >> 4, c = lane & 15;
  const SmallTiles<MX> of_x(wave, a.rp / 16, a.cp / 16);
  const SmallTiles<MN> of_n(wave, side / 16, side / 16);
  f32x4 x32[MX], acc_x[MX], acc_n[MN];
#pragma unroll
  for (int i = 0; i < MX; ++i) {
    const Small::half4 h = *X.at(of_x.row[i] + c, of_x.col[i] + q * 4);
    x32[i] = f32x4{(float)h[0], (float)h[1], (float)h[2], (float)h[3]};
  }
  // acc = the wave's tiles of a product; a depth is a multiple of 32.
  auto product = [&](const auto& tiles, auto& acc, int depth, auto left, auto right) {
    constexpr int N = sizeof(acc) / sizeof(acc[0]);
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    if constexpr (!small_ahead(MX, MN)) {
#pragma unroll 1
      for (int k = 0; k < depth; k += 32) {
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = mfma<_Float16>(right(tiles.col[i], k), left(tiles.row[i], k), acc[i]);
      }
      return;
    }
    s16x8 l[N], r[N];
#pragma unroll
    for (int i = 0; i < N; ++i) l[i] = left(tiles.row[i], 0), r[i] = right(tiles.col[i], 0);
#pragma unroll 1
    for (int k = 32; k < depth; k += 32) {      // the next fragments under way
      s16x8 l1[N], r1[N];
#pragma unroll
      for (int i = 0; i < N; ++i) l1[i] = left(tiles.row[i], k), r1[i] = right(tiles.col[i], k);
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = mfma<_Float16>(r[i], l[i], acc[i]);
#pragma unroll
      for (int i = 0; i < N; ++i) l[i] = l1[i], r[i] = r1[i];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = mfma<_Float16>(r[i], l[i], acc[i]);
  };
#pragma unroll 1
  for (int step = 0; step < a.steps; ++step) {
    const float d = step >= a.shift_from ? may_shift : 0.0f;
    if (tall) product(of_n, acc_n, wide, [&](int r, int k) { return X.across(r, k, lane); }, [&](int r, int k) { return X.across(r, k, lane); });
    else product(of_n, acc_n, wide, [&](int r, int k) { return X.along(r, k, lane); }, [&](int r, int k) { return X.along(r, k, lane); });
#pragma unroll
    for (int i = 0; i < MN; ++i) {
      const int row = of_n.row[i] + c, col = of_n.col[i] + q * 4;
      if (i < of_n.count) {
        Small::half4 h;
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = (_Float16)__builtin_fmaf(f * f, acc_n[i][k], row == col + k ? -d : 0.0f);
        *A.at(row, col) = h;
      }
    }
    __syncthreads();
    product(of_n, acc_n, side, [&](int r, int k) { return A.along(r, k, lane); }, [&](int r, int k) { return A.along(r, k, lane); });
    const float b = __builtin_fmaf(2.0f * a.c, d, a.b), c0 = __builtin_fmaf(__builtin_fmaf(a.c, d, a.b), d, a.a);
#pragma unroll
    for (int i = 0; i < MN; ++i) {
      const int row = of_n.row[i] + c, col = of_n.col[i] + q * 4;
      if (i < of_n.count) {
        const Small::half4 x = *A.at(row, col);
        Small::half4 h;
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = (_Float16)__builtin_fmaf(a.c, acc_n[i][k], b * (float)x[k]);
        *B.at(row, col) = h;
      }
    }
    __syncthreads();
    if (tall)
      product(of_x, acc_x, side, [&](int r, int k) { return X.along(r, k, lane); }, [&](int r, int k) { return B.along(r, k, lane); });
    else
      product(of_x, acc_x, side, [&](int r, int k) { return B.along(r, k, lane); }, [&](int r, int k) { return X.across(r, k, lane); });
    __syncthreads();        // nobody reads X any more
    const bool last = step + 1 == a.steps;
#pragma unroll
    for (int i = 0; i < MX; ++i) {
      const int row = of_x.row[i] + c, col = of_x.col[i] + q * 4;
      if (i < of_x.count) {
        float v[4];
        Small::half4 h;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x32[i][k] = v[k] = f * __builtin_fmaf(c0, x32[i][k], acc_x[i][k]);
          h[k] = (_Float16)v[k];
        }
        if (!last) *X.at(row, col) = h;
        else small_store(a, row, col, v);
      }
    }
    f = 1.0f;
    __syncthreads();
  }
}

// Small matrices with a side of up to 16.  Few entries' rounding to fp16 does not average
// out (2 x 2 with A, B and X in fp16: up to 0.014 off, 0.002 at the median), so these go the way
// of the large matrices with a short side: P in fp32 from A = X X^T, which is one tile of
// 16 x 16, and P X with P as two fp16 numbers along k.  Every wave forms P by itself: a
// product's result lies in a wave's registers as the next one's operands do (16 x 512: 8.3 us,
// most of it the load, the norm and a chain of 18 products; 2 x 2: 5.0).
constexpr int kShortThreads = 256;
template <typename T>
__global__ void __launch_bounds__(kShortThreads) ortho_short_kernel(const OrthoSmallArgs a) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  constexpr int kWaves = kShortThreads / 64, kPitchP = 80;      // bytes: 32 halves, and 16 to lie in other banks
  __shared__ double sums[kWaves];
  __shared__ f32x4 part[kWaves][64];
  __shared__ __attribute__((aligned(16))) char halves[kWaves][16 * kPitchP];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 15, q = lane >> 4;
  const bool tall = a.rows > a.cols;
  const int n = tall ? a.cols : a.rows, rp = tall ? a.rp : 16, cp = tall ? 16 : a.cp, wide = tall ? a.rp : a.cp;
  const Small X = {(ZK_LDS char*)smem, cp * 2 + 16};
  bool shifts;
  const float f = small_load<T, kShortThreads>(a, X, rp, cp, sums, shifts);

  // A: the waves take 32 k in turn, and join their sums in their order.
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int k = wave * 32; k < wide; k += kWaves * 32) {
    const s16x8 x = tall ? X.across(0, k, lane) : X.along(0, k, lane);
    acc = mfma<_Float16>(x, x, acc);
  }
  part[wave][lane] = acc;
  __syncthreads();
  // A lane has row c, columns 4 q to 4 q + 3, which as an operand are four k.
  f32x4 A, P, one;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) s += (double)part[w][lane][k];
    A[k] = (float)(s * (double)f * (double)f);
    one[k] = q * 4 + k == c && c < n ? 1.0f : 0.0f;
  }
  P = one;
  const auto product = [](const f32x4& l, const f32x4& r) {      // l r for symmetric r
    f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 4; ++k) d = __builtin_amdgcn_mfma_f32_16x16x4f32(r[k], l[k], d, 0, 0, 0);
    return d;
  };
#pragma unroll 1
  for (int step = 0; step < a.steps; ++step) {
    const f32x4 s = product(A, A);
    f32x4 Q;
#pragma unroll
    for (int k = 0; k < 4; ++k) Q[k] = __builtin_fmaf(a.c, s[k], __builtin_fmaf(a.b, A[k], a.a * one[k]));
    P = product(Q, P);
    A = product(product(Q, A), Q);
  }

  // P times a power of two that brings its largest entry to 2^12, as two halves.
  float m = 0.0f;
#pragma unroll
  for (int k = 0; k < 4; ++k) m = __builtin_fabsf(P[k]) > m ? __builtin_fabsf(P[k]) : m;
#pragma unroll
  for (int k = 32; k > 0; k >>= 1) {
    const float x = __shfl_xor(m, k);
    m = x > m ? x : m;
  }
  const int e = m > 0.0f && m < __builtin_inff() ? ilogbf(m) - 12 : 0;
  const Small H = {(ZK_LDS char*)(char*)halves[wave], kPitchP};
  Small::half4 hi, lo;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float x = ldexpf(P[k], -e);
    hi[k] = (_Float16)x;
    lo[k] = (_Float16)(x - (float)hi[k]);
  }
  *H.at(c, q * 4) = hi;
  *H.at(c, 16 + q * 4) = lo;
  __syncthreads();
  const s16x8 p = H.along(0, 0, lane);
  const float scale = ldexpf(f, e);
  for (int t = wave; t < wide / 16; t += kWaves) {
    // X's 16 rows or columns again for the second half of k.
    const int k0 = (q & 1) * 8 - q * 8;
    acc = f32x4{0.f, 0.f, 0.f, 0.f};
    if (tall) acc = mfma<_Float16>(p, X.along(t * 16, k0, lane), acc);
    else acc = mfma<_Float16>(X.across(t * 16, k0, lane), p, acc);
    float v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = scale * acc[k];
    small_store(a, (tall ? t * 16 : 0) + c, (tall ? 0 : t * 16) + q * 4, v);
  }
}

template <int EPI, int AF, int BF, int TILE>
int go(const OrthoArgs& a, int64_t blocks, void* stream) {
  return launch(&ortho_kernel<EPI, AF, BF, TILE>, a, blocks, kTileThreads[TILE], CoreOf<_Float16, AF, BF, TILE, true>::kLds, stream);
}
template <int EPI, int AF, int BF>
int go(const OrthoArgs& a, int tile, int64_t blocks, void* stream) {
  if (tile == kTile256) return go<EPI, AF, BF, kTile256>(a, blocks, stream);
  if (tile == kTile128) return go<EPI, AF, BF, kTile128>(a, blocks, stream);
  return go<EPI, AF, BF, kTile64>(a, blocks, stream);
}

}  // namespace

// A wave goes through as many tiles as its kernel was made for, so a rung takes about its
// own time whatever the tiles are; the rungs are at most 1.7 times apart from three on.
// Sides are 2, 4, 6 or 8 tiles where they are the shorter, so the n x n results 4, 16, 36
// or 64.
template <typename T, int MX>
int go_small(const OrthoSmallArgs& a, int64_t batch, int n_tiles, int lds, void* stream) {
  if constexpr (MX > 1) {
    if (n_tiles > 8) {
      if constexpr (MX > 5)
        if (n_tiles > 40) return launch(&ortho_small_kernel<T, MX, 8>, a, batch, kSmallThreads, lds, stream);
      if constexpr (MX > 3)
        if (n_tiles > 16) return launch(&ortho_small_kernel<T, MX, 5>, a, batch, kSmallThreads, lds, stream);
      return launch(&ortho_small_kernel<T, MX, 2>, a, batch, kSmallThreads, lds, stream);
    }
  }
  return launch(&ortho_small_kernel<T, MX, 1>, a, batch, kSmallThreads, lds, stream);
}
template <typename T>
int go_small(const OrthoSmallArgs& a, int64_t batch, int lds, void* stream) {
  const int side = (a.rp < a.cp ? a.rp : a.cp) / 16, tiles = (a.rp / 16) * (a.cp / 16), n = side * side;
  if (tiles <= 8) return go_small<T, 1>(a, batch, n, lds, stream);
  if (tiles <= 16) return go_small<T, 2>(a, batch, n, lds, stream);
  if (tiles <= 24) return go_small<T, 3>(a, batch, n, lds, stream);
  if (tiles <= 40) return go_small<T, 5>(a, batch, n, lds, stream);
  return go_small<T, 8>(a, batch, n, lds, stream);
}

int launch_ortho_small(const OrthoSmallArgs& a, int64_t batch, void* stream) {
  if (a.is_short) {
    const int lds = a.rows > a.cols ? a.rp * (16 * 2 + 16) : 16 * (a.cp * 2 + 16);
    return a.src_dt == ZERO_BF16 ? launch(&ortho_short_kernel<__bf16>, a, batch, kShortThreads, lds, stream)
                                 : launch(&ortho_short_kernel<_Float16>, a, batch, kShortThreads, lds, stream);
  }
  const int side = a.rp < a.cp ? a.rp : a.cp;
  const int lds = a.rp * (a.cp * 2 + 16) + 2 * side * (side * 2 + 16);
  return a.src_dt == ZERO_BF16 ? go_small<__bf16>(a, batch, lds, stream) : go_small<_Float16>(a, batch, lds, stream);
}

int launch_ortho_thin(const OrthoThinArgs& a, int64_t batch, void* stream) {
  const int lds = 4 * kThinSide * (kThinSide + 4) * 4;
  switch ((a.side + 15) / 16) {
    case 1: return launch(&ortho_thin_kernel<1>, a, batch, kThinThreads, lds, stream);
    case 2: return launch(&ortho_thin_kernel<2>, a, batch, kThinThreads, lds, stream);
    case 3: return launch(&ortho_thin_kernel<3>, a, batch, kThinThreads, lds, stream);
    default: return launch(&ortho_thin_kernel<4>, a, batch, kThinThreads, lds, stream);
  }
}

int launch_ortho_norm(const OrthoLoadArgs& a, int dt, void* stream) {
  const int64_t blocks = (int64_t)a.batch * a.norm_blocks;
  return dt == ZERO_BF16 ? launch(&ortho_norm_kernel<__bf16>, a, blocks, kLoadThreads, 0, stream)
                         : launch(&ortho_norm_kernel<_Float16>, a, blocks, kLoadThreads, 0, stream);
}

int launch_ortho_load(const OrthoLoadArgs& a, int dt, int64_t blocks, void* stream) {
  return dt == ZERO_BF16 ? launch(&ortho_load_kernel<__bf16>, a, blocks, kLoadThreads, 0, stream)
                         : launch(&ortho_load_kernel<_Float16>, a, blocks, kLoadThreads, 0, stream);
}

int launch_ortho(const OrthoArgs& a, int tile, int64_t blocks, void* stream) {
  if (a.epi == kGram)
    return a.tall ? go<kGram, kFormM, kFormM>(a, tile, blocks, stream) : go<kGram, kFormK, kFormK>(a, tile, blocks, stream);
  if (a.epi == kPoly) return go<kPoly, kFormK, kFormK>(a, tile, blocks, stream);
  return a.tall ? go<kNext, kFormK, kFormK>(a, tile, blocks, stream) : go<kNext, kFormK, kFormM>(a, tile, blocks, stream);
}

int launch_ortho_join(const OrthoArgs& a, int64_t blocks, void* stream) {
  if (a.epi == kGram) return launch(&ortho_join_kernel<kGram>, a, blocks, kJoinThreads, 0, stream);
  if (a.epi == kPoly) return launch(&ortho_join_kernel<kPoly>, a, blocks, kJoinThreads, 0, stream);
  return launch(&ortho_join_kernel<kNext>, a, blocks, kJoinThreads, 0, stream);
}

}  // namespace hidden
}  // namespace zk
