// zero_hidden_dev.h -- what zero_linear.hip and zero_muon.hip share: element
// access, tile shapes, partial sums and launching.
#pragma once

#include "zero_gemm.h"
#include "zero_hidden.h"

#pragma clang fp contract(off)

namespace zk {
namespace hidden {
namespace {

using namespace zk::gemm;

#define AS1 __attribute__((address_space(1)))

template <int DT>
struct ElemOf;
template <>
struct ElemOf<ZERO_F16> { typedef _Float16 T; };
template <>
struct ElemOf<ZERO_BF16> { typedef __bf16 T; };

// V consecutive 16-bit elements at element alignment, `have` of which exist.
template <typename T, int V>
__device__ __forceinline__ void load_row(const void* base, int64_t e, int have, float (&x)[V]) {
  typedef T tv __attribute__((ext_vector_type(V)));
  typedef tv __attribute__((aligned(2))) tvu;
  const AS1 T* p = (const AS1 T*)base + e;
  if (have >= V) {
    const tv v = *(const AS1 tvu*)p;
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = (float)v[i];
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = i < have ? (float)p[i] : 0.0f;
  }
}

// The same in two steps: the load, and its values when they are needed.
template <typename T, int V>
struct Row {
  typedef T tv __attribute__((ext_vector_type(V)));
  tv v;
  __device__ __forceinline__ void load(const void* base, int64_t e, int have) {
    typedef tv __attribute__((aligned(2))) tvu;
    const AS1 T* p = (const AS1 T*)base + e;
    if (have >= V) {
      v = *(const AS1 tvu*)p;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = i < have ? p[i] : (T)0.0f;
    }
  }
};

template <typename T, int V>
__device__ __forceinline__ void store_row(void* base, int64_t e, int have, const float (&x)[V]) {
  typedef T tv __attribute__((ext_vector_type(V)));
  typedef tv __attribute__((aligned(2))) tvu;
  AS1 T* p = (AS1 T*)base + e;
  if (have >= V) {
    tv v;
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = (T)x[i];
    *(AS1 tvu*)p = v;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < have) p[i] = (T)x[i];
  }
}

template <int TILE>
struct Shape;
template <>
struct Shape<kTile256> { static constexpr int BM = 256, BN = 256, WM = 2, WN = 4; };
template <>
struct Shape<kTile128> { static constexpr int BM = 128, BN = 128, WM = 2, WN = 2; };
template <>
struct Shape<kTile64> { static constexpr int BM = 64, BN = 64, WM = 2, WN = 2; };

template <typename T, int AF, int BF, int TILE, bool DIRECT>
using CoreOf = Core<T, AF, BF, Shape<TILE>::BM, Shape<TILE>::BN, Shape<TILE>::WM, Shape<TILE>::WN, DIRECT>;

// The work of one workgroup: a tile, whole or a piece of k of it.
struct Work {
  int z, im, in;        // which result, which tile
  int cut, split;       // which of the cut tiles (-1: whole), which piece
  int k0, k_end;
};

// UPPER: the result is symmetric, tiles on and above the diagonal only.
template <bool UPPER>
__device__ __forceinline__ void tile_at(const Product& p, int t, int& z, int& im, int& in) {
  z = t / p.tiles;
  if constexpr (UPPER) place_upper(t - z * p.tiles, im, in);
  else place(t - z * p.tiles, p.tm, p.tn, im, in);
}

template <bool UPPER>
__device__ __forceinline__ Work work_of(const Product& p, int b) {
  Work w;
  int tile;
  if (b < p.whole) {
    tile = die_order(b, p.whole);
    w.cut = -1;
    w.split = 0;
    w.k0 = 0;
    w.k_end = p.k;
  } else {
    // Pieces of one k lie together, so that a die's workgroups read the same rows.
    const int t = die_order(b - p.whole, p.cut * p.splits);
    w.split = t / p.cut;
    w.cut = t - w.split * p.cut;
    tile = p.whole + w.cut;
    w.k0 = w.split * p.k_piece;
    w.k_end = p.k - w.k0 < p.k_piece ? p.k : w.k0 + p.k_piece;
  }
  tile_at<UPPER>(p, tile, w.z, w.im, w.in);
  w.z = __builtin_amdgcn_readfirstlane(w.z);       // the root leaves them in vector registers
  w.im = __builtin_amdgcn_readfirstlane(w.im);
  w.in = __builtin_amdgcn_readfirstlane(w.in);
  return w;
}

__device__ __forceinline__ void store_part(const Product& p, const Work& w, int row, int col, const float (&v)[8]) {
  AS1 float* d = (AS1 float*)p.part + (((int64_t)w.cut * p.splits + w.split) * p.size + (row - w.im * p.size)) * p.size + (col - w.in * p.size);
  *(AS1 f32x4*)d = f32x4{v[0], v[1], v[2], v[3]};
  *(AS1 f32x4*)(d + 4) = f32x4{v[4], v[5], v[6], v[7]};
}

// Sums a workgroup's work (operands of several results za and zb elements apart);
// partial sums go where they are joined from.  Returns whether the tile is whole:
// tile (m0, n0) of result z.
template <bool UPPER, typename C>
__device__ __forceinline__ bool run_tile(C& core, ZK_LDS char* lds, const Product& p, int b, int64_t za, int64_t zb, int& z, int& m0,
                                         int& n0) {
  const Work w = work_of<UPPER>(p, b);
  z = w.z;
  m0 = w.im * p.size;
  n0 = w.in * p.size;
  core.run(lds, (const uint16_t*)p.a + z * za, p.lda, p.m, (const uint16_t*)p.b + z * zb, p.ldb, p.n, m0, n0, w.k0, w.k_end);
  if (w.cut < 0) return true;
  core.template each<int>(lds, m0, n0, false, [](int, int, int&) {}, [&](int row, int col, const float (&v)[8], int) {
    if (row < p.m && col < p.n) store_part(p, w, row, col, v);
  }, 0);
  return false;
}

// Four columns of a row of a cut tile from its pieces' sums, in the order of the
// pieces.
template <bool UPPER>
__device__ __forceinline__ bool join4(const Product& p, int64_t unit, int& z, int& row, int& col, float (&v)[4], bool& twice) {
  const int upr = p.size >> 2, per = p.size * upr;
  const int cut = (int)(unit / per), u = (int)(unit - (int64_t)cut * per);
  if (cut >= p.cut) return false;
  int im, in;
  tile_at<UPPER>(p, p.whole + cut, z, im, in);
  const int r = u / upr, c = u % upr * 4;
  row = im * p.size + r;
  col = in * p.size + c;
  twice = UPPER && im != in;
  if (row >= p.m || col >= p.n) return false;
  const AS1 f32x4* s = (const AS1 f32x4*)((const AS1 float*)p.part + ((int64_t)cut * p.splits * p.size + r) * p.size + c);
  const int64_t step = (int64_t)p.size * upr;
  f32x4 t = s[0];
  for (int i = 1; i < p.splits; ++i) {
    s += step;
    t += *s;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = t[i];
  return true;
}

template <typename K, typename A>
int launch(K kernel, const A& a, int64_t blocks, int threads, int lds, void* stream) {
  if (lds > 65536) {   // more than a launch is given without asking
    const hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) {
      (void)hipGetLastError();
      return (int)e;
    }
  }
  void* args[] = {(void*)&a};
  return (int)hipLaunchKernel((const void*)kernel, dim3((unsigned)blocks), dim3((unsigned)threads), args, (size_t)lds,
                              (hipStream_t)stream);
}

}  // namespace
}  // namespace hidden
}  // namespace zk
