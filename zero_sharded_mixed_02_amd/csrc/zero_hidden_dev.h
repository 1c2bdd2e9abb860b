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

template <int V>
__device__ __forceinline__ void store_part(const Product& p, float* part, int split, int row, int col, const float* v) {
  AS1 float* d = (AS1 float*)(part + ((int64_t)split * p.m + row) * p.n_pad + col);
#pragma unroll
  for (int i = 0; i < V; i += 4)
    if (col + i < p.n) *(AS1 f32x4*)(d + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
}

// Four columns of a row from the pieces' sums, in the order of the pieces.
__device__ __forceinline__ bool join4(const Product& p, const float* part, int64_t unit, int& row, int& col, float (&v)[4]) {
  const int upr = p.n_pad >> 2;
  if (unit >= (int64_t)p.m * upr) return false;
  row = (int)(unit / upr);
  col = (int)(unit - (int64_t)row * upr) * 4;
  const AS1 f32x4* s = (const AS1 f32x4*)(part + (int64_t)row * p.n_pad + col);
  const int64_t step = (int64_t)p.m * p.n_pad / 4;
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
