// Rows of the residual stream in registers: shared by the forward pass and the gradient.
//
// T threads share a row and hold V vectors of eight elements each: vector j of
// thread t is columns (j T + t) 8 onwards, so that a warp's accesses are whole
// lines. VEC: the width is a multiple of 8 and all rows start on 16-byte
// boundaries; otherwise elements are accessed one by one.
#pragma once

#include <utility>

#include "dropout.cuh"
#include "op_common.cuh"

namespace ma {

constexpr int kNormMaxWidth = 32768;  // 512 threads of eight vectors

struct NormArgs {
  int64_t n;
  int w;
  float eps;
  DropArgs drop;  // threshold 0: none
  const float* weight;
  const void *x, *residual;  // forward; residual may be NULL
  int64_t xs, rs;
  void* y;
  float* scales;  // forward, 8 bits
  void* res;      // forward: output, may be NULL
  const void *dy, *dres, *r;  // gradient; dres may be NULL
  int64_t dys, dress, ress;
  void *dx, *dr;  // dx may be NULL
  float *partial, *dweight;
};

cudaError_t residual_norm_forward(const NormArgs& a, int dtype, int stream_dtype, bool vec, cudaStream_t st);
cudaError_t residual_norm_backward(const NormArgs& a, int dtype, int stream_dtype, bool vec, cudaStream_t st);
int64_t residual_norm_backward_space(int64_t n, int w);  // bytes of partial sums

namespace {

template <typename T, bool VEC>
struct RowVec {
  RawVec<T, 8> raw;
  __device__ __forceinline__ void load(const T* row, int col, int w) {
    if (col < w) raw.load(row + col);
  }
  __device__ __forceinline__ void get(int col, int w, float (&v)[8]) const {
    if (col < w) {
      raw.get(v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 0.f;
    }
  }
};
template <typename T>
struct RowVec<T, false> {
  T v8[8];
  __device__ __forceinline__ void load(const T* row, int col, int w) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (col + e < w) v8[e] = row[col + e];
  }
  __device__ __forceinline__ void get(int col, int w, float (&v)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = col + e < w ? load1(&v8[e]) : 0.f;
  }
};

template <bool VEC, typename T>
__device__ __forceinline__ void store_row(T* row, int col, int w, const float (&v)[8]) {
  if constexpr (VEC) {
    if (col < w) store8(row + col, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (col + e < w) store1(row + col + e, v[e]);
  }
}

template <bool VEC>
__device__ __forceinline__ void load_weight(const float* weight, int col, int w, float (&v)[8]) {
  if constexpr (VEC) {
    if (col < w) {
      load8(weight + col, v);
      return;
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = col + e < w ? weight[col + e] : 0.f;
}

// Dropout of the eight elements from number `at` on. VEC: a multiple of 8.
template <bool VEC>
__device__ __forceinline__ void drop8_at(const DropKey& k, int64_t at, float (&x)[8]) {
  const uint32_t group = (uint32_t)(at >> 3);
  if (VEC || (at & 7) == 0) {
    drop8<1>(k, group, 0, *reinterpret_cast<float(*)[1][8]>(&x));
    return;
  }
  // the end of one group and the beginning of the next, the same shift for a whole row
  uint4 c[2] = {make_uint4(group, k.site, k.step0, k.step1), make_uint4(group + 1, k.site, k.step0, k.step1)};
  philox(c, k.k0, k.k1);
  uint32_t w[8] = {c[0].x, c[0].y, c[0].z, c[0].w, c[1].x, c[1].y, c[1].z, c[1].w};
  if (at & 4) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (at & 2) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  if (at & 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
  }
  drop8_by(k, make_uint4(w[0], w[1], w[2], w[3]), x);
}

// Of a thread's V vectors in the row whose first element is number `row0`.
template <bool VEC, int T, int V>
__device__ __forceinline__ void drop_row(const DropKey& k, int64_t row0, int t, float (&x)[V][8]) {
  if constexpr (VEC) {
    // in step where the registers allow it: 32765 rows of 2048 84 us, one by one 88; 16381 of 4096 86 and 91; eight
    // vectors, or four of wide rows, lose more by fewer warps
    constexpr int N = V == 2 || (V == 4 && T == 128) ? 2 : 1;
#pragma unroll
    for (int j = 0; j < V; j += N)
      drop8<N>(k, (uint32_t)(row0 >> 3) + (uint32_t)(j * T + t), T, *reinterpret_cast<float(*)[N][8]>(&x[j]));
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) drop8_at<false>(k, row0 + (j * T + t) * 8, x[j]);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}

}  // namespace
}  // namespace ma
