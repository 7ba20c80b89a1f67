// Rows of the residual stream in registers: shared by the forward pass and the gradient.
//
// T threads share a row and hold V vectors of eight elements each. Each warp has
// V segments of 256 elements. VEC: the width is a multiple of 8 and all rows
// start on 16-byte boundaries; a lane's vector is eight elements in sequence.
// Otherwise it is every 32nd element of the segment, accessed one by one, so
// that a warp's accesses lie together either way.
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

// The first column of vector j of thread t, and the step to the next.
template <bool VEC, int T>
__device__ __forceinline__ int col_of(int j, int t) {
  return VEC ? (j * T + t) * 8 : (j * T + (t & ~31)) * 8 + (t & 31);
}
template <bool VEC>
constexpr int kColStep = VEC ? 1 : 32;

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
  T one[8];
  __device__ __forceinline__ void load(const T* row, int col, int w) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (col + 32 * e < w) one[e] = row[col + 32 * e];
  }
  __device__ __forceinline__ void get(int col, int w, float (&v)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = col + 32 * e < w ? load1(&one[e]) : 0.f;
  }
};

template <bool VEC, typename T>
__device__ __forceinline__ void store_row(T* row, int col, int w, const float (&v)[8]) {
  if constexpr (VEC) {
    if (col < w) store8(row + col, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (col + 32 * e < w) store1(row + col + 32 * e, v[e]);
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
  for (int e = 0; e < 8; ++e) v[e] = col + kColStep<VEC> * e < w ? weight[col + kColStep<VEC> * e] : 0.f;
}

// Dropout of vector j of thread t in the row whose first element is number `row0`; by whole warps.
template <bool VEC, int T>
__device__ __forceinline__ void drop_vector(const DropKey& k, int64_t row0, int j, int t, float (&x)[8]) {
  if constexpr (VEC) {
    drop8<1>(k, (uint32_t)(row0 >> 3) + (uint32_t)(j * T + t), 0, *reinterpret_cast<float(*)[1][8]>(&x));
  } else {
    // The segment's 256 elements begin `shift` elements into a group: a lane forms the bits of one of its groups and
    // of the 33rd, and element 32 e of lane t finds its own with lane (shift + t) / 8 + 4 e.
    const int64_t first = row0 + (j * T + (t & ~31)) * 8;
    const int shift = (int)(first & 7), lane = t & 31, at = shift + lane;
    const uint32_t group = (uint32_t)(first >> 3);
    uint4 c[2] = {make_uint4(group + lane, k.site, k.step0, k.step1), make_uint4(group + 32, k.site, k.step0, k.step1)};
    philox(c, k.k0, k.k1);
    const uint32_t threshold = k.threshold_up >> 16;
    auto word = [&](const uint4& v) { return at & 4 ? (at & 2 ? v.w : v.z) : (at & 2 ? v.y : v.x); };
    const uint32_t last = word(c[1]);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int from = at / 8 + 4 * e;
      const uint4 v = make_uint4(__shfl_sync(0xffffffffu, c[0].x, from & 31), __shfl_sync(0xffffffffu, c[0].y, from & 31),
                                 __shfl_sync(0xffffffffu, c[0].z, from & 31), __shfl_sync(0xffffffffu, c[0].w, from & 31));
      const uint32_t w = from < 32 ? word(v) : last;
      const bool keep = (at & 1 ? w >> 16 : w & 0xFFFFu) >= threshold;
      x[e] = keep && k.factor != 0.f ? x[e] * k.factor : 0.f;
    }
  }
}

// Of a thread's V vectors.
template <bool VEC, int T, int V>
__device__ __forceinline__ void drop_row(const DropKey& k, int64_t row0, int t, float (&x)[V][8]) {
  // in step where the registers allow it: 32765 rows of 2048 84 us, one by one 88; 16381 of 4096 86 and 91; eight
  // vectors, or four of wide rows, lose more by fewer warps
  constexpr int N = VEC && (V == 2 || (V == 4 && T == 128)) ? 2 : 1;
  if constexpr (N > 1) {
#pragma unroll
    for (int j = 0; j < V; j += N)
      drop8<N>(k, (uint32_t)(row0 >> 3) + (uint32_t)(j * T + t), T, *reinterpret_cast<float(*)[N][8]>(&x[j]));
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) drop_vector<VEC, T>(k, row0, j, t, x[j]);
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
