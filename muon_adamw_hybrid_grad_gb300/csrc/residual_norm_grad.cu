// Gradient of the residual's addition with RMS norm.
//
//   g = dy w,  c = mean(g r) rstd^3,  dr = dres + rstd g - c r,
//   dx = drop(dr),  dw = sum over rows of dy r rstd
//
// One pass over dy, dres and r: both of a row's sums are formed together, so it
// waits once for its threads. Bound by HBM (three rows in, two out). Blocks are
// persistent: each keeps its columns' share of dw in registers over its rows,
// loads a row while it finishes the one before, and leaves one partial row; a
// second launch adds those up in a fixed order.
#include <algorithm>
#include <cmath>

#include "residual_norm.cuh"

namespace ma {
namespace {

template <int T>
struct RowGroups {
  static constexpr int kBlock = T < 256 ? 256 : T;
  static constexpr int kGroups = kBlock / T;  // rows at a time
};

constexpr int kMaxBlocks = 1024;  // rows of partial sums

template <int T>
__device__ __forceinline__ void group_barrier(int group) {
  if constexpr (RowGroups<T>::kGroups == 1)
    __syncthreads();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(T) : "memory");
}

template <typename TX, typename TS, int V, bool VEC>
struct GradRow {
  RowVec<TX, VEC> dy[V];
  RowVec<TS, VEC> r[V], dres[V];
  template <int T>
  __device__ __forceinline__ void load(const NormArgs& a, int64_t row, int t) {
    const TX* const py = static_cast<const TX*>(a.dy) + row * a.dys;
    const TS* const pr = static_cast<const TS*>(a.r) + row * a.ress;
#pragma unroll
    for (int j = 0; j < V; ++j) dy[j].load(py, (j * T + t) * 8, a.w);
#pragma unroll
    for (int j = 0; j < V; ++j) r[j].load(pr, (j * T + t) * 8, a.w);
    if (a.dres) {
      const TS* const pd = static_cast<const TS*>(a.dres) + row * a.dress;
#pragma unroll
      for (int j = 0; j < V; ++j) dres[j].load(pd, (j * T + t) * 8, a.w);
    }
  }
};

template <typename TX, typename TS, int T, int V, bool VEC>
__global__ void __launch_bounds__(RowGroups<T>::kBlock) residual_norm_grad_kernel(const __grid_constant__ NormArgs a) {
  constexpr int G = RowGroups<T>::kGroups;
  constexpr bool AHEAD = V <= 2;  // registers for a second row
  extern __shared__ float shared[];  // [2][G][T / 32][2] sums, then a row of dw
  float* const sums = shared;
  const int group = threadIdx.x / T, t = threadIdx.x % T, warp = t >> 5, lane = t & 31;
  pdl_wait();
  pdl_launch();
  const int64_t step = (int64_t)gridDim.x * G;
  DropKey key{};
  if (a.drop.threshold) key = drop_key(a.drop);
  float dw[V][8];
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[j][e] = 0.f;
  GradRow<TX, TS, V, VEC> next;
  int64_t row = (int64_t)blockIdx.x * G + group;
  if (AHEAD && row < a.n) next.template load<T>(a, row, t);
  for (int parity = 0; row < a.n; row += step, parity ^= 1) {
    GradRow<TX, TS, V, VEC> cur;
    if constexpr (AHEAD) {
      cur = next;
      if (row + step < a.n) next.template load<T>(a, row + step, t);
    } else {
      cur.template load<T>(a, row, t);
    }
    float ss = 0.f, gr = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = (j * T + t) * 8;
      float dy[8], r[8], w[8];
      cur.dy[j].get(col, a.w, dy);
      cur.r[j].get(col, a.w, r);
      load_weight<VEC>(a.weight, col, a.w, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ss = fmaf(r[e], r[e], ss);
        gr = fmaf(dy[e] * w[e], r[e], gr);
      }
    }
    ss = warp_sum(ss);
    gr = warp_sum(gr);
    if constexpr (T > 32) {
      float2* const at = reinterpret_cast<float2*>(sums) + (parity * G + group) * (T / 32);
      if (lane == 0) at[warp] = make_float2(ss, gr);
      group_barrier<T>(group);
      ss = gr = 0.f;
#pragma unroll
      for (int i = 0; i < T / 32; ++i) {
        const float2 v = at[i];
        ss += v.x;
        gr += v.y;
      }
    }
    const float rstd = rsqrtf(ss / (float)a.w + a.eps);
    const float c = gr / (float)a.w * rstd * rstd * rstd;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = (j * T + t) * 8;
      float dy[8], r[8], w[8], d[8];
      cur.dy[j].get(col, a.w, dy);
      cur.r[j].get(col, a.w, r);
      load_weight<VEC>(a.weight, col, a.w, w);
      if (a.dres) {
        cur.dres[j].get(col, a.w, d);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        d[e] += fmaf(rstd * dy[e], w[e], -c * r[e]);
        dw[j][e] = fmaf(dy[e], r[e] * rstd, dw[j][e]);
      }
      store_row<VEC>(static_cast<TS*>(a.dr) + row * a.w, col, a.w, d);
      if (a.dx) {
        if (a.drop.threshold && col < a.w) drop8_at<VEC>(key, row * a.w + col, d);
        store_row<VEC>(static_cast<TX*>(a.dx) + row * a.w, col, a.w, d);
      }
    }
  }
  // the groups' shares of dw, one after the other
  float* const sum = shared + 4 * G * (T / 32);
  if constexpr (G > 1) {
    for (int g = 0; g < G; ++g) {
      if (group == g) {
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float* const at = sum + ((j * 8 + e) * T + t);
            dw[j][e] += g ? *at : 0.f;
            *at = dw[j][e];
          }
      }
      __syncthreads();
    }
    if (group != G - 1) return;
  }
  float* const out = a.partial + (int64_t)blockIdx.x * a.w;
#pragma unroll
  for (int j = 0; j < V; ++j) store_row<VEC>(out, (j * T + t) * 8, a.w, dw[j]);
}

// dw from the blocks' rows: eight threads a column, then those eight.
__global__ void __launch_bounds__(256) residual_norm_join_kernel(const float* __restrict__ partial, int rows, int w,
                                                                 float* __restrict__ dweight) {
  __shared__ float sum[8][32];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, col = blockIdx.x * 32 + x;
  pdl_wait();
  pdl_launch();
  float s = 0.f;
  if (col < w) {
#pragma unroll 8
    for (int i = y; i < rows; i += 8) s += partial[(int64_t)i * w + col];
  }
  sum[y][x] = s;
  __syncthreads();
  if (y == 0 && col < w) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += sum[i][x];
    dweight[col] = s;
  }
}

template <typename TX, typename TS, int T, int V, bool VEC>
cudaError_t launch(const NormArgs& a, cudaStream_t st) {
  using R = RowGroups<T>;
  constexpr int kSmem = 4 * (4 * R::kGroups * (T / 32) + (R::kGroups > 1 ? T * V * 8 : 0));
  const auto kernel = residual_norm_grad_kernel<TX, TS, T, V, VEC>;
  int sms = 0, *err = nullptr, blocks = 0;
  cudaError_t e = op_device(&sms, &err);
  if (e != cudaSuccess) return e;
  if (a.n > 0) {
    static const int per_sm = [&] {
      int k = 0;
      return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&k, kernel, R::kBlock, kSmem) == cudaSuccess && k > 0 ? k : 1;
    }();
    blocks = (int)std::min<int64_t>(std::min(sms * per_sm, kMaxBlocks), (a.n + R::kGroups - 1) / R::kGroups);
    e = op_launch(kernel, dim3(blocks), dim3(R::kBlock), kSmem, st, 1, a);
    if (e != cudaSuccess) return e;
  }
  return op_launch(residual_norm_join_kernel, dim3((a.w + 31) / 32), dim3(256), 0, st, 1, (const float*)a.partial,
                   blocks, a.w, a.dweight);
}

template <typename TX, typename TS>
cudaError_t backward(const NormArgs& a, bool vec, cudaStream_t st) {
  const int units = (a.w + 7) / 8;
  if (!vec) {
    if (units <= 128) return launch<TX, TS, 64, 2, false>(a, st);
    if (units <= 1024) return launch<TX, TS, 256, 4, false>(a, st);
    return launch<TX, TS, 512, 8, false>(a, st);
  }
  if (units <= 32) return launch<TX, TS, 32, 1, true>(a, st);
  if (units <= 64) return launch<TX, TS, 32, 2, true>(a, st);
  if (units <= 128) return launch<TX, TS, 64, 2, true>(a, st);
  if (units <= 256) return launch<TX, TS, 128, 2, true>(a, st);
  if (units <= 512) return launch<TX, TS, 256, 2, true>(a, st);
  if (units <= 1024) return launch<TX, TS, 512, 2, true>(a, st);
  if (units <= 2048) return launch<TX, TS, 512, 4, true>(a, st);
  return launch<TX, TS, 512, 8, true>(a, st);
}

}  // namespace

int64_t residual_norm_backward_space(int64_t n, int w) { return std::min<int64_t>(n, kMaxBlocks) * w * 4 + 256; }

cudaError_t residual_norm_backward(const NormArgs& a, int dtype, int stream_dtype, bool vec, cudaStream_t st) {
  if (dtype == MA_DT_F32) return backward<float, float>(a, vec, st);
  return stream_dtype == MA_DT_F32 ? backward<__nv_bfloat16, float>(a, vec, st)
                                   : backward<__nv_bfloat16, __nv_bfloat16>(a, vec, st);
}

}  // namespace ma
