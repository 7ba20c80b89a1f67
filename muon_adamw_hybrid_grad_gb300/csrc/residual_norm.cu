// The residual's addition with RMS norm, forward, and the C entry points.
//
//   r = residual + drop(x),   y = w r / sqrt(mean(r^2) + eps)
//
// One pass: a row stays in registers between its sum of squares and its output,
// and the norm is of r in fp32, before r is rounded for the stream. With 8 bits
// a second reduction finds the row's largest |y|.
//
// Bound by HBM: two rows in, two out. Rows of up to 1024 elements are a warp's
// own, which needs no barrier, and a thread's loads are all in flight at once.
#include <cuda_fp8.h>

#include <cfloat>
#include <cmath>

#include "residual_norm.cuh"

namespace ma {
namespace {

constexpr int kMinThreads = 128;

template <int T>
struct RowThreads {
  static constexpr int kBlock = T == 32 ? kMinThreads : T;
  static constexpr int kRows = kBlock / T;
  static_assert(T == 32 || kRows == 1, "several warps share a row: one row to a block");
};

// Sum or maximum over the threads of a row, in an order of their own.
template <int T, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* shared) {
  v = MAX ? warp_max(v) : warp_sum(v);
  if constexpr (T > 32) {
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
    __syncthreads();
    v = shared[0];
#pragma unroll
    for (int i = 1; i < T / 32; ++i) v = MAX ? fmaxf(v, shared[i]) : v + shared[i];
  }
  return v;
}

template <typename TX, typename TS, int T, int V, bool VEC>
__global__ void __launch_bounds__(RowThreads<T>::kBlock) residual_norm_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float shared[2][32];
  const int t = T == 32 ? threadIdx.x & 31 : threadIdx.x;
  const int64_t row = (int64_t)blockIdx.x * RowThreads<T>::kRows + (T == 32 ? threadIdx.x >> 5 : 0);
  pdl_wait();
  pdl_launch();
  if (row >= a.n) return;  // whole rows
  const TX* const x = static_cast<const TX*>(a.x) + row * a.xs;
  const TS* const res = a.residual ? static_cast<const TS*>(a.residual) + row * a.rs : nullptr;
  RowVec<TX, VEC> rx[V];
  RowVec<TS, VEC> rr[V];
#pragma unroll
  for (int j = 0; j < V; ++j) rx[j].load(x, col_of<VEC, T>(j, t), a.w);
  if (res) {
#pragma unroll
    for (int j = 0; j < V; ++j) rr[j].load(res, col_of<VEC, T>(j, t), a.w);
  }
  float r[V][8];
#pragma unroll
  for (int j = 0; j < V; ++j) rx[j].get(col_of<VEC, T>(j, t), a.w, r[j]);
  if (a.drop.threshold) drop_row<VEC, T>(drop_key(a.drop), row * a.w, t, r);
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int col = col_of<VEC, T>(j, t);
    if (res) {
      float s[8];
      rr[j].get(col, a.w, s);
#pragma unroll
      for (int e = 0; e < 8; ++e) r[j][e] += s[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(r[j][e], r[j][e], ss);
    if (a.res) store_row<VEC>(static_cast<TS*>(a.res) + row * a.w, col, a.w, r[j]);
  }
  ss = row_reduce<T, false>(ss, shared[0]);
  const float rstd = rsqrtf(ss / (float)a.w + a.eps);
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int col = col_of<VEC, T>(j, t);
    float w[8];
    load_weight<VEC>(a.weight, col, a.w, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      r[j][e] *= rstd * w[e];
      top = fmaxf(top, fabsf(r[j][e]));
    }
    if (!a.scales) store_row<VEC>(static_cast<TX*>(a.y) + row * a.w, col, a.w, r[j]);
  }
  if (!a.scales) return;
  top = row_reduce<T, true>(top, shared[1]);
  if (t == 0) a.scales[row] = top / 448.f;
  // a factor that keeps 448 / top finite where top is next to nothing
  const float up = top < 1e-30f ? 0x1p64f : 1.f;
  const float inv = top > 0.f ? 448.f / (top * up) : 0.f;
  uint8_t* const q = static_cast<uint8_t*>(a.y) + row * a.w;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int col = col_of<VEC, T>(j, t);
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i] = __nv_cvt_float2_to_fp8x2(make_float2(r[j][2 * i] * up * inv, r[j][2 * i + 1] * up * inv), __NV_SATFINITE,
                                      __NV_E4M3);
    if constexpr (VEC) {
      if (col < a.w) *reinterpret_cast<uint2*>(q + col) = make_uint2(p[0] | p[1] << 16, p[2] | p[3] << 16);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (col + 32 * e < a.w) q[col + 32 * e] = (uint8_t)(p[e / 2] >> (8 * (e & 1)));
    }
  }
}

template <typename TX, typename TS, int T, int V, bool VEC>
cudaError_t launch(const NormArgs& a, cudaStream_t st) {
  const int64_t per = RowThreads<T>::kRows;
  return op_launch(residual_norm_kernel<TX, TS, T, V, VEC>, dim3((unsigned)((a.n + per - 1) / per)),
                   dim3(RowThreads<T>::kBlock), 0, st, 1, a);
}

template <typename TX, typename TS>
cudaError_t forward(const NormArgs& a, bool vec, cudaStream_t st) {
  const int units = (a.w + 7) / 8;
  if (!vec) {
    if (units <= 32) return launch<TX, TS, 32, 1, false>(a, st);
    if (units <= 128) return launch<TX, TS, 64, 2, false>(a, st);
    if (units <= 256) return launch<TX, TS, 128, 2, false>(a, st);
    if (units <= 384) return launch<TX, TS, 192, 2, false>(a, st);
    if (units <= 512) return launch<TX, TS, 128, 4, false>(a, st);
    if (units <= 1024) return launch<TX, TS, 256, 4, false>(a, st);
    return launch<TX, TS, 512, 8, false>(a, st);
  }
  // Two to four vectors a thread: enough loads in flight, and warps enough to hide the generator. 64M elements of bf16
  // without and with dropout: width 1024 with (threads, vectors) = (32, 4) 78 and 85 us, (64, 2) 77 and 83; 2048 with
  // (32, 8) 79 and 102, (128, 2) 77 and 84, (256, 1) 77 and 94; 8192 with (128, 8) 86, (256, 4) 85 and 100, (512, 2) 95
  // and 98; 16384 with (256, 8) 111 and 162, (512, 4) 104 and 111, (1024, 2) 105 and 134.
  if (units <= 32) return launch<TX, TS, 32, 1, true>(a, st);
  if (units <= 64) return launch<TX, TS, 32, 2, true>(a, st);
  if (units <= 128) return launch<TX, TS, 64, 2, true>(a, st);
  if (units <= 256) return launch<TX, TS, 128, 2, true>(a, st);
  if (units <= 384) return launch<TX, TS, 192, 2, true>(a, st);
  if (units <= 512) return launch<TX, TS, 128, 4, true>(a, st);
  if (units <= 1024) return launch<TX, TS, 256, 4, true>(a, st);
  if (units <= 2048) return launch<TX, TS, 512, 4, true>(a, st);
  return launch<TX, TS, 512, 8, true>(a, st);
}

ma_status check(const ma_residual_norm* d, const float* weight) {
  if (!d) return op_fail(MA_ERR_ARG, "the description must not be NULL");
  if (!op_dtype_ok(d->dtype) || !op_dtype_ok(d->stream_dtype))
    return op_fail(MA_ERR_DTYPE, "dtype %d or stream_dtype %d is neither MA_DT_F32 nor MA_DT_BF16", d->dtype,
                   d->stream_dtype);
  if (d->dtype == MA_DT_F32 && d->stream_dtype == MA_DT_BF16)
    return op_fail(MA_ERR_DTYPE, "a stream of bf16 takes no fp32 branch");
  if (d->n_tokens < 0 || d->n_tokens > (1ll << 30) || d->width < 1 || d->width > kNormMaxWidth)
    return op_fail(MA_ERR_SHAPE, "%lld tokens of %lld elements: outside [0, 2^30] or [1, %d]", (long long)d->n_tokens,
                   (long long)d->width, kNormMaxWidth);
  // squares below the smallest normal number may be lost: eps, which is at least that, outweighs them
  if (!((float)d->eps >= FLT_MIN) || !std::isfinite((float)d->eps))
    return op_fail(MA_ERR_ARG, "eps = %g is no positive normal number in fp32", d->eps);
  DropArgs drop;
  if (!drop_args(d->p, d->rng, d->site, &drop)) return op_fail(MA_ERR_ARG, "p = %g outside [0, 1]", d->p);
  if (drop.threshold) {
    if (!d->rng) return op_fail(MA_ERR_ARG, "dropout needs rng");
    if (!op_aligned(d->rng, 8)) return op_fail(MA_ERR_ALIGN, "rng is not aligned to 8 bytes");
    if (d->site < 0) return op_fail(MA_ERR_ARG, "site %d is negative", d->site);
    if (d->n_tokens * d->width > MA_DROPOUT_MAX_ELEMENTS)
      return op_fail(MA_ERR_SHAPE, "dropout of more than 2^35 elements");
  }
  if (!weight) return op_fail(MA_ERR_ARG, "weight must not be NULL");
  if (!op_aligned(weight, 4)) return op_fail(MA_ERR_ALIGN, "weight is not aligned to 4 bytes");
  return MA_OK;
}

// A tensor of d's rows; `vec` becomes false where they allow no 16-byte access.
ma_status check_rows(const ma_residual_norm* d, const char* name, const void* p, int dtype, int64_t stride, bool* vec) {
  const int64_t e = op_dtype_size(dtype);
  if (!p) return op_fail(MA_ERR_ARG, "%s must not be NULL", name);
  if (!op_aligned(p, e)) return op_fail(MA_ERR_ALIGN, "%s is not aligned to its elements", name);
  if (d->n_tokens > 1 && stride < d->width)
    return op_fail(MA_ERR_SHAPE, "%s has rows %lld apart, below the width", name, (long long)stride);
  if (!op_aligned(p, 16) || (d->n_tokens > 1 && stride * e % 16)) *vec = false;
  return MA_OK;
}

NormArgs args_of(const ma_residual_norm* d, const float* weight) {
  NormArgs a{};
  a.n = d->n_tokens;
  a.w = (int)d->width;
  a.eps = (float)d->eps;
  drop_args(d->p, d->rng, d->site, &a.drop);
  a.weight = weight;
  return a;
}

}  // namespace

cudaError_t residual_norm_forward(const NormArgs& a, int dtype, int stream_dtype, bool vec, cudaStream_t st) {
  if (dtype == MA_DT_F32) return forward<float, float>(a, vec, st);
  return stream_dtype == MA_DT_F32 ? forward<__nv_bfloat16, float>(a, vec, st)
                                   : forward<__nv_bfloat16, __nv_bfloat16>(a, vec, st);
}

}  // namespace ma

using namespace ma;

extern "C" {

ma_status muon_adamw_residual_norm(const ma_residual_norm* d, const void* x, int64_t x_stride, const void* residual,
                                   int64_t residual_stride, const float* weight, void* y, float* scales, void* res,
                                   void* cuda_stream) {
  ma_status st = check(d, weight);
  if (st != MA_OK) return st;
  if (d->n_tokens > 0) {
    bool vec = d->width % 8 == 0 && op_aligned(weight, 16);
    st = check_rows(d, "x", x, d->dtype, x_stride, &vec);
    if (st == MA_OK && residual) st = check_rows(d, "residual", residual, d->stream_dtype, residual_stride, &vec);
    if (st == MA_OK && res) st = check_rows(d, "res", res, d->stream_dtype, d->width, &vec);
    if (st == MA_OK && !scales) st = check_rows(d, "y", y, d->dtype, d->width, &vec);
    if (st != MA_OK) return st;
    if (scales) {
      if (!y) return op_fail(MA_ERR_ARG, "y must not be NULL");
      if (!op_aligned(scales, 4)) return op_fail(MA_ERR_ALIGN, "scales is not aligned to 4 bytes");
      if (!op_aligned(y, 8)) vec = false;
    }
    NormArgs a = args_of(d, weight);
    a.x = x;
    a.xs = x_stride;
    a.residual = residual;
    a.rs = residual_stride;
    a.y = y;
    a.scales = scales;
    a.res = res;
    const cudaError_t e = residual_norm_forward(a, d->dtype, d->stream_dtype, vec, static_cast<cudaStream_t>(cuda_stream));
    if (e != cudaSuccess) return op_cuda(e, "residual norm launch");
  }
  clear_last_error();
  return MA_OK;
}

ma_status muon_adamw_residual_norm_backward_workspace(const ma_residual_norm* d, int64_t* bytes) {
  if (!bytes) return op_fail(MA_ERR_ARG, "bytes must not be NULL");
  static const float one = 1.f;
  const ma_status st = check(d, &one);
  if (st != MA_OK) return st;
  *bytes = residual_norm_backward_space(d->n_tokens, (int)d->width);
  clear_last_error();
  return MA_OK;
}

ma_status muon_adamw_residual_norm_backward(const ma_residual_norm* d, const void* dy, int64_t dy_stride,
                                            const void* dres, int64_t dres_stride, const void* res, int64_t res_stride,
                                            const float* weight, void* dx, void* dresidual, float* dweight,
                                            void* workspace, int64_t workspace_bytes, void* cuda_stream) {
  ma_status st = check(d, weight);
  if (st != MA_OK) return st;
  if (!dweight) return op_fail(MA_ERR_ARG, "dweight must not be NULL");
  if (!op_aligned(dweight, 4)) return op_fail(MA_ERR_ALIGN, "dweight is not aligned to 4 bytes");
  if (!workspace || !op_aligned(workspace, 256))
    return op_fail(workspace ? MA_ERR_ALIGN : MA_ERR_ARG, "workspace is NULL or not 256-byte aligned");
  const int64_t need = residual_norm_backward_space(d->n_tokens, (int)d->width);
  if (workspace_bytes < need)
    return op_fail(MA_ERR_ARG, "workspace of %lld bytes, %lld are needed", (long long)workspace_bytes, (long long)need);
  bool vec = d->width % 8 == 0 && op_aligned(weight, 16);
  NormArgs a = args_of(d, weight);
  if (d->n_tokens > 0) {
    st = check_rows(d, "dy", dy, d->dtype, dy_stride, &vec);
    if (st == MA_OK && dres) st = check_rows(d, "dres", dres, d->stream_dtype, dres_stride, &vec);
    if (st == MA_OK) st = check_rows(d, "res", res, d->stream_dtype, res_stride, &vec);
    if (st == MA_OK) st = check_rows(d, "dresidual", dresidual, d->stream_dtype, d->width, &vec);
    if (st == MA_OK && dx) st = check_rows(d, "dx", dx, d->dtype, d->width, &vec);
    if (st != MA_OK) return st;
    if (!dx && (a.drop.threshold || d->dtype != d->stream_dtype))
      return op_fail(MA_ERR_ARG, "dx must not be NULL: it is not dresidual");
  }
  a.dy = dy;
  a.dys = dy_stride;
  a.dres = dres;
  a.dress = dres_stride;
  a.r = res;
  a.ress = res_stride;
  a.dx = dx;
  a.dr = dresidual;
  a.partial = static_cast<float*>(workspace);
  a.dweight = dweight;
  const cudaError_t e = residual_norm_backward(a, d->dtype, d->stream_dtype, vec, static_cast<cudaStream_t>(cuda_stream));
  if (e != cudaSuccess) return op_cuda(e, "residual norm gradient launch");
  clear_last_error();
  return MA_OK;
}

}  // extern "C"
