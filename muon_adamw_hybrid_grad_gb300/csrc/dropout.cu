// Dropout whose mask is never stored: forward and gradient are the same pass.
//
// Bound by HBM: a thread takes four groups of eight elements, its loads ahead of
// the generator's ten rounds, which two groups go through together (134 M
// elements of bf16 83 us, 6.5 TB/s; one by one 90, four together 123: too few
// warps).
#include <cmath>

#include "dropout.cuh"
#include "op_common.cuh"

namespace ma {

bool drop_args(double p, const int64_t* rng, int32_t site, DropArgs* out) {
  if (!(p >= 0.0 && p <= 1.0)) return false;
  const uint32_t t = (uint32_t)std::floor(p * 65536.0 + 0.5);
  *out = {rng, (uint32_t)site, t, t == 65536 ? 0.f : (float)(65536.0 / (65536.0 - t))};
  return true;
}

namespace {

constexpr int kThreads = 256;
constexpr int kGroups = 4;  // of eight elements, a thread
constexpr int kInStep = 2;  // of them through the generator together

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const T* __restrict__ x, int64_t n, DropArgs a,
                                                           T* __restrict__ out) {
  const int64_t g0 = (int64_t)blockIdx.x * (kThreads * kGroups) + threadIdx.x;
  const int64_t whole = n / 8;
  pdl_wait();
  pdl_launch();
  RawVec<T, 8> raw[kGroups];
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < kGroups; ++i)
      if (g0 + i * kThreads < whole) raw[i].load(x + (g0 + i * kThreads) * 8);
  }
  const DropKey key = drop_key(a);
#pragma unroll
  for (int i = 0; i < kGroups; i += kInStep) {
    if ((g0 + i * kThreads) * 8 >= n) break;
    float v[kInStep][8];
#pragma unroll
    for (int j = 0; j < kInStep; ++j) {
      const int64_t g = g0 + (i + j) * kThreads;
      if (VEC && g < whole) {
        raw[i + j].get(v[j]);
      } else {  // rows off 16-byte boundaries, or the last elements
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] = g * 8 + e < n ? load1(x + g * 8 + e) : 0.f;
      }
    }
    drop8(key, (uint32_t)g0 + i * kThreads, kThreads, v);
#pragma unroll
    for (int j = 0; j < kInStep; ++j) {
      const int64_t g = g0 + (i + j) * kThreads;
      if (VEC && g < whole) {
        store8(out + g * 8, v[j]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (g * 8 + e < n) store1(out + g * 8 + e, v[j][e]);
      }
    }
  }
}

template <typename T>
cudaError_t run(const void* x, int64_t n, const DropArgs& a, void* out, cudaStream_t st) {
  const int64_t per = (int64_t)kThreads * kGroups * 8;
  const dim3 grid((unsigned)((n + per - 1) / per));
  const T* in = static_cast<const T*>(x);
  T* to = static_cast<T*>(out);
  return op_aligned(x, 16) && op_aligned(out, 16)
             ? op_launch(dropout_kernel<T, true>, grid, dim3(kThreads), 0, st, 1, in, n, a, to)
             : op_launch(dropout_kernel<T, false>, grid, dim3(kThreads), 0, st, 1, in, n, a, to);
}

}  // namespace
}  // namespace ma

using namespace ma;

extern "C" ma_status muon_adamw_dropout(const void* x, int dtype, int64_t n, double p, const int64_t* rng,
                                        int32_t site, void* out, void* cuda_stream) {
  if (!op_dtype_ok(dtype)) return op_fail(MA_ERR_DTYPE, "dtype %d is neither MA_DT_F32 nor MA_DT_BF16", dtype);
  if (n < 0 || n > MA_DROPOUT_MAX_ELEMENTS)
    return op_fail(MA_ERR_SHAPE, "%lld elements outside [0, 2^35]", (long long)n);
  DropArgs a;
  if (!drop_args(p, rng, site, &a)) return op_fail(MA_ERR_ARG, "p = %g outside [0, 1]", p);
  if (site < 0) return op_fail(MA_ERR_ARG, "site %d is negative", site);
  if (!x || !out || !rng) return op_fail(MA_ERR_ARG, "x, rng and out must not be NULL");
  if (!op_aligned(x, op_dtype_size(dtype)) || !op_aligned(out, op_dtype_size(dtype)) || !op_aligned(rng, 8))
    return op_fail(MA_ERR_ALIGN, "x, out or rng is not aligned to its elements");
  if (n > 0) {
    const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    const cudaError_t e = dtype == MA_DT_BF16 ? run<__nv_bfloat16>(x, n, a, out, st) : run<float>(x, n, a, out, st);
    if (e != cudaSuccess) return op_cuda(e, "dropout launch");
  }
  clear_last_error();
  return MA_OK;
}
