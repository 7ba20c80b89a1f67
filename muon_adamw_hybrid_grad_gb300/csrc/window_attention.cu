// Causal attention with a sliding window and sink tokens, and its gradient.
//
// One warp to a query (forward, dq) or to a key (dk, dv), a head's elements
// spread over its lanes; scores, softmax statistics and sums in fp32.
#include <math.h>

#include "op_common.cuh"

namespace ma {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxDim = 128, kPer = kMaxDim / 32;

struct AttnArgs {
  int n, heads, kv_heads, dim, sinks, window, n_seqs;
  float scale;
  const int32_t* cu;
  const __nv_bfloat16 *q, *k, *v;
  int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs;
};

// The sample [b, e) of token t; empty where t lies behind the last one.
__device__ __forceinline__ int2 sample_of(const AttnArgs& a, int t) {
  if (!a.cu) return make_int2(0, a.n);
  int b = 0;
  for (int i = 1; i <= a.n_seqs; ++i) {
    const int e = min(max(a.cu[i], b), a.n);
    if (t < e) return make_int2(b, e);
    b = e;
  }
  return make_int2(t, t);
}

__device__ __forceinline__ void load_row(const __nv_bfloat16* p, int dim, int lane, float (&x)[kPer]) {
#pragma unroll
  for (int i = 0; i < kPer; ++i) x[i] = lane + 32 * i < dim ? __bfloat162float(p[lane + 32 * i]) : 0.f;
}
__device__ __forceinline__ void store_row(__nv_bfloat16* p, int dim, int lane, const float (&x)[kPer]) {
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (lane + 32 * i < dim) p[lane + 32 * i] = __float2bfloat16_rn(x[i]);
}
__device__ __forceinline__ float dot(const float (&x)[kPer], const float (&y)[kPer]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) s = fmaf(x[i], y[i], s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// f(j) for every key that query t of the sample [b, e) sees.
template <typename F>
__device__ __forceinline__ void each_key(const AttnArgs& a, int t, int2 smp, F f) {
  if (smp.x >= smp.y) return;
  const int lo = max(smp.x, t - a.window + 1), sink = min(min(smp.x + a.sinks, lo), t + 1);
  for (int j = smp.x; j < sink; ++j) f(j);
  for (int j = lo; j <= t; ++j) f(j);
}

__global__ void __launch_bounds__(kWarps * 32) window_forward_kernel(const __grid_constant__ AttnArgs a,
                                                                     __nv_bfloat16* __restrict__ out,
                                                                     float* __restrict__ lse) {
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x & 31, t = blockIdx.x * kWarps + (threadIdx.x >> 5), h = blockIdx.y;
  if (t >= a.n) return;
  const int g = h / (a.heads / a.kv_heads);
  float q[kPer], o[kPer] = {}, m = -INFINITY, l = 0.f;
  load_row(a.q + t * a.q_ts + h * a.q_hs, a.dim, lane, q);
  each_key(a, t, sample_of(a, t), [&](int j) {
    float k[kPer], v[kPer];
    load_row(a.k + j * a.k_ts + g * a.k_hs, a.dim, lane, k);
    load_row(a.v + j * a.v_ts + g * a.v_hs, a.dim, lane, v);
    const float s = dot(q, k) * a.scale, mn = fmaxf(m, s);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float f = expf(m - base), p = expf(s - base);
    l = l * f + p;
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] = fmaf(p, v[i], o[i] * f);
    m = mn;
  });
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll
  for (int i = 0; i < kPer; ++i) o[i] *= inv;
  store_row(out + ((int64_t)t * a.heads + h) * a.dim, a.dim, lane, o);
  if (lane == 0) lse[(int64_t)h * a.n + t] = l == 0.f ? -INFINITY : m + logf(l);
}

struct GradArgs {
  const __nv_bfloat16 *dout, *out;
  int64_t do_ts, do_hs;
  const float* lse;
  float* delta;  // [head][token]: sum of dout * out
  __nv_bfloat16 *dq, *dk, *dv;
};

__global__ void __launch_bounds__(kWarps * 32) window_dq_kernel(const __grid_constant__ AttnArgs a,
                                                                const __grid_constant__ GradArgs r) {
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x & 31, t = blockIdx.x * kWarps + (threadIdx.x >> 5), h = blockIdx.y;
  if (t >= a.n) return;
  const int g = h / (a.heads / a.kv_heads);
  float q[kPer], d[kPer], o[kPer], dq[kPer] = {};
  load_row(a.q + t * a.q_ts + h * a.q_hs, a.dim, lane, q);
  load_row(r.dout + t * r.do_ts + h * r.do_hs, a.dim, lane, d);
  load_row(r.out + ((int64_t)t * a.heads + h) * a.dim, a.dim, lane, o);
  const float delta = dot(d, o), lse = r.lse[(int64_t)h * a.n + t];
  if (lane == 0) r.delta[(int64_t)h * a.n + t] = delta;
  each_key(a, t, sample_of(a, t), [&](int j) {
    float k[kPer], v[kPer];
    load_row(a.k + j * a.k_ts + g * a.k_hs, a.dim, lane, k);
    load_row(a.v + j * a.v_ts + g * a.v_hs, a.dim, lane, v);
    const float p = expf(dot(q, k) * a.scale - lse), ds = p * (dot(d, v) - delta);
#pragma unroll
    for (int i = 0; i < kPer; ++i) dq[i] = fmaf(ds, k[i], dq[i]);
  });
#pragma unroll
  for (int i = 0; i < kPer; ++i) dq[i] *= a.scale;
  store_row(r.dq + ((int64_t)t * a.heads + h) * a.dim, a.dim, lane, dq);
}

__global__ void __launch_bounds__(kWarps * 32) window_dkv_kernel(const __grid_constant__ AttnArgs a,
                                                                 const __grid_constant__ GradArgs r) {
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x & 31, j = blockIdx.x * kWarps + (threadIdx.x >> 5), g = blockIdx.y;
  if (j >= a.n) return;
  const int2 smp = sample_of(a, j);
  float k[kPer], v[kPer], dk[kPer] = {}, dv[kPer] = {};
  load_row(a.k + j * a.k_ts + g * a.k_hs, a.dim, lane, k);
  load_row(a.v + j * a.v_ts + g * a.v_hs, a.dim, lane, v);
  const int last = j - smp.x < a.sinks ? smp.y : (int)min((int64_t)smp.y, (int64_t)j + a.window);
  const int per = a.heads / a.kv_heads;
  for (int h = g * per; h < (g + 1) * per; ++h) {
    for (int t = j; t < last; ++t) {
      float q[kPer], d[kPer];
      load_row(a.q + t * a.q_ts + h * a.q_hs, a.dim, lane, q);
      load_row(r.dout + t * r.do_ts + h * r.do_hs, a.dim, lane, d);
      const float p = expf(dot(q, k) * a.scale - r.lse[(int64_t)h * a.n + t]);
      const float ds = p * (dot(d, v) - r.delta[(int64_t)h * a.n + t]);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        dk[i] = fmaf(ds, q[i], dk[i]);
        dv[i] = fmaf(p, d[i], dv[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) dk[i] *= a.scale;
  store_row(r.dk + ((int64_t)j * a.kv_heads + g) * a.dim, a.dim, lane, dk);
  store_row(r.dv + ((int64_t)j * a.kv_heads + g) * a.dim, a.dim, lane, dv);
}

// ---- host ----
ma_status check_rows(const char* what, const void* p, int64_t ts, int64_t hs) {
  if (!p) return op_fail(MA_ERR_ARG, "%s must not be NULL", what);
  if (!op_aligned(p, 16) || ts % 8 != 0 || hs % 8 != 0)
    return op_fail(MA_ERR_ALIGN, "%s: the pointer and the token and head strides must keep 16-byte alignment", what);
  return MA_OK;
}

ma_status check_attn(const ma_window_attention* d) {
  if (!d) return op_fail(MA_ERR_ARG, "the description must not be NULL");
  if (d->n_tokens < 0 || d->n_tokens > (int64_t)1 << 30) return op_fail(MA_ERR_SHAPE, "n_tokens outside [0, 2^30]");
  if (d->n_heads < 1 || d->n_kv_heads < 1 || d->n_heads > 32768 || d->n_heads % d->n_kv_heads)
    return op_fail(MA_ERR_SHAPE, "%d query heads over %d key heads: no whole number of queries for each", d->n_heads,
                   d->n_kv_heads);
  if (d->head_dim < 8 || d->head_dim > kMaxDim || d->head_dim % 8)
    return op_fail(MA_ERR_SHAPE, "head_dim %d is no multiple of 8 in [8, %d]", d->head_dim, kMaxDim);
  if (d->window < 0) return op_fail(MA_ERR_ARG, "window must not be negative");
  if (d->sinks < 0 || d->sinks > 128) return op_fail(MA_ERR_ARG, "sinks outside [0, 128]");
  if (!(d->scale - d->scale == 0.0)) return op_fail(MA_ERR_ARG, "scale must be finite");
  if (d->n_seqs < 0 || (d->cu_seqlens && d->n_seqs < 1)) return op_fail(MA_ERR_ARG, "cu_seqlens needs n_seqs >= 1");
  if (!op_aligned(d->cu_seqlens, 4)) return op_fail(MA_ERR_ALIGN, "cu_seqlens is not aligned to 4 bytes");
  if (d->n_tokens == 0) return MA_OK;
  ma_status st = check_rows("q", d->q, d->q_token_stride, d->q_head_stride);
  if (st == MA_OK) st = check_rows("k", d->k, d->k_token_stride, d->k_head_stride);
  if (st == MA_OK) st = check_rows("v", d->v, d->v_token_stride, d->v_head_stride);
  return st;
}

AttnArgs args_of(const ma_window_attention* d) {
  AttnArgs a{};
  a.n = (int)d->n_tokens;
  a.heads = d->n_heads;
  a.kv_heads = d->n_kv_heads;
  a.dim = d->head_dim;
  a.sinks = d->sinks;
  a.window = (int)(d->window < d->n_tokens ? d->window : d->n_tokens);
  a.n_seqs = d->n_seqs;
  a.scale = (float)d->scale;
  a.cu = d->cu_seqlens;
  a.q = static_cast<const __nv_bfloat16*>(d->q);
  a.k = static_cast<const __nv_bfloat16*>(d->k);
  a.v = static_cast<const __nv_bfloat16*>(d->v);
  a.q_ts = d->q_token_stride;
  a.q_hs = d->q_head_stride;
  a.k_ts = d->k_token_stride;
  a.k_hs = d->k_head_stride;
  a.v_ts = d->v_token_stride;
  a.v_hs = d->v_head_stride;
  return a;
}

int64_t workspace_bytes_of(const ma_window_attention* d) {
  return ((int64_t)d->n_heads * d->n_tokens * 4 + 255) / 256 * 256 + 256;
}

}  // namespace
}  // namespace ma

using namespace ma;

extern "C" {

ma_status muon_adamw_window_attention(const ma_window_attention* d, void* out, float* lse, void* cuda_stream) {
  ma_status st = check_attn(d);
  if (st != MA_OK) return st;
  if (d->n_tokens > 0) {
    st = check_rows("out", out, 0, 0);
    if (st != MA_OK) return st;
    if (!lse) return op_fail(MA_ERR_ARG, "lse must not be NULL");
    if (!op_aligned(lse, 4)) return op_fail(MA_ERR_ALIGN, "lse is not aligned to 4 bytes");
    AttnArgs a = args_of(d);
    cudaError_t e = op_launch(window_forward_kernel, dim3((a.n + kWarps - 1) / kWarps, a.heads), dim3(kWarps * 32), 0,
                              static_cast<cudaStream_t>(cuda_stream), 1, a, static_cast<__nv_bfloat16*>(out), lse);
    if (e != cudaSuccess) return op_cuda(e, "attention launch");
  }
  clear_last_error();
  return MA_OK;
}

ma_status muon_adamw_window_attention_backward_workspace(const ma_window_attention* d, int64_t* bytes) {
  if (!bytes) return op_fail(MA_ERR_ARG, "bytes must not be NULL");
  ma_status st = check_attn(d);
  if (st != MA_OK) return st;
  *bytes = workspace_bytes_of(d);
  clear_last_error();
  return MA_OK;
}

ma_status muon_adamw_window_attention_backward(const ma_window_attention* d, const void* dout,
                                               int64_t dout_token_stride, int64_t dout_head_stride, const void* out,
                                               const float* lse, void* dq, void* dk, void* dv, void* workspace,
                                               int64_t workspace_bytes, void* cuda_stream) {
  ma_status st = check_attn(d);
  if (st != MA_OK) return st;
  if (d->n_tokens > 0) {
    st = check_rows("dout", dout, dout_token_stride, dout_head_stride);
    if (st == MA_OK) st = check_rows("out", out, 0, 0);
    if (st == MA_OK) st = check_rows("dq", dq, 0, 0);
    if (st == MA_OK) st = check_rows("dk", dk, 0, 0);
    if (st == MA_OK) st = check_rows("dv", dv, 0, 0);
    if (st != MA_OK) return st;
    if (!lse || !op_aligned(lse, 4)) return op_fail(lse ? MA_ERR_ALIGN : MA_ERR_ARG, "lse is NULL or not aligned to 4 bytes");
    if (!workspace || !op_aligned(workspace, 256))
      return op_fail(workspace ? MA_ERR_ALIGN : MA_ERR_ARG, "workspace is NULL or not 256-byte aligned");
    const int64_t need = workspace_bytes_of(d);
    if (workspace_bytes < need)
      return op_fail(MA_ERR_ARG, "workspace of %lld bytes, %lld are needed", (long long)workspace_bytes, (long long)need);
    AttnArgs a = args_of(d);
    GradArgs r{};
    r.dout = static_cast<const __nv_bfloat16*>(dout);
    r.out = static_cast<const __nv_bfloat16*>(out);
    r.do_ts = dout_token_stride;
    r.do_hs = dout_head_stride;
    r.lse = lse;
    r.delta = static_cast<float*>(workspace);
    r.dq = static_cast<__nv_bfloat16*>(dq);
    r.dk = static_cast<__nv_bfloat16*>(dk);
    r.dv = static_cast<__nv_bfloat16*>(dv);
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    const unsigned blocks = (a.n + kWarps - 1) / kWarps;
    cudaError_t e = op_launch(window_dq_kernel, dim3(blocks, a.heads), dim3(kWarps * 32), 0, s, 1, a, r);
    if (e == cudaSuccess) e = op_launch(window_dkv_kernel, dim3(blocks, a.kv_heads), dim3(kWarps * 32), 0, s, 1, a, r);
    if (e != cudaSuccess) return op_cuda(e, "attention gradient launch");
  }
  clear_last_error();
  return MA_OK;
}

}  // extern "C"
