// RMS norm of every query and key head and the position rotation, in one
// pass, and the gradient of both.
//
//   y = x r w,  r = 1 / sqrt(mean(x^2) + eps)       over a head's D elements
//   (a, b) -> (a cos - b sin, b cos + a sin)        for the rot / 2 pairs
//
// With dn the incoming gradient rotated back and z = x r:
//   dw += dn z,   g = dn w,   dx = r (g - z mean(g z)).
// r is computed again from x, which the gradient has to read anyway.
//
// A head's row is spread over LPH lanes of eight elements, so a warp holds
// 32 / LPH heads of one token and every access is 16 bytes. The token's cosines and sines
// stay in registers over all its heads. Everything is held in fp32 and rounded
// once when stored.
#include "op_common.cuh"

namespace ma {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kUnroll = 4;  // heads in flight per lane group

struct QkArgs {
  int64_t n;
  int heads, kv_heads, dim, rot;
  int neighbours, wide_pos;
  float eps, inv_dim;
  const void *q, *k;
  int64_t q_ts, q_hs, k_ts, k_hs;
  const float *qw, *kw, *cos, *sin;
  int64_t table_rows;
  const void* pos;
  int splits;  // blocks along y share a token's heads
};

struct Rotation {
  float c[8], s[8];  // per element: its pair's cosine, and the sine with the partner's sign
  int partner;       // lane that holds the partner element, or -1: the partner is in this lane
  bool on;
};

template <int LPH>
__device__ __forceinline__ Rotation load_rotation(const QkArgs& a, int64_t t, int gl, int lane, bool backward) {
  Rotation R;
  const int half = a.rot / 2;
  R.on = gl * 8 < a.rot;
  R.partner = lane;
#pragma unroll
  for (int i = 0; i < 8; ++i) R.c[i] = 1.f, R.s[i] = 0.f;
  int64_t p = a.wide_pos ? static_cast<const int64_t*>(a.pos)[t] : (int64_t)static_cast<const int32_t*>(a.pos)[t];
  p = p < 0 ? 0 : p >= a.table_rows ? a.table_rows - 1 : p;
  if (!R.on) return R;
  const float* ct = a.cos + p * half;
  const float* st = a.sin + p * half;
  if (a.neighbours) {
    const float4 c = *reinterpret_cast<const float4*>(ct + gl * 4), s = *reinterpret_cast<const float4*>(st + gl * 4);
    const float cv[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      R.c[2 * i] = R.c[2 * i + 1] = cv[i];
      R.s[2 * i] = backward ? sv[i] : -sv[i];
      R.s[2 * i + 1] = backward ? -sv[i] : sv[i];
    }
  } else {
    const bool lead = gl * 8 < half;
    R.partner = lead ? lane + half / 8 : lane - half / 8;
    const int f = lead ? gl * 8 : gl * 8 - half;
    load8(ct + f, R.c);
    load8(st + f, R.s);
    if (lead != backward) {
#pragma unroll
      for (int i = 0; i < 8; ++i) R.s[i] = -R.s[i];
    }
  }
  return R;
}

// x <- the rotated x. Every lane of the warp takes part.
__device__ __forceinline__ void rotate(float (&x)[8], const Rotation& R, bool neighbours) {
  if (neighbours) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float u = fmaf(x[i + 1], R.s[i], x[i] * R.c[i]), v = fmaf(x[i], R.s[i + 1], x[i + 1] * R.c[i + 1]);
      x[i] = u;
      x[i + 1] = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = __shfl_sync(0xffffffffu, x[i], R.partner);
      x[i] = fmaf(y, R.s[i], x[i] * R.c[i]);
    }
  }
}

template <int LPH>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The heads [h0, h1) of one tensor at token t, kUnroll at a time per lane group.
template <typename T, int LPH>
__device__ __forceinline__ void forward_heads(const T* x, int64_t hs, T* y, int h0, int h1, const float (&w)[8],
                                              const Rotation& R, const QkArgs& a, int group, int gl) {
  constexpr int GROUPS = 32 / LPH;
  const bool act = gl * 8 < a.dim;
  for (int h = h0; h < h1; h += GROUPS * kUnroll) {
    float v[kUnroll][8];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = 0.f;
      const int hh = h + u * GROUPS + group;
      if (act && hh < h1) load8(x + hh * hs + gl * 8, v[u]);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (h + u * GROUPS >= h1) break;  // the same for the whole warp
      const int hh = h + u * GROUPS + group;
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(v[u][i], v[u][i], s);
      const float r = rsqrtf(fmaf(group_sum<LPH>(s), a.inv_dim, a.eps));
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = v[u][i] * r * w[i];
      rotate(v[u], R, a.neighbours != 0);
      if (act && hh < h1) store8(y + (int64_t)hh * a.dim + gl * 8, v[u]);
    }
  }
}

// A block of kWarps warps takes a token each; with few tokens a token's heads
// are shared by `splits` blocks.
template <typename T, int LPH>
__global__ void __launch_bounds__(kThreads) qk_forward_kernel(const __grid_constant__ QkArgs a, T* __restrict__ qo,
                                                              T* __restrict__ ko) {
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x & 31, gl = lane & (LPH - 1), group = lane / LPH;
  float qw[8], kw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) qw[i] = kw[i] = 0.f;
  if (gl * 8 < a.dim && a.n > 0) {
    if (a.heads) load8(a.qw + gl * 8, qw);
    if (a.kv_heads) load8(a.kw + gl * 8, kw);
  }
  const int per = (a.heads + a.kv_heads + a.splits - 1) / a.splits;
  const int h0 = blockIdx.y * per, h1 = min(h0 + per, a.heads + a.kv_heads);
  for (int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); t < a.n; t += (int64_t)gridDim.x * kWarps) {
    const Rotation R = load_rotation<LPH>(a, t, gl, lane, false);
    forward_heads<T, LPH>(static_cast<const T*>(a.q) + t * a.q_ts, a.q_hs, qo + t * a.heads * a.dim, h0,
                          min(h1, a.heads), qw, R, a, group, gl);
    forward_heads<T, LPH>(static_cast<const T*>(a.k) + t * a.k_ts, a.k_hs, ko + t * a.kv_heads * a.dim,
                          max(h0 - a.heads, 0), h1 - a.heads, kw, R, a, group, gl);
  }
}

template <typename T, int LPH>
__device__ __forceinline__ void backward_heads(const T* x, int64_t hs, const T* dy, int64_t dhs, T* dx, int h0, int h1,
                                               const float (&w)[8], float (&dw)[8], const Rotation& R,
                                               const QkArgs& a, int group, int gl) {
  constexpr int GROUPS = 32 / LPH;
  constexpr int UNROLL = kUnroll / 2;
  const bool act = gl * 8 < a.dim;
  for (int h = h0; h < h1; h += GROUPS * UNROLL) {
    float v[UNROLL][8], d[UNROLL][8];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = d[u][i] = 0.f;
      const int hh = h + u * GROUPS + group;
      if (act && hh < h1) {
        load8(x + hh * hs + gl * 8, v[u]);
        load8(dy + hh * dhs + gl * 8, d[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      if (h + u * GROUPS >= h1) break;
      const int hh = h + u * GROUPS + group;
      rotate(d[u], R, a.neighbours != 0);
      float s = 0.f, m = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s = fmaf(v[u][i], v[u][i], s);
        m = fmaf(d[u][i] * w[i], v[u][i], m);
      }
      s = group_sum<LPH>(s);
      m = group_sum<LPH>(m);
      const float r = rsqrtf(fmaf(s, a.inv_dim, a.eps));
      const float mz = m * r * a.inv_dim;  // mean(g z)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float z = v[u][i] * r;
        dw[i] = fmaf(d[u][i], z, dw[i]);
        v[u][i] = r * fmaf(-z, mz, d[u][i] * w[i]);
      }
      if (act && hh < h1) store8(dx + (int64_t)hh * a.dim + gl * 8, v[u]);
    }
  }
}

// Persistent: each lane keeps its eight elements' weight gradients over all
// its heads; a block leaves one partial row [queries | keys] of 2 D sums.
template <typename T, int LPH>
__global__ void __launch_bounds__(kThreads) qk_backward_kernel(const __grid_constant__ QkArgs a,
                                                               const T* __restrict__ dqo, int64_t dq_ts,
                                                               int64_t dq_hs, const T* __restrict__ dko,
                                                               int64_t dk_ts, int64_t dk_hs, T* __restrict__ dq,
                                                               T* __restrict__ dk, float* __restrict__ partial) {
  __shared__ float sums[kWarps][2][256];
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gl = lane & (LPH - 1), group = lane / LPH;
  float qw[8], kw[8], dqw[8], dkw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) qw[i] = kw[i] = dqw[i] = dkw[i] = 0.f;
  if (gl * 8 < a.dim && a.n > 0) {
    if (a.heads) load8(a.qw + gl * 8, qw);
    if (a.kv_heads) load8(a.kw + gl * 8, kw);
  }
  const int per = (a.heads + a.kv_heads + a.splits - 1) / a.splits;
  const int h0 = blockIdx.y * per, h1 = min(h0 + per, a.heads + a.kv_heads);
  for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < a.n; t += (int64_t)gridDim.x * kWarps) {
    const Rotation R = load_rotation<LPH>(a, t, gl, lane, true);
    backward_heads<T, LPH>(static_cast<const T*>(a.q) + t * a.q_ts, a.q_hs, dqo + t * dq_ts, dq_hs,
                           dq + t * a.heads * a.dim, h0, min(h1, a.heads), qw, dqw, R, a, group, gl);
    backward_heads<T, LPH>(static_cast<const T*>(a.k) + t * a.k_ts, a.k_hs, dko + t * dk_ts, dk_hs,
                           dk + t * a.kv_heads * a.dim, max(h0 - a.heads, 0), h1 - a.heads, kw, dkw, R, a, group, gl);
  }
  // lane groups, then warps, in a fixed order
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int o = 16; o >= LPH; o >>= 1) {
      dqw[i] += __shfl_xor_sync(0xffffffffu, dqw[i], o);
      dkw[i] += __shfl_xor_sync(0xffffffffu, dkw[i], o);
    }
  }
  if (group == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sums[warp][0][gl * 8 + i] = dqw[i];
      sums[warp][1][gl * 8 + i] = dkw[i];
    }
  }
  __syncthreads();
  float* row = partial + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 2 * a.dim;
  for (int i = threadIdx.x; i < 2 * a.dim; i += kThreads) {
    const int which = i >= a.dim, e = which ? i - a.dim : i;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += sums[w][which][e];
    row[i] = s;
  }
}

// Adds the blocks' partial rows: 8 columns by 32 row walkers to a block.
__global__ void __launch_bounds__(kThreads) qk_weight_kernel(const float* __restrict__ partial, int rows, int dim,
                                                             float* __restrict__ dqw, float* __restrict__ dkw) {
  __shared__ float sums[32][9];
  pdl_launch();
  pdl_wait();
  const int c = threadIdx.x & 7, r = threadIdx.x >> 3, col = blockIdx.x * 8 + c;
  float s = 0.f;
  if (col < 2 * dim)
    for (int i = r; i < rows; i += 32) s += partial[(int64_t)i * 2 * dim + col];
  sums[r][c] = s;
  __syncthreads();
  if (r == 0 && col < 2 * dim) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += sums[i][c];
    float* out = col < dim ? dqw : dkw;
    if (out) out[col < dim ? col : col - dim] = s;
  }
}

// ---- host ----
ma_status check_tensor(const char* what, const void* p, int dtype, int64_t ts, int64_t hs, bool used) {
  if (!used) return MA_OK;
  if (!p) return op_fail(MA_ERR_ARG, "%s must not be NULL", what);
  const int64_t e = op_dtype_size(dtype);
  if (!op_aligned(p, 16) || ts * e % 16 != 0 || hs * e % 16 != 0)
    return op_fail(MA_ERR_ALIGN, "%s: the pointer and the token and head strides must keep 16-byte alignment", what);
  return MA_OK;
}

ma_status check_qk(const ma_qk_norm_rope* d) {
  if (!d) return op_fail(MA_ERR_ARG, "the description must not be NULL");
  if (!op_dtype_ok(d->dtype)) return op_fail(MA_ERR_DTYPE, "dtype %d is neither MA_DT_F32 nor MA_DT_BF16", d->dtype);
  if (d->n_tokens < 0 || d->n_tokens > ((int64_t)1 << 31) - 1) return op_fail(MA_ERR_SHAPE, "n_tokens outside [0, 2^31)");
  if (d->n_heads < 0 || d->n_kv_heads < 0 || d->n_heads + (int64_t)d->n_kv_heads < 1 || d->n_heads > 65536 ||
      d->n_kv_heads > 65536)
    return op_fail(MA_ERR_SHAPE, "head counts outside [0, 65536], or no head at all");
  if (d->head_dim < 8 || d->head_dim > 256 || d->head_dim % 8)
    return op_fail(MA_ERR_SHAPE, "head_dim %d is no multiple of 8 in [8, 256]", d->head_dim);
  if (d->rot_dim < 0 || d->rot_dim > d->head_dim || d->rot_dim % 16)
    return op_fail(MA_ERR_SHAPE, "rot_dim %d is no multiple of 16 in [0, head_dim]", d->rot_dim);
  if (d->neighbours != 0 && d->neighbours != 1) return op_fail(MA_ERR_ARG, "neighbours must be 0 or 1");
  if (!(d->eps >= 0.0) || !(d->eps - d->eps == 0.0)) return op_fail(MA_ERR_ARG, "eps must be finite and not negative");
  if (d->position_bytes != 4 && d->position_bytes != 8) return op_fail(MA_ERR_ARG, "position_bytes must be 4 or 8");
  if (d->n_tokens == 0) return MA_OK;
  if (!d->positions || !op_aligned(d->positions, d->position_bytes))
    return op_fail(d->positions ? MA_ERR_ALIGN : MA_ERR_ARG, "positions are NULL or not aligned to their size");
  if (d->rot_dim > 0) {
    if (d->table_rows < 1) return op_fail(MA_ERR_SHAPE, "the tables of cosines and sines need a row");
    if (!d->cos_table || !d->sin_table) return op_fail(MA_ERR_ARG, "cos_table and sin_table must not be NULL");
    if (!op_aligned(d->cos_table, 16) || !op_aligned(d->sin_table, 16))
      return op_fail(MA_ERR_ALIGN, "cos_table and sin_table must be 16-byte aligned");
  }
  if ((d->n_heads && !d->q_weight) || (d->n_kv_heads && !d->k_weight))
    return op_fail(MA_ERR_ARG, "q_weight and k_weight must not be NULL");
  if (!op_aligned(d->q_weight, 16) || !op_aligned(d->k_weight, 16))
    return op_fail(MA_ERR_ALIGN, "q_weight and k_weight must be 16-byte aligned");
  ma_status st = check_tensor("q", d->q, d->dtype, d->q_token_stride, d->q_head_stride, d->n_heads > 0);
  if (st == MA_OK) st = check_tensor("k", d->k, d->dtype, d->k_token_stride, d->k_head_stride, d->n_kv_heads > 0);
  return st;
}

QkArgs args_of(const ma_qk_norm_rope* d) {
  QkArgs a{};
  a.n = d->n_tokens;
  a.heads = d->n_heads;
  a.kv_heads = d->n_kv_heads;
  a.dim = d->head_dim;
  a.rot = d->rot_dim;
  a.neighbours = d->neighbours;
  a.wide_pos = d->position_bytes == 8;
  a.eps = (float)d->eps;
  a.inv_dim = 1.f / (float)d->head_dim;
  a.q = d->q;
  a.k = d->k;
  a.q_ts = d->q_token_stride;
  a.q_hs = d->q_head_stride;
  a.k_ts = d->k_token_stride;
  a.k_hs = d->k_head_stride;
  a.qw = d->q_weight;
  a.kw = d->k_weight;
  a.cos = d->cos_table;
  a.sin = d->sin_table;
  a.table_rows = d->table_rows;
  a.pos = d->positions;
  return a;
}

// Blocks along x (tokens) and the split of a token's heads: with fewer tokens
// than the GPU has places for warps, a token's heads go to several warps, down
// to one batch of unrolled heads for each.
dim3 grid_of(QkArgs& a, int lph, int unroll, int sms, int blocks_per_sm) {
  int64_t x = (a.n + kWarps - 1) / kWarps;
  const int64_t most = (int64_t)sms * blocks_per_sm;
  const int batches = (a.heads + a.kv_heads + 32 / lph * unroll - 1) / (32 / lph * unroll);
  int64_t y = x > 0 ? most / x : 1;
  if (y > batches) y = batches;
  if (y < 1) y = 1;
  if (x > most) x = most;
  if (x < 1) x = 1;
  a.splits = (int)y;
  return dim3((unsigned)x, (unsigned)y);
}

constexpr int kForwardBlocksPerSm = 8, kBackwardBlocksPerSm = 4;

int lanes_per_head(int dim) {
  int l = 1;
  while (l * 8 < dim) l *= 2;
  return l;
}

template <typename T, int LPH>
cudaError_t run_forward(QkArgs& a, void* qo, void* ko, int sms, cudaStream_t st) {
  const dim3 g = grid_of(a, LPH, kUnroll, sms, kForwardBlocksPerSm);
  return op_launch(qk_forward_kernel<T, LPH>, g, dim3(kThreads), 0, st, 1, a, static_cast<T*>(qo),
                   static_cast<T*>(ko));
}

struct BackwardPtrs {
  const void *dqo, *dko;
  int64_t dq_ts, dq_hs, dk_ts, dk_hs;
  void *dq, *dk;
  float *dqw, *dkw, *partial;
};

template <typename T, int LPH>
cudaError_t run_backward(QkArgs& a, const BackwardPtrs& b, int sms, cudaStream_t st) {
  const dim3 g = grid_of(a, LPH, kUnroll / 2, sms, kBackwardBlocksPerSm);
  cudaError_t e = op_launch(qk_backward_kernel<T, LPH>, g, dim3(kThreads), 0, st, 1, a, static_cast<const T*>(b.dqo),
                            b.dq_ts, b.dq_hs, static_cast<const T*>(b.dko), b.dk_ts, b.dk_hs, static_cast<T*>(b.dq),
                            static_cast<T*>(b.dk), b.partial);
  if (e != cudaSuccess) return e;
  return op_launch(qk_weight_kernel, dim3((unsigned)((2 * a.dim + 7) / 8)), dim3(kThreads), 0, st, 1,
                   static_cast<const float*>(b.partial), (int)(g.x * g.y), a.dim, b.dqw, b.dkw);
}

template <typename F>
cudaError_t by_lanes(int dim, F f) {
  switch (lanes_per_head(dim)) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 4: return f(std::integral_constant<int, 4>());
    case 8: return f(std::integral_constant<int, 8>());
    case 16: return f(std::integral_constant<int, 16>());
    default: return f(std::integral_constant<int, 32>());
  }
}

}  // namespace
}  // namespace ma

using namespace ma;

extern "C" {

ma_status muon_adamw_qk_norm_rope(const ma_qk_norm_rope* d, void* q_out, void* k_out, void* cuda_stream) {
  ma_status st = check_qk(d);
  if (st != MA_OK) return st;
  if (d->n_tokens > 0) {
    if ((d->n_heads && !q_out) || (d->n_kv_heads && !k_out)) return op_fail(MA_ERR_ARG, "q_out and k_out must not be NULL");
    if (!op_aligned(q_out, 16) || !op_aligned(k_out, 16))
      return op_fail(MA_ERR_ALIGN, "q_out and k_out must be 16-byte aligned");
    int sms = 0;
    cudaError_t e = op_num_sms(&sms);
    if (e != cudaSuccess) return op_cuda(e, "device query");
    QkArgs a = args_of(d);
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    e = by_lanes(a.dim, [&](auto l) {
      return d->dtype == MA_DT_BF16 ? run_forward<__nv_bfloat16, l.value>(a, q_out, k_out, sms, s)
                                    : run_forward<float, l.value>(a, q_out, k_out, sms, s);
    });
    if (e != cudaSuccess) return op_cuda(e, "query/key norm launch");
  }
  clear_last_error();
  return MA_OK;
}

ma_status muon_adamw_qk_norm_rope_backward_workspace(const ma_qk_norm_rope* d, int64_t* bytes) {
  if (!d || !bytes) return op_fail(MA_ERR_ARG, "the description and bytes must not be NULL");
  if (d->head_dim < 8 || d->head_dim > 256) return op_fail(MA_ERR_SHAPE, "head_dim outside [8, 256]");
  int sms = 0;
  cudaError_t e = op_num_sms(&sms);
  if (e != cudaSuccess) return op_cuda(e, "device query");
  // grid_of() gives at most this many blocks, each with one partial row
  *bytes = (int64_t)sms * kBackwardBlocksPerSm * 2 * d->head_dim * 4;
  clear_last_error();
  return MA_OK;
}

ma_status muon_adamw_qk_norm_rope_backward(const ma_qk_norm_rope* d, const void* dq_out, int64_t dq_token_stride,
                                           int64_t dq_head_stride, const void* dk_out, int64_t dk_token_stride,
                                           int64_t dk_head_stride, void* dq, void* dk, float* dq_weight,
                                           float* dk_weight, void* workspace, int64_t workspace_bytes,
                                           void* cuda_stream) {
  ma_status st = check_qk(d);
  if (st != MA_OK) return st;
  if (d->n_tokens > 0) {
    st = check_tensor("dq_out", dq_out, d->dtype, dq_token_stride, dq_head_stride, d->n_heads > 0);
    if (st == MA_OK) st = check_tensor("dk_out", dk_out, d->dtype, dk_token_stride, dk_head_stride, d->n_kv_heads > 0);
    if (st == MA_OK) st = check_tensor("dq", dq, d->dtype, 0, 0, d->n_heads > 0);
    if (st == MA_OK) st = check_tensor("dk", dk, d->dtype, 0, 0, d->n_kv_heads > 0);
    if (st != MA_OK) return st;
  }
  if ((d->n_heads && !dq_weight) || (d->n_kv_heads && !dk_weight))
    return op_fail(MA_ERR_ARG, "dq_weight and dk_weight must not be NULL");
  if (!op_aligned(dq_weight, 4) || !op_aligned(dk_weight, 4))
    return op_fail(MA_ERR_ALIGN, "dq_weight and dk_weight must be aligned to 4 bytes");
  int sms = 0;
  cudaError_t e = op_num_sms(&sms);
  if (e != cudaSuccess) return op_cuda(e, "device query");
  const int64_t need = (int64_t)sms * kBackwardBlocksPerSm * 2 * d->head_dim * 4;
  if (!workspace || !op_aligned(workspace, 16))
    return op_fail(workspace ? MA_ERR_ALIGN : MA_ERR_ARG, "workspace is NULL or not 16-byte aligned");
  if (workspace_bytes < need)
    return op_fail(MA_ERR_ARG, "workspace of %lld bytes, %lld are needed", (long long)workspace_bytes, (long long)need);
  QkArgs a = args_of(d);
  BackwardPtrs b{dq_out, dk_out, dq_token_stride, dq_head_stride, dk_token_stride, dk_head_stride,
                 dq, dk, dq_weight, dk_weight, static_cast<float*>(workspace)};
  if (!d->n_heads) b.dqw = nullptr;
  if (!d->n_kv_heads) b.dkw = nullptr;
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  e = by_lanes(a.dim, [&](auto l) {
    return d->dtype == MA_DT_BF16 ? run_backward<__nv_bfloat16, l.value>(a, b, sms, s)
                                  : run_backward<float, l.value>(a, b, sms, s);
  });
  if (e != cudaSuccess) return op_cuda(e, "query/key norm gradient launch");
  clear_last_error();
  return MA_OK;
}

}  // extern "C"
