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
// 32 / LPH heads of one token. A lane's eight elements are two quads chosen so
// that every rotated pair lies within one lane (element e and e + rot / 2, or
// neighbours): the rotation needs no exchange between lanes and a lane keeps
// four cosines and four sines for all of its token's heads. Everything is held
// in fp32 and rounded once when stored.
//
// The passes are bound by HBM. Each warp owns a ring of stages in shared memory
// that bulk copies fill: a unit's rows (up to `chunk` heads of one token, the
// queries first, then the keys; the gradient's incoming rows behind them) and
// the token's rows of the tables. Two stages a warp and 16 warps an SM keep
// 100 to 200 KB in flight on every SM, which a warp's registers could not
// hold. 32749 tokens of 16 + 8 heads of 128 in bf16 take 71 us (5.7 TB/s, 0.84 of
// the measured copy bandwidth), their gradient 121 us (5.0 TB/s, 0.74: a third
// stream to read, and warps issue in 64 % of the cycles); loads straight to
// registers took 153 and 180. A stage holds one token at most, so narrow tokens
// leave it part empty: of 8 + 1 heads of 64 an SM has 45 KB in flight, and 32749
// tokens take 31 us (2.5 TB/s), their gradient 45 (2.6); of 5 + 5 heads of 96 they
// take 45 (2.8) and 63 (3.0).
#include "op_common.cuh"
#include "tcgen05.cuh"

namespace ma {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kBlocksPerSm = 2;
constexpr int kStages = 2;
constexpr int kStageBytes = 6656;  // 24 heads of 128 in bf16 and their token's cosines and sines
constexpr int kErrRows = 0x301;

struct QkArgs {
  int64_t n;
  int heads, kv_heads, dim, rot;
  int neighbours, wide_pos;
  float eps, inv_dim;
  const void *q, *k;
  int64_t q_ts, q_hs, k_ts, k_hs;
  const void *dq, *dk;  // incoming gradients, or null
  int64_t dq_ts, dq_hs, dk_ts, dk_hs;
  const float *qw, *kw, *cos, *sin;
  int64_t table_rows;
  const void* pos;
  int chunk, chunks;  // heads of a unit; units of a token
  int* err;
};

// Four elements of a row in shared memory, and in the output.
__device__ __forceinline__ void get_quad(const __nv_bfloat16* p, float* x) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xFFFF0000u);
  x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xFFFF0000u);
}
__device__ __forceinline__ void get_quad(const float* p, float* x) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
__device__ __forceinline__ void put_quad(__nv_bfloat16* p, const float* x) {
  *reinterpret_cast<uint2*>(p) = make_uint2(op_pack_bf16(x[0], x[1]), op_pack_bf16(x[2], x[3]));
}
__device__ __forceinline__ void put_quad(float* p, const float* x) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}

// A lane's place: its two quads within a head, and its heads within a batch.
struct Place {
  int a, b;      // first element of each quad
  bool on, rot;  // it has elements; they are rotated
  int table;     // first of its four columns of the tables
  int group;
};
template <int LPH>
__device__ __forceinline__ Place place_of(const QkArgs& q) {
  const int lane = threadIdx.x & 31, gl = lane & (LPH - 1);
  Place p;
  p.group = lane / LPH;
  p.on = gl * 8 < q.dim;
  p.rot = gl * 8 < q.rot;
  p.table = gl * 4;
  const bool apart = p.rot && !q.neighbours;
  p.a = apart ? gl * 4 : gl * 8;
  p.b = apart ? q.rot / 2 + gl * 4 : gl * 8 + 4;
  return p;
}

__device__ __forceinline__ int64_t position(const QkArgs& a, int64_t t) {
  const int64_t p =
      a.wide_pos ? static_cast<const int64_t*>(a.pos)[t] : (int64_t)static_cast<const int32_t*>(a.pos)[t];
  return p < 0 ? 0 : p >= a.table_rows ? a.table_rows - 1 : p;
}

struct Angles {
  float c[4], s[4];
};

// Rotation by the angles, or back by them (BACK).
template <bool BACK>
__device__ __forceinline__ void turn(float& u, float& v, float c, float s) {
  const float x = u, y = v;
  u = BACK ? fmaf(y, s, x * c) : fmaf(-y, s, x * c);
  v = BACK ? fmaf(-x, s, y * c) : fmaf(x, s, y * c);
}
template <bool BACK>
__device__ __forceinline__ void rotate(float (&x)[8], const Angles& r, bool neighbours) {
  if (neighbours) {
#pragma unroll
    for (int i = 0; i < 4; ++i) turn<BACK>(x[2 * i], x[2 * i + 1], r.c[i], r.s[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) turn<BACK>(x[i], x[i + 4], r.c[i], r.s[i]);
  }
}

template <int LPH>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ void load_weights(const QkArgs& a, const Place& pl, float (&qw)[8], float (&kw)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) qw[i] = kw[i] = 0.f;
  if (!pl.on || a.n == 0) return;
  if (a.heads) get_quad(a.qw + pl.a, qw), get_quad(a.qw + pl.b, qw + 4);
  if (a.kv_heads) get_quad(a.kw + pl.a, kw), get_quad(a.kw + pl.b, kw + 4);
}

struct Unit {
  int64_t t;
  int h0, h1;  // heads, the keys' counted on from the queries'
};
__device__ __forceinline__ Unit unit_of(const QkArgs& a, int64_t u) {
  Unit r;
  r.t = a.chunks == 1 ? u : u / a.chunks;
  r.h0 = (int)(u - r.t * a.chunks) * a.chunk;
  r.h1 = min(r.h0 + a.chunk, a.heads + a.kv_heads);
  return r;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// The rows of heads [h0, h1) to consecutive places: one copy where the heads
// are consecutive in memory too, else one for each, spread over the lanes.
template <typename T>
__device__ __forceinline__ void copy_heads(uint32_t dst, const T* p, int64_t hs, int h0, int h1, int dim, uint32_t bar,
                                           int lane) {
  if (h0 >= h1) return;
  if (hs == dim) {
    if (lane == 0) bulk_load(dst, p + (int64_t)h0 * dim, (uint32_t)((h1 - h0) * dim * sizeof(T)), bar);
  } else {
    for (int h = h0 + lane; h < h1; h += 32)
      bulk_load(dst + (h - h0) * dim * (int)sizeof(T), p + h * hs, (uint32_t)(dim * sizeof(T)), bar);
  }
}

// A stage: x rows [chunk][dim], then the incoming gradients' rows (BACK), then
// the cosines and the sines.
template <typename T, bool BACK>
__device__ __forceinline__ void request(const QkArgs& a, const Unit& w, int64_t pos, uint32_t stage, uint32_t bar,
                                        int lane) {
  const uint32_t rows = (uint32_t)((w.h1 - w.h0) * a.dim * sizeof(T)), full = (uint32_t)(a.chunk * a.dim * sizeof(T));
  const uint32_t tab = (uint32_t)a.rot * 2;
  if (lane == 0) mbar_expect_tx(bar, rows * (BACK ? 2 : 1) + 2 * tab);
  __syncwarp();
  const int q1 = min(w.h1, a.heads), k0 = max(w.h0 - a.heads, 0), k1 = w.h1 - a.heads;
  const uint32_t kat = (uint32_t)(max(a.heads - w.h0, 0) * a.dim * sizeof(T));
  copy_heads(stage, static_cast<const T*>(a.q) + w.t * a.q_ts, a.q_hs, w.h0, q1, a.dim, bar, lane);
  copy_heads(stage + kat, static_cast<const T*>(a.k) + w.t * a.k_ts, a.k_hs, k0, k1, a.dim, bar, lane);
  if (BACK) {
    copy_heads(stage + full, static_cast<const T*>(a.dq) + w.t * a.dq_ts, a.dq_hs, w.h0, q1, a.dim, bar, lane);
    copy_heads(stage + full + kat, static_cast<const T*>(a.dk) + w.t * a.dk_ts, a.dk_hs, k0, k1, a.dim, bar, lane);
  }
  if (tab && lane == 0) {
    const uint32_t at = stage + full * (BACK ? 2 : 1);
    bulk_load(at, a.cos + pos * (a.rot / 2), tab, bar);
    bulk_load(at + tab, a.sin + pos * (a.rot / 2), tab, bar);
  }
}

// Forward, heads [h0, h1) of one tensor: x in shared memory, y in the output.
template <typename T, int LPH>
__device__ __forceinline__ void forward_heads(const QkArgs& a, const Place& pl, const T* x, T* y, int count,
                                              const float (&w)[8], const Angles& ang) {
  constexpr int GROUPS = 32 / LPH, U = 4;
  for (int h0 = 0; h0 < count; h0 += GROUPS * U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (h0 + u * GROUPS >= count) break;  // the same for the whole warp
      const int h = h0 + u * GROUPS + pl.group;
      const bool on = pl.on && h < count;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
      if (on) get_quad(x + h * a.dim + pl.a, v), get_quad(x + h * a.dim + pl.b, v + 4);
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(v[i], v[i], s);
      const float r = rsqrtf(fmaf(group_sum<LPH>(s), a.inv_dim, a.eps));
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = v[i] * r * w[i];
      rotate<false>(v, ang, a.neighbours != 0);
      if (on) put_quad(y + h * a.dim + pl.a, v), put_quad(y + h * a.dim + pl.b, v + 4);
    }
  }
}

template <typename T, int LPH>
__device__ __forceinline__ void backward_heads(const QkArgs& a, const Place& pl, const T* x, const T* dy, T* dx,
                                               int count, const float (&w)[8], float (&dw)[8], const Angles& ang) {
  constexpr int GROUPS = 32 / LPH, U = 4;
  for (int h0 = 0; h0 < count; h0 += GROUPS * U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (h0 + u * GROUPS >= count) break;
      const int h = h0 + u * GROUPS + pl.group;
      const bool on = pl.on && h < count;
      float v[8], d[8], g[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = d[i] = 0.f;
      if (on) {
        get_quad(x + h * a.dim + pl.a, v), get_quad(x + h * a.dim + pl.b, v + 4);
        get_quad(dy + h * a.dim + pl.a, d), get_quad(dy + h * a.dim + pl.b, d + 4);
      }
      rotate<true>(d, ang, a.neighbours != 0);
      float s = 0.f, m = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        g[i] = d[i] * w[i];
        s = fmaf(v[i], v[i], s);
        m = fmaf(g[i], v[i], m);
      }
      s = group_sum<LPH>(s);
      m = group_sum<LPH>(m);
      const float r = rsqrtf(fmaf(s, a.inv_dim, a.eps));
      const float mz = m * r * a.inv_dim;  // mean(g z)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float z = v[i] * r;
        dw[i] = fmaf(d[i], z, dw[i]);
        v[i] = r * fmaf(-z, mz, g[i]);
      }
      if (on) put_quad(dx + h * a.dim + pl.a, v), put_quad(dx + h * a.dim + pl.b, v + 4);
    }
  }
}

// Persistent over the units. Forward: qo, ko are the results; gradient (BACK):
// they are dq and dk, each lane keeps its eight elements' weight gradients over
// all its heads, and a block leaves one partial row [queries | keys] of 2 D sums.
template <typename T, int LPH, bool BACK>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    qk_norm_rope_kernel(const __grid_constant__ QkArgs a, T* __restrict__ qo, T* __restrict__ ko,
                        float* __restrict__ partial) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[kWarps * kStages];
  __shared__ int abort_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    abort_word = 0;
    for (int i = 0; i < kWarps * kStages; ++i) mbar_init(smem_u32(bars + i), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  pdl_launch();
  pdl_wait();
  const Place pl = place_of<LPH>(a);
  const int64_t units = a.n * a.chunks, step = (int64_t)gridDim.x * kWarps;
  const int64_t u0 = (int64_t)blockIdx.x + (int64_t)warp * gridDim.x;  // neighbouring units on different SMs
  uint8_t* const mine = smem + warp * kStages * kStageBytes;
  const uint32_t bar0 = smem_u32(bars + warp * kStages), full = (uint32_t)(a.chunk * a.dim * sizeof(T));
  float dqw[8], dkw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dqw[i] = dkw[i] = 0.f;
  int in_flight = 0;
  int64_t ahead = u0, pos_ahead = 0;  // the next unit to request, and its position
  if (ahead < units) pos_ahead = position(a, unit_of(a, ahead).t);
  auto ask = [&](int stage) {
    if (ahead >= units) return;
    request<T, BACK>(a, unit_of(a, ahead), pos_ahead, smem_u32(mine) + stage * kStageBytes, bar0 + 8 * stage, lane);
    ++in_flight;
    ahead += step;
    if (ahead < units) pos_ahead = position(a, unit_of(a, ahead).t);
  };
#pragma unroll
  for (int s = 0; s < kStages; ++s) ask(s);
  float qw[8], kw[8];
  load_weights(a, pl, qw, kw);
  uint32_t phase = 0;
  int stage = 0;
  for (int64_t u = u0; u < units; u += step) {
    const Unit w = unit_of(a, u);
    if (!__all_sync(0xffffffffu, mbar_wait(bar0 + 8 * stage, phase, &abort_word, a.err, kErrRows))) break;
    --in_flight;
    const T* x = reinterpret_cast<const T*>(mine + stage * kStageBytes);
    Angles ang;
    if (pl.rot) {
      const float* tab = reinterpret_cast<const float*>(mine + stage * kStageBytes + full * (BACK ? 2 : 1)) + pl.table;
      get_quad(tab, ang.c);
      get_quad(tab + a.rot / 2, ang.s);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) ang.c[i] = 1.f, ang.s[i] = 0.f;
    }
    const int qn = max(min(w.h1, a.heads) - w.h0, 0), k0 = max(w.h0 - a.heads, 0), kn = w.h1 - w.h0 - qn;
    T* yq = qo + (w.t * a.heads + w.h0) * a.dim;
    T* yk = ko + (w.t * a.kv_heads + k0) * a.dim;
    if constexpr (BACK) {
      const T* d = reinterpret_cast<const T*>(mine + stage * kStageBytes + full);
      backward_heads<T, LPH>(a, pl, x, d, yq, qn, qw, dqw, ang);
      backward_heads<T, LPH>(a, pl, x + qn * a.dim, d + qn * a.dim, yk, kn, kw, dkw, ang);
    } else {
      forward_heads<T, LPH>(a, pl, x, yq, qn, qw, ang);
      forward_heads<T, LPH>(a, pl, x + qn * a.dim, yk, kn, kw, ang);
    }
    __syncwarp();  // every lane has read the stage
    ask(stage);
    if (++stage == kStages) stage = 0, phase ^= 1;
  }
  // after a wait that ran out: copies still on their way land before the block leaves
  for (; in_flight > 0; --in_flight) {
    drain_wait(bar0 + 8 * stage, phase);
    if (++stage == kStages) stage = 0, phase ^= 1;
  }
  if constexpr (BACK) {
    // lane groups, then warps, in a fixed order; the stages are free now
    float* sums = reinterpret_cast<float*>(smem);  // [warp][2][dim]
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int o = 16; o >= LPH; o >>= 1) {
        dqw[i] += __shfl_xor_sync(0xffffffffu, dqw[i], o);
        dkw[i] += __shfl_xor_sync(0xffffffffu, dkw[i], o);
      }
    }
    __syncthreads();
    if (pl.group == 0 && pl.on) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = i < 4 ? pl.a + i : pl.b + i - 4;
        sums[(warp * 2 + 0) * a.dim + e] = dqw[i];
        sums[(warp * 2 + 1) * a.dim + e] = dkw[i];
      }
    }
    __syncthreads();
    float* row = partial + (int64_t)blockIdx.x * 2 * a.dim;
    for (int i = threadIdx.x; i < 2 * a.dim; i += kThreads) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += sums[w * 2 * a.dim + i];
      row[i] = s;
    }
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
  if (col < 2 * dim) {
#pragma unroll 8
    for (int i = r; i < rows; i += 32) s += partial[(int64_t)i * 2 * dim + col];
  }
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

// Heads of a unit: as many as a stage holds, fewer (down to one pass of a
// warp's lane groups) while there are fewer units than warps on the GPU (50 tokens
// of 16 + 16 heads of 64: 2.8 us, with whole stages 3.9; 1000 tokens: 3.8 and 4.7).
void set_units(QkArgs& a, int lph, int esize, bool back, int sms) {
  const int groups = 32 / lph, total = a.heads + a.kv_heads;
  const int most = (kStageBytes - 4 * a.rot) / (a.dim * esize * (back ? 2 : 1));
  int64_t pieces = (total + most - 1) / most;
  const int64_t warps = (int64_t)sms * kBlocksPerSm * kWarps;
  if (a.n > 0 && a.n * pieces < warps) {
    pieces = warps / a.n;
    const int64_t finest = (total + groups - 1) / groups;
    if (pieces > finest) pieces = finest;
    const int64_t coarsest = (total + most - 1) / most;
    if (pieces < coarsest) pieces = coarsest;
  }
  a.chunk = (int)((total + pieces - 1) / pieces);
  a.chunks = (total + a.chunk - 1) / a.chunk;
}
int64_t blocks_of(const QkArgs& a, int sms) {
  const int64_t need = (a.n * a.chunks + kWarps - 1) / kWarps, most = (int64_t)sms * kBlocksPerSm;
  return need < 1 ? 1 : need < most ? need : most;
}

int lanes_per_head(int dim) {
  int l = 1;
  while (l * 8 < dim) l *= 2;
  return l;
}

template <typename T, int LPH, bool BACK>
cudaError_t run_rows(QkArgs& a, void* qo, void* ko, float* partial, int sms, int64_t* blocks, cudaStream_t st) {
  constexpr size_t smem = (size_t)kWarps * kStages * kStageBytes;
  cudaError_t e = op_smem_limit<qk_norm_rope_kernel<T, LPH, BACK>>((int)smem);
  if (e != cudaSuccess) return e;
  set_units(a, LPH, sizeof(T), BACK, sms);
  *blocks = blocks_of(a, sms);
  return op_launch(qk_norm_rope_kernel<T, LPH, BACK>, dim3((unsigned)*blocks), dim3(kThreads), smem, st, 1, a,
                   static_cast<T*>(qo), static_cast<T*>(ko), partial);
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
    QkArgs a = args_of(d);
    cudaError_t e = op_device(&sms, &a.err);
    if (e != cudaSuccess) return op_cuda(e, "device query");
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    int64_t blocks;
    e = by_lanes(a.dim, [&](auto l) {
      return d->dtype == MA_DT_BF16
                 ? run_rows<__nv_bfloat16, l.value, false>(a, q_out, k_out, nullptr, sms, &blocks, s)
                 : run_rows<float, l.value, false>(a, q_out, k_out, nullptr, sms, &blocks, s);
    });
    if (e != cudaSuccess) return op_cuda(e, "query/key norm launch");
  }
  clear_last_error();
  return MA_OK;
}

ma_status muon_adamw_qk_norm_rope_backward_workspace(const ma_qk_norm_rope* d, int64_t* bytes) {
  if (!d || !bytes) return op_fail(MA_ERR_ARG, "the description and bytes must not be NULL");
  if (d->head_dim < 8 || d->head_dim > 256) return op_fail(MA_ERR_SHAPE, "head_dim outside [8, 256]");
  int sms = 0, *err = nullptr;
  cudaError_t e = op_device(&sms, &err);
  if (e != cudaSuccess) return op_cuda(e, "device query");
  // one partial row for each block
  *bytes = (int64_t)sms * kBlocksPerSm * 2 * d->head_dim * 4;
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
  QkArgs a = args_of(d);
  cudaError_t e = op_device(&sms, &a.err);
  if (e != cudaSuccess) return op_cuda(e, "device query");
  const int64_t need = (int64_t)sms * kBlocksPerSm * 2 * d->head_dim * 4;
  if (!workspace || !op_aligned(workspace, 16))
    return op_fail(workspace ? MA_ERR_ALIGN : MA_ERR_ARG, "workspace is NULL or not 16-byte aligned");
  if (workspace_bytes < need)
    return op_fail(MA_ERR_ARG, "workspace of %lld bytes, %lld are needed", (long long)workspace_bytes, (long long)need);
  a.dq = dq_out;
  a.dk = dk_out;
  a.dq_ts = dq_token_stride;
  a.dq_hs = dq_head_stride;
  a.dk_ts = dk_token_stride;
  a.dk_hs = dk_head_stride;
  float* partial = static_cast<float*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  int64_t blocks = 0;
  e = by_lanes(a.dim, [&](auto l) {
    return d->dtype == MA_DT_BF16 ? run_rows<__nv_bfloat16, l.value, true>(a, dq, dk, partial, sms, &blocks, s)
                                  : run_rows<float, l.value, true>(a, dq, dk, partial, sms, &blocks, s);
  });
  if (e == cudaSuccess)
    e = op_launch(qk_weight_kernel, dim3((unsigned)((2 * a.dim + 7) / 8)), dim3(kThreads), 0, s, 1,
                  static_cast<const float*>(partial), (int)blocks, a.dim, d->n_heads ? dq_weight : nullptr,
                  d->n_kv_heads ? dk_weight : nullptr);
  if (e != cudaSuccess) return op_cuda(e, "query/key norm gradient launch");
  clear_last_error();
  return MA_OK;
}

}  // extern "C"
