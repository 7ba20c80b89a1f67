// Gradient of the residual's addition with RMS norm.
//
//   g = dy w,  n = r rstd,  dr = dres + rstd (g - n mean(g n)),
//   dx = drop(dr),  dw = sum over rows of dy n
//
// The sum over the row is of g r, and c = mean(g r) rstd^2 is taken times n: with
// rstd^3 times r it would leave fp32's range for rows of 1e-13 or 1e13 and beyond.
//
// One pass over dy, dres and r: both of a row's sums are formed together, so it
// waits once for its threads. Bound by HBM (three rows in, two out). Blocks are
// persistent: each keeps its columns' share of dw in registers over its rows
// and leaves one partial row; a second launch adds those up in a fixed order.
//
// residual_norm_ring_kernel takes rows that allow 16-byte accesses: bulk copies
// bring them into a ring of shared memory that a group of T threads owns. From 128
// elements of bf16 a row on 96 to 200 KB are in flight on an SM, where registers
// for a row ahead would be a quarter of that (32749 rows of 2048: 103 us with
// dropout, 139 by registers; 71 and 105 without). Narrower rows have a warp's
// lanes and the ring's eight places half empty and take what those of 128 do
// (400000 rows of 8, 64 and 128: 113, 115 and 115 us). The barrier of the row's
// sums is also the one behind which its place in the ring is free.
// residual_norm_grad_kernel takes the others: rows off 16-byte boundaries and of
// more than 8192 elements.
#include <algorithm>
#include <cmath>

#include "pairs.cuh"
#include "residual_norm.cuh"
#include "tcgen05.cuh"

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
    for (int j = 0; j < V; ++j) dy[j].load(py, col_of<VEC, T>(j, t), a.w);
#pragma unroll
    for (int j = 0; j < V; ++j) r[j].load(pr, col_of<VEC, T>(j, t), a.w);
    if (a.dres) {
      const TS* const pd = static_cast<const TS*>(a.dres) + row * a.dress;
#pragma unroll
      for (int j = 0; j < V; ++j) dres[j].load(pd, col_of<VEC, T>(j, t), a.w);
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
      const int col = col_of<VEC, T>(j, t);
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
    const float c = gr / (float)a.w * rstd * rstd;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = col_of<VEC, T>(j, t);
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
        const float n = r[e] * rstd;
        d[e] = fmaf(-c, n, fmaf(rstd * dy[e], w[e], d[e]));
        dw[j][e] = fmaf(dy[e], n, dw[j][e]);
      }
      store_row<VEC>(static_cast<TS*>(a.dr) + row * a.w, col, a.w, d);
      if (a.dx) {
        if (a.drop.threshold) drop_vector<VEC, T>(key, row * a.w, j, t, d);
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
  for (int j = 0; j < V; ++j) store_row<VEC>(out, col_of<VEC, T>(j, t), a.w, dw[j]);
}

// ---- rows through a ring of shared memory ----

constexpr int kRingThreads = 512;
constexpr int kRingBytes = 200 * 1024;  // of rows, at most
constexpr int kMaxStages = 8;
constexpr int kErrRow = 0x401;

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// Eight elements as four pairs.
__device__ __forceinline__ void load_pairs(const __nv_bfloat16* p, uint64_t (&x)[4]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ void load_pairs(const float* p, uint64_t (&x)[4]) {
  const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(p), b = *reinterpret_cast<const ulonglong2*>(p + 4);
  x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
}

template <typename TX, typename TS, int T, int V>
__global__ void __launch_bounds__(kRingThreads, 1)
    residual_norm_ring_kernel(const __grid_constant__ NormArgs a, int stages, int* err) {
  constexpr int G = kRingThreads / T;
  extern __shared__ __align__(128) uint8_t ring[];  // [group][stage][dy, r, dres]
  __shared__ uint64_t bars[G * kMaxStages];
  __shared__ float2 sums[2][G][T / 32];
  __shared__ int abort_word;
  volatile int* const abort_flag = &abort_word;
  const int group = threadIdx.x / T, t = threadIdx.x % T, warp = t >> 5, lane = t & 31;
  const int x_bytes = a.w * (int)sizeof(TX), s_bytes = a.w * (int)sizeof(TS);
  const int row_bytes = x_bytes + s_bytes * (a.dres ? 2 : 1);
  uint8_t* const rows = ring + (int64_t)group * stages * row_bytes;
  const uint32_t bar0 = smem_u32(bars + group * kMaxStages);
  if (threadIdx.x == 0) {
    for (int i = 0; i < G * kMaxStages; ++i) mbar_init(smem_u32(bars + i), 1);
    abort_word = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  __syncthreads();
  pdl_wait();
  pdl_launch();
  const int64_t step = (int64_t)gridDim.x * G, row0 = (int64_t)blockIdx.x * G + group;
  auto fetch = [&](int64_t row, int stage) {  // by the group's first thread
    const uint32_t dst = smem_u32(rows + stage * row_bytes), bar = bar0 + 8 * stage;
    mbar_expect_tx(bar, (uint32_t)row_bytes);
    bulk_load(dst, static_cast<const TX*>(a.dy) + row * a.dys, (uint32_t)x_bytes, bar);
    bulk_load(dst + x_bytes, static_cast<const TS*>(a.r) + row * a.ress, (uint32_t)s_bytes, bar);
    if (a.dres)
      bulk_load(dst + x_bytes + s_bytes, static_cast<const TS*>(a.dres) + row * a.dress, (uint32_t)s_bytes, bar);
  };
  if (t == 0)
    for (int i = 0; i < stages; ++i)
      if (row0 + i * step < a.n) fetch(row0 + i * step, i);
  DropKey key{};
  if (a.drop.threshold) key = drop_key(a.drop);
  uint64_t w[V][4], dw[V][4];
#pragma unroll
  for (int j = 0; j < V; ++j) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[j][i] = dw[j][i] = 0;
    if ((j * T + t) * 8 < a.w) load_pairs(a.weight + (j * T + t) * 8, w[j]);
  }
  int stage = 0, parity = 0;
  uint32_t phase = 0;
  for (int64_t row = row0; row < a.n; row += step, parity ^= 1) {
    // where the wait runs out the error word is set and the rows that follow are not valid; the loop goes on, so that
    // no thread waits for another at a barrier
    mbar_wait(bar0 + 8 * stage, phase, abort_flag, err, kErrRow);
    const uint8_t* const at = rows + stage * row_bytes;
    uint64_t dy[V][4], r[V][4], d[V][4], ss = 0, gr = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = (j * T + t) * 8;
#pragma unroll
      for (int i = 0; i < 4; ++i) dy[j][i] = r[j][i] = d[j][i] = 0;
      if (col < a.w) {
        load_pairs(reinterpret_cast<const TX*>(at) + col, dy[j]);
        load_pairs(reinterpret_cast<const TS*>(at + x_bytes) + col, r[j]);
        if (a.dres) load_pairs(reinterpret_cast<const TS*>(at + x_bytes + s_bytes) + col, d[j]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ss = fma2(r[j][i], r[j][i], ss);
        gr = fma2(mul2(dy[j][i], w[j][i]), r[j][i], gr);
      }
    }
    float ss0, ss1, gr0, gr1;
    unpack2(ss, ss0, ss1);
    unpack2(gr, gr0, gr1);
    ss0 = warp_sum(ss0 + ss1);
    gr0 = warp_sum(gr0 + gr1);
    if constexpr (T > 32) {
      if (lane == 0) sums[parity][group][warp] = make_float2(ss0, gr0);
      if constexpr (G == 1)
        __syncthreads();
      else
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(T) : "memory");
      ss0 = gr0 = 0.f;
#pragma unroll
      for (int i = 0; i < T / 32; ++i) {
        const float2 v = sums[parity][group][i];
        ss0 += v.x;
        gr0 += v.y;
      }
    } else {
      __syncwarp();
    }
    // every thread has read the row
    if (t == 0 && row + stages * step < a.n) fetch(row + stages * step, stage);
    if (++stage == stages) {
      stage = 0;
      phase ^= 1u;
    }
    const float rstd = rsqrtf(ss0 / (float)a.w + a.eps);
    const float c = gr0 / (float)a.w * rstd * rstd;
    const uint64_t rstd2 = pack2(rstd, rstd), c2 = pack2(-c, -c);
    float v[V][8];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = (j * T + t) * 8;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t n = mul2(rstd2, r[j][i]), g = mul2(rstd2, dy[j][i]);
        dw[j][i] = fma2(dy[j][i], n, dw[j][i]);
        unpack2(fma2(c2, n, fma2(g, w[j][i], d[j][i])), v[j][2 * i], v[j][2 * i + 1]);
      }
      if (col < a.w) store8(static_cast<TS*>(a.dr) + row * a.w + col, v[j]);
    }
    if (a.dx) {
      if (a.drop.threshold) drop_row<true, T>(key, row * a.w, t, v);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int col = (j * T + t) * 8;
        if (col < a.w) store8(static_cast<TX*>(a.dx) + row * a.w + col, v[j]);
      }
    }
  }
  // the groups' shares of dw, added up in their order
  if (*abort_flag && t == 0)  // copies in flight land before the ring is written to
    for (int i = 0; i < stages; ++i, phase ^= stage + 1 == stages, stage = stage + 1 == stages ? 0 : stage + 1)
      drain_wait(bar0 + 8 * stage, phase);
  __syncthreads();
  float* const shares = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) reinterpret_cast<uint64_t*>(shares)[(j * 4 + i) * kRingThreads + threadIdx.x] = dw[j][i];
  __syncthreads();
  // pair q of a row is pair q % 4 of vector q / 4, which thread q / 4 % T of every group holds
  for (int q = threadIdx.x; q < a.w / 2; q += kRingThreads) {
    const int vec = q / 4;
    const float2* const from =
        reinterpret_cast<const float2*>(shares) + (vec / T * 4 + q % 4) * kRingThreads + vec % T;
    float2 s = from[0];
#pragma unroll
    for (int g = 1; g < G; ++g) {
      s.x += from[g * T].x;
      s.y += from[g * T].y;
    }
    reinterpret_cast<float2*>(a.partial + (int64_t)blockIdx.x * a.w)[q] = s;
  }
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

cudaError_t join(const NormArgs& a, int blocks, cudaStream_t st) {
  return op_launch(residual_norm_join_kernel, dim3((a.w + 31) / 32), dim3(256), 0, st, 1, (const float*)a.partial,
                   blocks, a.w, a.dweight);
}

template <typename TX, typename TS, int T, int V, bool VEC>
cudaError_t launch(const NormArgs& a, cudaStream_t st) {
  using R = RowGroups<T>;
  constexpr int kSmem = 4 * (4 * R::kGroups * (T / 32) + (R::kGroups > 1 ? T * V * 8 : 0));
  const auto kernel = residual_norm_grad_kernel<TX, TS, T, V, VEC>;
  int sms = 0, *err = nullptr, per_sm = 0;
  cudaError_t e = op_device(&sms, &err);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, R::kBlock, kSmem);
  if (e != cudaSuccess) return e;
  const int blocks = (int)std::min<int64_t>(std::min(sms * std::max(per_sm, 1), kMaxBlocks),
                                            (a.n + R::kGroups - 1) / R::kGroups);
  e = op_launch(kernel, dim3(blocks), dim3(R::kBlock), kSmem, st, 1, a);
  return e == cudaSuccess ? join(a, blocks, st) : e;
}

template <typename TX, typename TS>
int ring_stages(const NormArgs& a, int groups) {
  const int row = a.w * (int)(sizeof(TX) + sizeof(TS) * (a.dres ? 2 : 1));
  return std::min(kMaxStages, kRingBytes / (row * groups));
}

template <typename TX, typename TS, int T, int V>
cudaError_t launch_ring(const NormArgs& a, cudaStream_t st) {
  constexpr int kGroups = kRingThreads / T;
  const auto kernel = residual_norm_ring_kernel<TX, TS, T, V>;
  int sms = 0, *err = nullptr;
  cudaError_t e = op_device(&sms, &err);
  if (e == cudaSuccess) e = op_smem_limit<residual_norm_ring_kernel<TX, TS, T, V>>(kRingBytes);
  if (e != cudaSuccess) return e;
  const int stages = ring_stages<TX, TS>(a, kGroups);
  const int row = a.w * (int)(sizeof(TX) + sizeof(TS) * (a.dres ? 2 : 1));
  const int smem = std::max(stages * kGroups * row, kRingThreads * V * 32);  // the rows, then the shares of dw
  if (a.n <= 2 * kGroups && op_aligned(a.dweight, 8)) {
    // two rows a group at most: one block, whose partial row is the whole sum
    NormArgs one = a;
    one.partial = a.dweight;
    return op_launch(kernel, dim3(1), dim3(kRingThreads), smem, st, 1, one, stages, err);
  }
  const int blocks = (int)std::min<int64_t>(sms, (a.n + kGroups - 1) / kGroups);
  e = op_launch(kernel, dim3(blocks), dim3(kRingThreads), smem, st, 1, a, stages, err);
  return e == cudaSuccess ? join(a, blocks, st) : e;
}

template <typename TX, typename TS>
cudaError_t backward(const NormArgs& a, bool vec, cudaStream_t st) {
  const int units = (a.w + 7) / 8;
  if (a.n == 0) return join(a, 0, st);
  if (!vec) {
    if (units <= 32) return launch<TX, TS, 32, 1, false>(a, st);
    if (units <= 128) return launch<TX, TS, 64, 2, false>(a, st);
    if (units <= 256) return launch<TX, TS, 128, 2, false>(a, st);
    if (units <= 512) return launch<TX, TS, 256, 2, false>(a, st);
    if (units <= 1024) return launch<TX, TS, 512, 2, false>(a, st);
    return launch<TX, TS, 512, 8, false>(a, st);
  }
  if (units <= 32) return launch_ring<TX, TS, 32, 1>(a, st);
  if (units <= 64) return launch_ring<TX, TS, 32, 2>(a, st);
  if (units <= 128) return launch_ring<TX, TS, 64, 2>(a, st);
  if (units <= 256) return launch_ring<TX, TS, 128, 2>(a, st);
  if (units <= 512) return launch_ring<TX, TS, 256, 2>(a, st);
  if (units <= 1024) return launch_ring<TX, TS, 512, 2>(a, st);
  // Wider rows from registers: 64M elements of rows of 16384 take 106 us, through a ring of two rows, whose threads
  // would hold four vectors each, 121.
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
