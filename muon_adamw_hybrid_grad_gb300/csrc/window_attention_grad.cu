// Gradient of the sliding-window attention.
//
// With P = exp2(c S - lse2) (the forward pass's softmax weights, from its
// saved lse), dP = dO V^T, delta_i = dO_i . O_i:
//   dS = P (dP - delta),  dV = P^T dO,  dK = scale dS^T Q,  dQ = scale dS K.
//
// window_stats_kernel  lse2 and delta of every query and head.
// window_dq_kernel     a CTA to 128 queries of a head, walking their key tiles.
// window_dkv_kernel    a CTA to 128 keys of a key head, walking the query
//                      tiles of every head that reads it.
// window_sink_kernel   joins the partial sums of the sink keys.
//
// Seven products instead of the five that one kernel would need, because S and
// dP are formed twice: dQ would otherwise have to be added up by atomics in an
// order that changes from run to run, or stored in fp32 once per key tile.
//
// The sink keys are seen by every query of a sample. Their gradients are cut
// into chunks of kSinkChunk query tiles, each a work item of its own whose
// fp32 sums window_sink_kernel adds in a fixed order.
#include "window_attention.cuh"

namespace ma {
namespace {

constexpr int kThreads = 320;
constexpr int kErrDq = 0x202, kErrDkv = 0x203, kErrAlign = 0x204;

// ---- lse2 and delta ----
// A group of 16 lanes to a (token, head), eight elements a lane.
__global__ void __launch_bounds__(256) window_stats_kernel(const __grid_constant__ AttnArgs a,
                                                           const __nv_bfloat16* __restrict__ dout, int64_t do_ts,
                                                           int64_t do_hs, const __nv_bfloat16* __restrict__ out,
                                                           const float* __restrict__ lse, float* __restrict__ lse2,
                                                           float* __restrict__ delta) {
  pdl_launch();
  pdl_wait();
  const int gl = threadIdx.x & 15;
  const int64_t total = (int64_t)a.n * a.heads, step = (int64_t)gridDim.x * 16;
  // whole warps stay in the loop for the sum across lanes
  for (int64_t u0 = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 5) * 2; u0 < total; u0 += step) {
    const int64_t u = u0 + ((threadIdx.x >> 4) & 1);
    float s = 0.f;
    int64_t t = 0;
    int h = 0;
    if (u < total) {
      t = u / a.heads;
      h = (int)(u - t * a.heads);
      if (gl * 8 < a.dim) {
        float x[8], y[8];
        load8(dout + t * do_ts + h * do_hs + gl * 8, x);
        load8(out + u * a.dim + gl * 8, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(x[i], y[i], s);
      }
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (u < total && gl == 0) {
      const float l = lse[(int64_t)h * a.n + t];
      lse2[(int64_t)h * a.n + t] = l == -INFINITY ? INFINITY : l * 1.4426950408889634f;
      delta[(int64_t)h * a.n + t] = s;
    }
  }
}

// ---- dQ ----
// Warps 0-7: a thread to a query and half of a tile's keys (warps 0-3 the
// first 64, 4-7 the others); warp 8: TMA; warp 9: tcgen05.mma.
// TMEM: S of even steps | S of odd steps | dP | dQ. dS (bf16) overwrites the S
// it came from, each half in the first 32 of its own 64 columns. S of the next
// tile is formed while the threads work on this one's, and dP of the next as
// soon as this one's has been read.
template <int DP>
struct DqSmem {
  static constexpr uint32_t TILE = kAttnTile * DP * 2;
  static constexpr int SLOTS = DP == 128 ? 5 : 8;
  static constexpr uint32_t RING = 2 * TILE;  // after Q and dO
  static constexpr uint32_t BARS = RING + SLOTS * TILE;
  // full[SLOTS], empty[SLOTS], q full, q empty, s full[2], dp full, dp empty, ds full, dq full, drain
  static constexpr int NBARS = 2 * SLOTS + 9;
  static constexpr uint32_t BYTES = BARS + NBARS * 8 + 16;
  static_assert(BYTES <= 232448, "shared memory per CTA");
};

struct DqItem {
  SampleTile t;
  KeyTiles k;
  int steps, head, kv;
  __device__ __forceinline__ int tile(int n) const { return k.sink ? (n == 0 ? 0 : k.lo + n - 1) : k.lo + n; }
};
__device__ __forceinline__ DqItem dq_item(const AttnArgs& a, int item, int lane) {
  DqItem w;
  const int tile = item / a.heads;
  w.head = item - tile * a.heads;
  w.kv = w.head / (a.heads / a.kv_heads);
  w.t = find_unit(a, tile, lane, [](int len, bool) { return (len + kAttnTile - 1) / kAttnTile; });
  w.t.p0 = w.t.index * kAttnTile;
  w.k = key_tiles(a, w.t.live, w.t.len, w.t.p0);
  w.steps = (w.k.sink ? 1 : 0) + max(0, w.k.hi - w.k.lo + 1);
  return w;
}

// The tile of S (64 columns of it) as softmax weights: v <- exp2(c v - lse2).
// Key k0 + col is visible to query i for col <= last and (col >= first or col < sink).
__device__ __forceinline__ void weights(uint32_t (&v)[2][32], float c, float shift, bool masked, int col0, int last,
                                        int first, int sink) {
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      float p = ex2(fmaf(__uint_as_float(v[x][j]), c, shift));
      if (masked) {
        const int col = col0 + 32 * x + j;
        if (col > last || (col < first && col >= sink)) p = 0.f;
      }
      v[x][j] = __float_as_uint(p);
    }
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
    window_dq_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ CUtensorMap tmDO, __nv_bfloat16* __restrict__ dq, int* __restrict__ err) {
  using SM = DqSmem<DP>;
  extern __shared__ __align__(1024) uint8_t smem[];
  // two words after the barriers: the TMEM base and the abort flag
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SM::BARS + SM::NBARS * 8);
  volatile int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = smem_u32(smem), bars = base + SM::BARS;
  Ring<SM::SLOTS> ring{base + SM::RING, bars, bars + SM::SLOTS * 8, SM::TILE};
  const uint32_t q_full = bars + 2 * SM::SLOTS * 8, q_empty = q_full + 8, s_full = q_full + 16, dp_full = q_full + 32,
                 dp_empty = q_full + 40, ds_full = q_full + 48, dq_full = q_full + 56, drain = q_full + 64;
  if (base & 1023u) {  // the swizzle's phase is that of the address
    if (threadIdx.x == 0) atomicCAS(err, 0, kErrAlign);
    return;
  }
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < SM::SLOTS; ++i) mbar_init(ring.full + 8 * i, 1), mbar_init(ring.empty + 8 * i, 1);
    mbar_init(q_full, 1), mbar_init(q_empty, 1), mbar_init(s_full, 1), mbar_init(s_full + 8, 1), mbar_init(dp_full, 1);
    mbar_init(dp_empty, 256), mbar_init(ds_full, 256), mbar_init(dq_full, 1), mbar_init(drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 9) tmem_alloc<1>(smem_u32(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch();
  pdl_wait();
  const int items = a.heads * count_units(a, lane, [](int len, bool) { return (len + kAttnTile - 1) / kAttnTile; });
  bool ok = true;

  if (warp < 8) {
    const int half = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    uint32_t step = 0, dq_ph = 0;  // step: over all items; the S slot starts at 0 for each
    uint32_t s_ph[2] = {0, 0};
    for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
      const DqItem w = dq_item(a, item, lane);
      const int i = w.t.p0 + row;
      const int64_t t = (int64_t)w.t.b + i;
      const bool mine = i < w.t.len;
      const float lse2 = mine ? a.lse2[(int64_t)w.head * a.n + t] : INFINITY;
      const float delta = mine ? a.delta[(int64_t)w.head * a.n + t] : 0.f;
      for (int n = 0; n < w.steps && ok; ++n, ++step) {
        const uint32_t slot = n & 1;
        ok = __all_sync(0xffffffffu, mbar_wait(s_full + 8 * slot, s_ph[slot], abort_flag, err, kErrDq));
        if (!ok) break;
        s_ph[slot] ^= 1;
        tc_fence_after();
        const uint32_t ts = tmem + lanes + 128u * slot + 64u * half;
        uint32_t p[2][32], g[2][32];
        tmem_ld_32x32b_x32(ts, p[0]);
        tmem_ld_32x32b_x32(ts + 32, p[1]);
        tmem_ld_wait();
        const int k0 = w.tile(n) * kAttnTile;
        const bool masked = !tile_full(a, w.t.p0, k0);
        if (masked)
          weights(p, a.scale_log2, -lse2, true, 64 * half, i - k0, i - a.window + 1 - k0, a.sinks - k0);
        else
          weights(p, a.scale_log2, -lse2, false, 0, 0, 0, 0);
        ok = __all_sync(0xffffffffu, mbar_wait(dp_full, step & 1, abort_flag, err, kErrDq));
        if (!ok) break;
        tc_fence_after();
        tmem_ld_32x32b_x32(tmem + lanes + 256u + 64u * half, g[0]);
        tmem_ld_32x32b_x32(tmem + lanes + 256u + 64u * half + 32, g[1]);
        tmem_ld_wait();
        tc_fence_before();
        mbar_arrive(dp_empty);
        uint32_t ds[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const int x = j >> 4, e = (2 * j) & 31;
          float d0 = __uint_as_float(p[x][e]) * (__uint_as_float(g[x][e]) - delta);
          float d1 = __uint_as_float(p[x][e + 1]) * (__uint_as_float(g[x][e + 1]) - delta);
          if (masked) {
            // a value row of another sample may hold anything
            if (p[x][e] == 0u) d0 = 0.f;
            if (p[x][e + 1] == 0u) d1 = 0.f;
          }
          ds[j] = op_pack_bf16(d0, d1);
        }
        tmem_st_32x32b_x32(ts, ds);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(ds_full);
      }
      if (!ok) break;
      if (w.steps) {
        ok = __all_sync(0xffffffffu, mbar_wait(dq_full, dq_ph, abort_flag, err, kErrDq));
        if (!ok) break;
        dq_ph ^= 1;
        tc_fence_after();
      }
      __nv_bfloat16* po = dq + (t * a.heads + w.head) * a.dim;
#pragma unroll 1
      for (int c = half * (DP / 2); c < (half + 1) * (DP / 2); c += 32) {
        uint32_t o[32];
        if (w.steps) {
          tmem_ld_32x32b_x32(tmem + lanes + 384u + c, o);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = 0u;
        }
        if (mine) {
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            if (c + j < a.dim) {
              uint32_t r[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                r[e] = op_pack_bf16(__uint_as_float(o[j + 2 * e]) * a.scale, __uint_as_float(o[j + 2 * e + 1]) * a.scale);
              *reinterpret_cast<uint4*>(po + c + j) = make_uint4(r[0], r[1], r[2], r[3]);
            }
          }
        }
      }
      tc_fence_before();
    }
  } else if (warp == 8) {
    uint32_t pos = 0, q_ph = 1, q_loads = 0;
    for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
      const DqItem w = dq_item(a, item, lane);
      for (int n = 0; n < w.steps && ok; ++n) {
        const int token = w.t.b + w.tile(n) * kAttnTile;
        for (int kv = 0; kv < 2 && ok; ++kv) {
          ok = mbar_wait(ring.empty_bar(pos), ring.empty_parity(pos), abort_flag, err, kErrDq);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) {
            mbar_expect_tx(ring.full_bar(pos), SM::TILE);
            load_tile<DP>(ring.slot(pos), kv ? &tmV : &tmK, token, w.kv, ring.full_bar(pos));
          }
          ++pos;
          if (n == 0 && kv == 0) {
            ok = mbar_wait(q_empty, q_ph, abort_flag, err, kErrDq);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            q_ph ^= 1;
            ++q_loads;
            if (lane == 0) {
              mbar_expect_tx(q_full, 2 * SM::TILE);
              load_tile<DP>(base, &tmQ, w.t.b + w.t.p0, w.head, q_full);
              load_tile<DP>(base + SM::TILE, &tmDO, w.t.b + w.t.p0, w.head, q_full);
            }
          }
        }
      }
    }
    for (uint32_t k = pos > SM::SLOTS ? pos - SM::SLOTS : 0; k < pos; ++k)
      drain_wait(ring.full_bar(k), ring.full_parity(k));
    if (q_loads) drain_wait(q_full, (q_loads - 1) & 1);
  } else {
    uint32_t pos = 0, q_ph = 0, step = 0;
    for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
      const DqItem w = dq_item(a, item, lane);
      if (w.steps == 0) continue;
      ok = __all_sync(0xffffffffu, mbar_wait(q_full, q_ph, abort_flag, err, kErrDq));
      if (!ok) break;
      q_ph ^= 1;
      // S of step n into its slot, dP of step n
      auto wait_tile = [&](uint32_t k) {
        ok = mbar_wait(ring.full_bar(k), ring.full_parity(k), abort_flag, err, kErrDq);
        ok = __all_sync(0xffffffffu, ok);
        return ok;
      };
      auto issue_s = [&](int n) {
        const uint32_t k = pos + 2 * n;
        if (!wait_tile(k)) return false;
        const int valid = w.t.len - w.tile(n) * kAttnTile;
        if (valid < kAttnTile) clear_rows<DP>(ring.slot(k), valid, lane);
        tc_fence_after();
        if (lane == 0) {
          mma_abt<DP>(tmem + 128u * (n & 1), base, ring.slot(k));
          umma_commit<1>(s_full + 8 * (n & 1));
        }
        __syncwarp();
        return true;
      };
      auto issue_dp = [&](int n) {
        const uint32_t k = pos + 2 * n + 1;
        if (!wait_tile(k)) return false;
        tc_fence_after();
        if (lane == 0) {
          mma_abt<DP>(tmem + 256u, base + SM::TILE, ring.slot(k));
          umma_commit<1>(dp_full);
          umma_commit<1>(ring.empty_bar(k));
        }
        __syncwarp();
        return true;
      };
      if (!issue_s(0) || !issue_dp(0)) break;
      if (w.steps > 1 && !issue_s(1)) break;
      for (int n = 0; n < w.steps && ok; ++n, ++step) {
        if (n + 1 < w.steps) {
          ok = __all_sync(0xffffffffu, mbar_wait(dp_empty, step & 1, abort_flag, err, kErrDq));
          if (!ok || !issue_dp(n + 1)) break;
        } else {
          ok = __all_sync(0xffffffffu, mbar_wait(dp_empty, step & 1, abort_flag, err, kErrDq));
          if (!ok) break;
        }
        ok = __all_sync(0xffffffffu, mbar_wait(ds_full, step & 1, abort_flag, err, kErrDq));
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
          mma_ab<DP>(tmem + 384u, tmem + 128u * (n & 1), 64, ring.slot(pos + 2 * n), n > 0);
          umma_commit<1>(ring.empty_bar(pos + 2 * n));
        }
        __syncwarp();
        if (n + 2 < w.steps && !issue_s(n + 2)) break;
      }
      if (!ok) break;
      if (lane == 0) {
        umma_commit<1>(dq_full);
        umma_commit<1>(q_empty);
      }
      __syncwarp();
      pos += 2 * w.steps;
    }
    if (lane == 0) {
      umma_commit<1>(drain);
      drain_wait(drain, 0);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc<1>(tmem, 512);
}

// ---- dK and dV ----
// Scores are formed transposed, S^T = K Q^T and dP^T = V dO^T, so that P^T and
// dS^T stand in TMEM as the left operands of dV += P^T dO and dK += dS^T Q.
// Warps 0-7: a thread to a key and half of a tile's queries; warp 8: TMA;
// warp 9: tcgen05.mma. TMEM: S^T | dP^T | dV | dK; P^T overwrites S^T and dS^T
// dP^T, each half in the first 32 of its own 64 columns. While the threads form
// P^T of a step the tensor core runs the step before's dK and this one's dP^T;
// while they form dS^T it runs dV and the next step's S^T.
template <int DP>
struct DkvSmem {
  static constexpr uint32_t TILE = kAttnTile * DP * 2;
  static constexpr int SLOTS = DP == 128 ? 5 : 8;
  static constexpr uint32_t RING = 2 * TILE;  // after K and V
  static constexpr uint32_t STATS = RING + SLOTS * TILE;  // [2][lse2, delta][128] of the query tiles
  static constexpr uint32_t BARS = STATS + 2 * 2 * kAttnTile * 4;
  // full[SLOTS], empty[SLOTS], kv full, done, s full, dp full, p full, ds full, stats full, drain
  static constexpr int NBARS = 2 * SLOTS + 8;
  static constexpr uint32_t BYTES = BARS + NBARS * 8 + 16;
  static_assert(BYTES <= 232448, "shared memory per CTA");
};

// First query tile that only the sinks reach in tile 0.
__device__ __forceinline__ int first_sink_tile(const AttnArgs& a) {
  return a.window == 0 ? 0 : (kAttnTile - 1 + a.window - 1) / kAttnTile + 1;
}
__device__ __forceinline__ int sink_chunks(const AttnArgs& a, int len, bool live) {
  if (!live || a.sinks == 0) return 0;
  const int left = (len + kAttnTile - 1) / kAttnTile - first_sink_tile(a);
  return left > 0 ? (left + kSinkChunk - 1) / kSinkChunk : 0;
}

struct DkvItem {
  SampleTile t;     // the key tile
  int kv, q_lo, nq; // query tiles q_lo .. q_lo + nq - 1, for each head of the group
  int64_t slot;     // partial slot of the sink keys, -1: none
  bool sink_only;   // a chunk for the sink keys alone
};
__device__ __forceinline__ DkvItem dkv_item(const AttnArgs& a, int item, int sink_items, int lane) {
  DkvItem w;
  w.sink_only = item < sink_items;
  const int u = (w.sink_only ? item : item - sink_items) / a.kv_heads;
  w.kv = (w.sink_only ? item : item - sink_items) - u * a.kv_heads;
  if (w.sink_only) {
    w.t = find_unit(a, u, lane, [&](int len, bool live) { return sink_chunks(a, len, live); });
    const int tiles = (w.t.len + kAttnTile - 1) / kAttnTile;
    w.q_lo = first_sink_tile(a) + w.t.index * kSinkChunk;
    w.nq = max(0, min(kSinkChunk, tiles - w.q_lo));
    w.slot = (int64_t)a.n_seqs + u;
    w.t.p0 = 0;
  } else {
    w.t = find_unit(a, u, lane, [](int len, bool) { return (len + kAttnTile - 1) / kAttnTile; });
    w.t.p0 = w.t.index * kAttnTile;
    const int tiles = (w.t.len + kAttnTile - 1) / kAttnTile;
    w.q_lo = w.t.index;
    w.nq = 0;
    if (w.t.live && a.window > 0) {
      const int hi = (int)min((int64_t)tiles - 1, ((int64_t)w.t.p0 + kAttnTile - 1 + a.window - 1) / kAttnTile);
      w.nq = hi - w.q_lo + 1;
    }
    w.slot = a.sinks > 0 && w.t.index == 0 && w.t.live ? w.t.sample : -1;
  }
  return w;
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
    window_dkv_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ CUtensorMap tmDO, __nv_bfloat16* __restrict__ dk,
                      __nv_bfloat16* __restrict__ dv, float* __restrict__ partial, int64_t partial_slots,
                      int* __restrict__ err) {
  using SM = DkvSmem<DP>;
  extern __shared__ __align__(1024) uint8_t smem[];
  // two words after the barriers: the TMEM base and the abort flag
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SM::BARS + SM::NBARS * 8);
  volatile int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = smem_u32(smem), bars = base + SM::BARS;
  Ring<SM::SLOTS> ring{base + SM::RING, bars, bars + SM::SLOTS * 8, SM::TILE};
  const uint32_t kv_full = bars + 2 * SM::SLOTS * 8, done = kv_full + 8, s_full = kv_full + 16, dp_full = kv_full + 24,
                 p_full = kv_full + 32, ds_full = kv_full + 40, stat_full = kv_full + 48, drain = kv_full + 56;
  float* stats = reinterpret_cast<float*>(smem + SM::STATS);
  if (base & 1023u) {  // the swizzle's phase is that of the address
    if (threadIdx.x == 0) atomicCAS(err, 0, kErrAlign);
    return;
  }
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < SM::SLOTS; ++i) mbar_init(ring.full + 8 * i, 1), mbar_init(ring.empty + 8 * i, 1);
    mbar_init(kv_full, 1), mbar_init(done, 1), mbar_init(s_full, 1), mbar_init(dp_full, 1), mbar_init(p_full, 256);
    mbar_init(ds_full, 256), mbar_init(stat_full, 256), mbar_init(drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 9) tmem_alloc<1>(smem_u32(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch();
  pdl_wait();
  const int group = a.heads / a.kv_heads;
  const int sink_items =
      a.kv_heads * count_units(a, lane, [&](int len, bool live) { return sink_chunks(a, len, live); });
  const int items = sink_items +
                    a.kv_heads * count_units(a, lane, [](int len, bool) { return (len + kAttnTile - 1) / kAttnTile; });
  bool ok = true;

  if (warp < 8) {
    const int half = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + 64u * half, tg = ts + 128u;
    uint32_t step = 0, done_ph = 0;
    for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
      const DkvItem w = dkv_item(a, item, sink_items, lane);
      const int steps = group * w.nq;
      // threads 0-127 bring lse2 of a query tile, threads 128-255 delta
      auto stat = [&](int n) {
        const int h = w.kv * group + n / w.nq, i = (w.q_lo + n % w.nq) * kAttnTile + row;
        if (i >= w.t.len) return half ? 0.f : INFINITY;
        return (half ? a.delta : a.lse2)[(int64_t)h * a.n + w.t.b + i];
      };
      if (steps) {
        stats[(step & 1) * 256 + threadIdx.x] = stat(0);
        mbar_arrive(stat_full);
      }
      for (int n = 0; n < steps && ok; ++n, ++step) {
        const float next = n + 1 < steps ? stat(n + 1) : 0.f;
        const float* st = stats + (step & 1) * 256 + 64 * half;
        ok = __all_sync(0xffffffffu, mbar_wait(stat_full, step & 1, abort_flag, err, kErrDkv));
        if (!ok) break;
        ok = __all_sync(0xffffffffu, mbar_wait(s_full, step & 1, abort_flag, err, kErrDkv));
        if (!ok) break;
        tc_fence_after();
        uint32_t p[2][32], g[2][32], r[32];
        tmem_ld_32x32b_x32(ts, p[0]);
        tmem_ld_32x32b_x32(ts + 32, p[1]);
        tmem_ld_wait();
        const int q0 = (w.q_lo + n % w.nq) * kAttnTile;
        // query q0 + col sees key j for col >= from and (col <= to or j < sinks)
        const int j = w.t.p0 + row, from = j - q0;
        const int to = j < a.sinks ? kAttnTile : (int)min((int64_t)j + a.window - 1 - q0, (int64_t)kAttnTile);
        const bool masked = !tile_full(a, q0, w.t.p0);
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 l4 = *reinterpret_cast<const float4*>(st + 32 * x + e);
            const float l[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              float q = ex2(fmaf(__uint_as_float(p[x][e + y]), a.scale_log2, -l[y]));
              if (masked) {
                const int col = 64 * half + 32 * x + e + y;
                if (col < from || col > to) q = 0.f;
              }
              p[x][e + y] = __float_as_uint(q);
            }
          }
#pragma unroll
        for (int e = 0; e < 32; ++e)
          r[e] = op_pack_bf16(__uint_as_float(p[e >> 4][(2 * e) & 31]), __uint_as_float(p[e >> 4][((2 * e) & 31) + 1]));
        tmem_st_32x32b_x32(ts, r);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(p_full);
        ok = __all_sync(0xffffffffu, mbar_wait(dp_full, step & 1, abort_flag, err, kErrDkv));
        if (!ok) break;
        tc_fence_after();
        tmem_ld_32x32b_x32(tg, g[0]);
        tmem_ld_32x32b_x32(tg + 32, g[1]);
        tmem_ld_wait();
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 d4 = *reinterpret_cast<const float4*>(st + 128 + 32 * x + e);
            const float d[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
            for (int y = 0; y < 4; y += 2)
              r[16 * x + (e + y) / 2] =
                  op_pack_bf16(__uint_as_float(p[x][e + y]) * (__uint_as_float(g[x][e + y]) - d[y]),
                               __uint_as_float(p[x][e + y + 1]) * (__uint_as_float(g[x][e + y + 1]) - d[y + 1]));
          }
        tmem_st_32x32b_x32(tg, r);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(ds_full);
        if (n + 1 < steps) {
          // every thread has read the buffer's last contents: it arrived after them for this step
          stats[((step + 1) & 1) * 256 + threadIdx.x] = next;
          mbar_arrive(stat_full);
        }
      }
      if (!ok) break;
      if (steps) {
        ok = __all_sync(0xffffffffu, mbar_wait(done, done_ph, abort_flag, err, kErrDkv));
        if (!ok) break;
        done_ph ^= 1;
        tc_fence_after();
      }
      // warps 0-3 store dV, warps 4-7 dK
      const int j = w.t.p0 + row;
      const float f = half ? a.scale : 1.f;
      const bool part = w.slot >= 0 && j < a.sinks;
      float* pp = partial + ((w.slot * a.kv_heads + w.kv) * 2 + half) * (int64_t)a.sinks * a.dim + (int64_t)j * a.dim;
      __nv_bfloat16* po = (half ? dk : dv) + (((int64_t)w.t.b + j) * a.kv_heads + w.kv) * a.dim;
      const bool mine = j < w.t.len && (part ? w.slot < partial_slots : !w.sink_only);
#pragma unroll 1
      for (int c = 0; c < DP; c += 32) {
        uint32_t o[32];
        if (steps) {
          tmem_ld_32x32b_x32(tmem + lanes + 256u + 128u * half + c, o);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
        if (mine) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            if (c + e < a.dim) {
              float x[8];
#pragma unroll
              for (int y = 0; y < 8; ++y) x[y] = __uint_as_float(o[e + y]) * f;
              if (part)
                store8(pp + c + e, x);
              else
                store8(po + c + e, x);
            }
          }
        }
      }
      tc_fence_before();
    }
  } else if (warp == 8) {
    uint32_t pos = 0, kv_ph = 1, kv_loads = 0;
    for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
      const DkvItem w = dkv_item(a, item, sink_items, lane);
      const int steps = group * w.nq;
      for (int n = 0; n < steps && ok; ++n) {
        const int h = w.kv * group + n / w.nq, token = w.t.b + (w.q_lo + n % w.nq) * kAttnTile;
        for (int x = 0; x < 2 && ok; ++x) {
          ok = mbar_wait(ring.empty_bar(pos), ring.empty_parity(pos), abort_flag, err, kErrDkv);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) {
            mbar_expect_tx(ring.full_bar(pos), SM::TILE);
            load_tile<DP>(ring.slot(pos), x ? &tmDO : &tmQ, token, h, ring.full_bar(pos));
          }
          ++pos;
          if (n == 0 && x == 0) {
            // keys and values once the item before has done with its own
            ok = mbar_wait(done, kv_ph, abort_flag, err, kErrDkv);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            kv_ph ^= 1;
            ++kv_loads;
            if (lane == 0) {
              mbar_expect_tx(kv_full, 2 * SM::TILE);
              load_tile<DP>(base, &tmK, w.t.b + w.t.p0, w.kv, kv_full);
              load_tile<DP>(base + SM::TILE, &tmV, w.t.b + w.t.p0, w.kv, kv_full);
            }
          }
        }
      }
    }
    for (uint32_t k = pos > SM::SLOTS ? pos - SM::SLOTS : 0; k < pos; ++k)
      drain_wait(ring.full_bar(k), ring.full_parity(k));
    if (kv_loads) drain_wait(kv_full, (kv_loads - 1) & 1);
  } else {
    uint32_t pos = 0, kv_ph = 0, step = 0;
    for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
      const DkvItem w = dkv_item(a, item, sink_items, lane);
      const int steps = group * w.nq;
      if (steps == 0) continue;
      ok = __all_sync(0xffffffffu, mbar_wait(kv_full, kv_ph, abort_flag, err, kErrDkv));
      if (!ok) break;
      kv_ph ^= 1;
      // x = 0: S^T of step n from its queries; 1: dP^T from its output gradients
      auto issue = [&](int n, int x) {
        const uint32_t k = pos + 2 * n + x;
        ok = mbar_wait(ring.full_bar(k), ring.full_parity(k), abort_flag, err, kErrDkv);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return false;
        const int valid = w.t.len - (w.q_lo + n % w.nq) * kAttnTile;
        if (valid < kAttnTile) clear_rows<DP>(ring.slot(k), valid, lane);
        tc_fence_after();
        if (lane == 0) {
          mma_abt<DP>(tmem + 128u * x, base + x * SM::TILE, ring.slot(k));
          umma_commit<1>(x ? dp_full : s_full);
        }
        __syncwarp();
        return true;
      };
      if (!issue(0, 0) || !issue(0, 1)) break;
      for (int n = 0; n < steps && ok; ++n, ++step) {
        ok = __all_sync(0xffffffffu, mbar_wait(p_full, step & 1, abort_flag, err, kErrDkv));
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
          mma_ab<DP>(tmem + 256u, tmem, 64, ring.slot(pos + 2 * n + 1), n > 0);
          umma_commit<1>(ring.empty_bar(pos + 2 * n + 1));
        }
        __syncwarp();
        if (n + 1 < steps && !issue(n + 1, 0)) break;
        ok = __all_sync(0xffffffffu, mbar_wait(ds_full, step & 1, abort_flag, err, kErrDkv));
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
          mma_ab<DP>(tmem + 384u, tmem + 128u, 64, ring.slot(pos + 2 * n), n > 0);
          umma_commit<1>(ring.empty_bar(pos + 2 * n));
        }
        __syncwarp();
        if (n + 1 < steps && !issue(n + 1, 1)) break;
      }
      if (!ok) break;
      if (lane == 0) umma_commit<1>(done);
      __syncwarp();
      pos += 2 * steps;
    }
    if (lane == 0) {
      umma_commit<1>(drain);
      drain_wait(drain, 0);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc<1>(tmem, 512);
}

// dK and dV of the sink keys: the first tile's own sums, then the chunks'.
__global__ void __launch_bounds__(256) window_sink_kernel(const __grid_constant__ AttnArgs a,
                                                          const float* __restrict__ partial, int64_t partial_slots,
                                                          __nv_bfloat16* __restrict__ dk,
                                                          __nv_bfloat16* __restrict__ dv) {
  __shared__ int first_chunk;
  pdl_launch();
  pdl_wait();
  const int sample = blockIdx.x, kv = blockIdx.y;
  if (threadIdx.x < 32) {
    // chunks of the samples before this one
    int sum = 0;
    if (a.cu)
      for (int i = threadIdx.x; i < sample; i += 32) {
        int b, len;
        sample_span(a, i, b, len);
        sum += sink_chunks(a, len, true);
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (threadIdx.x == 0) first_chunk = sum;
  }
  __syncthreads();
  int b = 0, len = a.n;
  if (a.cu) sample_span(a, sample, b, len);
  const int chunks = sink_chunks(a, len, true), rows = min(a.sinks, len);
  const int64_t per = (int64_t)a.sinks * a.dim, slot = (int64_t)a.kv_heads * 2 * per;
  for (int e = threadIdx.x; e < 2 * rows * a.dim; e += 256) {
    const int which = e >= rows * a.dim, x = which ? e - rows * a.dim : e;
    const float* p = partial + (kv * 2 + which) * per + x;
    float s = p[sample * slot];
    for (int c = 0; c < chunks; ++c) {
      const int64_t at = (int64_t)a.n_seqs + first_chunk + c;
      if (at < partial_slots) s += p[at * slot];
    }
    const int row = x / a.dim;
    (which ? dk : dv)[(((int64_t)b + row) * a.kv_heads + kv) * a.dim + (x - row * a.dim)] = __float2bfloat16_rn(s);
  }
}

template <int DP>
cudaError_t run_backward(const AttnArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                         const CUtensorMap& dout, const AttnGrad& g, int* err, int sms, cudaStream_t st) {
  const int64_t tiles = attn_max_tiles(a.n, a.n_seqs, kAttnTile);
  cudaError_t e = op_smem_limit<window_dq_kernel<DP>>((int)DqSmem<DP>::BYTES);
  if (e == cudaSuccess) e = op_smem_limit<window_dkv_kernel<DP>>((int)DkvSmem<DP>::BYTES);
  if (e != cudaSuccess) return e;
  int64_t grid = tiles * a.heads;
  e = op_launch(window_dq_kernel<DP>, dim3((unsigned)(grid < sms ? grid : sms)), dim3(kThreads), DqSmem<DP>::BYTES, st,
                1, a, q, k, v, dout, g.dq, err);
  if (e != cudaSuccess) return e;
  grid = (tiles + g.partial_slots) * a.kv_heads;
  return op_launch(window_dkv_kernel<DP>, dim3((unsigned)(grid < sms ? grid : sms)), dim3(kThreads),
                   DkvSmem<DP>::BYTES, st, 1, a, q, k, v, dout, g.dk, g.dv, g.partial, g.partial_slots, err);
}

}  // namespace

cudaError_t attn_backward(AttnArgs a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                          const CUtensorMap& dout, const AttnGrad& g, int* err, int sms, cudaStream_t st) {
  const int64_t rows = ((int64_t)a.n * a.heads + 15) / 16, most = (int64_t)sms * 8;
  cudaError_t e = op_launch(window_stats_kernel, dim3((unsigned)(rows < most ? rows : most)), dim3(256), 0, st, 1, a,
                            g.dout, g.do_ts, g.do_hs, g.out, g.lse, g.lse2, g.delta);
  if (e != cudaSuccess) return e;
  a.lse2 = g.lse2;
  a.delta = g.delta;
  e = a.dim > 64 ? run_backward<128>(a, q, k, v, dout, g, err, sms, st)
                 : run_backward<64>(a, q, k, v, dout, g, err, sms, st);
  if (e != cudaSuccess || a.sinks == 0) return e;
  return op_launch(window_sink_kernel, dim3((unsigned)a.n_seqs, (unsigned)a.kv_heads), dim3(256), 0, st, 1, a,
                   static_cast<const float*>(g.partial), g.partial_slots, g.dk, g.dv);
}

}  // namespace ma
