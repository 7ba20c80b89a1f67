// Gradient of the sliding-window attention.
//
// With P = exp2(c S - lse2) (the forward pass's softmax weights, lse2 = log2(e)
// times its saved lse), dP = dO V^T, delta_i = dO_i . O_i:
//   dS = P (dP - delta),  dV = P^T dO,  dK = scale dS^T Q,  dQ = scale dS K.
//
// window_stats_kernel  lse2 and delta of every query and head.
// window_grad_kernel   dkv_part: 128 keys of a key head, walking the query tiles
//                      of every head that reads it; then dq_part: 128 queries of
//                      a head, walking their key tiles.
//
// Seven products instead of the five that one kernel would need, because S and
// dP are formed twice: dQ would otherwise have to be added up by atomics in an
// order that changes from run to run, or stored in fp32 once per key tile.
//
// Bound by the tensor cores where samples are long: 16384 tokens of 16 heads of 128
// over 8 key heads, all keys visible, take 2.3 ms, 1659 TFLOP/s of products formed
// (0.88 of the measured bf16 peak). With a window of 1024 and four sinks 440 us, of
// which the statistics are 25 (8192 tokens over 16 key heads: 222 us, without sinks
// 204). There a dK/dV step takes 2950 cycles for 2048 of products, since S^T of the
// next queries waits for dV, which waits for P^T in its place, a dQ step 2130 for 1536;
// edge tiles, the sinks' own steps and the ends of items are the rest. Six samples of 7
// to 1021 tokens (16 heads of 64, window 256): 52 us, bound by the latency of items of
// three steps: a CTA has about 16 steps in all, of some 5000 cycles each for 1000 of
// products, since the ends of its items do not overlap (dq_part has one buffer each
// for Q and dO and one accumulator, for heads of up to 64 too).
//
// Heads of other widths run at the next of 64 and 128: 8192 tokens of 16 heads over 8,
// window 1024, four sinks, take 158 us of 32, 163 of 64, 201 to 210 of 72 to 128.
//
// The sink keys are seen by every query of a sample. Their gradients are cut
// into chunks of kSinkChunk query tiles, each a work item of its own; the CTA that
// ends the last of a sample's adds their fp32 sums in a fixed order (a launch of its
// own for that took 9 us at 16384 tokens and 4 at short samples).
#include <limits.h>

#include "window_attention.cuh"

namespace ma {
namespace {

constexpr int kMathWarps = 16;
constexpr int kThreads = (kMathWarps + 4) * 32;
constexpr int kTma = kMathWarps, kMmaA = kMathWarps + 1, kMmaB = kMathWarps + 2;  // and the clearing warp
// of the 96 registers a thread is launched with: 16 * 104 + 4 * 64 = 20 * 96
constexpr int kMathRegs = 104, kOtherRegs = 64;
constexpr int kErrDq = 0x202, kErrDkv = 0x203, kErrAlign = 0x204;

// ---- lse2 and delta ----
// A group of 16 lanes to a (token, head), eight elements a lane. Bound by HBM: 134 MB
// in 25 us (5.4 TB/s) at 16384 tokens of 16 heads of 128. (Four rows of a group in
// flight took 36 us, with 77 registers; 16 tokens of one head to a block 28.)
__global__ void __launch_bounds__(256) window_stats_kernel(const __grid_constant__ AttnArgs a,
                                                           const __nv_bfloat16* __restrict__ dout, int64_t do_ts,
                                                           int64_t do_hs, const __nv_bfloat16* __restrict__ out,
                                                           int64_t o_ts, int64_t o_hs, const float* __restrict__ lse, float* __restrict__ nlse2,
                                                           float* __restrict__ ndelta, int* __restrict__ counter) {
  pdl_launch();
  pdl_wait();
  // the next launch's counters: of dQ items, and of the sink items of each sample and key head
  const int64_t counters = 1 + (int64_t)a.n_seqs * a.kv_heads;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < counters; i += (int64_t)gridDim.x * 256) counter[i] = 0;
  const int gl = threadIdx.x & 15;
  // 16 rows (token, head) a block and step; the row advances without a division
  const int step = gridDim.x * 16, up_t = step / a.heads, up_h = step - up_t * a.heads;
  const int64_t first = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  int t = (int)min(first / a.heads, (int64_t)a.n), h = (int)(first - first / a.heads * a.heads);
  // whole warps stay in the loop for the sum across lanes
  while (__any_sync(0xffffffffu, t < a.n)) {
    float s = 0.f;
    if (t < a.n && gl * 8 < a.dim) {
      float x[8], y[8];
      load8(dout + t * do_ts + h * do_hs + gl * 8, x);
      load8(out + t * o_ts + h * o_hs + gl * 8, y);
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(x[i], y[i], s);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (t < a.n && gl == 0) {
      const int64_t at = (int64_t)h * a.n + t;
      const float l = lse[at];
      nlse2[at] = l == -INFINITY ? -INFINITY : l * -1.4426950408889634f;
      ndelta[at] = -s;
    }
    t += up_t, h += up_h;
    if (h >= a.heads) h -= a.heads, ++t;
  }
}

// ---- dQ ----
// Warps 0-15: a thread to a query and a block of 32 of a tile's keys (warps 0-3
// the first block, and so on); warp 16: TMA; warps 17 and 18: tcgen05.mma, the
// one S and dQ, the other dP; warp 19: clears the key and value rows of other
// samples and stores the finished tiles. Sixteen warps rather than eight with twice
// the keys: a step's chain of waits, TMEM reads and exponentials is what bounds this.
// TMEM: S of even steps | S of odd steps | dP | dQ. dS (bf16) overwrites the S
// it came from, each block in the first 16 of its own 32 columns. S of the next
// tile is formed while the threads work on this one's, and dP of the next as
// soon as this one's has been read.
template <int DP>
struct GradSmem {
  static constexpr uint32_t TILE = kAttnTile * DP * 2;
  static constexpr int SLOTS = DP == 128 ? 5 : 8;
  // dK/dV: buffers for K and V, and for S^T in TMEM. Heads of up to 64 leave room for two of each: the next item's
  // operands are there when it begins, and S^T of a step is formed while the threads hold the weights of the one
  // before.
  static constexpr int KV = DP == 128 ? 1 : 2, NS = DP == 128 ? 1 : 2;
  static constexpr uint32_t RING = 2 * KV * TILE;              // after K and V, or Q and dO
  static constexpr uint32_t STATS = RING + SLOTS * TILE;       // dkv: [2][nlse2, ndelta][128] of the query tiles
  static constexpr uint32_t BARS = STATS + 2 * 2 * kAttnTile * 4;
  static constexpr int NBARS = 8 * SLOTS + 45;  // dK/dV's and dQ's
  static constexpr uint32_t BYTES = BARS + NBARS * 8 + 32;
  static_assert(BYTES <= 232448, "shared memory per CTA");
};

struct DqItem {
  SampleTile t;
  KeyTiles k;
  int steps, head, kv;
  bool staged;  // leaves through the ring, in the position after the last values
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
  w.staged = w.steps > 0 && w.t.p0 + kAttnTile <= w.t.len;
  return w;
}

__device__ __forceinline__ void parts_sync() {
  tc_fence_before();
  asm volatile("barrier.sync 1, %0;" ::"n"(kThreads) : "memory");
  tc_fence_after();
}

// dQ items go to the CTAs in the order in which they come for them, so that those
// whose dK/dV items took longer take fewer (static shares: 6 % longer on short
// samples, 1 % at 16384 tokens; all keys of 8192 visible 700 us, drawn 618, and drawn
// with the last tiles first 590). The TMA warp draws an item's number
// from a counter, one item ahead of its loads, and posts it to the other warps.
constexpr int kPosts = 4;
struct DqPosts {
  uint32_t full, empty, data;  // barriers and numbers, [kPosts] each
  uint32_t nth;                // the next to be posted or taken

  // By the TMA warp.
  __device__ __forceinline__ int post(int* counter, int lane, bool& ok, volatile int* abort_flag, int* err) {
    int item = INT_MAX;
    if (lane == 0 && ok) {
      const uint32_t at = nth % kPosts;
      ok = mbar_wait_in(empty + 8 * at, (nth / kPosts & 1) ^ 1, abort_flag, err, kErrDq);
      if (ok) {
        item = atomicAdd(counter, 1);
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(data + 4 * at), "r"(item) : "memory");
        mbar_arrive(full + 8 * at);
      }
    }
    ++nth;
    ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
    return __shfl_sync(0xffffffffu, item, 0);
  }
  // By each of the other warps, once for each number.
  __device__ __forceinline__ int take(int lane, bool& ok, volatile int* abort_flag, int* err) {
    const uint32_t at = nth % kPosts;
    int item = INT_MAX;
    ok = ok && mbar_wait_warp(full + 8 * at, nth / kPosts & 1, abort_flag, err, kErrDq);
    if (ok) {
      asm volatile("ld.shared.b32 %0, [%1];" : "=r"(item) : "r"(data + 4 * at) : "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + 8 * at);
    }
    ++nth;
    return item;
  }
};

template <int DP>
struct DqBarriers {
  static constexpr int COUNT = 4 * GradSmem<DP>::SLOTS + 13 + 2 * kPosts;
};

template <int DP, bool MATH>
__device__ __forceinline__ void dq_part(const AttnArgs& a, const CUtensorMap& tmQ, const CUtensorMap& tmK,
                                        const CUtensorMap& tmV, const CUtensorMap& tmDO, const CUtensorMap& tmDQ,
                                        __nv_bfloat16* __restrict__ dq, int* __restrict__ err, volatile int* abort_flag,
                                        uint32_t base, uint32_t bars, uint32_t tmem, uint32_t numbers, int* counter,
                                        bool set_up) {
  using SM = GradSmem<DP>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Ring<SM::SLOTS> ring{base + SM::RING, bars, bars + SM::SLOTS * 8, bars + SM::SLOTS * 16, SM::TILE};
  // full[SLOTS], empty[SLOTS], raw[SLOTS], staged[SLOTS], then
  const uint32_t staged = bars + 3 * SM::SLOTS * 8, own = bars + 4 * SM::SLOTS * 8, q_full = own, q_empty = own + 8, do_full = own + 16,
                 do_empty = own + 24, s_full = own + 32, dp_full = own + 48, dp_empty = own + 56, ds_full = own + 64,
                 dq_full = own + 80, drain = own + 88;
  DqPosts posts{own + 104, own + 104 + 8 * kPosts, numbers, 0};
  static_assert(DqBarriers<DP>::COUNT == 4 * SM::SLOTS + 104 / 8 + 2 * kPosts, "barriers");
  if (set_up) {
    ring.init(1);
    for (int i = 0; i < SM::SLOTS; ++i) mbar_init(staged + 8 * i, kMathWarps / (DP == 64 ? 2 : 1));
    mbar_init(q_full, 1), mbar_init(q_empty, 1), mbar_init(do_full, 1), mbar_init(do_empty, 1);
    mbar_init(s_full, 1), mbar_init(s_full + 8, 1), mbar_init(dp_full, 1), mbar_init(dp_empty, kMathWarps);
    mbar_init(ds_full, kMathWarps), mbar_init(ds_full + 8, kMathWarps), mbar_init(dq_full, 1), mbar_init(drain, 1), mbar_init(drain + 8, 1);
    for (int i = 0; i < kPosts; ++i) mbar_init(posts.full + 8 * i, 1), mbar_init(posts.empty + 8 * i, kMathWarps + 3);
    return;
  }
  const int items = a.heads * count_units(a, lane, [](int len, bool) { return (len + kAttnTile - 1) / kAttnTile; });
  const int few = sink_columns(a);
  // the last tiles first: where the window lets them, they meet the most keys
  auto nth_item = [&](int n) { return dq_item(a, items - 1 - n, lane); };
  bool ok = true;
  int item = INT_MAX;
  if (!MATH && warp == kTma) item = posts.post(counter, lane, ok, abort_flag, err);
  // every product and copy of the first part has ended
  parts_sync();
  ok = __all_sync(0xffffffffu, ok && *abort_flag == 0);
  if (MATH || warp != kTma) item = posts.take(lane, ok, abort_flag, err);

  if constexpr (MATH) {
    const int blk = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    uint32_t step = 0, s_ph = 0, dq_ph = 0;  // step: over all items; s_ph: a bit per S slot
    Cursor<SM::SLOTS> cur;
    const uint64_t scale2 = pack2(a.scale_log2, a.scale_log2);
    const bool wide = rows_wide(dq, a.dim);
    DqItem next;
    if (item < items) next = nth_item(item);
    while (item < items && ok) {
      const DqItem w = next;
      const int i = w.t.p0 + row;
      const int64_t t = (int64_t)w.t.b + i;
      const bool mine = i < w.t.len;
      const float nlse2 = mine ? a.nlse2[(int64_t)w.head * a.n + t] : -INFINITY;
      const float ndelta = mine ? a.ndelta[(int64_t)w.head * a.n + t] : 0.f;
      const uint64_t shift2 = pack2(nlse2, nlse2), delta2 = pack2(ndelta, ndelta);
      for (int n = 0; n < w.steps && ok; ++n, ++step) {
        const uint32_t slot = n & 1, ts = tmem + lanes + 128u * slot + 32u * blk;
        const int k0 = w.tile(n) * kAttnTile + 32 * blk;  // of this block
        ok = mbar_wait_warp(s_full + 8 * slot, s_ph >> slot & 1, abort_flag, err, kErrDq);
        if (!ok) break;
        s_ph ^= 1u << slot;
        tc_fence_after();
        uint32_t p[32], g[32], ds[16];
        tmem_ld_32x32b_x32(ts, p);
        tmem_ld_wait();
        bool seen = true;
        if (!tile_full(a, w.t.p0, w.tile(n) * kAttnTile)) {
          // key k0 + col is visible for col < end and (col >= first or col < sink); past the sinks' columns of
          // a tile that is there for them alone no score has been formed
          const int cols = w.k.sink && n == 0 ? few - 32 * blk : 32;
          const int end = min(i - k0 + 1, cols), first = i - k0 - a.window + 1, sink = min(a.sinks - k0, end);
          const uint32_t m = bit_range(first, end) | bit_range(0, sink);
          seen = __any_sync(0xffffffffu, m != 0u);
          if (seen && !__all_sync(0xffffffffu, m == 0xffffffffu)) mask_block(p, m);
        }
        if (seen) {
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            float u, v;
            unpack2(fma2(pack2(p[j], p[j + 1]), scale2, shift2), u, v);
            p[j] = __float_as_uint(ex2(u));
            p[j + 1] = __float_as_uint(ex2(v));
          }
        }
        ok = mbar_wait_warp(dp_full, step & 1, abort_flag, err, kErrDq);
        if (!ok) break;
        tc_fence_after();
        tmem_ld_32x32b_x32(tmem + lanes + 256u + 32u * blk, g);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(dp_empty);
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          float u, v;
          unpack2(mul2(pack2(p[j], p[j + 1]), add2(pack2(g[j], g[j + 1]), delta2)), u, v);
          ds[j / 2] = seen ? op_pack_bf16(u, v) : 0u;
        }
        tmem_st_32x32b_x16(ts, ds);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ds_full + 8 * slot);
      }
      if (!ok) break;
      item = posts.take(lane, ok, abort_flag, err);
      if (item < items) next = nth_item(item);
      if (w.steps) {
        ok = mbar_wait_warp(dq_full, dq_ph, abort_flag, err, kErrDq);
        if (!ok) break;
        dq_ph ^= 1;
        tc_fence_after();
      }
      cur.skip(2 * w.steps);
      // a quarter of the columns to each four warps (of 64: half to each of the first eight)
      if (w.staged) {
        if (32 * blk < DP) {
          ok = mbar_wait_warp(cur.full(ring), cur.phase, abort_flag, err, kErrDq);
          if (!ok) break;
          stage_row(tmem + lanes + 384u, 32 * blk, 32 * blk + 32, a.scale, false, cur.data(ring), row);
          __syncwarp();
          if (lane == 0) mbar_arrive(staged + 8 * cur.slot);
        }
        cur.advance();
      } else if (32 * blk < DP)
        store_row(tmem + lanes + 384u, 32 * blk, 32 * blk + 32, a.scale, w.steps == 0,
                  dq + (t * a.heads + w.head) * a.dim, mine, a.dim, wide);
      tc_fence_before();
    }
  } else if (warp == kTma) {
    Cursor<SM::SLOTS> cur;
    uint32_t loads = 0, raw_phase = 0;
    while (item < items && ok) {
      const DqItem w = nth_item(item);
      item = posts.post(counter, lane, ok, abort_flag, err);
      if (lane == 0) {
        for (int n = 0; n < w.steps && ok; ++n) {
          const int at = w.tile(n) * kAttnTile;
          for (int kv = 0; kv < 2 && ok; ++kv) {
            if (n == 0) {
              // Q before the first keys, dO before the first values
              ok = mbar_wait_in(kv ? do_empty : q_empty, (loads & 1) ^ 1, abort_flag, err, kErrDq);
              if (!ok) break;
              mbar_expect_tx(kv ? do_full : q_full, SM::TILE);
              load_tile<DP>(base + kv * SM::TILE, kv ? &tmDO : &tmQ, w.t.b + w.t.p0, w.head, kv ? do_full : q_full);
            }
            ok = mbar_wait_in(cur.empty(ring), cur.phase ^ 1, abort_flag, err, kErrDq);
            if (!ok) break;
            fill_slot<DP>(ring, cur, kv ? &tmV : &tmK, w.t.b + at, w.kv, w.t.len - at, raw_phase);
            cur.advance();
          }
        }
        if (w.steps) ++loads;
        if (w.staged && ok) {
          ok = mbar_wait_in(cur.empty(ring), cur.phase ^ 1, abort_flag, err, kErrDq);
          if (ok) {
            mbar_arrive(cur.full(ring));
            cur.advance();
          }
        }
      }
      ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
    }
    if (lane == 0) {
      drain_ring(ring, cur, raw_phase);
      if (loads) {
        // (after a wait that ran out dO's last copy may not have been asked for: this wait is bounded too)
        drain_wait(q_full, (loads - 1) & 1);
        drain_wait(do_full, (loads - 1) & 1);
      }
    }
    __syncwarp();
  } else if (warp == kMmaA) {
    // S of the next steps, dQ
    Cursor<SM::SLOTS> sc;  // the next S's key tile
    uint32_t q_ph = 0, ds_ph = 0;  // ds_ph: a bit per S slot
    const uint32_t tm = warp_uniform(tmem);
    DqItem next;
    if (item < items) next = nth_item(item);
    while (item < items && ok) {
      const int steps = warp_uniform(next.steps), sink = warp_uniform((int)next.k.sink),
                out = warp_uniform((int)next.staged);
      if (steps == 0) {
        item = posts.take(lane, ok, abort_flag, err);
        if (item < items) next = nth_item(item);
        continue;
      }
      Cursor<SM::SLOTS> qc = sc;  // the next dQ's key tile
      auto issue_s = [&](int n) {
        if (!mbar_wait_warp(sc.full(ring), sc.phase, abort_flag, err, kErrDq)) return false;
        tc_fence_after();
        mma_abt<DP>(tm + 128u * (n & 1), base, sc.data(ring), n == 0 && sink ? few : kAttnTile);
        umma_commit_warp(s_full + 8 * (n & 1));
        if (n == steps - 1) umma_commit_warp(q_empty);
        sc.skip(2);
        return true;
      };
      ok = mbar_wait_warp(q_full, q_ph, abort_flag, err, kErrDq) && issue_s(0) && (steps == 1 || issue_s(1));
      q_ph ^= 1;
      item = posts.take(lane, ok, abort_flag, err);
      if (item < items) next = nth_item(item);
      for (int n = 0; n < steps && ok; ++n) {
        // (a barrier to each slot of S: the threads need nothing of this warp for the step after, so that they
        // may be through with it before this wait, and one barrier's phases would have passed twice)
        const uint32_t slot = n & 1;
        if (!(ok = mbar_wait_warp(ds_full + 8 * slot, ds_ph >> slot & 1, abort_flag, err, kErrDq))) break;
        ds_ph ^= 1u << slot;
        tc_fence_after();
        if (n > 0 || !sink)
          mma_ab<DP, 32>(tm + 384u, tm + 128u * (n & 1), qc.data(ring), n > 0);
        else
          mma_ab_few<DP, 32>(tm + 384u, tm, qc.data(ring), false, few);
        umma_commit_warp(qc.empty(ring));
        qc.skip(2);
        if (n + 2 < steps) ok = issue_s(n + 2);
      }
      if (ok) umma_commit_warp(dq_full);
      if (out) sc.advance();
    }
    umma_commit_warp(drain);
    if (lane == 0) drain_wait(drain, 0);
    __syncwarp();
  } else if (warp == kMmaB) {
    // dP, once the threads have read the one before
    Cursor<SM::SLOTS> pc;  // a key tile, then its value tile
    uint32_t q_ph = 0, step = 0;
    const uint32_t tm = warp_uniform(tmem);
    DqItem next;
    if (item < items) next = nth_item(item);
    while (item < items && ok) {
      const int steps = warp_uniform(next.steps), sink = warp_uniform((int)next.k.sink),
                out = warp_uniform((int)next.staged);
      item = posts.take(lane, ok, abort_flag, err);
      if (item < items) next = nth_item(item);
      if (steps == 0) continue;
      ok = ok && mbar_wait_warp(do_full, q_ph, abort_flag, err, kErrDq);
      q_ph ^= 1;
      for (int n = 0; n < steps && ok; ++n, ++step) {
        pc.advance();
        // (parity of the step before; the very first passes)
        ok = mbar_wait_warp(dp_empty, (step & 1) ^ 1, abort_flag, err, kErrDq) &&
             mbar_wait_warp(pc.full(ring), pc.phase, abort_flag, err, kErrDq);
        if (!ok) break;
        tc_fence_after();
        mma_abt<DP>(tm + 256u, base + SM::TILE, pc.data(ring), n == 0 && sink ? few : kAttnTile);
        umma_commit_warp(dp_full);
        umma_commit_warp(pc.empty(ring));
        if (n == steps - 1) umma_commit_warp(do_empty);
        pc.advance();
      }
      if (out) pc.advance();
    }
    umma_commit_warp(drain + 8);
    if (lane == 0) drain_wait(drain + 8, 0);
    __syncwarp();
  } else {
    Cursor<SM::SLOTS> cur;
    uint32_t raw_phase = 0, staged_phase = 0;
    while (item < items && ok) {
      const DqItem w = nth_item(item);
      item = posts.take(lane, ok, abort_flag, err);
      if (w.steps == 0) continue;
      cur.skip(2 * w.steps - 2);
      const int valid = w.t.len - w.tile(w.steps - 1) * kAttnTile;  // only the last tile can be ragged
      for (int kv = 0; kv < 2; ++kv) {
        if (valid < kAttnTile && ok)
          ok = clear_slot<DP>(ring, cur, valid, raw_phase, lane, abort_flag, err, kErrDq);
        cur.advance();
      }
      if (w.staged && ok) {
        ok = store_slot<DP>(ring, cur, staged, staged_phase, &tmDQ, w.t.b + w.t.p0, w.head, 1, lane, abort_flag, err,
                            kErrDq);
        cur.advance();
      }
    }
  }
}

// ---- dK and dV ----
// Scores are formed transposed, S^T = K Q^T and dP^T = V dO^T, so that P^T and
// dS^T stand in TMEM as the left operands of dV += P^T dO and dK += dS^T Q.
// Warps 0-15: a thread to a key and a block of 32 of a tile's queries; warp 16:
// TMA; warps 17 and 18: tcgen05.mma, the one dV and the next step's S^T, the other
// dK and the next dP^T, issued behind them; warp 19: clears rows of Q and dO that
// belong to other samples, and stores the finished tiles. TMEM: S^T | dP^T | dV | dK,
// and for heads of up to 64 a second S^T behind them; P^T overwrites S^T and dS^T
// dP^T, each block in the first 16 of its own 32 columns. While the threads form P^T
// of a step the tensor core runs the step before's dK and this one's dP^T; while
// they form dS^T it runs dV and the next step's S^T (with two buffers S^T is formed a
// step earlier: 8192 tokens of 16 heads of 64 over 8, window 1024, four sinks, take
// 163 us, of 72 209).
//
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
  int64_t slot;     // partial slot of the sink keys, -1: none (no other item sees any of them)
  bool sink_only;   // a chunk for the sink keys alone
  bool staged;      // dV and dK leave through the ring, in the positions after the last step's tiles
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
    w.slot = w.t.index == 0 && sink_chunks(a, w.t.len, w.t.live) > 0 ? w.t.sample : -1;
  }
  w.staged = w.slot < 0 && w.nq > 0 && w.t.p0 + kAttnTile <= w.t.len;
  return w;
}

// dK and dV of a sample's sink keys, by all threads that hold scores: the first
// tile's own sums, then the chunks' in their order.
__device__ __forceinline__ void sum_sinks(const AttnArgs& a, const SampleTile& t, int kv, const float* partial,
                                          int64_t partial_slots, __nv_bfloat16* __restrict__ dk,
                                          __nv_bfloat16* __restrict__ dv, int lane) {
  int before = 0;  // chunks of the samples before this one
  if (a.cu)
    for (int i = lane; i < t.sample; i += 32) {
      int b, len;
      sample_span(a, i, b, len);
      before += sink_chunks(a, len, true);
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  const int rows = min(a.sinks, t.len);
  const int64_t per = (int64_t)a.sinks * a.dim, slot = (int64_t)a.kv_heads * 2 * per, at = (int64_t)a.n_seqs + before;
  const int64_t n = min((int64_t)sink_chunks(a, t.len, true), partial_slots - at);
  for (int e = threadIdx.x; e < 2 * rows * a.dim; e += kMathWarps * 32) {
    const int which = e >= rows * a.dim, x = which ? e - rows * a.dim : e;
    const float* p = partial + (kv * 2 + which) * per + x;
    float s = __ldcg(p + t.sample * slot);
#pragma unroll 8
    for (int64_t c = 0; c < n; ++c) s += __ldcg(p + (at + c) * slot);
    const int row = x / a.dim;
    (which ? dk : dv)[(((int64_t)t.b + row) * a.kv_heads + kv) * a.dim + (x - row * a.dim)] = __float2bfloat16_rn(s);
  }
}

template <int DP>
struct DkvBarriers {
  static constexpr int COUNT = 4 * GradSmem<DP>::SLOTS + 24;
};

template <int DP, bool MATH>
__device__ __forceinline__ void dkv_part(const AttnArgs& a, const CUtensorMap& tmQ, const CUtensorMap& tmK,
                                         const CUtensorMap& tmV, const CUtensorMap& tmDO, const CUtensorMap& tmDK,
                                         const CUtensorMap& tmDV, __nv_bfloat16* __restrict__ dk, __nv_bfloat16* __restrict__ dv,
                                         float* __restrict__ partial, int64_t partial_slots, int* __restrict__ err,
                                         volatile int* abort_flag, float* stats, int* __restrict__ arrived,
                                         uint32_t last_word, uint32_t base, uint32_t bars, uint32_t tmem, int cta, int ctas, int sink_items, int items, bool set_up) {
  using SM = GradSmem<DP>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Ring<SM::SLOTS> ring{base + SM::RING, bars, bars + SM::SLOTS * 8, bars + SM::SLOTS * 16, SM::TILE};
  // full[SLOTS], empty[SLOTS], raw[SLOTS], staged[SLOTS], then
  const uint32_t staged = bars + 3 * SM::SLOTS * 8, own = bars + 4 * SM::SLOTS * 8, k_full = own, k_empty = own + 16,
                 v_full = own + 32, v_empty = own + 48, s_full = own + 64, p_full = own + 80, dp_full = own + 96,
                 ds_full = own + 104, stat_full = own + 112, done = own + 120, drain = own + 128, turn = own + 144,
                 summed = own + 176, told = own + 184;
  static_assert(DkvBarriers<DP>::COUNT == 4 * SM::SLOTS + (184 + 8) / 8, "barriers");
  constexpr int KV = SM::KV, NS = SM::NS;
  if (set_up) {
    ring.init(2);
    for (int i = 0; i < SM::SLOTS; ++i) mbar_init(staged + 8 * i, kMathWarps / 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full + 8 * i, 1), mbar_init(k_empty + 8 * i, 1), mbar_init(v_full + 8 * i, 1), mbar_init(v_empty + 8 * i, 1);
      mbar_init(s_full + 8 * i, 1), mbar_init(p_full + 8 * i, kMathWarps);
    }
    mbar_init(dp_full, 1), mbar_init(ds_full, kMathWarps), mbar_init(summed, kMathWarps), mbar_init(told, 1);
    mbar_init(stat_full, kMathWarps * 32), mbar_init(done, 2), mbar_init(drain, 1), mbar_init(drain + 8, 1);
    for (int i = 0; i < 4; ++i) mbar_init(turn + 8 * i, 1);
    return;
  }
  const int group = a.heads / a.kv_heads;
  bool ok = true;
  // The first items, the sinks' among them, go to the CTAs in turn, the others the other way round: the CTAs that
  // begin with a long one are the last to get one more.
  auto at = [&](int i) { return i == 0 ? cta : i * ctas + ctas - 1 - cta; };

  if constexpr (MATH) {
    const int blk = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tg = tmem + lanes + 32u * blk + 128u;
    uint32_t step = 0, done_ph = 0, slot_ph = 0;
    Cursor<SM::SLOTS> cur;
    const uint64_t scale2 = pack2(a.scale_log2, a.scale_log2);
    const bool wide = rows_wide(dk, a.dim) && rows_wide(dv, a.dim);
    DkvItem upcoming = dkv_item(a, cta, sink_items, lane);
    for (int i = 0, item = cta; item < items && ok; item = at(++i)) {
      const DkvItem w = upcoming;
      const int steps = group * w.nq, row0 = w.t.p0 + (row & ~31), j = w.t.p0 + row;
      // threads 0-127 bring nlse2 of a query tile, threads 128-255 ndelta. (Rows past the sample's end get zeros:
      // their rows of Q and dO are zero too, and nothing comes of their weights.)
      auto bring = [&](uint32_t to_step, int head, int tile) {
        if (warp < 8) {
          const int i = tile * kAttnTile + row;
          const bool on = i < w.t.len;
          copy4(smem_u32(stats + (to_step & 1) * 256 + threadIdx.x),
                (warp < 4 ? a.nlse2 : a.ndelta) + (on ? (int64_t)head * a.n + w.t.b + i : 0), on);
        }
        // every thread arrives, those without a copy too: a warp that is behind then holds the phase after its own
        copies_arrive(stat_full);
      };
      int head = w.kv * group, tile = w.q_lo;  // of the step
      if (steps) bring(step, head, tile);
      for (int n = 0; n < steps && ok; ++n, ++step) {
        const int q0 = tile * kAttnTile;
        if (++tile == w.q_lo + w.nq) tile = w.q_lo, ++head;
        const float* st = stats + (step & 1) * 256 + 32 * blk;
        // (the second buffer of S^T lies behind dK)
        const uint32_t slot = step % NS, ts = tg - 128u + 384u * slot;
        ok = mbar_wait_warp(stat_full, step & 1, abort_flag, err, kErrDkv) &&
             mbar_wait_warp(s_full + 8 * slot, step / NS & 1, abort_flag, err, kErrDkv);
        if (!ok) break;
        tc_fence_after();
        uint32_t p[32], g[32], r[16];
        tmem_ld_32x32b_x32(ts, p);
        tmem_ld_wait();
        bool seen = true;
        if (!tile_full(a, q0, w.t.p0)) {
          // query qb + col sees key j for col >= from and col < to
          const int qb = q0 + 32 * blk, from = j - qb;
          const int to = j < a.sinks ? 32 : (int)min((int64_t)from + a.window, (int64_t)32);
          const uint32_t m = bit_range(from, to);
          seen = __any_sync(0xffffffffu, m != 0u);
          if (seen && !__all_sync(0xffffffffu, m == 0xffffffffu)) mask_block(p, m);
        }
        if (seen) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const ulonglong2 l = *reinterpret_cast<const ulonglong2*>(st + e);
            float u, v;
            unpack2(fma2(pack2(p[e], p[e + 1]), scale2, l.x), u, v);
            p[e] = __float_as_uint(ex2(u));
            p[e + 1] = __float_as_uint(ex2(v));
            unpack2(fma2(pack2(p[e + 2], p[e + 3]), scale2, l.y), u, v);
            p[e + 2] = __float_as_uint(ex2(u));
            p[e + 3] = __float_as_uint(ex2(v));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) p[e] = 0u;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) r[e] = op_pack_bf16(__uint_as_float(p[2 * e]), __uint_as_float(p[2 * e + 1]));
        tmem_st_32x32b_x16(ts, r);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + 8 * slot);
        ok = mbar_wait_warp(dp_full, step & 1, abort_flag, err, kErrDkv);
        if (!ok) break;
        tc_fence_after();
        // every warp is through with the step before, whose buffer this is: dP^T was formed after their dS^T
        if (n + 1 < steps) bring(step + 1, head, tile);
        tmem_ld_32x32b_x32(tg, g);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const ulonglong2 d = *reinterpret_cast<const ulonglong2*>(st + 128 + e);
          float u, v;
          unpack2(mul2(pack2(p[e], p[e + 1]), add2(pack2(g[e], g[e + 1]), d.x)), u, v);
          r[e / 2] = op_pack_bf16(u, v);
          unpack2(mul2(pack2(p[e + 2], p[e + 3]), add2(pack2(g[e + 2], g[e + 3]), d.y)), u, v);
          r[e / 2 + 1] = op_pack_bf16(u, v);
        }
        tmem_st_32x32b_x16(tg, r);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ds_full);
      }
      if (!ok) break;
      if (at(i + 1) < items) upcoming = dkv_item(a, at(i + 1), sink_items, lane);
      if (steps) {
        ok = mbar_wait_warp(done, done_ph, abort_flag, err, kErrDkv);
        if (!ok) break;
        done_ph ^= 1;
        tc_fence_after();
      }
      // warps 0-7 store dV, warps 8-15 dK, half of the columns to each four; the sink keys' rows go to their partial
      // slot in fp32
      const int which = blk >> 1, c0 = (blk & 1) * (DP / 2), c1 = c0 + DP / 2;
      const float f = which ? a.scale : 1.f;
      const uint32_t acc = tmem + lanes + 256u + DP * which;
      const int sinks = w.slot >= 0 ? a.sinks : 0;
      if (row0 < sinks) {
        float* pp = partial + ((w.slot * a.kv_heads + w.kv) * 2 + which) * (int64_t)a.sinks * a.dim + (int64_t)j * a.dim;
        const bool mine = j < sinks && j < w.t.len && w.slot < partial_slots;
#pragma unroll 1
        for (int c = c0; c < c1; c += 32) {
          uint32_t o[32];
          if (steps) {
            tmem_ld_32x32b_x32(acc + c, o);
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
                store8(pp + c + e, x);
              }
            }
          }
        }
      }
      cur.skip(2 * steps);
      if (w.staged) {
        const Cursor<SM::SLOTS> mine = which ? cur.next() : cur;
        ok = mbar_wait_warp(mine.full(ring), mine.phase, abort_flag, err, kErrDkv);
        if (!ok) break;
        stage_row(acc, c0, c1, f, false, mine.data(ring), row);
        __syncwarp();
        if (lane == 0) mbar_arrive(staged + 8 * mine.slot);
        cur.skip(2);
      } else if (!w.sink_only)
        store_row(acc, c0, c1, f, steps == 0, (which ? dk : dv) + (((int64_t)w.t.b + j) * a.kv_heads + w.kv) * a.dim,
                  j < w.t.len && j >= sinks, a.dim, wide);
      if (w.slot >= 0) {
        // the last of a sample's items to come here adds up its sink keys' rows
        __threadfence();
        __syncwarp();
        if (lane == 0) mbar_arrive(summed);
        if (warp == 0) {
          ok = mbar_wait_warp(summed, slot_ph, abort_flag, err, kErrDkv);
          if (ok && lane == 0) {
            const int all = 1 + sink_chunks(a, w.t.len, true);
            const int before = atomicAdd(arrived + (int64_t)w.t.sample * a.kv_heads + w.kv, 1);
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(last_word), "r"((int)(before + 1 == all)) : "memory");
            mbar_arrive(told);
          }
        }
        ok = ok && mbar_wait_warp(told, slot_ph, abort_flag, err, kErrDkv);
        if (!ok) break;
        slot_ph ^= 1;
        int last;
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(last) : "r"(last_word) : "memory");
        if (last) {
          __threadfence();
          sum_sinks(a, w.t, w.kv, partial, partial_slots, dk, dv, lane);
        }
      }
      tc_fence_before();
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // (after a wait that ran out)
  } else if (warp == kTma) {
    Cursor<SM::SLOTS> cur;
    uint32_t loads = 0, raw_phase = 0;
    for (int i = 0, item = cta; item < items && ok; item = at(++i)) {
      const DkvItem w = dkv_item(a, item, sink_items, lane);
      if (lane == 0) {
        const int steps = group * w.nq;
        int head = w.kv * group, tile = w.q_lo;
        for (int n = 0; n < steps && ok; ++n) {
          const int at = tile * kAttnTile;
          for (int x = 0; x < 2 && ok; ++x) {
            if (n == 0) {
              // K before the first queries, V before the first output gradients
              const uint32_t b = loads % KV, full = (x ? v_full : k_full) + 8 * b;
              ok = mbar_wait_in((x ? v_empty : k_empty) + 8 * b, (loads / KV & 1) ^ 1, abort_flag, err, kErrDkv);
              if (!ok) break;
              mbar_expect_tx(full, SM::TILE);
              load_tile<DP>(base + (x * KV + b) * SM::TILE, x ? &tmV : &tmK, w.t.b + w.t.p0, w.kv, full);
            }
            ok = mbar_wait_in(cur.empty(ring), cur.phase ^ 1, abort_flag, err, kErrDkv);
            if (!ok) break;
            fill_slot<DP>(ring, cur, x ? &tmDO : &tmQ, w.t.b + at, head, w.t.len - at, raw_phase);
            cur.advance();
          }
          if (++tile == w.q_lo + w.nq) tile = w.q_lo, ++head;
        }
        if (steps) ++loads;
        for (int x = 0; w.staged && x < 2 && ok; ++x) {
          ok = mbar_wait_in(cur.empty(ring), cur.phase ^ 1, abort_flag, err, kErrDkv);
          if (!ok) break;
          mbar_arrive(cur.full(ring));
          cur.advance();
        }
      }
      ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
    }
    if (lane == 0) {
      drain_ring(ring, cur, raw_phase);
      for (uint32_t i = loads > KV ? loads - KV : 0; i < loads; ++i) {
        drain_wait(k_full + 8 * (i % KV), i / KV & 1);
        drain_wait(v_full + 8 * (i % KV), i / KV & 1);
      }
    }
    __syncwarp();
  } else if (warp < kMmaB + 1) {
    // x = 0: S^T of Q, then dV += P^T dO; x = 1: dP^T of dO, then dK += dS^T Q
    const int x = warp_uniform(warp - kMmaA);
    Cursor<SM::SLOTS> cur;  // a step's query tile; its output gradients follow it
    uint32_t nth = 0, turns = 0;        // items with steps, steps whose first product has been reached
    const uint32_t tm = warp_uniform(tmem), to = tm + 256u + (uint32_t)DP * x;
    DkvItem upcoming = dkv_item(a, cta, sink_items, lane);
    for (int i = 0, item = cta; item < items && ok; item = at(++i)) {
      const int steps = warp_uniform(group * upcoming.nq), out = warp_uniform((int)upcoming.staged);
      if (at(i + 1) < items) upcoming = dkv_item(a, at(i + 1), sink_items, lane);
      if (steps == 0) continue;
      const uint32_t b = nth % KV, kt = base + (x * KV + b) * SM::TILE;
      ok = mbar_wait_warp((x ? v_full : k_full) + 8 * b, nth / KV & 1, abort_flag, err, kErrDkv);
      ++nth;
      Cursor<SM::SLOTS> other;  // the second product's right-hand tile, of the step before
      // S^T, or dP^T, of step n, which is the `turns`th of all
      auto first = [&](int n) {
        const Cursor<SM::SLOTS> c = x ? cur.next() : cur;
        const uint32_t slot = x ? 0 : turns % NS;
        if (!mbar_wait_warp(c.full(ring), c.phase, abort_flag, err, kErrDkv)) return false;
        tc_fence_after();
        mma_abt<DP>(tm + (x ? 128u : 384u * slot), kt, c.data(ring));
        umma_commit_warp(x ? dp_full : s_full + 8 * slot);
        if (x == 0 && lane == 0) mbar_arrive(turn + 8 * (turns & 3));
        umma_commit_warp(c.empty(ring));
        if (n == steps - 1) umma_commit_warp((x ? v_empty : k_empty) + 8 * b);
        return true;
      };
      // dV, or dK, of the `at`th step
      auto second = [&](bool add, uint32_t at) {
        const uint32_t slot = x ? 0 : at % NS;
        if (!(mbar_wait_warp(other.full(ring), other.phase, abort_flag, err, kErrDkv) &&
              mbar_wait_warp(x ? ds_full : p_full + 8 * slot, (x ? at : at / NS) & 1, abort_flag, err, kErrDkv)))
          return false;
        tc_fence_after();
        mma_ab<DP, 32>(to, tm + (x ? 128u : 384u * slot), other.data(ring), add);
        umma_commit_warp(other.empty(ring));
        return true;
      };
      // step n issues the second product of step n - 1 and the first of step n, S^T ahead of dV where it has a buffer
      for (int n = 0; n <= steps && ok; ++n) {
        // dK behind the next step's S^T: the threads' next work waits for that
        if (x == 1 && n < steps)
          if (!(ok = mbar_wait_warp(turn + 8 * (turns & 3), turns >> 2 & 1, abort_flag, err, kErrDkv))) break;
        const bool ahead = NS == 2 && x == 0;
        if (ahead && n < steps && !(ok = first(n))) break;
        if (n > 0 && !(ok = second(n > 1, turns - 1))) break;
        if (n == steps) break;
        if (!ahead && !(ok = first(n))) break;
        other = x ? cur : cur.next();
        cur.skip(2);
        ++turns;
      }
      if (ok) umma_commit_warp(done);
      if (out) cur.skip(2);
    }
    umma_commit_warp(drain + 8 * x);
    if (lane == 0) drain_wait(drain + 8 * x, 0);
    __syncwarp();
  } else {
    Cursor<SM::SLOTS> cur;
    uint32_t raw_phase = 0, staged_phase = 0;
    for (int i = 0, item = cta; item < items && ok; item = at(++i)) {
      const DkvItem w = dkv_item(a, item, sink_items, lane);
      const int valid = w.t.len - (w.q_lo + w.nq - 1) * kAttnTile;  // of a head's last query tile
      if (w.nq > 0)
        for (int h = 0; h < group; ++h) {
          cur.skip(2 * w.nq - 2);
          for (int x = 0; x < 2; ++x) {
            if (valid < kAttnTile && ok)
              ok = clear_slot<DP>(ring, cur, valid, raw_phase, lane, abort_flag, err, kErrDkv);
            cur.advance();
          }
        }
      for (int x = 0; w.staged && x < 2 && ok; ++x) {
        ok = store_slot<DP>(ring, cur, staged, staged_phase, x ? &tmDK : &tmDV, w.t.b + w.t.p0, w.kv, 2, lane, abort_flag,
                            err, kErrDkv);
        cur.advance();
      }
    }
  }
}

// dK and dV, then dQ: one persistent CTA per SM runs its items of the one and then
// its items of the other, so that no SM waits in between for the slowest.
template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
    window_grad_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const __grid_constant__ CUtensorMap tmDO, const __grid_constant__ CUtensorMap tmDQ,
                       const __grid_constant__ CUtensorMap tmDK, const __grid_constant__ CUtensorMap tmDV,
                       __nv_bfloat16* __restrict__ dq,
                       __nv_bfloat16* __restrict__ dk, __nv_bfloat16* __restrict__ dv, float* __restrict__ partial,
                       int64_t partial_slots, int* __restrict__ counter, int* __restrict__ err) {
  using SM = GradSmem<DP>;
  extern __shared__ __align__(1024) uint8_t smem[];
  // words after the barriers: the TMEM base, the abort flag, the posted numbers
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SM::BARS + SM::NBARS * 8);
  volatile int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  const uint32_t numbers = smem_u32(tmem_slot + 2);
  float* stats = reinterpret_cast<float*>(smem + SM::STATS);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = smem_u32(smem), bars = base + SM::BARS, bars2 = bars + DkvBarriers<DP>::COUNT * 8;
  static_assert(DkvBarriers<DP>::COUNT + DqBarriers<DP>::COUNT == SM::NBARS, "barriers");
  if (base & 1023u) {  // the swizzle's phase is that of the address
    if (threadIdx.x == 0) atomicCAS(err, 0, kErrAlign);
    return;
  }
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    dkv_part<DP, false>(a, tmQ, tmK, tmV, tmDO, tmDK, tmDV, dk, dv, partial, partial_slots, err, abort_flag, stats, nullptr, 0, base, bars, 0, 0, 1, 0, 0,
                 true);
    dq_part<DP, false>(a, tmQ, tmK, tmV, tmDO, tmDQ, dq, err, abort_flag, base, bars2, 0, 0, nullptr, true);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaA) tmem_alloc<1>(smem_u32(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch();
  pdl_wait();
  const int cta = blockIdx.x, ctas = gridDim.x;
  const int sink_items =
      a.kv_heads * count_units(a, lane, [&](int len, bool live) { return sink_chunks(a, len, live); });
  const int items = sink_items +
                    a.kv_heads * count_units(a, lane, [](int len, bool) { return (len + kAttnTile - 1) / kAttnTile; });
  // (the registers are given by one instruction for all four warps of a group)
  if (warp < kMathWarps) {
    regs_up<kMathRegs>();
    dkv_part<DP, true>(a, tmQ, tmK, tmV, tmDO, tmDK, tmDV, dk, dv, partial, partial_slots, err, abort_flag, stats, counter + 1, numbers + 4 * kPosts, base, bars, tmem,
                       cta, ctas, sink_items, items, false);
    dq_part<DP, true>(a, tmQ, tmK, tmV, tmDO, tmDQ, dq, err, abort_flag, base, bars2, tmem, numbers, counter, false);
  } else {
    regs_down<kOtherRegs>();
    dkv_part<DP, false>(a, tmQ, tmK, tmV, tmDO, tmDK, tmDV, dk, dv, partial, partial_slots, err, abort_flag, stats, counter + 1, numbers + 4 * kPosts, base, bars,
                        tmem, cta, ctas, sink_items, items, false);
    dq_part<DP, false>(a, tmQ, tmK, tmV, tmDO, tmDQ, dq, err, abort_flag, base, bars2, tmem, numbers, counter, false);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaA) tmem_dealloc<1>(tmem, 512);
}

template <int DP>
cudaError_t run_backward(const AttnArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                         const CUtensorMap& dout, const AttnGrad& g, int* err, int sms, cudaStream_t st) {
  const int64_t tiles = attn_max_tiles(a.n, a.n_seqs, kAttnTile), most = tiles * a.heads;
  const cudaError_t e = op_smem_limit<window_grad_kernel<DP>>((int)GradSmem<DP>::BYTES);
  if (e != cudaSuccess) return e;
  return op_launch(window_grad_kernel<DP>, dim3((unsigned)(most < sms ? most : sms)), dim3(kThreads),
                   GradSmem<DP>::BYTES, st, 1, a, q, k, v, dout, g.tm_dq, g.tm_dk, g.tm_dv, g.dq, g.dk, g.dv, g.partial, g.partial_slots, g.counter, err);
}

}  // namespace

cudaError_t attn_backward(AttnArgs a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                          const CUtensorMap& dout, const AttnGrad& g, int* err, int sms, cudaStream_t st) {
  const int64_t rows = ((int64_t)a.n * a.heads + 15) / 16, most = (int64_t)sms * 8;
  cudaError_t e = op_launch(window_stats_kernel, dim3((unsigned)(rows < most ? rows : most)), dim3(256), 0, st, 1, a,
                            g.dout, g.do_ts, g.do_hs, g.out, g.o_ts, g.o_hs, g.lse, g.nlse2, g.ndelta, g.counter);
  if (e != cudaSuccess) return e;
  a.nlse2 = g.nlse2;
  a.ndelta = g.ndelta;
  return a.dim > 64 ? run_backward<128>(a, q, k, v, dout, g, err, sms, st)
                    : run_backward<64>(a, q, k, v, dout, g, err, sms, st);
}

}  // namespace ma
