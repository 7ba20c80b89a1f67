// Causal attention with a sliding window and sink tokens, forward pass, and
// the C entry points of the operator.
//
// One pass over the keys with the running maximum m and sum l of the softmax:
//   S = Q K^T,  P = exp2(c S - m),  l += rowsum(P),  O += P V,  c = scale log2(e)
// and out = O / l, lse = (m + log2 l) ln 2.
//
// window_forward_kernel (one persistent CTA per SM, 384 threads) works on two
// tiles of 128 queries that share their keys and values: the same queries of
// two heads that read one key head, or, where heads do not pair, two
// neighbouring tiles of one head.
//   warps 0-3, 4-7  softmax of the first and of the second tile, a thread to a
//                   query: S from TMEM, P (bf16) back to TMEM over S;
//   warp 8          TMA: the two query tiles, then key and value tiles into a
//                   ring;
//   warps 9, 10     tcgen05.mma of the first and of the second tile: S = Q K^T
//                   from shared memory, O += P V with P from TMEM. One tile's
//                   products run while the other's softmax does. A warp issues
//                   a product in 400 cycles and spends as much on the barriers
//                   around it, a product runs for 520: one warp for both tiles
//                   left the tensor core idle half the time (174 us for 16360
//                   tokens of 16 heads of 128, window 1024);
//   warp 11         clears the rows of a sample's last value tile that belong to
//                   other samples, and stores the finished tiles.
// TMEM: S0 | S1 | O0 | O1, 128 columns each (heads of up to 64 leave half of each O
// idle).
//
// Finished tiles leave through two positions of the ring and TMA (see stage_row),
// tiles with rows of other samples from the threads' registers.
//
// Bound by the chain of a step: S, its softmax in one thread a row, P V, and S of the
// next keys, which takes P's place. A step of both tiles takes 3500 cycles, of which
// the four products fill 2048 and a softmax takes 1950 (maximum 380, exponentials,
// sum and rounding 1060, TMEM and barriers the rest); it is bound by issue, so that
// exponentials as polynomials beside the special-function unit cost 12 to 20 %.
// 16384 tokens of 16 heads of 128 over 8 key heads, all keys visible: 772 us, 1425
// TFLOP/s (0.76 of the measured bf16 peak). Window 1024 and four sinks: 73 us for
// 8192 tokens; 139 us for 16360 in packed samples, 800 TFLOP/s counting visible
// pairs, nine tiles being formed for eight tiles' worth of keys. 50 tokens of 16 heads
// of 64: 6.3 us, the latency of one step and its set-up.
//
// Heads of other widths run at the next of 64 and 128, the columns past their own
// zero: 8192 tokens of 16 heads over 8 with window 1024 and four sinks take 65 us of
// 32 or 64, 72 to 74 of 72, 80, 96 or 128.
//
// O is rescaled only when a row's maximum has grown by more than 2^8 since it
// was last taken as m: P then stays below 2^8 and sums in fp32 lose nothing.
#include "window_attention.cuh"

namespace ma {
namespace {

constexpr int kThreads = 384;
// of the 168 registers a thread is launched with: 8 softmax warps and 4 others, 8 * 208 + 4 * 80 <= 12 * 168
constexpr int kSoftmaxRegs = 208, kOtherRegs = 80;
constexpr int kErrForward = 0x201, kErrAlign = 0x204;

template <int DP>
struct FwdSmem {
  static constexpr uint32_t TILE = kAttnTile * DP * 2;
  static constexpr int SLOTS = DP == 128 ? 4 : 8;
  static constexpr uint32_t RING = 2 * TILE;
  static constexpr uint32_t BARS = RING + SLOTS * TILE;
  // full[SLOTS], empty[SLOTS], raw[SLOTS], q full, q empty, s full[2], p full[2], o full[2], drain[2], turn[SLOTS / 2],
  // staged[SLOTS]
  static constexpr int NBARS = 4 * SLOTS + 10 + SLOTS / 2;
  static constexpr uint32_t BYTES = BARS + NBARS * 8 + 16;
  static_assert(BYTES <= 232448, "shared memory per CTA");
};

// The key tiles two query tiles meet, as one list: tile 0 for the sinks where
// no window reaches it, then lo .. hi. Query tile s uses the steps a[s] .. b[s]
// of it in full, and step 0 for the sinks where z[s] (written out, a0 to z1, so
// that they stay in registers).
struct PairTiles {
  int lo, steps, sink;
  int a0, b0, a1, b1;
  bool z0, z1;
  __device__ __forceinline__ int tile(int n) const { return sink && n == 0 ? 0 : lo + n - sink; }
  __device__ __forceinline__ bool whole(int s, int n) const { return n >= (s ? a1 : a0) && n <= (s ? b1 : b0); }
  __device__ __forceinline__ bool use(int s, int n) const { return whole(s, n) || (n == 0 && (s ? z1 : z0)); }
};
__device__ __forceinline__ PairTiles pair_tiles(const AttnArgs& a, const SampleTile& t, int step) {
  PairTiles p;
  const KeyTiles r0 = key_tiles(a, t.live, t.len, t.p0), r1 = key_tiles(a, t.live, t.len, t.p0 + step);
  p.sink = r0.sink ? 1 : 0;
  p.lo = r0.lo;
  p.steps = p.sink + max(0, max(r0.hi, r1.hi) - p.lo + 1);
  const bool w0 = r0.hi >= r0.lo, w1 = r1.hi >= r1.lo;
  p.a0 = w0 ? p.sink : 1;
  p.b0 = w0 ? p.sink + r0.hi - p.lo : 0;
  p.a1 = w1 ? p.sink + r1.lo - p.lo : 1;
  p.b1 = w1 ? p.sink + r1.hi - p.lo : 0;
  p.z0 = r0.sink;
  p.z1 = r1.sink;
  return p;
}

struct FwdItem {
  SampleTile t;
  PairTiles k;
  int head0, head1, kv;
  bool staged;  // both tiles leave through the ring, two positions after the last values
};

// Work item: a pair of query tiles. by_head: of two heads, which meet the same keys,
// else of one head, whose two tiles meet one key tile more (8192 tokens of 16 heads,
// window 1024: 73 us over 8 key heads, 79 us over 16).
//
// FRO: the last tiles come first, which meet the most keys, and the CTAs take them to
// and fro: every second round of items (the last one may be short) goes round the
// other way.
template <bool FRO>
__device__ __forceinline__ FwdItem fwd_item(const AttnArgs& a, int nth, int items, int units, int lane) {
  int item = nth;
  if constexpr (FRO) {
    const int ctas = gridDim.x, turn = nth / ctas, at = nth - turn * ctas, round = min(ctas, items - turn * ctas);
    item = items - 1 - (turn * ctas + (turn & 1 ? round - 1 - at : at));
  }
  const bool by_head = units * 2 == a.heads;
  const int rows = by_head ? kAttnTile : 2 * kAttnTile;
  const int tile = item / units, u = item - tile * units;
  FwdItem w;
  w.t = find_unit(a, tile, lane, [rows](int len, bool) { return (len + rows - 1) / rows; });
  w.t.p0 = w.t.index * rows;
  w.k = pair_tiles(a, w.t, by_head ? 0 : kAttnTile);
  w.head0 = by_head ? 2 * u : u;
  w.head1 = by_head ? 2 * u + 1 : u;
  w.kv = w.head0 / (a.heads / a.kv_heads);
  w.staged = w.k.steps > 0 && w.t.p0 + rows <= w.t.len;
  return w;
}

template <int DP, bool FRO>
__global__ void __launch_bounds__(kThreads, 1)
    window_forward_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap tmQ,
                          const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                          const __grid_constant__ CUtensorMap tmO, __nv_bfloat16* __restrict__ out, float* __restrict__ lse, int* __restrict__ err, int units) {
  using SM = FwdSmem<DP>;
  extern __shared__ __align__(1024) uint8_t smem[];
  // two words after the barriers: the TMEM base and the abort flag
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SM::BARS + SM::NBARS * 8);
  volatile int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = smem_u32(smem), bars = base + SM::BARS;
  Ring<SM::SLOTS> ring{base + SM::RING, bars, bars + SM::SLOTS * 8, bars + SM::SLOTS * 16, SM::TILE};
  const uint32_t q_full = bars + 3 * SM::SLOTS * 8, q_empty = q_full + 8, s_full = q_full + 16, p_full = q_full + 32,
                 o_full = q_full + 48, drain = q_full + 64, turn = q_full + 80, staged = turn + 4 * SM::SLOTS;
  if (base & 1023u) {  // the swizzle's phase is that of the address
    if (threadIdx.x == 0) atomicCAS(err, 0, kErrAlign);
    return;
  }
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    ring.init(2);
    mbar_init(q_full, 1), mbar_init(q_empty, 2), mbar_init(drain, 1), mbar_init(drain + 8, 1);
    for (int i = 0; i < SM::SLOTS / 2; ++i) mbar_init(turn + 8 * i, 1);
    for (int i = 0; i < SM::SLOTS; ++i) mbar_init(staged + 8 * i, 4);
    for (int s = 0; s < 2; ++s) mbar_init(s_full + 8 * s, 1), mbar_init(p_full + 8 * s, 128), mbar_init(o_full + 8 * s, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 9) tmem_alloc<1>(smem_u32(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch();
  pdl_wait();
  const int rows = units * 2 == a.heads ? kAttnTile : 2 * kAttnTile;
  const int items = units * count_units(a, lane, [rows](int len, bool) { return (len + rows - 1) / rows; });
  bool ok = true;
  // (one instruction for all four warps of a group)
  if (warp < 8)
    regs_up<kSoftmaxRegs>();
  else
    regs_down<kOtherRegs>();

  if (warp < 8) {
    // ---- softmax ----
    const int s = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + 128u * s + lanes, to = tmem + 256u + 128u * s + lanes;
    const bool wide = rows_wide(out, a.dim);
    uint32_t s_ph = 0, o_ph = 0;
    Cursor<SM::SLOTS> cur;
    FwdItem next = fwd_item<FRO>(a, blockIdx.x, items, units, lane);
    for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
      const FwdItem w = next;
      const int p0 = w.t.p0 + (w.head0 == w.head1 ? s * kAttnTile : 0), i = p0 + row, row0 = p0 + (row & ~31);
      float m = -INFINITY, l = 0.f;
      bool any = false;
      for (int n = 0; n < w.k.steps && ok; ++n) {
        if (!w.k.use(s, n)) continue;
        const int k0 = w.k.tile(n) * kAttnTile;
        ok = mbar_wait_warp(s_full + 8 * s, s_ph, abort_flag, err, kErrForward);
        if (!ok) break;
        s_ph ^= 1;
        tc_fence_after();
        Blocks seen = kAllBlocks;
        if (!tile_full(a, p0, k0)) {
          // key k0 + col is visible for col < end and (col >= first or col < sink); past the sinks' columns of
          // a tile that is there for them alone no score has been formed
          const int cols = w.k.whole(s, n) ? kAttnTile : sink_columns(a);
          const int end = min(i - k0 + 1, cols), first = i - a.window + 1 - k0, sink = min(a.sinks - k0, end);
          seen = key_blocks(a, row0, k0, cols, 4);
          mask_tile(ts, seen,
                    [&](int c) { return bit_range(first - 32 * c, end - 32 * c) | bit_range(0, sink - 32 * c); });
        }
        uint32_t v[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(ts + 32 * c, v[c]);
        tmem_ld_wait();
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c >= seen.lo && c < seen.hi) {
#pragma unroll
            for (int j = 0; j < 32; ++j) mx[j & 3] = fmaxf(mx[j & 3], __uint_as_float(v[c][j]));
          }
        const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
        const bool grow = mt > m + 8.f;
        if (__any_sync(0xffffffffu, grow)) {
          const float f = grow ? ex2(m - mt) : 1.f;
          if (grow) m = mt;
          l *= f;
          if (any) {
#pragma unroll 1
            for (int c = 0; c < DP; c += 32) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(to + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_st_32x32b_x32(to + c, o);
            }
          }
        }
        any = true;
        const float shift = m == -INFINITY ? 0.f : -m;
        const uint64_t shift2 = pack2(shift, shift), scale2 = pack2(a.scale_log2, a.scale_log2);
        uint64_t sum0 = 0, sum1 = 0;  // two sums each
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t p[16];
          if (c >= seen.lo && c < seen.hi) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              float x, y;
              unpack2(fma2(pack2(v[c][2 * j], v[c][2 * j + 1]), scale2, shift2), x, y);
              x = ex2(x);
              y = ex2(y);
              if (j & 1)
                sum1 = add2(sum1, pack2(x, y));
              else
                sum0 = add2(sum0, pack2(x, y));
              p[j] = op_pack_bf16(x, y);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) p[j] = 0u;
          }
          tmem_st_32x32b_x16(ts + 16 * c, p);
        }
        float l0, l1;
        unpack2(add2(sum0, sum1), l0, l1);
        l += l0 + l1;
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(p_full + 8 * s);
      }
      if (!ok) break;
      if (item + (int)gridDim.x < items) next = fwd_item<FRO>(a, item + gridDim.x, items, units, lane);
      if (any) {
        ok = mbar_wait_warp(o_full + 8 * s, o_ph, abort_flag, err, kErrForward);
        if (!ok) break;
        o_ph ^= 1;
        tc_fence_after();
      }
      // a query that saw no key: zeros and -infinity
      const float inv = any ? 1.f / l : 0.f;
      const int head = s ? w.head1 : w.head0;
      const int64_t t = (int64_t)w.t.b + i;
      cur.skip(2 * w.k.steps);
      if (w.staged) {
        const Cursor<SM::SLOTS> mine = s ? cur.next() : cur;
        ok = mbar_wait_warp(mine.full(ring), mine.phase, abort_flag, err, kErrForward);
        if (!ok) break;
        stage_row(to, 0, DP, inv, !any, mine.data(ring), row);
        __syncwarp();
        if (lane == 0) mbar_arrive(staged + 8 * mine.slot);
        cur.skip(2);
      } else {
        store_row(to, 0, DP, inv, !any, out + (t * a.heads + head) * a.dim, i < w.t.len, a.dim, wide);
      }
      if (i < w.t.len)
        lse[(int64_t)head * a.n + t] = any ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
      tc_fence_before();
    }
  } else if (warp == 8) {
    // ---- TMA ----
    Cursor<SM::SLOTS> cur;
    uint32_t loads = 0, raw_phase = 0;
    for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
      const FwdItem w = fwd_item<FRO>(a, item, items, units, lane);
      if (lane == 0) {
        for (int n = 0; n < w.k.steps && ok; ++n) {
          const int at = w.k.tile(n) * kAttnTile;
          for (int kv = 0; kv < 2 && ok; ++kv) {
            ok = mbar_wait_in(cur.empty(ring), cur.phase ^ 1, abort_flag, err, kErrForward);
            if (!ok) break;
            // value rows of another sample are cleared; keys of another are masked in S
            fill_slot<DP>(ring, cur, kv ? &tmV : &tmK, w.t.b + at, w.kv, kv ? w.t.len - at : kAttnTile, raw_phase);
            cur.advance();
            if (n == 0 && kv == 0) {
              // the queries after the first keys: their buffer is free once the item before has formed its last S
              ok = mbar_wait_in(q_empty, (loads & 1) ^ 1, abort_flag, err, kErrForward);
              if (!ok) break;
              ++loads;
              mbar_expect_tx(q_full, 2 * SM::TILE);
              load_tile<DP>(base, &tmQ, w.t.b + w.t.p0, w.head0, q_full);
              load_tile<DP>(base + SM::TILE, &tmQ, w.t.b + w.t.p0 + (w.head0 == w.head1 ? kAttnTile : 0), w.head1, q_full);
            }
          }
        }
        for (int s = 0; w.staged && s < 2 && ok; ++s) {
          ok = mbar_wait_in(cur.empty(ring), cur.phase ^ 1, abort_flag, err, kErrForward);
          if (!ok) break;
          mbar_arrive(cur.full(ring));
          cur.advance();
        }
      }
      ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
    }
    if (lane == 0) {
      // every copy has landed before the CTA leaves
      drain_ring(ring, cur, raw_phase);
      if (loads) drain_wait(q_full, (loads - 1) & 1);
    }
    __syncwarp();
  } else if (warp < 11) {
    // ---- MMA ----
    Cursor<SM::SLOTS> cur;
    uint32_t q_ph = 0, p_ph = 0, turns = 0;
    const int s = warp_uniform(warp - 9), few = sink_columns(a);
    const uint32_t ts = warp_uniform(tmem) + 128u * s, to = ts + 256u, qt = base + s * SM::TILE;
    const uint32_t sf = s_full + 8 * s, pf = p_full + 8 * s, of = o_full + 8 * s;
    FwdItem next = fwd_item<FRO>(a, blockIdx.x, items, units, lane);
    for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
      const int steps = warp_uniform(next.k.steps), first = warp_uniform(s ? next.k.a1 : next.k.a0),
                last = warp_uniform(s ? next.k.b1 : next.k.b0), sink = warp_uniform((int)(s ? next.k.z1 : next.k.z0)), staged_out = warp_uniform((int)next.staged);
      if (steps == 0 || !(ok = mbar_wait_warp(q_full, q_ph, abort_flag, err, kErrForward))) {
        if (item + (int)gridDim.x < items) next = fwd_item<FRO>(a, item + gridDim.x, items, units, lane);
        continue;
      }
      q_ph ^= 1;
      const int end = last >= first ? last : sink - 1;  // the last step that this tile uses
      bool pend = false, whole = false, begun = false;
      Cursor<SM::SLOTS> vc;  // the value tile of the step before
      // step n issues O += P V of tile n - 1 and S of tile n. Tiles that only the other warp uses are waited for
      // and released all the same: a slot's release counts both warps once for each of its fills.
      //
      // The second tile's products of a step are issued behind the first's. Issued freely they would run in turns,
      // both softmaxes would start when both S are there, and products and softmaxes would alternate instead of
      // overlapping (4000 cycles a step of both tiles instead of 2700).
      for (int n = 0; n <= steps; ++n) {
        // (the first tile's warp is never as many turns ahead as there are barriers: the slot of its keys would not
        // be free)
        const uint32_t my_turn = turn + 8 * (turns % (SM::SLOTS / 2)), turn_ph = turns / (SM::SLOTS / 2) & 1;
        if (n < steps && s == 1 && !(ok = mbar_wait_warp(my_turn, turn_ph, abort_flag, err, kErrForward))) break;
        if (n > 0) {
          if (!(ok = mbar_wait_warp(vc.full(ring), vc.phase, abort_flag, err, kErrForward))) break;
          if (pend) {
            if (!(ok = mbar_wait_warp(pf, p_ph, abort_flag, err, kErrForward))) break;
            p_ph ^= 1;
            tc_fence_after();
            if (whole)
              mma_ab<DP, 16>(to, ts, vc.data(ring), begun);
            else
              mma_ab_few<DP, 16>(to, ts, vc.data(ring), begun, few);
            if (n - 1 == end) umma_commit_warp(of);
            begun = true;
          }
          umma_commit_warp(vc.empty(ring));
        }
        if (n == steps) break;
        if (!(ok = mbar_wait_warp(cur.full(ring), cur.phase, abort_flag, err, kErrForward))) break;
        whole = n >= first && n <= last;
        pend = whole || (n == 0 && sink);
        if (pend) {
          tc_fence_after();
          mma_abt<DP>(ts, qt, cur.data(ring), whole ? kAttnTile : few);
          umma_commit_warp(sf);
        }
        if (s == 0 && lane == 0) mbar_arrive(my_turn);
        ++turns;
        umma_commit_warp(cur.empty(ring));
        if (n == steps - 1) umma_commit_warp(q_empty);
        cur.advance();
        vc = cur;
        cur.advance();
        if (n == 0 && item + (int)gridDim.x < items) next = fwd_item<FRO>(a, item + gridDim.x, items, units, lane);
      }
      if (staged_out) cur.skip(2);
    }
    umma_commit_warp(drain + 8 * s);
    if (lane == 0) drain_wait(drain + 8 * s, 0);
    __syncwarp();
  } else {
    // ---- rows of other samples, staged tiles ----
    Cursor<SM::SLOTS> cur;
    uint32_t raw_phase = 0, staged_phase = 0;
    for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
      const FwdItem w = fwd_item<FRO>(a, item, items, units, lane);
      if (w.k.steps == 0) continue;
      cur.skip(2 * w.k.steps - 1);
      const int valid = w.t.len - w.k.tile(w.k.steps - 1) * kAttnTile;  // only the last tile can be ragged
      if (valid < kAttnTile) ok = clear_slot<DP>(ring, cur, valid, raw_phase, lane, abort_flag, err, kErrForward);
      cur.advance();
      for (int s = 0; w.staged && s < 2 && ok; ++s) {
        ok = store_slot<DP>(ring, cur, staged, staged_phase, &tmO,
                            w.t.b + w.t.p0 + (s && w.head0 == w.head1 ? kAttnTile : 0), s ? w.head1 : w.head0, 2, lane,
                            abort_flag, err, kErrForward);
        cur.advance();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc<1>(tmem, 512);
}

template <int DP, bool FRO>
cudaError_t run_forward(const AttnArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                        const CUtensorMap& o, __nv_bfloat16* out, float* lse, int* err, int sms, cudaStream_t st) {
  const int group = a.heads / a.kv_heads;
  const int units = group % 2 == 0 ? a.heads / 2 : a.heads;
  const int rows = group % 2 == 0 ? kAttnTile : 2 * kAttnTile;
  const int64_t most = attn_max_tiles(a.n, a.cu ? a.n_seqs : 1, rows) * units;
  const cudaError_t e = op_smem_limit<window_forward_kernel<DP, FRO>>((int)FwdSmem<DP>::BYTES);
  if (e != cudaSuccess) return e;
  return op_launch(window_forward_kernel<DP, FRO>, dim3((unsigned)(most < sms ? most : sms)), dim3(kThreads),
                   FwdSmem<DP>::BYTES, st, 1, a, q, k, v, o, out, lse, err, units);
}

// ---- host ----
ma_status check_rows(const char* what, const void* p, int64_t dim, int64_t tokens, int64_t heads, int64_t ts,
                     int64_t hs) {
  if (!p) return op_fail(MA_ERR_ARG, "%s must not be NULL", what);
  if (!op_aligned(p, 16) || ts % 8 != 0 || hs % 8 != 0)
    return op_fail(MA_ERR_ALIGN, "%s: the pointer and the token and head strides must keep 16-byte alignment", what);
  if ((tokens > 1 && ts < dim) || (heads > 1 && hs < dim))
    return op_fail(MA_ERR_SHAPE, "%s: a token or head stride below head_dim", what);
  return MA_OK;
}

ma_status check_attn(const ma_window_attention* d) {
  if (!d) return op_fail(MA_ERR_ARG, "the description must not be NULL");
  if (d->n_tokens < 0 || d->n_tokens > (int64_t)1 << 30) return op_fail(MA_ERR_SHAPE, "n_tokens outside [0, 2^30]");
  if (d->n_heads < 1 || d->n_kv_heads < 1 || d->n_heads > 1024 || d->n_heads % d->n_kv_heads)
    return op_fail(MA_ERR_SHAPE, "%d query heads over %d key heads: no whole number of queries for each, or over 1024",
                   d->n_heads, d->n_kv_heads);
  if (d->head_dim < 8 || d->head_dim > 128 || d->head_dim % 8)
    return op_fail(MA_ERR_SHAPE, "head_dim %d is no multiple of 8 in [8, 128]", d->head_dim);
  if (d->window < 0) return op_fail(MA_ERR_ARG, "window must not be negative");
  if (d->sinks < 0 || d->sinks > kAttnTile) return op_fail(MA_ERR_ARG, "sinks outside [0, %d]", kAttnTile);
  if (!(d->scale > 0.0) || !(d->scale - d->scale == 0.0)) return op_fail(MA_ERR_ARG, "scale must be finite and positive");
  if (d->n_seqs < 0 || (d->cu_seqlens && d->n_seqs < 1)) return op_fail(MA_ERR_ARG, "cu_seqlens needs n_seqs >= 1");
  if (!op_aligned(d->cu_seqlens, 4)) return op_fail(MA_ERR_ALIGN, "cu_seqlens is not aligned to 4 bytes");
  if (((d->cu_seqlens ? d->n_seqs : 0) + d->n_tokens / kAttnTile + 2) * d->n_heads >= (int64_t)1 << 31)
    return op_fail(MA_ERR_SHAPE, "too many tokens, samples and heads");
  if (d->n_tokens == 0) return MA_OK;
  ma_status st = check_rows("q", d->q, d->head_dim, d->n_tokens, d->n_heads, d->q_token_stride, d->q_head_stride);
  if (st == MA_OK)
    st = check_rows("k", d->k, d->head_dim, d->n_tokens, d->n_kv_heads, d->k_token_stride, d->k_head_stride);
  if (st == MA_OK)
    st = check_rows("v", d->v, d->head_dim, d->n_tokens, d->n_kv_heads, d->v_token_stride, d->v_head_stride);
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
  a.n_seqs = d->cu_seqlens ? d->n_seqs : 1;
  a.scale = (float)d->scale;
  a.scale_log2 = (float)(d->scale * 1.4426950408889634);
  a.cu = d->cu_seqlens;
  return a;
}

struct Maps {
  CUtensorMap q, k, v, dout, out;
};

// The operator's own tensors lie without gaps.
bool dense_map(CUtensorMap* tm, const void* base, const ma_window_attention* d, int heads) {
  return attn_map(tm, base, d->head_dim, d->n_tokens, heads, (int64_t)heads * d->head_dim, d->head_dim);
}

bool maps_of(const ma_window_attention* d, Maps* m) {
  return attn_map(&m->q, d->q, d->head_dim, d->n_tokens, d->n_heads, d->q_token_stride, d->q_head_stride) &&
         attn_map(&m->k, d->k, d->head_dim, d->n_tokens, d->n_kv_heads, d->k_token_stride, d->k_head_stride) &&
         attn_map(&m->v, d->v, d->head_dim, d->n_tokens, d->n_kv_heads, d->v_token_stride, d->v_head_stride);
}

// Workspace of the gradient: lse2 and delta [head][token], then the partial
// sums of the sink keys, one slot for each sample and each chunk, then the counters.
struct GradSpace {
  int64_t stats, slots, slot_bytes, counter, bytes;
};
GradSpace grad_space(const ma_window_attention* d) {
  GradSpace g;
  const int64_t seqs = d->cu_seqlens ? d->n_seqs : 1;
  g.stats = ((int64_t)d->n_heads * d->n_tokens * 4 + 255) / 256 * 256;
  g.slots = d->sinks > 0 ? 2 * seqs + attn_max_tiles(d->n_tokens, seqs, kAttnTile) / kSinkChunk + 1 : 0;
  g.slot_bytes = (int64_t)d->n_kv_heads * 2 * d->sinks * d->head_dim * 4;
  g.counter = 2 * g.stats + g.slots * g.slot_bytes;
  g.bytes = g.counter + (1 + seqs * d->n_kv_heads) * 4 + 256;
  return g;
}

}  // namespace

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

bool attn_map(CUtensorMap* tm, const void* base, int dim, int64_t tokens, int64_t heads, int64_t token_stride,
              int64_t head_stride) {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  if (!fn) return false;
  // the stride of a single token or head is never used, but has to be a legal one
  if (tokens <= 1) token_stride = dim;
  if (heads <= 1) head_stride = dim;
  const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)tokens, (cuuint64_t)heads};
  const cuuint64_t strides[2] = {(cuuint64_t)token_stride * 2, (cuuint64_t)head_stride * 2};
  const cuuint32_t box[3] = {64, kAttnTile, 1}, estr[3] = {1, 1, 1};
  return fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t attn_forward(const AttnArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                         const CUtensorMap& o, __nv_bfloat16* out, float* lse, int* err, int sms, cudaStream_t st) {
  // Items that differ go longest first, to and fro: where the window is more than an eighth of all tokens (all keys of
  // 16384 visible: 772 us, in plain order 865; of 8192 208 and 249). Below they are alike, and in plain order only the
  // last keys of a tile have not been read before (window 1024 of 16384: 134 us, the other way 138; 16360 tokens in
  // eight samples 136 and 143). The samples' own lengths, which set how much the items differ, are not known here.
  // Beside the bound little hangs on it: windows of 2047 in plain order and 2049 to and fro take 223 and 219 us of one
  // sample of 16384 tokens, 145 and 147 of eight of 2048.
  const bool fro = (int64_t)a.window * 8 > a.n;
  if (a.dim > 64)
    return fro ? run_forward<128, true>(a, q, k, v, o, out, lse, err, sms, st)
               : run_forward<128, false>(a, q, k, v, o, out, lse, err, sms, st);
  return fro ? run_forward<64, true>(a, q, k, v, o, out, lse, err, sms, st)
             : run_forward<64, false>(a, q, k, v, o, out, lse, err, sms, st);
}

}  // namespace ma

using namespace ma;

extern "C" {

ma_status muon_adamw_window_attention(const ma_window_attention* d, void* out, float* lse, void* cuda_stream) {
  ma_status st = check_attn(d);
  if (st != MA_OK) return st;
  if (d->n_tokens > 0) {
    st = check_rows("out", out, 0, 1, 1, 0, 0);
    if (st != MA_OK) return st;
    if (!lse) return op_fail(MA_ERR_ARG, "lse must not be NULL");
    if (!op_aligned(lse, 4)) return op_fail(MA_ERR_ALIGN, "lse is not aligned to 4 bytes");
    int sms = 0, *err = nullptr;
    cudaError_t e = op_device(&sms, &err);
    if (e != cudaSuccess) return op_cuda(e, "device query");
    Maps m;
    if (!maps_of(d, &m) || !dense_map(&m.out, out, d, d->n_heads))
      return op_fail(MA_ERR_CUDA, "cuTensorMapEncodeTiled refused a tensor");
    e = attn_forward(args_of(d), m.q, m.k, m.v, m.out, static_cast<__nv_bfloat16*>(out), lse, err, sms,
                     static_cast<cudaStream_t>(cuda_stream));
    if (e != cudaSuccess) return op_cuda(e, "attention launch");
  }
  clear_last_error();
  return MA_OK;
}

ma_status muon_adamw_window_attention_backward_workspace(const ma_window_attention* d, int64_t* bytes) {
  if (!bytes) return op_fail(MA_ERR_ARG, "bytes must not be NULL");
  ma_status st = check_attn(d);
  if (st != MA_OK) return st;
  *bytes = grad_space(d).bytes;
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
    st = check_rows("dout", dout, d->head_dim, d->n_tokens, d->n_heads, dout_token_stride, dout_head_stride);
    // (a single token or head has no stride)
    const bool dense = d->out_token_stride == 0 && d->out_head_stride == 0;
    const int64_t o_ts = dense ? (int64_t)d->n_heads * d->head_dim : d->out_token_stride;
    const int64_t o_hs = dense ? d->head_dim : d->out_head_stride;
    if (st == MA_OK) st = check_rows("out", out, d->head_dim, d->n_tokens, d->n_heads, o_ts, o_hs);
    if (st == MA_OK) st = check_rows("dq", dq, 0, 1, 1, 0, 0);
    if (st == MA_OK) st = check_rows("dk", dk, 0, 1, 1, 0, 0);
    if (st == MA_OK) st = check_rows("dv", dv, 0, 1, 1, 0, 0);
    if (st != MA_OK) return st;
    if (!lse || !op_aligned(lse, 4)) return op_fail(lse ? MA_ERR_ALIGN : MA_ERR_ARG, "lse is NULL or not aligned to 4 bytes");
    if (!workspace || !op_aligned(workspace, 256))
      return op_fail(workspace ? MA_ERR_ALIGN : MA_ERR_ARG, "workspace is NULL or not 256-byte aligned");
    const GradSpace sp = grad_space(d);
    if (workspace_bytes < sp.bytes)
      return op_fail(MA_ERR_ARG, "workspace of %lld bytes, %lld are needed", (long long)workspace_bytes,
                     (long long)sp.bytes);
    int sms = 0, *err = nullptr;
    cudaError_t e = op_device(&sms, &err);
    if (e != cudaSuccess) return op_cuda(e, "device query");
    Maps m;
    AttnGrad g{};
    if (!maps_of(d, &m) ||
        !attn_map(&m.dout, dout, d->head_dim, d->n_tokens, d->n_heads, dout_token_stride, dout_head_stride) ||
        !dense_map(&g.tm_dq, dq, d, d->n_heads) || !dense_map(&g.tm_dk, dk, d, d->n_kv_heads) ||
        !dense_map(&g.tm_dv, dv, d, d->n_kv_heads))
      return op_fail(MA_ERR_CUDA, "cuTensorMapEncodeTiled refused a tensor");
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    g.dout = static_cast<const __nv_bfloat16*>(dout);
    g.out = static_cast<const __nv_bfloat16*>(out);
    g.do_ts = dout_token_stride;
    g.do_hs = dout_head_stride;
    g.o_ts = o_ts;
    g.o_hs = o_hs;
    g.lse = lse;
    g.nlse2 = reinterpret_cast<float*>(ws);
    g.ndelta = reinterpret_cast<float*>(ws + sp.stats);
    g.partial = reinterpret_cast<float*>(ws + 2 * sp.stats);
    g.partial_slots = sp.slots;
    g.counter = reinterpret_cast<int*>(ws + sp.counter);
    g.dq = static_cast<__nv_bfloat16*>(dq);
    g.dk = static_cast<__nv_bfloat16*>(dk);
    g.dv = static_cast<__nv_bfloat16*>(dv);
    e = attn_backward(args_of(d), m.q, m.k, m.v, m.dout, g, err, sms, static_cast<cudaStream_t>(cuda_stream));
    if (e != cudaSuccess) return op_cuda(e, "attention gradient launch");
  }
  clear_last_error();
  return MA_OK;
}

}  // extern "C"
