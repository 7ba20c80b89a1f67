// Products grouped by expert on the 5th-generation tensor cores (sm_103a).
//
//   forward   out[t]  = W_e x[t]              D[outer, token] = W[outer, inner]  x^T
//   input     dx[t]   = W_e^T dout[t]         D[inner, token] = W^T[inner, outer] dout^T
//   weights   dW_e    = sum_t dout[t] x[t]^T  D[outer, inner] = dout^T x
//
// In the first two the tokens are the products' N side and the weights their M
// side: N goes in steps of 32, so that an expert's last tokens, or its only few,
// cost what they are, where the M side would round them up to 256. Weights are
// read as they lie (K-major forward, MN-major for dx), nothing is transposed in
// memory. The third sums over an expert's tokens: its last block of 64 reaches
// into the next expert, and a warp of its own clears those rows before the
// product, so that whatever they hold meets no product.
//
// Persistent pairs of CTAs (a cluster of two) run tcgen05.mma.cta_group::2 with
// M = 256, N <= 256: each CTA loads its own 128 rows of the left operand and its
// half of the right one, 32 KB a block of 64, which is what the L2 delivers to
// an SM in the 512 cycles of the block's products; with a CTA for itself it
// would be 48 KB.
//   warps 0, 11  TMA loads of the left and of the right operand into a ring of
//              six stages
//   warp 1     products, issued by the even CTA; two accumulators of 256 columns, in turn, or one and the sum of its
//              runs (kRun)
//   warps 2-9  results from TMEM: transposed where tokens are columns, out
//              through shared memory and TMA; tiles with other experts' tokens
//              by plain stores of the rows that are theirs
//   warp 10    clears the rows behind an expert's tokens (third product)
// Which unit belongs to whom follows from the offsets, which only the device
// knows: every CTA adds them up for itself first.
//
// Every wait is bounded; where one runs out the error word is set, copies and
// products in flight end, and TMEM is freed. A wait spans a run's
// blocks at most, but for warp 10's: the units before the next one with rows to
// clear, any number of them, go by meanwhile. Its limit counts from the last
// progress of the loads.
#include <math.h>

#include <algorithm>

#include "op_common.cuh"
#include "tcgen05.cuh"

namespace ma {
namespace {

constexpr int kTile = 256;       // M of a pair, and the most N
constexpr int kHalf = kTile / 2;
constexpr int kBlock = 64;       // of the contraction
constexpr int kMidBox = 64, kSmallBox = 16;  // rows of the copies of smaller token tiles
constexpr int kOperand = kHalf * kBlock * 2;  // 16 KB: a CTA's part of one operand in a stage
constexpr int kStage = 2 * kOperand;
constexpr int kPanel = kBlock * 64 * 2;  // MN-major: 64 columns of a block's 64 rows
constexpr int kWarps = 12;
constexpr int kThreads = kWarps * 32;
constexpr int kStoreWarps = 8;
constexpr int kMaxExperts = 512;
// Blocks that one accumulator adds up. The tensor cores cut off toward zero what a sum cannot hold, so that a long
// one loses in proportion to its length (4096 tokens 4.4e-6, a million 1.2e-3; of terms of one sign 1.4e-5 and 6.8e-3).
// Longer sums are those of runs of this many blocks, which the warps that store add up in the other accumulator, to
// nearest. For results in bf16 8192 terms, 3.5e-5 of themselves at most; for fp32 2048: 2.1e-6, with 4096 4.4e-6 and
// with 1024 1.0e-6, at 5, 1 and 12 % more time (8192 tokens, 2048 -> 2048; 44.4 us in one run).
constexpr int kRun = 128, kRunF32 = 32;  // kRunF32: of an fp32 gradient of the weights
constexpr int kRaster = 8;  // token (or inner) tiles that walk together along the features
constexpr uint32_t kTmemColumns = 512;

// error codes of the waits that ran out
constexpr int kErrLoad = 0x501, kErrProduct = 0x502, kErrStore = 0x503, kErrClear = 0x504, kErrAlign = 0x505;

// Division of numbers below 2^31 by a divisor that the host knows: every warp takes every unit apart, and a division
// takes longer than the products of a small one.
struct Divisor {
  uint32_t d, mul, shift;  // mul 0: a power of two
};

struct ExpertArgs {
  // the product whose columns are tokens: out, or dx
  CUtensorMap a, b, b_mid, b_small, out;
  int m, k;  // rows of D; the contraction, 0: no such product
  Divisor band;  // units of kRaster token tiles
  void* dst;
  // the weights' gradients
  CUtensorMap wa, wb, wout;
  int wm, wn;  // rows (0: no such product) and columns
  Divisor wunits, wband;  // units of an expert; of kRaster column tiles
  void* grad;
  int accumulate;
  int rounds;  // units of these that take as long as one of dx
  const int32_t* offsets;
  int tokens, experts;
  int* err;
};

struct Layout {
  static constexpr int kStages = 6;
  // results on their way out, 32 rows of 64 bytes, two a warp: one is written while the other is read
  static constexpr int kTileBytes = 2048, kTiles = 2;
  static constexpr int kStore = kStages * kStage;
  static constexpr int kTable = kStore + kStoreWarps * kTiles * kTileBytes;
  static constexpr int kBars = kTable + (kMaxExperts + 4) * 4;
  // full, empty, tail, fixed [stage]; accumulator full, free [2]; drain
  static constexpr int kNumBars = 4 * kStages + 5;
  static constexpr int kBytes = kBars + kNumBars * 8 + 16;
  static_assert(kBars % 8 == 0, "barriers");
  static_assert(kBytes <= 232448, "shared memory of a CTA");
};

// Everything below is issued by a converged warp, and the instructions elect the
// thread: addresses stay warp-uniform, as the instructions take them. From a
// branch of one lane a block's two copies took 360 cycles to issue, and bound
// small tiles.

// The four steps of a block, KA and KB further in the operands' descriptors each.
template <int KA, int KB>
__device__ __forceinline__ void umma_block_warp(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                uint32_t accumulate) {
  static_assert(kBlock == 64, "four steps of 16");
  asm volatile(
      "{\n\t.reg .pred p, q, t;\n\t"
      ".reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "add.s64 a1, %1, %5;\n\tadd.s64 a2, %1, %6;\n\tadd.s64 a3, %1, %7;\n\t"
      "add.s64 b1, %2, %8;\n\tadd.s64 b2, %2, %9;\n\tadd.s64 b3, %2, %10;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.eq.b32 t, 0, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], a1, b1, %3, t;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], a2, b2, %3, t;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], a3, b3, %3, t;\n\t}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "n"(KA), "n"(2 * KA), "n"(3 * KA), "n"(KB), "n"(2 * KB),
      "n"(3 * KB)
      : "memory");
}
__device__ __forceinline__ void umma_pair_warp(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// The products issued so far have ended: one arrival on the barrier at this offset in each CTA of the pair.
__device__ __forceinline__ void commit_pair_warp(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}\n" ::"r"(
          bar),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void commit_own_warp(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(bar)
      : "memory");
}
// An arrival at a barrier of either CTA of threads that have read TMEM (behind tc_fence_before). Nothing else is
// handed over, so that it need not wait for their writes to be visible in the cluster: that took 2500 cycles a unit.
__device__ __forceinline__ void arrive_either(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// A wait whose outcome is the whole warp's, on a barrier at which the other CTA arrives too.
__device__ __forceinline__ bool mbar_wait_warp_cluster(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                                       int* err, int code) {
  if (__all_sync(0xffffffffu, mbar_try_wait<true>(bar, parity))) return true;
  return __all_sync(0xffffffffu, mbar_wait_loop<true>(bar, parity, abort_flag, err, code));
}
// A wait during which the CTA may have any amount of work: it runs out once `progress`, a word of shared memory, has
// stood still for the limit.
__device__ __forceinline__ bool mbar_wait_warp_while(uint32_t bar, uint32_t parity, volatile int* progress,
                                                     volatile int* abort_flag, int* err, int code) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  bool ok = false;
  int seen = *progress;
  uint64_t since = global_timer();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) {
      ok = true;
      break;
    }
    if ((it & 63u) != 0) continue;
    if (*abort_flag) break;
    const int at = *progress;
    const uint64_t now = global_timer();
    if (at != seen) {
      seen = at;
      since = now;
    } else if (now - since > kWaitLimitNs) {
      *abort_flag = 1;
      atomicCAS(err, 0, code);
      break;
    }
  }
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ void expect_warp(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}\n" ::"r"(bar),
      "r"(bytes)
      : "memory");
}
__device__ __forceinline__ void load_warp(uint32_t dst, const CUtensorMap* tm, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];\n\t}\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// A copy into this CTA that counts on barrier `bar` of the pair's even CTA, a cluster address.
__device__ __forceinline__ void load_pair_warp(uint32_t dst, const CUtensorMap* tm, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3, %4}], [%5];\n\t}\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// Stores out of shared memory, a group each, and the wait until at most the last one still reads it.
__device__ __forceinline__ void store_2d_warp(const CUtensorMap* tm, uint32_t src, int x, int y) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];\n\t"
      "@q cp.async.bulk.commit_group;\n\t}\n" ::"l"(reinterpret_cast<uint64_t>(tm)),
      "r"(src), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void store_3d_warp(const CUtensorMap* tm, uint32_t src, int x, int y, int z) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];\n\t"
      "@q cp.async.bulk.commit_group;\n\t}\n" ::"l"(reinterpret_cast<uint64_t>(tm)),
      "r"(src), "r"(x), "r"(y), "r"(z)
      : "memory");
}
template <int LEFT>
__device__ __forceinline__ void stores_read_warp() {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q cp.async.bulk.wait_group.read %0;\n\t}\n" ::"n"(LEFT)
      : "memory");
  __syncwarp();
}
__device__ __forceinline__ uint32_t pack(uint32_t lo, uint32_t hi) {
  return op_pack_bf16(__uint_as_float(lo), __uint_as_float(hi));
}

// What a pair works on: rows m0 to m0 + 255 of D and `n` of its columns.
struct Unit {
  bool weights;  // of the weights' gradients
  int expert, m0, n0, n;
  int at, count;  // the unit's tokens
  int blocks;     // of the contraction; 0: zeros
};
template <bool BACK>
__device__ __forceinline__ bool is_weights(const Unit& u) {
  return BACK && u.weights;
}

// Expert e's tokens are bound[e] to bound[e + 1]; e = experts: those behind the last. `tokens` units of the product
// over tokens come first, in ascending order, so that each warp looks for a unit's expert from its last one on.
struct Units {
  const int* bound;
  int tokens, all;
  int expert, first;  // `first`: that expert's first unit
};

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Which units a pair takes, one of `pairs`: in turn; but the pairs with one unit of the product over tokens more than
// the others leave the first `early` units of the weights' gradients to those.
template <bool BACK>
struct Deal {
  int pair, pairs, tokens, weights, extra, early;
  __device__ __forceinline__ Deal(const ExpertArgs& a, const Units& all, int pair_, int pairs_)
      : pair(pair_), pairs(pairs_), tokens(all.tokens), weights(all.all - all.tokens) {
    extra = !BACK ? 0 : tokens < pairs ? tokens : tokens % pairs;
    early = extra ? (int)min((int64_t)a.rounds * (pairs - extra), (int64_t)weights) : 0;
  }
  __device__ __forceinline__ int begin() const { return !BACK || pair < tokens ? pair : weights_from(); }
  __device__ __forceinline__ int after(int pos) const {
    if (!BACK) return pos + pairs;
    if (pos < tokens) return pos + pairs < tokens ? pos + pairs : weights_from();
    int i = pos - tokens;
    if (i < early) {
      i += pairs - extra;
      return tokens + (i < early ? i : early + pair);
    }
    return pos + pairs;
  }
  __device__ __forceinline__ int weights_from() const {
    return tokens + (pair >= extra && pair - extra < early ? pair - extra : early + pair);
  }
};

__device__ __forceinline__ int divide(int n, const Divisor& d) {
  return d.mul ? (int)(__umulhi((uint32_t)n, d.mul) >> d.shift) : n >> d.shift;
}
// Of r below 2^18 by at most kRaster.
__device__ __forceinline__ int divide_small(int r, int by) {
  return by == kRaster ? r / kRaster : __float2int_rz(__fdividef((float)r + 0.5f, (float)by));
}

template <bool BACK>
__device__ __forceinline__ Unit unit_at(const ExpertArgs& a, Units& all, int pos) {
  Unit u;
  u.weights = pos >= all.tokens;
  if (is_weights<BACK>(u)) {
    const int nt = ceil_div(a.wn, kTile);
    u.expert = divide(pos - all.tokens, a.wunits);
    const int local = pos - all.tokens - u.expert * (int)a.wunits.d;
    const int group = divide(local, a.wband), width = min(kRaster, nt - group * kRaster);
    const int r = local - group * (int)a.wband.d, row = divide_small(r, width);
    u.m0 = row * kTile;
    u.n0 = (group * kRaster + r - row * width) * kTile;
    u.n = a.wn - u.n0 > kHalf ? kTile : kHalf;
    u.at = all.bound[u.expert];
    u.count = all.bound[u.expert + 1] - u.at;
    u.blocks = ceil_div(u.count, kBlock);
  } else {
    const int mt = ceil_div(a.m, kTile);
    int begin, count, tt;
    for (;; ++all.expert, all.first += tt * mt) {
      begin = all.bound[all.expert];
      count = all.bound[all.expert + 1] - begin;
      tt = ceil_div(count, kTile);
      if (pos < all.first + tt * mt) break;
    }
    const int local = pos - all.first;
    const int group = divide(local, a.band), width = min(kRaster, tt - group * kRaster);
    const int r = local - group * (int)a.band.d, row = divide_small(r, width);
    // token tiles of one size; the last is never empty, since count > 256 (tt - 1)
    const int per = ((tt == 1 ? count : ceil_div(count, tt)) + 31) & ~31, tile = group * kRaster + r - row * width;
    u.expert = all.expert;
    u.m0 = row * kTile;
    u.n0 = 0;
    u.at = begin + tile * per;
    u.count = min(per, count - tile * per);
    u.n = (u.count + 31) & ~31;
    u.blocks = u.expert < a.experts ? ceil_div(a.k, kBlock) : 0;
  }
  return u;
}

// Rows of a token tile's copies into a CTA: its half of the tile, or more where one copy beats several.
__device__ __forceinline__ int token_rows(const Unit& u) {
  const int half = u.n / 2;
  return half <= 2 * kSmallBox ? half : half <= kMidBox ? kMidBox : kHalf;
}

template <bool BACK, bool F32>
__device__ __forceinline__ int run_of(const Unit& u) {
  return F32 && is_weights<BACK>(u) ? kRunF32 : kRun;
}

// Bytes that land in a CTA for one block.
template <bool BACK>
__device__ __forceinline__ uint32_t stage_bytes(const Unit& u) {
  return (uint32_t)(kOperand + (is_weights<BACK>(u) ? u.n / 2 / 64 * kPanel : token_rows(u) * kBlock * 2));
}

template <bool BACK, typename LOAD>
__device__ __forceinline__ void load_left(const ExpertArgs& a, const Unit& u, int block, uint32_t stage, uint32_t rank,
                                          LOAD load) {
  const int k0 = block * kBlock, m0 = u.m0 + (int)rank * kHalf;
  if constexpr (!BACK) {
    load(stage, &a.a, k0, m0, u.expert);
  } else {
    const CUtensorMap* const map = u.weights ? &a.wa : &a.a;
    const int y = u.weights ? u.at + k0 : k0, z = u.weights ? 0 : u.expert;
    for (int p = 0; p < kHalf / 64; ++p) load(stage + p * kPanel, map, m0 + p * 64, y, z);
  }
}

template <bool BACK, typename LOAD>
__device__ __forceinline__ void load_right(const ExpertArgs& a, const Unit& u, int block, uint32_t stage, uint32_t rank,
                                           LOAD load) {
  const int k0 = block * kBlock;
  const uint32_t sb = stage + kOperand;
  if (is_weights<BACK>(u)) {
    const int n0 = u.n0 + (int)rank * (u.n / 2);
    load(sb, &a.wb, n0, u.at + k0, 0);
    if (u.n == kTile) load(sb + kPanel, &a.wb, n0 + 64, u.at + k0, 0);
  } else {
    const int t0 = u.at + (int)rank * (u.n / 2), rows = token_rows(u);
    if (rows > 2 * kSmallBox) {
      load(sb, rows == kHalf ? &a.b : &a.b_mid, k0, t0, 0);
    } else {
      load(sb, &a.b_small, k0, t0, 0);
      if (rows > kSmallBox) load(sb + kSmallBox * kBlock * 2, &a.b_small, k0, t0 + kSmallBox, 0);
    }
  }
}

// 32 rows of D by 32 columns, D's rows the lanes: tokens are columns, so the
// block leaves transposed, a row of 32 features for each token.
__device__ __forceinline__ void store_tokens(const ExpertArgs& a, const Unit& u, int row0, int c0,
                                             const uint32_t (&r)[32], uint8_t* tiles, int& turn, int lane) {
  uint8_t* const tile = tiles + turn * Layout::kTileBytes;
  turn ^= 1;
  stores_read_warp<1>();  // this tile's last store has read it
  // rows of 64 bytes, 16-byte chunk q of row t at q ^ (t / 2 % 4): lanes 2 k and 2 k + 1 swap, the even one writes
  // the pair's even tokens, the odd one its odd ones
  uint8_t* const to = tile + (lane & 1) * 64 + ((lane >> 1) & 3) * 4;
  const uint32_t sel = (lane & 1) ? 0x3276u : 0x5410u;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const uint32_t mine = pack(r[2 * j], r[2 * j + 1]);
    const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, 1);
    *reinterpret_cast<uint32_t*>(to + 2 * j * 64 + (((lane >> 3) ^ (j & 3)) << 4)) = __byte_perm(mine, other, sel);
  }
  if (c0 + 32 <= u.count) {
    fence_proxy_async_smem();
    __syncwarp();
    store_2d_warp(&a.out, smem_u32(tile), row0, u.at + c0);
    return;
  }
  __syncwarp();
  const int q = lane & 3;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = i * 8 + (lane >> 2);
    if (c0 + t < u.count && row0 + q * 8 < a.m)
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.dst) + (int64_t)(u.at + c0 + t) * a.m + row0 + q * 8) =
          *reinterpret_cast<const uint4*>(tile + t * 64 + ((q ^ ((t >> 1) & 3)) << 4));
  }
  __syncwarp();
  // an empty group, so that the tiles' turns and the groups stay in step
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t@q cp.async.bulk.commit_group;\n\t}\n" ::: "memory");
}

// What an expert's gradient holds so far in a lane's 32 columns of a block, as it lies in memory.
template <bool F32>
struct Before {
  uint4 v[F32 ? 8 : 4];
  __device__ __forceinline__ void load(const ExpertArgs& a, const Unit& u, int row, int col) {
    const uint4* const p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.grad) +
                                                          (((int64_t)u.expert * a.wm + row) * a.wn + col) * (F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (F32 ? 8 : 4); ++i)
      if (row < a.wm && col + i * (F32 ? 4 : 8) < a.wn) v[i] = p[i];
  }
  __device__ __forceinline__ float get(int e) const {
    const uint4 x = v[e / (F32 ? 4 : 8)];
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    if constexpr (F32) return __uint_as_float(w[e % 4]);
    return __uint_as_float(e & 1 ? w[e / 2 % 4] & 0xFFFF0000u : w[e / 2 % 4] << 16);
  }
};

// 32 rows of an expert's gradient by 32 columns, a row to a lane. `turn`: the tile that is next.
template <bool F32>
__device__ __forceinline__ void store_weights(const ExpertArgs& a, const Unit& u, int row0, int col0,
                                              const uint32_t (&r)[32], uint8_t* tiles, int& turn, int lane) {
#pragma unroll
  for (int h = 0; h < (F32 ? 2 : 1); ++h, turn ^= 1) {
    uint8_t* const tile = tiles + turn * Layout::kTileBytes;
    stores_read_warp<1>();  // this tile's last store has read it
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint4 v;
      if constexpr (F32)
        v = make_uint4(r[16 * h + 4 * q], r[16 * h + 4 * q + 1], r[16 * h + 4 * q + 2], r[16 * h + 4 * q + 3]);
      else
        v = make_uint4(pack(r[8 * q], r[8 * q + 1]), pack(r[8 * q + 2], r[8 * q + 3]), pack(r[8 * q + 4], r[8 * q + 5]),
                       pack(r[8 * q + 6], r[8 * q + 7]));
      *reinterpret_cast<uint4*>(tile + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)) = v;
    }
    fence_proxy_async_smem();
    __syncwarp();
    // (the second half of 32 fp32 columns may lie outside: nothing of it is written)
    store_3d_warp(&a.wout, smem_u32(tile), col0 + 16 * h, row0, u.expert);
  }
}

// A run's sum with that of the runs before it, to `to`: every second 32 columns of this warp's rows in TMEM.
__device__ __forceinline__ void add_run(uint32_t run, uint32_t before, uint32_t to, int c0, int columns, bool first) {
  for (; c0 < columns; c0 += 64) {
    uint32_t r[32], s[32];
    tmem_ld_32x32b_x32(run + (uint32_t)c0, r);
    if (!first) tmem_ld_32x32b_x32(before + (uint32_t)c0, s);
    tmem_ld_wait();
    if (!first) {
#pragma unroll
      for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) + __uint_as_float(s[e]));
    }
    tmem_st_32x32b_x32(to + (uint32_t)c0, r);
  }
  tmem_st_wait();
}

// BACK: dx and the weights' gradients in one launch, the units of both dealt out as they come.
template <bool BACK, bool F32>
__global__ void __launch_bounds__(kThreads, 1) expert_matmul_kernel(const __grid_constant__ ExpertArgs a) {
  using L = Layout;
  constexpr int S = L::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023) {  // the operands' swizzle counts on it; in both CTAs alike
    if (threadIdx.x == 0) atomicCAS(a.err, 0, kErrAlign);
    return;
  }
  int* const bound = reinterpret_cast<int*>(smem + L::kTable);
  uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(bars + L::kNumBars);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* const progress = abort_flag + 1;  // blocks that warp 0 has loaded, every 64
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t full = smem_u32(bars), empty = full + 8 * S, tail = empty + 8 * S, fixed = tail + 8 * S;
  const uint32_t acc_full = fixed + 8 * S, acc_free = acc_full + 16, drain = acc_free + 16;
  const uint32_t rank = cluster_ctarank();

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
      mbar_init(tail + 8 * s, 1);
      mbar_init(fixed + 8 * s, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + 8 * i, 1);
      mbar_init(acc_free + 8 * i, 2 * kStoreWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = *progress = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (warp == 1) tmem_alloc<2>(smem_u32(tmem_slot), kTmemColumns);
  pdl_wait();
  pdl_launch();
  if (warp == 0) {
    // the experts' bounds, kept in order and in range whatever the offsets hold, and their units
    int before = 0, units = 0;
    const int mt = ceil_div(a.m, kTile);
    if (lane == 0) bound[0] = 0;
    for (int e0 = 0; e0 <= a.experts; e0 += 32) {
      const int e = e0 + lane;  // bound[e + 1]; the last one is where the tokens end
      int b = e < a.experts ? min(max(a.offsets[e + 1], 0), a.tokens) : a.tokens;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, b, d);
        if (lane >= d) b = max(b, o);
      }
      b = max(b, before);
      int begin = __shfl_up_sync(0xffffffffu, b, 1);
      if (lane == 0) begin = before;
      before = __shfl_sync(0xffffffffu, b, 31);
      units += ceil_div(b - begin, kTile) * mt;
      if (e <= a.experts) bound[e + 1] = b;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) units += __shfl_xor_sync(0xffffffffu, units, d);
    if (lane == 0) bound[kMaxExperts + 3] = a.k > 0 ? units : 0;
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the other CTA's barriers are there before a copy or a commit reaches them
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Units tab{bound, bound[kMaxExperts + 3], 0, 0, 0};
  tab.all = tab.tokens + (BACK ? a.experts * ceil_div(a.wm, kTile) * ceil_div(a.wn, kTile) : 0);
  const Deal<BACK> deal(a, tab, blockIdx.x / 2, gridDim.x / 2);

  if (warp == 0 || warp == kWarps - 1) {
    // ---- loads, a warp for each operand: issuing a copy takes some 100 cycles ----
    const bool left = warp == 0;
    int stage = 0, issued = 0;
    uint32_t phase = 0;
    bool ok = true;
    const uint32_t s0 = smem_u32(smem), full_pair = mapa_shared(full, 0);
    for (int pos = deal.begin(); pos < tab.all && ok; pos = deal.after(pos)) {
      const Unit u = unit_at<BACK>(a, tab, pos);
      const uint32_t bytes = stage_bytes<BACK>(u);
      for (int b = 0; b < u.blocks; ++b) {
        if (BACK && left && (b & 63) == 0 && lane == 0) *progress = issued + 1;
        if (!mbar_wait_warp(empty + 8 * stage, phase ^ 1u, abort_flag, a.err, kErrLoad)) {
          ok = false;
          break;
        }
        const uint32_t at = s0 + (uint32_t)(stage * kStage);
        if (is_weights<BACK>(u) && b == u.blocks - 1 && u.count % kBlock != 0) {
          // rows of the next expert in it: lands on a barrier of this CTA's, and is cleared before it is full
          const uint32_t bar = tail + 8 * stage;
          auto load = [&](uint32_t dst, const CUtensorMap* tm, int x, int y, int z) { load_warp(dst, tm, x, y, z, bar); };
          if (left) {
            expect_warp(bar, bytes);
            load_left<BACK>(a, u, b, at, rank, load);
          } else {
            load_right<BACK>(a, u, b, at, rank, load);
          }
        } else {
          const uint32_t bar = full_pair + 8 * stage;
          auto load = [&](uint32_t dst, const CUtensorMap* tm, int x, int y, int z) {
            load_pair_warp(dst, tm, x, y, z, bar);
          };
          if (left) {
            if (rank == 0) expect_warp(full + 8 * stage, 2 * bytes);
            load_left<BACK>(a, u, b, at, rank, load);
          } else {
            load_right<BACK>(a, u, b, at, rank, load);
          }
        }
        ++issued;
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // copies in flight land before the CTA leaves: those of the odd CTA count on the even one's barriers
    if (left && rank == 0) {
      for (int i = 0; i < min(issued, S); ++i) {
        if (--stage < 0) {
          stage = S - 1;
          phase ^= 1u;
        }
        drain_wait(full + 8 * stage, phase);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      // ---- products ----
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;  // acc_phase: a bit an accumulator
      bool ok = true;
      const uint32_t s0 = smem_u32(smem);
      // MN-major: panels of 64 columns, sixteen rows of the contraction 2 KB further
      constexpr int kStepA = BACK ? 128 : 2;
      const uint64_t a0 = BACK ? sdesc(s0, kPanel, 1024) : sdesc(s0, 16, 1024);
      const uint64_t b_k = sdesc(s0 + kOperand, 16, 1024), b_mn = sdesc(s0 + kOperand, kPanel, 1024);
      for (int pos = deal.begin(); pos < tab.all && ok; pos = deal.after(pos)) {
        const Unit u = unit_at<BACK>(a, tab, pos);
        if (u.blocks == 0) continue;
        const bool weights = is_weights<BACK>(u);
        const uint32_t idesc = idesc_bf16(kTile, u.n, weights) | (BACK ? 1u << 15 : 0u);
        const uint32_t d = tmem + (uint32_t)(acc * kTile);
        const int run = run_of<BACK, F32>(u);
        for (int b0 = 0; b0 < u.blocks; b0 += run) {
          ok = mbar_wait_warp_cluster(acc_free + 8 * acc, (acc_phase >> acc & 1u) ^ 1u, abort_flag, a.err, kErrProduct);
          if (!ok) break;
          tc_fence_after();
          const int end = min(b0 + run, u.blocks);
          for (int b = b0; b < end; ++b) {
            if (!mbar_wait_warp_cluster(full + 8 * stage, phase, abort_flag, a.err, kErrProduct)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t off = (uint32_t)stage * (uint32_t)(kStage >> 4);
            const uint64_t ad = a0 + off;
            if (!weights) {
              umma_block_warp<kStepA, 2>(d, ad, b_k + off, idesc, b != b0 ? 1u : 0u);
            } else {
              const int left = u.count - b * kBlock;
              if (left > kBlock - 16) {
                umma_block_warp<kStepA, 128>(d, ad, b_mn + off, idesc, b != b0 ? 1u : 0u);
              } else {
                for (int i = 0; i * 16 < left; ++i)
                  umma_pair_warp(d, ad + kStepA * i, b_mn + off + 128 * i, idesc, ((b - b0) | i) != 0 ? 1u : 0u);
              }
            }
            commit_pair_warp(empty + 8 * stage);
            if (++stage == S) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          commit_pair_warp(acc_full + 8 * acc);
          acc_phase ^= 1u << acc;
        }
        // the sum of several runs is in the other accumulator, until its tile has left and this one is free
        if (u.blocks <= run) acc ^= 1;
      }
      commit_own_warp(drain);  // products in flight end before TMEM is freed
      drain_wait(drain, 0);
      __syncwarp();
    }
  } else if (warp < 2 + kStoreWarps) {
    // ---- results ----
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    uint8_t* const tiles = smem + L::kStore + (warp - 2) * L::kTiles * L::kTileBytes;
    int acc = 0, turn = 0;
    uint32_t acc_phase = 0;
    for (int pos = deal.begin(); pos < tab.all; pos = deal.after(pos)) {
      const Unit u = unit_at<BACK>(a, tab, pos);
      const bool weights = is_weights<BACK>(u), adds = weights && a.accumulate != 0;
      const int row0 = u.m0 + (int)rank * kHalf + quarter * 32;
      const int columns = weights ? min(u.n, a.wn - u.n0) : u.count, run = run_of<BACK, F32>(u);
      const bool inside = row0 < (weights ? a.wm : a.m);
      const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
      const uint32_t t0 = lanes + (uint32_t)(acc * kTile), sum0 = lanes + (uint32_t)((acc ^ 1) * kTile);
      Before<F32> next;
      if (adds && u.blocks > 0) next.load(a, u, row0 + lane, u.n0 + 32 * half);
      bool ok = true;
      for (int b = run; u.blocks > 0; b += run) {
        const bool got = mbar_wait(acc_full + 8 * acc, acc_phase >> acc & 1u, abort_flag, a.err, kErrStore);
        ok = __all_sync(0xffffffffu, got);
        if (!ok) break;
        tc_fence_after();
        const bool last = b >= u.blocks;
        // the sum so far lies in the other accumulator, whose last tile this warp has read, and in the end in this one
        if (__builtin_expect(inside && u.blocks > run, 0)) add_run(t0, sum0, last ? t0 : sum0, 32 * half, columns, b == run);
        if (last) break;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_either(mapa_shared(acc_free + 8 * acc, 0));
        acc_phase ^= 1u << acc;
      }
      if (!ok) break;
      if (inside && !(adds && u.blocks == 0)) {
        for (int c0 = 32 * half; c0 < columns; c0 += 64) {
          const Before<F32> before = next;
          if (adds && c0 + 64 < columns) next.load(a, u, row0 + lane, u.n0 + c0 + 64);
          uint32_t r[32];
          if (u.blocks > 0) {
            tmem_ld_32x32b_x32(t0 + (uint32_t)c0, r);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = 0;
          }
          if (weights) {
            if (adds) {
#pragma unroll
              for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) + before.get(e));
            }
            store_weights<F32>(a, u, row0, u.n0 + c0, r, tiles, turn, lane);
          } else {
            store_tokens(a, u, row0, c0, r, tiles, turn, lane);
          }
        }
      }
      if (u.blocks > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_either(mapa_shared(acc_free + 8 * acc, 0));
        acc_phase ^= 1u << acc;
        if (u.blocks <= run) acc ^= 1;
      }
    }
    stores_read_warp<0>();  // the stores have read shared memory
  } else if (BACK) {
    // ---- rows behind an expert's tokens ----
    int issued = 0;
    uint32_t tail_phase = 0, fixed_phase = 0;  // a bit a stage
    for (int pos = deal.begin(); pos < tab.all; pos = deal.after(pos)) {
      const Unit u = unit_at<BACK>(a, tab, pos);
      issued += u.blocks;
      const int left = u.count % kBlock;
      if (!u.weights || left == 0) continue;
      const int stage = (issued - 1) % S;
      if (!mbar_wait_warp_while(tail + 8 * stage, (tail_phase >> stage) & 1u, progress, abort_flag, a.err, kErrClear))
        break;
      tail_phase ^= 1u << stage;
      const int end = (left + 15) & ~15;  // products go in steps of 16
      uint8_t* const at = smem + stage * kStage;
      const int panels = kHalf / 64 + u.n / 2 / 64;  // the left operand's, then the right one's
      for (int p = 0; p < panels; ++p)
        for (int i = left * 8 + lane; i < end * 8; i += 32)
          *reinterpret_cast<uint4*>(at + p * kPanel + i * 16) = make_uint4(0, 0, 0, 0);
      fence_proxy_async_smem();
      __syncwarp();
      if (rank != 0) {
        if (lane == 0) mbar_arrive_cluster(mapa_shared(fixed + 8 * stage, 0));
        continue;
      }
      if (!mbar_wait_warp_cluster(fixed + 8 * stage, (fixed_phase >> stage) & 1u, abort_flag, a.err, kErrClear)) break;
      fixed_phase ^= 1u << stage;
      fence_proxy_async_smem();
      if (lane == 0) mbar_arrive(full + 8 * stage);
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither leaves while the other may reach its shared memory or TMEM
  tc_fence_after();
  if (warp == 1) tmem_dealloc<2>(tmem, kTmemColumns);
}

// ---- host ----

// A row-major tensor [z][y][x] of 16-byte aligned rows.
bool map3(CUtensorMap* tm, const void* base, bool f32, int64_t x, int64_t y, int64_t z, int64_t sy, int64_t sz,
          int box_x, int box_y, CUtensorMapSwizzle swizzle) {
  const int64_t e = f32 ? 4 : 2;
  // the stride of a single row or matrix is never used, but has to be a legal one
  if (y <= 1) sy = x;
  if (z <= 1) sz = sy;
  const cuuint64_t dims[3] = {(cuuint64_t)x, (cuuint64_t)y, (cuuint64_t)z};
  const cuuint64_t strides[2] = {(cuuint64_t)(sy * e), (cuuint64_t)(sz * e)};
  const cuuint32_t box[3] = {(cuuint32_t)box_x, (cuuint32_t)box_y, 1}, step[3] = {1, 1, 1};
  return op_tensor_map(tm, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims,
                       strides, box, step, swizzle);
}

bool map2(CUtensorMap* tm, const void* base, int64_t x, int64_t y, int box_x, int box_y, CUtensorMapSwizzle swizzle) {
  const cuuint64_t dims[2] = {(cuuint64_t)x, (cuuint64_t)y}, strides[1] = {(cuuint64_t)(x * 2)};
  const cuuint32_t box[2] = {(cuuint32_t)box_x, (cuuint32_t)box_y}, step[2] = {1, 1};
  return op_tensor_map(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, step, swizzle);
}

template <bool BACK, bool F32>
cudaError_t launch(ExpertArgs& a, int sms, int64_t most_units, cudaStream_t st) {
  using L = Layout;
  cudaError_t e = op_smem_limit<expert_matmul_kernel<BACK, F32>>(L::kBytes);
  if (e != cudaSuccess) return e;
  const int64_t pairs = std::max<int64_t>(1, std::min<int64_t>(sms / 2, most_units));
  return op_launch(expert_matmul_kernel<BACK, F32>, dim3((unsigned)(2 * pairs)), dim3(kThreads), L::kBytes, st, 2, a);
}

ma_status check(const ma_expert_matmul* d, bool weight) {
  if (!d) return op_fail(MA_ERR_ARG, "the description must not be NULL");
  if (d->n_experts < 1 || d->n_experts > kMaxExperts)
    return op_fail(MA_ERR_SHAPE, "%d experts: outside [1, %d]", d->n_experts, kMaxExperts);
  if (d->inner < 8 || d->inner > 1 << 20 || d->inner % 8 || d->outer < 8 || d->outer > 1 << 20 || d->outer % 8)
    return op_fail(MA_ERR_SHAPE, "inner %d or outer %d is no multiple of 8 in [8, 2^20]", d->inner, d->outer);
  // (rows and a CTA's blocks are counted in 31 bits)
  if (d->n_tokens < 0 || d->n_tokens > 1ll << 28)
    return op_fail(MA_ERR_SHAPE, "%lld tokens: outside [0, 2^28]", (long long)d->n_tokens);
  const int64_t wide = (std::max(d->inner, d->outer) + kTile - 1) / kTile;
  const int64_t narrow = (std::min(d->inner, d->outer) + kTile - 1) / kTile;
  if ((d->n_tokens / kTile + d->n_experts + 1) * wide > INT32_MAX / 2 || d->n_experts * wide * narrow > INT32_MAX / 2)
    return op_fail(MA_ERR_SHAPE, "%lld tokens and %d experts of %d x %d are too many for a call",
                   (long long)d->n_tokens, d->n_experts, d->outer, d->inner);
  if (!d->offsets) return op_fail(MA_ERR_ARG, "offsets must not be NULL");
  if (!op_aligned(d->offsets, 4)) return op_fail(MA_ERR_ALIGN, "offsets is not aligned to 4 bytes");
  if (d->n_tokens > 0 && weight) {
    if (!d->weight) return op_fail(MA_ERR_ARG, "weight must not be NULL");
    if (d->weight_row_stride > 1ll << 38 || d->weight_expert_stride > 1ll << 38)
      return op_fail(MA_ERR_SHAPE, "a stride of the weights is above 2^38");
    if (d->weight_row_stride < d->inner ||
        (d->n_experts > 1 && d->weight_expert_stride < (d->outer - 1) * d->weight_row_stride + d->inner))
      return op_fail(MA_ERR_SHAPE, "the weights' rows or matrices overlap");
    if (!op_aligned(d->weight, 16) || d->weight_row_stride % 8 || (d->n_experts > 1 && d->weight_expert_stride % 8))
      return op_fail(MA_ERR_ALIGN, "the weights' rows do not start on 16-byte boundaries");
  }
  return MA_OK;
}

ma_status check_rows(const char* name, const void* p, int64_t n, int64_t width, int64_t stride) {
  if (!p) return op_fail(MA_ERR_ARG, "%s must not be NULL", name);
  if (n > 1 && (stride < width || stride > 1ll << 38))
    return op_fail(MA_ERR_SHAPE, "%s has rows %lld apart: below the width, or above 2^38", name, (long long)stride);
  if (!op_aligned(p, 16) || (n > 1 && stride % 8))
    return op_fail(MA_ERR_ALIGN, "%s does not have its rows on 16-byte boundaries", name);
  return MA_OK;
}

ma_status refused_map() { return op_fail(MA_ERR_CUDA, "cuTensorMapEncodeTiled refused a tensor"); }

Divisor divisor(int64_t d) {
  uint32_t s = 0;
  while ((2ll << s) <= d) ++s;  // 2^s <= d < 2^(s + 1)
  if ((1ll << s) == d) return {(uint32_t)d, 0, s};
  // with e = mul d - 2^(32 + s) <= d: n e < 2^31 2^(s + 1), so that the quotient's fraction is not carried over
  return {(uint32_t)d, (uint32_t)((1ull << (32 + s)) / (uint64_t)d + 1), s};
}

ExpertArgs args_of(const ma_expert_matmul* d, int* err) {
  ExpertArgs a{};
  a.offsets = d->offsets;
  a.tokens = (int)d->n_tokens;
  a.experts = d->n_experts;
  a.err = err;
  return a;
}

constexpr CUtensorMapSwizzle kWide = CU_TENSOR_MAP_SWIZZLE_128B, kNarrow = CU_TENSOR_MAP_SWIZZLE_64B;

// Units of a product whose columns are tokens, at most.
int64_t token_units(const ExpertArgs& a) {
  return ((int64_t)a.tokens / kTile + std::min(a.experts + 1, a.tokens)) * ((a.m + kTile - 1) / kTile);
}

}  // namespace
}  // namespace ma

using namespace ma;

extern "C" {

ma_status muon_adamw_expert_matmul(const ma_expert_matmul* d, void* out, void* cuda_stream) {
  ma_status st = check(d, true);
  if (st != MA_OK) return st;
  if (d->n_tokens > 0) {
    st = check_rows("x", d->x, d->n_tokens, d->inner, d->x_stride);
    if (st == MA_OK) st = check_rows("out", out, d->n_tokens, d->outer, d->outer);
    if (st != MA_OK) return st;
    int sms = 0, *err = nullptr;
    cudaError_t e = op_device(&sms, &err);
    if (e != cudaSuccess) return op_cuda(e, "device query");
    ExpertArgs a = args_of(d, err);
    a.m = d->outer;
    a.k = d->inner;
    a.band = divisor(kRaster * ((a.m + kTile - 1) / kTile));
    a.dst = out;
    if (!map3(&a.a, d->weight, false, d->inner, d->outer, d->n_experts, d->weight_row_stride, d->weight_expert_stride,
              kBlock, kHalf, kWide) ||
        !map3(&a.b, d->x, false, d->inner, d->n_tokens, 1, d->x_stride, 0, kBlock, kHalf, kWide) ||
        !map3(&a.b_mid, d->x, false, d->inner, d->n_tokens, 1, d->x_stride, 0, kBlock, kMidBox, kWide) ||
        !map3(&a.b_small, d->x, false, d->inner, d->n_tokens, 1, d->x_stride, 0, kBlock, kSmallBox, kWide) ||
        !map2(&a.out, out, d->outer, d->n_tokens, 32, 32, kNarrow))
      return refused_map();
    e = launch<false, false>(a, sms, token_units(a), static_cast<cudaStream_t>(cuda_stream));
    if (e != cudaSuccess) return op_cuda(e, "expert product launch");
  }
  clear_last_error();
  return MA_OK;
}

ma_status muon_adamw_expert_matmul_backward(const ma_expert_matmul* d, const void* dout, int64_t dout_stride,
                                            void* dx, void* dweight, int grad_dtype, int accumulate,
                                            void* cuda_stream) {
  ma_status st = check(d, dx != nullptr);
  if (st != MA_OK) return st;
  if (!op_dtype_ok(grad_dtype))
    return op_fail(MA_ERR_DTYPE, "grad_dtype %d is neither MA_DT_F32 nor MA_DT_BF16", grad_dtype);
  if (accumulate != 0 && accumulate != 1) return op_fail(MA_ERR_ARG, "accumulate %d is neither 0 nor 1", accumulate);
  if (d->n_tokens > 0) {
    st = check_rows("dout", dout, d->n_tokens, d->outer, dout_stride);
    if (st == MA_OK && dweight) st = check_rows("x", d->x, d->n_tokens, d->inner, d->x_stride);
    if (st == MA_OK && dx) st = check_rows("dx", dx, d->n_tokens, d->inner, d->inner);
    if (st != MA_OK) return st;
  }
  if (dweight && !op_aligned(dweight, 16)) return op_fail(MA_ERR_ALIGN, "dweight is not aligned to 16 bytes");
  int sms = 0, *err = nullptr;
  cudaError_t e = op_device(&sms, &err);
  if (e != cudaSuccess) return op_cuda(e, "device query");
  const cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  const bool f32 = grad_dtype == MA_DT_F32;
  if (d->n_tokens == 0) {
    if (dweight && !accumulate) {
      e = cudaMemsetAsync(dweight, 0, (size_t)d->n_experts * d->outer * d->inner * op_dtype_size(grad_dtype), s);
      if (e != cudaSuccess) return op_cuda(e, "expert weight gradient");
    }
  } else if (dx || dweight) {
    ExpertArgs a = args_of(d, err);
    int64_t units = 0;
    if (dx) {
      a.m = d->inner;
      a.k = d->outer;
      a.band = divisor(kRaster * ((a.m + kTile - 1) / kTile));
      a.dst = dx;
      if (!map3(&a.a, d->weight, false, d->inner, d->outer, d->n_experts, d->weight_row_stride,
                d->weight_expert_stride, 64, kBlock, kWide) ||
          !map3(&a.b, dout, false, d->outer, d->n_tokens, 1, dout_stride, 0, kBlock, kHalf, kWide) ||
          !map3(&a.b_mid, dout, false, d->outer, d->n_tokens, 1, dout_stride, 0, kBlock, kMidBox, kWide) ||
          !map3(&a.b_small, dout, false, d->outer, d->n_tokens, 1, dout_stride, 0, kBlock, kSmallBox, kWide) ||
          !map2(&a.out, dx, d->inner, d->n_tokens, 32, 32, kNarrow))
        return refused_map();
      units += token_units(a);
    }
    if (dweight) {
      a.wm = d->outer;
      a.wn = d->inner;
      const int64_t mt = (a.wm + kTile - 1) / kTile, nt = (a.wn + kTile - 1) / kTile;
      a.wunits = divisor(mt * nt);
      a.wband = divisor(mt * kRaster);
      a.grad = dweight;
      a.accumulate = accumulate;
      if (!map3(&a.wa, dout, false, d->outer, d->n_tokens, 1, dout_stride, 0, 64, kBlock, kWide) ||
          !map3(&a.wb, d->x, false, d->inner, d->n_tokens, 1, d->x_stride, 0, 64, kBlock, kWide) ||
          !map3(&a.wout, dweight, f32, d->inner, d->outer, d->n_experts, d->inner, (int64_t)d->outer * d->inner,
                f32 ? 16 : 32, 32, kNarrow))
        return refused_map();
      units += d->n_experts * mt * nt;
    }
    // a unit of dx has its contraction's blocks, one of the weights its expert's tokens' or, for few, the time of nine
    a.rounds = (d->outer + kBlock - 1) / kBlock / (int)std::max<int64_t>(d->n_tokens / d->n_experts / kBlock, 9);
    e = f32 ? launch<true, true>(a, sms, units, s) : launch<true, false>(a, sms, units, s);
    if (e != cudaSuccess) return op_cuda(e, "expert gradient launch");
  }
  clear_last_error();
  return MA_OK;
}

}  // extern "C"
