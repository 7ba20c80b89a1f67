// Shared by the forward and gradient kernels of the sliding-window attention:
// arguments, how samples are cut into tiles, which tiles a tile of queries or
// keys meets, and the shared-memory ring that feeds the tensor cores.
#pragma once

#include <math.h>

#include "op_common.cuh"
#include "tcgen05.cuh"

namespace ma {

constexpr int kAttnTile = 128;  // queries or keys of a tile: the M of an MMA

struct AttnArgs {
  int n, heads, kv_heads, dim, sinks, window, n_seqs;
  float scale, scale_log2;  // scale, and scale * log2(e): scores enter exp2
  const int32_t* cu;
  const float* nlse2;       // gradient: -lse * log2(e), -infinity for a query that sees nothing [head][token]
  const float* ndelta;      // gradient: -dout . out [head][token]
};

// A 3-D map (element, token, head) of a bf16 tensor with 64 x 128 x 1 boxes in
// the 128-byte swizzle: a tile is one or two panels of 64 elements by 128
// tokens. Elements past head_dim and tokens past n read as zero.
bool attn_map(CUtensorMap* tm, const void* base, int dim, int64_t tokens, int64_t heads, int64_t token_stride,
              int64_t head_stride);

cudaError_t attn_forward(const AttnArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                         const CUtensorMap& o, __nv_bfloat16* out, float* lse, int* err, int sms, cudaStream_t st);

struct AttnGrad {
  const __nv_bfloat16 *dout, *out;
  int64_t do_ts, do_hs, o_ts, o_hs;
  const float* lse;
  float *nlse2, *ndelta, *partial;
  int64_t partial_slots;
  __nv_bfloat16 *dq, *dk, *dv;
  int* counter;  // 1 + n_seqs kv_heads, zeroed and counted by the launches
  CUtensorMap tm_dq, tm_dk, tm_dv;
};
cudaError_t attn_backward(AttnArgs a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                          const CUtensorMap& dout, const AttnGrad& g, int* err, int sms, cudaStream_t st);

// Query tiles of a chunk of the gradient for sink keys (see dkv_part).
constexpr int kSinkChunk = 8;

// Upper bound of the tiles of `rows` tokens that any cut into samples gives,
// the tokens behind the last sample counting as one more.
inline int64_t attn_max_tiles(int64_t n, int64_t n_seqs, int rows) { return n / rows + n_seqs + 1; }

#ifdef __CUDACC__
namespace {

// First token of sample i as the kernels read cu: clamped to [0, n].
__device__ __forceinline__ int sample_bound(const AttnArgs& a, int i) {
  return i == 0 ? 0 : min(max(__ldg(a.cu + i), 0), a.n);
}

struct SampleTile {
  int b, len;   // the sample's first token and length
  int p0;       // the tile's first row, counted from the sample's first token
  int sample;   // its number
  int index;    // the tile's number within its sample
  bool live;    // false: tokens behind the last sample, which see nothing
};

// Sample i of [0, n_seqs], the last being the tokens behind the samples.
__device__ __forceinline__ void sample_span(const AttnArgs& a, int i, int& b, int& len) {
  b = sample_bound(a, i);
  const int e = i == a.n_seqs ? a.n : max(sample_bound(a, i + 1), b);
  len = max(e - b, 0);
}

// The unit `u` of the samples' consecutive units, `count(len, live)` to a
// sample; found by a whole warp, 32 samples at a time.
template <typename F>
__device__ __forceinline__ SampleTile find_unit(const AttnArgs& a, int u, int lane, F count) {
  SampleTile t;
  if (a.cu == nullptr) {
    t.b = 0, t.len = a.n, t.sample = 0, t.index = u, t.live = true, t.p0 = 0;
    return t;
  }
  int base = 0;
  for (int i0 = 0; i0 <= a.n_seqs; i0 += 32) {
    const int i = i0 + lane;
    int b = 0, len = 0, c = 0;
    if (i <= a.n_seqs) {
      sample_span(a, i, b, len);
      c = count(len, i < a.n_seqs);
    }
    int incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const uint32_t over = __ballot_sync(0xffffffffu, u < base + incl);
    if (over) {
      const int src = __ffs(over) - 1;
      t.b = __shfl_sync(0xffffffffu, b, src);
      t.len = __shfl_sync(0xffffffffu, len, src);
      t.index = u - base - __shfl_sync(0xffffffffu, incl - c, src);
      t.sample = i0 + src;
      t.live = t.sample < a.n_seqs;
      t.p0 = 0;
      return t;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  t.b = a.n, t.len = 0, t.p0 = 0, t.sample = a.n_seqs, t.index = 0, t.live = false;
  return t;
}

// All samples' units, by a whole warp.
template <typename F>
__device__ __forceinline__ int count_units(const AttnArgs& a, int lane, F count) {
  if (a.cu == nullptr) return count(a.n, true);
  int sum = 0;
  for (int i0 = 0; i0 <= a.n_seqs; i0 += 32) {
    const int i = i0 + lane;
    if (i <= a.n_seqs) {
      int b, len;
      sample_span(a, i, b, len);
      sum += count(len, i < a.n_seqs);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// Key tiles (of 128 keys, counted from the sample's first) that the 128
// queries from p0 see: lo .. hi through the window, and tile 0 through the
// sinks where lo is past it.
struct KeyTiles {
  int lo, hi;
  bool sink;
};
__device__ __forceinline__ KeyTiles key_tiles(const AttnArgs& a, bool live, int len, int p0) {
  KeyTiles r{0, -1, false};
  if (!live || p0 >= len) return r;
  if (a.window == 0) return KeyTiles{1, 0, a.sinks > 0};
  r.lo = max(0, p0 - a.window + 1) / kAttnTile;
  r.hi = p0 / kAttnTile;
  r.sink = a.sinks > 0 && r.lo > 0;
  return r;
}

// Every one of 128 queries from q0 sees every one of 128 keys from k0.
__device__ __forceinline__ bool tile_full(const AttnArgs& a, int q0, int k0) {
  return k0 + kAttnTile - 1 <= q0 && (q0 + kAttnTile - 1 - k0 < a.window || k0 + kAttnTile - 1 < a.sinks);
}

// Bits [lo, hi) of a word, the bounds clamped to [0, 32].
__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {
  lo = max(lo, 0);
  hi = min(hi, 32);
  return hi <= lo ? 0u : (0xffffffffu >> (32 - (hi - lo))) << lo;
}

// What 32 rows of a tile of scores see of its blocks of 32 columns: nothing
// outside blocks lo .. hi - 1, all of block c where bit c of `all` is set.
struct Blocks {
  int lo, hi;
  uint32_t all;
};
constexpr Blocks kAllBlocks{0, 4, 15u};

// Masks the blocks of a tile of scores in TMEM that are neither all seen nor
// unseen: -infinity in column 32 c + j of block c where bit j of seen(c) is 0. A
// loop of its own over the few tiles at a sample's and a window's edges: masks
// woven into the unrolled arithmetic made it so long that fetching its
// instructions cost 4000 cycles a tile.
template <typename F>
__device__ __forceinline__ void mask_tile(uint32_t taddr, const Blocks& b, F seen) {
#pragma unroll 1
  for (int c = b.lo; c < b.hi; ++c) {
    if (b.all >> c & 1u) continue;
    const uint32_t m = seen(c);
    uint32_t v[32];
    tmem_ld_32x32b_x32(taddr + 32 * c, v);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (!(m >> j & 1u)) v[j] = 0xff800000u;
    tmem_st_32x32b_x32(taddr + 32 * c, v);
  }
  tmem_st_wait();
}

// Masks one block of scores the same way, by the bits of m.
__device__ __forceinline__ void mask_block(uint32_t (&v)[32], uint32_t m) {
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (!(m >> j & 1u)) v[j] = 0xff800000u;
}

// Blocks lo .. of a tile of keys from k0 (of `blocks` blocks) that 32 queries
// from q0 see; cols: score columns that have been formed.
__device__ __forceinline__ Blocks key_blocks(const AttnArgs& a, int q0, int k0, int cols, int blocks) {
  Blocks b;
  b.hi = max(0, min(min(blocks, (cols + 31) / 32), (q0 + 31 - k0) / 32 + 1));
  if (q0 + 31 < k0) b.hi = 0;
  const int first = q0 - a.window + 1 - k0;  // first column that the first query's window reaches
  b.lo = k0 < a.sinks ? 0 : min(max(first, 0) / 32, b.hi);
  b.all = 0;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (32 * c + 31 < cols && 32 * c + 31 <= q0 - k0 && (32 * c >= first + 31 || k0 + 32 * c + 31 < a.sinks)) b.all |= 1u << c;
  return b;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ uint64_t pack2(uint32_t x, uint32_t y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Columns that the products of a tile cover which only the sinks make visible.
__device__ __forceinline__ int sink_columns(const AttnArgs& a) { return (a.sinks + 31) / 32 * 32; }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A ring of equal slots that one thread fills by TMA in a fixed order of tiles
// and the MMA warp empties in the same order. Position k of that order uses
// slot k % SLOTS.
//
// A tile whose last rows belong to another sample takes a way round: its copy
// signals the slot's `raw` barrier, a warp clears those rows and then signals
// `full`. raw_phase (a bit per slot) is kept by each of the two.
template <int SLOTS>
struct Ring {
  uint32_t data, full, empty, raw, slot_bytes;
  static constexpr int BARS = 3 * SLOTS;
  __device__ __forceinline__ void init(int users) const {  // MMA warps that release a slot
    for (int i = 0; i < SLOTS; ++i) mbar_init(full + 8 * i, 1), mbar_init(empty + 8 * i, users), mbar_init(raw + 8 * i, 1);
  }
};

// A position of the ring's order: its slot, and the parity of its barriers'
// phases there.
template <int SLOTS>
struct Cursor {
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ void advance() {
    if (++slot == SLOTS) slot = 0, phase ^= 1;
  }
  __device__ __forceinline__ Cursor next() const {
    Cursor c = *this;
    c.advance();
    return c;
  }
  __device__ __forceinline__ void skip(uint32_t n) {
    slot += n;
    phase ^= slot / SLOTS & 1;
    slot %= SLOTS;
  }
  __device__ __forceinline__ uint32_t data(const Ring<SLOTS>& r) const { return r.data + slot * r.slot_bytes; }
  __device__ __forceinline__ uint32_t full(const Ring<SLOTS>& r) const { return r.full + slot * 8; }
  __device__ __forceinline__ uint32_t empty(const Ring<SLOTS>& r) const { return r.empty + slot * 8; }
  __device__ __forceinline__ uint32_t raw(const Ring<SLOTS>& r) const { return r.raw + slot * 8; }
};

// One tile of 128 tokens from `token` of head `head`: DP / 64 panels.
template <int DP>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* tm, int token, int head, uint32_t bar) {
#pragma unroll
  for (int p = 0; p < DP / 64; ++p) tma_load_3d(dst + p * (kAttnTile * 128), tm, p * 64, token, head, bar);
}

// D[128 x cols] = A B^T over DP elements, both operands K-major tiles; cols: the
// first rows of B, a multiple of 32.
// Issued by a whole warp, as all products here.
template <int DP>
__device__ __forceinline__ void mma_abt(uint32_t d_tmem, uint32_t a, uint32_t b, int cols = kAttnTile) {
  const uint32_t id = idesc_bf16(128, cols, false);
  const uint64_t da = sdesc(a, 16, 1024), db = sdesc(b, 16, 1024);
#pragma unroll
  for (int p = 0; p < DP / 64; ++p)
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
      umma_bf16_warp(d_tmem, da + (p * (kAttnTile * 128 / 16) + 2 * kk), db + (p * (kAttnTile * 128 / 16) + 2 * kk), id,
                     (p | kk) != 0 ? 1u : 0u);
}

// D[128 x DP] (+)= A B with A bf16 in TMEM (128 x 128, each 32 columns of it in 16
// TMEM columns, STEP after the 32 before) and B a tile whose 128 rows are the
// inner dimension.
template <int DP, int STEP>
__device__ __forceinline__ void mma_ab(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, bool add) {
  const uint32_t id = idesc_bf16(128, DP, true);
  const uint64_t db = sdesc(b, kAttnTile * 128, 1024);
#pragma unroll
  for (int ks = 0; ks < 8; ++ks)
    umma_bf16_ts_warp(d_tmem, a_tmem + (ks >> 1) * STEP + (ks & 1) * 8, db + 128u * ks, id,
                      ks != 0 ? 1u : (uint32_t)add);
}
// The same with an inner dimension of `cols`, a multiple of 32.
template <int DP, int STEP>
__device__ __forceinline__ void mma_ab_few(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, bool add, int cols) {
  const uint32_t id = idesc_bf16(128, DP, true);
  const uint64_t db = sdesc(b, kAttnTile * 128, 1024);
#pragma unroll 1
  for (int ks = 0; ks * 16 < cols; ++ks)
    umma_bf16_ts_warp(d_tmem, a_tmem + (ks >> 1) * STEP + (ks & 1) * 8, db + 128u * ks, id, add || ks != 0);
}

// Columns c0 .. c1 - 1 (multiples of 32) of this thread's row of an accumulator
// in TMEM, times f and rounded to bf16, to its row of the output; zero: zeros, TMEM
// holds nothing. `wide`: rows lie on 32-byte boundaries, and a lane stores whole
// 32-byte sectors. For tiles with rows of other samples: each row is a line of its
// own, and the 128 rows of a CTA take 3000 cycles to leave.
__device__ __forceinline__ void store_row(uint32_t taddr, int c0, int c1, float f, bool zero, __nv_bfloat16* out, bool mine,
                                          int dim, bool wide) {
#pragma unroll 1
  for (int c = c0; c < c1; c += 32) {
    uint32_t r[16];
    if (!zero) {
      uint32_t o[32];
      tmem_ld_32x32b_x32(taddr + c, o);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 16; ++j) r[j] = op_pack_bf16(__uint_as_float(o[2 * j]) * f, __uint_as_float(o[2 * j + 1]) * f);
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) r[j] = 0u;
    }
    if (!mine) continue;
    if (wide) {
#pragma unroll
      for (int j = 0; j < 16; j += 8)
        if (c + 2 * j < dim)
          asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out + c + 2 * j), "r"(r[j]),
                       "r"(r[j + 1]), "r"(r[j + 2]), "r"(r[j + 3]), "r"(r[j + 4]), "r"(r[j + 5]), "r"(r[j + 6]),
                       "r"(r[j + 7])
                       : "memory");
    } else {
#pragma unroll
      for (int j = 0; j < 16; j += 4)
        if (c + 2 * j < dim) *reinterpret_cast<uint4*>(out + c + 2 * j) = make_uint4(r[j], r[j + 1], r[j + 2], r[j + 3]);
    }
  }
}
// Rows of `dim` elements from p on are on 32-byte boundaries.
__device__ __forceinline__ bool rows_wide(const void* p, int dim) {
  return dim % 16 == 0 && (reinterpret_cast<uintptr_t>(p) & 31) == 0;
}

// The same to a tile in shared memory, laid out as TMA reads it, for tiles whose
// rows all belong to the sample: a position of the ring that no load fills. The
// threads go on at once, a warp without other work hands the tile to TMA and frees
// the position when it has been read. (At 16384 tokens of 16 heads of 128, window
// 1024, the gradient kernel takes 391 us, with rows stored by their threads 426.)
__device__ __forceinline__ void stage_row(uint32_t taddr, int c0, int c1, float f, bool zero, uint32_t tile, int row) {
#pragma unroll 1
  for (int c = c0; c < c1; c += 32) {
    uint32_t o[32];
    if (!zero) {
      tmem_ld_32x32b_x32(taddr + c, o);
      tmem_ld_wait();
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] = 0u;
    }
    const uint32_t at = tile + (c >> 6) * (kAttnTile * 128) + row * 128, first = (c & 63) >> 3;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t r[4];
#pragma unroll
      for (int x = 0; x < 4; ++x)
        r[x] = op_pack_bf16(__uint_as_float(o[8 * j + 2 * x]) * f, __uint_as_float(o[8 * j + 2 * x + 1]) * f);
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + (((first + j) ^ (row & 7)) << 4)), "r"(r[0]),
                   "r"(r[1]), "r"(r[2]), "r"(r[3])
                   : "memory");
    }
  }
  fence_proxy_async_smem();
}

// An asynchronous copy of four bytes to shared memory (zero where !on), and the
// arrival on a barrier when this thread's copies have landed.
__device__ __forceinline__ void copy4(uint32_t dst, const float* src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(on ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Zeros in the rows of a tile from `rows` on, by a whole warp: tokens there
// belong to another sample, and a product with a zero weight must not take a
// NaN or an infinity from them. A warp of its own does this, for a sample's
// last tile only; the products wait for it there.
template <int DP>
__device__ __forceinline__ void clear_rows(uint32_t tile, int rows, int lane) {
  for (int i = rows * 8 + lane; i < kAttnTile * 8; i += 32) {
#pragma unroll
    for (int p = 0; p < DP / 64; ++p)
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + p * (kAttnTile * 128) + i * 16), "r"(0)
                   : "memory");
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// Fills a position of the ring (one lane issues; the slot is free): `valid` rows
// of the tile belong to the sample.
template <int DP, int SLOTS>
__device__ __forceinline__ void fill_slot(const Ring<SLOTS>& ring, const Cursor<SLOTS>& k, const CUtensorMap* tm,
                                          int token, int head, int valid, uint32_t& raw_phase) {
  const bool ragged = valid < kAttnTile;
  const uint32_t bar = ragged ? k.raw(ring) : k.full(ring);
  mbar_expect_tx(bar, ring.slot_bytes);
  load_tile<DP>(k.data(ring), tm, token, head, bar);
  if (ragged) raw_phase ^= 1u << k.slot;
}

// The clearing warp's part for a ragged tile.
template <int DP, int SLOTS>
__device__ __forceinline__ bool clear_slot(const Ring<SLOTS>& ring, const Cursor<SLOTS>& k, int valid,
                                           uint32_t& raw_phase, int lane, volatile int* abort_flag, int* err,
                                           int code) {
  if (!mbar_wait_warp(k.raw(ring), raw_phase >> k.slot & 1, abort_flag, err, code)) return false;
  raw_phase ^= 1u << k.slot;
  clear_rows<DP>(k.data(ring), valid, lane);
  if (lane == 0) mbar_arrive(k.full(ring));
  return true;
}

// A staged tile's position: the warps that write it wait for `full`, which the
// producer grants by itself, and arrive on `staged`; this warp then stores the tile
// and frees the position for the `users` of a slot.
template <int DP, int SLOTS>
__device__ __forceinline__ bool store_slot(const Ring<SLOTS>& ring, const Cursor<SLOTS>& k, uint32_t staged,
                                           uint32_t& staged_phase, const CUtensorMap* tm, int token, int head, int users,
                                           int lane, volatile int* abort_flag, int* err, int code) {
  if (!mbar_wait_warp(staged + 8 * k.slot, staged_phase >> k.slot & 1, abort_flag, err, code)) return false;
  staged_phase ^= 1u << k.slot;
  if (lane == 0) {
#pragma unroll
    for (int p = 0; p < DP / 64; ++p) tma_store_3d(tm, k.data(ring) + p * (kAttnTile * 128), p * 64, token, head);
    bulk_commit();
    bulk_wait_read_all();
    for (int u = 0; u < users; ++u) mbar_arrive(k.empty(ring));
  }
  __syncwarp();
  return true;
}

// Every copy of the ring has landed, `cur` being the first position not filled:
// the last of each slot, to either barrier. (A slot never filled waits for
// nothing. Where the CTA gave up, a cleared tile's `full` may never come; the
// wait for it is bounded like any other.)
template <int SLOTS>
__device__ __forceinline__ void drain_ring(const Ring<SLOTS>& ring, const Cursor<SLOTS>& cur, uint32_t raw_phase) {
  for (uint32_t s = 0; s < SLOTS; ++s) {
    drain_wait(ring.raw + 8 * s, (raw_phase >> s & 1) ^ 1);
    // slots before the cursor were filled in its own round, the others in the round before
    drain_wait(ring.full + 8 * s, s < cur.slot ? cur.phase : cur.phase ^ 1);
  }
}

}  // namespace
#endif

}  // namespace ma
