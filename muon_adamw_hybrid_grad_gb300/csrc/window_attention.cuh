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
  const float* lse2;        // gradient: lse * log2(e), +infinity for a query that sees nothing [head][token]
  const float* delta;       // gradient: dout . out [head][token]
};

// A 3-D map (element, token, head) of a bf16 tensor with 64 x 128 x 1 boxes in
// the 128-byte swizzle: a tile is one or two panels of 64 elements by 128
// tokens. Elements past head_dim and tokens past n read as zero.
bool attn_map(CUtensorMap* tm, const void* base, int dim, int64_t tokens, int64_t heads, int64_t token_stride,
              int64_t head_stride);

cudaError_t attn_forward(const AttnArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                         __nv_bfloat16* out, float* lse, int* err, int sms, cudaStream_t st);

struct AttnGrad {
  const __nv_bfloat16 *dout, *out;
  int64_t do_ts, do_hs;
  const float* lse;
  float *lse2, *delta, *partial;
  int64_t partial_slots;
  __nv_bfloat16 *dq, *dk, *dv;
};
cudaError_t attn_backward(AttnArgs a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                          const CUtensorMap& dout, const AttnGrad& g, int* err, int sms, cudaStream_t st);

// Query tiles of a chunk of the gradient for sink keys (see window_dkv_kernel).
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

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A ring of equal slots that one thread fills by TMA in a fixed order of tiles
// and the MMA warp empties in the same order. Position k of that order uses
// slot k % SLOTS.
template <int SLOTS>
struct Ring {
  uint32_t data, full, empty, slot_bytes;
  __device__ __forceinline__ uint32_t slot(uint32_t k) const { return data + (k % SLOTS) * slot_bytes; }
  __device__ __forceinline__ uint32_t full_bar(uint32_t k) const { return full + (k % SLOTS) * 8; }
  __device__ __forceinline__ uint32_t empty_bar(uint32_t k) const { return empty + (k % SLOTS) * 8; }
  __device__ __forceinline__ uint32_t full_parity(uint32_t k) const { return (k / SLOTS) & 1; }
  // of the wait before position k is filled (its slot's last user has finished)
  __device__ __forceinline__ uint32_t empty_parity(uint32_t k) const { return ((k / SLOTS) & 1) ^ 1; }
};

// One tile of 128 tokens from `token` of head `head`: DP / 64 panels.
template <int DP>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* tm, int token, int head, uint32_t bar) {
#pragma unroll
  for (int p = 0; p < DP / 64; ++p) tma_load_3d(dst + p * (kAttnTile * 128), tm, p * 64, token, head, bar);
}

// D[128 x 128] = A B^T over DP elements, both operands K-major tiles.
template <int DP>
__device__ __forceinline__ void mma_abt(uint32_t d_tmem, uint32_t a, uint32_t b) {
  const uint32_t id = idesc_bf16(128, 128, false);
#pragma unroll
  for (int p = 0; p < DP / 64; ++p) {
    const uint64_t da = sdesc(a + p * (kAttnTile * 128), 16, 1024), db = sdesc(b + p * (kAttnTile * 128), 16, 1024);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) umma_bf16<1>(d_tmem, da + 2u * kk, db + 2u * kk, id, (p | kk) != 0 ? 1u : 0u);
  }
}

// D[128 x DP] (+)= A B with A bf16 in TMEM (128 x 128: 64 columns, the second
// half of them `half_step` columns after the first) and B a tile whose 128
// rows are the inner dimension.
template <int DP>
__device__ __forceinline__ void mma_ab(uint32_t d_tmem, uint32_t a_tmem, uint32_t half_step, uint32_t b, bool add) {
  const uint32_t id = idesc_bf16(128, DP, true);
  const uint64_t db = sdesc(b, kAttnTile * 128, 1024);
#pragma unroll
  for (int ks = 0; ks < 8; ++ks)
    umma_bf16_ts(d_tmem, a_tmem + (ks >> 2) * half_step + (ks & 3) * 8, db + 128u * ks, id, (add || ks != 0) ? 1u : 0u);
}

// Zeros in the rows of a tile from `rows` on, by a whole warp: tokens there
// belong to another sample, and a product with a zero weight must not take a
// NaN or an infinity from them.
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

}  // namespace
#endif

}  // namespace ma
