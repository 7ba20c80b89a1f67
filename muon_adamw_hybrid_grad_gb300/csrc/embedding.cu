// Embedding lookup with scaling, and its dense gradient from sorted tokens.
//
//   out[t]  = scale * weight[ids[t]]                    (zero where ids[t] is no row)
//   grad[v] = scale * sum over {t : ids[t] = v} dout[t]  (+ grad[v] when accumulating)
//
// The gradient is deterministic: each id's rows are added in the order of their
// positions (within groups of fixed size) in fp32. Two ways lead there:
//   - up to kDirectTokens tokens, one launch: every block owns some rows of the
//     gradient, picks their tokens out of all ids and writes each row once;
//   - more tokens: a stable radix sort brings the tokens into the order
//     (id, position), then runs of equal ids are added up.
#include <limits.h>

#include "op_common.cuh"

namespace ma {
namespace {

constexpr int kThreads = 256;

// ids as written by the caller: int32 or int64. Anything outside [0, vocab) is
// no token and maps to `vocab`.
__device__ __forceinline__ uint32_t read_id(const void* ids, bool wide, int64_t t, uint32_t vocab) {
  const int64_t v = wide ? static_cast<const int64_t*>(ids)[t] : (int64_t)static_cast<const int32_t*>(ids)[t];
  return (v < 0 || v >= (int64_t)vocab) ? vocab : (uint32_t)v;
}

// ---- lookup ----
// blockDim.x threads take VEC columns each, blockDim.y token groups of ROWS
// tokens whose rows are loaded before any is stored. Bound by HBM: 65521 tokens of
// 2048 bf16 columns, ids drawn by a Zipf law, take 64 us (5.3 TB/s of distinct rows
// read and rows written, 0.78 of the measured copy bandwidth; each repeated row is
// read from L2 again); 61 tokens of 256 columns 3.7 us, the launch.
template <typename W, typename O, int VEC>
__global__ void __launch_bounds__(kThreads) embedding_kernel(const W* __restrict__ weight, int64_t wstride,
                                                             uint32_t vocab, int width, const void* __restrict__ ids,
                                                             int wide, int64_t n, float scale, O* __restrict__ out,
                                                             int64_t ostride) {
  constexpr int ROWS = 4;
  pdl_launch();
  pdl_wait();
  const int64_t t0 = ((int64_t)blockIdx.x * blockDim.y + threadIdx.y) * ROWS;
  uint32_t id[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) id[r] = t0 + r < n ? read_id(ids, wide != 0, t0 + r, vocab) : vocab;
  for (int c = (int)(threadIdx.x + blockDim.x * blockIdx.y) * VEC; c < width; c += (int)(blockDim.x * gridDim.y) * VEC) {
    RawVec<W, VEC> raw[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
      if (id[r] < vocab) raw[r].load(weight + (int64_t)id[r] * wstride + c);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      if (t0 + r >= n) break;
      float x[VEC];
      raw[r].get(x);
#pragma unroll
      for (int i = 0; i < VEC; ++i) x[i] = id[r] < vocab ? x[i] * scale : 0.f;
      store_vec<VEC>(out + (t0 + r) * ostride + c, x);
    }
  }
}

// ---- gradient of few tokens: one launch ----
// Blocks b + B y own rows b, b + B, b + 2 B, ... (neighbouring ids are of like
// frequency in most vocabularies, so consecutive rows would load the first
// blocks with all the frequent ones) and the 32 VEC columns of slab y. Their
// warps read all ids, each a contiguous part, and keep the tokens of the block's
// rows in order; then every row is written once: zeros, or the sum over its
// tokens, eight rows of dout in flight. A warp takes a row of up to kFewTokens
// tokens; the warps share a row of more, each the part of its own ids.
//
// Bound by the writes of a dense gradient: 93 us for 16 tokens of 151936 x 2048
// (bf16, 6.7 TB/s). Against the sorted form, ids drawn by a Zipf law: 6.2 us (22)
// at 1024 tokens of 1000 x 256, 105 (119) at 1024 of 151936 x 2048, 117 (122) at
// 4096 of these. Where all tokens have one id its row's block takes longest: 113
// (117) at 1024, 172 (126) at 4096. Past that the reading of all ids by all blocks
// costs more than the sort.
constexpr int kDirectTokens = 4096;
constexpr int kDirectRows = 4096;  // rows of a block, at most: its counters lie in shared memory
constexpr int kDirectWarps = kThreads / 32;
constexpr uint32_t kFewTokens = 16;

struct DirectArgs {
  const void* ids;
  int wide, n;
  uint32_t vocab;
  int width;
  float scale;
  int accumulate;
  int64_t dstride, gstride;
};

template <typename D, typename G, int VEC>
__global__ void __launch_bounds__(kThreads) embedding_direct_kernel(const __grid_constant__ DirectArgs a,
                                                                    const D* __restrict__ dout, G* __restrict__ grad) {
  extern __shared__ uint32_t list[];  // [warp][per]: row of the block << 12 | position; then a counter per row
  __shared__ int count[kDirectWarps];
  __shared__ float sums[kDirectWarps][32][VEC + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t B = gridDim.x, b = blockIdx.x;
  const int rows = (int)((a.vocab - b + B - 1) / B);
  const int per = ((a.n + kDirectWarps - 1) / kDirectWarps + 31) / 32 * 32;
  uint32_t* tokens = list + kDirectWarps * per;
  for (int i = threadIdx.x; i < rows; i += kThreads) tokens[i] = 0;
  __syncthreads();
  pdl_launch();
  pdl_wait();
  {
    constexpr int AHEAD = 4;
    uint32_t* mine = list + warp * per;
    int found = 0;
    const int t1 = min((warp + 1) * per, a.n);
    for (int t0 = warp * per; t0 < t1; t0 += 32 * AHEAD) {
      uint32_t id[AHEAD];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int t = t0 + 32 * u + lane;
        id[u] = t < t1 ? read_id(a.ids, a.wide != 0, t, a.vocab) : a.vocab;
      }
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const uint32_t r = id[u] / B;
        const bool hit = id[u] < a.vocab && id[u] - r * B == b;
        const uint32_t hits = __ballot_sync(0xffffffffu, hit);
        if (hit) {
          mine[found + __popc(hits & ((1u << lane) - 1))] = r << 12 | (uint32_t)(t0 + 32 * u + lane);
          atomicAdd(tokens + r, 1u);
        }
        found += __popc(hits);
      }
    }
    if (lane == 0) count[warp] = found;
  }
  __syncthreads();
  const int c = (int)(blockIdx.y * 32 + lane) * VEC;
  // s += the rows of the tokens of the block's row r in list q, in order
  auto add_list = [&](float (&s)[VEC], uint32_t r, int q) {
    for (int e0 = 0; e0 < count[q]; e0 += 32) {
      const uint32_t entry = e0 + lane < count[q] ? list[q * per + e0 + lane] : UINT_MAX;
      uint32_t hits = __ballot_sync(0xffffffffu, (entry >> 12) == r && e0 + lane < count[q]);
      while (hits) {
        RawVec<D, VEC> raw[8];
        int m = 0;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          if (hits) {
            const int t = (int)(__shfl_sync(0xffffffffu, entry, __ffs(hits) - 1) & 4095u);
            hits &= hits - 1;
            if (c < a.width) raw[u].load(dout + (int64_t)t * a.dstride + c);
            ++m;
          }
        }
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (u < m) {
            float x[VEC];
            raw[u].get(x);
#pragma unroll
            for (int i = 0; i < VEC; ++i) s[i] += x[i];
          }
      }
    }
  };
  auto write = [&](uint32_t r, const float (&s)[VEC]) {
    if (c >= a.width) return;
    G* p = grad + (int64_t)(b + r * B) * a.gstride + c;
    float y[VEC];
    if (a.accumulate) {
      load_vec<VEC>(p, y);
#pragma unroll
      for (int i = 0; i < VEC; ++i) y[i] = fmaf(s[i], a.scale, y[i]);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) y[i] = s[i] * a.scale;
    }
    store_vec<VEC>(p, y);
  };
  // rows of no token, whole ones shared out over the slabs, and of few: every eighth row to a warp (the first rows of
  // a block are those of the most frequent ids)
  for (int r0 = 0; r0 < rows; r0 += 32 * kDirectWarps) {
    const int row = r0 + lane * kDirectWarps + warp;
    const uint32_t mine = row < rows ? tokens[row] : UINT_MAX;
    if (!a.accumulate) {
      float zero[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) zero[i] = 0.f;
      const bool ours = mine == 0u && (row / kDirectWarps) % gridDim.y == blockIdx.y;
      for (uint32_t left = __ballot_sync(0xffffffffu, ours); left; left &= left - 1) {
        const uint32_t r = r0 + (__ffs(left) - 1) * kDirectWarps + warp;
        G* p = grad + (int64_t)(b + r * B) * a.gstride;
        for (int x = lane * VEC; x < a.width; x += 32 * VEC) store_vec<VEC>(p + x, zero);
      }
    }
    for (uint32_t left = __ballot_sync(0xffffffffu, mine >= 1u && mine <= kFewTokens); left; left &= left - 1) {
      const uint32_t r = r0 + (__ffs(left) - 1) * kDirectWarps + warp;
      float s[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) s[i] = 0.f;
      for (int q = 0; q < kDirectWarps; ++q) add_list(s, r, q);
      write(r, s);
    }
  }
  // rows of many, by all warps
  for (int r0 = 0; r0 < rows; r0 += 32) {
    for (uint32_t left = __ballot_sync(0xffffffffu, r0 + lane < rows && tokens[r0 + lane] > kFewTokens); left;
         left &= left - 1) {
      const uint32_t r = r0 + __ffs(left) - 1;
      float s[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) s[i] = 0.f;
      add_list(s, r, warp);
#pragma unroll
      for (int i = 0; i < VEC; ++i) sums[warp][lane][i] = s[i];
      __syncthreads();
      if (warp == 0) {
#pragma unroll
        for (int q = 1; q < kDirectWarps; ++q)
#pragma unroll
          for (int i = 0; i < VEC; ++i) s[i] += sums[q][lane][i];
        write(r, s);
      }
      __syncthreads();
    }
  }
}

// ---- gradient: sort, then sum ----
// The first cluster sorts the tokens by id (stable least-significant-digit
// radix sort over the cluster's CTAs, digit totals exchanged through
// distributed shared memory); every other CTA meanwhile fills the gradient
// with zeros, which hides the sort behind the writes of a large vocabulary: 105 us
// for 151936 x 2048 in bf16 (5.9 TB/s, where the one-launch form writes the same
// zeros at 6.7; why has not been found), the sort of 32749 ids among them. The sums
// then take 35 us and the joins 16. (Zeros shared out over all three launches, so
// that the sums read beside them: 153 to 158 us in all, as against 156.) With
// accumulate there are no zeros and the sort stands alone: 89 us at 32749 tokens,
// 33 at 4097; the one-launch form 36 at 4096, 20 at 777.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortCluster = 8;
constexpr int kDigitBits = 9;  // two passes cover ids below 2^18
constexpr int kDigits = 1 << kDigitBits;
constexpr size_t kSortSmem = (size_t)kSortWarps * kDigits * 4 + 2 * kDigits * 4 + 64 * 4;

struct SortArgs {
  const void* ids;
  int wide;
  int64_t n;
  uint32_t vocab;
  int passes, bits;            // digits of `bits` bits
  uint32_t *key0, *pos0, *key1, *pos1;  // ping-pong buffers; the last pass writes key0/pos0
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t ld_dsmem(const uint32_t* p, uint32_t rank) {
  uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), r, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(r) : "memory");
  return v;
}

__device__ void sort_tokens(const SortArgs& a, uint32_t* sm) {
  uint32_t* hist = sm;                             // [warp][digit]
  uint32_t* total = sm + kSortWarps * kDigits;     // this CTA's count of each digit
  uint32_t* wsum = total + 2 * kDigits;            // block scan
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  // contiguous runs of whole 32-token groups: CTA, then warp
  const int64_t groups = (a.n + 31) / 32;
  const int64_t per_cta = (groups + kSortCluster - 1) / kSortCluster;
  const int64_t per_warp = (per_cta + kSortWarps - 1) / kSortWarps;
  int64_t g0 = (int64_t)rank * per_cta + warp * per_warp;
  int64_t g1 = min(min(g0 + per_warp, (int64_t)(rank + 1) * per_cta), groups);
  for (int pass = 0; pass < a.passes; ++pass) {
    const bool first = pass == 0;
    // the last pass writes buffer 0, so the one before it writes buffer 1
    const bool to0 = ((a.passes - 1 - pass) & 1) == 0;
    const uint32_t* skey = to0 ? a.key1 : a.key0;
    const uint32_t* spos = to0 ? a.pos1 : a.pos0;
    uint32_t* dkey = to0 ? a.key0 : a.key1;
    uint32_t* dpos = to0 ? a.pos0 : a.pos1;
    const int shift = pass * a.bits;
    const uint32_t mask = (1u << a.bits) - 1;
    for (int i = tid; i < kSortWarps * kDigits; i += kSortThreads) hist[i] = 0;
    __syncthreads();
    uint32_t* mine = hist + warp * kDigits;
    for (int64_t g = g0; g < g1; ++g) {
      const int64_t t = g * 32 + lane;
      if (t < a.n) {
        const uint32_t key = first ? read_id(a.ids, a.wide != 0, t, a.vocab) : __ldcg(skey + t);
        atomicAdd(mine + ((key >> shift) & mask), 1u);
      }
    }
    __syncthreads();
    // per digit: exclusive scan over this CTA's warps, and the CTA's total
    if (tid < kDigits) {
      uint32_t s = 0;
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = hist[w * kDigits + tid];
        hist[w * kDigits + tid] = s;
        s += c;
      }
      total[tid] = s;
    }
    cluster_barrier();
    // digits below this one over the whole cluster, plus this digit in lower CTAs
    uint32_t all = 0, lower = 0;
    if (tid < kDigits) {
      for (int r = 0; r < kSortCluster; ++r) {
        const uint32_t c = ld_dsmem(total + tid, r);
        if (r < (int)rank) lower += c;
        all += c;
      }
    }
    uint32_t incl = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    if (warp == 0) {
      uint32_t w = wsum[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
      }
      wsum[32 + lane] = w;
    }
    __syncthreads();
    if (tid < kDigits) {
      const uint32_t base = incl - all + (warp > 0 ? wsum[32 + warp - 1] : 0) + lower;
      for (int w = 0; w < kSortWarps; ++w) hist[w * kDigits + tid] += base;
    }
    __syncthreads();
    for (int64_t g = g0; g < g1; ++g) {
      const int64_t t = g * 32 + lane;
      const bool on = t < a.n;
      uint32_t key = 0, pos = 0;
      if (on) {
        key = first ? read_id(a.ids, a.wide != 0, t, a.vocab) : __ldcg(skey + t);
        pos = first ? (uint32_t)t : __ldcg(spos + t);
      }
      const uint32_t d = (key >> shift) & mask;
      const uint32_t peers = __match_any_sync(0xffffffffu, on ? d : 0xffffffffu);
      const uint32_t before = __popc(peers & ((1u << lane) - 1));
      uint32_t at = 0;
      if (on) at = mine[d] + before;
      __syncwarp();
      if (on) {
        if (before == 0) mine[d] += __popc(peers);
        dkey[at] = key;
        dpos[at] = pos;
      }
      __syncwarp();
    }
    // the cluster's writes are visible to the cluster after its barrier
    __threadfence();
    cluster_barrier();
  }
}

__global__ void __launch_bounds__(kSortThreads) embedding_sort_kernel(const __grid_constant__ SortArgs a,
                                                                      uint8_t* __restrict__ grad, int64_t row_bytes,
                                                                      int64_t stride_bytes, int64_t rows, int vec) {
  extern __shared__ __align__(16) uint32_t sort_sm[];
  pdl_launch();
  pdl_wait();
  if (blockIdx.x < kSortCluster) {
    sort_tokens(a, sort_sm);
  } else {
    const int64_t nth = (int64_t)(gridDim.x - kSortCluster) * kSortThreads;
    const int64_t me = (int64_t)(blockIdx.x - kSortCluster) * kSortThreads + threadIdx.x;
    if (stride_bytes == row_bytes) row_bytes *= rows, stride_bytes = row_bytes, rows = 1;
    const int unit = vec ? 16 : 2;
    const int64_t per_row = row_bytes / unit;
    if (rows == 1) {
      for (int64_t i = me; i < per_row; i += nth) {
        if (vec)
          reinterpret_cast<uint4*>(grad)[i] = make_uint4(0, 0, 0, 0);
        else
          reinterpret_cast<uint16_t*>(grad)[i] = 0;
      }
    } else {
      // a CTA to a row, so that no index is divided
      for (int64_t r = blockIdx.x - kSortCluster; r < rows; r += gridDim.x - kSortCluster) {
        uint8_t* row = grad + r * stride_bytes;
        for (int64_t i = threadIdx.x; i < per_row; i += kSortThreads) {
          if (vec)
            reinterpret_cast<uint4*>(row)[i] = make_uint4(0, 0, 0, 0);
          else
            reinterpret_cast<uint16_t*>(row)[i] = 0;
        }
      }
    }
  }
}

// Sums of dout over runs of equal ids. Bound by reading dout: 121 MB in 35 us. (Chunks
// of 8 or 32 tokens, 4 or 16 loads in flight, or more blocks an SM: 0 to 8 us more.)
// A chunk of kChunkTokens sorted tokens belongs
// to one row of threads; a run inside it is written to the gradient at once,
// a run that reaches over a border leaves fp32 partial sums: slot 0 of a chunk
// holds the run that came in from the chunk before, slot 1 the run that starts
// here and goes on.
constexpr int kChunkTokens = 16;

struct SumArgs {
  const uint32_t *key, *pos;
  int64_t n;
  uint32_t vocab;
  int width;
  float scale;
  int accumulate;
  int64_t dstride, gstride;
  float* partial;  // [chunk][2][width]
};

template <int VEC, typename G>
__device__ __forceinline__ void write_grad(G* grad, const SumArgs& a, uint32_t key, int c, const float (&s)[VEC]) {
  float y[VEC];
  G* p = grad + (int64_t)key * a.gstride + c;
  if (a.accumulate) {
    load_vec<VEC>(p, y);
#pragma unroll
    for (int i = 0; i < VEC; ++i) y[i] = fmaf(s[i], a.scale, y[i]);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) y[i] = s[i] * a.scale;
  }
  store_vec<VEC>(p, y);
}

template <typename D, typename G, int VEC>
__global__ void __launch_bounds__(kThreads) embedding_sum_kernel(const __grid_constant__ SumArgs a,
                                                                 const D* __restrict__ dout, G* __restrict__ grad) {
  constexpr int AHEAD = 8;
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t chunk = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const int64_t t0 = chunk * kChunkTokens;
  if (t0 >= a.n) return;  // the same for a whole warp
  const int m = (int)min((int64_t)kChunkTokens, a.n - t0);
  // the chunk's ids and positions, a lane to a token, and the ids beside it
  const uint32_t my_key = lane < m ? a.key[t0 + lane] : a.vocab, my_pos = lane < m ? a.pos[t0 + lane] : 0;
  const uint32_t before = t0 > 0 ? a.key[t0 - 1] : UINT_MAX;
  const uint32_t after = t0 + m < a.n ? a.key[t0 + m] : UINT_MAX;
  const int c = (int)(threadIdx.x + blockDim.x * blockIdx.y) * VEC;
  float* part = a.partial + chunk * 2 * a.width + c;
  float s[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) s[i] = 0.f;
  uint32_t cur = __shfl_sync(0xffffffffu, my_key, 0);
  bool came_in = cur == before;
  for (int t = 0; t < m && cur < a.vocab; t += AHEAD) {
    RawVec<D, VEC> raw[AHEAD];
    uint32_t key[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      key[u] = __shfl_sync(0xffffffffu, my_key, t + u);
      const uint32_t pos = __shfl_sync(0xffffffffu, my_pos, t + u);
      if (key[u] < a.vocab && c < a.width) raw[u].load(dout + (int64_t)pos * a.dstride + c);
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      if (t + u >= m) break;
      if (key[u] != cur) {
        if (c < a.width) {
          if (came_in)
            store_vec<VEC>(part, s);
          else
            write_grad<VEC>(grad, a, cur, c, s);
        }
        came_in = false;
        cur = key[u];
        if (cur >= a.vocab) break;  // ids of no token are last
#pragma unroll
        for (int i = 0; i < VEC; ++i) s[i] = 0.f;
      }
      float x[VEC];
      raw[u].get(x);
#pragma unroll
      for (int i = 0; i < VEC; ++i) s[i] += x[i];
    }
  }
  if (cur < a.vocab && c < a.width) {
    if (came_in)
      store_vec<VEC>(part, s);
    else if (cur == after)
      store_vec<VEC>(part + a.width, s);
    else
      write_grad<VEC>(grad, a, cur, c, s);
  }
}

constexpr int kJoinChunks = 8;  // chunks of a block

// Joins the runs that reach over a border, at the chunk where they start. A warp
// takes 32 VEC columns of one or two such slabs, and the block's other warps walk
// along with it: each takes every WALKERS-th partial sum of the run,
// four of them in flight, and the walkers' sums are added in their order.
template <typename G, int VEC>
__global__ void __launch_bounds__(kThreads) embedding_join_kernel(const __grid_constant__ SumArgs a,
                                                                  G* __restrict__ grad, int slabs) {
  constexpr int WARPS = kThreads / 32, AHEAD = 4;
  __shared__ float sums[WARPS][32][VEC + 1];
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, slab = warp % slabs, walker = warp / slabs;
  const int walkers = WARPS / slabs;
  const int c = (lane + 32 * (slab + slabs * (int)blockIdx.y)) * VEC;
  // which of this block's chunks start a run that goes on
  bool starts = false;
  {
    const int64_t t0 = ((int64_t)blockIdx.x * kJoinChunks + lane) * kChunkTokens, t1 = t0 + kChunkTokens;
    if (lane < kJoinChunks && t1 < a.n) {
      const uint32_t first = a.key[t0], cur = a.key[t1 - 1], next = a.key[t1];
      const uint32_t before = t0 > 0 ? a.key[t0 - 1] : UINT_MAX;
      starts = cur < a.vocab && next == cur && !(before == cur && first == cur);
    }
  }
  for (uint32_t left = __ballot_sync(0xffffffffu, starts); left; left &= left - 1) {
    const int64_t chunk = (int64_t)blockIdx.x * kJoinChunks + __ffs(left) - 1;
    const uint32_t cur = a.key[(chunk + 1) * kChunkTokens];
    // the first chunk behind the run, looked for 32 chunks at a time
    int64_t end = chunk + 1;
    for (uint32_t same = 0xffffffffu; same == 0xffffffffu;) {
      const int64_t at = (end + lane) * kChunkTokens;
      same = __ballot_sync(0xffffffffu, at < a.n && a.key[at] == cur);
      end += __ffs(~same) ? __ffs(~same) - 1 : 32;
    }
    float s[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) s[i] = 0.f;
    if (c < a.width) {
      if (walker == 0) load_vec<VEC>(a.partial + (chunk * 2 + 1) * a.width + c, s);
      for (int64_t k = chunk + 1 + walker; k < end; k += AHEAD * walkers) {
        float y[AHEAD][VEC];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
          if (k + u * walkers < end) load_vec<VEC>(a.partial + (k + u * walkers) * 2 * a.width + c, y[u]);
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
          if (k + u * walkers < end) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) s[i] += y[u][i];
          }
      }
    }
    if (walkers > 1) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) sums[warp][lane][i] = s[i];
      __syncthreads();
      if (walker == 0)
        for (int w = 1; w < walkers; ++w)
#pragma unroll
          for (int i = 0; i < VEC; ++i) s[i] += sums[w * slabs + slab][lane][i];
      __syncthreads();
    }
    if (walker == 0 && c < a.width) write_grad<VEC>(grad, a, cur, c, s);
  }
}

// ---- host ----
struct Plan {
  int64_t chunks;
  int64_t key_bytes, bytes;
};

Plan plan_backward(int64_t n, int64_t width) {
  Plan p;
  p.chunks = (n + kChunkTokens - 1) / kChunkTokens;
  p.key_bytes = (n * 4 + 255) / 256 * 256;
  p.bytes = 4 * p.key_bytes + p.chunks * 2 * ((width + 7) / 8 * 8) * 4 + 256;
  return p;
}

// Threads of a block: x over the columns, y over rows.
dim3 block_of(int64_t width, int vec) {
  int64_t cols = (width + vec - 1) / vec;
  int x = 32;
  while (x < kThreads && x < cols) x *= 2;
  return dim3((unsigned)x, (unsigned)(kThreads / x));
}

ma_status check_rows(const char* what, const void* p, int dt, int64_t stride, int64_t width, int64_t rows) {
  if (!op_dtype_ok(dt)) return op_fail(MA_ERR_DTYPE, "%s: dtype %d is neither MA_DT_F32 nor MA_DT_BF16", what, dt);
  if (rows > 0 && !p) return op_fail(MA_ERR_ARG, "%s must not be NULL", what);
  if (!op_aligned(p, op_dtype_size(dt))) return op_fail(MA_ERR_ALIGN, "%s is not aligned to its element size", what);
  if (stride < width) return op_fail(MA_ERR_SHAPE, "%s: row stride %lld below the width", what, (long long)stride);
  return MA_OK;
}

ma_status check_common(int64_t vocab, int64_t width, const void* ids, int id_bytes, int64_t n, double scale) {
  if (vocab < 1 || vocab > ((int64_t)1 << 30)) return op_fail(MA_ERR_SHAPE, "vocab outside [1, 2^30]");
  if (width < 1 || width > ((int64_t)1 << 20)) return op_fail(MA_ERR_SHAPE, "width outside [1, 2^20]");
  if (n < 0 || n > ((int64_t)1 << 30)) return op_fail(MA_ERR_SHAPE, "n_tokens outside [0, 2^30]");
  if (id_bytes != 4 && id_bytes != 8) return op_fail(MA_ERR_ARG, "id_bytes must be 4 or 8");
  if (n > 0 && !ids) return op_fail(MA_ERR_ARG, "ids must not be NULL");
  if (!op_aligned(ids, id_bytes)) return op_fail(MA_ERR_ALIGN, "ids are not aligned to their size");
  if (!(scale - scale == 0.0)) return op_fail(MA_ERR_ARG, "scale must be finite");
  return MA_OK;
}

// 8-element accesses: whole vectors, and rows on 16-byte boundaries. (65536 tokens of
// 2048 columns: 82 us, of 2047 columns, an element at a time, 158; the gradient of
// 32768 tokens 161 and 243.)
bool rows_vec(const void* p, int dt, int64_t stride, int64_t width) {
  return width % 8 == 0 && op_aligned(p, 16) && stride * op_dtype_size(dt) % 16 == 0;
}

template <typename W, typename O>
cudaError_t run_lookup(bool vec, const void* weight, int64_t wstride, int64_t vocab, int64_t width, const void* ids,
                       int wide, int64_t n, float scale, void* out, int64_t ostride, cudaStream_t st) {
  const dim3 b = block_of(width, vec ? 8 : 1);
  const dim3 g((unsigned)((n + 4 * b.y - 1) / (4 * b.y)), 1);
  if (vec)
    return op_launch(embedding_kernel<W, O, 8>, g, b, 0, st, 1, static_cast<const W*>(weight), wstride,
                     (uint32_t)vocab, (int)width, ids, wide, n, scale, static_cast<O*>(out), ostride);
  return op_launch(embedding_kernel<W, O, 1>, g, b, 0, st, 1, static_cast<const W*>(weight), wstride, (uint32_t)vocab,
                   (int)width, ids, wide, n, scale, static_cast<O*>(out), ostride);
}

template <typename D, typename G, int VEC>
cudaError_t run_sums(const SumArgs& a, int64_t chunks, const void* dout, void* grad, cudaStream_t st) {
  const dim3 b = block_of(a.width, VEC);
  const dim3 g((unsigned)((chunks + b.y - 1) / b.y), (unsigned)((a.width + b.x * VEC - 1) / (b.x * VEC)));
  cudaError_t e = op_launch(embedding_sum_kernel<D, G, VEC>, g, b, 0, st, 1, a, static_cast<const D*>(dout),
                            static_cast<G*>(grad));
  if (e != cudaSuccess || chunks < 2) return e;
  const int all = (a.width + 32 * VEC - 1) / (32 * VEC);
  int slabs = 1;
  while (slabs < all && slabs < 2) slabs *= 2;
  return op_launch(embedding_join_kernel<G, VEC>, 
                   dim3((unsigned)((chunks + kJoinChunks - 2) / kJoinChunks), (unsigned)((all + slabs - 1) / slabs)), dim3(kThreads), 0, st, 1, a, static_cast<G*>(grad), slabs);
}

// Blocks along x of the one-launch gradient: up to eight an SM over all slabs.
int64_t direct_blocks(int64_t vocab, int64_t width, int vec, int sms) {
  const int64_t slabs = (width + 32 * vec - 1) / (32 * vec), most = (8 * (int64_t)sms + slabs - 1) / slabs;
  return vocab < most ? vocab : most;
}

template <typename D, typename G, int VEC>
cudaError_t run_direct(const DirectArgs& a, int64_t blocks, const void* dout, void* grad, cudaStream_t st) {
  const int per = ((a.n + kDirectWarps - 1) / kDirectWarps + 31) / 32 * 32;
  const int64_t rows = (a.vocab + blocks - 1) / blocks;
  return op_launch(embedding_direct_kernel<D, G, VEC>,
                   dim3((unsigned)blocks, (unsigned)((a.width + 32 * VEC - 1) / (32 * VEC))), dim3(kThreads),
                   (size_t)(kDirectWarps * per + rows) * 4, st, 1, a, static_cast<const D*>(dout),
                   static_cast<G*>(grad));
}

// f(dout type, gradient type, vector width) for the call's own.
template <typename F>
cudaError_t by_types(bool vec, int dout_dtype, int grad_dtype, F f) {
  typedef __nv_bfloat16 B;
  const bool db = dout_dtype == MA_DT_BF16, gb = grad_dtype == MA_DT_BF16;
  const std::integral_constant<int, 8> v;
  const std::integral_constant<int, 1> o;
  if (vec) return db ? (gb ? f(B(), B(), v) : f(B(), 0.f, v)) : (gb ? f(0.f, B(), v) : f(0.f, 0.f, v));
  return db ? (gb ? f(B(), B(), o) : f(B(), 0.f, o)) : (gb ? f(0.f, B(), o) : f(0.f, 0.f, o));
}

}  // namespace
}  // namespace ma

using namespace ma;

extern "C" {

ma_status muon_adamw_embedding(const void* weight, int weight_dtype, int64_t weight_stride, int64_t vocab,
                               int64_t width, const void* ids, int id_bytes, int64_t n_tokens, double scale,
                               void* out, int out_dtype, int64_t out_stride, void* cuda_stream) {
  ma_status st = check_common(vocab, width, ids, id_bytes, n_tokens, scale);
  if (st == MA_OK) st = check_rows("weight", weight, weight_dtype, weight_stride, width, vocab);
  if (st == MA_OK) st = check_rows("out", out, out_dtype, out_stride, width, n_tokens);
  if (st != MA_OK) return st;
  if (n_tokens > 0) {
    const bool vec = rows_vec(weight, weight_dtype, weight_stride, width) && rows_vec(out, out_dtype, out_stride, width);
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    const int wide = id_bytes == 8;
    const float sc = (float)scale;
    cudaError_t e;
    if (weight_dtype == MA_DT_BF16)
      e = out_dtype == MA_DT_BF16
              ? run_lookup<__nv_bfloat16, __nv_bfloat16>(vec, weight, weight_stride, vocab, width, ids, wide, n_tokens,
                                                         sc, out, out_stride, s)
              : run_lookup<__nv_bfloat16, float>(vec, weight, weight_stride, vocab, width, ids, wide, n_tokens, sc,
                                                 out, out_stride, s);
    else
      e = out_dtype == MA_DT_BF16 ? run_lookup<float, __nv_bfloat16>(vec, weight, weight_stride, vocab, width, ids,
                                                                     wide, n_tokens, sc, out, out_stride, s)
                                  : run_lookup<float, float>(vec, weight, weight_stride, vocab, width, ids, wide,
                                                             n_tokens, sc, out, out_stride, s);
    if (e != cudaSuccess) return op_cuda(e, "embedding launch");
  }
  clear_last_error();
  return MA_OK;
}

ma_status muon_adamw_embedding_backward_workspace(int64_t n_tokens, int64_t vocab, int64_t width, int64_t* bytes) {
  if (!bytes) return op_fail(MA_ERR_ARG, "bytes must not be NULL");
  ma_status st = check_common(vocab, width, bytes, 8, n_tokens, 1.0);
  if (st != MA_OK) return st;
  *bytes = plan_backward(n_tokens, width).bytes;
  clear_last_error();
  return MA_OK;
}

ma_status muon_adamw_embedding_backward(const void* dout, int dout_dtype, int64_t dout_stride, const void* ids,
                                        int id_bytes, int64_t n_tokens, double scale, void* grad, int grad_dtype,
                                        int64_t grad_stride, int64_t vocab, int64_t width, int accumulate,
                                        void* workspace, int64_t workspace_bytes, void* cuda_stream) {
  ma_status st = check_common(vocab, width, ids, id_bytes, n_tokens, scale);
  if (st == MA_OK) st = check_rows("dout", dout, dout_dtype, dout_stride, width, n_tokens);
  if (st == MA_OK) st = check_rows("grad", grad, grad_dtype, grad_stride, width, vocab);
  if (st != MA_OK) return st;
  if (accumulate != 0 && accumulate != 1) return op_fail(MA_ERR_ARG, "accumulate must be 0 or 1");
  const Plan p = plan_backward(n_tokens, width);
  if (!workspace) return op_fail(MA_ERR_ARG, "workspace must not be NULL");
  if (!op_aligned(workspace, 256)) return op_fail(MA_ERR_ALIGN, "workspace is not 256-byte aligned");
  if (workspace_bytes < p.bytes)
    return op_fail(MA_ERR_ARG, "workspace of %lld bytes, %lld are needed", (long long)workspace_bytes,
                   (long long)p.bytes);
  if (n_tokens == 0 && accumulate) {
    clear_last_error();
    return MA_OK;
  }
  int sms = 0, *err = nullptr;
  cudaError_t e = op_device(&sms, &err);
  if (e != cudaSuccess) return op_cuda(e, "device query");
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  const bool vec = rows_vec(dout, dout_dtype, dout_stride, width) && rows_vec(grad, grad_dtype, grad_stride, width);
  const int64_t blocks = direct_blocks(vocab, width, vec ? 8 : 1, sms);
  if (n_tokens <= kDirectTokens && (vocab + blocks - 1) / blocks <= kDirectRows) {
    DirectArgs d{};
    d.ids = ids;
    d.wide = id_bytes == 8;
    d.n = (int)n_tokens;
    d.vocab = (uint32_t)vocab;
    d.width = (int)width;
    d.scale = (float)scale;
    d.accumulate = accumulate;
    d.dstride = dout_stride;
    d.gstride = grad_stride;
    e = by_types(vec, dout_dtype, grad_dtype, [&](auto x, auto y, auto v) {
      return run_direct<decltype(x), decltype(y), v.value>(d, blocks, dout, grad, s);
    });
    if (e != cudaSuccess) return op_cuda(e, "embedding gradient launch");
    clear_last_error();
    return MA_OK;
  }
  SortArgs a{};
  a.ids = ids;
  a.wide = id_bytes == 8;
  a.n = n_tokens;
  a.vocab = (uint32_t)vocab;
  int bits = 1;
  while (((int64_t)1 << bits) <= vocab) ++bits;  // keys 0 .. vocab
  a.passes = n_tokens > 0 ? (bits + kDigitBits - 1) / kDigitBits : 0;
  a.bits = a.passes > 0 ? (bits + a.passes - 1) / a.passes : 0;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.key0 = reinterpret_cast<uint32_t*>(ws);
  a.pos0 = reinterpret_cast<uint32_t*>(ws + p.key_bytes);
  a.key1 = reinterpret_cast<uint32_t*>(ws + 2 * p.key_bytes);
  a.pos1 = reinterpret_cast<uint32_t*>(ws + 3 * p.key_bytes);
  const int64_t gsize = op_dtype_size(grad_dtype);
  const int64_t fill = accumulate ? 0 : vocab * width * gsize;
  int64_t fill_ctas = (fill + 64 * kSortThreads - 1) / (64 * kSortThreads);  // four 16-byte stores a thread at least
  if (fill_ctas > 2 * sms) fill_ctas = 2 * sms;
  const unsigned grid = (unsigned)(kSortCluster + (fill_ctas + kSortCluster - 1) / kSortCluster * kSortCluster);
  e = op_smem_limit<embedding_sort_kernel>((int)kSortSmem);
  if (e != cudaSuccess) return op_cuda(e, "embedding sort attributes");
  e = op_launch(embedding_sort_kernel, dim3(grid), dim3(kSortThreads), kSortSmem, s, kSortCluster, a,
                static_cast<uint8_t*>(grad), width * gsize, grad_stride * gsize, accumulate ? (int64_t)0 : vocab,
                (int)(op_aligned(grad, 16) && width * gsize % 16 == 0 && grad_stride * gsize % 16 == 0));
  if (e != cudaSuccess) return op_cuda(e, "embedding sort launch");
  if (n_tokens > 0) {
    SumArgs u{};
    u.key = a.key0;
    u.pos = a.pos0;
    u.n = n_tokens;
    u.vocab = (uint32_t)vocab;
    u.width = (int)width;
    u.scale = (float)scale;
    u.accumulate = accumulate;
    u.dstride = dout_stride;
    u.gstride = grad_stride;
    u.partial = reinterpret_cast<float*>(ws + 4 * p.key_bytes);
    e = by_types(vec, dout_dtype, grad_dtype, [&](auto x, auto y, auto v) {
      return run_sums<decltype(x), decltype(y), v.value>(u, p.chunks, dout, grad, s);
    });
    if (e != cudaSuccess) return op_cuda(e, "embedding sum launch");
  }
  clear_last_error();
  return MA_OK;
}

}  // extern "C"
