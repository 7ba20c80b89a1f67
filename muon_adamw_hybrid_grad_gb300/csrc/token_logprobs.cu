// Log probabilities of given tokens with entropy and top alternatives, and their gradient.
//
// Forward, one pass over a row: each thread keeps its own running maximum m, the
// sum s of 2^a and the sum u of a 2^a, a = (x - m) scale log2(e). It adds those
// of a group of 32 elements at a time (one by one, what lies below a step of s was
// lost: 1.3e-6 of every log probability of 4093 rows of 151936, now 6e-8), and
// the threads' are joined at the end:
//   lse = m scale + ln s,  entropy = ln s - ln(2) u / s.
// Sums are kept relative to the maximum, so that neither entropy nor a log
// probability is a difference of large numbers.
//
// The alternatives cost the pass next to nothing: a group's maximum, which the
// softmax needs anyway, is kept in shared memory. The threshold is the k-th
// largest of 32 maxima, each over the threads of one lane of every warp: it is at
// most the k-th largest element, since k lanes have an element that reaches it. So
// only groups whose maximum reaches it are read again, some 25 of thousands, and
// their few candidates ranked by comparison.
//
// A row of the large vocabulary has a block; where rows are few, a cluster of up
// to eight blocks shares one and joins through distributed shared memory.
// Bound by HBM for many rows, by latency for few.
//
// Gradient: an element-wise pass, bound by HBM (one row in, one out).
#include <math.h>

#include <algorithm>
#include <cmath>

#include "op_common.cuh"
#include "pairs.cuh"
#include "tcgen05.cuh"

namespace ma {
namespace {

constexpr int kThreads = 128;
constexpr int kVecs = 4;  // vectors of eight elements in a group
constexpr int kStep = kThreads * kVecs;  // vectors of a block's pass
constexpr int kGradThreads = 256;
constexpr int kGradStep = kGradThreads * kVecs;
constexpr int kMaxTop = 32;
constexpr int kListed = 512;  // candidates above the threshold, and as many that equal it
constexpr int kMaxVocab = 1 << 20;
constexpr int kMaxParts = 8;
constexpr int kMaxGroupBytes = (kMaxVocab / (kStep * 8) + 1) * kThreads * 4;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct LogprobArgs {
  const void* logits;
  const void* ids;
  int64_t n, stride, out_stride;
  int vocab, id_bytes, top, parts;
  float scale;
  float *logprobs, *entropy, *lse, *top_logprobs;
  int64_t* top_ids;
  const float *dlogprobs, *dentropy, *entropy_in, *lse_in;
  void* dlogits;
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ void fill(RawVec<__nv_bfloat16, 8>& r) {
  r.v = make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);  // -infinity
}
__device__ __forceinline__ void fill(RawVec<float, 8>& r) {
  r.a = r.b = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
}

// The largest of a group's elements, NaN if there is one.
template <int N>
__device__ __forceinline__ float group_max(const RawVec<__nv_bfloat16, 8> (&r)[N]) {
  __nv_bfloat162 m[4];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t w[4] = {r[i].v.x, r[i].v.y, r[i].v.z, r[i].v.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&w[q]);
      m[q] = i == 0 ? x : __hmax2_nan(m[q], x);
    }
  }
  m[0] = __hmax2_nan(__hmax2_nan(m[0], m[1]), __hmax2_nan(m[2], m[3]));
  return max_nan(__low2float(m[0]), __high2float(m[0]));
}
template <int N>
__device__ __forceinline__ float group_max(const RawVec<float, 8> (&r)[N]) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < N; ++i)
    m = max_nan(m, max_nan(max_nan(max_nan(r[i].a.x, r[i].a.y), max_nan(r[i].a.z, r[i].a.w)),
                           max_nan(max_nan(r[i].b.x, r[i].b.y), max_nan(r[i].b.z, r[i].b.w))));
  return m;
}

// Softmax sums relative to their maximum m; m -infinity: nothing so far.
struct Sums {
  float m, s, u;
};
// The same sums relative to `m`, which is at least x.m.
__device__ __forceinline__ Sums rebase(const Sums& x, float m, float c) {
  if (x.m == -INFINITY) return {m, 0.f, 0.f};
  const float d = (x.m - m) * c, f = ex2(d);
  // where nothing is left the difference may be infinite
  return {m, f * x.s, f == 0.f ? f * x.u : f * fmaf(d, x.s, x.u)};
}
__device__ __forceinline__ Sums join(const Sums& x, const Sums& y, float c) {
  const float m = max_nan(x.m, y.m);
  const Sums a = rebase(x, m, c), b = rebase(y, m, c);
  return {m, a.s + b.s, a.u + b.u};
}

// An element's place in the order of the alternatives: by value, the lowest
// index first among equal ones. NaN counts as -infinity.
__device__ __forceinline__ uint32_t rank_bits(float x) {
  x = x != x ? -INFINITY : x + 0.f;  // one zero
  const uint32_t b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t rank_key(float x, uint32_t index) {
  return (uint64_t)rank_bits(x) << 32 | (0xFFFFFFFFu - index);
}
__device__ __forceinline__ float key_value(uint64_t key) {
  const uint32_t b = (uint32_t)(key >> 32);
  return __uint_as_float(b & 0x80000000u ? b & 0x7FFFFFFFu : ~b);
}
__device__ __forceinline__ uint32_t key_index(uint64_t key) { return 0xFFFFFFFFu - (uint32_t)key; }

__device__ __forceinline__ int64_t token_id(const LogprobArgs& a, int64_t row) {
  return a.id_bytes == 8 ? __ldg(static_cast<const long long*>(a.ids) + row)
                         : (int64_t)__ldg(static_cast<const int*>(a.ids) + row);
}

__device__ __forceinline__ uint64_t ld_cluster_u64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// A row as its elements up to the first 16-byte boundary, vectors of eight, and the rest.
template <typename T>
struct Row {
  const T* p;
  int head, vecs, tail;
  __device__ __forceinline__ Row(const T* row, int vocab) : p(row) {
    const int off = (int)(reinterpret_cast<uintptr_t>(row) & 15);
    head = min(off ? (16 - off) / (int)sizeof(T) : 0, vocab);
    vecs = (vocab - head) / 8;
    tail = vocab - head - vecs * 8;
  }
  __device__ __forceinline__ int index(int vec) const { return head + vec * 8; }
  // the edge element of thread t, -1 for none
  __device__ __forceinline__ int edge(int t) const {
    return t < head ? t : t >= 32 && t - 32 < tail ? head + vecs * 8 + t - 32 : -1;
  }
};

constexpr int kHits = 512;  // groups that reach the threshold

struct TopShared {
  float best[kThreads];
  uint32_t hits[kHits];
  uint64_t list[2 * kListed];  // above the threshold, then equal to it
  uint64_t chosen[kMaxTop];
  uint64_t warp_best[kThreads / 32];
  int warp_count[kThreads / 32];
  int hit, above, equal;
};

// The block's `top` first elements of vectors [v0, v1), and of the row's edges
// with `edges`, into sh.chosen in their order; 0 where there are fewer.
template <typename T>
__device__ void choose_top(const Row<T>& row, int v0, int v1, bool edges, int top, float best, const T* groups,
                           TopShared& sh) {
  const int t = threadIdx.x, lane = t & 31;
  sh.best[t] = best;
  if (t < kMaxTop) sh.chosen[t] = 0;
  if (t == 0) sh.hit = sh.above = sh.equal = 0;
  __syncthreads();
  // the threshold: the top-th largest of 32 maxima, each of the threads of one lane. It is met by as many elements
  // as are wanted; with fewer lanes that hold any it is -infinity, and everything is a candidate
  float mine = sh.best[lane];
#pragma unroll
  for (int i = 1; i < kThreads / 32; ++i) mine = fmaxf(mine, sh.best[i * 32 + lane]);
  int rank = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const float b = __shfl_sync(0xffffffffu, mine, i);
    rank += b > mine || (b == mine && i < lane);
  }
  const float limit = __shfl_sync(0xffffffffu, mine, __ffs(__ballot_sync(0xffffffffu, rank == top - 1)) - 1);
  const uint32_t limit_bits = rank_bits(limit);
  const bool everything = limit == -INFINITY;
  auto offer = [&](float x, int index) {
    if (!(x >= limit) && !everything) return;
    const uint64_t key = rank_key(x, (uint32_t)index);
    if ((uint32_t)(key >> 32) > limit_bits) {
      const int at = atomicAdd(&sh.above, 1);
      if (at < kListed) sh.list[at] = key;
    } else {
      const int at = atomicAdd(&sh.equal, 1);
      if (at < kListed) sh.list[kListed + at] = key;
    }
  };
  auto of_vector = [&](int vec, auto&& f) {
    float x[8];
    load8(row.p + row.index(vec), x);
#pragma unroll
    for (int e = 0; e < 8; ++e) f(x[e], row.index(vec) + e);
  };
  // every element of this thread whose group reaches the threshold
  auto each = [&](auto&& f) {
    int g = t;
    for (int v = v0; v < v1; v += kStep, g += kThreads) {
      if (load1(groups + g) < limit) continue;
      for (int j = 0; j < kVecs; ++j)
        if (v + j * kThreads + t < v1) of_vector(v + j * kThreads + t, f);
    }
    if (edges && row.edge(t) >= 0) f(load1(row.p + row.edge(t)), row.edge(t));
  };
  // the groups that reach it, looked at 32 at a time, and then their vectors shared out over all threads
  if (best >= limit) {
    const int all = (v1 - v0 + kStep - 1) / kStep;
    for (int i0 = 0; i0 < all; i0 += 32) {
      uint32_t reach = 0;
#pragma unroll 8
      for (int i = 0; i < 32; ++i)
        if (i0 + i < all) reach |= (uint32_t)!(load1(groups + (i0 + i) * kThreads + t) < limit) << i;
      for (; reach; reach &= reach - 1) {
        const int at = atomicAdd(&sh.hit, 1);
        if (at < kHits) sh.hits[at] = (uint32_t)((i0 + __ffs(reach) - 1) * kThreads + t);
      }
    }
  }
  __syncthreads();
  const int hit = sh.hit;
  if (hit > kHits) {
    each(offer);
  } else {
    for (int i = t; i < hit * kVecs; i += kThreads) {
      const int g = (int)sh.hits[i / kVecs];
      const int vec = v0 + g / kThreads * kStep + i % kVecs * kThreads + g % kThreads;
      if (vec < v1) of_vector(vec, offer);
    }
    if (edges && row.edge(t) >= 0) offer(load1(row.p + row.edge(t)), row.edge(t));
  }
  __syncthreads();
  int above = sh.above, equal = sh.equal;
  if (above > kListed) {
    // a few threads hold more large elements than the list takes: one element a pass
    uint64_t before = ~0ull;
    for (int r = 0; r < top; ++r) {
      uint64_t mine = 0;
      each([&](float x, int index) {
        const uint64_t key = rank_key(x, (uint32_t)index);
        if (key < before && key > mine) mine = key;
      });
      for (int d = 16; d > 0; d >>= 1) mine = max(mine, __shfl_xor_sync(0xffffffffu, mine, d));
      if ((t & 31) == 0) sh.warp_best[t >> 5] = mine;
      __syncthreads();
      before = 0;
#pragma unroll
      for (int i = 0; i < kThreads / 32; ++i) before = max(before, (uint64_t)sh.warp_best[i]);
      if (t == 0) sh.chosen[r] = before;
      __syncthreads();
    }
    return;
  }
  if (equal > kListed) {
    // ties without end, as in a masked row: the first ones in the order of their indices. The vectors hold enough
    // of them, so that the edge behind them, whose indices are the largest, is not needed.
    int found = 0;
    if (edges) {
      if (t < 32) {
        const bool tie = t < row.head && rank_bits(load1(row.p + t)) == limit_bits;
        const uint32_t votes = __ballot_sync(0xffffffffu, tie);
        if (tie) sh.list[kListed + __popc(votes & ((1u << t) - 1))] = rank_key(limit, (uint32_t)t);
        if (t == 0) sh.warp_count[0] = __popc(votes);
      }
      __syncthreads();
      found = sh.warp_count[0];
      __syncthreads();
    }
    for (int v = v0; v < v1 && found < top; v += kThreads) {
      uint32_t ties = 0;
      if (v + t < v1) {
        float x[8];
        load8(row.p + row.index(v + t), x);
#pragma unroll
        for (int e = 0; e < 8; ++e) ties |= (uint32_t)(rank_bits(x[e]) == limit_bits) << e;
      }
      const int mine = __popc(ties);
      int upto = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, upto, d);
        if ((t & 31) >= d) upto += o;
      }
      if ((t & 31) == 31) sh.warp_count[t >> 5] = upto;
      __syncthreads();
      int place = found + upto - mine, total = 0;
#pragma unroll
      for (int i = 0; i < kThreads / 32; ++i) {
        const int c = sh.warp_count[i];
        if (i < (t >> 5)) place += c;
        total += c;
      }
      for (; ties; ties &= ties - 1, ++place)
        if (place < top) sh.list[kListed + place] = rank_key(limit, (uint32_t)(row.index(v + t) + __ffs(ties) - 1));
      found += total;
      __syncthreads();
    }
    equal = min(found, top);
  }
  for (int i = t; i < above + equal; i += kThreads) {
    const uint64_t key = sh.list[i < above ? i : kListed + i - above];
    int r = 0;
#pragma unroll 8
    for (int k = 0; k < above; ++k) r += sh.list[k] > key;
#pragma unroll 8
    for (int k = 0; k < equal; ++k) r += sh.list[kListed + k] > key;
    if (r < top) sh.chosen[r] = key;
  }
  __syncthreads();
}

// A thread's running sums, in pairs.
struct Running {
  float m;
  uint64_t s, u;
  // gm is above m, or one of them is NaN, which stays
  __device__ __forceinline__ void raise(float gm, float c) {
    gm = max_nan(gm, m);
    const float f = m == -INFINITY ? 0.f : ex2((m - gm) * c);
    const float d = f == 0.f ? 0.f : (m - gm) * c;
    u = mul2(pack2(f, f), fma2(pack2(d, d), s, u));
    s = mul2(pack2(f, f), s);
    m = gm;
  }
  __device__ __forceinline__ void add(float x, float y, float c) {
    const uint64_t a = mul2(add2(pack2(x, y), pack2(-m, -m)), pack2(c, c));
    float p, q;
    unpack2(a, p, q);
    // -infinity would meet a zero
    p = max_nan(p, -1e30f);
    q = max_nan(q, -1e30f);
    const uint64_t e = pack2(ex2(p), ex2(q));
    s = add2(s, e);
    u = fma2(e, pack2(p, q), u);
  }
  // A group's vectors: their own sums first, so that a long row's are not added to one by one.
  template <typename T, int N>
  __device__ __forceinline__ void add_group(const RawVec<T, 8> (&raw)[N], float c) {
    Running group{m, 0, 0};
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float x[8];
      raw[j].get(x);
#pragma unroll
      for (int e = 0; e < 8; e += 2) group.add(x[e], x[e + 1], c);
    }
    s = add2(s, group.s);
    u = add2(u, group.u);
  }
  __device__ __forceinline__ Sums sums() const {
    float s0, s1, u0, u1;
    unpack2(s, s0, s1);
    unpack2(u, u0, u1);
    return {m, s0 + s1, u0 + u1};
  }
};

// The sums of a block of THREADS: of each warp relative to its maximum, then of the block.
template <int THREADS>
__device__ __forceinline__ Sums block_sums(const Running& run, float c, Sums (&warps)[THREADS / 32]) {
  Sums all = run.sums();
  float m = all.m;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
  all = rebase(all, m, c);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    all.s += __shfl_xor_sync(0xffffffffu, all.s, d);
    all.u += __shfl_xor_sync(0xffffffffu, all.u, d);
  }
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = all;
  __syncthreads();
  m = warps[0].m;
#pragma unroll
  for (int i = 1; i < THREADS / 32; ++i) m = max_nan(m, warps[i].m);
  all = {m, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) {
    const Sums w = rebase(warps[i], m, c);
    all.s += w.s;
    all.u += w.u;
  }
  return all;
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(kThreads) token_logprobs_kernel(const __grid_constant__ LogprobArgs a) {
  extern __shared__ uint8_t shared[];
  T* const groups = reinterpret_cast<T*>(shared);  // TOP: the maximum of every thread's groups
  __shared__ Sums warp_sums[kThreads / 32];
  __shared__ Sums part_sums;
  __shared__ TopShared sh;
  const int t = threadIdx.x;
  const int64_t at = blockIdx.x / a.parts;
  const int part = (int)(blockIdx.x - at * a.parts);
  pdl_wait();
  pdl_launch();
  const Row<T> row(static_cast<const T*>(a.logits) + at * a.stride, a.vocab);
  const int share = (row.vecs + a.parts * kStep - 1) / (a.parts * kStep) * kStep;
  const int v0 = min(part * share, row.vecs), v1 = min(v0 + share, row.vecs);
  const bool edges = part == 0;
  const float c = a.scale * kLog2e;

  // the given token's logit, by the thread that needs it
  int64_t id = -1;
  float given = 0.f;
  if (edges && t == 0) {
    id = token_id(a, at);
    if (id >= 0 && id < a.vocab) given = load1(row.p + id);
  }
  Running run{-INFINITY, 0, 0};
  float best = -INFINITY;
  RawVec<T, 8> next[kVecs];
  auto fetch = [&](int v) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int vec = v + j * kThreads + t;
      if (vec < v1)
        next[j].load(row.p + row.index(vec));
      else
        fill(next[j]);
    }
  };
  if (v0 < v1) fetch(v0);
  int g = t;
  for (int v = v0; v < v1; v += kStep, g += kThreads) {
    RawVec<T, 8> cur[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) cur[j] = next[j];
    if (v + kStep < v1) fetch(v + kStep);
    const float gm = group_max(cur);
    if (TOP) {
      store1(groups + g, gm);  // as it was read: nothing is rounded
      best = fmaxf(best, gm);
    }
    if (!(gm <= run.m)) run.raise(gm, c);
    if (run.m != -INFINITY) run.add_group(cur, c);
  }
  if (edges && row.edge(t) >= 0) {
    const float x = load1(row.p + row.edge(t));
    best = fmaxf(best, x);
    if (!(x <= run.m)) run.raise(x, c);
    if (run.m != -INFINITY) run.add(x, -INFINITY, c);
  }
  Sums all = block_sums<kThreads>(run, c, warp_sums);
  if constexpr (TOP) choose_top(row, v0, v1, edges, a.top, best, groups, sh);

  if (a.parts > 1) {
    // the cluster's first block reads the others' results
    if (t == 0) part_sums = all;
    cluster_sync();
    if (part == 0) {
      const uint32_t theirs = smem_u32(&part_sums);
      for (int i = 1; i < a.parts; ++i) {
        const uint32_t p = mapa_shared(theirs, i);
        all = join(all, {ld_cluster_f32(p), ld_cluster_f32(p + 4), ld_cluster_f32(p + 8)}, c);
      }
      if constexpr (TOP) {
        const uint32_t lists = smem_u32(sh.chosen);
        for (int i = t; i < a.parts * a.top; i += kThreads)
          sh.list[i] = ld_cluster_u64(mapa_shared(lists, i / a.top) + 8 * (i % a.top));
      }
    }
    // the others may leave once this block has read
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    if (part != 0) {
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
      return;
    }
    __syncthreads();
    if constexpr (TOP) {
      for (int k = t; k < a.parts * a.top; k += kThreads) {
        const uint64_t key = sh.list[k];
        int r = 0;
#pragma unroll 8
        for (int i = 0; i < a.parts * a.top; ++i) r += sh.list[i] > key;
        if (key != 0 && r < a.top) sh.chosen[r] = key;
      }
      __syncthreads();
    }
  }
  const bool empty = all.m == -INFINITY;
  const float log_s = logf(all.s);
  if (t == 0) {
    const bool inside = id >= 0 && id < a.vocab;
    a.logprobs[at] = !inside ? 0.f : empty ? -INFINITY : (given - all.m) * a.scale - log_s;
    a.entropy[at] = empty ? 0.f : log_s - kLn2 * (all.u / all.s);
    a.lse[at] = empty ? -INFINITY : fmaf(all.m, a.scale, log_s);
  }
  if constexpr (TOP) {
    if (t < a.top) {
      const uint64_t key = sh.chosen[t];
      a.top_logprobs[at * a.top + t] = empty ? -INFINITY : (key_value(key) - all.m) * a.scale - log_s;
      a.top_ids[at * a.top + t] = (int64_t)key_index(key);
    }
  }
  if (a.parts > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ---- gradient ----
// d_v = scale (dlogprob (1[v = id] - p_v) - dentropy p_v (log p_v + entropy))

struct GradRow {
  float shift, rest, c, base, slope, given;  // d = 2^a (base + slope a) [+ given], a = (x - shift - rest) c
  int64_t id;
  bool empty;
};

// Above this magnitude of lse its rounding, half a step of fp32, would change a row's probabilities by more than 2^-14
// of themselves for bf16 logits, whose gradient is rounded to 2^-9, and 2^-19 for fp32. Far above it ln s would be lost,
// as in a row of the type's lowest value alone, or lse be infinite. There each block forms the row's sums once more:
// 4093 bf16 rows of 151936 3.8 ms, usual ones 0.37; 2046 fp32 rows 2.1 and 0.36; 8000 fp32 rows of 8000 113 and 79 us.
template <typename T>
constexpr float kLseMax = sizeof(T) == 2 ? 2048.f : 64.f;

// The row's maximum and the logarithm of its sum, by the whole block.
template <typename T>
__device__ __forceinline__ float2 row_sums(const Row<T> row, float c) {
  __shared__ Sums warps[kGradThreads / 32];
  const int t = threadIdx.x;
  Running run{-INFINITY, 0, 0};
  RawVec<T, 8> next;
  if (t < row.vecs) next.load(row.p + row.index(t));
#pragma unroll 1
  for (int v = t; v < row.vecs; v += kGradThreads) {
    const RawVec<T, 8> cur[1] = {next};
    if (v + kGradThreads < row.vecs) next.load(row.p + row.index(v + kGradThreads));
    const float m = group_max(cur);
    if (!(m <= run.m)) run.raise(m, c);
    if (run.m != -INFINITY) run.add_group(cur, c);
  }
  if (row.edge(t) >= 0) {
    const float x = load1(row.p + row.edge(t));
    if (!(x <= run.m)) run.raise(x, c);
    if (run.m != -INFINITY) run.add(x, -INFINITY, c);
  }
  const Sums all = block_sums<kGradThreads>(run, c, warps);
  return make_float2(all.m, all.m == -INFINITY ? 0.f : logf(all.s));
}

__device__ __forceinline__ GradRow grad_row(const LogprobArgs& a, int64_t at, float lse) {
  GradRow g;
  const float h = a.dentropy ? __ldg(a.dentropy + at) : 0.f;
  g.id = token_id(a, at);
  const float l = a.dlogprobs && g.id >= 0 && g.id < a.vocab ? __ldg(a.dlogprobs + at) : 0.f;
  // lse / scale in two parts: its rounding would scale the whole row
  g.shift = lse / a.scale;
  g.rest = fmaf(-g.shift, a.scale, lse) / a.scale;
  g.c = a.scale * kLog2e;
  g.given = a.scale * l;
  g.base = -a.scale * (h == 0.f ? l : fmaf(h, __ldg(a.entropy_in + at), l));
  g.slope = -a.scale * h * kLn2;
  g.empty = false;  // which it may be above kLseMax only
  return g;
}

__device__ __forceinline__ float grad_of(const GradRow& g, float x) {
  const float a = max_nan((x - g.shift - g.rest) * g.c, -1000.f);  // where 2^a is 0, and a times the slope no infinity
  return g.empty ? 0.f : ex2(a) * fmaf(g.slope, a, g.base);
}

template <typename T>
__device__ __forceinline__ void grad_single(const GradRow& g, const T* row, T* out, int i) {
  store1(out + i, grad_of(g, load1(row + i)) + (i == g.id && !g.empty ? g.given : 0.f));
}

// A block's part of a row whose lse is above kLseMax, element by element. It is called behind the usual rows' path and
// keeps nothing across row_sums, so that it costs those neither registers nor a branch that waits for lse.
template <typename T>
__device__ __noinline__ void grad_large(const LogprobArgs& a, int64_t at, int part, T* out) {
  const T* const p = static_cast<const T*>(a.logits) + at * a.stride;
  const float lse = __ldg(a.lse_in + at);
  GradRow g = grad_row(a, at, lse);
  const int begin = part * kGradStep * 8 + threadIdx.x, end = min(a.vocab, (part + 1) * kGradStep * 8);
  // No sums for a row that no gradient reaches. Nor, where lse is -infinity, for a part of masked logits without the
  // given token, or in which that has no gradient: whatever the row's other logits are.
  bool look = g.given != 0.f || g.base != 0.f || g.slope != 0.f || lse == INFINITY;
  if (look && lse == -INFINITY) {
    bool any = false;
    for (int i = begin; i < end; i += kGradThreads) any |= load1(p + i) > -INFINITY || (i == g.id && g.given != 0.f);
    look = __syncthreads_or(any);
  }
  g.empty = !look;
  if (look) {
    const float2 sums = row_sums(Row<T>(p, a.vocab), g.c);
    g.shift = sums.x;
    g.rest = sums.y / a.scale;
    g.empty = sums.x == -INFINITY;
  }
  for (int i = begin; i < end; i += kGradThreads) grad_single(g, p, out, i);
}

// (fp32 for four blocks an SM, which it would have anyway: with other registers 81 us in place of 79 for 8000 rows of 8000)
template <typename T>
__global__ void __launch_bounds__(kGradThreads, sizeof(T) == 2 ? 0 : 4)
    token_logprobs_grad_kernel(const __grid_constant__ LogprobArgs a) {
  const int t = threadIdx.x;
  const int64_t at = blockIdx.x / a.parts;
  const int part = (int)(blockIdx.x - at * a.parts);
  pdl_wait();
  pdl_launch();
  const Row<T> row(static_cast<const T*>(a.logits) + at * a.stride, a.vocab);
  T* const out = static_cast<T*>(a.dlogits) + at * a.out_stride;
  bool large;
  if (((reinterpret_cast<uintptr_t>(row.p) ^ reinterpret_cast<uintptr_t>(out)) & 15) != 0) {
    // rows that lie differently: no boundary is both's
    const float lse = __ldg(a.lse_in + at);
    const GradRow g = grad_row(a, at, lse);
    large = fabsf(lse) > kLseMax<T>;
    const int end = large ? 0 : min(a.vocab, (part + 1) * kGradStep * 8);
    for (int i = part * kGradStep * 8 + t; i < end; i += kGradThreads) grad_single(g, row.p, out, i);
  } else {
    const int v0 = part * kGradStep;
    RawVec<T, 8> raw[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int vec = v0 + j * kGradThreads + t;
      if (vec < row.vecs) raw[j].load(row.p + row.index(vec));
    }
    const float lse = __ldg(a.lse_in + at);
    const GradRow g = grad_row(a, at, lse);
    large = fabsf(lse) > kLseMax<T>;
    const int vecs = large ? 0 : row.vecs;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int vec = v0 + j * kGradThreads + t;
      if (vec >= vecs) break;
      const int i = row.index(vec);
      float x[8];
      raw[j].get(x);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = grad_of(g, x[e]);
      if (g.id >= i && g.id < i + 8) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (i + e == g.id) x[e] += g.given;
      }
      store8(out + i, x);
    }
    if (part == 0 && row.edge(t) >= 0 && !large) grad_single(g, row.p, out, row.edge(t));
  }
  if (large) grad_large(a, at, part, out);
}

ma_status check(const ma_token_logprobs* d) {
  if (!d) return op_fail(MA_ERR_ARG, "the description must not be NULL");
  if (!op_dtype_ok(d->dtype)) return op_fail(MA_ERR_DTYPE, "dtype %d is neither MA_DT_F32 nor MA_DT_BF16", d->dtype);
  if (d->id_bytes != 4 && d->id_bytes != 8) return op_fail(MA_ERR_ARG, "id_bytes %d is neither 4 nor 8", d->id_bytes);
  if (d->n_tokens < 0 || d->n_tokens > (1ll << 30) || d->vocab < 1 || d->vocab > kMaxVocab)
    return op_fail(MA_ERR_SHAPE, "%lld tokens of %lld logits: outside [0, 2^30] or [1, 2^20]", (long long)d->n_tokens,
                   (long long)d->vocab);
  // the gradient's blocks of 8192 logits, and a cluster's, are numbered in 31 bits
  const int64_t parts = std::max<int64_t>((d->vocab + kGradStep * 8 - 1) / (kGradStep * 8), 1);
  if (d->n_tokens * parts > INT32_MAX)
    return op_fail(MA_ERR_SHAPE, "%lld tokens of %lld logits are too many for a call", (long long)d->n_tokens,
                   (long long)d->vocab);
  if (!(d->scale >= 1e-30 && d->scale <= 1e30))  // its products and quotients stay normal fp32 numbers
    return op_fail(MA_ERR_ARG, "scale = %g outside [1e-30, 1e30]", d->scale);
  if (d->n_tokens == 0) return MA_OK;
  if (!d->logits || !d->ids) return op_fail(MA_ERR_ARG, "logits and ids must not be NULL");
  if (!op_aligned(d->logits, op_dtype_size(d->dtype)) || !op_aligned(d->ids, d->id_bytes))
    return op_fail(MA_ERR_ALIGN, "logits or ids is not aligned to its elements");
  if (d->n_tokens > 1 && d->stride < d->vocab)
    return op_fail(MA_ERR_SHAPE, "logits has rows %lld apart, below the vocabulary", (long long)d->stride);
  return MA_OK;
}

LogprobArgs args_of(const ma_token_logprobs* d) {
  LogprobArgs a{};
  a.logits = d->logits;
  a.ids = d->ids;
  a.n = d->n_tokens;
  a.stride = d->stride;
  a.vocab = (int)d->vocab;
  a.id_bytes = d->id_bytes;
  a.scale = (float)d->scale;
  return a;
}

template <typename T, bool TOP>
cudaError_t forward(LogprobArgs& a, cudaStream_t st) {
  int sms = 0, *err = nullptr;
  cudaError_t e = op_device(&sms, &err);
  if (e != cudaSuccess) return e;
  a.parts = 1;
  const int64_t steps = (a.vocab / 8 + kStep - 1) / kStep;
  // A cluster to a row where blocks would be few; the larger the clusters, the slower they are dispatched. Times with
  // 1, 2, 4, 8 blocks a row of 151936 (no alternatives): 1 row 13.9, 8.9, 6.5, 5.1 us; 64 rows 14.1, 9.0, 7.4, 7.6;
  // 150 rows 14.1, 10.6, 17.1, 13.6; 300 rows 22.2, 17.5, 21.5, 23.4; 900 rows 62, 58, 56, 64.
  // The rule does less well for shorter rows: of 32000 it lies within a fifth of the best, of 8192 up to 300 rows take
  // 3.0 to 3.6 us in clusters of 2 and 2.5 to 2.7 in single blocks (with alternatives 6.0 to 7.2 and 5.0 to 5.5).
  for (int k = 4; a.parts < kMaxParts && 2 * a.parts * a.n <= (int64_t)k * sms && steps >= 2 * a.parts; --k) a.parts *= 2;
  const int64_t per = (steps + a.parts - 1) / a.parts;
  if (TOP) {
    e = op_smem_limit<token_logprobs_kernel<T, TOP>>(kMaxGroupBytes);
    if (e != cudaSuccess) return e;
  }
  return op_launch(token_logprobs_kernel<T, TOP>, dim3((unsigned)(a.n * a.parts)), dim3(kThreads),
                   TOP ? (size_t)std::max<int64_t>(per, 1) * kThreads * sizeof(T) : 0, st, a.parts, a);
}

}  // namespace
}  // namespace ma

using namespace ma;

extern "C" {

ma_status muon_adamw_token_logprobs(const ma_token_logprobs* d, int32_t top, float* logprobs, float* entropy,
                                    float* lse, float* top_logprobs, int64_t* top_ids, void* cuda_stream) {
  const ma_status st = check(d);
  if (st != MA_OK) return st;
  if (top < 0 || top > kMaxTop || top > d->vocab)
    return op_fail(MA_ERR_ARG, "top = %d outside [0, %d], or above the vocabulary", top, kMaxTop);
  if (d->n_tokens > 0) {
    if (!logprobs || !entropy || !lse || (top > 0 && (!top_logprobs || !top_ids)))
      return op_fail(MA_ERR_ARG, "the results must not be NULL");
    if (!op_aligned(logprobs, 4) || !op_aligned(entropy, 4) || !op_aligned(lse, 4) ||
        (top > 0 && (!op_aligned(top_logprobs, 4) || !op_aligned(top_ids, 8))))
      return op_fail(MA_ERR_ALIGN, "a result is not aligned to its elements");
    LogprobArgs a = args_of(d);
    a.top = top;
    a.logprobs = logprobs;
    a.entropy = entropy;
    a.lse = lse;
    a.top_logprobs = top_logprobs;
    a.top_ids = top_ids;
    const cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    const cudaError_t e = d->dtype == MA_DT_BF16
                              ? (top ? forward<__nv_bfloat16, true>(a, s) : forward<__nv_bfloat16, false>(a, s))
                              : (top ? forward<float, true>(a, s) : forward<float, false>(a, s));
    if (e != cudaSuccess) return op_cuda(e, "log probabilities launch");
  }
  clear_last_error();
  return MA_OK;
}

ma_status muon_adamw_token_logprobs_backward(const ma_token_logprobs* d, const float* dlogprobs,
                                             const float* dentropy, const float* entropy, const float* lse,
                                             void* dlogits, int64_t dlogits_stride, void* cuda_stream) {
  const ma_status st = check(d);
  if (st != MA_OK) return st;
  if (d->n_tokens > 0) {
    if (!lse || !dlogits || (dentropy && !entropy))
      return op_fail(MA_ERR_ARG, "lse, dlogits and, with dentropy, entropy must not be NULL");
    if (!op_aligned(dlogprobs, 4) || !op_aligned(dentropy, 4) || !op_aligned(entropy, 4) || !op_aligned(lse, 4) ||
        !op_aligned(dlogits, op_dtype_size(d->dtype)))
      return op_fail(MA_ERR_ALIGN, "a tensor is not aligned to its elements");
    if (d->n_tokens > 1 && dlogits_stride < d->vocab)
      return op_fail(MA_ERR_SHAPE, "dlogits has rows %lld apart, below the vocabulary", (long long)dlogits_stride);
    LogprobArgs a = args_of(d);
    a.dlogprobs = dlogprobs;
    a.dentropy = dentropy;
    a.entropy_in = entropy;
    a.lse_in = lse;
    a.dlogits = dlogits;
    a.out_stride = dlogits_stride;
    a.parts = std::max((a.vocab + kGradStep * 8 - 1) / (kGradStep * 8), 1);
    // each of a row's blocks may read all of it while the others write (above kLseMax)
    if (dlogits == d->logits && a.parts > 1)
      return op_fail(MA_ERR_ARG, "dlogits are the logits, with more than %d of them in a row", kGradStep * 8);
    const dim3 grid((unsigned)(a.n * a.parts));
    const cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    const cudaError_t e = d->dtype == MA_DT_BF16
                              ? op_launch(token_logprobs_grad_kernel<__nv_bfloat16>, grid, dim3(kGradThreads), 0, s, 1, a)
                              : op_launch(token_logprobs_grad_kernel<float>, grid, dim3(kGradThreads), 0, s, 1, a);
    if (e != cudaSuccess) return op_cuda(e, "log probabilities gradient launch");
  }
  clear_last_error();
  return MA_OK;
}

}  // extern "C"
