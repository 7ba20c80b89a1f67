// Which elements dropout keeps, recomputed wherever it is asked for.
//
// Sixteen bits for each element from Philox4x32-10 (Salmon, Moraes, Dror and
// Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011): the key is the
// 64-bit seed, the counter the element's group of eight, the call's site and
// the 64-bit step. A call of the generator gives a group's 128 bits: word i / 2
// of the result has element i in its low half where i is even. An element is
// kept where its bits are at least `threshold`, p in units of 2^-16. Sixteen
// bits instead of 32 halve the integer work, which would otherwise take as long
// as the memory does.
#pragma once

#include <stdint.h>

namespace ma {

struct DropArgs {
  const int64_t* rng;  // seed, step
  uint32_t site, threshold;
  float factor;  // 1 / (1 - p), 0 where nothing is kept
};

namespace {

struct DropKey {
  uint32_t k0, k1, site, step0, step1;
  uint32_t threshold_up;  // the threshold in the upper half
  float factor;
};

__device__ __forceinline__ DropKey drop_key(const DropArgs& a) {
  const uint64_t seed = (uint64_t)__ldg(a.rng), step = (uint64_t)__ldg(a.rng + 1);
  return {(uint32_t)seed, (uint32_t)(seed >> 32), a.site, (uint32_t)step, (uint32_t)(step >> 32), a.threshold << 16,
          a.factor};
}

// Ten rounds over N counters in step, which form each round's keys once.
template <int N>
__device__ __forceinline__ void philox(uint4 (&c)[N], uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const uint64_t a = (uint64_t)c[j].x * 0xD2511F53u, b = (uint64_t)c[j].z * 0xCD9E8D57u;
      c[j] = make_uint4((uint32_t)(b >> 32) ^ c[j].y ^ k0, (uint32_t)b, (uint32_t)(a >> 32) ^ c[j].w ^ k1, (uint32_t)a);
    }
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
}

// Eight elements by their bits, four words of them. Dropped ones become 0 whatever they hold.
__device__ __forceinline__ void drop8_by(const DropKey& k, const uint4& bits, float (&x)[8]) {
  if (k.factor == 0.f) {  // p = 1, whose threshold no 16 bits reach
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.f;
    return;
  }
  const uint32_t w[4] = {bits.x, bits.y, bits.z, bits.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // the threshold lies in the upper half: the high element compares as it is, the low one moved up
    x[2 * i] = w[i] << 16 >= k.threshold_up ? x[2 * i] * k.factor : 0.f;
    x[2 * i + 1] = w[i] >= k.threshold_up ? x[2 * i + 1] * k.factor : 0.f;
  }
}

// The eight elements of each of N groups, `stride` apart from `group` on.
template <int N>
__device__ __forceinline__ void drop8(const DropKey& k, uint32_t group, uint32_t stride, float (&x)[N][8]) {
  uint4 c[N];
#pragma unroll
  for (int j = 0; j < N; ++j) c[j] = make_uint4(group + j * stride, k.site, k.step0, k.step1);
  philox(c, k.k0, k.k1);
#pragma unroll
  for (int j = 0; j < N; ++j) drop8_by(k, c[j], x[j]);
}

}  // namespace

// Of a probability and where the generator stands; false if p is outside [0, 1].
bool drop_args(double p, const int64_t* rng, int32_t site, DropArgs* out);

}  // namespace ma
