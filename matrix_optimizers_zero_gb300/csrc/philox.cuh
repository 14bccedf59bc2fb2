// Counter-based random numbers: Philox4x32-10 (Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", 2011). A number depends only
// on its element's index, the seed and the offset, so a mask or a rounding
// can be drawn again in any launch order and never needs to be stored.
//
// One call gives 128 bits for a group of eight consecutive elements, 16 bits
// each: element i takes half i % 2 (low first) of word (i % 8) / 2 of the
// call whose counter is (i / 8, offset), both 64-bit, under the key `seed`.
// 16 bits an element (probabilities in steps of 2^-16) instead of 32 halve
// the integer work: at 32 bits it would bound the streaming kernels instead
// of memory (10 rounds are 20 wide multiplies and 40 logic operations).
#pragma once

#include <cstdint>

namespace mo {

// Seed and offset of a launch; `offset_dev`, when set, is added to `offset`
// when the kernel runs (a captured step can advance it between replays).
struct RandomArgs {
  uint64_t seed = 0;
  uint64_t offset = 0;
  const uint64_t* offset_dev = nullptr;
};

// A launch's dropout: an element is kept where its number is at least
// `threshold` (out of 65536); threshold 0 keeps all.
struct DropArgs {
  RandomArgs rnd;
  uint32_t threshold = 0;
  float factor = 1.0f;   // 65536 / (65536 - threshold); 0 when nothing is kept
};

#ifdef __CUDACC__

struct Philox {
  uint32_t k0, k1, o0, o1;

  __device__ __forceinline__ Philox() : k0(0), k1(0), o0(0), o1(0) {}
  __device__ __forceinline__ Philox(const RandomArgs& a, uint64_t stream = 0) {
    const uint64_t o = a.offset + (a.offset_dev != nullptr ? *a.offset_dev : 0) + stream;
    k0 = uint32_t(a.seed);
    k1 = uint32_t(a.seed >> 32);
    o0 = uint32_t(o);
    o1 = uint32_t(o >> 32);
  }

  // the eight 16-bit numbers of group j, two a word
  __device__ __forceinline__ uint4 group(uint64_t j) const { return group(uint32_t(j >> 32), uint32_t(j)); }
  // (calls that share the upper half share two of the twenty products)
  __device__ __forceinline__ uint4 group(uint32_t j_hi, uint32_t j_lo) const {
    uint32_t a = j_lo, b = j_hi, c = o0, d = o1, x = k0, y = k1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
      const uint64_t p = uint64_t(a) * 0xD2511F53u;
      const uint64_t q = uint64_t(c) * 0xCD9E8D57u;
      a = uint32_t(q >> 32) ^ b ^ x;
      b = uint32_t(q);
      c = uint32_t(p >> 32) ^ d ^ y;
      d = uint32_t(p);
      x += 0x9E3779B9u;
      y += 0xBB67AE85u;
    }
    return make_uint4(a, b, c, d);
  }

  // the number of one element (a whole call for it: for ragged edges)
  __device__ __forceinline__ uint32_t element(uint64_t i) const {
    const uint4 g = group(i >> 3);
    const uint32_t k = uint32_t(i & 7u);
    const uint32_t w = k < 4 ? (k < 2 ? g.x : g.y) : (k < 6 ? g.z : g.w);
    return (k & 1u) ? w >> 16 : w & 0xFFFFu;
  }
};

// The number of element k (0-7) of a group.
__device__ __forceinline__ uint32_t philox_half(const uint4& g, int k) {
  const uint32_t w = k < 4 ? (k < 2 ? g.x : g.y) : (k < 6 ? g.z : g.w);
  return (k & 1) ? w >> 16 : w & 0xFFFFu;
}

#endif  // __CUDACC__

}  // namespace mo
