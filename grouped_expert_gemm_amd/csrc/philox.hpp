// Counter-based random bits for dropout: Philox4x32-10 (Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", 2011). Value i of a tensor takes 16 of the 128
// bits that the generator gives for the counter (i / 8, offset), 64 bits each, and the key
// `seed`: half i % 8 of its four words, low halves first. Nothing but (seed, offset) is kept
// between the passes that need the same mask.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "geg_launch.hpp"

namespace geg {

struct PhiloxState {
  uint32_t k0, k1, c2, c3;
  __device__ __forceinline__ explicit PhiloxState(const DropoutArgs& d) {
    uint64_t key = d.seed, off = d.offset;
    if (d.dev) {
      key = d.dev[0];
      off += d.dev[1];
    }
    k0 = (uint32_t)key;
    k1 = (uint32_t)(key >> 32);
    c2 = (uint32_t)off;
    c3 = (uint32_t)(off >> 32);
  }
  // The 8 x 16 bits of values 8 block .. 8 block + 7, two per word.
  __device__ __forceinline__ void bits(uint64_t block, uint32_t w[4]) const {
    uint32_t a = (uint32_t)block, b = (uint32_t)(block >> 32), c = c2, d = c3, x = k0, y = k1;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
      const uint64_t p = (uint64_t)0xD2511F53u * a, q = (uint64_t)0xCD9E8D57u * c;
      a = (uint32_t)(q >> 32) ^ b ^ x;
      b = (uint32_t)q;
      c = (uint32_t)(p >> 32) ^ d ^ y;
      d = (uint32_t)p;
      x += 0x9E3779B9u;
      y += 0xBB67AE85u;
    }
    w[0] = a;
    w[1] = b;
    w[2] = c;
    w[3] = d;
  }
};

// Whether value i (of the 8) stays.
__device__ __forceinline__ bool philox_kept(const uint32_t w[4], int i, uint32_t threshold) {
  return ((w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu) >= threshold;
}

}  // namespace geg
