// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", 2011): four random words from a counter and a key, in ten
// rounds of two 32 x 32-bit products.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nvfp4 {

__device__ __forceinline__ void philox(uint32_t (&c)[4], uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)0xD2511F53u * c[0], b = (uint64_t)0xCD9E8D57u * c[2];
    const uint32_t n0 = (uint32_t)(b >> 32) ^ c[1] ^ k0, n2 = (uint32_t)(a >> 32) ^ c[3] ^ k1;
    c[1] = (uint32_t)b;
    c[3] = (uint32_t)a;
    c[0] = n0;
    c[2] = n2;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
}

// Dropout's random bits: eight neighbours of a row, columns 8 v to 8 v + 7 of
// row t, take the eight halves of one counter's words.
struct Mask8 {
  uint32_t w[4];
  __device__ __forceinline__ Mask8(uint32_t v, uint32_t t, uint64_t seed, uint64_t offset) {
    w[0] = v;
    w[1] = t;
    w[2] = (uint32_t)offset;
    w[3] = (uint32_t)(offset >> 32);
    philox(w, (uint32_t)seed, (uint32_t)(seed >> 32));
  }
  __device__ __forceinline__ bool keeps(int i, uint32_t cut) const {
    return (i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu) >= cut;
  }
};

}  // namespace nvfp4
