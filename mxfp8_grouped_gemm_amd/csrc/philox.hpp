// philox.hpp -- the counter-based generator of the dropout masks: Philox4x32
// with 10 rounds (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", 2011).  A mask is a function of (seed, offset, element), so
// it is computed wherever it is needed and never stored.
//
// Element i of a tensor (its index in row-major order, whatever the strides)
// takes 16 bits: half i % 2 (0: the low one) of word (i % 8) / 2 at counter
// (i / 8, offset), the key being the seed.  It is dropped where those bits are
// below thr = round(65536 p), and scaled by 65536 / (65536 - thr) elsewhere:
// the expectation is kept exactly for the p that is applied, a multiple of
// 2^-16.  16 bits an element, because a counter's 10 rounds cost about 100
// instructions, 40 of them multiplications at a quarter of the rate: one a
// 4 elements would bound the kernel by arithmetic, one an 8 elements does not.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mx {

struct DropoutRule {
  uint32_t thr;         // 0: nothing is dropped (rng is not read); 65536: everything
  float scale;          // 65536 / (65536 - thr); 0 with thr == 65536
  const int64_t* rng;   // device: seed, offset
};

struct PhiloxKey {
  uint32_t k0, k1, o0, o1;
  __device__ __forceinline__ explicit PhiloxKey(const int64_t* rng) {
    const uint64_t s = uint64_t(rng[0]), o = uint64_t(rng[1]);
    k0 = uint32_t(s);
    k1 = uint32_t(s >> 32);
    o0 = uint32_t(o);
    o1 = uint32_t(o >> 32);
  }
};

// the 8 x 16 bits of counter g
__device__ __forceinline__ uint4 philox(const PhiloxKey& key, uint64_t g) {
  uint32_t x0 = uint32_t(g), x1 = uint32_t(g >> 32), x2 = key.o0, x3 = key.o1, k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = uint64_t(x0) * 0xD2511F53u, b = uint64_t(x2) * 0xCD9E8D57u;
    x0 = uint32_t(b >> 32) ^ x1 ^ k0;
    x1 = uint32_t(b);
    x2 = uint32_t(a >> 32) ^ x3 ^ k1;
    x3 = uint32_t(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(x0, x1, x2, x3);
}

// element j (0..7) of a counter's group: kept?
__device__ __forceinline__ bool philox_keep(const uint4& w, int j, uint32_t thr) {
  const uint32_t x = j < 2 ? w.x : j < 4 ? w.y : j < 6 ? w.z : w.w;
  return ((j & 1) ? x >> 16 : x & 0xffffu) >= thr;
}

}  // namespace mx
