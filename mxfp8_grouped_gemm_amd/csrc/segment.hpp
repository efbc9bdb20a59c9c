// segment.hpp -- reductions over segments of L consecutive lanes (L a power of
// two up to 64) that stay in the register file: quad_perm, row_half_mirror and
// row_mirror DPP moves within 16 lanes, v_permlane16_swap / v_permlane32_swap
// beyond.  After each step every lane of the reduced group holds the same
// value, so a mirror serves as the exchange with the other half.  Each step
// combines two values with a commutative operation: all lanes of a segment end
// with the same bits.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mx {
namespace seg {

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
  return uint32_t(__builtin_amdgcn_update_dpp(0, int(x), CTRL, 0xf, 0xf, true));
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;

template <int L, class Op>
__device__ __forceinline__ uint32_t reduce(uint32_t x, const Op& op) {
  static_assert(L >= 1 && L <= 64 && (L & (L - 1)) == 0, "a power of two");
#if defined(__HIP_DEVICE_COMPILE__)
  if constexpr (L > 1) x = op(x, dpp<kXor1>(x));
  if constexpr (L > 2) x = op(x, dpp<kXor2>(x));
  if constexpr (L > 4) x = op(x, dpp<kHalfMirror>(x));
  if constexpr (L > 8) x = op(x, dpp<kMirror>(x));
  if constexpr (L > 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    x = op(r[0], r[1]);
  }
  if constexpr (L > 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    x = op(r[0], r[1]);
  }
#endif
  return x;
}
template <int L>
__device__ __forceinline__ float sum(float v) {
  return __uint_as_float(reduce<L>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
template <int L>
__device__ __forceinline__ float max(float v) {   // NaN only where every value is NaN
  return __uint_as_float(reduce<L>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
template <int L>
__device__ __forceinline__ uint32_t umax(uint32_t v) {
  return reduce<L>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int L>
__device__ __forceinline__ uint32_t umin(uint32_t v) {
  return reduce<L>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}


// Sum over the lanes of a wave that are congruent modulo L (the same column of
// the wave's 64 / L segments), in every lane: exact exchanges (quad_perm,
// rotations within 16 lanes, row swaps), since lanes of a segment differ.
constexpr int kRor4 = 0x124, kRor8 = 0x128;
template <int L>
__device__ __forceinline__ float across(float v) {
#if defined(__HIP_DEVICE_COMPILE__)
  auto add = [&](uint32_t b) { v += __uint_as_float(b); };
  if constexpr (L <= 1) add(dpp<kXor1>(__float_as_uint(v)));
  if constexpr (L <= 2) add(dpp<kXor2>(__float_as_uint(v)));
  if constexpr (L <= 8) add(dpp<kRor8>(__float_as_uint(v)));
  if constexpr (L <= 4) add(dpp<kRor4>(__float_as_uint(v)));
  if constexpr (L <= 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (L <= 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
#endif
  return v;
}
// the two words of a double move the same way
template <int L>
__device__ __forceinline__ double across(double v) {
#if defined(__HIP_DEVICE_COMPILE__)
  auto add = [&](auto move) { v += __hiloint2double(int(move(__double2hiint(v))), int(move(__double2loint(v)))); };
  if constexpr (L <= 1) add([](int x) { return dpp<kXor1>(x); });
  if constexpr (L <= 2) add([](int x) { return dpp<kXor2>(x); });
  if constexpr (L <= 8) add([](int x) { return dpp<kRor8>(x); });
  if constexpr (L <= 4) add([](int x) { return dpp<kRor4>(x); });
  auto swap = [&](auto rows) {
    const auto hi = rows(__double2hiint(v)), lo = rows(__double2loint(v));
    v = __hiloint2double(int(hi[0]), int(lo[0])) + __hiloint2double(int(hi[1]), int(lo[1]));
  };
  if constexpr (L <= 16) swap([](int x) { return __builtin_amdgcn_permlane16_swap(x, x, false, false); });
  if constexpr (L <= 32) swap([](int x) { return __builtin_amdgcn_permlane32_swap(x, x, false, false); });
#endif
  return v;
}

}  // namespace seg
}  // namespace mx
