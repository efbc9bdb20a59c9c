// router_rows.hpp -- rows of router logits in registers, shared by the router
// forward and the auxiliary losses.  L lanes take one row, EPL columns each: 8
// (L = E / 8 rounded up to a power of two, from one lane for 8 experts to a
// whole wave for 512), more past 512 experts.  A lane holds runs of four columns,
// run q of lane l at column 4 (l + L q): the lanes of a row read and write
// consecutive runs (16 bytes of fp32, 8 of bf16) where E % 4 == 0 (VEC: every run is
// then aligned, and inside the row or past it).
#pragma once
#include <type_traits>

#include "kernels.hpp"
#include "mx_device.hpp"
#include "segment.hpp"

namespace mx {
namespace rows {

// exp(d) for d <= 0 through v_exp_f32: d * log2 e rounds once, 2^-24 |d| of the
// result (results under 2^-126 may be 0).
__device__ __forceinline__ float exp_fast(float d) { return __builtin_amdgcn_exp2f(d * 1.4426950408889634f); }

// log(s) through v_log_f32, for sums of exponentials (s in [1, 4096]): v_log_f32 is
// within about an ulp, and so is the product
__device__ __forceinline__ float log_fast(float s) { return __builtin_amdgcn_logf(s) * 0.6931471805599453f; }
// 1 / s through v_rcp_f32, within about an ulp of any s whose reciprocal is a normal
// number: sums of exponentials, and balance.hip's counts (tokens, sequences times
// selections: whole numbers up to 2^31, rounded to fp32)
__device__ __forceinline__ float rcp_fast(float s) { return __builtin_amdgcn_rcpf(s); }

__device__ __forceinline__ float value(float v) { return v; }
__device__ __forceinline__ float value(uint16_t v) { return bf16_to_f32(v); }

// the column that lane holds in x[j]
template <int L>
__device__ __forceinline__ int column(int lane, int j) {
  return 4 * (lane + L * (j >> 2)) + (j & 3);
}

// x[j] = logit of column<L>(lane, j), -inf past E
template <int L, int EPL, bool VEC, class LT>
__device__ __forceinline__ void load(const LT* row, int E, int lane, float (&x)[EPL]) {
#pragma unroll
  for (int j = 0; j < EPL; j += 4) {
    const int c = column<L>(lane, j);
    if constexpr (VEC) {
      if (c < E) {
        if constexpr (std::is_same_v<LT, float>) {
          const float4 a = *reinterpret_cast<const float4*>(row + c);
          x[j] = a.x; x[j + 1] = a.y; x[j + 2] = a.z; x[j + 3] = a.w;
        } else {
          const uint2 a = *reinterpret_cast<const uint2*>(row + c);
          x[j] = __uint_as_float(a.x << 16); x[j + 1] = __uint_as_float(a.x & 0xffff0000u);
          x[j + 2] = __uint_as_float(a.y << 16); x[j + 3] = __uint_as_float(a.y & 0xffff0000u);
        }
      } else {
        x[j] = x[j + 1] = x[j + 2] = x[j + 3] = -INFINITY;
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {   // past E: the last column again, so that no load hangs on a branch
        const float v = value(row[c + k < E ? c + k : E - 1]);
        x[j + k] = c + k < E ? v : -INFINITY;
      }
    }
  }
}

// the same columns of an fp32 row
template <int L, int EPL, bool VEC>
__device__ __forceinline__ void store(float* row, int E, int lane, const float (&x)[EPL]) {
#pragma unroll
  for (int j = 0; j < EPL; j += 4) {
    const int c = column<L>(lane, j);
    if constexpr (VEC) {
      if (c < E) *reinterpret_cast<float4*>(row + c) = float4{x[j], x[j + 1], x[j + 2], x[j + 3]};
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (c + k < E) row[c + k] = x[j + k];
    }
  }
}

// Softmax of a row over its L lanes: x becomes p; false (x = 0) where no logit
// is above -inf.
template <int L, int EPL>
__device__ __forceinline__ bool softmax(float (&x)[EPL], float& lse) {
  float m = x[0];
#pragma unroll
  for (int j = 1; j < EPL; ++j) m = fmaxf(m, x[j]);
  m = seg::max<L>(m);
  const bool some = m > -INFINITY;
  if (!some) m = 0.f;   // exp(-inf - 0) = 0
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    x[j] = exp_fast(x[j] - m);
    s += x[j];
  }
  s = seg::sum<L>(s);
  const float inv = some ? rcp_fast(s) : 0.f;
#pragma unroll
  for (int j = 0; j < EPL; ++j) x[j] *= inv;
  lse = some ? m + log_fast(s) : 0.f;
  return some;
}

// f(L, EPL, VEC) for E experts
template <int N> using Int = std::integral_constant<int, N>;
template <class F>
void by_experts(int64_t E, const F& f) {
  auto go = [&](auto L, auto EPL) {
    if (E % 4 == 0) f(L, EPL, std::true_type{});
    else f(L, EPL, std::false_type{});
  };
  if (E <= 8) go(Int<1>{}, Int<8>{});
  else if (E <= 16) go(Int<2>{}, Int<8>{});
  else if (E <= 32) go(Int<4>{}, Int<8>{});
  else if (E <= 64) go(Int<8>{}, Int<8>{});
  else if (E <= 128) go(Int<16>{}, Int<8>{});
  else if (E <= 256) go(Int<32>{}, Int<8>{});
  else if (E <= 512) go(Int<64>{}, Int<8>{});
  else if (E <= 1024) go(Int<64>{}, Int<16>{});
  else if (E <= 2048) go(Int<64>{}, Int<32>{});
  else go(Int<64>{}, Int<64>{});
}
inline int lanes(int64_t E) {
  int l = 1;
  while (l < 64 && l * 8 < E) l *= 2;
  return l;
}

// tokens of one launch: L threads each, under 2^32 in all
inline int64_t max_tokens(int64_t E) { return ((int64_t(1) << 32) - 65536) / lanes(E); }

}  // namespace rows
}  // namespace mx
