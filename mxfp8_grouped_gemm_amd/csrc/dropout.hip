// dropout.hip -- dropout with a residual, and its backward.
//
//   y = residual + (keep(i) ? x * scale : 0)     fp32, rounded once
// The mask comes from philox.hpp's counters, so the backward (the same kernel
// on dy, no residual) recomputes it; a dropped element gives 0 whatever it
// holds.  Bound by memory: 2 or 3 element sizes an element.  A thread takes the
// 8 elements of one counter.  Measured: 16384 x 4096 bf16 with a residual 58 us,
// 6.9 TB/s (rows 4104 apart 65); 5003 x 1501 fp32 without 9.5 us, 6.3 TB/s.
// Rows at a stride whose width or stride is no whole number of 8 columns or 16 bytes
// go element by element (16384 x 4095 in rows of 4096: 239 us, 1.7 TB/s, fp32 627; contiguous
// 59 and 138): a counter's 8 elements lie across two rows and at any alignment there.
#include "kernels.hpp"
#include "mx_device.hpp"
#include "philox.hpp"
#include "swiglu.hpp"

namespace mx {

namespace {
constexpr int kThreads = 256;

template <bool BF16>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&v)[8]) {
  if constexpr (BF16) {
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = lo_bf16(a[k]);
      v[2 * k + 1] = hi_bf16(a[k]);
    }
  } else {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    const float4 a = q[0], b = q[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}
template <bool BF16>
__device__ __forceinline__ void store8(void* p, int64_t at, const float (&v)[8]) {
  if constexpr (BF16) {
    store_nt(static_cast<uint16_t*>(p) + at, make_uint4(bf16x2_pack(v[0], v[1]), bf16x2_pack(v[2], v[3]),
                                                        bf16x2_pack(v[4], v[5]), bf16x2_pack(v[6], v[7])));
  } else {
    float* q = static_cast<float*>(p) + at;
    store_nt(q, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
    store_nt(q + 4, make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])));
  }
}
template <bool BF16>
__device__ __forceinline__ float load1(const void* p, int64_t at) {
  if constexpr (BF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[at]);
  else return static_cast<const float*>(p)[at];
}
template <bool BF16>
__device__ __forceinline__ void store1(void* p, int64_t at, float v) {
  if constexpr (BF16) static_cast<uint16_t*>(p)[at] = uint16_t(bf16x2_pack(v, 0.f));
  else static_cast<float*>(p)[at] = v;
}

// How the elements lie: kFlat, all tensors contiguous; kRows, every row a whole
// number of counters at 8-element-aligned addresses; kAny, element by element.
constexpr int kFlat = 0, kRows = 1, kAny = 2;

template <bool BF16, bool RES, int MODE>
__global__ void __launch_bounds__(kThreads) dropout_kernel(DropoutArgs p) {
  const int64_t n = p.rows * p.cols;
  const int64_t g = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (g * 8 >= n) return;
  uint4 w = make_uint4(0u, 0u, 0u, 0u);
  if (p.rule.thr) w = philox(PhiloxKey(p.rule.rng), uint64_t(g));   // thr == 0: every element is kept
  int64_t ax = g * 8, ar = ax, ay = ax;
  if constexpr (MODE == kRows) {
    const int64_t per = p.cols / 8, r = g / per, c = (g - r * per) * 8;
    ax = r * p.ldx + c;
    ar = r * p.ldr + c;
    ay = r * p.ldy + c;
  }
  if (MODE != kAny && g * 8 + 8 <= n) {
    float x[8], res[8];
    load8<BF16>(p.x, ax, x);
    if constexpr (RES) load8<BF16>(p.residual, ar, res);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float v = philox_keep(w, j, p.rule.thr) ? x[j] * p.rule.scale : 0.f;
      x[j] = RES ? v + res[j] : v;
    }
    store8<BF16>(p.y, ay, x);
    return;
  }
  for (int j = 0; j < 8 && g * 8 + j < n; ++j) {
    const int64_t i = g * 8 + j, r = i / p.cols, c = i - r * p.cols;
    float v = philox_keep(w, j, p.rule.thr) ? load1<BF16>(p.x, r * p.ldx + c) * p.rule.scale : 0.f;
    if constexpr (RES) v += load1<BF16>(p.residual, r * p.ldr + c);
    store1<BF16>(p.y, r * p.ldy + c, v);
  }
}

template <bool BF16, bool RES>
void go(const DropoutArgs& p, int mode, unsigned grid, hipStream_t st) {
  if (mode == kFlat) dropout_kernel<BF16, RES, kFlat><<<grid, kThreads, 0, st>>>(p);
  else if (mode == kRows) dropout_kernel<BF16, RES, kRows><<<grid, kThreads, 0, st>>>(p);
  else dropout_kernel<BF16, RES, kAny><<<grid, kThreads, 0, st>>>(p);
}
}  // namespace

hipError_t launch_dropout(const DropoutArgs& p, hipStream_t st) {
  const int64_t n = p.rows * p.cols, grid = ((n + 7) / 8 + kThreads - 1) / kThreads;
  if (grid == 0) return hipSuccess;
  if (grid > kMaxGrid256) return hipErrorInvalidValue;
  const int64_t per16 = p.bf16 ? 8 : 4;   // elements of 16 bytes
  auto whole = [&](int64_t ld) { return ld % per16 == 0; };
  int mode = kAny;
  if (p.rows == 1 || (p.ldx == p.cols && p.ldy == p.cols && (!p.residual || p.ldr == p.cols))) mode = kFlat;
  else if (p.cols % 8 == 0 && whole(p.ldx) && whole(p.ldy) && (!p.residual || whole(p.ldr))) mode = kRows;
  if (p.bf16) {
    if (p.residual) go<true, true>(p, mode, unsigned(grid), st);
    else go<true, false>(p, mode, unsigned(grid), st);
  } else {
    if (p.residual) go<false, true>(p, mode, unsigned(grid), st);
    else go<false, false>(p, mode, unsigned(grid), st);
  }
  return hipGetLastError();
}

}  // namespace mx
