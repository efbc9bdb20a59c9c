// quantize_t.hip -- MXFP8 quantisation of a batch of matrices along their rows,
// written transposed: x [G][R][C] bf16 -> codes [G][C][R], scales [G][C][R/32],
// so that the quantised axis (the one a product contracts over) is contiguous.
//
// Bound by memory: 2 bytes read and 1.03 written an element.  A workgroup takes
// 128 rows x 128 columns; wave w rows 32w .. 32w + 31 (one group), lane l the
// columns 2l and 2l + 1, so each of its 32 loads is 256 consecutive bytes of a
// row and a lane holds two whole groups in registers.  The codes go through LDS,
// where 8 lanes then write a column's 128 bytes at once.  16 matrices of 2048 x 2816:
// 48 us, 5.8 TB/s (a copy of 1 GiB runs at 5.1); 77 us with each lane storing its own
// 32-byte pieces.  Loads and stores go through the caches: nontemporal loads cost rows
// that start inside a line a quarter (1184 x 2116: 41 -> 52 us) and the others a tenth,
// nontemporal stores 3 us of the 48.
// Widths that are no whole lines cost by the lines that a tile's 256-byte pieces of a row
// touch, three in place of two: 22 x 1184 x 2176 31 us, 5.6 TB/s, 2116 36, 4.6, and 2115 42, 4.0,
// where every other row is shifted by half a word besides (rows of whole lines in the
// result, 1280 for 1184, change neither).
#include <type_traits>

#include "kernels.hpp"
#include "mx_device.hpp"

namespace mx {

namespace {
constexpr int kT = 128;        // tile: rows and columns
constexpr int kPitch = kT + 16;   // LDS bytes of a column's codes

// PAIRED: C even, so a lane's two columns are one aligned word.
template <int FMT, bool PAIRED>
__global__ void __launch_bounds__(256) quantize_t_kernel(const uint16_t* __restrict__ x, int64_t R, int64_t C,
                                                         int tiles_r, int tiles_c, uint8_t* __restrict__ codes,
                                                         uint8_t* __restrict__ scales) {
  const int tc = blockIdx.x % tiles_c, rest = blockIdx.x / tiles_c, tr = rest % tiles_r;
  const int64_t m = rest / tiles_r;
  const int lane = threadIdx.x & 63;
  const int64_t r0 = int64_t(tr) * kT + 32 * (threadIdx.x >> 6), c = int64_t(tc) * kT + 2 * lane;
  __shared__ __attribute__((aligned(16))) uint8_t tile[kT * kPitch];
  __shared__ uint32_t tile_scales[kT];
  const bool in = r0 < R && c < C, two = c + 1 < C;
  const uint16_t* src = x + (m * R + r0) * C + c;
  uint32_t w[32], am = 0;
#pragma unroll
  for (int r = 0; r < 32; ++r) w[r] = 0;
  if constexpr (PAIRED) {
    if (in) {
#pragma unroll
      for (int r = 0; r < 32; ++r) w[r] = *reinterpret_cast<const uint32_t*>(src + r * C);
    }
  } else if (int64_t(blockIdx.x) + 1 < gridDim.x) {
    // odd C: every other row's pairs straddle two words, the second of which is the next lane's first
    // (22 matrices of 1184 x 2115: 42 us, 75 with 2-byte loads).  A word may reach past the tile, not past x:
    // the last tile takes the other way.
    const uint32_t* words = reinterpret_cast<const uint32_t*>(x);
    if (r0 < R) {   // whole waves
      uint32_t tail[32];
#pragma unroll
      for (int r = 0; r < 32; ++r) {
        const int64_t at = (m * R + r0 + r) * C + (c < C ? c : C - 1);
        w[r] = words[at >> 1];
        tail[r] = lane == 63 && (at & 1) && two ? words[(at >> 1) + 1] : 0u;
      }
#pragma unroll
      for (int r = 0; r < 32; ++r) {
        const uint32_t next = uint32_t(__builtin_amdgcn_update_dpp(int(tail[r]), int(w[r]), 0x130, 0xf, 0xf, false));
        const bool odd = ((m * R + r0 + r) * C & 1) != 0;   // c is even
        w[r] = odd ? (w[r] >> 16) | (next << 16) : w[r];
        w[r] = two ? w[r] : c < C ? w[r] & 0xffffu : 0u;
      }
    }
  } else if (in) {
#pragma unroll
    for (int r = 0; r < 32; ++r) w[r] = uint32_t(src[r * C]) | (two ? uint32_t(src[r * C + 1]) << 16 : 0u);
  }
#pragma unroll
  for (int r = 0; r < 32; ++r) am = absmax_bf16x2(am, w[r]);
  const int X0 = scale_exp<FMT>(am << 16), X1 = scale_exp<FMT>(am & 0xffff0000u);
  const uint32_t lim = bf16_limit<FMT>(X0) | (bf16_limit<FMT>(X1) << 16);
  const float s0 = cvt_scale(X0), s1 = cvt_scale(X1);
  uint32_t p0[8], p1[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const uint32_t a = clamp_bf16x2(w[4 * q], lim), b = clamp_bf16x2(w[4 * q + 1], lim);
    const uint32_t d = clamp_bf16x2(w[4 * q + 2], lim), e = clamp_bf16x2(w[4 * q + 3], lim);
    p0[q] = encode_bf16x4<FMT>(lo_halves(a, b), lo_halves(d, e), s0);
    p1[q] = encode_bf16x4<FMT>(hi_halves(a, b), hi_halves(d, e), s1);
  }
  const int wave = threadIdx.x >> 6;
  uint4* dst = reinterpret_cast<uint4*>(tile + 2 * lane * kPitch + 32 * wave);
  dst[0] = make_uint4(p0[0], p0[1], p0[2], p0[3]);
  dst[1] = make_uint4(p0[4], p0[5], p0[6], p0[7]);
  dst += kPitch / 16;
  dst[0] = make_uint4(p1[0], p1[1], p1[2], p1[3]);
  dst[1] = make_uint4(p1[4], p1[5], p1[6], p1[7]);
  uint8_t* sc = reinterpret_cast<uint8_t*>(tile_scales + 2 * lane) + wave;
  sc[0] = uint8_t(X0 + 127);
  sc[4] = uint8_t(X1 + 127);
  __syncthreads();
  const int64_t c0 = int64_t(tc) * kT, row0 = m * C + c0, first = int64_t(tr) * kT;   // of the result
  const int q = threadIdx.x & 7;
  if (first + 16 * q < R) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int col = 32 * k + (threadIdx.x >> 3);
      if (c0 + col < C)
        *reinterpret_cast<uint4*>(codes + (row0 + col) * R + first + 16 * q) = *reinterpret_cast<const uint4*>(tile + col * kPitch + 16 * q);
    }
  }
  if (threadIdx.x < kT && c0 + threadIdx.x < C) {
    const uint32_t v = tile_scales[threadIdx.x];
    uint8_t* to = scales + (row0 + threadIdx.x) * (R / 32) + first / 32;
    if (R % 128 == 0 && (reinterpret_cast<uintptr_t>(scales) & 3) == 0) {   // scales: of any alignment
      *reinterpret_cast<uint32_t*>(to) = v;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (first + 32 * k < R) to[k] = uint8_t(v >> (8 * k));
    }
  }
}
}  // namespace

int64_t quantize_t_grid(int64_t G, int64_t R, int64_t C) {
  const int64_t tr = (R + kT - 1) / kT, tc = (C + kT - 1) / kT;
  if (tr > kMaxGrid256 || tc > kMaxGrid256 || tr * tc > kMaxGrid256 || G > kMaxGrid256) return kMaxGrid256 + 1;
  return G * tr * tc;
}

hipError_t launch_quantize_t(const uint16_t* x, int64_t G, int64_t R, int64_t C, int fmt, uint8_t* codes,
                             uint8_t* scales, hipStream_t st) {
  const int64_t grid = quantize_t_grid(G, R, C);
  if (grid == 0) return hipSuccess;
  if (grid > kMaxGrid256) return hipErrorInvalidValue;
  const int tr = int((R + kT - 1) / kT), tc = int((C + kT - 1) / kT);
  auto go = [&](auto f, auto paired) {
    quantize_t_kernel<f(), paired()><<<unsigned(grid), 256, 0, st>>>(x, R, C, tr, tc, codes, scales);
  };
  auto kind = [&](auto f) {
    if (C % 2 == 0) go(f, std::true_type{});
    else go(f, std::false_type{});
  };
  if (fmt == kE4M3) kind(std::integral_constant<int, kE4M3>{});
  else kind(std::integral_constant<int, kE5M2>{});
  return hipGetLastError();
}

}  // namespace mx
