// moe_fwd_down.hip -- the MoE forward's down projection where the contraction is
// short: each routed slot's row in scaled fp16.
//
// Per block b of expert e (tile rows = slots, columns = hidden index h,
// contraction over Ip): row[p][h] = sum_i deq(Q(s))[p][i] deq(Wd[e])[h][i], fp32
// in the accumulators, summed over a token's slots by the last kernel.  With a
// short contraction the rows' trip through memory is most of the time (T = 32768,
// I = 256, top-8: 1.6 GB written and read as fp32, against 0.2 TFLOP), so they are
// stored as fp16 times a power of two per row and 128 columns: the largest value
// lies in [2^14, 2^15), a value down to 2^-29 of it keeps 11 significant bits, so a
// term of the sum is off by at most 2^-12 of itself, an eighth of half a step of
// the bf16 result.  The scale is a row's own: no token's values touch another's.
// Long contractions (I >= 4096) keep fp32 rows and Phase 3's kernel
// (moe_phase3.hip), whose last round of tiles is cut along K.
#include <type_traits>

#include "gemm_v3.hpp"
#include "kernels.hpp"
#include "moe_tiles.hpp"
#include "mx_device.hpp"
#include "segment.hpp"

namespace mx {

namespace {
using v2::v16f;

template <int BM, int BN>
struct DownLds {
  static constexpr int PITCH = BN * 2 + 16;   // bytes of a staged fp16 row
  static constexpr int SCALES = BM * PITCH;   // then a scale per row and 128 columns
  static constexpr int BYTES = SCALES + BM * (BN / 128) * 4;
};

template <int BM, int BN, bool RAG>
__global__ void __launch_bounds__(v2::kThreads) fwd_down_kernel(MoeFwdDownArgs p) {
  using L = DownLds<BM, BN>;
  constexpr int SMEM = v3::smem_bytes(BM, BN) > L::BYTES ? v3::smem_bytes(BM, BN) : L::BYTES;
  static_assert(SMEM <= 160 * 1024, "LDS");
  __shared__ __attribute__((aligned(16))) uint8_t smem[SMEM];
  constexpr int FM = BM / 64, FN = BN / 64;
  static_assert(BN / 2 <= 128 && 128 % (BN / 2) == 0, "a wave's columns lie in one run of 128");
  BlockTiles bt;
  if (!block_tile(p.tile_start, p.flag, BM, int(p.N), blockIdx.x, p.rr_tiles, bt)) return;
  int tm, tn;
  v2::grouped_tile<8>(bt.local, bt.slots, p.tiles_n, tm, tn);
  const int64_t m0 = int64_t(tm) * BM, n0 = int64_t(tn) * BN, sbase = int64_t(bt.b) * p.B, e = p.b2e[bt.b], P = p.N * p.B;
  v16f acc[FM][FN];
  {
    v3::Op<BM> A;
    v3::Op<BN> B;
    v3::ScaleDma<BM, BN> sd;
    v3::setup_rows_sm(A, p.inter_codes, sbase + m0, sbase + p.B, P, p.Ip);
    v3::setup_rows(B, p.w_codes + e * p.H * p.I, n0, p.H, p.I);
    v3::setup_scales(sd, p.inter_scales, sbase + m0, P, P * (p.Ip / 32), p.w_scales + e * p.H * (p.Ip / 32), n0, p.H,
                     p.H * (p.Ip / 32));
    v3::mainloop<BM, BN, v3::kFp8, kE4M3, kE4M3, v3::KMapPlain, RAG ? 2 : 0>(A, B, &sd, int(p.Ip / v3::SK),
                                                                            v3::KMapPlain{}, smem, acc, uint32_t(p.I));
  }
  __syncthreads();   // the ring is done
  const int lane = threadIdx.x & 63, h = lane >> 5, r = lane & 31, wave = threadIdx.x >> 6, wm = wave >> 1, wn = wave & 1;
  float* scales = reinterpret_cast<float*>(smem + L::SCALES);
  uint32_t* half_max = reinterpret_cast<uint32_t*>(scales);   // BN == 128: a row's run spans both wave columns
  // largest magnitude of each of the lane's rows over the wave's columns
  uint32_t top[FM][16];
  v2::static_for<FM>([&](auto FI) {
    v2::static_for<16>([&](auto Q) {
      uint32_t m = 0;
      v2::static_for<FN>([&](auto FJ) { m = max(m, abs_bits(acc[FI][FJ][int(Q)])); });
      top[int(FI)][int(Q)] = seg::umax<32>(m);
    });
  });
  auto row_of = [&](int fi, int q) { return wm * (BM / 2) + 32 * fi + 8 * (q >> 2) + 4 * h + (q & 3); };
  if constexpr (BN == 128) {
    // exchange with the other wave column
    if (r == 0 && wn == 1)
      v2::static_for<FM>([&](auto FI) {
        v2::static_for<16>([&](auto Q) { half_max[row_of(FI, Q)] = top[int(FI)][int(Q)]; });
      });
    __syncthreads();
    if (wn == 0) {
      v2::static_for<FM>([&](auto FI) {
        v2::static_for<16>([&](auto Q) { top[int(FI)][int(Q)] = max(top[int(FI)][int(Q)], half_max[row_of(FI, Q)]); });
      });
    }
    __syncthreads();
    if (r == 0 && wn == 0)
      v2::static_for<FM>([&](auto FI) {
        v2::static_for<16>([&](auto Q) { half_max[row_of(FI, Q)] = top[int(FI)][int(Q)]; });
      });
    __syncthreads();
    if (wn == 1)
      v2::static_for<FM>([&](auto FI) {
        v2::static_for<16>([&](auto Q) { top[int(FI)][int(Q)] = half_max[row_of(FI, Q)]; });
      });
    __syncthreads();
  }
  v2::static_for<FM>([&](auto FI) {
    v2::static_for<16>([&](auto Q) {
      constexpr int q = Q;
      // biased exponent of the largest, at least 15 so that both scales are normal numbers
      const uint32_t ex = max(top[int(FI)][q] >> 23, 15u);
      const float mul = __uint_as_float((268u - ex) << 23);   // 2^(141 - ex): the largest in [2^14, 2^15)
      const int row = row_of(FI, q);
      uint8_t* dst = smem + row * L::PITCH + (wn * (BN / 2) + r) * 2;
      v2::static_for<FN>([&](auto FJ) {
        *reinterpret_cast<_Float16*>(dst + 64 * int(FJ)) = _Float16(acc[FI][FJ][q] * mul);
      });
      if (r == 0 && (BN == 256 || wn == 0))
        scales[row * (BN / 128) + (BN == 256 ? wn : 0)] = __uint_as_float((ex - 14u) << 23);
    });
  });
  __syncthreads();
  // 16-byte runs of whole rows; slots past the extent store too (their rows are not read)
  constexpr int RUNS = BN / 8;
  for (int k = threadIdx.x; k < BM * RUNS; k += v2::kThreads) {
    const int row = k / RUNS, c = k % RUNS;
    if (n0 + 8 * c < p.H)   // H % 32 == 0
      store_nt(p.rows + (sbase + m0 + row) * p.H + n0 + 8 * c, *reinterpret_cast<const uint4*>(smem + row * L::PITCH + 16 * c));
  }
  const int64_t hs = (p.H + 127) / 128;
  for (int k = threadIdx.x; k < BM * (BN / 128); k += v2::kThreads) {
    const int row = k / (BN / 128);
    const int64_t c = n0 / 128 + k % (BN / 128);
    if (c < hs) p.row_scale[(sbase + m0 + row) * hs + c] = scales[k];
  }
}

struct Shape {
  int m, n;
};
// 256 x 256 from blocks and contractions that are long enough (as Phase 3); 128 x 128, two workgroups a CU,
// where 128 x 256 tiles would leave CUs idle or half their columns empty
Shape down_shape(const MoeFwdDownArgs& p) {
  if (p.I >= 1024 && p.B >= 256 && p.H >= 256) return {256, 256};
  if (p.H <= 128 || p.N * (p.B / 128) * ((p.H + 255) / 256) < 256) return {128, 128};
  return {128, 256};
}

template <int BM, int BN>
hipError_t go(MoeFwdDownArgs p, hipStream_t st) {
  p.tiles_n = int((p.H + BN - 1) / BN);
  const int64_t blocks = (p.N * (p.B / BM) * p.tiles_n + 7) & ~int64_t(7);
  if (blocks > kMaxGrid256) return hipErrorInvalidValue;
  if (p.I % 128) fwd_down_kernel<BM, BN, true><<<unsigned(blocks), v2::kThreads, 0, st>>>(p);
  else fwd_down_kernel<BM, BN, false><<<unsigned(blocks), v2::kThreads, 0, st>>>(p);
  return hipGetLastError();
}
}  // namespace

bool fwd_down_fits(int64_t I) { return I < 4096 || I % 128 != 0; }

TileRangeJob fwd_down_ranges(const MoeFwdDownArgs& p) {
  const Shape t = down_shape(p);
  return {t.m, int((p.H + t.n - 1) / t.n), int(p.B), p.tile_start, nullptr, 0, 0, p.rr_tiles};
}

hipError_t launch_fwd_down(const MoeFwdDownArgs& p, hipStream_t st) {
  const Shape t = down_shape(p);
  if (t.m == 256) return go<256, 256>(p, st);
  return t.n == 256 ? go<128, 256>(p, st) : go<128, 128>(p, st);
}

}  // namespace mx
