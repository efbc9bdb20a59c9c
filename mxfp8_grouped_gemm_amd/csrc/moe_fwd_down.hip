// moe_fwd_down.hip -- the MoE forward's down projection where the contraction is
// short: each routed slot's row in scaled fp16.
//
// Per block b of expert e (tile rows = hidden index h, tile columns = slots,
// contraction over Ip): row[p][h] = sum_i deq(Q(s))[p][i] deq(Wd[e])[h][i], fp32
// in the accumulators, summed over a token's slots by the last kernel.  With a
// short contraction the rows' trip through memory is most of the time (T = 32768,
// I = 256, top-8: 1.6 GB written and read as fp32, against 0.2 TFLOP), so they are
// stored as fp16 times a power of two per row and 64 columns: the largest value
// lies in [2^14, 2^15), a value down to 2^-28 of it is a normal fp16 number of 11
// significant bits, so a term of the sum is off by at most 2^-11 of itself, an eighth
// of the 2^-8 of the bf16 result's rounding; a smaller one by at most 2^-25, that is
// 2^-39 of the largest.  The scale is a row's own: no token's values touch another's.
// With the slots as tile columns a lane holds 32 of a slot's 64 values, the lane 32
// away the rest, and 4 of them in a row: one exchange a maximum, 8-byte stores.
// 32768 slots, H = 2048, I = 1408: 145 us, 1.3 PFLOP/s.  I <= 256 has a kernel of its own
// (moe_fwd_down_short.hip).  Long contractions (I >= 4096) keep fp32 rows and Phase 3's kernel
// (moe_phase3.hip), whose last round of tiles is cut along K.
#include "gemm_v3.hpp"
#include "kernels.hpp"
#include "moe_tiles.hpp"
#include "mx_device.hpp"

namespace mx {

namespace {
using v2::v16f;

// Staged results: a slot's fp16 values, BM of them, then its scales.
template <int BM, int BN>
struct DownLds {
  static constexpr int PITCH = BM * 2 + 16;   // bytes of a slot
  static constexpr int SCALES = BN * PITCH;
  static constexpr int BYTES = SCALES + BN * (BM / 64) * 4;
};

template <int BM, int BN, bool RAG>
__global__ void __launch_bounds__(v2::kThreads) fwd_down_kernel(MoeFwdDownArgs p) {
  using L = DownLds<BM, BN>;
  constexpr int SMEM = v3::smem_bytes(BM, BN) > L::BYTES ? v3::smem_bytes(BM, BN) : L::BYTES;
  static_assert(SMEM <= 160 * 1024, "LDS");
  __shared__ __attribute__((aligned(16))) uint8_t smem[SMEM];
  constexpr int FM = BM / 64, FN = BN / 64, NS = BM / 64;   // NS: runs of 64 values a slot
  BlockTiles bt;
  if (!block_tile(p.tile_start, p.flag, BN, int(p.N), blockIdx.x, p.rr_tiles, bt)) return;
  int tm, tn;
  v2::grouped_tile<8>(bt.local, p.tiles_m, bt.slots, tm, tn);
  const int64_t m0 = int64_t(tm) * BM, n0 = int64_t(tn) * BN, sbase = int64_t(bt.b) * p.B, e = p.b2e[bt.b], P = p.N * p.B;
  v16f acc[FM][FN];
  {
    v3::Op<BM> A;
    v3::Op<BN> B;
    v3::ScaleDma<BM, BN> sd;
    v3::setup_rows(A, p.w_codes + e * p.H * p.I, m0, p.H, p.I);
    v3::setup_rows_sm(B, p.inter_codes, sbase + n0, sbase + p.B, P, p.Ip);
    v3::setup_scales(sd, p.w_scales + e * p.H * (p.Ip / 32), m0, p.H, p.H * (p.Ip / 32), p.inter_scales, sbase + n0, P,
                     P * (p.Ip / 32));
    v3::mainloop<BM, BN, v3::kFp8, kE4M3, kE4M3, v3::KMapPlain, RAG>(A, B, &sd, int(p.Ip / v3::SK), v3::KMapPlain{},
                                                                   smem, acc, uint32_t(p.I));
  }
  __syncthreads();   // the ring is done
  const int lane = threadIdx.x & 63, h = lane >> 5, r = lane & 31, wave = threadIdx.x >> 6, wm = wave >> 1, wn = wave & 1;
  float* scales = reinterpret_cast<float*>(smem + L::SCALES);
  v2::static_for<FN>([&](auto FJ) {
    const int slot = wn * (BN / 2) + 32 * int(FJ) + r;
    uint8_t* dst = smem + slot * L::PITCH + (wm * (BM / 2) + 4 * h) * 2;
    v2::static_for<FM / 2>([&](auto RUN) {
      // 64 values of the slot: fragments 2 RUN and 2 RUN + 1, half of each in this lane
      uint32_t m = 0;
      v2::static_for<2>([&](auto F) {
        v2::static_for<16>([&](auto Q) { m = max(m, abs_bits(acc[2 * int(RUN) + int(F)][FJ][int(Q)])); });
      });
#if defined(__HIP_DEVICE_COMPILE__)
      {
        const auto x = __builtin_amdgcn_permlane32_swap(m, m, false, false);
        m = max(uint32_t(x[0]), uint32_t(x[1]));
      }
#endif
      float mul, scale;
      f16_row_scale(m, mul, scale);
      if (h == 0) scales[slot * NS + wm * (NS / 2) + int(RUN)] = scale;
      v2::static_for<2>([&](auto F) {
        constexpr int fi = 2 * int(RUN) + int(F);
        v2::static_for<4>([&](auto K) {
          constexpr int q = 4 * int(K);
          const v16f& c = acc[fi][FJ];
          *reinterpret_cast<uint2*>(dst + (32 * fi + 8 * int(K)) * 2) =
              make_uint2(f16x2_pack(c[q] * mul, c[q + 1] * mul), f16x2_pack(c[q + 2] * mul, c[q + 3] * mul));
        });
      });
    });
  });
  __syncthreads();
  // 16-byte runs of whole rows; slots past the extent store too (their rows are not read)
  constexpr int RUNS = BM / 8;
  static_assert(BN * RUNS % v2::kThreads == 0, "whole passes");
  {
    const int c = threadIdx.x % RUNS, s0 = threadIdx.x / RUNS;
    if (m0 + 8 * c < p.H) {   // H % 32 == 0
      uint16_t* dst = p.rows + (sbase + n0 + s0) * p.H + m0 + 8 * c;
      const uint8_t* src = smem + s0 * L::PITCH + 16 * c;
      constexpr int STEP = v2::kThreads / RUNS;
#pragma unroll 8
      for (int k = 0; k < BN / STEP; ++k)
        store_nt(dst + int64_t(k) * STEP * p.H, *reinterpret_cast<const uint4*>(src + k * STEP * L::PITCH));
    }
  }
  const int64_t hs = (p.H + 63) / 64;
  for (int k = threadIdx.x; k < BN * NS; k += v2::kThreads) {
    const int slot = k / NS;
    const int64_t c = m0 / 64 + k % NS;
    if (c < hs) p.row_scale[(sbase + n0 + slot) * hs + c] = scales[k];
  }
}

struct Shape {
  int m, n;
};
// 256 x 256 with one workgroup a CU where the work is several rounds of such tiles, else 128 x 128, two a CU.  The whole
// forward at 128 -> 256 in us, by routed slots (of 4 to 16 experts; *: 64) and H; left of | the rule takes 128:
//   8192, 2048   I = 1024 119 -> 129, 1408 127 -> 138, 2112 181 -> 190, 2816 199 -> 209 |
//   32768, 1024  1024 195 -> 204, 2048 326 -> 332, 2816 411 -> 416 | 3968 561 -> 545
//   32768, 2048  1024 300 -> 313, 1408 369 -> 375, 1664 421 -> 420 | 2048 508 -> 497, 2816 677 -> 647
//   32768, 4096  512 352 -> 368, 704 435 -> 454 | 1024 527 -> 541, 1408 656 -> 649, 2048 921 -> 905
//   65536, 1024  1024 351 -> 360, 1408 453 -> 458 | 2048 633 -> 609
//   65536, 2048  512 380 -> 383, 704 469 -> 478 | 1024 581 -> 587, 1408 759 -> 732, 2048 1050 -> 973
//   65536*, 2048 512 434 -> 434, 704 553 -> 529 | 1024 691 -> 655, 2048 1233 -> 1169
//   131072, 2048 512 712 -> 713, 704 922 -> 899 | 1024 1162 -> 1117, 2048 2077 -> 1941
Shape down_shape(const MoeFwdDownArgs& p) {
  if (p.I >= 1024 && p.N * p.B * p.H * p.I >= int64_t(1) << 37 && p.B >= 256 && p.H >= 256) return {256, 256};
  return {128, 128};
}

template <int BM, int BN>
hipError_t go(MoeFwdDownArgs p, hipStream_t st) {
  p.tiles_m = int((p.H + BM - 1) / BM);
  const int64_t blocks = (p.N * (p.B / BN) * p.tiles_m + 7) & ~int64_t(7);
  if (blocks > kMaxGrid256) return hipErrorInvalidValue;
  if (p.I % 128) fwd_down_kernel<BM, BN, true><<<unsigned(blocks), v2::kThreads, 0, st>>>(p);
  else fwd_down_kernel<BM, BN, false><<<unsigned(blocks), v2::kThreads, 0, st>>>(p);
  return hipGetLastError();
}
}  // namespace

// fp16 rows up to where their bytes no longer matter enough to give up bits for them.  The whole forward with fp32
// rows -> fp16, 32768 routed slots: H = 4096: I = 1024 621 -> 545 us, 2048 986 -> 910, 4096 1762 -> 1651, 8192 3044 -> 3019;
// H = 2048: 350 -> 316, 532 -> 500, 942 -> 908, 1770 -> 1761; 262144 slots of H = 1536, I = 256 1099 -> 775; T = 256,
// H = 128, I = 256 21.5 -> 19.3.  (A ragged contraction takes them at any length: Phase 3's kernel reads whole pairs.)
bool fwd_down_fits(int64_t I) { return I < 4096 || I % 128 != 0; }

TileRangeJob fwd_down_ranges(const MoeFwdDownArgs& p) {
  if (p.Ip <= 256) return fwd_down_short_ranges(p);
  const Shape t = down_shape(p);
  return {t.n, int((p.H + t.m - 1) / t.m), int(p.B), p.tile_start, nullptr, 0, 0, p.rr_tiles};
}

hipError_t launch_fwd_down(const MoeFwdDownArgs& p, hipStream_t st) {
  if (p.Ip <= 256) return launch_fwd_down_short(p, st);
  return down_shape(p).m == 256 ? go<256, 256>(p, st) : go<128, 128>(p, st);
}

}  // namespace mx
