// moe_fwd_down_short.hip -- the MoE forward's second product for I <= 256
// (moe_fwd_down.hip's, its rows and scales): P x H results of a contraction
// that one tile's operands hold whole, so the results' bytes are the work
// (262 144 routed slots, H = 1536: 805 MB of rows, 206 GFLOP).
//
// A workgroup keeps its 128 slots' codes in registers and goes through H 128
// rows at a time: the next rows' codes come to LDS while this tile's products
// run, and its results leave while the next tile's run.  One wait a tile, on
// loads that were issued before the products, and none on the stores of the
// tile at hand; two workgroups a CU.  That case takes 265 us, 340 with a
// workgroup a tile, whose loads, products and stores follow each other.
// Few slots: H is split over workgroups, so that each CU has some.
#include "gemm_v3.hpp"
#include "kernels.hpp"
#include "moe_tiles.hpp"
#include "mx_device.hpp"

namespace mx {

namespace {
using v2::v16f;
constexpr int kSide = 128;                       // slots, and h a tile
constexpr int kStage = kSide * 64;               // LDS bytes of 64 columns of a tile's weight rows
constexpr int kPitch = 64 * 2 + 16;              // of a slot's 64 staged results
constexpr int kWaveStage = 64 * kPitch;          // a wave's 64 slots

// KS: stages of 64 columns (Ip / 64)
template <int KS>
__global__ void __launch_bounds__(v2::kThreads, 2) fwd_down_short_kernel(MoeFwdDownArgs p) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ __attribute__((aligned(16))) uint8_t smem[KS * kStage + 4 * 256 + 4 * kWaveStage];
  uint8_t* const swords = smem + KS * kStage;   // scale words: pair w >> 1, rows 64 (w & 1) .. by wave w
  BlockTiles bt;
  if (!block_tile(p.tile_start, p.flag, kSide, int(p.N), blockIdx.x, p.rr_tiles, bt)) return;
  int tm, tn;
  v2::grouped_tile<8>(bt.local, p.tiles_m, bt.slots, tm, tn);
  const int64_t s0 = int64_t(bt.b) * p.B + int64_t(tn) * kSide, e = p.b2e[bt.b], P = p.N * p.B;
  const int t1 = min((tm + 1) * p.tiles_wg, int((p.H + kSide - 1) / kSide));
  const int lane = threadIdx.x & 63, h = lane >> 5, r = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave >> 1, wn = wave & 1;

  // Weight rows by the DMA: instruction j of stage s fills 16 rows x 64 bytes.  Offsets from the expert's first
  // byte: rows past H lie past the descriptor, columns past I are sent there.
  const v3::v4i dA = v3::rsrc(v2::make_rsrc(p.w_codes + e * p.H * p.I, uint32_t(p.H * p.I)));
  const v3::v4i dS = v3::rsrc(v2::make_rsrc(p.w_scales + e * p.H * (p.Ip / 32), uint32_t(p.H * (p.Ip / 32))));
  uint32_t off[2];
  const uint32_t col = 16u * ((threadIdx.x & 3) ^ ((threadIdx.x >> 4) & 3));   // dma_row's rows share a swizzle
#pragma unroll
  for (int j = 0; j < 2; ++j) off[j] = uint32_t(v3::dma_row<kSide>(j) * p.I) + col;
  auto load = [&](int t) {
    const uint32_t first = uint32_t(t) * kSide * uint32_t(p.I);
    v2::static_for<KS>([&](auto S) {
      v2::static_for<2>([&](auto J) {
        v3::dma16(dA, v3::lds_addr(smem) + uint32_t(S) * kStage + uint32_t(wave * 32 + 16 * int(J)) * 64,
                  64 * uint32_t(S) + col < uint32_t(p.I) ? first + off[J] + 64 * uint32_t(S) : v3::kOOB, 0);
      });
    });
    const int64_t row = int64_t(t) * kSide + 64 * (wave & 1) + lane;
    v3::dma4(dS, v3::lds_addr(swords) + uint32_t(wave) * 256,
             row < p.H && (wave >> 1) < KS / 2 ? uint32_t(((wave >> 1) * p.H + row) * 4) : v3::kOOB, 0);
  };
  load(tm * p.tiles_wg);

  uint4 fb[KS][2][2];   // the slots' codes and scale words
  uint32_t sb[KS / 2][2];
  v2::static_for<2>([&](auto J) {
    const int64_t slot = s0 + wn * 64 + 32 * int(J) + r;
    v2::static_for<KS>([&](auto S) {
      fb[S][J][0] = *reinterpret_cast<const uint4*>(p.inter_codes + stage_major_off(slot, 64 * int(S) + 16 * h, P, p.Ip));
      fb[S][J][1] = *reinterpret_cast<const uint4*>(p.inter_codes + stage_major_off(slot, 64 * int(S) + 32 + 16 * h, P, p.Ip));
    });
    v2::static_for<KS / 2>([&](auto Q) {
      sb[Q][J] = reinterpret_cast<const uint32_t*>(p.inter_scales)[int(Q) * P + slot] >> (8 * h);
    });
  });
  uint8_t* const stage = swords + 4 * 256 + wave * kWaveStage;
  const int64_t hs = (p.H + 63) / 64;
  auto barrier = [] {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  barrier();
  for (int t = tm * p.tiles_wg; t < t1; ++t) {
    uint4 fa[KS][2][2];
    uint32_t sa[KS / 2][2];
    v2::static_for<2>([&](auto F) {
      const int row = wm * 64 + 32 * int(F) + r;
      v2::static_for<KS>([&](auto S) {
        const uint8_t* q = smem + int(S) * kStage + row * 64;
        fa[S][F][0] = *reinterpret_cast<const uint4*>(q + 16 * (h ^ v3::swz(row)));
        fa[S][F][1] = *reinterpret_cast<const uint4*>(q + 16 * ((2 + h) ^ v3::swz(row)));
      });
      v2::static_for<KS / 2>([&](auto Q) {
        sa[Q][F] = *reinterpret_cast<const uint32_t*>(swords + (2 * int(Q) + wm) * 256 + (32 * int(F) + r) * 4) >> (8 * h);
      });
    });
    barrier();   // every wave holds its rows
    if (t + 1 < t1) load(t + 1);
    v16f acc[2][2];
    v2::static_for<KS>([&](auto S) {
      v2::static_for<2>([&](auto F) {
        v2::static_for<2>([&](auto J) {
          constexpr int s = S;
          if constexpr (s == 0) acc[F][J] = v16f{};
          acc[F][J] = v3::mma<kE4M3, kE4M3, 2 * (s & 1)>(fa[S][F], fb[S][J], acc[F][J], int(sa[s / 2][F]), int(sb[s / 2][J]));
        });
      });
    });
    const int64_t m0 = int64_t(t) * kSide + wm * 64;   // the wave's 64 values of a slot
    float scale[2];
    v2::static_for<2>([&](auto J) {
      uint32_t m = 0;
      v2::static_for<2>([&](auto F) { v2::static_for<16>([&](auto Q) { m = max(m, abs_bits(acc[F][J][int(Q)])); }); });
      const auto x = __builtin_amdgcn_permlane32_swap(m, m, false, false);
      m = max(uint32_t(x[0]), uint32_t(x[1]));
      float mul;
      f16_row_scale(m, mul, scale[J]);
      uint8_t* dst = stage + (32 * int(J) + r) * kPitch + 8 * h;
      v2::static_for<2>([&](auto F) {
        v2::static_for<4>([&](auto K) {
          constexpr int q = 4 * int(K);
          const v16f& c = acc[F][J];
          *reinterpret_cast<uint2*>(dst + 64 * int(F) + 16 * int(K)) =
              make_uint2(f16x2_pack(c[q] * mul, c[q + 1] * mul), f16x2_pack(c[q + 2] * mul, c[q + 3] * mul));
        });
      });
    });
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the next rows (and the last tile's stores, a tile old)
    wave_lds_order();   // the staging is the wave's own
    const int c = lane & 7;
    if (m0 + 8 * c < p.H) {   // H % 32 == 0
      uint16_t* dst = p.rows + (s0 + wn * 64 + (lane >> 3)) * p.H + m0 + 8 * c;
      const uint8_t* src = stage + (lane >> 3) * kPitch + 16 * c;
#pragma unroll
      for (int k = 0; k < 8; ++k) store_nt(dst + 8 * k * p.H, *reinterpret_cast<const uint4*>(src + 8 * k * kPitch));
    }
    if (h == 0 && m0 < p.H) {
#pragma unroll
      for (int j = 0; j < 2; ++j) p.row_scale[(s0 + wn * 64 + 32 * j + r) * hs + m0 / 64] = scale[j];
    }
    barrier();   // every wave's share of the next rows has landed
  }
#endif
}

int tiles_h(const MoeFwdDownArgs& p) { return int((p.H + kSide - 1) / kSide); }
// h tiles a workgroup: as many as leave kWgs workgroups, if every slot were routed (H = 1536: 265 us with all 12,
// 270 with 6, 281 with 3)
int tiles_wg(const MoeFwdDownArgs& p) {
  constexpr int64_t kWgs = 2048;
  const int64_t n = p.N * (p.B / kSide) * tiles_h(p) / kWgs;
  return int(n < 1 ? 1 : n < tiles_h(p) ? n : tiles_h(p));
}
int parts(const MoeFwdDownArgs& p) { return (tiles_h(p) + tiles_wg(p) - 1) / tiles_wg(p); }
}  // namespace

TileRangeJob fwd_down_short_ranges(const MoeFwdDownArgs& p) {
  return {kSide, parts(p), int(p.B), p.tile_start, nullptr, 0, 0, p.rr_tiles};
}

hipError_t launch_fwd_down_short(MoeFwdDownArgs p, hipStream_t st) {
  p.tiles_m = parts(p);
  p.tiles_wg = tiles_wg(p);
  const int64_t blocks = (p.N * (p.B / kSide) * p.tiles_m + 7) & ~int64_t(7);
  if (blocks > kMaxGrid256 || p.Ip > 256) return hipErrorInvalidValue;
  if (p.Ip == 128) fwd_down_short_kernel<2><<<unsigned(blocks), v2::kThreads, 0, st>>>(p);
  else fwd_down_short_kernel<4><<<unsigned(blocks), v2::kThreads, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace mx
