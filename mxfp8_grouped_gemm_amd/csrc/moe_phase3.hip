// moe_phase3.hip -- Phase 3 of the MoE backward (P1, "Blockwise MM Backward
// MXFP8 Kernel API Reference": Phase 3; P3, sonic-moe functional/backward.py:
// _up_projection_backward_act, the input-gradient product).
//
// Per block b (tile rows = slot p, columns = hidden index h, contraction over 2I):
//   dX_slot[p][h] = sum_{j,i} deq(dGU)[p][j][i] * deq(W_gate_up[e])[h][j][i]
//   stored per slot in fp32; the finalisation sums each token's slots (they
//   sit in different blocks) in expert order, so dX is deterministic.
#include "moe_phase3.hpp"

namespace mx {

using v2::KMapPlain;

// dx_slot += the other parts of each cut tile, in part order.  One workgroup
// per 16 rows of a cut tile: ids x + 8 (i * BM / 16 + slab) for tile i of XCD
// x; a thread takes one 4-column group of 4 rows, all of its loads issued
// before the sums.
template <int BM, int BN>
__global__ void __launch_bounds__(256) p3_fixup_kernel(Phase3Args p) {
  constexpr int NSL = BM / 16, CG = BN / 4;   // slabs per tile, 4-column groups per row
  static_assert(CG * 4 == 256, "a thread per 4-column group and row of 4");
  const int x = blockIdx.x % 8, rest = blockIdx.x / 8, i = rest / NSL, slab = rest % NSL;
  const TailCut c = p3_cuts(p)[x];
  if (i >= c.tail) return;
  const P3Pos tp = p3_pos<BM, BN>(p, 8 * (c.nx - c.tail + i) + x);
  if (tp.b < 0) return;
  const int col = (threadIdx.x % CG) * 4, r0 = slab * 16 + threadIdx.x / CG;
  if (tp.n0 + col >= p.H) return;   // H % 32 == 0: a group is all inside or all outside
  const float* part = p3_part_tiles(p) + int64_t(c.base + i * (c.S - 1)) * (BM * BN);
  float* out = p.dx_slot + (int64_t(tp.b) * p.B + tp.m0) * p.H + tp.n0 + col;
  float4 v[4], q[kCutMaxParts - 1][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = r0 + 4 * j;
    v[j] = *reinterpret_cast<const float4*>(out + int64_t(r) * p.H);
#pragma unroll
    for (int k = 0; k < kCutMaxParts - 1; ++k)
      q[k][j] = k < c.S - 1 ? *reinterpret_cast<const float4*>(part + int64_t(k) * (BM * BN) + r * BN + col)
                            : make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
#pragma unroll
    for (int k = 0; k < kCutMaxParts - 1; ++k) {
      if (k < c.S - 1) {
        v[j].x += q[k][j].x;
        v[j].y += q[k][j].y;
        v[j].z += q[k][j].z;
        v[j].w += q[k][j].w;
      }
    }
    *reinterpret_cast<float4*>(out + int64_t(r0 + 4 * j) * p.H) = v[j];
  }
}

// 2I not a multiple of 128 bytes: one tile per workgroup on the v2 loop.
template <int BM, int BN, int FG, int FW>
__global__ void __launch_bounds__(v2::kThreads) phase3_generic(Phase3Args p) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[2 * (BM + BN) * v2::BK];
  constexpr int FM = BM / 64, FN = BN / 64;
  const P3Pos tp = p3_pos<BM, BN>(p, blockIdx.x);
  if (tp.b < 0) return;
  const int64_t e = p.b2e[tp.b];
  const int wave = threadIdx.x >> 6;
  const int64_t sbase = int64_t(tp.b) * p.B, twoI = 2 * p.I;
  v2::Operand<BM, FM> A;
  v2::Operand<BN, FN> B;
  v2::setup_rows(A, p.dgu_row_codes + sbase * twoI, p.dgu_row_scales + sbase * (twoI / 32), tp.m0, p.B, twoI,
                 twoI / 32, (wave >> 1) * (BM / 2));
  v2::setup_rows(B, p.wgu_codes + e * p.H * twoI, p.wgu_scales + e * p.H * (twoI / 32), tp.n0, p.H, twoI,
                 twoI / 32, (wave & 1) * (BN / 2));
  v16f acc[FM][FN];
  v2::mainloop<BM, BN, v2::kFp8, FG, FW, true>(A, B, int((twoI + v2::BK - 1) / v2::BK), KMapPlain{twoI}, smem,
                                                acc);
  p3_store<BM, BN>(p, tp, acc);
}

// Aligned: one tile per workgroup.
template <int BM, int BN, int FG, int FW>
__global__ void __launch_bounds__(v2::kThreads) phase3_ring(Phase3Args p) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[v3::smem_bytes(BM, BN)];
  phase3_tile<BM, BN, FG, FW>(p, blockIdx.x, smem);
}

// Completes p for tiles of BM x BN.
static hipError_t plan(Phase3Args& p, int BM, int BN, TileRangeJob& job) {
  p.tiles_m = int((p.B + BM - 1) / BM);
  p.tiles_n = int((p.H + BN - 1) / BN);
  const int64_t total = (int64_t(p.tiles_m) * p.tiles_n * p.N + 7) & ~int64_t(7);   // every tile, rounded to 8
  if (total + kP3MaxExtra > INT32_MAX) return hipErrorInvalidValue;
  p.grid_main = int(total);
  p.npairs = int(2 * p.I / 128);
  job = phase3_ranges(p);
  p.conc = job.conc;
  return hipSuccess;
}

template <int BM, int BN>
static hipError_t phase3_launch(Phase3Args p, int fg, int fw, bool generic, hipStream_t st) {
  // the ring's LDS keeps these tiles at one workgroup per CU, so the CU count
  // is the number resident at once (TailCut)
  static_assert(2 * v3::smem_bytes(BM, BN) > 160 * 1024, "one workgroup per CU");
  TileRangeJob job;
  hipError_t e = plan(p, BM, BN, job);
  if (e != hipSuccess) return e;
  if (!p.ranges_done) {
    e = launch_tile_ranges(p.flag, p.N, job, st);
    if (e != hipSuccess) return e;
  }
  if (generic) {
    const unsigned grid = unsigned(p.grid_main);
    if (fg == 0 && fw == 0) phase3_generic<BM, BN, 0, 0><<<grid, v2::kThreads, 0, st>>>(p);
    else if (fg == 0) phase3_generic<BM, BN, 0, 1><<<grid, v2::kThreads, 0, st>>>(p);
    else if (fw == 0) phase3_generic<BM, BN, 1, 0><<<grid, v2::kThreads, 0, st>>>(p);
    else phase3_generic<BM, BN, 1, 1><<<grid, v2::kThreads, 0, st>>>(p);
  } else {
    const unsigned grid = unsigned(p.grid_main + p.conc);   // p.conc extra workgroups for the cut parts
    if (fg == 0 && fw == 0) phase3_ring<BM, BN, 0, 0><<<grid, v2::kThreads, 0, st>>>(p);
    else if (fg == 0) phase3_ring<BM, BN, 0, 1><<<grid, v2::kThreads, 0, st>>>(p);
    else if (fw == 0) phase3_ring<BM, BN, 1, 0><<<grid, v2::kThreads, 0, st>>>(p);
    else phase3_ring<BM, BN, 1, 1><<<grid, v2::kThreads, 0, st>>>(p);
    if (p.conc) p3_fixup_kernel<BM, BN><<<unsigned(p.conc * (BM / 16)), 256, 0, st>>>(p);
  }
  return hipGetLastError();
}

// Tile shape: 256 x 256 when the block and H allow, else 128 x 256; 2I not a
// multiple of 128 bytes (unaligned scale rows / ragged last K stage): the v2
// loop at 128 x 256.  A short contraction (2I < 1024: a few ring stages per
// tile) also takes 128 x 256 tiles: with the rows stored through LDS, they
// measured 5% faster at 2I = 512 than 128 x 128 tiles at two per CU.
static bool phase3_wide(const Phase3Args& p) {
  return (2 * p.I) % v2::BK == 0 && 2 * p.I >= 1024 && p.B >= 256 && p.H >= 256;
}
TileRangeJob phase3_ranges(const Phase3Args& p) {
  const int bm = phase3_wide(p) ? 256 : 128, bn = 256, npairs = int(2 * p.I / 128);
  // the cut needs the ring, the parts buffer, whole XCDs of CUs (at most
  // kP3MaxExtra: the extra workgroups and part tiles) and at least two parts'
  // worth of stage pairs
  const bool cut = p.parts && phase3_parts_bytes(p) > 0 && p.conc >= 8 && p.conc % 8 == 0 && p.conc <= kP3MaxExtra;
  return {bm, int((p.H + bn - 1) / bn), int(p.B), p.tile_start, cut ? reinterpret_cast<TailCut*>(p.parts) : nullptr,
          cut ? p.conc : 0, npairs, p.rr_tiles};
}
hipError_t launch_phase3(const Phase3Args& p, int fg, int fw, hipStream_t st) {
  if (phase3_wide(p)) return phase3_launch<256, 256>(p, fg, fw, false, st);
  return phase3_launch<128, 256>(p, fg, fw, (2 * p.I) % v2::BK != 0, st);
}

bool phase3_small(Phase3Args& p, unsigned& grid) {
  TileRangeJob job;
  if (phase3_wide(p) || (2 * p.I) % v2::BK != 0 || !p.ranges_done || plan(p, 128, 256, job) != hipSuccess) return false;
  grid = unsigned(p.grid_main);
  return p.conc == 0;   // no tile cut along K
}

int64_t phase3_max_tiles(const Phase3Args& p) {
  const int64_t bm = phase3_wide(p) ? 256 : 128, bn = 256;
  return p.N * ((p.B + bm - 1) / bm) * ((p.H + bn - 1) / bn);
}

// The parts buffer: the 8 XCDs' cuts (256 bytes), then the later parts' tiles:
// fewer than the extra workgroups, and at most kCutMaxParts - 1 per tile.
// Empty where nothing can be cut (the v2 loop, or too few stage pairs).
int64_t phase3_parts_bytes(const Phase3Args& p) {
  if ((2 * p.I) % v2::BK != 0 || 2 * p.I / 128 < 2 * kCutMinPairs) return 0;
  const int64_t bm = phase3_wide(p) ? 256 : 128, bn = 256;
  int64_t tiles = (kCutMaxParts - 1) * phase3_max_tiles(p);
  tiles = tiles < kP3MaxExtra ? tiles : kP3MaxExtra;
  return 256 + tiles * bm * bn * 4;
}

}  // namespace mx
