// moe_phase3.hpp -- one tile of Phase 3, shared by the kernels of
// moe_phase3.hip and the small MoE layers' joint launch (moe_grads.hip).
#pragma once
#include "gemm_v2.hpp"
#include "gemm_v3.hpp"
#include "kernels.hpp"
#include "moe_tiles.hpp"
#include "mx_device.hpp"

namespace mx {

using v2::v16f;

// ---------------------------------------------------------------------------
// Phase 3 tiles: block b, rows = slots m0.., columns = hidden index n0..
// Live tiles only (moe_tiles.hpp): block b's slot tiles up to its extent, times
// the H tiles.  b < 0: no tile.
struct P3Pos {
  int b;
  int64_t m0, n0;
};
template <int BM, int BN>
__device__ __forceinline__ P3Pos p3_pos(const Phase3Args& p, int wg) {
  BlockTiles bt;
  if (!block_tile(p.tile_start, p.flag, BM, int(p.N), wg, p.rr_tiles, bt)) return P3Pos{-1, 0, 0};
  int tm, tn;
  v2::grouped_tile<8>(bt.local, bt.slots, p.tiles_n, tm, tn);
  return P3Pos{bt.b, int64_t(tm) * BM, int64_t(tn) * BN};
}

// ---------------------------------------------------------------------------
// The last round of tiles, cut along K (moe_tiles.hpp, TailCut; the cut of each
// XCD is computed with the tile ranges).  A cut tile's own workgroup runs its
// first part and stores its rows to dx_slot as usual; extra workgroups after
// the main grid (ids x mod 8 again: the same XCD, after its last round has
// started) run the other parts and store their fp32 tiles to the parts
// buffer; p3_fixup_kernel then adds those into dx_slot in part order, so the
// result stays the same from run to run.
constexpr int kP3MaxExtra = 256;   // extra workgroups (and part tiles) at most

__device__ __forceinline__ const TailCut* p3_cuts(const Phase3Args& p) {
  return reinterpret_cast<const TailCut*>(p.parts);
}
__device__ __forceinline__ float* p3_part_tiles(const Phase3Args& p) {
  return reinterpret_cast<float*>(p.parts + 256);
}

// What workgroup wg runs: a whole tile, the first part of a cut tile (its own
// id), or another part (ids from grid_main on), and where that part goes.
struct P3Work {
  P3Pos tp;        // tp.b < 0: nothing
  int pair0, npairs;
  int part_slot;   // >= 0: the fp32 tile goes to part tile part_slot
};
template <int BM, int BN>
__device__ __forceinline__ P3Work p3_work(const Phase3Args& p, int wg) {
  P3Work w{P3Pos{-1, 0, 0}, 0, p.npairs, -1};
  const bool extra = wg >= p.grid_main;
  if (p.conc <= 0) {
    if (!extra) w.tp = p3_pos<BM, BN>(p, wg);
    return w;
  }
  const int e = extra ? wg - p.grid_main : wg;
  const int x = e % 8, q = e / 8;
  const TailCut c = p3_cuts(p)[x];
  int main_wg = wg, part = 0;
  bool cut;
  if (extra) {
    if (q >= c.tail * (c.S - 1)) return w;   // also every extra id when nothing is cut
    const int i = q / (c.S - 1);
    part = 1 + q % (c.S - 1);
    main_wg = 8 * (c.nx - c.tail + i) + x;
    w.part_slot = c.base + q;
    cut = true;
  } else {
    cut = q >= c.nx - c.tail && q < c.nx;   // tail == 0: never
  }
  w.tp = p3_pos<BM, BN>(p, main_wg);
  if (cut) {
    w.pair0 = part * p.npairs / c.S;
    w.npairs = (part + 1) * p.npairs / c.S - w.pair0;
  }
  return w;
}

// stage s of a part that starts at stage s0
struct P3KMap {
  int s0;
  __device__ __forceinline__ uint32_t operator()(int s) const { return uint32_t(s + s0) * v3::SK; }
};

// A part's fp32 tile, row-major BM x BN (lanes of a fragment row write 128
// consecutive bytes).
template <int BM, int BN>
__device__ __forceinline__ void p3_store_part(float* dst, const v16f (&acc)[BM / 64][BN / 64]) {
  v2::static_for<BM / 64>([&](auto FI) {
    v2::static_for<16>([&](auto Q) {
      float* row = dst + v2::acc_row<BM, BN>(FI, Q) * BN;
      v2::static_for<BN / 64>([&](auto FJ) { row[v2::acc_col<BM, BN>(FJ)] = acc[FI][FJ][int(Q)]; });
    });
  });
}

// dX rows of one tile.  Every slot of the tile stores its row: a padding
// slot's dGU row is zeros, so its row is zeros too, and the finalisation
// reads only routed slots' rows.  (Storing only routed rows made every store
// wait for a load of the slot's token.)  Tiles lie inside one block (BM <= B).
template <int BM, int BN>
__device__ __forceinline__ void p3_store(const Phase3Args& p, const P3Pos& tp, const v16f (&acc)[BM / 64][BN / 64]) {
  const int64_t sbase = int64_t(tp.b) * p.B;
  v2::static_for<BM / 64>([&](auto FI) {
    v2::static_for<16>([&](auto Q) {
      const int64_t s = tp.m0 + v2::acc_row<BM, BN>(FI, Q);
      float* dst = p.dx_slot + (sbase + s) * p.H;
      v2::static_for<BN / 64>([&](auto FJ) {
        const int64_t hh = tp.n0 + v2::acc_col<BM, BN>(FJ);
        if (hh < p.H) dst[hh] = acc[FI][FJ][int(Q)];
      });
    });
  });
}

// The same rows through LDS (the ring's, free after the main loop), in passes
// of R rows padded by 16 bytes: every thread then stores 16-byte runs, so each
// store instruction writes whole row segments (BN * 4 bytes) instead of
// 128-byte pieces of 2 rows.  Nontemporal stores: the rows ([P, H] fp32, the
// largest output) are read once, by the finalisation, after the other phases;
// measured 24% faster on the fine workload (H = 1536, 2I = 512), 10% with
// 2I = 2816, 1% with 2I = 28672.
template <int BM, int BN, int SMEM>
__device__ __forceinline__ void p3_store_staged(const Phase3Args& p, const P3Pos& tp,
                                                const v16f (&acc)[BM / 64][BN / 64], uint8_t* smem) {
  constexpr int RB = BN * 4 + 16;                       // bytes per staged row
  constexpr int R = (SMEM / RB) >= BM ? BM : BM / 2;    // rows per pass
  static_assert(R * RB <= SMEM && BM % R == 0 && (BM / 2) % 32 == 0, "staging passes");
  const int64_t sbase = int64_t(tp.b) * p.B;
  const int wave = threadIdx.x >> 6;
  constexpr int CPR = BN * 4 / 16;                      // 16-byte runs per row
  v2::static_for<BM / R>([&](auto PASS) {
    __syncthreads();                                    // the ring, or the previous pass, is done
    // pass PASS holds tile rows [PASS * R, PASS * R + R): R == BM, or the waves
    // whose half of the rows (wave >> 1) is PASS
    if (R == BM || (wave >> 1) == int(PASS)) {
      v2::static_for<BM / 64>([&](auto FI) {
        v2::static_for<16>([&](auto Q) {
          const int r = v2::acc_row<BM, BN>(FI, Q) - int(PASS) * R;
          v2::static_for<BN / 64>([&](auto FJ) {
            *reinterpret_cast<float*>(smem + r * RB + v2::acc_col<BM, BN>(FJ) * 4) = acc[FI][FJ][int(Q)];
          });
        });
      });
    }
    __syncthreads();
    // a thread keeps one 16-byte column run and walks the rows RPP apart
    constexpr int RPP = v2::kThreads / CPR;   // rows per pass
    static_assert(v2::kThreads % CPR == 0 && R % RPP == 0, "passes of whole rows");
    const int ch = threadIdx.x % CPR, r0 = threadIdx.x / CPR;
    const int64_t hh = tp.n0 + ch * 4;
    if (hh < p.H) {
      float* dst = p.dx_slot + (sbase + tp.m0 + int(PASS) * R + r0) * p.H + hh;
      const uint8_t* src = smem + r0 * RB + ch * 16;
#pragma unroll 8
      for (int q = 0; q < R / RPP; ++q)
        store_nt(dst + int64_t(q) * RPP * p.H, *reinterpret_cast<const uint4*>(src + q * (RPP * RB)));
    }
  });
}

// One aligned tile, on the four-slot ring loop (its deeper look-ahead measured
// 4% faster here than the pair-slot ring).
template <int BM, int BN, int FG, int FW>
__device__ __forceinline__ void phase3_tile(const Phase3Args& p, int wg, uint8_t* smem) {
  constexpr int FM = BM / 64, FN = BN / 64;
  const P3Work w = p3_work<BM, BN>(p, wg);
  const P3Pos& tp = w.tp;
  if (tp.b < 0) return;
  const int64_t e = p.b2e[tp.b];
  const int64_t sbase = int64_t(tp.b) * p.B, twoI = 2 * p.I;
  v3::Op<BM> A;
  v3::Op<BN> B;
  v3::ScaleDma<BM, BN> sd;
  const int64_t P = p.N * p.B;
  // dGU stage-major over all P slots (the tile's rows stop at its block's end);
  // W_gate_up row-major, as the caller holds it
  v3::setup_rows_sm(A, p.dgu_row_codes, sbase + tp.m0, sbase + p.B, P, twoI);
  v3::setup_rows(B, p.wgu_codes + e * p.H * twoI, tp.n0, p.H, twoI);
  // pair-major scales: dGU along I over all P slots; W_gate_up re-laid per expert
  v3::setup_scales(sd, p.dgu_row_scales, sbase + tp.m0, P, P * (twoI / 32), p.wgu_scales + e * p.H * (twoI / 32),
                   tp.n0, p.H, p.H * (twoI / 32));
  v16f acc[FM][FN];
  v3::mainloop<BM, BN, v3::kFp8, FG, FW>(A, B, &sd, 2 * w.npairs, P3KMap{2 * w.pair0}, smem, acc);
  if (w.part_slot >= 0)
    p3_store_part<BM, BN>(p3_part_tiles(p) + int64_t(w.part_slot) * (BM * BN), acc);
  else
    p3_store_staged<BM, BN, v3::smem_bytes(BM, BN)>(p, tp, acc, smem);
}

}  // namespace mx
