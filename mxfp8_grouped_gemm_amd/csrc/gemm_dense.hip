// gemm_dense.hip -- MXFP8 NT GEMM with a bf16 store, for
//   * the dense backward (P2, "Matmul MXFP8 Backward Kernel API Reference"):
//       dX [M,K] = dY [M,N] . W^T [K,N]^T      (contraction over N)
//       dW [N,K] = dY^T [N,M] . X^T [K,M]^T    (contraction over M)
//   * the MoE weight gradients (P1 Phases 2 and 4), one group per expert,
//     whose contraction runs over the expert's blocks of token slots:
//       dW_gate_up[e] [H,2I] = X_tok [H,P] . dGU_tok [2I,P]^T
//       dW_down[e]    [I,H]  = inter_tok [I,P] . gy_tok [H,P]^T
//     where the K columns of expert e are the slots of the blocks
//     list[off[e] .. off[e+1]) (B slots each).
#include <type_traits>
#include <utility>

#include "gemm_store.hpp"

namespace mx {

// K column of stage s.  Grouped: the block list is read through the constant
// address space (a scalar load: the main loop only waits on vector loads for
// its DMA), and block sizes are powers of two >= 128 (shift = log2(blk/128)).
typedef const __attribute__((address_space(4))) int32_t* const_i32_ptr;
struct KMapGrouped {
  const int32_t* list;   // null: plain K range [0, K)
  int b0, blk, shift;
  int64_t K;
  __device__ __forceinline__ void operator()(int s, uint32_t& kc, int& kv) const {
    if (list) {
      const int blkid = ((const_i32_ptr)(uintptr_t)list)[b0 + (s >> shift)];
      kc = uint32_t(blkid) * uint32_t(blk) + uint32_t(s & ((1 << shift) - 1)) * v2::BK;
      kv = v2::BK;
    } else {
      const int64_t q = int64_t(s) * v2::BK;
      kc = uint32_t(q);
      const int64_t rem = K - q;
      kv = rem < v2::BK ? int(rem) : v2::BK;
    }
  }
};

// Unaligned shapes (ragged K or scale rows not 4-byte aligned): one tile per
// workgroup on the two-stage loop.
template <int BM, int BN, int FA, int FB>
__global__ void __launch_bounds__(v2::kThreads) gemm_store_generic(GemmStoreArgs p) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[2 * (BM + BN) * v2::BK];
  constexpr int FM = BM / 64, FN = BN / 64;
  const TilePos tp = tile_pos<BM, BN>(p, blockIdx.x, p.groups);
  if (tp.g < 0) return;
  const int wave = threadIdx.x >> 6;
  v2::Operand<BM, FM> A;
  v2::Operand<BN, FN> B;
  v2::setup_rows(A, p.a_codes, p.a_scales, tp.m0, p.M, p.lda, p.lda / 32, (wave >> 1) * (BM / 2));
  v2::setup_rows(B, p.b_codes, p.b_scales, tp.n0, p.N, p.ldb, p.ldb / 32, (wave & 1) * (BN / 2));
  KMapGrouped km{p.blk_list, 0, p.blk, 31 - __builtin_clz(unsigned(p.blk / v2::BK) | 1u), p.K};
  int nstages;
  if (p.blk_list) {
    km.b0 = p.blk_off[tp.g];
    nstages = int((int64_t(p.blk_off[tp.g + 1] - km.b0) * p.blk) / v2::BK);
  } else {
    nstages = int((p.K + v2::BK - 1) / v2::BK);
  }
  v2::v16f acc[FM][FN];
  v2::mainloop<BM, BN, v2::kFp8, FA, FB, true>(A, B, nstages, km, smem, acc);
  store_tile<BM, BN>(p, tp.g, tp.m0, tp.n0, acc);
}

// Aligned shapes: one tile per workgroup on a ring loop.
template <int BM, int BN, int FA, int FB, bool LIST, bool PAIR>
__global__ void __launch_bounds__(v2::kThreads) gemm_store_ring(GemmStoreArgs p) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[gemm_store_smem<BM, BN, PAIR>()];
  gemm_store_tile<BM, BN, FA, FB, LIST, PAIR>(p, blockIdx.x, smem);
}

template <int BM, int BN>
static void launch_generic(const GemmStoreArgs& p, int fa, int fb, unsigned grid, hipStream_t st) {
  if (fa == 0 && fb == 0) gemm_store_generic<BM, BN, 0, 0><<<grid, v2::kThreads, 0, st>>>(p);
  else if (fa == 0) gemm_store_generic<BM, BN, 0, 1><<<grid, v2::kThreads, 0, st>>>(p);
  else if (fb == 0) gemm_store_generic<BM, BN, 1, 0><<<grid, v2::kThreads, 0, st>>>(p);
  else gemm_store_generic<BM, BN, 1, 1><<<grid, v2::kThreads, 0, st>>>(p);
}

template <int BM, int BN, bool LIST, bool PAIR>
static void launch_ring(const GemmStoreArgs& p, int fa, int fb, unsigned grid, hipStream_t st) {
  if (fa == 0 && fb == 0) gemm_store_ring<BM, BN, 0, 0, LIST, PAIR><<<grid, v2::kThreads, 0, st>>>(p);
  else if (fa == 0) gemm_store_ring<BM, BN, 0, 1, LIST, PAIR><<<grid, v2::kThreads, 0, st>>>(p);
  else if (fb == 0) gemm_store_ring<BM, BN, 1, 0, LIST, PAIR><<<grid, v2::kThreads, 0, st>>>(p);
  else gemm_store_ring<BM, BN, 1, 1, LIST, PAIR><<<grid, v2::kThreads, 0, st>>>(p);
}

struct GemmStorePlan {
  bool generic, big;
  unsigned grid;
};
// Completes p for a launch: the operands swapped (C^T = B . A^T, so that the store is
// along the output's rows, see store_tile), the tile shape and counts.
static hipError_t plan(GemmStoreArgs& p, int groups, int& fa, int& fb, GemmStorePlan& q) {
  std::swap(p.a_codes, p.b_codes);
  std::swap(p.a_scales, p.b_scales);
  std::swap(p.lda, p.ldb);
  std::swap(p.M, p.N);
  std::swap(fa, fb);
  // every stage full and scale rows 4-byte aligned -> the ring; otherwise the v2 loop
  q.generic = (p.lda % v2::BK) || (p.ldb % v2::BK) || (!p.blk_list && (p.K % v2::BK)) ||
                (p.blk_list && (p.blk % v2::BK));
  // stage-major operands: only the four-slot ring reads them
  if (p.stage_major && (q.generic || p.pair)) return hipErrorInvalidValue;
  // larger tiles once there are enough of them to fill the chip
  q.big = !q.generic && p.M >= 256 && p.N >= 256 &&
          ((p.M + 255) / 256) * ((p.N + 255) / 256) * int64_t(groups) >= 200;
  const int W = q.big ? 256 : 128;
  p.tiles_m = int((p.M + W - 1) / W);
  p.tiles_n = int((p.N + W - 1) / W);
  const int64_t per_group = int64_t(p.tiles_m) * p.tiles_n;
  const int64_t total = per_group * groups;
  if (total > INT32_MAX) return hipErrorInvalidValue;
  p.total = int(total);
  p.groups = groups;
  // rotating eighths (tile_pos): room for ceil(G / 8) * P workgroups per XCD
  const int64_t launched = (per_group % 8 && groups > 1) ? 8 * ((groups + 7) / 8) * per_group : total;
  if (launched > INT32_MAX) return hipErrorInvalidValue;
  q.grid = unsigned(launched);
  return hipSuccess;
}

bool gemm_store_small(GemmStoreArgs& p, int groups, unsigned& grid) {
  int fa = 0, fb = 0;
  GemmStorePlan q;
  if (p.M <= 0 || p.N <= 0 || groups <= 0 || plan(p, groups, fa, fb, q) != hipSuccess) return false;
  grid = q.grid;
  return !q.generic && !q.big && !p.pair && p.blk_list;
}

hipError_t launch_gemm_store(GemmStoreArgs p, int groups, int fa, int fb, hipStream_t st) {
  if (p.M <= 0 || p.N <= 0 || groups <= 0) return hipSuccess;
  GemmStorePlan q;
  const hipError_t err = plan(p, groups, fa, fb, q);
  if (err != hipSuccess) return err;
  const unsigned grid = q.grid;
  if (q.generic) {
    launch_generic<128, 128>(p, fa, fb, grid, st);
    return hipGetLastError();
  }
  if (q.big) {
    if (p.blk_list) {
      if (p.pair) launch_ring<256, 256, true, true>(p, fa, fb, grid, st);
      else launch_ring<256, 256, true, false>(p, fa, fb, grid, st);
    } else {
      if (p.pair) launch_ring<256, 256, false, true>(p, fa, fb, grid, st);
      else launch_ring<256, 256, false, false>(p, fa, fb, grid, st);
    }
  } else {
    if (p.blk_list) launch_ring<128, 128, true, false>(p, fa, fb, grid, st);
    else launch_ring<128, 128, false, false>(p, fa, fb, grid, st);
  }
  return hipGetLastError();
}

}  // namespace mx
