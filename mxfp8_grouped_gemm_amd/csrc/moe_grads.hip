// moe_grads.hip -- Phases 3, 2 and 4 of a small MoE layer in one launch.
//
// The three products only depend on the epilogue, so where all their tiles run
// at once (a workgroup per CU) one launch takes as long as the longest of them:
// the first n3 workgroups run Phase 3's tiles, then Phase 2's, then Phase 4's.  The
// tiles are those of the separate kernels, to the bit.  Measured at T = 256,
// H = 128, I = 256, E = 4, top-2 (28 tiles of 2 to 8 ring stages, all latency): 8.8 us
// against 8.4 + 5.2 + 5.2 in three launches.  With more tiles than CUs the
// phases keep their own tile orders and shapes.
#include "gemm_store.hpp"
#include "moe_phase3.hpp"

namespace mx {

namespace {
constexpr int kSmem3 = v3::smem_bytes(128, 256), kSmem24 = gemm_store_smem<128, 128, false>();
}

template <int FG, int FW, int FA>
__global__ void __launch_bounds__(v2::kThreads) moe_grads_kernel(Phase3Args p3, int n3, GemmStoreArgs g2, int n2,
                                                                 GemmStoreArgs g4) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[kSmem3 > kSmem24 ? kSmem3 : kSmem24];
  const int wg = blockIdx.x;
  if (wg < n3) {
    phase3_tile<128, 256, FG, FW>(p3, wg, smem);
  } else {
    const bool two = wg < n3 + n2;
    const GemmStoreArgs g = two ? g2 : g4;
    gemm_store_tile<128, 128, FG, FA, true, false>(g, wg - (two ? n3 : n3 + n2), smem);
  }
}

bool moe_grads_fit(Phase3Args p3, GemmStoreArgs g2, GemmStoreArgs g4, int groups, int cus) {
  unsigned n3, n2, n4;
  return phase3_small(p3, n3) && gemm_store_small(g2, groups, n2) && gemm_store_small(g4, groups, n4) &&
         int64_t(n3) + n2 + n4 <= cus;
}

hipError_t launch_moe_grads(Phase3Args p3, GemmStoreArgs g2, GemmStoreArgs g4, int groups, int fg, int fw, int fa,
                            hipStream_t st) {
  unsigned n3, n2, n4;
  if (!phase3_small(p3, n3) || !gemm_store_small(g2, groups, n2) || !gemm_store_small(g4, groups, n4))
    return hipErrorInvalidValue;
  auto go = [&](auto FG, auto FW, auto FA) {
    moe_grads_kernel<FG(), FW(), FA()><<<n3 + n2 + n4, v2::kThreads, 0, st>>>(p3, int(n3), g2, int(n2), g4);
  };
  using E4 = std::integral_constant<int, kE4M3>;
  using E5 = std::integral_constant<int, kE5M2>;
  auto act = [&](auto FG, auto FW) {
    if (fa == kE4M3) go(FG, FW, E4{});
    else go(FG, FW, E5{});
  };
  auto weight = [&](auto FG) {
    if (fw == kE4M3) act(FG, E4{});
    else act(FG, E5{});
  };
  if (fg == kE4M3) weight(E4{});
  else weight(E5{});
  return hipGetLastError();
}

}  // namespace mx
