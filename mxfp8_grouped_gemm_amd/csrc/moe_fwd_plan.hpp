// moe_fwd_plan.hpp -- how the MoE forward's preparation (moe_fwd_prep.hip) is
// launched: host arithmetic on the sizes alone, without HIP.
#pragma once
#include <stdint.h>

namespace mx {

// Threads that one launch takes: the runtime runs a grid's threads modulo 2^32,
// without an error.
constexpr int64_t kMaxLaunchThreads = (int64_t(1) << 32) - 1;

constexpr int kPrepThreads = 256;
// A small layer (slots, T * E): one workgroup of kSmallThreads sets up its slots beside the others.  T = 1500, 23
// blocks of 256: 10.0 us (15.6 with 256 threads), where two launches took 6.2 and 7.6.
constexpr int64_t kSmallSlots = 8192, kSmallPairs = 32768;
constexpr int kSmallThreads = 1024;

struct FwdPrepPlan {
  bool small;
  int threads;             // of a workgroup
  int64_t nq, ns, nf;      // workgroups: X, the weights' scales, the inverse map's fill (not small)
  int64_t grid;            // of all, and a small layer's one for the slots
};
inline FwdPrepPlan fwd_prep_plan(int64_t T, int64_t H, int64_t I, int64_t E, int64_t N, int64_t B, bool x_by_slot) {
  auto up = [](int64_t v, int64_t n) { return (v + n - 1) / n; };
  const int64_t Hp = up(H, 128) * 128, Ip = up(I, 128) * 128;
  // 64 rows x 32 words of scales each (PairsJob)
  const int64_t ns = E * (up(2 * I, 64) * up(Hp, 4096) + up(H, 64) * up(Ip, 4096));
  auto plan = [&](bool small) {
    FwdPrepPlan p{small, small ? kSmallThreads : kPrepThreads, 0, ns, 0, 0};
    const int64_t want = up(T * (Hp / 8), int64_t(4) * p.threads);
    p.nq = x_by_slot ? N * B / 32 * up(Hp, 256) : want < 65536 ? want : 65536;
    p.nf = small ? 0 : up(T * E, 4 * kPrepThreads);
    p.grid = p.nq + p.ns + p.nf + (small ? 1 : 0);
    return p;
  };
  const FwdPrepPlan p = plan(N * B <= kSmallSlots && T * E <= kSmallPairs && !x_by_slot);
  // so many experts or weight rows that workgroups of kSmallThreads pass what one launch takes
  return p.small && p.grid > kMaxLaunchThreads / kSmallThreads ? plan(false) : p;
}

}  // namespace mx
