// router_fwd.hip -- the router forward: per token the K largest of its E logits
// (equal logits: the lower expert first), their scores, and the scores in the
// masked [T, E] layout that the MoE layer reads.
//
//   softmax over top-k, and renormalised top-k over softmax:
//       y_k = exp(z_k - m) / sum over the selection of exp(z - m)
//       (the renormalisation cancels the sum over all experts)
//   top-k over softmax:  y_k = exp(z_k - m) / sum over all experts
//   top-k:               y_k = z_k
// m is the token's largest logit.  An expert at -inf is closed to the token: it
// is never selected.  A masked token selects nothing.  A selection that finds
// no expert left holds id -1 (what the routing blocks drop) and score 0.
//
// HBM-bound: a row is E logits read and E affinities written, plus K ids and
// scores.  L lanes take one row and hold its columns lane, lane + L, ... in
// registers as 32-bit keys whose unsigned order is the logits' order; a
// selection is one maximum over the segment's lanes and one minimum over the
// columns that reach it, in registers (segment.hpp).  The lane that owns a
// selected column writes its id and score.
#include <type_traits>

#include "kernels.hpp"
#include "mx_device.hpp"
#include "segment.hpp"

namespace mx {

namespace {
constexpr int kThreads = 256;

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return bf16_to_f32(*p); }

// Unsigned order = the order of the values, -0 = +0, and -inf and NaN below
// every other key (0: closed, never selected).
__device__ __forceinline__ uint32_t order_key(float z) {
  const uint32_t b = __float_as_uint(z + 0.f);   // -0 + 0 = +0
  const uint32_t k = b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
  return z > -INFINITY ? k : 0u;                 // false for NaN
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}

enum { kOverSelection, kOverAll, kRaw };
}  // namespace

template <int L, int EPL, int SCORE, class LT>
__global__ void __launch_bounds__(kThreads) router_fwd_kernel(RouterFwdArgs p) {
  const int lane = threadIdx.x % L;
  const int64_t t = int64_t(blockIdx.x) * (kThreads / L) + threadIdx.x / L;
  if (t >= p.T) return;   // whole segments leave together
  const int E = int(p.E), K = int(p.K);
  const LT* row = static_cast<const LT*>(p.logits) + t * p.E;
  const bool live = !p.mask || p.mask[t] != 0;
  float z[EPL];
  uint32_t key[EPL];
  int rank[EPL];   // the column's place among the selected, -1: not selected
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = lane + L * j;
    z[j] = live && e < E ? load_logit(row + e) : -INFINITY;
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    key[j] = order_key(z[j]);
    rank[j] = -1;
  }
  uint32_t top = 0;
  int found = 0;
  for (int k = 0; k < K; ++k) {
    uint32_t best = key[0];
    int at = 0;
#pragma unroll
    for (int j = 1; j < EPL; ++j)
      if (key[j] > best) { best = key[j]; at = j; }
    const uint32_t most = seg::umax<L>(best);
    if (k == 0) top = most;
    if (most == 0) break;   // nothing open is left (the same in the whole segment)
    const uint32_t mine = best == most ? uint32_t(lane + L * at) : 0xffffffffu;
    const bool won = seg::umin<L>(mine) == mine && best == most;
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (won && j == at) { rank[j] = k; key[j] = 0; }
    found = k + 1;
  }
  const float m = key_value(top);
  float s = 0.f, inv = 0.f;
  if (SCORE != kRaw && found > 0) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      // closed experts: exp(-inf) = 0; a NaN logit reaches the sum over all
      z[j] = lane + L * j < E && (SCORE == kOverAll || rank[j] >= 0) ? expf(z[j] - m) : 0.f;
      s += z[j];
    }
    inv = 1.f / seg::sum<L>(s);
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = lane + L * j;
    const float y = rank[j] < 0 ? 0.f : SCORE == kRaw ? z[j] + 0.f : z[j] * inv;
    if (rank[j] >= 0) {
      p.idx[t * K + rank[j]] = e;
      p.scores[t * K + rank[j]] = y;
    }
    if (p.aff && e < E) p.aff[t * p.E + e] = y;
  }
  for (int k = found + lane; k < K; k += L) {
    p.idx[t * K + k] = -1;
    p.scores[t * K + k] = 0.f;
  }
}

template <int L, int EPL>
static void router_fwd_go(const RouterFwdArgs& p, hipStream_t st) {
  const int64_t rows = kThreads / L;
  const unsigned grid = unsigned((p.T + rows - 1) / rows);
  const int score = p.mode == kRouterTopk ? kRaw
                    : p.mode == kRouterSoftmaxOverTopk || p.renorm ? kOverSelection : kOverAll;
  auto go = [&](auto lt) {
    using LT = decltype(lt);
    if (score == kRaw) router_fwd_kernel<L, EPL, kRaw, LT><<<grid, kThreads, 0, st>>>(p);
    else if (score == kOverSelection) router_fwd_kernel<L, EPL, kOverSelection, LT><<<grid, kThreads, 0, st>>>(p);
    else router_fwd_kernel<L, EPL, kOverAll, LT><<<grid, kThreads, 0, st>>>(p);
  };
  if (p.bf16) go(uint16_t{});
  else go(float{});
}

hipError_t launch_router_fwd(const RouterFwdArgs& p, hipStream_t st) {
  if (p.T <= 0) return hipSuccess;
  if (p.E > kRouterFwdMaxExperts || (p.T + 3) / 4 > int64_t(INT32_MAX)) return hipErrorInvalidValue;
  if (p.E <= 8) router_fwd_go<8, 1>(p, st);
  else if (p.E <= 16) router_fwd_go<8, 2>(p, st);
  else if (p.E <= 32) router_fwd_go<8, 4>(p, st);
  else if (p.E <= 64) router_fwd_go<8, 8>(p, st);
  else if (p.E <= 128) router_fwd_go<16, 8>(p, st);
  else if (p.E <= 256) router_fwd_go<32, 8>(p, st);
  else if (p.E <= 512) router_fwd_go<64, 8>(p, st);
  else if (p.E <= 1024) router_fwd_go<64, 16>(p, st);
  else if (p.E <= 2048) router_fwd_go<64, 32>(p, st);
  else router_fwd_go<64, 64>(p, st);
  return hipGetLastError();
}

}  // namespace mx
