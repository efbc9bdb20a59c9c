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
// HBM-bound by its bytes: a row is E logits read and E affinities written, plus
// K ids and scores (T = 32768, E = 128, K = 8: 35.7 MB in 11.6 us on the GPU, 10.5 us a
// call in a row of calls, 3.4 TB/s; an elementwise pass over as many bytes takes
// 6.4 us).  What it has to be kept from is the arithmetic of the selection: K
// rounds of a maximum over a row cost more than the traffic (16.6 us).  So, for
// up to 8 selections of up to 512 experts, each lane sorts its 8 columns
// (router_rows.hpp) and log2 L exchanges merge the lanes' lists, keeping 8:
// the elementwise maxima of one list and the other reversed are the 8 largest
// of both, a bitonic sequence that three steps sort.  All on 32-bit words that
// carry the column in their low bits: exact for bf16 logits (16 bits each).
// An fp32 logit loses log2(8 L) low bits to the column; rows where that could
// have changed the selection or its order (two candidates equal in the bits
// left, which is seen after the merge) send their wave to the exact rounds, as
// do more selections or experts (T = 4096: E = 128, K = 8 5.4 us, K = 16 7.2, K = 32 11.8;
// E = 1024, K = 8 13.9).  What bounds it now: about 350 vector instructions
// a wave of four rows (half of the time), then the load, the four LDS exchanges and
// the store of a single round of waves, which do not overlap.
#include "kernels.hpp"
#include "router_rows.hpp"

namespace mx {

namespace {
constexpr int kThreads = 256;
enum { kOverSelection, kOverAll, kRaw };

// Unsigned order = the order of the values, -0 = +0; 0 for -inf and NaN (closed).
__device__ __forceinline__ uint32_t order_key(float z) {
  const uint32_t b = __float_as_uint(z + 0.f);   // -0 + 0 = +0
  const uint32_t k = b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
  return z > -INFINITY ? k : 0u;                 // false for NaN
}

__device__ __forceinline__ void cswap(uint32_t& a, uint32_t& b) {   // descending
  const uint32_t hi = a > b ? a : b, lo = a > b ? b : a;
  a = hi;
  b = lo;
}
// 8 words, descending: Batcher's odd-even merge sort, 19 exchanges
__device__ __forceinline__ void sort8(uint32_t (&v)[8]) {
  cswap(v[0], v[1]); cswap(v[2], v[3]); cswap(v[4], v[5]); cswap(v[6], v[7]);
  cswap(v[0], v[2]); cswap(v[1], v[3]); cswap(v[4], v[6]); cswap(v[5], v[7]);
  cswap(v[1], v[2]); cswap(v[5], v[6]);
  cswap(v[0], v[4]); cswap(v[1], v[5]); cswap(v[2], v[6]); cswap(v[3], v[7]);
  cswap(v[2], v[4]); cswap(v[3], v[5]);
  cswap(v[1], v[2]); cswap(v[3], v[4]); cswap(v[5], v[6]);
}
// a bitonic sequence of 8, descending
__device__ __forceinline__ void bitonic8(uint32_t (&v)[8]) {
  cswap(v[0], v[4]); cswap(v[1], v[5]); cswap(v[2], v[6]); cswap(v[3], v[7]);
  cswap(v[0], v[2]); cswap(v[1], v[3]); cswap(v[4], v[6]); cswap(v[5], v[7]);
  cswap(v[0], v[1]); cswap(v[2], v[3]); cswap(v[4], v[5]); cswap(v[6], v[7]);
}
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t umin(uint32_t a, uint32_t b) { return a < b ? a : b; }
// the order of the lowest finite value, -3.4e38 (bf16: its own lowest is above); -inf is below
constexpr uint32_t kOpen = 0x00800000u;

// the 8 largest of this lane's sorted list and another's (x(k): the other's entry k)
template <class X>
__device__ __forceinline__ void merge8(uint32_t (&v)[8], const X& x) {
  uint32_t o[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) o[k] = umax(v[k], x(7 - k));
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = o[k];
  bitonic8(v);
}
// the 8 largest of the segment's L lists, in every lane.  The mirrors work as
// in segment.hpp: the lists of a reduced group's lanes are equal by then.
template <int L>
__device__ __forceinline__ void merge_lanes(uint32_t (&v)[8]) {
#if defined(__HIP_DEVICE_COMPILE__)
  if constexpr (L > 1) merge8(v, [&](int k) { return seg::dpp<seg::kXor1>(v[k]); });
  if constexpr (L > 2) merge8(v, [&](int k) { return seg::dpp<seg::kXor2>(v[k]); });
  if constexpr (L > 4) merge8(v, [&](int k) { return seg::dpp<seg::kHalfMirror>(v[k]); });
  if constexpr (L > 8) merge8(v, [&](int k) { return seg::dpp<seg::kMirror>(v[k]); });
  // a row swap gives both halves' entries at once, to both halves
  auto swap_merge = [&](auto swap) {
    uint32_t a[8], b[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const auto r = swap(v[k]);
      a[k] = r[0];
      b[k] = r[1];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = umax(a[k], b[7 - k]);
    bitonic8(v);
  };
  if constexpr (L > 16)
    swap_merge([](uint32_t x) { return __builtin_amdgcn_permlane16_swap(x, x, false, false); });
  if constexpr (L > 32)
    swap_merge([](uint32_t x) { return __builtin_amdgcn_permlane32_swap(x, x, false, false); });
#endif
}

// One row by K rounds of a maximum over its lanes, exact for any K and E.
template <int L, int EPL, bool VEC, int SCORE>
__device__ __forceinline__ void select_rounds(const RouterFwdArgs& p, int64_t t, int lane, float (&z)[EPL]) {
  const int E = int(p.E), K = int(p.K);
  uint32_t key[EPL];
  int rank[EPL];   // the column's place among the selected, -1: not selected
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    key[j] = order_key(z[j]);
    rank[j] = -1;
  }
  float m = -INFINITY;   // the largest logit that is not closed
#pragma unroll
  for (int j = 0; j < EPL; ++j) m = fmaxf(m, z[j]);
  m = seg::max<L>(m);
  int found = 0;
  for (int k = 0; k < K; ++k) {
    uint32_t best = key[0];
    int at = 0;
#pragma unroll
    for (int j = 1; j < EPL; ++j)
      if (key[j] > best) { best = key[j]; at = j; }
    const uint32_t most = seg::umax<L>(best);
    if (most == 0) break;   // nothing open is left (the same in the whole segment)
    const uint32_t mine = best == most ? uint32_t(rows::column<L>(lane, at)) : 0xffffffffu;
    const bool won = seg::umin<L>(mine) == mine && best == most;
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (won && j == at) { rank[j] = k; key[j] = 0; }
    found = k + 1;
  }
  float inv = 0.f;
  if (SCORE != kRaw && found > 0) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      // closed experts: exp(-inf) = 0; a NaN logit reaches the sum over all
      z[j] = SCORE == kOverAll || rank[j] >= 0 ? rows::exp_fast(z[j] - m) : 0.f;
      s += z[j];
    }
    inv = rows::rcp_fast(seg::sum<L>(s));
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    z[j] = rank[j] < 0 ? 0.f : SCORE == kRaw ? z[j] + 0.f : z[j] * inv;
    if (rank[j] >= 0) {
      p.idx[t * K + rank[j]] = rows::column<L>(lane, j);
      p.scores[t * K + rank[j]] = z[j];
    }
  }
  if (p.aff) rows::store<L, EPL, VEC>(p.aff + t * p.E, E, lane, z);
  for (int k = found + lane; k < K; k += L) {
    p.idx[t * K + k] = -1;
    p.scores[t * K + k] = 0.f;
  }
}
}  // namespace

template <int L, int EPL, bool VEC, int SCORE, class LT>
__global__ void __launch_bounds__(kThreads) router_fwd_kernel(RouterFwdArgs p) {
  const int lane = threadIdx.x % L;
  const int64_t t = int64_t(blockIdx.x) * (kThreads / L) + threadIdx.x / L;
  if (t >= p.T) return;   // whole segments leave together
  float z[EPL];
  rows::load<L, EPL, VEC>(static_cast<const LT*>(p.logits) + t * p.E, int(p.E), lane, z);
  if (p.mask && !p.mask[t]) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) z[j] = -INFINITY;
  }
  select_rounds<L, EPL, VEC, SCORE>(p, t, lane, z);
}

// The merge: K <= 8, E <= 8 L <= 512.
template <int L, bool VEC, int SCORE, class LT>
__global__ void __launch_bounds__(kThreads) router_merge_kernel(RouterFwdArgs p) {
  constexpr bool BF16 = std::is_same_v<LT, uint16_t>;
  constexpr uint32_t COLS = BF16 ? 0xffffu : uint32_t(8 * L - 1);   // the word's column bits (complemented)
  constexpr int R = 64 / L, KL = L < 8 ? 8 / L : 1;                 // selections of one lane
  __shared__ float zs[kThreads * 8];   // each wave's rows, 8 L columns each
  const int lane = threadIdx.x % L, slot = (threadIdx.x & 63) / L;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t0 = int64_t(blockIdx.x) * (kThreads / L) + wave * R;   // the wave's first row
  if (t0 >= p.T) return;   // whole waves leave
  const bool in = slot < p.T - t0;
  const int E = int(p.E), K = int(p.K);
  float z[8];
  const int row = in ? slot : 0;
  rows::load<L, 8, VEC>(static_cast<const LT*>(p.logits) + t0 * p.E + row * E, E, lane, z);
  if (!in || (p.mask && !p.mask[t0 + slot])) {
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] = -INFINITY;
  }
  // words: the logit's order with the column, complemented, in the low bits;
  // closed columns are below kOpen
  uint32_t v[8], own[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t b = __float_as_uint(fmaxf(z[j] + 0.f, -INFINITY));   // -0 + 0 = +0, NaN: -inf
    own[j] = v[j] = ((b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u)) & ~COLS) | (COLS - rows::column<L>(lane, j));
  }
  sort8(v);
  merge_lanes<L>(v);
  if (!BF16) {
    // Equal high bits: neighbours in the order (up to one past the last
    // selection), or, with 8 selections, a column that is not among them with
    // the last: then more than 8 of the row's words reach its high bits.
    uint32_t near = 0xffffffffu;
#pragma unroll
    for (int k = 0; k < 7; ++k) near = umin(near, (v[k] ^ v[k + 1]) | (k < K ? 0u : 0xffffffffu));
    int reach = 0;
    if (K == 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) reach += __popcll(__ballot(own[j] >= (v[7] & ~COLS)));
    }
    if (__ballot(near <= COLS) || reach > 8 * R) {
      // closed columns are no clash: look again, without them
      bool clash = false;
      uint32_t last = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k + 1 < 8) clash |= k + 1 < K && v[k + 1] >= kOpen && (v[k] ^ v[k + 1]) <= COLS;
        if (k + 1 == K) last = v[k];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) clash |= last >= kOpen && own[j] < last && (own[j] ^ last) <= COLS;
      if (__ballot(clash)) {   // the whole wave: no lane of a segment leaves alone
        if (in) select_rounds<L, 8, VEC, SCORE>(p, t0 + slot, lane, z);
        return;
      }
    }
  }
  // The selections go to one lane each (several where L < 8), which reads
  // their logits from the row in LDS.  All within the wave.
  float* zr = zs + (wave * R + slot) * 8 * L;
  float4* lo = reinterpret_cast<float4*>(zr) + lane;   // the lane's two runs
  float4* hi = lo + L;
  *lo = float4{z[0], z[1], z[2], z[3]};
  *hi = float4{z[4], z[5], z[6], z[7]};
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  int col[KL];
  float y[KL];
#pragma unroll
  for (int i = 0; i < KL; ++i) {
    uint32_t w = 0;
#pragma unroll
    for (int k = i * L; k < i * L + L && k < 8; ++k)
      if (lane == k - i * L) w = k < K ? v[k] : 0u;
    col[i] = w >= kOpen ? int(COLS - (w & COLS)) : -1;
    y[i] = w >= kOpen ? zr[col[i]] : -INFINITY;
  }
  if (SCORE != kRaw) {
    // v[0] is the largest: its logit is m; +inf - +inf makes the row NaN
    const float m = v[0] >= kOpen ? zr[COLS - (v[0] & COLS)] : 0.f;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < KL; ++i) {
      y[i] = rows::exp_fast(y[i] - m);
      if (SCORE == kOverSelection) s += y[i];
    }
    if (SCORE == kOverAll) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s += rows::exp_fast(z[j] - m);
    }
    s = seg::sum<L>(s);
    const float inv = s != 0.f ? rows::rcp_fast(s) : 0.f;   // 0: nothing open
#pragma unroll
    for (int i = 0; i < KL; ++i) y[i] *= inv;
  }
  const int64_t out = t0 * K;
  if (in) {
#pragma unroll
    for (int i = 0; i < KL; ++i) {
      const int k = lane + i * L;
      if (k < K) {
        y[i] = col[i] >= 0 ? y[i] + 0.f : 0.f;
        p.idx[out + slot * K + k] = col[i];
        p.scores[out + slot * K + k] = y[i];
      }
    }
  }
  if (!p.aff) return;
  // the row again: zeros, the scores, and back
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  *lo = *hi = float4{0.f, 0.f, 0.f, 0.f};
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int i = 0; i < KL; ++i)
    if (lane + i * L < K && col[i] >= 0) zr[col[i]] = y[i];
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  const float4 a = *lo, b = *hi;
  const float w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (in) rows::store<L, 8, VEC>(p.aff + t0 * p.E + slot * E, E, lane, w);
}

int64_t router_max_tokens(int64_t E) { return rows::max_tokens(E); }

hipError_t launch_router_fwd(const RouterFwdArgs& p, hipStream_t st) {
  if (p.T <= 0) return hipSuccess;
  const int64_t r = kThreads / rows::lanes(p.E);
  if (p.E > kRouterFwdMaxExperts || p.T > rows::max_tokens(p.E)) return hipErrorInvalidValue;
  const unsigned grid = unsigned((p.T + r - 1) / r);
  const int score = p.mode == kRouterTopk ? kRaw
                    : p.mode == kRouterSoftmaxOverTopk || p.renorm ? kOverSelection : kOverAll;
  rows::by_experts(p.E, [&](auto L, auto EPL, auto vec) {
    auto go = [&](auto sc, auto lt) {
      if constexpr (EPL() == 8) {
        if (p.K <= 8) {
          router_merge_kernel<L(), vec(), sc(), decltype(lt)><<<grid, kThreads, 0, st>>>(p);
          return;
        }
      }
      router_fwd_kernel<L(), EPL(), vec(), sc(), decltype(lt)><<<grid, kThreads, 0, st>>>(p);
    };
    auto kind = [&](auto sc) {
      if (p.bf16) go(sc, uint16_t{});
      else go(sc, float{});
    };
    if (score == kRaw) kind(rows::Int<kRaw>{});
    else if (score == kOverSelection) kind(rows::Int<kOverSelection>{});
    else kind(rows::Int<kOverAll>{});
  });
  return hipGetLastError();
}

}  // namespace mx
