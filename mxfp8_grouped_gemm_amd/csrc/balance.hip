// balance.hip -- the router's auxiliary losses: per-expert counts, the load-
// balance loss per sequence and the z loss, and their gradient on the logits.
//
// With p_t = softmax over all E logits of token t, lse_t its log-sum-exp, n_s
// the tokens of sequence s that take part, S' the sequences that have any, n
// their tokens in all, and c_se the selections of expert e in sequence s:
//   balance = (b / S') sum_s E sum_e (c_se / (K n_s)) (1 / n_s) sum_{t in s} p_te
//   z       = (z / n) sum_t lse_t^2
//   d_te    = g_b p_te (w_se - sum_j w_sj p_tj) + g_z (2 z / n) lse_t p_te,
//             w_se = b E c_se / (S' K n_s^2)
// A token takes part if it lies in a sequence, its mask byte is not 0 and one of
// its logits is above -inf.
//
// Forward, two launches.  The first cuts the tokens into chunks, one workgroup
// each; a workgroup goes through the sequences that meet its chunk and writes,
// for each, the sums of p per expert, the counts, the tokens and the sum of
// lse^2 to record chunk + sequence (moving along the tokens raises one of the
// two each time, so the records of different pairs never meet).  The second
// adds a sequence's records in chunk order, and the last of its workgroups to
// finish the sequences' terms in sequence order: no floating-point atomics, the
// same bits on every run.
// HBM-bound: E logits and K ids a token; backward E logits read, E gradients
// written.
#include <type_traits>

#include "kernels.hpp"
#include "mx_device.hpp"
#include "segment.hpp"

namespace mx {

namespace {
constexpr int kThreads = 256;
constexpr int kTile = 64;   // experts of one workgroup of the second launch

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return bf16_to_f32(*p); }

// first token of sequence s (s in [0, S]), kept in [0, T]
__device__ __forceinline__ int64_t seq_at(const BalanceArgs& p, int64_t s) {
  if (!p.seq) return s ? p.T : 0;
  const int64_t v = p.seq[s];
  return v < 0 ? 0 : v > p.T ? p.T : v;
}
// the last s in [0, S] whose sequence starts at or before token t; -1 if none
__device__ __forceinline__ int64_t seq_of(const BalanceArgs& p, int64_t t) {
  if (!p.seq) return t < p.T ? 0 : 1;
  int64_t lo = 0, hi = p.S + 1;   // entries before lo are <= t, from hi on > t
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (seq_at(p, mid) <= t) lo = mid + 1;
    else hi = mid;
  }
  return lo - 1;
}

// One row's softmax over all experts by L lanes: x[j] becomes p at column
// lane + L j; returns false where no logit is above -inf (x is 0 then).
template <int L, int EPL, class LT>
__device__ __forceinline__ bool row_softmax(const LT* row, int E, int lane, float (&x)[EPL], float& lse) {
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = lane + L * j;
    x[j] = e < E ? load_logit(row + e) : -INFINITY;
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j) m = fmaxf(m, x[j]);
  m = seg::max<L>(m);
  const bool some = m > -INFINITY;
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    x[j] = some && lane + L * j < E ? expf(x[j] - m) : 0.f;
    s += x[j];
  }
  s = seg::sum<L>(s);
  const float inv = some ? 1.f / s : 0.f;
#pragma unroll
  for (int j = 0; j < EPL; ++j) x[j] *= inv;
  lse = some ? m + logf(s) : 0.f;
  return some;
}
}  // namespace

template <int L, int EPL, class LT>
__global__ void __launch_bounds__(kThreads) balance_chunk_kernel(BalanceArgs p) {
  constexpr int R = kThreads / L;          // rows at a time
  constexpr int W = kThreads / 64;
  __shared__ float lp[W][L * EPL];
  __shared__ int hist[L * EPL];
  __shared__ float lz[W];
  __shared__ int ln[W];
  const int lane = threadIdx.x % L, slot = threadIdx.x / L, wave = threadIdx.x >> 6;
  const int E = int(p.E), K = int(p.K);
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.done = 0;   // read by the next launch only
  const int64_t c0 = int64_t(blockIdx.x) * p.chunk;
  const int64_t c1 = c0 + p.chunk < p.T ? c0 + p.chunk : p.T;
  if (c0 >= c1) return;
  int64_t s = seq_of(p, c0);
  for (s = s < 0 ? 0 : s; s < p.S; ++s) {
    const int64_t a = seq_at(p, s), b = seq_at(p, s + 1);
    if (a >= c1) break;
    const int64_t lo = a > c0 ? a : c0, hi = b < c1 ? b : c1;
    if (lo >= hi) continue;
    for (int e = threadIdx.x; e < E; e += kThreads) hist[e] = 0;
    __syncthreads();
    float acc[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) acc[j] = 0.f;
    float z2 = 0.f;
    int n = 0;
    for (int64_t t = lo + slot; t < hi; t += R) {
      if (p.mask && !p.mask[t]) continue;
      float x[EPL], lse;
      if (!row_softmax<L, EPL>(static_cast<const LT*>(p.logits) + t * p.E, E, lane, x, lse)) continue;
#pragma unroll
      for (int j = 0; j < EPL; ++j) acc[j] += x[j];
      if (lane == 0) {
        z2 += lse * lse;
        ++n;
      }
      for (int k = lane; k < K; k += L) {
        const int e = p.idx[t * K + k];
        if (e >= 0 && e < E) atomicAdd(&hist[e], 1);
      }
    }
    // the wave's row slots, then the waves
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      float v = acc[j];
      for (int o = L; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
      if ((threadIdx.x & 63) < L) lp[wave][lane + L * j] = v;
    }
    for (int o = 1; o < 64; o <<= 1) {
      z2 += __shfl_xor(z2, o, 64);
      n += __shfl_xor(n, o, 64);
    }
    if ((threadIdx.x & 63) == 0) { lz[wave] = z2; ln[wave] = n; }
    __syncthreads();
    const int64_t rec = int64_t(blockIdx.x) + s;
    for (int e = threadIdx.x; e < E; e += kThreads) {
      float v = lp[0][e];
#pragma unroll
      for (int w = 1; w < W; ++w) v += lp[w][e];
      p.part_p[rec * p.E + e] = v;
      p.part_c[rec * p.E + e] = hist[e];
    }
    if (threadIdx.x == 0) {
      float v = lz[0];
      int m = ln[0];
#pragma unroll
      for (int w = 1; w < W; ++w) { v += lz[w]; m += ln[w]; }
      p.part_z[rec] = v;
      p.part_n[rec] = m;
    }
    __syncthreads();   // before the next sequence's histogram
  }
}

// Grid (S, tiles of kTile experts): thread (q, e) adds every fourth record of
// its sequence for expert e.
__global__ void __launch_bounds__(kThreads) balance_sum_kernel(BalanceArgs p) {
  constexpr int Q = kThreads / kTile;
  __shared__ float sp[Q][kTile];
  __shared__ int sc[Q][kTile];
  __shared__ int sn[kThreads];
  __shared__ float sz[kThreads];
  __shared__ bool last;
  const int64_t s = blockIdx.x;
  const int tid = threadIdx.x, q = tid / kTile, col = tid % kTile;
  const int64_t e = int64_t(blockIdx.y) * kTile + col;
  const int64_t a = seq_at(p, s), b = seq_at(p, s + 1);
  const int64_t f = a < b ? a / p.chunk : 0, l = a < b ? (b - 1) / p.chunk : -1;   // its chunks
  float v = 0.f;
  int c = 0;
  if (e < p.E)
    for (int64_t k = f + q; k <= l; k += Q) {
      v += p.part_p[(k + s) * p.E + e];
      c += p.part_c[(k + s) * p.E + e];
    }
  sp[q][col] = v;
  sc[q][col] = c;
  int n = 0;
  float z = 0.f;
  for (int64_t k = f + tid; k <= l; k += kThreads) {
    n += p.part_n[k + s];
    z += p.part_z[k + s];
  }
  sn[tid] = n;
  sz[tid] = z;
  __syncthreads();
  for (int o = kThreads / 2; o; o >>= 1) {
    if (tid < o) {
      sn[tid] += sn[tid + o];
      sz[tid] += sz[tid + o];
    }
    __syncthreads();
  }
  n = sn[0];
  if (q == 0) {
    for (int i = 1; i < Q; ++i) {
      v += sp[i][col];
      c += sc[i][col];
    }
    if (e < p.E) p.counts[s * p.E + e] = c;
    // the tile's share of sum_e c_se sum_t p_te / n_s^2
    double d = n > 0 ? double(c) * double(v) / (double(n) * double(n)) : 0.;
    for (int o = 1; o < kTile; o <<= 1) d += __shfl_xor(d, o, 64);
    if (tid == 0) {
      p.term[s * gridDim.y + blockIdx.y] = d;
      if (blockIdx.y == 0) {
        p.num[s] = n;
        p.term_z[s] = sz[0];
      }
      __threadfence();
      last = atomicAdd(p.done, 1u) == gridDim.x * gridDim.y - 1;
    }
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  // all sequences' terms, in an order that does not depend on who is last
  __shared__ double db[kThreads], dz[kThreads];
  __shared__ int di[kThreads], dl[kThreads];
  double tb = 0., tz = 0.;
  int all = 0, live = 0;
  const volatile double* term = p.term;
  const volatile float* term_z = p.term_z;
  const volatile int32_t* num = p.num;
  for (int64_t i = tid; i < p.S * gridDim.y; i += kThreads) tb += term[i];
  for (int64_t i = tid; i < p.S; i += kThreads) {
    tz += term_z[i];
    all += num[i];
    live += num[i] > 0;
  }
  db[tid] = tb; dz[tid] = tz; di[tid] = all; dl[tid] = live;
  __syncthreads();
  for (int o = kThreads / 2; o; o >>= 1) {
    if (tid < o) {
      db[tid] += db[tid + o];
      dz[tid] += dz[tid + o];
      di[tid] += di[tid + o];
      dl[tid] += dl[tid + o];
    }
    __syncthreads();
  }
  if (tid == 0) {
    all = di[0];
    live = dl[0];
    p.num[p.S] = live;
    p.num[p.S + 1] = all;
    p.loss[0] = live ? float(double(p.balance_coef) * double(p.E) * db[0] / (double(p.K) * live)) : 0.f;
    p.loss[1] = all ? float(double(p.z_coef) * dz[0] / all) : 0.f;
  }
}

template <int L, int EPL, class LT>
__global__ void __launch_bounds__(kThreads) balance_bwd_kernel(BalanceArgs p) {
  const int lane = threadIdx.x % L;
  const int64_t t = int64_t(blockIdx.x) * (kThreads / L) + threadIdx.x / L;
  if (t >= p.T) return;   // whole segments leave together
  const int E = int(p.E);
  float* out = p.dlogits + t * p.E;
  const int64_t s = seq_of(p, t);
  float x[EPL], lse = 0.f;
  bool part = s >= 0 && s < p.S && t < seq_at(p, s + 1) && (!p.mask || p.mask[t] != 0);
  if (part) part = row_softmax<L, EPL>(static_cast<const LT*>(p.logits) + t * p.E, E, lane, x, lse);
  if (!part) {
    if (!p.accumulate)
      for (int e = lane; e < E; e += L) out[e] = 0.f;
    return;
  }
  const float gb = p.dloss ? p.dloss[0] : 1.f, gz = p.dloss ? p.dloss[1] : 1.f;
  const float n = float(p.num[s]), live = float(p.num[p.S]), all = float(p.num[p.S + 1]);
  const float fb = gb * (p.balance_coef * float(p.E) / (live * float(p.K) * n)) / n;
  const float fz = gz * (2.f * p.z_coef / all) * lse;
  float w[EPL], dot = 0.f;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = lane + L * j;
    w[j] = e < E ? fb * float(p.counts[s * p.E + e]) : 0.f;
    dot += w[j] * x[j];
  }
  dot = seg::sum<L>(dot) - fz;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = lane + L * j;
    if (e < E) {
      const float d = x[j] * (w[j] - dot);
      out[e] = p.accumulate ? out[e] + d : d;
    }
  }
}

namespace {
// f(L, EPL) for E experts: L = E / 8 rounded up to a power of two in [8, 64]
template <int N> using Int = std::integral_constant<int, N>;
template <class F>
void by_experts(int64_t E, const F& f) {
  if (E <= 8) f(Int<8>{}, Int<1>{});
  else if (E <= 16) f(Int<8>{}, Int<2>{});
  else if (E <= 32) f(Int<8>{}, Int<4>{});
  else if (E <= 64) f(Int<8>{}, Int<8>{});
  else if (E <= 128) f(Int<16>{}, Int<8>{});
  else if (E <= 256) f(Int<32>{}, Int<8>{});
  else if (E <= 512) f(Int<64>{}, Int<8>{});
  else if (E <= 1024) f(Int<64>{}, Int<16>{});
  else if (E <= 2048) f(Int<64>{}, Int<32>{});
  else f(Int<64>{}, Int<64>{});
}
int rows_at_a_time(int64_t E) { return E <= 64 ? 32 : E <= 128 ? 16 : E <= 256 ? 8 : 4; }
}  // namespace

// Tokens of one chunk: one round of rows, or more where that would make over
// 1024 chunks.
int64_t balance_chunk_tokens(int64_t T, int64_t E) {
  const int64_t r = rows_at_a_time(E);
  const int64_t c = (T + 1023) / 1024;
  return c <= r ? r : (c + r - 1) / r * r;
}

hipError_t launch_balance_fwd(const BalanceArgs& p, hipStream_t st) {
  const int64_t chunks = (p.T + p.chunk - 1) / p.chunk;
  const unsigned grid = unsigned(chunks > 0 ? chunks : 1);
  by_experts(p.E, [&](auto L, auto EPL) {
    if (p.bf16) balance_chunk_kernel<L(), EPL(), uint16_t><<<grid, kThreads, 0, st>>>(p);
    else balance_chunk_kernel<L(), EPL(), float><<<grid, kThreads, 0, st>>>(p);
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  balance_sum_kernel<<<dim3(unsigned(p.S), unsigned((p.E + kTile - 1) / kTile)), kThreads, 0, st>>>(p);
  return hipGetLastError();
}

hipError_t launch_balance_bwd(const BalanceArgs& p, hipStream_t st) {
  if (p.T <= 0) return hipSuccess;
  const int64_t rows = rows_at_a_time(p.E);
  const unsigned grid = unsigned((p.T + rows - 1) / rows);
  by_experts(p.E, [&](auto L, auto EPL) {
    if (p.bf16) balance_bwd_kernel<L(), EPL(), uint16_t><<<grid, kThreads, 0, st>>>(p);
    else balance_bwd_kernel<L(), EPL(), float><<<grid, kThreads, 0, st>>>(p);
  });
  return hipGetLastError();
}

}  // namespace mx
