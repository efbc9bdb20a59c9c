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
// Forward, two launches (one for few tokens, see balance_one).  The first cuts
// the tokens into chunks, one workgroup each; a workgroup goes through its rows
// a round at a time and through the sequences that meet each round, and writes,
// for each sequence, the sums of p per expert, the counts, the tokens and the
// sum of lse^2 to record chunk + sequence (moving along the tokens raises one
// of the two each time, so the records of different pairs never meet).  The
// second adds a sequence's records in an order fixed by the sizes, and the last
// of its workgroups to finish the sequences' terms likewise: no floating-point
// atomics, the same bits on every run.
// HBM-bound by its bytes: E logits and K ids a token; backward E logits read, E
// gradients written (rows in registers, router_rows.hpp).  T = 32768, E = 128,
// K = 8, 16 sequences: chunks 8.4 us (17.8 MB), sums 7.2 us (latency: records,
// one atomic, the last workgroup's terms), gradient 9.2 us (33.6 MB, 3.7 TB/s;
// an elementwise pass over as many bytes takes 6.4 us).  T = 16384, E = 8: 5.7
// and 3.7 us (one workgroup, which needs no one else's terms), all of it latency.
#include "kernels.hpp"
#include "router_rows.hpp"

namespace mx {

namespace {
constexpr int kBwdThreads = 256;
constexpr int kSumThreads = 1024;
constexpr int kTile = 32;        // experts of one workgroup of the second launch
constexpr int kChunks = 512;     // two workgroups of the first launch per CU

// threads of the chunk kernel: its LDS holds a row of E sums per wave
constexpr int chunk_threads(int EPL) { return EPL > 8 ? 256 : 512; }

// first token of sequence s (s in [0, S]), kept in [0, T]
__device__ __forceinline__ int64_t seq_at(const BalanceArgs& p, int64_t s) {
  if (!p.seq) return s ? p.T : 0;
  const int64_t v = p.seq[s];
  return v < 0 ? 0 : v > p.T ? p.T : v;
}

// The part of seq_starts around token t, found by the whole wave, 64 entries a
// step: `lo` and this lane's entry lo + lane (past every token behind the last
// one), such that lo = 0 or entry lo is at or before t, and the first entry past
// t is among the 64 or just behind them.
__device__ __forceinline__ int64_t seq_window(const BalanceArgs& p, int64_t t, int64_t& v) {
  const int lane = threadIdx.x & 63;
  int64_t lo = 0, n = p.S + 1;
  while (n > 64) {
    const int64_t step = (n + 63) / 64;
    const int c = __popcll(__ballot(lane * step < n && seq_at(p, lo + lane * step) <= t));
    if (c == 0) break;   // entry 0 is past t
    n = n - (c - 1) * step < step ? n - (c - 1) * step : step;
    lo += (c - 1) * step;
  }
  v = lo + lane <= p.S ? seq_at(p, lo + lane) : p.T + 1;
  return lo;
}
// Goes through the sequences from the one that may hold token t on (the last one
// that starts at or before it, or the first): s and its bounds a, b, the same
// in the whole wave.  64 starts are held in the wave's lanes.
struct SeqCursor {
  int64_t s, a, b;
  int64_t lo, v;   // this lane holds entry lo + lane
  __device__ __forceinline__ SeqCursor(const BalanceArgs& p, int64_t t) : s(0), a(0), b(p.T), lo(0), v(0) {
    if (!p.seq) return;
    lo = seq_window(p, t, v);
    const int c = __popcll(__ballot(v <= t));
    s = lo + c > 0 ? lo + c - 1 : 0;
    a = entry(p, s);
    b = entry(p, s + 1);
  }
  __device__ __forceinline__ int64_t entry(const BalanceArgs& p, int64_t i) {
    if (i > p.S) return p.T;   // behind the last sequence: not looked at
    if (i < lo || i >= lo + 64) {
      lo = i;
      v = i + (threadIdx.x & 63) <= p.S ? seq_at(p, i + (threadIdx.x & 63)) : p.T;
    }
    return __shfl(int(v), int(i - lo), 64);   // T < 2^31
  }
  __device__ __forceinline__ void next(const BalanceArgs& p) {
    ++s;
    a = b;
    b = p.seq ? entry(p, s + 1) : p.T;
  }
};
// The same for each of the wave's 64 / L rows t0, t0 + 1, ... by its own lanes.
template <int L>
__device__ __forceinline__ int64_t seq_of_rows(const BalanceArgs& p, int64_t t0) {
  if (!p.seq) return t0 < p.T ? 0 : 1;   // rows past T are not looked at
  constexpr int R = 64 / L;
  const int lane = threadIdx.x & 63;
  int64_t v;
  const int64_t lo = seq_window(p, t0, v);
  int c = __popcll(__ballot(v <= t0));
  const uint64_t end = __ballot(v <= t0 + R - 1);
  if (end == ~uint64_t(0)) {   // starts past the window may lie among these rows: each row by itself
    const int64_t t = t0 + lane / L;
    int64_t l = lo, h = p.S + 1;
    while (l < h) {
      const int64_t mid = (l + h) >> 1;
      if (seq_at(p, mid) <= t) l = mid + 1;
      else h = mid;
    }
    return l - 1;
  }
  if (__popcll(end) != c) {
#pragma unroll 4
    for (int r = 1; r < R; ++r) {
      const int k = __popcll(__ballot(v <= t0 + r));
      if (lane / L == r) c = k;
    }
  }
  return lo - 1 + c;
}
// tb = sum_s sum_e c_se sum_t p_te / n_s^2, tz = sum_t lse_t^2
__device__ __forceinline__ void write_totals(const BalanceArgs& p, double tb, double tz, int all, int live) {
  p.num[p.S] = live;
  p.num[p.S + 1] = all;
  p.loss[0] = live ? float(double(p.balance_coef) * double(p.E) * tb / (double(p.K) * live)) : 0.f;
  p.loss[1] = all ? float(double(p.z_coef) * tz / all) : 0.f;
}
}  // namespace

// ALL: one workgroup takes every token and sequence and writes the results.
template <int L, int EPL, bool VEC, class LT, bool ALL>
__global__ void __launch_bounds__(chunk_threads(EPL)) balance_chunk_kernel(BalanceArgs p) {
  constexpr int THREADS = chunk_threads(EPL);
  constexpr int R = THREADS / L;   // rows at a time
  constexpr int W = THREADS / 64;
  constexpr int IDS = (kRouterMaxK + L - 1) / L;   // ids of one lane, K <= 32
  __shared__ float lp[W][L * EPL];
  __shared__ int hist[L * EPL];
  __shared__ double lz[W];
  __shared__ int ln[W];
  const int lane = threadIdx.x % L, slot = threadIdx.x / L, wave = threadIdx.x >> 6;
  const int E = int(p.E), K = int(p.K);
  if (!ALL && blockIdx.x == 0 && threadIdx.x == 0) *p.done = 0;   // read by the next launch only
  const int64_t c0 = int64_t(blockIdx.x) * p.chunk;
  const int64_t c1 = !ALL && c0 + p.chunk < p.T ? c0 + p.chunk : p.T;
  if (!ALL && c0 >= c1) return;
  double term = 0., term_z = 0.;   // ALL: this thread's share of the balance sum, the z sum
  int all = 0, live_seqs = 0;
  const LT* logits = static_cast<const LT*>(p.logits);
  // a round's rows and ids are loaded one round ahead, the first ones while the
  // sequence is looked up
  float nx[EPL];
  int nid[IDS];
  bool nlive = false;
  auto fetch = [&](int64_t t) {
    if (t >= c1) return;
    rows::load<L, EPL, VEC>(logits + t * p.E, E, lane, nx);
#pragma unroll
    for (int k = 0; k < IDS; ++k) nid[k] = lane + L * k < K ? p.idx[t * K + lane + L * k] : -1;
    nlive = !p.mask || p.mask[t] != 0;
  };
  fetch(c0 + slot);
  float acc[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) acc[j] = 0.f;
  // lse^2 in fp64: the square of a token whose logits are all the type's lowest value passes fp32
  double z2 = 0.;
  float n = 0.f;   // whole numbers, at most a chunk's tokens
  for (int e = threadIdx.x; e < E; e += THREADS) hist[e] = 0;
  SeqCursor q(p, ALL ? -1 : c0);
  __syncthreads();
  // writes what has been gathered for sequence q.s, and starts the next
  auto flush = [&]() {
    // the wave's row slots, then the waves
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const float v = seg::across<L>(acc[j]);
      acc[j] = 0.f;
      if ((threadIdx.x & 63) < L) lp[wave][rows::column<L>(lane, j)] = v;
    }
    z2 = seg::across<L>(z2);   // the rows' first lanes hold it
    n = seg::sum<64>(n);
    if ((threadIdx.x & 63) == 0) { lz[wave] = z2; ln[wave] = int(n); }
    z2 = 0.;
    n = 0.f;
    __syncthreads();
    double zs = 0.;
    int ns = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) { zs += lz[w]; ns += ln[w]; }
    const int64_t rec = ALL ? q.s : int64_t(blockIdx.x) + q.s;
    double d = 0.;
    for (int e = threadIdx.x; e < E; e += THREADS) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) v += lp[w][e];
      const int c = hist[e];
      hist[e] = 0;
      if constexpr (ALL) {
        p.counts[rec * p.E + e] = c;
        d += double(c) * double(v);
      } else {
        p.part_p[rec * p.E + e] = v;
        p.part_c[rec * p.E + e] = c;
      }
    }
    if constexpr (ALL) {
      if (ns > 0) term += d / (double(ns) * double(ns));
      term_z += zs;
      all += ns;
      live_seqs += ns > 0;
      if (threadIdx.x == 0) p.num[rec] = ns;
    } else if (threadIdx.x == 0) {
      p.part_z[rec] = zs;
      p.part_n[rec] = ns;
    }
    __syncthreads();
  };
  auto zeros = [&]() {
    for (int e = threadIdx.x; e < E; e += THREADS) p.counts[q.s * p.E + e] = 0;
    if (threadIdx.x == 0) p.num[q.s] = 0;
  };
  for (int64_t t0 = c0; t0 < c1; t0 += R) {
    const int64_t t = t0 + slot, t1 = t0 + R < c1 ? t0 + R : c1;
    float x[EPL], lse = 0.f;
    int id[IDS];
    bool live = t < c1 && nlive;
#pragma unroll
    for (int j = 0; j < EPL; ++j) x[j] = live ? nx[j] : -INFINITY;
#pragma unroll
    for (int k = 0; k < IDS; ++k) id[k] = nid[k];
    fetch(t + R);
    live = rows::softmax<L, EPL>(x, lse) && live;
    // the sequences that meet this round; their sums go on into the next one
    // where they do not end here
    while (q.s < p.S && q.a < t1) {
      if (live && t >= q.a && t < q.b) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) acc[j] += x[j];
        if (lane == 0) {
          z2 += double(lse) * double(lse);
          n += 1.f;
        }
#pragma unroll
        for (int k = 0; k < IDS; ++k)
          if (id[k] >= 0 && id[k] < E) atomicAdd(&hist[id[k]], 1);
      }
      const bool ends = q.b <= t1;
      if (!ends ? t1 == c1 : (q.a > c0 ? q.a : c0) < q.b) flush();
      else if (ALL && ends) zeros();   // an empty sequence (it has no record)
      if (!ends) break;
      q.next(p);
    }
  }
  if constexpr (ALL) {
    for (; q.s < p.S; q.next(p)) zeros();   // behind the last token
    __shared__ double red[W];
    for (int o = 1; o < 64; o <<= 1) term += __shfl_xor(term, o, 64);
    if ((threadIdx.x & 63) == 0) red[wave] = term;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < W; ++w) term += red[w];
      write_totals(p, term, term_z, all, live_seqs);
    }
  }
}

// Values that the last workgroup reads from the others: stored and loaded as
// agent-scope atomics, which pass through the XCDs' L2s, and waited for before
// the workgroup counts itself as done.  (Fences would write back and
// invalidate whole L2s: 3 of the kernel's 8 us.)
template <class T>
__device__ __forceinline__ void publish(T* p, T v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <class T>
__device__ __forceinline__ T published(const T* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Grid (S, tiles of kTile experts): thread (q, col) adds every 32nd record of
// its sequence for one expert, so that 512 records are 16 loads in flight.
__global__ void __launch_bounds__(kSumThreads) balance_sum_kernel(BalanceArgs p) {
  constexpr int Q = kSumThreads / kTile, W = kSumThreads / 64;
  static_assert(kTile == 32, "two record groups a wave");
  __shared__ float sp[W][kTile];
  __shared__ double sz[W];
  __shared__ int sc[W][kTile], sn[W];
  __shared__ bool last;
  const bool only = gridDim.x * gridDim.y == 1;
  const int64_t s = blockIdx.x;
  const int tid = threadIdx.x, q = tid / kTile, col = tid % kTile, wave = tid >> 6;
  const int64_t e = int64_t(blockIdx.y) * kTile + col;
  const int64_t a = seq_at(p, s), b = seq_at(p, s + 1);
  const int64_t f = a < b ? a / p.chunk : 0, l = a < b ? (b - 1) / p.chunk : -1;   // its chunks
  float v = 0.f;
  int c = 0;
  if (e < p.E) {
#pragma unroll 8
    for (int64_t k = f + q; k <= l; k += Q) {
      v += p.part_p[(k + s) * p.E + e];
      c += p.part_c[(k + s) * p.E + e];
    }
  }
  int n = 0;
  double z = 0.;
  for (int64_t k = f + tid; k <= l; k += kSumThreads) {
    n += p.part_n[k + s];
    z += p.part_z[k + s];
  }
  v += __shfl_xor(v, 32, 64);
  c += __shfl_xor(c, 32, 64);
  for (int o = 1; o < 64; o <<= 1) {
    n += __shfl_xor(n, o, 64);
    z += __shfl_xor(z, o, 64);
  }
  if ((tid & 63) < kTile) {
    sp[wave][col] = v;
    sc[wave][col] = c;
  }
  if ((tid & 63) == 0) { sn[wave] = n; sz[wave] = z; }
  __syncthreads();
  if (tid < kTile) {
    n = 0;
    z = 0.;
    v = 0.f;
    c = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      v += sp[i][col];
      c += sc[i][col];
      n += sn[i];
      z += sz[i];
    }
    if (e < p.E) p.counts[s * p.E + e] = c;
    // the tile's share of sum_e c_se sum_t p_te / n_s^2
    double d = n > 0 ? double(c) * double(v) / (double(n) * double(n)) : 0.;
    for (int o = 1; o < kTile; o <<= 1) d += __shfl_xor(d, o, 64);
    if (tid == 0 && only) {   // all there is
      p.num[s] = n;
      write_totals(p, d, z, n, n > 0);
    } else if (tid == 0) {
      publish(&p.term[s * gridDim.y + blockIdx.y], d);
      if (blockIdx.y == 0) {
        publish(&p.num[s], n);
        publish(&p.term_z[s], z);
      }
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the published values have reached memory
      last = __hip_atomic_fetch_add(p.done, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x * gridDim.y - 1;
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
  }
  if (only) return;
  __syncthreads();
  if (!last) return;
  // all sequences' terms, in an order that does not depend on who is last
  __shared__ double db[W], dz[W];
  __shared__ int di[W], dl[W];
  double tb = 0., tz = 0.;
  int all = 0, live = 0;
  for (int64_t i = tid; i < p.S * gridDim.y; i += kSumThreads) tb += published(&p.term[i]);
  for (int64_t i = tid; i < p.S; i += kSumThreads) {
    tz += published(&p.term_z[i]);
    const int k = published(&p.num[i]);
    all += k;
    live += k > 0;
  }
  for (int o = 1; o < 64; o <<= 1) {
    tb += __shfl_xor(tb, o, 64);
    tz += __shfl_xor(tz, o, 64);
    all += __shfl_xor(all, o, 64);
    live += __shfl_xor(live, o, 64);
  }
  if ((tid & 63) == 0) { db[wave] = tb; dz[wave] = tz; di[wave] = all; dl[wave] = live; }
  __syncthreads();
  if (tid < W) {
    tb = db[tid]; tz = dz[tid]; all = di[tid]; live = dl[tid];
    for (int o = 1; o < W; o <<= 1) {
      tb += __shfl_xor(tb, o, 64);
      tz += __shfl_xor(tz, o, 64);
      all += __shfl_xor(all, o, 64);
      live += __shfl_xor(live, o, 64);
    }
    if (tid == 0) {
      write_totals(p, tb, tz, all, live);
    }
  }
}

template <int L, int EPL, bool VEC, class LT>
__global__ void __launch_bounds__(kBwdThreads) balance_bwd_kernel(BalanceArgs p) {
  const int lane = threadIdx.x % L, slot = (threadIdx.x & 63) / L;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t0 = int64_t(blockIdx.x) * (kBwdThreads / L) + wave * (64 / L);   // the wave's first row
  if (t0 >= p.T) return;   // whole waves leave
  const bool in = slot < p.T - t0;
  const int E = int(p.E), off = slot * E;   // 32-bit offsets from the wave's rows
  const LT* logits = static_cast<const LT*>(p.logits) + t0 * p.E;
  float* out = p.dlogits + t0 * p.E;
  // the row is under way while its sequence is looked up
  float x[EPL], lse = 0.f;
  bool part = in && (!p.mask || p.mask[t0 + slot] != 0);
  if (in) {
    rows::load<L, EPL, VEC>(logits + off, E, lane, x);
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j) x[j] = -INFINITY;
  }
  const float gb = p.dloss ? p.dloss[0] : 1.f, gz = p.dloss ? p.dloss[1] : 1.f;
  const float live = float(p.num[p.S]), all = float(p.num[p.S + 1]);
  const int64_t s = seq_of_rows<L>(p, t0);
  if (!in) return;
  part = part && s >= 0 && s < p.S;
  const float n = part ? float(p.num[s]) : 1.f;
  part = rows::softmax<L, EPL>(x, lse) && part;
  if (!part) {
    if (!p.accumulate) {
#pragma unroll
      for (int j = 0; j < EPL; ++j) x[j] = 0.f;
      rows::store<L, EPL, VEC>(out + off, E, lane, x);
    }
    return;
  }
  const float rn = rows::rcp_fast(n);
  const float fb = gb * (p.balance_coef * float(p.E) * rows::rcp_fast(live * float(p.K))) * rn * rn;
  const float fz = gz * (2.f * p.z_coef * rows::rcp_fast(all)) * lse;
  const int32_t* counts = p.counts + s * p.E;
  float w[EPL], dot = 0.f;
#pragma unroll
  for (int j = 0; j < EPL; j += 4) {
    const int c = rows::column<L>(lane, j);
    if constexpr (VEC) {
      const int4 k = c < E ? *reinterpret_cast<const int4*>(counts + c) : int4{0, 0, 0, 0};
      w[j] = float(k.x); w[j + 1] = float(k.y); w[j + 2] = float(k.z); w[j + 3] = float(k.w);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) w[j + k] = c + k < E ? float(counts[c + k]) : 0.f;
    }
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    w[j] *= fb;
    dot += w[j] * x[j];
  }
  dot = seg::sum<L>(dot) - fz;
#pragma unroll
  for (int j = 0; j < EPL; ++j) x[j] *= w[j] - dot;
  if (p.accumulate) {
    rows::load<L, EPL, VEC>(static_cast<const float*>(out + off), E, lane, w);
#pragma unroll
    for (int j = 0; j < EPL; ++j) x[j] += w[j];
  }
  rows::store<L, EPL, VEC>(out + off, E, lane, x);
}

// Tokens of one chunk: a round of the workgroup's rows, or as many as keep to
// kChunks chunks; fewer where several sequences would fall into one chunk, as
// each costs its workgroup about 1.5 us of reduction: a sequence's mean length,
// but no less than 4 tokens and no more than 2 kChunks chunks (1000 tokens of 8
// experts in 64 sequences: 60 -> 14 us).
int64_t balance_chunk_tokens(int64_t T, int64_t E, int64_t S) {
  const int64_t r = chunk_threads(E > 512 ? 16 : 8) / rows::lanes(E);
  const int64_t c = (T + kChunks - 1) / kChunks;
  const int64_t most = c <= r ? r : (c + r - 1) / r * r;
  const int64_t least = (T + 2 * kChunks - 1) / (2 * kChunks);
  int64_t few = (T + S - 1) / S;   // the mean
  few = few > least ? few : least;
  few = few > 4 ? few : 4;
  return few < most ? few : most;
}

// One workgroup for everything, in one launch, where the tokens make at most two
// rounds of its rows, in few sequences (each is a reduction of its own): measured with
// 8 experts and 300 tokens 5.9 us against 8.1 in one sequence, 11.0 against 13.0
// in 4, 17.6 against 16.1 in 8; 60 experts and 128 tokens 5.1 against 9.1, 8.9 against 11.1 in 4
// and 14.1 against 11.9 in 8.
static bool balance_one(const BalanceArgs& p) {
  const int64_t round = chunk_threads(p.E > 512 ? 16 : 8) / rows::lanes(p.E);
  return p.T <= 2 * round && p.S <= 4;
}

hipError_t launch_balance_fwd(const BalanceArgs& p, hipStream_t st) {
  const int64_t chunks = (p.T + p.chunk - 1) / p.chunk;
  const bool one = balance_one(p);
  rows::by_experts(p.E, [&](auto L, auto EPL, auto vec) {
    constexpr int threads = chunk_threads(EPL());
    auto go = [&](auto lt, auto all, unsigned grid) {
      balance_chunk_kernel<L(), EPL(), vec(), decltype(lt), all()><<<grid, threads, 0, st>>>(p);
    };
    auto kind = [&](auto lt) {
      if (one) go(lt, std::true_type{}, 1u);
      else go(lt, std::false_type{}, unsigned(chunks > 0 ? chunks : 1));
    };
    if (p.bf16) kind(uint16_t{});
    else kind(float{});
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || one) return e;
  balance_sum_kernel<<<dim3(unsigned(p.S), unsigned((p.E + kTile - 1) / kTile)), kSumThreads, 0, st>>>(p);
  return hipGetLastError();
}

hipError_t launch_balance_bwd(const BalanceArgs& p, hipStream_t st) {
  if (p.T <= 0) return hipSuccess;
  const int64_t r = kBwdThreads / rows::lanes(p.E);
  const unsigned grid = unsigned((p.T + r - 1) / r);
  rows::by_experts(p.E, [&](auto L, auto EPL, auto vec) {
    if (p.bf16) balance_bwd_kernel<L(), EPL(), vec(), uint16_t><<<grid, kBwdThreads, 0, st>>>(p);
    else balance_bwd_kernel<L(), EPL(), vec(), float><<<grid, kBwdThreads, 0, st>>>(p);
  });
  return hipGetLastError();
}

}  // namespace mx
