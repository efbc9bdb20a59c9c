// moe_fwd_prep.hip -- what the MoE forward makes before its two products.
//
//   fwd_prep_kernel   X along H to codes (rows padded to Hp with zeros, scales
//                     pair-major), both weights' scales pair-major and padded,
//                     and slot_of filled with -1; for a small layer one more
//                     workgroup does the rest as well
//   fwd_slots_kernel  a workgroup per block: its slots' tokens and affinities, the
//                     inverse map and its extent; the last one to finish makes the
//                     tile ranges of the two products (up to kListMax blocks)
//   fwd_ranges_kernel the ranges of more blocks, a workgroup for each product
// X is bound by memory (32768 x 1536: 151 MB read and written in 42 us, 3.6 TB/s);
// the rest is launches and latency (T = 256, E = 4: one launch of 5 us where four of
// 2.5 to 4 us stood).
#include "kernels.hpp"
#include "moe_fwd_plan.hpp"
#include "moe_tiles.hpp"
#include "mx_device.hpp"

namespace mx {

namespace {
constexpr int kThreads = kPrepThreads;
constexpr int kSmallBlocks = int(kSmallSlots / 128);

// ---------------------------------------------------------------------------
// X: a thread takes 8 columns, 4 lanes a group of 32.
// The codes of a lane's 8 columns (its group's other lanes beside it) and their scale.
__device__ __forceinline__ uint2 quant_x8(const uint4& v, int& X) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) m = absmax_bf16x2(m, w[k]);
  m = max(m & 0xffffu, m >> 16);
  m = max(m, uint32_t(__shfl_xor(int(m), 1, 64)));
  m = max(m, uint32_t(__shfl_xor(int(m), 2, 64)));
  X = scale_exp<kE4M3>(m << 16);
  const uint32_t lim = bf16_limit<kE4M3>(X) * 0x10001u;
  const float s = cvt_scale(X);
  return make_uint2(encode_bf16x4<kE4M3>(clamp_bf16x2(w[0], lim), clamp_bf16x2(w[1], lim), s),
                    encode_bf16x4<kE4M3>(clamp_bf16x2(w[2], lim), clamp_bf16x2(w[3], lim), s));
}
template <int TH>
__device__ __forceinline__ void quant_x(const MoeFwdPrep& p, unsigned wg, unsigned wgs) {
  constexpr int U = 4;   // chunks of a thread, their loads issued together
  const uint32_t per = uint32_t(p.Hp / 8), n = uint32_t(p.T) * per, stride = wgs * TH;   // T * Hp < 2^32
  for (uint32_t c0 = wg * TH + threadIdx.x; c0 < n; c0 += U * stride) {
    uint4 v[U];
    uint32_t row[U], col[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t c = c0 + u * stride;
      row[u] = c / per;
      col[u] = (c - row[u] * per) * 8;
      v[u] = make_uint4(0u, 0u, 0u, 0u);
      if (c < n && col[u] < p.H) v[u] = *reinterpret_cast<const uint4*>(p.x + int64_t(row[u]) * p.H + col[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      int X;
      const uint2 q = quant_x8(v[u], X);   // n is a multiple of 16: a group's lanes stay together
      if (c0 + u * stride < n) {
        *reinterpret_cast<uint2*>(p.x_codes + int64_t(row[u]) * p.Hp + col[u]) = q;
        if ((col[u] & 31) == 0)
          p.x_scales[((col[u] >> 7) * p.T + row[u]) * 4 + (col[u] >> 5 & 3)] = col[u] < p.H ? uint8_t(X + 127) : uint8_t(0);
      }
    }
  }
}

__device__ __forceinline__ int64_t valid_tokens(const MoeFwdPrep& p) {
  const int64_t n = p.nvalid ? int64_t(*p.nvalid) : p.T;
  return n < 0 ? 0 : (n < p.T ? n : p.T);
}

// X as slots: each slot's token's row again, codes stage-major over the P slots (zeros in padding).  A
// workgroup takes 32 slots x 256 columns, 2 KB of consecutive codes at a time.
__device__ __forceinline__ void quant_slots(const MoeFwdPrep& p, unsigned id) {
  constexpr int U = 4;
  const unsigned per = unsigned((p.Hp + 255) / 256), g = id / per;
  const int64_t P = p.N * p.B, slot = int64_t(g) * 32 + threadIdx.x / 8, e = p.b2e[slot / p.B], t = p.tpid[slot];
  const bool ok = t >= 0 && t < valid_tokens(p) && e >= 0 && e < p.E;
  const int64_t col0 = int64_t(id - g * per) * 256 + (threadIdx.x & 7) * 8;
  uint4 v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t c = col0 + 64 * u;
    v[u] = ok && c < p.H ? *reinterpret_cast<const uint4*>(p.x + t * p.H + c) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t c = col0 + 64 * u;
    int X;
    const uint2 q = quant_x8(v[u], X);
    if (c < p.Hp) {   // Hp % 128 == 0
      *reinterpret_cast<uint2*>(p.x_codes + stage_major_off(slot, c, P, p.Hp)) = q;
      if ((c & 31) == 0) p.x_scales[((c >> 7) * P + slot) * 4 + (c >> 5 & 3)] = c < p.H ? uint8_t(X + 127) : uint8_t(0);
    }
  }
}

// Weight scales [E][rows][G] -> [E][kp][rows][4], bytes from G on 0: a workgroup
// turns 64 rows x 32 words through LDS.
struct PairsJob {
  const uint8_t* in;
  uint32_t* out;
  int64_t rows, G, kp;
  unsigned gx, gy, n;   // workgroups: along the words, the rows, in all
};
PairsJob pairs_job(const uint8_t* in, uint8_t* out, int64_t E, int64_t rows, int64_t k) {
  PairsJob j{in, reinterpret_cast<uint32_t*>(out), rows, k / 32, (k + 127) / 128, 0, 0, 0};
  j.gx = unsigned((j.kp + 31) / 32);
  j.gy = unsigned((rows + 63) / 64);
  j.n = unsigned(E) * j.gx * j.gy;
  return j;
}
template <int TH>
__device__ __forceinline__ void scale_pairs(const PairsJob& j, unsigned id, uint32_t (*tile)[65]) {
  const unsigned per = j.gx * j.gy, g = id / per, yx = id - g * per, y = yx / j.gx, x = yx - y * j.gx;
  const int64_t p0 = int64_t(x) * 32, r0 = int64_t(y) * 64;
  const uint8_t* src = j.in + g * j.rows * j.G;
  uint32_t* dst = j.out + g * j.rows * j.kp;
#pragma unroll
  for (int k = 0; k < 2048 / TH; ++k) {
    const int i = threadIdx.x + TH * k, r = i >> 5, q = i & 31;
    if (r0 + r < j.rows && p0 + q < j.kp) {
      const uint8_t* s = src + (r0 + r) * j.G + 4 * (p0 + q);
      uint32_t w = 0;
      if (j.G % 4 == 0) {
        w = *reinterpret_cast<const uint32_t*>(s);
      } else {
        const int64_t left = j.G - 4 * (p0 + q);
#pragma unroll
        for (int b = 0; b < 4; ++b) w |= b < left ? uint32_t(s[b]) << (8 * b) : 0u;
      }
      tile[q][r] = w;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2048 / TH; ++k) {
    const int i = threadIdx.x + TH * k, q = i >> 6, r = i & 63;
    if (r0 + r < j.rows && p0 + q < j.kp) dst[(p0 + q) * j.rows + r0 + r] = tile[q][r];
  }
}

// ---------------------------------------------------------------------------
// Tile ranges (moe_tiles.hpp) of any number of blocks by one workgroup of TH
// threads, or (TH = 64) by one wave of any; ext(b): block b's extent.  One pass over the blocks for the totals,
// one for the starts and the map: TH blocks at a time, a block's map entries
// by as many lanes as it has tiles, from starts held in LDS (39 blocks of 448 tiles:
// 12 us less than a thread a block).
template <int TH>
struct RangeLds {
  uint64_t wave[TH / 64];
  int32_t c[TH], start[TH], dead[TH];
};
template <int TH, class Ext>
__device__ __forceinline__ void make_ranges(const Ext& ext, int N, const TileRangeJob& j, RangeLds<TH>& lds) {
  const int tid = TH == 64 ? threadIdx.x & 63 : threadIdx.x;
  auto sync = [] {
    if constexpr (TH == 64) wave_lds_order();
    else __syncthreads();
  };
  const int lane = tid & 63, wave = tid >> 6, cmax = (j.blk + j.W - 1) / j.W * j.other;
  // tiles of fully live blocks (with rr) in the high word, of the others in the low
  auto word = [&](int c) { return j.rr && c == cmax ? uint64_t(c) << 32 : uint64_t(c); };
  auto sum_waves = [&](uint64_t x, uint64_t& before) {   // x: lane 63's is the wave's; returns the sum, before: of earlier waves
    sync();
    if (lane == 63) lds.wave[wave] = x;
    sync();
    uint64_t all = 0;
    before = 0;
    for (int w = 0; w < TH / 64; ++w) {
      const uint64_t s = lds.wave[w];
      before += w < wave ? s : 0;
      all += s;
    }
    return all;
  };
  uint64_t mine = 0, before;
  for (int b = tid; b < N; b += TH) mine += word((ext(b) + j.W - 1) / j.W * j.other);
  for (int o = 32; o > 0; o >>= 1) mine += __shfl_xor(static_cast<unsigned long long>(mine), o, 64);
  const uint64_t sum = sum_waves(mine, before);
  const int nfull = int(sum >> 32), total = nfull + int32_t(sum);
  int32_t* map = j.start + N + 1;
  uint64_t carry = 0;   // of earlier blocks
  for (int b0 = 0; b0 < N; b0 += TH) {
    const int b = b0 + tid, c = b < N ? (ext(b) + j.W - 1) / j.W * j.other : 0;
    uint64_t x = word(c);
    for (int o = 1; o < 64; o <<= 1) {
      const uint64_t y = __shfl_up(static_cast<unsigned long long>(x), o, 64);
      if (lane >= o) x += y;
    }
    const uint64_t chunk = sum_waves(x, before);
    before += carry + x - word(c);
    carry += chunk;
    const int32_t start = j.rr && c == cmax ? int32_t(before >> 32) : nfull + int32_t(before);
    const int32_t dead = total + b * cmax - int32_t(before >> 32) - int32_t(before);
    lds.c[tid] = c;
    lds.start[tid] = start;
    lds.dead[tid] = dead;
    if (b < N) {
      j.start[b] = start;
      if (j.dead) j.dead[b] = dead;
    }
    sync();
    const int L = cmax > 16 ? 64 : cmax > 4 ? 16 : 4, nb = min(TH, N - b0);
    for (int k = tid / L; k < nb; k += TH / L) {
      const int cc = lds.c[k], s = lds.start[k], d = lds.dead[k] - cc;
      for (int t = tid % L; t < (j.dead ? cmax : cc); t += L) map[t < cc ? s + t : d + t] = b0 + k;
    }
  }
  if (tid == 0) j.start[N] = total;
  if (j.cut && tid < 8) {   // the tail cut of each XCD
    TailCut k = tail_cut_one(total, tid, j.rr, j.conc, j.npairs);
    const int mineb = k.tail * (k.S - 1);
    int base = mineb;
    for (int o = 1; o < 8; o <<= 1) {
      const int y = __shfl_up(base, o, 8);
      if (tid >= o) base += y;
    }
    k.base = base - mineb;
    j.cut[tid] = k;
  }
}

// Four slots s + k step below end (in a block of expert(s)): tokens and
// affinities (padding: -1, 0), the inverse map; routed(s) for each that has a token.
// Padding is what holds no token below the count of valid ones, or lies in a block
// of no expert.  The four's loads are issued together.
template <class Expert, class Routed>
__device__ __forceinline__ void put_slots(const MoeFwdPrep& p, int64_t s0, int64_t step, int64_t end, int64_t Tv,
                                          const Expert& expert, const Routed& routed) {
  int64_t t[4], e[4];
  float a[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t s = s0 + k * step;
    t[k] = s < end ? int64_t(p.tpid[s]) : -1;
    e[k] = s < end ? expert(s) : -1;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (t[k] >= Tv || e[k] < 0 || e[k] >= p.E) t[k] = -1;
    a[k] = t[k] >= 0 ? p.aff[t[k] * p.E + e[k]] : 0.f;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t s = s0 + k * step;
    if (s >= end) continue;
    p.slot_tok[s] = t[k] >= 0 ? int32_t(t[k]) : -1;
    p.slot_aff[s] = a[k];
    if (t[k] >= 0) {
      p.slot_of[t[k] * p.E + e[k]] = int32_t(s);
      routed(s);
    }
  }
}
// SMALL: workgroup 0 does the whole set-up of the slots.
template <bool SMALL>
__global__ void __launch_bounds__(SMALL ? kSmallThreads : kThreads) fwd_prep_kernel(MoeFwdPrep p, PairsJob j0, PairsJob j1,
                                                                                         unsigned nq) {
  constexpr int TH = SMALL ? kSmallThreads : kThreads;
  __shared__ uint32_t tile[32][65];
  const unsigned wg = blockIdx.x;
  if constexpr (SMALL) {
    if (wg == 0) {
      __shared__ int ext[kSmallBlocks];
      __shared__ RangeLds<64> lds[2];
      for (int64_t k = threadIdx.x; k < p.T * p.E; k += TH) p.slot_of[k] = -1;
      for (int b = threadIdx.x; b < p.N; b += TH) ext[b] = 0;
      __syncthreads();
      const int64_t Tv = valid_tokens(p);
      const int P = int(p.N * p.B), B = int(p.B);
      for (int s = threadIdx.x; s < P; s += 4 * TH)
        put_slots(p, s, TH, P, Tv, [&](int64_t q) { return int64_t(p.b2e[int(q) / B]); },
                  [&](int64_t q) { atomicMax(&ext[int(q) / B], int(q) % B + 1); });
      __syncthreads();
      for (int b = threadIdx.x; b < p.N; b += TH) p.flag[b] = ext[b];
      const int w = threadIdx.x >> 6;   // a wave for each product
      if (w < 2) make_ranges<64>([&](int b) { return ext[b]; }, int(p.N), p.jobs[w], lds[w]);
      return;
    }
  }
  unsigned id = wg - (SMALL ? 1 : 0);
  if (id == 0 && threadIdx.x == 0) *p.done = 0;   // read by the next launch only
  if (id < nq) {
    if (!SMALL && p.x_by_slot) return quant_slots(p, id);
    quant_x<TH>(p, id, nq);
    return;
  }
  id -= nq;
  if (id < j0.n) {
    scale_pairs<TH>(j0, id, tile);
    return;
  }
  id -= j0.n;
  if (id < j1.n) {
    scale_pairs<TH>(j1, id, tile);
    return;
  }
  id -= j1.n;
  const int64_t n = p.T * p.E, i = (int64_t(id) * TH + threadIdx.x) * 4;
  if (i + 4 <= n) {
    *reinterpret_cast<int4*>(p.slot_of + i) = int4{-1, -1, -1, -1};
  } else {
    for (int64_t k = i; k < n; ++k) p.slot_of[k] = -1;
  }
}

__global__ void __launch_bounds__(kThreads) fwd_slots_kernel(MoeFwdPrep p, int ranges) {
  __shared__ int red[kThreads / 64], exts[kListMax];
  __shared__ RangeLds<kThreads> lds;
  __shared__ int last;
  const int b = blockIdx.x;
  const int64_t Tv = valid_tokens(p), e = p.b2e[b];
  int ext = 0;
  const int64_t first = int64_t(b) * p.B;
  for (int64_t s = first + threadIdx.x; s < first + p.B; s += 4 * kThreads)   // ascending per thread
    put_slots(p, s, kThreads, first + p.B, Tv, [&](int64_t) { return e; }, [&](int64_t q) { ext = int(q - first) + 1; });
  for (int o = 32; o > 0; o >>= 1) ext = max(ext, __shfl_xor(ext, o, 64));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = ext;
  __syncthreads();
  if (threadIdx.x == 0) {
    ext = max(max(red[0], red[1]), max(red[2], red[3]));
    if (ranges) {   // published at agent scope: the last workgroup reads all of them
      __hip_atomic_store(p.flag + b, ext, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      last = __hip_atomic_fetch_add(p.done, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
    } else {
      p.flag[b] = ext;
    }
  }
  if (!ranges) return;
  __syncthreads();
  if (!last) return;
  for (int q = threadIdx.x; q < p.N; q += kThreads)   // N <= kListMax
    exts[q] = __hip_atomic_load(p.flag + q, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  for (int k = 0; k < 2; ++k) make_ranges<kThreads>([&](int q) { return exts[q]; }, int(p.N), p.jobs[k], lds);
}

constexpr int kRangeThreads = 1024;
__global__ void __launch_bounds__(kRangeThreads) fwd_ranges_kernel(MoeFwdPrep p) {
  __shared__ RangeLds<kRangeThreads> lds;
  make_ranges<kRangeThreads>([&](int b) { return p.flag[b]; }, int(p.N), p.jobs[blockIdx.x], lds);
}
}  // namespace

hipError_t launch_fwd_prep(const MoeFwdPrep& p, hipStream_t st) {
  const FwdPrepPlan plan = fwd_prep_plan(p.T, p.H, p.I, p.E, p.N, p.B, p.x_by_slot);
  if (plan.grid > kMaxLaunchThreads / plan.threads) return hipErrorInvalidValue;
  const PairsJob j0 = pairs_job(p.wgu_scales, p.wgu_pairs, p.E, 2 * p.I, p.H);
  const PairsJob j1 = pairs_job(p.wd_scales, p.wd_pairs, p.E, p.H, p.I);
  const unsigned grid = unsigned(plan.grid), nq = unsigned(plan.nq);
  if (plan.small) {
    fwd_prep_kernel<true><<<grid, kSmallThreads, 0, st>>>(p, j0, j1, nq);
  } else {
    fwd_prep_kernel<false><<<grid, kThreads, 0, st>>>(p, j0, j1, nq);
    const bool ranges = p.N <= kListMax;
    fwd_slots_kernel<<<unsigned(p.N), kThreads, 0, st>>>(p, ranges ? 1 : 0);
    if (!ranges) fwd_ranges_kernel<<<2, kRangeThreads, 0, st>>>(p);
  }
  return hipGetLastError();
}

}  // namespace mx
