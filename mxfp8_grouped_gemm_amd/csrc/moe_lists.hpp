// moe_lists.hpp -- one workgroup's part in the MoE backward's block lists: the
// expert lists, or the tile ranges of one GEMM.  Shared by the set-up's kernel
// (moe_aux.hip) and the small layers' gather (quantize.hip).
#pragma once
#include "kernels.hpp"
#include "moe_tiles.hpp"

namespace mx {

// Per-expert lists of occupied blocks in ascending order, for up to MAX blocks
// and experts: one workgroup of MAX threads, a thread per block.  The counts by LDS atomics,
// the offsets by a scan over the experts, and a block's place in its list by
// counting the blocks before it with its expert (N / 4 reads of four at a
// time, the same address in every lane).
// eb: LDS for an occupied block's expert, else -1 (16-byte aligned); cnt, wsum: LDS
template <int MAX>
__device__ __forceinline__ void expert_lists(const int32_t* __restrict__ b2e, const int32_t* __restrict__ flag, int N,
                                             int E, int32_t* __restrict__ off, int32_t* __restrict__ list, int32_t* eb,
                                             int32_t* cnt, int32_t* wsum) {
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  int e = -1;
  if (t < N && flag[t] != 0) e = b2e[t];
  if (e < 0 || e >= E) e = -1;
  eb[t] = e;
  cnt[t] = 0;
  __syncthreads();
  if (e >= 0) atomicAdd(&cnt[e], 1);
  __syncthreads();
  const int c = cnt[t];
  int x = c;
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(x, o, 64);
    if (lane >= o) x += y;
  }
  if (lane == 63) wsum[wave] = x;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < wave; ++w) before += wsum[w];
  const int pos = before + x - c;   // expert t's first entry
  cnt[t] = pos;
  if (t < E) off[t] = pos;
  if (t == E - 1) off[E] = pos + c;
  __syncthreads();
  if (e >= 0) {
    int rank = 0;
    const int4* q = reinterpret_cast<const int4*>(eb);
#pragma unroll 4
    for (int b = 0; b < N; b += 4) {
      const int4 v = q[b >> 2];
      rank += (v.x == e && b < t) + (v.y == e && b + 1 < t) + (v.z == e && b + 2 < t) + (v.w == e && b + 3 < t);
    }
    list[cnt[e] + rank] = t;
  }
}

// tile_ranges_kernel's results for up to MAX blocks, a thread each
template <int MAX>
__device__ __forceinline__ void tile_ranges_of(const int32_t* __restrict__ ext, int N, const TileRangeJob& j, int cmax,
                                               int32_t* wfull, int32_t* wpart) {
  const int b = threadIdx.x, lane = b & 63, wave = b >> 6;
  const int c = b < N ? (ext[b] + j.W - 1) / j.W * j.other : 0;
  const bool full = j.rr && c == cmax;
  int xf = full ? c : 0, xp = full ? 0 : c;
  for (int o = 1; o < 64; o <<= 1) {
    const int yf = __shfl_up(xf, o, 64), yp = __shfl_up(xp, o, 64);
    if (lane >= o) {
      xf += yf;
      xp += yp;
    }
  }
  if (lane == 63) {
    wfull[wave] = xf;
    wpart[wave] = xp;
  }
  __syncthreads();
  int bf = 0, bp = 0, tf = 0, tp = 0;
  for (int w = 0; w < MAX / 64; ++w) {
    bf += w < wave ? wfull[w] : 0;
    bp += w < wave ? wpart[w] : 0;
    tf += wfull[w];
    tp += wpart[w];
  }
  const int total = tf + tp;
  const int t0 = full ? bf + xf - c : tf + bp + xp - c;   // partly filled blocks after the full ones
  if (b < N) {
    j.start[b] = t0;
    int32_t* map = j.start + N + 1;
    for (int t = t0; t < t0 + c; ++t) map[t] = b;
  }
  if (b == 0) {
    j.start[N] = total;
    if (j.cut) {   // the tail cut of each XCD
      int base = 0;
      for (int x = 0; x < 8; ++x) {
        TailCut k = tail_cut_one(total, x, j.rr, j.conc, j.npairs);
        k.base = base;
        base += k.tail * (k.S - 1);
        j.cut[x] = k;
      }
    }
  }
}

inline int full_tiles(const TileRangeJob& j) { return (j.blk + j.W - 1) / j.W * j.other; }   // of a block all live

}  // namespace mx
