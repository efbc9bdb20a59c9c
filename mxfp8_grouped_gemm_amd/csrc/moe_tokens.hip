// moe_tokens.hip -- the MoE forward for few tokens (decoding): the layer of
// moe_fwd.hip straight from the router's selections, without block lists.
//
// Bound by the bytes of the selected experts' weights: an expert has a handful
// of rows, so a product is a stream of weights past a few columns.  They are read
// once where an expert has no more pairs than a workgroup has columns (`columns`:
// 32, or 64 from an average of 16 on), and once more for every further so many.
// Selections ("pairs" t * K + k) keep their index as row of every
// intermediate.  A tile is 64 weight rows of one expert (32 gate rows and the
// same 32 up rows; or 64 rows of the down projection) times up to NCOL of the
// expert's pairs.  Each wave streams whole 128-byte lines of weight rows
// straight to an LDS ring of its own (no barrier in the loop), scales and the
// columns' codes with them, and either
//   KS = 1: walks whole tiles, the ring running on from one to the next, or
//   KS = 4: shares one tile's contraction with the workgroup's other waves
//           (and, in the down projection, with other workgroups): where there
//           are too few tiles to fill the CUs.
// Up to kFewTokens tokens, a workgroup finds its expert's pairs by scanning the
// ids and quantises X as it reads it, and the last workgroup to finish a tile of
// the down projection adds up the splits and selections: two launches.  More
// tokens: a launch before that lists the pairs by expert and quantises X, and
// one after that adds up.
// Measured: T = 1, two experts of H = 4096, I = 14336: 51 + 26 us, 4.7 TB/s of weights;
// T = 200 over 128 experts of H = 1536, I = 256: 5 + 37 + 21 + 7 us, 2.7 TB/s in the
// products, where each workgroup's 393 KB leave no time to hide the chain before its
// first load (5 us) or its epilogue; T = 1, eight of those: 9.3 + 9.6 us, all latency.
#include <type_traits>

#include "gemm_v4.hpp"
#include "kernels.hpp"
#include "mx_device.hpp"
#include "swiglu.hpp"

namespace mx {

namespace {
using v2::v16f;
constexpr int kWaves = 4;
constexpr int kRows = 64;                    // weight rows of a tile
constexpr int kStagePitch = 36;              // words a row of the waves' sums
constexpr int kStageBytes = kWaves * kRows * kStagePitch * 4;
constexpr int kFewTokens = 4;                // NCOL of the two-launch form, whose columns are bf16 X

template <int NCOL, bool BF16X>
struct TokLds {
  // pairs (128 bytes of K) in a wave's ring: as many as LDS holds, with two workgroups on a CU up to 8 columns
  static constexpr int SLOTS = NCOL == 32 ? 3 : 2;
  static constexpr int A = kRows * 128, B = NCOL * (BF16X ? 256 : 128);
  static constexpr int SLOT = A + B + 256 + (BF16X ? 0 : 256);   // then a scale word a row (and a column)
  static constexpr int RING = kWaves * SLOTS * SLOT;
  static constexpr int BYTES = RING > kStageBytes ? RING : kStageBytes;
};

// 16 bytes a lane into LDS at m0 + 16 * lane, past the caches' reuse: weights are
// read once a call (240 MB of them 46 us with the hint, 53 without, as plain loads).
__device__ __forceinline__ void dma16_once(const v3::v4i& rs, uint32_t lds, uint32_t voff, uint32_t soff) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, %3 offen nt lds"
               :
               : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(voff), "s"(rs),
                 "s"(__builtin_amdgcn_readfirstlane(soff))
               : "memory");
#endif
}

// What a workgroup works on: expert e, and n, how many columns from c0 on.
struct Unit {
  int e, n;
};
// From the lists (launch_tok_prep): unit blockIdx.y is an expert's run of up to NCOL pairs.
template <int NCOL>
__device__ __forceinline__ Unit tok_unit_listed(const MoeTokensArgs& p, int32_t* cols) {
  const int u = blockIdx.y;
  const int nu = p.units[0];
  const int e = p.units[1 + 3 * u], lo = p.units[2 + 3 * u], n = p.units[3 + 3 * u];
  if (u >= nu) return Unit{0, 0};   // entries behind nu are not written, and not used
  if (int(threadIdx.x) < n) cols[threadIdx.x] = p.list[lo + threadIdx.x];   // n <= NCOL
  __syncthreads();
  return Unit{e, n};
}
// By scanning the ids (T <= kFewTokens).  A unit is an expert, or, where there
// are fewer pairs than experts, a pair, which stands for its expert if it is the
// first to select it (n = 0 if not).
template <int NCOL>
__device__ __forceinline__ Unit tok_unit_scanned(const MoeTokensArgs& p, int c0, int32_t* cols, int* cnt) {
  const int M = int(p.T * p.K), lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  static_assert(kFewTokens * 32 <= 64 * kWaves, "a pair a lane (K <= 32)");
  const int u = blockIdx.y, j = threadIdx.x;
  const int e = p.by_pair ? p.idx[u] : u;
  const int id = j < M ? p.idx[j] : -1;
  if (e < 0 || e >= p.E) return Unit{0, 0};
  const uint64_t mask = __ballot(id == e);
  if (lane == 0) cnt[wave] = __popcll(mask);
  if (j == u) cnt[kWaves] = __popcll(mask & ((uint64_t(1) << lane) - 1));   // u's rank in its wave
  __syncthreads();
  int rank = __popcll(mask & ((uint64_t(1) << lane) - 1)), n = 0, before = cnt[kWaves];
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    rank += w < wave ? cnt[w] : 0;
    before += w < (u >> 6) ? cnt[w] : 0;
    n += cnt[w];
  }
  if (p.by_pair && before > 0) return Unit{0, 0};
  if (id == e && rank >= c0 && rank < c0 + NCOL) cols[rank - c0] = j;
  __syncthreads();
  return Unit{e, n};
}
template <int NCOL, bool SCAN>
__device__ __forceinline__ Unit tok_unit(const MoeTokensArgs& p, int c0, int32_t* cols, int* cnt) {
  if constexpr (SCAN) return tok_unit_scanned<NCOL>(p, c0, cols, cnt);
  else return c0 == 0 ? tok_unit_listed<NCOL>(p, cols) : Unit{0, 0};
}

// 16 bf16 of a group of 32, the other 16 in the lane 32 away, as E4M3 codes;
// returns the scale byte.
__device__ __forceinline__ uint32_t tok_quantise(const uint4 (&v)[2], uint4& codes) {
  const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) m = absmax_bf16x2(m, w[k]);
  m = max(m & 0xffffu, m >> 16);
#if defined(__HIP_DEVICE_COMPILE__)
  {
    const auto x = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    m = max(uint32_t(x[0]), uint32_t(x[1]));
  }
#endif
  const int X = scale_exp<kE4M3>(m << 16);
  const uint32_t lim = bf16_limit<kE4M3>(X) * 0x10001u;
  const float s = cvt_scale(X);
  uint32_t c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    c[k] = encode_bf16x4<kE4M3>(clamp_bf16x2(w[2 * k], lim), clamp_bf16x2(w[2 * k + 1], lim), s);
  codes = make_uint4(c[0], c[1], c[2], c[3]);
  return uint32_t(X + 127);
}

// A wave's stream: nk pairs (first, first + step, ..) of K elements of each of
// ntiles tiles.  w, ws: the expert's codes and scales, rows of K bytes (wrows of
// them); row(q), q < 64: tile 0's source rows; tile t's lie t * trows further
// down.  x, xs: the columns' codes and scales, or bf16 rows (BF16X), col(q): source
// row or -1.  done(t, acc) takes a tile's sums.  EXACT: on the bf16 MFMA, from the
// codes' exact values: the gate/up sums are rounded to codes again, and the scaled
// MFMA's truncation of small products would move some of those to a neighbour, once
// in some ten thousand groups a scale, which a call of a few hundred groups shows in
// full (y 0.0047 off the formula where its rounding to bf16 is 0.0017).  The stream
// of weights hides the difference.
template <int NCOL, bool GENERIC, bool BF16X, bool EXACT>
struct TokLoop {
  static constexpr int FN = NCOL <= 32 ? 1 : 2;
  static constexpr int XB = BF16X ? 2 : 1;                                     // bytes an element of the columns
  static constexpr int NA = kRows / 8, NB = (NCOL * XB + 7) / 8;               // DMA instructions of 1 KB
  static constexpr int PER = NA + NB + (GENERIC ? 0 : BF16X ? 1 : 2);          // of a pair
  static_assert(!BF16X || NCOL == 4, "one instruction: 4 rows of 256 bytes");
  using L = TokLds<NCOL, BF16X>;
  static constexpr int S = L::SLOTS;

  template <class Row, class Col, class Done>
  __device__ __forceinline__ static void run(const uint8_t* w, const uint8_t* ws, int64_t wrows, const void* x,
                                             const uint8_t* xs, int64_t xrows, int K, int first, int step, int nk,
                                             int ntiles, int64_t trows, uint8_t* ring, const Row& row, const Col& col,
                                             const Done& done) {
#if defined(__HIP_DEVICE_COMPILE__)
    const int lane = threadIdx.x & 63, h = lane >> 5, r = lane & 31, G = K / 32;
    const v3::v4i rw = v3::rsrc(v2::make_rsrc(w, uint32_t(wrows * K)));
    const v3::v4i rx = v3::rsrc(v2::make_rsrc(x, uint32_t(xrows * K * XB)));
    const v3::v4i rws = v3::rsrc(v2::make_rsrc(ws, uint32_t(wrows * G)));
    const v3::v4i rxs = v3::rsrc(v2::make_rsrc(xs, uint32_t(BF16X ? 0 : xrows * G)));
    uint32_t offa[NA], offb[NB], offs[2];
#pragma unroll
    for (int j = 0; j < NA; ++j) {   // LDS row q: lane l fills its physical chunk l & 7
      const int q = 8 * j + (lane >> 3);
      offa[j] = uint32_t(row(q) * K + 16 * ((lane & 7) ^ v4::swz(q)));
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int q = BF16X ? lane >> 4 : 8 * j + (lane >> 3);
      const int64_t src = q < NCOL ? col(q) : -1;
      const int c = BF16X ? (lane & 15) ^ (q << 2) : (lane & 7) ^ v4::swz(q);
      offb[j] = src >= 0 ? uint32_t(src * K * XB + 16 * c) : v3::kOOB;
    }
    {
      const int64_t b = !BF16X && lane < NCOL ? col(lane) : -1;
      offs[0] = uint32_t(row(lane) * G);
      offs[1] = b >= 0 ? uint32_t(b * G) : v3::kOOB;
    }
    const uint32_t base = v3::lds_addr(ring);
    const int total = nk * ntiles;
    // the next pair to load: n-th of all, pair iu of tile it
    int in = 0, iu = 0, it = 0;
    uint32_t islot = 0;
    auto issue = [&]() {
      const bool live = in < total;
      const uint32_t u = uint32_t(first + iu * step);
      const uint32_t kc = live ? u * 128u : 0u, slot = base + islot * L::SLOT;
      const uint32_t trow = live ? uint32_t(it * trows) : 0u;
      v3::v4i ra = rw, rb = rx, rc = rws, rd = rxs;   // past the end: no records, zeros without memory traffic
      ra[2] = live ? ra[2] : 0;
      rb[2] = live ? rb[2] : 0;
      rc[2] = live ? rc[2] : 0;
      rd[2] = live ? rd[2] : 0;
      // a ragged last pair: chunks past K read as zeros (K % 32 == 0: whole chunks)
#pragma unroll
      for (int j = 0; j < NA; ++j) {
        uint32_t off = offa[j] + trow * uint32_t(K);   // rows past the expert's lie past the descriptor's end
        if (GENERIC && int(kc) + 16 * ((lane & 7) ^ v4::swz(8 * j + (lane >> 3))) >= K) off = v3::kOOB;
        dma16_once(ra, slot + j * 1024u, off, kc);
      }
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        uint32_t off = offb[j];
        const int c = BF16X ? ((lane & 15) ^ (lane >> 4 << 2)) >> 1 : (lane & 7) ^ v4::swz(8 * j + (lane >> 3));
        if (GENERIC && int(kc) + 16 * c >= K) off = v3::kOOB;
        v3::dma16(rb, slot + L::A + j * 1024u, off, kc * XB);
      }
      if constexpr (!GENERIC) {
        v3::dma4(rc, slot + L::A + L::B, offs[0] + trow * uint32_t(G), kc >> 5);
        if constexpr (!BF16X) v3::dma4(rd, slot + L::A + L::B + 256, offs[1], kc >> 5);
      }
      ++in;
      islot = islot + 1 == S ? 0 : islot + 1;
      if (++iu == nk) {
        iu = 0;
        ++it;
      }
    };
#pragma unroll
    for (int k = 0; k < S; ++k) issue();
    int at = 0;   // slot of the next pair to use
    for (int t = 0; t < ntiles; ++t) {
      v16f acc[2][FN];
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int q = 0; q < 16; ++q) acc[f][j][q] = 0.f;
      for (int i = 0; i < nk; ++i) {
        const uint8_t* slot = ring + at * L::SLOT;
        at = at + 1 == S ? 0 : at + 1;
        // this pair has landed once only the later ones' loads remain
        asm volatile("s_waitcnt vmcnt(%0)" : : "n"((S - 1) * PER) : "memory");
        __builtin_amdgcn_sched_barrier(0);
        uint4 fa[2][2][2], fb[2][FN][2];   // [stage][fragment][chunk]
        uint4 xv[2][2][2];                 // BF16X: [stage][chunk], 32 bytes each
        uint32_t sa[2], sb[FN];
#pragma unroll
        for (int P = 0; P < 2; ++P) {
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const int q = 32 * f + r;
#pragma unroll
            for (int c = 0; c < 2; ++c)
              fa[P][f][c] = *reinterpret_cast<const uint4*>(slot + q * 128 + 16 * ((4 * P + 2 * c + h) ^ v4::swz(q)));
          }
          // columns past NCOL repeat, and are not used
          if constexpr (BF16X) {
            const int q = r % NCOL;
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int b = 0; b < 2; ++b)
                xv[P][c][b] = *reinterpret_cast<const uint4*>(slot + L::A + q * 256 +
                                                              16 * ((2 * (4 * P + 2 * c + h) + b) ^ (q << 2)));
          } else {
#pragma unroll
            for (int j = 0; j < FN; ++j) {
              const int q = NCOL < 32 ? r % NCOL : 32 * j + r;
#pragma unroll
              for (int c = 0; c < 2; ++c)
                fb[P][j][c] = *reinterpret_cast<const uint4*>(slot + L::A + q * 128 + 16 * ((4 * P + 2 * c + h) ^ v4::swz(q)));
            }
          }
        }
        const uint32_t* sc = reinterpret_cast<const uint32_t*>(slot + L::A + L::B);
        if constexpr (!GENERIC) {
#pragma unroll
          for (int f = 0; f < 2; ++f) sa[f] = sc[32 * f + r];
          if constexpr (!BF16X) {
#pragma unroll
            for (int j = 0; j < FN; ++j) sb[j] = sc[64 + (NCOL < 32 ? r % NCOL : 32 * j + r)];
          }
        } else {
          // scale rows that are not whole words: byte by byte, groups past K as 0
          const int u4 = 4 * (first + i * step);
          auto word = [&](const uint8_t* s, int64_t src) -> uint32_t {
            uint32_t v = 0;
            if (src >= 0)
              for (int g = 0; g < 4; ++g)
                if (u4 + g < G) v |= uint32_t(s[src * G + u4 + g]) << (8 * g);
            return v;
          };
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const int64_t src = row(32 * f + r) + t * trows;
            sa[f] = word(ws, src < wrows ? src : -1);
          }
          if constexpr (!BF16X) {
#pragma unroll
            for (int j = 0; j < FN; ++j) sb[j] = word(xs, col(NCOL < 32 ? r % NCOL : 32 * j + r));
          }
        }
        // every read of the slot is back before its next pair is loaded
        asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
        __builtin_amdgcn_sched_barrier(0);
        issue();
        if constexpr (BF16X) {
          sb[0] = 0;
#pragma unroll
          for (int P = 0; P < 2; ++P)
#pragma unroll
            for (int c = 0; c < 2; ++c) sb[0] |= tok_quantise(xv[P][c], fb[P][0][c]) << (8 * (2 * P + c));
        }
        v2::static_for<2>([&](auto P) {
          v2::static_for<2>([&](auto F) {
            v2::static_for<FN>([&](auto J) {
              if constexpr (EXACT) {
                using R = v3::Ring<128, 128, v3::kFp8Bf16, kE4M3, kE4M3, v3::KMapPlain>;
                v2::static_for<4>([&](auto C) {   // 16 columns each
                  acc[F][J] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(R::template step_operand<kE4M3, P, C>(fa[P][F], sa[F]),
                                                                      R::template step_operand<kE4M3, P, C>(fb[P][J], sb[J]),
                                                                      acc[F][J], 0, 0, 0);
                });
              } else {
                acc[F][J] = v3::mma<kE4M3, kE4M3, 2 * int(P)>(fa[P][F], fb[P][J], acc[F][J], int(sa[F] >> (8 * h)),
                                                              int(sb[J] >> (8 * h)));
              }
            });
          });
        });
      }
      done(t, acc);
    }
    asm volatile("s_waitcnt vmcnt(0)" : : : "memory");   // the loads past the end have landed too
#endif
  }
};

// Wave's sums of fragment column J to LDS: word [wave][row][column].
template <int FN>
__device__ __forceinline__ void tok_stage(float* st, const v16f (&acc)[2][FN], int J) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = lane >> 5, r = lane & 31;
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int q = 0; q < 16; ++q)
      st[(wave * kRows + 32 * f + 8 * (q >> 2) + 4 * h + (q & 3)) * kStagePitch + r] = acc[f][J][q];
}
__device__ __forceinline__ float tok_sum(const float* st, int row, int c) {
  float v = st[row * kStagePitch + c];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) v += st[(w * kRows + row) * kStagePitch + c];
  return v;
}
__device__ __forceinline__ float tok_act(bool geglu, float g) { return geglu ? gate_act<true>(g) : gate_act<false>(g); }

// Values that another workgroup of the same launch reads: stores and loads at
// agent scope (fences would write back whole L2s).
__device__ __forceinline__ void publish(float* p, float v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float published(const float* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <int NCOL, bool GENERIC, int KS>
__global__ void __launch_bounds__(64 * kWaves) tok_gate_up_kernel(MoeTokensArgs p) {
  constexpr bool FEW = NCOL == kFewTokens;
  using Loop = TokLoop<NCOL, GENERIC, FEW, true>;
  using L = TokLds<NCOL, FEW>;
  constexpr int FN = Loop::FN;
  __shared__ __attribute__((aligned(16))) uint8_t smem[L::BYTES];
  __shared__ int32_t cols[NCOL];
  __shared__ int cnt[kWaves + 1];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);   // uniform: descriptors stay scalar
  const int lane = threadIdx.x & 63, h = lane >> 5, r = lane & 31;
  // the counts of finished workgroups that the next launch uses start at 0
  if (FEW && blockIdx.y == 0)
    for (int64_t k = blockIdx.x * 256 + threadIdx.x; k < (p.H + kRows - 1) / kRows; k += gridDim.x * 256) p.done[k] = 0;
  const int np = int((p.H + 127) / 128), tiles = int(p.I / 32);   // I % 32 == 0
  const int t0 = KS == 1 ? int(blockIdx.x) * kWaves + wave : int(blockIdx.x);
  const int tstep = KS == 1 ? int(gridDim.x) * kWaves : tiles;
  const int nt = t0 < tiles ? (tiles - t0 + tstep - 1) / tstep : 0;
  for (int c0 = 0;; c0 += NCOL) {
    const Unit un = tok_unit<NCOL, FEW>(p, c0, cols, cnt);
    if (c0 >= un.n) return;
    const int64_t e = un.e;
    const int nc = un.n - c0 < NCOL ? un.n - c0 : NCOL;
    const int first = KS == 1 ? 0 : wave, step = KS == 1 ? 1 : kWaves;
    // KS = 4: what the one tile's epilogue needs, loaded ahead of the stream
    uint2 bias_g = make_uint2(0u, 0u), bias_u = bias_g;
    float score[FN];
    if constexpr (KS == 4) {
      const int c = threadIdx.x >> 3, k = threadIdx.x & 7;
      if (p.b1) {
        const uint16_t* b = p.b1 + e * 2 * p.I + int64_t(t0) * 32 + 4 * k;
        bias_g = *reinterpret_cast<const uint2*>(b);
        bias_u = *reinterpret_cast<const uint2*>(b + p.I);
      }
#pragma unroll
      for (int J = 0; J < FN; ++J) score[J] = p.on_i && 32 * J + c < nc ? p.scores[cols[32 * J + c]] : 1.f;
    }
    Loop::run(
        p.w_codes + e * 2 * p.I * p.H, p.w_scales + e * 2 * p.I * (p.H / 32), 2 * p.I,
        FEW ? static_cast<const void*>(p.x) : p.x_codes, p.x_scales, p.T, int(p.H), first, step,
        np > first ? (np - first + step - 1) / step : 0, nt, int64_t(tstep) * 32, smem + wave * L::SLOTS * L::SLOT,
        [&](int q) -> int64_t { return (q >> 5) * p.I + int64_t(t0) * 32 + (q & 31); },
        [&](int q) -> int64_t { return q < nc ? cols[q] / int(p.K) : -1; },
        [&](int t, const v16f (&acc)[2][FN]) {
          const int64_t i0 = (t0 + int64_t(t) * tstep) * 32;
          if constexpr (KS == 1) {
            const uint16_t* b1 = p.b1 ? p.b1 + e * 2 * p.I + i0 : nullptr;
            // a lane holds gate and up of 16 of the 32 i, the lane 32 away the rest
            float bg[16], bu[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) bg[q] = bu[q] = 0.f;
            if (b1) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint2 g = *reinterpret_cast<const uint2*>(b1 + 4 * h + 8 * k);
                const uint2 u = *reinterpret_cast<const uint2*>(b1 + p.I + 4 * h + 8 * k);
                bg[4 * k] = lo_bf16(g.x); bg[4 * k + 1] = hi_bf16(g.x); bg[4 * k + 2] = lo_bf16(g.y); bg[4 * k + 3] = hi_bf16(g.y);
                bu[4 * k] = lo_bf16(u.x); bu[4 * k + 1] = hi_bf16(u.x); bu[4 * k + 2] = lo_bf16(u.y); bu[4 * k + 3] = hi_bf16(u.y);
              }
            }
#pragma unroll
            for (int J = 0; J < FN; ++J) {
              const bool in = 32 * J + r < nc;
              const int64_t pair = in ? cols[32 * J + r] : 0;
              const float a = p.on_i && in ? p.scores[pair] : 1.f;
              float v[16];
              uint32_t m = 0;
#pragma unroll
              for (int q = 0; q < 16; ++q) {
                v[q] = tok_act(p.geglu, acc[0][J][q] + bg[q]) * (acc[1][J][q] + bu[q]) * a;
                m = max(m, abs_bits(v[q]));
              }
#if defined(__HIP_DEVICE_COMPILE__)
              {
                const auto x = __builtin_amdgcn_permlane32_swap(m, m, false, false);
                m = max(uint32_t(x[0]), uint32_t(x[1]));
              }
              const int X = scale_exp<kE4M3>(m);
              const float inv = inv_scale(X);
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) w[k] = encode4<kE4M3>(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3], inv);
              // word k of half h: rows 8k + 4h .. + 3.  Half 0 takes rows 0..15, half 1 rows 16..31.
              const auto x = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
              const auto y = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
              if (in) {
                *reinterpret_cast<uint4*>(p.s_codes + pair * p.I + i0 + 16 * h) = make_uint4(x[0], x[1], y[0], y[1]);
                if (h == 0) p.s_scales[pair * (p.I / 32) + i0 / 32] = uint8_t(X + 127);
              }
#endif
            }
          } else {
            float* st = reinterpret_cast<float*>(smem);
#pragma unroll
            for (int J = 0; J < FN; ++J) {
#if defined(__HIP_DEVICE_COMPILE__)
              asm volatile("s_waitcnt vmcnt(0)" : : : "memory");   // this wave's ring is quiet
#endif
              __syncthreads();   // the rings, or the previous columns, are done with
              tok_stage<FN>(st, acc, J);
              __syncthreads();
              // thread: column c, rows 4 k .. + 3
              const int c = threadIdx.x >> 3, k = threadIdx.x & 7;
              if (32 * J + c < nc) {
                const int64_t pair = cols[32 * J + c];
                const float bg[4] = {lo_bf16(bias_g.x), hi_bf16(bias_g.x), lo_bf16(bias_g.y), hi_bf16(bias_g.y)};
                const float bu[4] = {lo_bf16(bias_u.x), hi_bf16(bias_u.x), lo_bf16(bias_u.y), hi_bf16(bias_u.y)};
                float v[4];
                uint32_t m = 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  const float g = tok_sum(st, 4 * k + q, c) + bg[q], u = tok_sum(st, 32 + 4 * k + q, c) + bu[q];
                  v[q] = tok_act(p.geglu, g) * u * score[J];
                  m = max(m, abs_bits(v[q]));
                }
                m = max(m, uint32_t(__shfl_xor(int(m), 1, 64)));
                m = max(m, uint32_t(__shfl_xor(int(m), 2, 64)));
                m = max(m, uint32_t(__shfl_xor(int(m), 4, 64)));
                const int X = scale_exp<kE4M3>(m);
                *reinterpret_cast<uint32_t*>(p.s_codes + pair * p.I + i0 + 4 * k) =
                    encode4<kE4M3>(v[0], v[1], v[2], v[3], inv_scale(X));
                if (k == 0) p.s_scales[pair * (p.I / 32) + i0 / 32] = uint8_t(X + 127);
              }
            }
          }
        });
    __syncthreads();   // the columns and the staging are rewritten
  }
}

// LAST (few tokens, KS = 4): the workgroup that finishes a tile last adds up
// the tile's splits and selections, in order, and writes the result.
template <int NCOL, bool GENERIC, int KS>
__global__ void __launch_bounds__(64 * kWaves) tok_down_kernel(MoeTokensArgs p) {
  constexpr bool FEW = NCOL == kFewTokens, LAST = FEW && KS == 4;
  using Loop = TokLoop<(NCOL < 8 ? 8 : NCOL), GENERIC, false, false>;
  using L = TokLds<(NCOL < 8 ? 8 : NCOL), false>;
  constexpr int FN = Loop::FN;
  __shared__ __attribute__((aligned(16))) uint8_t smem[L::BYTES];
  __shared__ int32_t cols[NCOL];
  __shared__ int cnt[kWaves + 1];
  __shared__ int last, ids[LAST ? kFewTokens * 32 : 1];
  __shared__ float scores[LAST ? kFewTokens * 32 : 1];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, h = lane >> 5, r = lane & 31;
  const int64_t M = p.T * p.K;
  if (LAST && threadIdx.x < M) {   // for the last sum; a dropped selection: -1
    const int e = p.idx[threadIdx.x];
    ids[threadIdx.x] = e >= 0 && e < p.E ? e : -1;
    scores[threadIdx.x] = p.on_i ? 1.f : p.scores[threadIdx.x];
  }
  const int np = int((p.I + 127) / 128), tiles = int((p.H + kRows - 1) / kRows);
  const int t0 = KS == 1 ? int(blockIdx.x) * kWaves + wave : int(blockIdx.x);
  const int tstep = KS == 1 ? int(gridDim.x) * kWaves : tiles;
  const int nt = t0 < tiles ? (tiles - t0 + tstep - 1) / tstep : 0;
  for (int c0 = 0;; c0 += NCOL) {
    const Unit un = tok_unit<NCOL, FEW>(p, c0, cols, cnt);
    if (c0 >= un.n) break;
    const int64_t e = un.e;
    const int nc = un.n - c0 < NCOL ? un.n - c0 : NCOL;
    const int first = KS == 1 ? 0 : int(blockIdx.z) * kWaves + wave, step = KS == 1 ? 1 : p.splits * kWaves;
    Loop::run(
        p.wd_codes + e * p.H * p.I, p.wd_scales + e * p.H * (p.I / 32), p.H, p.s_codes, p.s_scales, M, int(p.I), first,
        step, np > first ? (np - first + step - 1) / step : 0, nt, int64_t(tstep) * kRows, smem + wave * L::SLOTS * L::SLOT,
        [&](int q) -> int64_t { return int64_t(t0) * kRows + q; },
        [&](int q) -> int64_t { return q < nc ? int64_t(cols[q]) : -1; },
        [&](int t, const v16f (&acc)[2][FN]) {
          const int64_t h0 = (t0 + int64_t(t) * tstep) * kRows;
          if constexpr (KS == 1) {
#pragma unroll
            for (int J = 0; J < FN; ++J) {
              if (32 * J + r < nc) {
                float* dst = p.rows + int64_t(cols[32 * J + r]) * p.H + h0 + 4 * h;
#pragma unroll
                for (int f = 0; f < 2; ++f)
                  if (h0 + 32 * f < p.H) {   // H % 32 == 0
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                      *reinterpret_cast<float4*>(dst + 32 * f + 8 * k) =
                          make_float4(acc[f][J][4 * k], acc[f][J][4 * k + 1], acc[f][J][4 * k + 2], acc[f][J][4 * k + 3]);
                  }
              }
            }
          } else {
            float* st = reinterpret_cast<float*>(smem);
#pragma unroll
            for (int J = 0; J < FN; ++J) {
#if defined(__HIP_DEVICE_COMPILE__)
              asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
#endif
              __syncthreads();
              tok_stage<FN>(st, acc, J);
              __syncthreads();
              // thread: column c, rows 8 k .. + 7
              const int c = threadIdx.x >> 3, k = threadIdx.x & 7;
              if (32 * J + c < nc && h0 + 8 * k < p.H) {
                float* dst = p.rows + (blockIdx.z * M + cols[32 * J + c]) * p.H + h0 + 8 * k;
                float v[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] = tok_sum(st, 8 * k + q, c);
                if constexpr (LAST) {
#pragma unroll
                  for (int q = 0; q < 8; ++q) publish(dst + q, v[q]);
                } else {
                  *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
                  *reinterpret_cast<float4*>(dst + 4) = make_float4(v[4], v[5], v[6], v[7]);
                }
              }
            }
          }
        });
    __syncthreads();
  }
  if constexpr (LAST) {
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("s_waitcnt vmcnt(0)" : : : "memory");   // what this thread published has reached memory
#endif
    __syncthreads();
    if (threadIdx.x == 0)
      last = __hip_atomic_fetch_add(p.done + blockIdx.x, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
             gridDim.y * gridDim.z - 1;
    __syncthreads();
    if (!last) return;
    // thread: a token, one row of the tile; kBatch of its rows loaded at a time
    constexpr int kBatch = 8;
    const int64_t t = threadIdx.x >> 6, hh = int64_t(blockIdx.x) * kRows + lane;
    if (t >= p.T || hh >= p.H) return;
    const int K = int(p.K), S = p.splits;
    const float res = p.residual ? bf16_to_f32(p.residual[t * p.H + hh]) : 0.f;
    float acc = 0.f, x = 0.f;
    for (int j0 = 0; j0 < K * S; j0 += kBatch) {
      float v[kBatch];
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        const int j = j0 + q, k = j / S, s = j - k * S;
        v[q] = j < K * S && ids[t * K + k] >= 0 ? published(p.rows + (s * M + t * K + k) * p.H + hh) : 0.f;
      }
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        const int j = j0 + q, k = j / S, s = j - k * S;
        if (j >= K * S) continue;
        x += v[q];
        if (s == S - 1) {
          const int e = ids[t * K + k];
          if (e >= 0) acc += scores[t * K + k] * (x + (p.b2 ? bf16_to_f32(p.b2[int64_t(e) * p.H + hh]) : 0.f));
          x = 0.f;
        }
      }
    }
    acc += res;
    p.out[t * p.H + hh] = uint16_t(bf16x2_pack(acc, 0.f));
  }
}

// out[t] = residual[t] + the sum over selections k, in order, of a (the sum of
// the splits' rows + b2): a thread per 8 columns of a token.
__global__ void __launch_bounds__(64) tok_combine_kernel(MoeTokensArgs p) {
  const int64_t C = p.H / 8, c = int64_t(blockIdx.x) * 64 + threadIdx.x, t = blockIdx.y, M = p.T * p.K;
  if (c >= C) return;
  float acc[8] = {};
  constexpr int U = 4;   // selections whose rows are loaded together
  for (int k0 = 0; k0 < p.K; k0 += U) {
    float a[U], x[U][8] = {};
    int e[U];
    uint4 b[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int64_t pair = t * p.K + k0 + j;
      e[j] = k0 + j < p.K ? p.idx[pair] : -1;
      if (e[j] >= p.E) e[j] = -1;
      a[j] = p.on_i || e[j] < 0 ? 1.f : p.scores[pair];
    }
    for (int s = 0; s < p.splits; ++s) {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        if (e[j] < 0) continue;
        const float4* row = reinterpret_cast<const float4*>(p.rows + (s * M + t * p.K + k0 + j) * p.H + 8 * c);
        const float4 v = row[0], w = row[1];
        x[j][0] += v.x; x[j][1] += v.y; x[j][2] += v.z; x[j][3] += v.w;
        x[j][4] += w.x; x[j][5] += w.y; x[j][6] += w.z; x[j][7] += w.w;
      }
    }
    if (p.b2) {
#pragma unroll
      for (int j = 0; j < U; ++j)
        b[j] = e[j] >= 0 ? *reinterpret_cast<const uint4*>(p.b2 + int64_t(e[j]) * p.H + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const uint32_t w[4] = {b[j].x, b[j].y, b[j].z, b[j].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          x[j][2 * q] += lo_bf16(w[q]);
          x[j][2 * q + 1] += hi_bf16(w[q]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (e[j] >= 0) {
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[q] += a[j] * x[j][q];
      }
  }
  if (p.residual) {
    const uint4 b = *reinterpret_cast<const uint4*>(p.residual + t * p.H + 8 * c);
    const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      acc[2 * j] += lo_bf16(w[j]);
      acc[2 * j + 1] += hi_bf16(w[j]);
    }
  }
  *reinterpret_cast<uint4*>(p.out + t * p.H + 8 * c) =
      make_uint4(bf16x2_pack(acc[0], acc[1]), bf16x2_pack(acc[2], acc[3]), bf16x2_pack(acc[4], acc[5]),
                 bf16x2_pack(acc[6], acc[7]));
}

// Columns a workgroup works on at once: what an expert has, on average, twice over.
int columns(int64_t T, int64_t E, int64_t K) { return T <= kFewTokens ? kFewTokens : T <= 8 ? 8 : T * K <= 16 * E ? 32 : 64; }
// Experts with pairs, at most.
int64_t busy_units(int64_t T, int64_t E, int64_t K) { return T * K < E ? T * K : E; }
// Units, at most: a listed expert has one for every `columns` pairs.
int64_t units_of(int64_t T, int64_t E, int64_t K) {
  return busy_units(T, E, K) + (T <= kFewTokens ? 0 : T * K / columns(T, E, K));
}
// Whole tiles a wave (KS = 1) where that gives every CU a workgroup.
bool whole_tiles(int64_t tiles, int64_t units) { return tiles * units >= 256 * kWaves; }

template <int NCOL>
void go(const MoeTokensArgs& p, hipStream_t st) {
  const int64_t nu = p.nunits, t1 = p.I / 32, t2 = (p.H + kRows - 1) / kRows, busy = busy_units(p.T, p.E, p.K);
  // KS = 1: as many workgroups as the CUs hold at once (by their LDS), each wave with its share of the tiles
  const int64_t room = NCOL <= 8 ? 512 : 256;
  auto wgs = [&](int64_t tiles) {
    const int64_t most = (tiles + kWaves - 1) / kWaves, want = (room + busy - 1) / busy;
    return unsigned(want < most ? want : most);
  };
  auto first = [&](auto generic) {
    if (whole_tiles(t1, busy)) tok_gate_up_kernel<NCOL, generic(), 1><<<dim3(wgs(t1), unsigned(nu)), 64 * kWaves, 0, st>>>(p);
    else tok_gate_up_kernel<NCOL, generic(), 4><<<dim3(unsigned(t1), unsigned(nu)), 64 * kWaves, 0, st>>>(p);
  };
  if (p.H % 128) first(std::true_type{});
  else first(std::false_type{});
  const bool whole = whole_tiles(t2, busy);
  auto second = [&](auto generic) {
    if (whole) tok_down_kernel<NCOL, generic(), 1><<<dim3(wgs(t2), unsigned(nu)), 64 * kWaves, 0, st>>>(p);
    else tok_down_kernel<NCOL, generic(), 4><<<dim3(unsigned(t2), unsigned(nu), unsigned(p.splits)), 64 * kWaves, 0, st>>>(p);
  };
  if (p.I % 128) second(std::true_type{});
  else second(std::false_type{});
  if (NCOL == kFewTokens && !whole) return;   // the last workgroups have added up
  tok_combine_kernel<<<dim3(unsigned((p.H / 8 + 63) / 64), unsigned(p.T)), 64, 0, st>>>(p);
}
}  // namespace

// The down projection's contraction is split over workgroups until there are
// two for each of 256 CUs, with at least 2 pairs of K a wave.
int64_t tokens_splits(int64_t T, int64_t H, int64_t I, int64_t E, int64_t K) {
  const int64_t tiles = (H + kRows - 1) / kRows, nu = busy_units(T, E, K), np = (I + 127) / 128;
  if (whole_tiles(tiles, nu)) return 1;
  int64_t s = (512 + tiles * nu - 1) / (tiles * nu);
  if (s > np / (2 * kWaves)) s = np / (2 * kWaves);
  return s < 1 ? 1 : s > 8 ? 8 : s;
}
int64_t tokens_units(int64_t T, int64_t E, int64_t K) { return units_of(T, E, K); }
bool tokens_few(int64_t T) { return T <= kFewTokens; }

hipError_t launch_moe_tokens(MoeTokensArgs p, hipStream_t st) {
  p.nunits = int(units_of(p.T, p.E, p.K));
  p.by_pair = p.T * p.K < p.E;
  if (tokens_few(p.T)) {
    go<kFewTokens>(p, st);
    return hipGetLastError();
  }
  const int ncol = columns(p.T, p.E, p.K);
  const hipError_t e = launch_tok_prep(p, ncol, st);
  if (e != hipSuccess) return e;
  if (ncol == 8) go<8>(p, st);
  else if (ncol == 32) go<32>(p, st);
  else go<64>(p, st);
  return hipGetLastError();
}

}  // namespace mx
