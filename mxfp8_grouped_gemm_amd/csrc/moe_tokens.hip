// moe_tokens.hip -- the MoE forward for few tokens (decoding): the layer of
// moe_fwd.hip straight from the router's selections, without block lists.
//
// Bound by the bytes of the selected experts' weights, each read once: an
// expert has a handful of rows, so a product is a stream of weights past a few
// columns.  Selections ("pairs" t * K + k) keep their index as row of every
// intermediate.  A workgroup takes 64 weight rows of one expert (32 gate rows
// and the same 32 up rows; or 64 rows of the down projection) and the expert's
// pairs, NCOL at a time, found by scanning the ids; its 4 waves split the
// contraction, each with an LDS ring of its own (no barrier in the loop), and
// add up at the end in wave order.  Whole 128-byte lines of weight rows go
// straight to LDS; scales and the columns' codes go with them.
//   launch 1  X along H to codes               (launch_quant_rows)
//   launch 2  gate/up, activation, product, s to codes
//   launch 3  down projection, per pair and split of the contraction, fp32
//   launch 4  the sum over splits and selections, biases, residual
#include "gemm_v4.hpp"
#include "kernels.hpp"
#include "mx_device.hpp"
#include "swiglu.hpp"

namespace mx {

namespace {
using v2::v16f;
constexpr int kWaves = 4;
constexpr int kRows = 64;                    // weight rows a workgroup
constexpr int kStagePitch = 36;              // words a row of the waves' sums
constexpr int kStageBytes = kWaves * kRows * kStagePitch * 4;
constexpr int kSlots = 2;                    // pairs (128 bytes of K) in a wave's ring

template <int NCOL>
struct TokLds {
  static constexpr int A = kRows * 128, B = NCOL * 128, SLOT = A + B + 512;   // then a scale word a row and column
  static constexpr int RING = kWaves * kSlots * SLOT;
  static constexpr int BYTES = RING > kStageBytes ? RING : kStageBytes;
};

// The columns of unit u (of gridDim.y): entries c0 .. c0 + NCOL - 1 of the
// ascending list of pairs that select its expert; n: how many there are in all.
// A unit is an expert, or, where there are fewer pairs than experts, a pair,
// which stands for its expert if it is the first to select it (n = 0 if not).
struct Unit {
  int e, n;
};
template <int NCOL>
__device__ __forceinline__ Unit tok_unit(const MoeTokensArgs& p, int c0, int32_t* cols, int* cnt) {
  const int M = int(p.T * p.K), lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int u = blockIdx.y;
  const int e = p.by_pair ? p.idx[u] : u;
  if (e < 0 || e >= p.E) return Unit{0, 0};
  // each wave a quarter of the pairs, counted, then listed from its first rank on
  const int per = (M + kWaves - 1) / kWaves, lo = wave * per, hi = lo + per < M ? lo + per : M;
  int mine = 0, before_u = 0;
  for (int j0 = lo; j0 < hi; j0 += 64) {
    const int j = j0 + lane;
    const uint64_t hit = __ballot(j < hi && p.idx[j] == e);
    mine += __popcll(hit);
    before_u += __popcll(__ballot(j < u && (hit >> lane & 1)));
  }
  if (lane == 0) {
    cnt[wave] = mine;
    cnt[kWaves + wave] = before_u;
  }
  __syncthreads();
  int rank = 0, n = 0, before = 0;
  for (int w = 0; w < kWaves; ++w) {
    rank += w < wave ? cnt[w] : 0;
    n += cnt[w];
    before += cnt[kWaves + w];
  }
  if (p.by_pair && before > 0) return Unit{0, 0};
  for (int j0 = lo; j0 < hi; j0 += 64) {
    const int j = j0 + lane;
    const bool hit = j < hi && p.idx[j] == e;
    const uint64_t mask = __ballot(hit);
    const int q = rank + __popcll(mask & ((uint64_t(1) << lane) - 1)) - c0;
    if (hit && q >= 0 && q < NCOL) cols[q] = j;
    rank += __popcll(mask);
  }
  __syncthreads();
  return Unit{e, n};
}

// One wave's share of a product: pairs [u0, u1) of K bytes past 64 weight rows
// (row(q), q < 64: source row or -1) and NCOL columns (col(q): source row or -1).
template <int NCOL, bool GENERIC>
struct TokLoop {
  static constexpr int FN = NCOL <= 32 ? 1 : 2;
  static constexpr int NA = kRows / 8, NB = NCOL / 8;          // DMA instructions: 8 rows of 128 bytes each
  static constexpr int PER = NA + NB + (GENERIC ? 0 : 2);      // of a pair
  using L = TokLds<NCOL>;

  template <class Row, class Col>
  __device__ __forceinline__ static void run(const uint8_t* w, const uint8_t* ws, int64_t wrows, const uint8_t* x,
                                             const uint8_t* xs, int64_t xrows, int K, int u0, int u1, uint8_t* ring,
                                             const Row& row, const Col& col, v16f (&acc)[2][FN]) {
#if defined(__HIP_DEVICE_COMPILE__)
    const int lane = threadIdx.x & 63, h = lane >> 5, r = lane & 31, G = K / 32;
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[f][j][q] = 0.f;
    const v3::v4i rw = v3::rsrc(v2::make_rsrc(w, uint32_t(wrows * K)));
    const v3::v4i rx = v3::rsrc(v2::make_rsrc(x, uint32_t(xrows * K)));
    const v3::v4i rws = v3::rsrc(v2::make_rsrc(ws, uint32_t(wrows * G)));
    const v3::v4i rxs = v3::rsrc(v2::make_rsrc(xs, uint32_t(xrows * G)));
    uint32_t offa[NA], offb[NB], offs[2];
    auto code_off = [&](int q, int64_t src) -> uint32_t {   // LDS row q: lane l its physical chunk l & 7
      return src >= 0 ? uint32_t(src * K + 16 * ((lane & 7) ^ v4::swz(q))) : v3::kOOB;
    };
#pragma unroll
    for (int j = 0; j < NA; ++j) offa[j] = code_off(8 * j + (lane >> 3), row(8 * j + (lane >> 3)));
#pragma unroll
    for (int j = 0; j < NB; ++j) offb[j] = code_off(8 * j + (lane >> 3), col(8 * j + (lane >> 3)));
    {
      const int64_t a = row(lane), b = lane < NCOL ? col(lane) : -1;
      offs[0] = a >= 0 ? uint32_t(a * G) : v3::kOOB;
      offs[1] = b >= 0 ? uint32_t(b * G) : v3::kOOB;
    }
    const uint32_t base = v3::lds_addr(ring);
    auto issue = [&](int u) {
      const bool live = u < u1;
      const uint32_t kc = live ? uint32_t(u) * 128u : 0u, slot = base + uint32_t((u - u0) & (kSlots - 1)) * L::SLOT;
      v3::v4i ra = rw, rb = rx, rc = rws, rd = rxs;   // past the end: no records, zeros without memory traffic
      ra[2] = live ? ra[2] : 0;
      rb[2] = live ? rb[2] : 0;
      rc[2] = live ? rc[2] : 0;
      rd[2] = live ? rd[2] : 0;
      // a ragged last pair: chunks past K read as zeros (K % 32 == 0: whole chunks)
      auto in_k = [&](int j, uint32_t off) -> uint32_t {
        if constexpr (!GENERIC) return off;
        const int q = 8 * j + (lane >> 3);
        return int(kc) + 16 * ((lane & 7) ^ v4::swz(q)) < K ? off : v3::kOOB;
      };
#pragma unroll
      for (int j = 0; j < NA; ++j) v3::dma16(ra, slot + j * 1024u, in_k(j, offa[j]), kc);
#pragma unroll
      for (int j = 0; j < NB; ++j) v3::dma16(rb, slot + L::A + j * 1024u, in_k(j, offb[j]), kc);
      if constexpr (!GENERIC) {
        v3::dma4(rc, slot + L::A + L::B, offs[0], kc >> 5);
        v3::dma4(rd, slot + L::A + L::B + 256, offs[1], kc >> 5);
      }
    };
#pragma unroll
    for (int k = 0; k < kSlots; ++k) issue(u0 + k);
    for (int u = u0; u < u1; ++u) {
      const uint8_t* slot = ring + ((u - u0) & (kSlots - 1)) * L::SLOT;
      // this pair has landed once only the later ones' loads remain
      asm volatile("s_waitcnt vmcnt(%0)" : : "n"((kSlots - 1) * PER) : "memory");
      __builtin_amdgcn_sched_barrier(0);
      uint4 fa[2][2][2], fb[2][FN][2];   // [stage][fragment][chunk]
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
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const int q = NCOL < 32 ? r % NCOL : 32 * j + r;   // columns past NCOL repeat, and are not used
#pragma unroll
          for (int c = 0; c < 2; ++c)
            fb[P][j][c] = *reinterpret_cast<const uint4*>(slot + L::A + q * 128 + 16 * ((4 * P + 2 * c + h) ^ v4::swz(q)));
        }
      }
      const uint32_t* sc = reinterpret_cast<const uint32_t*>(slot + L::A + L::B);
      if constexpr (!GENERIC) {
#pragma unroll
        for (int f = 0; f < 2; ++f) sa[f] = sc[32 * f + r];
#pragma unroll
        for (int j = 0; j < FN; ++j) sb[j] = sc[64 + (NCOL < 32 ? r % NCOL : 32 * j + r)];
      } else {
        // scale rows that are not whole words: byte by byte, groups past K as 0
        auto word = [&](const uint8_t* s, int64_t src) -> uint32_t {
          uint32_t v = 0;
          if (src >= 0)
            for (int g = 0; g < 4; ++g)
              if (4 * u + g < G) v |= uint32_t(s[src * G + 4 * u + g]) << (8 * g);
          return v;
        };
#pragma unroll
        for (int f = 0; f < 2; ++f) sa[f] = word(ws, row(32 * f + r));
#pragma unroll
        for (int j = 0; j < FN; ++j) sb[j] = word(xs, col(NCOL < 32 ? r % NCOL : 32 * j + r));
      }
      // every read of the slot is back before its next pair is loaded
      asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
      __builtin_amdgcn_sched_barrier(0);
      issue(u + kSlots);
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[f][j] = v3::mma<kE4M3, kE4M3, 0>(fa[0][f], fb[0][j], acc[f][j], int(sa[f] >> (8 * h)), int(sb[j] >> (8 * h)));
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[f][j] = v3::mma<kE4M3, kE4M3, 2>(fa[1][f], fb[1][j], acc[f][j], int(sa[f] >> (8 * h)), int(sb[j] >> (8 * h)));
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

template <int NCOL, bool GENERIC, bool GEGLU>
__global__ void __launch_bounds__(64 * kWaves) tok_gate_up_kernel(MoeTokensArgs p) {
  constexpr int FN = TokLoop<NCOL, GENERIC>::FN;
  __shared__ __attribute__((aligned(16))) uint8_t smem[TokLds<NCOL>::BYTES];
  __shared__ int32_t cols[NCOL];
  __shared__ int cnt[2 * kWaves];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);   // uniform: descriptors stay scalar
  const int64_t i0 = int64_t(blockIdx.x) * 32;   // I % 32 == 0
  for (int c0 = 0;; c0 += NCOL) {
    const Unit un = tok_unit<NCOL>(p, c0, cols, cnt);
    if (c0 >= un.n) return;
    const int64_t e = un.e;
    const int nc = un.n - c0 < NCOL ? un.n - c0 : NCOL;
    const int np = int((p.H + 127) / 128);
    v16f acc[2][FN];
    TokLoop<NCOL, GENERIC>::run(
        p.w_codes + e * 2 * p.I * p.H, p.w_scales + e * 2 * p.I * (p.H / 32), 2 * p.I, p.x_codes, p.x_scales, p.T,
        int(p.H), wave * np / kWaves, (wave + 1) * np / kWaves, smem + wave * kSlots * TokLds<NCOL>::SLOT,
        [&](int q) -> int64_t { return (q >> 5) * p.I + i0 + (q & 31); },
        [&](int q) -> int64_t { return q < nc ? cols[q] / int(p.K) : -1; }, acc);
    float* st = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int J = 0; J < FN; ++J) {
      __syncthreads();   // the rings, or the previous columns, are done with
      tok_stage<FN>(st, acc, J);
      __syncthreads();
      // thread: column c, rows 4 k .. + 3
      const int c = threadIdx.x >> 3, k = threadIdx.x & 7;
      if (32 * J + c < nc) {
        const int64_t pair = cols[32 * J + c];
        const float a = p.on_i ? p.scores[pair] : 1.f;
        float v[4];
        uint32_t m = 0;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          float g = tok_sum(st, 4 * k + t, c), u = tok_sum(st, 32 + 4 * k + t, c);
          if (p.b1) {
            const uint16_t* b = p.b1 + e * 2 * p.I + i0 + 4 * k + t;
            g += bf16_to_f32(b[0]);
            u += bf16_to_f32(b[p.I]);
          }
          v[t] = gate_act<GEGLU>(g) * u * a;
          m = max(m, abs_bits(v[t]));
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
    __syncthreads();   // the columns and the staging are rewritten
  }
}

template <int NCOL, bool GENERIC>
__global__ void __launch_bounds__(64 * kWaves) tok_down_kernel(MoeTokensArgs p) {
  constexpr int FN = TokLoop<NCOL, GENERIC>::FN;
  __shared__ __attribute__((aligned(16))) uint8_t smem[TokLds<NCOL>::BYTES];
  __shared__ int32_t cols[NCOL];
  __shared__ int cnt[2 * kWaves];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), part = blockIdx.z * kWaves + wave, parts = p.splits * kWaves;
  const int64_t h0 = int64_t(blockIdx.x) * kRows, M = p.T * p.K;
  for (int c0 = 0;; c0 += NCOL) {
    const Unit un = tok_unit<NCOL>(p, c0, cols, cnt);
    if (c0 >= un.n) return;
    const int64_t e = un.e;
    const int nc = un.n - c0 < NCOL ? un.n - c0 : NCOL;
    const int np = int((p.I + 127) / 128);
    v16f acc[2][FN];
    TokLoop<NCOL, GENERIC>::run(
        p.wd_codes + e * p.H * p.I, p.wd_scales + e * p.H * (p.I / 32), p.H, p.s_codes, p.s_scales, M, int(p.I),
        part * np / parts, (part + 1) * np / parts, smem + wave * kSlots * TokLds<NCOL>::SLOT,
        [&](int q) -> int64_t { return h0 + q < p.H ? h0 + q : -1; },
        [&](int q) -> int64_t { return q < nc ? int64_t(cols[q]) : -1; }, acc);
    float* st = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int J = 0; J < FN; ++J) {
      __syncthreads();
      tok_stage<FN>(st, acc, J);
      __syncthreads();
      // thread: column c, rows 8 k .. + 7
      const int c = threadIdx.x >> 3, k = threadIdx.x & 7;
      if (32 * J + c < nc && h0 + 8 * k < p.H) {   // H % 32 == 0
        float* dst = p.rows + (int64_t(blockIdx.z) * M + cols[32 * J + c]) * p.H + h0 + 8 * k;
        float v[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) v[t] = tok_sum(st, 8 * k + t, c);
        *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(dst + 4) = make_float4(v[4], v[5], v[6], v[7]);
      }
    }
    __syncthreads();
  }
}

// out[t] = residual[t] + the sum over selections k, in order, of a (the sum of
// the splits' rows + b2): a thread per 8 columns of a token.
__global__ void __launch_bounds__(64) tok_combine_kernel(MoeTokensArgs p) {
  const int64_t C = p.H / 8, c = int64_t(blockIdx.x) * 64 + threadIdx.x, t = blockIdx.y, M = p.T * p.K;
  if (c >= C) return;
  float acc[8] = {};
  for (int k = 0; k < p.K; ++k) {
    const int64_t pair = t * p.K + k;
    const int e = p.idx[pair];
    if (e < 0 || e >= p.E) continue;
    const float a = p.on_i ? 1.f : p.scores[pair];
    float x[8] = {};
    for (int s = 0; s < p.splits; ++s) {
      const float4* row = reinterpret_cast<const float4*>(p.rows + (s * M + pair) * p.H + 8 * c);
      const float4 v = row[0], w = row[1];
      x[0] += v.x; x[1] += v.y; x[2] += v.z; x[3] += v.w;
      x[4] += w.x; x[5] += w.y; x[6] += w.z; x[7] += w.w;
    }
    if (p.b2) {
      const uint4 b = *reinterpret_cast<const uint4*>(p.b2 + int64_t(e) * p.H + 8 * c);
      const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[2 * j] += lo_bf16(w[j]);
        x[2 * j + 1] += hi_bf16(w[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] += a * x[j];
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

int64_t units(const MoeTokensArgs& p) { return p.T * p.K < p.E ? p.T * p.K : p.E; }

template <int NCOL>
void gate_up(const MoeTokensArgs& p, dim3 grid, hipStream_t st) {
  auto go = [&](auto generic, auto geglu) { tok_gate_up_kernel<NCOL, generic(), geglu()><<<grid, 64 * kWaves, 0, st>>>(p); };
  auto kind = [&](auto generic) {
    if (p.geglu) go(generic, std::true_type{});
    else go(generic, std::false_type{});
  };
  if (p.H % 128) kind(std::true_type{});
  else kind(std::false_type{});
}
template <int NCOL>
void down(const MoeTokensArgs& p, dim3 grid, hipStream_t st) {
  if (p.I % 128) tok_down_kernel<NCOL, true><<<grid, 64 * kWaves, 0, st>>>(p);
  else tok_down_kernel<NCOL, false><<<grid, 64 * kWaves, 0, st>>>(p);
}
}  // namespace

// The down projection's contraction is split over workgroups until there are
// two for each of 256 CUs, with at least 2 pairs of K a wave.
int64_t tokens_splits(int64_t T, int64_t H, int64_t I, int64_t E, int64_t K) {
  const int64_t wgs = (T * K < E ? T * K : E) * ((H + kRows - 1) / kRows), np = (I + 127) / 128;
  int64_t s = (512 + wgs - 1) / wgs;
  if (s > np / (2 * kWaves)) s = np / (2 * kWaves);
  return s < 1 ? 1 : s > 8 ? 8 : s;
}

hipError_t launch_moe_tokens(MoeTokensArgs p, const uint16_t* x, hipStream_t st) {
  hipError_t e = launch_quant_rows(x, p.T, p.H, kE4M3, p.x_codes, p.x_scales, st);
  if (e != hipSuccess) return e;
  const unsigned nu = unsigned(units(p));
  p.by_pair = p.T * p.K < p.E;
  const dim3 g1(unsigned(p.I / 32), nu), g2(unsigned((p.H + kRows - 1) / kRows), nu, unsigned(p.splits));
  // columns a workgroup works on at once: what an expert has, on average, twice over
  const int ncol = p.T <= 8 ? 8 : p.T * p.K <= 16 * p.E ? 32 : 64;
  if (ncol == 8) gate_up<8>(p, g1, st);
  else if (ncol == 32) gate_up<32>(p, g1, st);
  else gate_up<64>(p, g1, st);
  if (ncol == 8) down<8>(p, g2, st);
  else if (ncol == 32) down<32>(p, g2, st);
  else down<64>(p, g2, st);
  tok_combine_kernel<<<dim3(unsigned((p.H / 8 + 63) / 64), unsigned(p.T)), 64, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace mx
