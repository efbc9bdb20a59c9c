// moe_fwd_gate_up.hpp -- the MoE forward's first product: both projections of
// the routed gated feed-forward block, its activation and the product of the
// two in one kernel.  The template and its launcher; the tile shapes are
// instantiated in moe_fwd_gate_up_*.hip so they compile in parallel.
//
// Per block b of expert e (tile rows = gate and up rows, tile columns = block
// slot p, contraction over H, on the scaled fp8 MFMA):
//   g[i][p] = sum_h deq(Wg)[i][h] deq(Q(x_tok))[h] + b1[0][i],  u likewise
//   s = act(g) u (times the slot's affinity with the affinity on I), fp32
//   s -> MXFP8 E4M3, groups of 32 along i: the down projection's operand
//   g, u -> the checkpoint that moe_bwd_mxfp8 reads, [N][2][I][B]: bf16, or
//           MXFP8 codes and scales of the bf16 values, groups of 32 along the
//           slots (one rounding more than from fp32, so that the 8-bit
//           checkpoint is the bf16 one, quantised)
// s is rounded once, to its code: from the fp32 sums, not the bf16 checkpoint.
// The scaled MFMA truncates small products (some 5e-5 of a result's size in all),
// which moves 0.16% of the codes to a neighbour, and once in some ten thousand
// groups the scale: y is then 0.0020 off the formula (norm of the difference over
// y's) where its own rounding to bf16 is 0.0017.  Where there are few tiles
// (fwd_few_tiles), a call of few groups could meet such a one to its whole extent,
// and its time goes by latency: there the products are the codes' exact bf16 values
// on the bf16 MFMA (kFp8Bf16), at half the rate.
//
// A tile of BM rows holds BM / 2 gate rows and the same BM / 2 up rows, as
// fragments of 32 in turn: a lane's accumulators then hold gate and up of the
// same 16 (i, p), 16 of a group's 32 i with the lane's other half holding the
// rest, so activation, product and group maxima stay in registers.  The tile
// columns are the slots, whose X code rows are gathered by token (or lie in the slots'
// order, fwd_x_by_slot).  Tiles cover
// i up to Ip, the contraction of the down projection in whole pairs: groups from
// I on get zeros.  Workgroups whose tile holds no routed slot write the
// checkpoint's zeros there.
//
// Measured (256 x 256 tiles but the last): 32768 slots, H = 4096, I = 14336, 3.5 ms,
// 2.2 PFLOP/s; H = 2048, I = 1408, 8-bit checkpoint, 285 us, 1.33 PFLOP/s; 262144 slots,
// H = 1536, I = 256, bf16 checkpoint, 400 us, 1.03 PFLOP/s.  Without their stages (two of
// them only) these take 0.7 ms, 129 and 179 us: what bounds the short contractions is the
// start of a tile (its block, expert, tokens, first loads: a chain of latencies) and its
// epilogue, which one workgroup a CU does not overlap.
#pragma once
#include "gemm_v2.hpp"
#include "gemm_v3.hpp"
#include "kernels.hpp"
#include "moe_tiles.hpp"
#include "mx_device.hpp"
#include "swiglu.hpp"

namespace mx {

using v2::v16f;

// Tile row r -> row of the expert's [2I] weight rows (gate, then up), or -1
// past I.  i0: the tile's first i.
template <int BM>
__device__ __forceinline__ int64_t fwd_weight_row(int r, int64_t i0, int64_t I) {
  const int w = r / (BM / 2), f = (r % (BM / 2)) / 32;
  const int64_t i = i0 + w * (BM / 4) + (f >> 1) * 32 + (r & 31);
  return i < I ? (f & 1) * I + i : -1;
}

// This workgroup's tile: block b, slot tile tn, i tile tm; live: it holds a
// routed slot.  false: nothing to do.
struct FwdTile {
  int b, tm, tn;
  bool live;
};
template <int BN>
__device__ __forceinline__ bool fwd_tile_of(const MoeFwdArgs& p, bool want_dead, FwdTile& t) {
  const int N = int(p.N), wg = blockIdx.x;
  const int total = p.tile_start[N], t8 = (total + 7) & ~7;
  const int id = wg < t8 && !p.rr_tiles ? v2::xcd_remap(wg, t8) : wg;
  t.live = id < total;
  if (!t.live && (!want_dead || id >= N * p.tiles_m * int(p.B / BN))) return false;
  t.b = p.tile_start[N + 1 + id];
  const int slots = (p.flag[t.b] + BN - 1) / BN;
  if (t.live) {
    v2::grouped_tile<8>(id - p.tile_start[t.b], p.tiles_m, slots, t.tm, t.tn);
  } else {
    const int local = id - p.dead[t.b];
    t.tn = slots + local / p.tiles_m;
    t.tm = local % p.tiles_m;
  }
  return true;
}

// The checkpoint of a tile without routed slots: zeros (scale byte 0: an all-zero group's).
template <int BM, int BN, int CK>
__device__ __forceinline__ void fwd_zero_ckpt(const MoeFwdArgs& p, const FwdTile& t) {
  const int64_t i0 = int64_t(t.tm) * (BM / 2), s0 = int64_t(t.tn) * BN;
  const int rows = p.I - i0 < BM / 2 ? int(p.I - i0) : BM / 2;   // not positive: past I
  constexpr int RUNS = BN * (CK == 1 ? 2 : 1) / 16;             // 16-byte runs a row
  for (int part = 0; part < 2; ++part) {
    const int64_t row0 = (int64_t(t.b) * 2 + part) * p.I + i0;
    for (int k = threadIdx.x; k < rows * RUNS; k += v2::kThreads) {
      const int64_t at = (row0 + k / RUNS) * p.B + s0;
      uint8_t* dst = (CK == 1 ? reinterpret_cast<uint8_t*>(p.ckpt + at) : p.ck8_codes + at) + 16 * (k % RUNS);
      store_nt(dst, make_uint4(0u, 0u, 0u, 0u));
    }
    if constexpr (CK != 1) {
      for (int k = threadIdx.x; k < rows * (BN / 128); k += v2::kThreads)
        *reinterpret_cast<uint32_t*>(p.ck8_scales + (row0 + k / (BN / 128)) * (p.B / 32) + s0 / 32 + 4 * (k % (BN / 128))) = 0u;
    }
  }
}

// One fragment pair's checkpoint (32 rows i x 32 slots, words gate | up << 16)
// through LDS, turned so that a lane holds 8 consecutive slots of a row:
// 4 lanes then store 64 consecutive bytes (bf16) or 32 (codes).  A row's 32
// slots are a group of the 8-bit checkpoint: 4 lanes share its maximum.
constexpr int kCkPitch = 36;   // words a row; 16-byte reads
constexpr int kCkWaveBytes = 32 * kCkPitch * 4;
template <int CK>   // 1: bf16, 2 + format: MXFP8
__device__ __forceinline__ void fwd_store_ckpt(const MoeFwdArgs& p, int b, int64_t i, int64_t s, const uint32_t* lds) {
  const int lane = threadIdx.x & 63, c = lane & 3;
#pragma unroll
  for (int it = 0; it < 2; ++it) {
    const int r = 16 * it + (lane >> 2);
    const uint4 a = *reinterpret_cast<const uint4*>(lds + r * kCkPitch + 8 * c);
    const uint4 d = *reinterpret_cast<const uint4*>(lds + r * kCkPitch + 8 * c + 4);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, d.x, d.y, d.z, d.w};
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      uint32_t v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = part ? hi_halves(w[2 * k], w[2 * k + 1]) : lo_halves(w[2 * k], w[2 * k + 1]);
      const int64_t row = (int64_t(b) * 2 + part) * p.I + i + r;
      if constexpr (CK == 1) {
        store_nt(p.ckpt + row * p.B + s + 8 * c, make_uint4(v[0], v[1], v[2], v[3]));
      } else {
        constexpr int F = CK - 2;
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) m = absmax_bf16x2(m, v[k]);
        m = max(m & 0xffffu, m >> 16);
        m = max(m, uint32_t(__shfl_xor(int(m), 1, 64)));
        m = max(m, uint32_t(__shfl_xor(int(m), 2, 64)));
        const int X = scale_exp<F>(m << 16);
        const float sc = cvt_scale(X);
        const uint32_t lo = encode_bf16x4<F>(v[0], v[1], sc), hi = encode_bf16x4<F>(v[2], v[3], sc);   // they saturate
        *reinterpret_cast<uint2*>(p.ck8_codes + row * p.B + s + 8 * c) = make_uint2(lo, hi);
        if (c == 0) p.ck8_scales[row * (p.B / 32) + s / 32] = uint8_t(X + 127);
      }
    }
  }
}

template <int BM, int BN, int ELEM, bool RAG, bool GEGLU, int CK>
__global__ void __launch_bounds__(v2::kThreads) fwd_gate_up_kernel(MoeFwdArgs p) {
  constexpr int SMEM = v3::smem_bytes(BM, BN);
  static_assert(SMEM >= 4 * kCkWaveBytes, "the checkpoint's staging fits the ring");
  __shared__ __attribute__((aligned(16))) uint8_t smem[SMEM];
  constexpr int FM = BM / 64, FN = BN / 64;
  FwdTile tile;
  if (!fwd_tile_of<BN>(p, CK != 0, tile)) return;
  if (CK != 0 && !tile.live) {
    fwd_zero_ckpt<BM, BN, CK>(p, tile);
    return;
  }
  const int b = tile.b;
  const int64_t i0 = int64_t(tile.tm) * (BM / 2), n0 = int64_t(tile.tn) * BN;
  const int64_t sbase = int64_t(b) * p.B, e = p.b2e[b], P = p.N * p.B;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, h = lane >> 5, r = lane & 31;
  const int wm = wave >> 1, wn = wave & 1;
  const int32_t* st = p.slot_tok + sbase;
  const int64_t B_ = p.B, I_ = p.I;
  auto tok_of = [&](int q) -> int64_t { const int64_t s = n0 + q; return s < B_ ? int64_t(st[s]) : -1; };
  auto row_of = [&](int q) -> int64_t { return fwd_weight_row<BM>(q, i0, I_); };
  const uint8_t* wc = p.w_codes + e * 2 * p.I * p.H;
  const uint8_t* ws = p.w_scales + e * 2 * p.I * (p.Hp / 32);
  v16f acc[FM][FN];
  if (i0 < p.I) {   // else the tile lies between I and Ip: no products
    v3::ScaleDma<BM, BN> sd;
    const int64_t xr = p.x_by_slot ? P : p.T;
    v3::setup_scales_map(sd, ws, 2 * p.I, 2 * p.I * (p.Hp / 32), row_of, p.x_scales, xr, xr * (p.Hp / 32),
                         [&](int q) -> int64_t { return p.x_by_slot ? (q < BN ? sbase + n0 + q : -1) : tok_of(q); });
    // the four-slot ring, also for these row-major operands (256 x 256: 3.6 ms against 3.9 on the pair-slot
    // ring at H = 4096, 287 us against 332 at H = 2048)
    v3::Op<BM> A;
    v3::Op<BN> B;
    v3::setup_gather(A, wc, 2 * p.I, p.H, row_of);
    if (p.x_by_slot) v3::setup_rows_sm(B, p.x_codes, sbase + n0, sbase + p.B, P, p.Hp);
    else v3::setup_gather(B, p.x_codes, p.T, p.Hp, tok_of);
    v3::mainloop<BM, BN, ELEM, kE4M3, kE4M3, v3::KMapPlain, RAG>(A, B, &sd, int(p.Hp / v3::SK), v3::KMapPlain{}, smem,
                                                                   acc, uint32_t(p.H));
  }
  if constexpr (CK != 0) __syncthreads();   // every wave is done with the ring: its bytes stage the checkpoint
  uint32_t* stage = reinterpret_cast<uint32_t*>(smem + wave * kCkWaveBytes);
  saturate_fp8_conversions();
  // this lane's slots.  A slot without a token has X rows of zeros, so g = u = 0 without a bias.
  bool ok[FN];
  float aff[FN];
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int64_t s = sbase + n0 + wn * (BN / 2) + 32 * j + r;   // BN divides B: inside the block
    ok[j] = p.slot_tok[s] >= 0;
    aff[j] = p.on_i ? p.slot_aff[s] : 1.f;
  }
  v2::static_for<FM / 2>([&](auto Q) {
    const int64_t i = i0 + wm * (BM / 4) + 32 * int(Q);   // the group's first i; I % 32 == 0: all of it or nothing
    if (i >= p.I) {   // up to Ip: zeros
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int64_t slot = sbase + n0 + wn * (BN / 2) + 32 * j + r;
        *reinterpret_cast<uint4*>(p.inter_codes + stage_major_off(slot, i + 16 * h, P, p.Ip)) = make_uint4(0u, 0u, 0u, 0u);
        if (h == 0) p.inter_scales[((i >> 7) * P + slot) * 4 + (i >> 5 & 3)] = 0;
      }
    } else {
      if (p.b1) {
        const uint16_t* row = p.b1 + e * 2 * p.I + i + 4 * h;
        v2::static_for<4>([&](auto K) {
          const uint2 g = *reinterpret_cast<const uint2*>(row + 8 * int(K));
          const uint2 u = *reinterpret_cast<const uint2*>(row + p.I + 8 * int(K));
          const float bg[4] = {lo_bf16(g.x), hi_bf16(g.x), lo_bf16(g.y), hi_bf16(g.y)};
          const float bu[4] = {lo_bf16(u.x), hi_bf16(u.x), lo_bf16(u.y), hi_bf16(u.y)};
          v2::static_for<FN>([&](auto J) {
            v2::static_for<4>([&](auto D) {
              constexpr int k = 4 * int(K) + int(D);
              acc[2 * int(Q)][J][k] = ok[J] ? acc[2 * int(Q)][J][k] + bg[int(D)] : 0.f;
              acc[2 * int(Q) + 1][J][k] = ok[J] ? acc[2 * int(Q) + 1][J][k] + bu[int(D)] : 0.f;
            });
          });
        });
      }
      v2::static_for<FN>([&](auto J) {
        const int64_t s = n0 + wn * (BN / 2) + 32 * int(J);   // the fragment's first slot
        float v[16];
        uint32_t m = 0;
        v2::static_for<16>([&](auto K) {
          constexpr int k = K;
          const float g = acc[2 * int(Q)][J][k], u = acc[2 * int(Q) + 1][J][k];
          v[k] = gate_act<GEGLU>(g) * u;
          if constexpr (CK != 0) stage[(8 * (k >> 2) + 4 * h + (k & 3)) * kCkPitch + r] = bf16x2_pack(g, u);
        });
        if (p.on_i) {
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] *= aff[J];
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) m = max(m, abs_bits(v[k]));
#if defined(__HIP_DEVICE_COMPILE__)
        {
          const auto x = __builtin_amdgcn_permlane32_swap(m, m, false, false);
          m = max(uint32_t(x[0]), uint32_t(x[1]));
        }
        const int X = scale_exp<kE4M3>(m);
        const float sc = cvt_scale(X);
        uint32_t w[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) w[t] = encode_f32x4(v[4 * t], v[4 * t + 1], v[4 * t + 2], v[4 * t + 3], sc);
        // word t of half h: rows 8t + 4h .. + 3.  Half 0 takes rows 0..15, half 1 rows 16..31.
        const auto x = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
        const auto y = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
        const int64_t slot = sbase + s + r, at = i + 16 * h;
        *reinterpret_cast<uint4*>(p.inter_codes + stage_major_off(slot, at, P, p.Ip)) = make_uint4(x[0], x[1], y[0], y[1]);
        if (h == 0) p.inter_scales[((i >> 7) * P + slot) * 4 + (i >> 5 & 3)] = uint8_t(X + 127);
#endif
        if constexpr (CK != 0) {
          wave_lds_order();
          fwd_store_ckpt<CK>(p, b, i, s, stage);
          wave_lds_order();
        }
      });
    }
  });
}

// ---------------------------------------------------------------------------
template <int BM, int BN, int ELEM>
hipError_t fwd_gate_up_launch(MoeFwdArgs p, hipStream_t st) {
  p.tiles_m = int(p.Ip / (BM / 2));
  const int64_t blocks = (int64_t(p.tiles_m) * (p.B / BN) * p.N + 7) & ~int64_t(7);   // every tile, rounded to 8
  if (blocks > kMaxGrid256) return hipErrorInvalidValue;
  auto go = [&](auto rag, auto geglu, auto ck) {
    fwd_gate_up_kernel<BM, BN, ELEM, rag(), geglu(), ck()><<<unsigned(blocks), v2::kThreads, 0, st>>>(p);
  };
  auto kind = [&](auto rag, auto geglu) {
    if (p.ckpt) go(rag, geglu, std::integral_constant<int, 1>{});
    else if (!p.ck8_codes) go(rag, geglu, std::integral_constant<int, 0>{});
    else if (p.ck8_fmt == kE4M3) go(rag, geglu, std::integral_constant<int, 2 + kE4M3>{});
    else go(rag, geglu, std::integral_constant<int, 2 + kE5M2>{});
  };
  auto act = [&](auto rag) {
    if (p.geglu) kind(rag, std::true_type{});
    else kind(rag, std::false_type{});
  };
  if (p.H % 128) act(std::true_type{});
  else act(std::false_type{});
  return hipGetLastError();
}

}  // namespace mx
