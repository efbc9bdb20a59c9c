// moe_fwd.hip -- the MoE forward around its two products: the gate/up kernel at
// 128 x 128 tiles and the tile-shape dispatch, the slots' set-up, the
// checkpoint's dead tiles, and the sum over a token's slots.
//
// The down projection is Phase 3's kernel (moe_phase3.hip): rows = slots, the
// contraction over I instead of 2I, each slot's fp32 row stored on its own.
#include "moe_fwd_gate_up.hpp"
#include "moe_lists.hpp"
#include "philox.hpp"

namespace mx {

template hipError_t fwd_gate_up_launch<128, 128, false>(MoeFwdArgs, hipStream_t);
extern template hipError_t fwd_gate_up_launch<128, 128, true>(MoeFwdArgs, hipStream_t);
extern template hipError_t fwd_gate_up_launch<256, 256, false>(MoeFwdArgs, hipStream_t);
extern template hipError_t fwd_gate_up_launch<256, 128, false>(MoeFwdArgs, hipStream_t);

namespace {
struct Tile {
  int m, n;
};
Tile fwd_tile(const MoeFwdArgs& p) {
  if (p.H % 128 != 0 || p.I < 128) return {128, 128};
  return {256, p.B >= 256 ? 256 : 128};
}
}  // namespace

TileRangeJob fwd_gate_up_ranges(const MoeFwdArgs& p) {
  const Tile t = fwd_tile(p);
  return {t.n, int((p.I + t.m / 2 - 1) / (t.m / 2)), int(p.B), p.tile_start, nullptr, 0, 0, p.rr_tiles};
}

hipError_t launch_fwd_gate_up(const MoeFwdArgs& p, hipStream_t st) {
  if (p.H % 128 != 0) return fwd_gate_up_launch<128, 128, true>(p, st);
  const Tile t = fwd_tile(p);
  if (t.m == 128) return fwd_gate_up_launch<128, 128, false>(p, st);
  return t.n == 256 ? fwd_gate_up_launch<256, 256, false>(p, st) : fwd_gate_up_launch<256, 128, false>(p, st);
}

// ---------------------------------------------------------------------------
// The checkpoint's slots behind a block's last live tile: zeros (and scale byte
// 0, an all-zero group's).  One workgroup per 16 rows of a block.
namespace {
constexpr int kDeadRows = 16;
__global__ void __launch_bounds__(256) fwd_dead_ckpt_kernel(MoeFwdArgs p, int W, int parts) {
  const int b = blockIdx.x / parts, part = blockIdx.x % parts;
  const int64_t s0 = int64_t((p.flag[b] + W - 1) / W) * W;   // the first slot of no live tile
  if (s0 >= p.B) return;
  const int64_t r0 = int64_t(part) * kDeadRows, rows = 2 * p.I - r0 < kDeadRows ? 2 * p.I - r0 : kDeadRows;
  const int64_t base = int64_t(b) * 2 * p.I + r0;
  const int per = int((p.B - s0) * (p.ckpt ? 2 : 1) / 16);   // 16-byte runs a row
  for (int k = threadIdx.x; k < rows * per; k += 256) {
    const int64_t row = base + k / per, c = k % per;
    uint8_t* dst = p.ckpt ? reinterpret_cast<uint8_t*>(p.ckpt + row * p.B + s0) : p.ck8_codes + row * p.B + s0;
    store_nt(dst + 16 * c, make_uint4(0u, 0u, 0u, 0u));
  }
  if (!p.ckpt) {
    const int words = int((p.B - s0) / 128);   // of 4 scale bytes; W % 128 == 0
    for (int k = threadIdx.x; k < rows * words; k += 256)
      *reinterpret_cast<uint32_t*>(p.ck8_scales + (base + k / words) * (p.B / 32) + s0 / 32 + 4 * (k % words)) = 0u;
  }
}
}  // namespace

hipError_t launch_fwd_dead_ckpt(const MoeFwdArgs& p, hipStream_t st) {
  const int64_t parts = (2 * p.I + kDeadRows - 1) / kDeadRows;
  if (parts * p.N > kMaxGrid256) return hipErrorInvalidValue;
  fwd_dead_ckpt_kernel<<<unsigned(parts * p.N), 256, 0, st>>>(p, fwd_tile(p).n, int(parts));
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// out[t] = residual[t] + drop( sum over t's slots, in expert order, of
// a (row + b2) ), fp32, rounded once; with the affinity on I the rows carry it
// already.  A team of TPT threads per token (whole waves), each wave finding
// the token's slots by itself, 64 experts a ballot, and a thread summing 8
// columns: 16-byte stores, and one counter of the dropout mask.
namespace {
template <int TPT>
__global__ void __launch_bounds__(256) fwd_combine_kernel(MoeCombineArgs p) {
  const int64_t t = int64_t(blockIdx.x) * (256 / TPT) + threadIdx.x / TPT;
  if (t >= p.T) return;
  const int lane = threadIdx.x & 63, me = threadIdx.x % TPT;
  const int64_t C = p.H / 8;
  for (int64_t c0 = 0; c0 < C; c0 += TPT) {
    const int64_t c = c0 + me;
    const bool in = c < C;
    float acc[8] = {};
    for (int64_t e0 = 0; e0 < p.E; e0 += 64) {
      const int32_t so = e0 + lane < p.E ? p.slot_of[t * p.E + e0 + lane] : -1;
      uint64_t live = __ballot(so >= 0);
      while (live) {
        // up to 4 slots at a time, their rows loaded before the first is added
        constexpr int U = 4;
        float4 v[U][2];
        float a[U];
        uint4 bias[U];
        int n = 0;
#pragma unroll
        for (int k = 0; k < U; ++k) {
          a[k] = 0.f;
          if (live) {
            const int l = __ffsll(static_cast<unsigned long long>(live)) - 1;
            live &= live - 1;
            const int64_t s = __builtin_amdgcn_readlane(so, l);
            a[k] = p.slot_aff ? p.slot_aff[s] : 1.f;
            if (in) {
              const f32x4_t* row = reinterpret_cast<const f32x4_t*>(p.rows + s * p.H + 8 * c);
              const f32x4_t x = __builtin_nontemporal_load(row), y = __builtin_nontemporal_load(row + 1);
              v[k][0] = make_float4(x[0], x[1], x[2], x[3]);
              v[k][1] = make_float4(y[0], y[1], y[2], y[3]);
              if (p.b2) bias[k] = *reinterpret_cast<const uint4*>(p.b2 + (e0 + l) * p.H + 8 * c);
            }
            n = k + 1;
          }
        }
        if (!in) continue;
#pragma unroll
        for (int k = 0; k < U; ++k) {
          if (k >= n) continue;
          float x[8] = {v[k][0].x, v[k][0].y, v[k][0].z, v[k][0].w, v[k][1].x, v[k][1].y, v[k][1].z, v[k][1].w};
          if (p.b2) {
            const uint32_t w[4] = {bias[k].x, bias[k].y, bias[k].z, bias[k].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              x[2 * j] += lo_bf16(w[j]);
              x[2 * j + 1] += hi_bf16(w[j]);
            }
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[j] += a[k] * x[j];
        }
      }
    }
    if (!in) continue;
    if (p.drop.thr) {
      const uint4 w = philox(PhiloxKey(p.drop.rng), uint64_t(t * C + c));
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = philox_keep(w, j, p.drop.thr) ? acc[j] * p.drop.scale : 0.f;
    }
    if (p.residual) {
      const uint4 x = *reinterpret_cast<const uint4*>(p.residual + t * p.H + 8 * c);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[2 * j] += lo_bf16(w[j]);
        acc[2 * j + 1] += hi_bf16(w[j]);
      }
    }
    store_nt(p.out + t * p.H + 8 * c, make_uint4(bf16x2_pack(acc[0], acc[1]), bf16x2_pack(acc[2], acc[3]),
                                                 bf16x2_pack(acc[4], acc[5]), bf16x2_pack(acc[6], acc[7])));
  }
}
}  // namespace

hipError_t launch_fwd_combine(const MoeCombineArgs& p, hipStream_t st) {
  const int tpt = p.H <= 512 ? 64 : p.H <= 1024 ? 128 : 256;   // 8 columns a thread
  const int64_t per = 256 / tpt, grid = (p.T + per - 1) / per;
  if (grid > kMaxGrid256) return hipErrorInvalidValue;
  if (tpt == 64) fwd_combine_kernel<64><<<unsigned(grid), 256, 0, st>>>(p);
  else if (tpt == 128) fwd_combine_kernel<128><<<unsigned(grid), 256, 0, st>>>(p);
  else fwd_combine_kernel<256><<<unsigned(grid), 256, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace mx
