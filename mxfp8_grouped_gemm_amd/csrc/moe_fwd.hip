// moe_fwd.hip -- the MoE forward around its two products: the gate/up kernel at
// 128 x 128 tiles and the tile-shape dispatch, and the sum over a token's slots.
#include "moe_fwd_gate_up.hpp"
#include "philox.hpp"

namespace mx {

template hipError_t fwd_gate_up_launch<128, 128, v3::kFp8>(MoeFwdArgs, hipStream_t);
extern template hipError_t fwd_gate_up_launch<128, 128, v3::kFp8Bf16>(MoeFwdArgs, hipStream_t);
extern template hipError_t fwd_gate_up_launch<256, 256, v3::kFp8>(MoeFwdArgs, hipStream_t);

namespace {
// No more tiles of 128 x 128 than the CUs hold at once (two each): their side is 128 and their products
// exact (T = 1500, 246 tiles: 14 us against 12).
bool fwd_few_tiles(int64_t I, int64_t N, int64_t B) { return N * (B / 128) * ((I + 127) / 128 * 2) <= 512; }
// The tile's side: 256 from contractions and blocks that are long enough for one workgroup a CU
// (H = 4096: 3.6 ms against 5.1 at 128; H = 2048: 290 us against 308), else 128, two workgroups a CU
// (blocks of 128 slots, H = 1536: 390 us against 420 at 256 x 128).  The whole forward of 32768 slots at 128 -> 256 in us,
// in brackets of 131072: H = 1024: I = 512 123 -> 137 (395 -> 418), 1408 229 -> 248 (793 -> 874), 8192 1000 -> 1058
// (3839 -> 4062); H = 1280: I = 1408 266 -> 276 (968 -> 1018); H = 1536: 165 -> 173 (571 -> 566), 322 -> 316 (1158 -> 1141),
// 1439 -> 1402 (5588 -> 5363); H = 2048: 202 -> 209 (734 -> 705), 400 -> 372 (1536 -> 1412).
int fwd_side(int64_t H, int64_t I, int64_t N, int64_t B) {
  return I < 128 || B < 256 || H < 1536 || fwd_few_tiles(I, N, B) ? 128 : 256;
}
}  // namespace

// Every slot's X row by itself and stage-major costs the preparation 0.25 ns a KB of it and spares each 256-row
// tile's reads half lines: H = 4096, I = 14336, 40k slots: preparation 62 -> 98 us, products 3.65 -> 3.44 ms.
// The whole forward, by token -> by slot, top-2 (each row twice) and, in brackets, top-4, 32768 routed slots:
// H = 4096: I = 4096 1.72 -> 1.73 ms (1.70 -> 1.75), 6144 2.47 -> 2.41 (2.42 -> 2.43), 8192 3.21 -> 3.11 (3.12 -> 3.07),
// 14336 5.15 -> 4.96; H = 2048: I = 4096 (0.92 -> 0.94), 8192 1.85 -> 1.82 (1.73 -> 1.76), 11264 (2.31 -> 2.26).
// 4096 routed slots: within 2% either way up to I = 14336.
bool fwd_x_by_slot(int64_t H, int64_t I, int64_t N, int64_t B) {
  return I >= 8192 && fwd_side(H, I, N, B) == 256 &&
         (H + 127) / 128 * 4 <= (int64_t(1) << 30) / (N * B);   // one launch, 32-bit offsets
}

TileRangeJob fwd_gate_up_ranges(const MoeFwdArgs& p) {
  const int side = fwd_side(p.H, p.I, p.N, p.B);
  return {side, int(p.Ip / (side / 2)), int(p.B), p.tile_start, nullptr, 0, 0, p.rr_tiles, p.dead};
}

hipError_t launch_fwd_gate_up(const MoeFwdArgs& p, hipStream_t st) {
  if (fwd_few_tiles(p.I, p.N, p.B)) return fwd_gate_up_launch<128, 128, v3::kFp8Bf16>(p, st);
  return fwd_side(p.H, p.I, p.N, p.B) == 128 ? fwd_gate_up_launch<128, 128, v3::kFp8>(p, st)
                                             : fwd_gate_up_launch<256, 256, v3::kFp8>(p, st);
}

// ---------------------------------------------------------------------------
// out[t] = residual[t] + drop( sum over t's slots, in expert order, of
// a (row + b2) ), fp32, rounded once; with the affinity on I the rows carry it
// already.  A team of TPT threads per token (whole waves), each wave finding
// the token's slots by itself, 64 experts a ballot, and a thread summing 8
// columns: 16-byte stores, and one counter of the dropout mask.  Bound by the
// rows' bytes: 262144 of H = 1536 in fp16, 906 MB with the result, 181 us, 5.0 TB/s
// (eight slots at a time, more registers, 196).
namespace {
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
template <int TPT, bool F16>
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
        float4 v[F16 ? 1 : U][2];
        u32x4_t v16[F16 ? U : 1];
        float a[U], sc[F16 ? U : 1];
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
              if constexpr (F16) {
                v16[k] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p.rows16 + s * p.H + 8 * c));
                sc[k] = p.row_scale[s * ((p.H + 63) / 64) + c / 8];
              } else {
                const f32x4_t* row = reinterpret_cast<const f32x4_t*>(p.rows + s * p.H + 8 * c);
                const f32x4_t x = __builtin_nontemporal_load(row), y = __builtin_nontemporal_load(row + 1);
                v[k][0] = make_float4(x[0], x[1], x[2], x[3]);
                v[k][1] = make_float4(y[0], y[1], y[2], y[3]);
              }
              if (p.b2) bias[k] = *reinterpret_cast<const uint4*>(p.b2 + (e0 + l) * p.H + 8 * c);
            }
            n = k + 1;
          }
        }
        if (!in) continue;
#pragma unroll
        for (int k = 0; k < U; ++k) {
          if (k >= n) continue;
          float x[8];
          if constexpr (F16) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t pair = v16[k][j];   // (a bit cast of the vector's element itself gives element 0)
              const f16x2_t q = __builtin_bit_cast(f16x2_t, pair);
              x[2 * j] = float(q[0]) * sc[k];
              x[2 * j + 1] = float(q[1]) * sc[k];
            }
          } else {
            x[0] = v[k][0].x; x[1] = v[k][0].y; x[2] = v[k][0].z; x[3] = v[k][0].w;
            x[4] = v[k][1].x; x[5] = v[k][1].y; x[6] = v[k][1].z; x[7] = v[k][1].w;
          }
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
  auto go = [&](auto f16) {
    if (tpt == 64) fwd_combine_kernel<64, f16()><<<unsigned(grid), 256, 0, st>>>(p);
    else if (tpt == 128) fwd_combine_kernel<128, f16()><<<unsigned(grid), 256, 0, st>>>(p);
    else fwd_combine_kernel<256, f16()><<<unsigned(grid), 256, 0, st>>>(p);
  };
  if (p.rows16) go(std::true_type{});
  else go(std::false_type{});
  return hipGetLastError();
}

}  // namespace mx
