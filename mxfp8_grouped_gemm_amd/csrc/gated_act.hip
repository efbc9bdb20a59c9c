// gated_act.hip -- the gated activation (SwiGLU, GeGLU) with its gate/up
// checkpoint in MXFP8, forward and backward.
//
// gate_up [R][2][C]: row r's gate g = [r][0][c] and up u = [r][1][c].
//   forward:  inter = bf16(act(g) u) from the bf16 inputs; g and u each as
//             codes and one E8M0 scale per 32 along C (the library's MXFP8
//             rule), the only thing the backward needs
//   backward: g, u = code * 2^X, dGate = bf16(d u act'(g)), dUp = bf16(d act(g))
// inter, dGate and dUp are rounded once, from fp32.  With slot ids (C a whole
// number of periods B, element c at slot c % B of block r), the elements of
// slots without a token count as zero: they do not reach their group's scale,
// and their outputs are zero.
//
// HBM-bound: forward 4 bytes read and 2 + 2 + 2/32 written an element, backward
// 2 + 2/32 + 2 read and 4 written.  One thread takes 8 consecutive elements
// (16-byte bf16 accesses); the four threads of a group share its largest
// magnitude by two DPP moves.  The bf16 results are stored with the nontemporal
// hint (5% faster at 135 to 576 MB a pass).  The inputs are loaded with it
// where a pass moves more than the 256 MB infinity cache holds (forward 442 MB:
// 74.7 -> 69.2 us, backward 576 MB: 92.8 -> 90 us); below that they may still
// lie there from the kernel that wrote them (135 MB: 21.8 us without, 24.2 with).
#include <type_traits>

#include "kernels.hpp"
#include "mx_device.hpp"
#include "segment.hpp"
#include "swiglu.hpp"

namespace mx {

namespace {
constexpr int kThreads = 256;
constexpr int64_t kInfinityCacheBytes = int64_t(256) << 20;

template <bool NT>
__device__ __forceinline__ uint4 load16(const void* q) {
  if constexpr (NT) {
    const u32x4_t v = __builtin_nontemporal_load(static_cast<const u32x4_t*>(q));
    return uint4{v[0], v[1], v[2], v[3]};
  } else {
    return *static_cast<const uint4*>(q);
  }
}
template <bool NT>
__device__ __forceinline__ uint2 load8(const void* q) {
  if constexpr (NT) {
    const u32x2_t v = __builtin_nontemporal_load(static_cast<const u32x2_t*>(q));
    return uint2{v[0], v[1]};
  } else {
    return *static_cast<const uint2*>(q);
  }
}

// This thread's row and run of 8 columns; runs are numbered below 2^31 (the
// launcher's bound), so the divisions are 32-bit ones.
struct Place {
  uint32_t r, c8;
  bool in;
  __device__ __forceinline__ explicit Place(const GatedActArgs& p) {
    const uint32_t v = blockIdx.x * kThreads + threadIdx.x, per = uint32_t(p.C / 8);
    in = v < uint32_t(p.R) * per;
    r = v / per;
    c8 = v - r * per;
  }
};

// bit k: slot of element 8 c8 + k holds a token (B a multiple of 8)
__device__ __forceinline__ uint32_t live_bits(const GatedActArgs& p, const Place& q) {
  const int4* id = reinterpret_cast<const int4*>(p.slot_id + q.r * p.B + q.c8 % uint32_t(p.B / 8) * 8);
  const int4 a = id[0], b = id[1];
  const int v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) m |= uint32_t(v[k] >= 0 && v[k] < p.T) << k;
  return m;
}
// bf16 pairs with the elements of dead slots zeroed
__device__ __forceinline__ void keep_live(uint32_t (&w)[4], uint32_t live) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    w[k] &= (live >> (2 * k) & 1 ? 0xffffu : 0u) | (live >> (2 * k + 1) & 1 ? 0xffff0000u : 0u);
}

// 8 elements' codes and their group's scale byte (the group's four threads are
// consecutive lanes of a quad)
template <int FMT>
__device__ __forceinline__ void encode8(const uint32_t (&w)[4], uint8_t* codes, uint8_t* scale, bool first) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) m = absmax_bf16x2(m, w[k]);
  m = max(m & 0xffffu, m >> 16);
  m = seg::umax<4>(m);
  const int X = scale_exp<FMT>(m << 16);
  const float inv = inv_scale(X);
  *reinterpret_cast<uint2*>(codes) =
      uint2{encode4<FMT>(lo_bf16(w[0]), hi_bf16(w[0]), lo_bf16(w[1]), hi_bf16(w[1]), inv),
            encode4<FMT>(lo_bf16(w[2]), hi_bf16(w[2]), lo_bf16(w[3]), hi_bf16(w[3]), inv)};
  if (first) *scale = uint8_t(X + 127);
}

// 2^X of an E8M0 byte (byte 0: 2^-127, an fp32 subnormal)
__device__ __forceinline__ float scale_value(uint32_t b) { return __uint_as_float(b ? b << 23 : 0x400000u); }
// four codes of a word
template <int FMT>
__device__ __forceinline__ void decode4(uint32_t w, float s, float* v) {
  if (FMT == kE4M3) {
    const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), false), b = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), true);
    v[0] = a[0] * s; v[1] = a[1] * s; v[2] = b[0] * s; v[3] = b[1] * s;
  } else {
    const auto a = __builtin_amdgcn_cvt_pk_f32_bf8(int(w), false), b = __builtin_amdgcn_cvt_pk_f32_bf8(int(w), true);
    v[0] = a[0] * s; v[1] = a[1] * s; v[2] = b[0] * s; v[3] = b[1] * s;
  }
}
}  // namespace

template <int FMT, bool GEGLU, bool SLOTS, bool NT>
__global__ void __launch_bounds__(kThreads) gated_act_fwd_kernel(GatedActArgs p) {
  const Place q(p);
  if (!q.in) return;   // C % 32 == 0: quads leave together
  const int64_t r = q.r, c = int64_t(q.c8) * 8, at = r * 2 * p.C + c;
  const uint4 g4 = load16<NT>(p.gate_up + at);
  const uint4 u4 = load16<NT>(p.gate_up + at + p.C);
  uint32_t g[4] = {g4.x, g4.y, g4.z, g4.w}, u[4] = {u4.x, u4.y, u4.z, u4.w};
  if (SLOTS) {
    const uint32_t live = live_bits(p, q);
    keep_live(g, live);
    keep_live(u, live);
  }
  uint32_t o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    o[k] = bf16x2_rne(gate_act<GEGLU>(lo_bf16(g[k])) * lo_bf16(u[k]), gate_act<GEGLU>(hi_bf16(g[k])) * hi_bf16(u[k]));
  store_nt(p.inter + r * p.C + c, uint4{o[0], o[1], o[2], o[3]});
  const bool first = (threadIdx.x & 3) == 0;
  encode8<FMT>(g, p.codes + at, p.scales + at / 32, first);
  encode8<FMT>(u, p.codes + at + p.C, p.scales + (at + p.C) / 32, first);
}

template <int FMT, bool GEGLU, bool SLOTS, bool NT>
__global__ void __launch_bounds__(kThreads) gated_act_bwd_kernel(GatedActArgs p) {
  const Place q(p);
  if (!q.in) return;
  const int64_t r = q.r, c = int64_t(q.c8) * 8, at = r * 2 * p.C + c;
  const uint4 d4 = load16<NT>(p.dinter + r * p.C + c);
  const uint2 gc = load8<NT>(p.codes_in + at);
  const uint2 uc = load8<NT>(p.codes_in + at + p.C);
  const float sg = scale_value(p.scales_in[at / 32]), su = scale_value(p.scales_in[(at + p.C) / 32]);
  uint32_t d[4] = {d4.x, d4.y, d4.z, d4.w};
  float g[8], u[8];
  decode4<FMT>(gc.x, sg, g);
  decode4<FMT>(gc.y, sg, g + 4);
  decode4<FMT>(uc.x, su, u);
  decode4<FMT>(uc.y, su, u + 4);
  const uint32_t live = SLOTS ? live_bits(p, q) : 0xffu;
  uint32_t og[4], ou[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float dg[2], du[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = 2 * k + h;
      const float x = h ? hi_bf16(d[k]) : lo_bf16(d[k]);
      float act, dact;
      gate_act_d<GEGLU>(g[i], act, dact);
      dg[h] = x * u[i] * dact;
      du[h] = x * act;
      if (SLOTS && !(live >> i & 1)) dg[h] = du[h] = 0.f;
    }
    og[k] = bf16x2_rne(dg[0], dg[1]);
    ou[k] = bf16x2_rne(du[0], du[1]);
  }
  store_nt(p.dgate_up + at, uint4{og[0], og[1], og[2], og[3]});
  store_nt(p.dgate_up + at + p.C, uint4{ou[0], ou[1], ou[2], ou[3]});
}

namespace {
template <class F>
hipError_t dispatch(const GatedActArgs& p, const F& f) {
  const int64_t n = p.R * (p.C / 8), grid = (n + kThreads - 1) / kThreads;
  if (n == 0) return hipSuccess;
  if (n > int64_t(1) << 31) return hipErrorInvalidValue;
  const bool nt = p.R * p.C > kInfinityCacheBytes / 8;   // 8.06 bytes an element
  auto slots = [&](auto fmt, auto geglu, auto with) {
    if (nt) f(fmt, geglu, with, std::true_type{}, unsigned(grid));
    else f(fmt, geglu, with, std::false_type{}, unsigned(grid));
  };
  auto act = [&](auto fmt, auto geglu) {
    if (p.slot_id) slots(fmt, geglu, std::true_type{});
    else slots(fmt, geglu, std::false_type{});
  };
  auto kind = [&](auto fmt) {
    if (p.geglu) act(fmt, std::true_type{});
    else act(fmt, std::false_type{});
  };
  if (p.fmt == kE4M3) kind(std::integral_constant<int, kE4M3>{});
  else kind(std::integral_constant<int, kE5M2>{});
  return hipGetLastError();
}
}  // namespace

hipError_t launch_gated_act_fwd(const GatedActArgs& p, hipStream_t st) {
  return dispatch(p, [&](auto fmt, auto geglu, auto slots, auto nt, unsigned grid) {
    gated_act_fwd_kernel<fmt(), geglu(), slots(), nt()><<<grid, kThreads, 0, st>>>(p);
  });
}
hipError_t launch_gated_act_bwd(const GatedActArgs& p, hipStream_t st) {
  return dispatch(p, [&](auto fmt, auto geglu, auto slots, auto nt, unsigned grid) {
    gated_act_bwd_kernel<fmt(), geglu(), slots(), nt()><<<grid, kThreads, 0, st>>>(p);
  });
}

}  // namespace mx
