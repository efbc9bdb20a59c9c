// api_fwd.cpp -- the C ABI of the MoE forward, its few-token form, dropout and
// the transposed quantiser (include/mxfp8_moe.h): argument validation,
// workspace carving and the launch sequence on the caller's stream.
#include <climits>
#include <cmath>

#include "../../include/mxfp8_moe.h"
#include "api_util.hpp"
#include "kernels.hpp"

using namespace mx_api;

// The rule of a dropout probability: false unless 0 <= p <= 1.
static bool dropout_rule(double p, const int64_t* rng, mx::DropoutRule& r) {
  if (!(p >= 0. && p <= 1.)) return false;
  r.thr = uint32_t(std::floor(p * 65536. + 0.5));
  r.scale = r.thr < 65536 ? float(65536. / (65536. - r.thr)) : 0.f;
  r.rng = rng;
  return true;
}

extern "C" {

int mxfp8_quantize_transposed(const uint16_t* x, int64_t batch, int64_t rows, int64_t cols, int fmt, uint8_t* codes,
                              uint8_t* scales, void* stream) {
  const char* me = "mxfp8_quantize_transposed";
  if (batch < 0 || rows < 0 || cols < 0) return fail(MXFP8_ERR_INVALID_ARG, "%s: negative shape", me);
  if (!valid_fmt(fmt)) return fail(MXFP8_ERR_INVALID_ARG, "%s: fmt %d is not E4M3/E5M2", me, fmt);
  if (rows % 32) return fail(MXFP8_ERR_INVALID_ARG, "%s: rows %% 32 != 0", me);
  if (batch == 0 || rows == 0 || cols == 0) return ok();
  if (!x || !codes || !scales) return fail(MXFP8_ERR_INVALID_ARG, "%s: null pointer", me);
  if (!aligned16(x) || !aligned16(codes))
    return fail(MXFP8_ERR_INVALID_ARG, "%s: x and codes must be 16-byte aligned", me);
  if (mx::quantize_t_grid(batch, rows, cols) > mx::kMaxGrid256)
    return fail(MXFP8_ERR_UNSUPPORTED, "%s: more than %lld tiles of 128 x 128", me, (long long)mx::kMaxGrid256);
  return hip_status(mx::launch_quantize_t(x, batch, rows, cols, fmt, codes, scales, static_cast<hipStream_t>(stream)),
                    me);
}

/* ---- dropout ------------------------------------------------------------- */

static int dropout_run(const char* me, const dropout_add_args* a, bool backward, void* stream) {
  if (!a) return fail(MXFP8_ERR_INVALID_ARG, "%s: null args", me);
  if (a->rows < 0 || a->cols < 0) return fail(MXFP8_ERR_INVALID_ARG, "%s: negative shape", me);
  if (a->type != MXFP8_TYPE_F32 && a->type != MXFP8_TYPE_BF16)
    return fail(MXFP8_ERR_INVALID_ARG, "%s: type %d is not F32/BF16", me, a->type);
  mx::DropoutArgs d{};
  if (!dropout_rule(a->p, a->rng, d.rule))
    return fail(MXFP8_ERR_INVALID_ARG, "%s: p must be in [0, 1] (got %g)", me, a->p);
  if (backward && a->residual) return fail(MXFP8_ERR_INVALID_ARG, "%s: the backward takes no residual", me);
  if (a->rows == 0 || a->cols == 0) return ok();
  if (a->rows > (int64_t(1) << 34) / a->cols) return fail(MXFP8_ERR_UNSUPPORTED, "%s: rows * cols beyond 2^34", me);
  const int64_t lds[3] = {a->ldx, a->ldy, a->residual ? a->ldr : a->cols};
  for (int64_t ld : lds)
    if (ld < a->cols || ld > (int64_t(1) << 40) / a->rows)
      return fail(MXFP8_ERR_INVALID_ARG, "%s: a leading dimension is below cols or reaches past 2^40 elements", me);
  if (!a->x || !a->y || (d.rule.thr && !a->rng)) return fail(MXFP8_ERR_INVALID_ARG, "%s: null pointer", me);
  const void* al[3] = {a->x, a->residual, a->y};
  for (const void* q : al)
    if (!aligned16(q)) return fail(MXFP8_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", me);
  if (reinterpret_cast<uintptr_t>(a->rng) & 7u) return fail(MXFP8_ERR_INVALID_ARG, "%s: rng must be 8-byte aligned", me);
  d.x = a->x; d.residual = a->residual; d.y = a->y;
  d.rows = a->rows; d.cols = a->cols;
  d.ldx = a->ldx; d.ldr = a->residual ? a->ldr : a->cols; d.ldy = a->ldy;
  d.bf16 = a->type == MXFP8_TYPE_BF16;
  return hip_status(mx::launch_dropout(d, static_cast<hipStream_t>(stream)), me);
}

int dropout_add_fwd(const dropout_add_args* a, void* stream) { return dropout_run("dropout_add_fwd", a, false, stream); }
int dropout_add_bwd(const dropout_add_args* a, void* stream) { return dropout_run("dropout_add_bwd", a, true, stream); }

/* ---- MoE forward --------------------------------------------------------- */

namespace {
struct FwdLayout {
  size_t x_codes, x_scales, wgu_pairs, wd_pairs, inter_codes, inter_scales, rows, row_scale, parts, tiles1, dead, tiles2,
      slot_of, slot_tok, slot_aff, flag, done, total;
};
int64_t up128(int64_t v) { return (v + 127) & ~int64_t(127); }
}  // namespace

static void fwd_layout(const moe_fwd_mxfp8_args* a, FwdLayout* L) {
  const int64_t T = a->T, H = a->H, I = a->I, E = a->E, N = a->N, B = a->block_size, P = N * B;
  const int64_t Hp = up128(H), Ip = up128(I);
  const bool f16 = mx::fwd_down_fits(I);
  size_t o = 0;
  auto put = [&](size_t& field, int64_t bytes) {
    field = o;
    o = up256(o + size_t(bytes));
  };
  const int64_t xr = mx::fwd_x_by_slot(H, a->I, a->N, a->block_size) ? P : T;
  put(L->x_codes, xr * Hp);
  put(L->x_scales, xr * (Hp / 32));
  put(L->wgu_pairs, E * 2 * I * (Hp / 32));
  put(L->wd_pairs, E * H * (Ip / 32));
  put(L->inter_codes, P * Ip);
  put(L->inter_scales, P * (Ip / 32));
  put(L->rows, P * H * (f16 ? 2 : 4));
  put(L->row_scale, f16 ? P * ((H + 63) / 64) * 4 : 0);
  mx::Phase3Args q{};
  q.H = H; q.I = I / 2; q.N = N; q.B = B;
  put(L->parts, f16 ? 0 : mx::phase3_parts_bytes(q));
  // tile starts [N+1], then the tile -> block map over every tile a block can have at the smallest tile
  put(L->tiles1, (N + 1 + N * (Ip / 64) * (B / 128)) * 4);
  put(L->dead, N * 4);
  put(L->tiles2, (N + 1 + N * (B / 128) * ((H + 127) / 128)) * 4);
  put(L->slot_of, T * E * 4);
  put(L->slot_tok, P * 4);
  put(L->slot_aff, P * 4);
  put(L->flag, N * 4);
  put(L->done, 4);
  L->total = o;
}

static int fwd_check_shapes(const moe_fwd_mxfp8_args* a) {
  const char* me = "moe_fwd_mxfp8";
  if (!a) return fail(MXFP8_ERR_INVALID_ARG, "%s: null args", me);
  const int64_t T = a->T, H = a->H, I = a->I, E = a->E, N = a->N, B = a->block_size;
  if (T <= 0 || H <= 0 || I <= 0 || E <= 0 || N <= 0 || B <= 0)
    return fail(MXFP8_ERR_INVALID_ARG, "%s: sizes must be positive", me);
  if (H % 32 || I % 32)
    return fail(MXFP8_ERR_INVALID_ARG, "%s: H and I must be multiples of 32 (got %lld, %lld)", me, (long long)H,
                (long long)I);
  if (B != 128 && B != 256 && B != 512 && B != 1024)
    return fail(MXFP8_ERR_UNSUPPORTED, "%s: block_size %lld not in {128,256,512,1024}", me, (long long)B);
  // X's code rows, an expert's weight rows and the slots' scales are read through one buffer each, at 32-bit offsets
  const int64_t big = int64_t(1) << 40;
  if (T > big || H > big || I > big || E > big || N > big || N > INT32_MAX / B || T > INT32_MAX / E ||
      T > INT32_MAX / up128(H) || I > INT32_MAX / 2 / up128(H) || up128(I) > INT32_MAX / H ||
      N * B > (int64_t(1) << 24) || 2 * I > (int64_t(1) << 23) || N * B > INT32_MAX / (up128(I) / 32))
    return fail(MXFP8_ERR_UNSUPPORTED, "%s: sizes beyond 32-bit indexing", me);
  // one launch of each product, of the weights' scales and of the tokens
  if (N * (up128(I) / 64) * (B / 128) > mx::kMaxGrid256 - 8 || N * ((H + 127) / 128) * (B / 128) > mx::kMaxGrid256 - 512 ||
      E > (int64_t(1) << 23) / ((2 * I + 63) / 64 * ((H + 4095) / 4096) + (H + 63) / 64 * ((I + 4095) / 4096)) ||
      T > mx::kMaxGrid256)
    return fail(MXFP8_ERR_UNSUPPORTED, "%s: more tiles than one launch takes", me);
  return MXFP8_OK;
}

size_t moe_fwd_mxfp8_workspace_size(const moe_fwd_mxfp8_args* a) {
  if (fwd_check_shapes(a)) return 0;
  FwdLayout L;
  fwd_layout(a, &L);
  return L.total;
}

int moe_fwd_mxfp8(const moe_fwd_mxfp8_args* a, void* ws, size_t ws_bytes, void* stream) {
  const char* me = "moe_fwd_mxfp8";
  int rc = fwd_check_shapes(a);
  if (rc) return rc;
  if (a->affinity_on != 0 && a->affinity_on != 1)
    return fail(MXFP8_ERR_INVALID_ARG, "%s: affinity_on must be 0 (H) or 1 (I)", me);
  if (a->activation != MXFP8_ACT_SWIGLU && a->activation != MXFP8_ACT_GEGLU)
    return fail(MXFP8_ERR_INVALID_ARG, "%s: activation must be 0 (SwiGLU) or 1 (GeGLU)", me);
  if (a->affinity_on == 1 && (a->gate_up_proj_bias || a->down_proj_bias))
    return fail(MXFP8_ERR_UNSUPPORTED, "%s: a bias with the affinity on I is not supported", me);
  mx::DropoutRule drop{};
  if (!dropout_rule(a->dropout_p, a->dropout_rng, drop))
    return fail(MXFP8_ERR_INVALID_ARG, "%s: dropout_p must be in [0, 1] (got %g)", me, a->dropout_p);
  const void* req[] = {a->hidden_states, a->expert_affinities_masked, a->gate_up_codes, a->gate_up_scales,
                       a->down_codes, a->down_scales, a->token_position_to_id, a->block_to_expert,
                       a->output_hidden_states};
  for (const void* q : req)
    if (!q) return fail(MXFP8_ERR_INVALID_ARG, "%s: a required pointer is null", me);
  if (drop.thr && !a->dropout_rng) return fail(MXFP8_ERR_INVALID_ARG, "%s: dropout needs dropout_rng", me);
  const void* opt[] = {a->gate_up_proj_bias, a->down_proj_bias, a->gate_up_proj_act_checkpoint_T,
                       a->gate_up_checkpoint_codes, a->gate_up_checkpoint_scales, a->residual};
  for (const void* q : req)
    if (!aligned16(q)) return fail(MXFP8_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", me);
  for (const void* q : opt)
    if (!aligned16(q)) return fail(MXFP8_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", me);
  if (!a->gate_up_checkpoint_codes != !a->gate_up_checkpoint_scales)
    return fail(MXFP8_ERR_INVALID_ARG, "%s: gate_up_checkpoint_codes and _scales go together", me);
  if (a->gate_up_checkpoint_codes && a->gate_up_proj_act_checkpoint_T)
    return fail(MXFP8_ERR_INVALID_ARG, "%s: one gate/up checkpoint, in bf16 or in MXFP8, not both", me);
  if (a->gate_up_checkpoint_codes && !valid_fmt(a->fmt_checkpoint))
    return fail(MXFP8_ERR_INVALID_ARG, "%s: fmt_checkpoint must be E4M3 (0) or E5M2 (1)", me);
  if ((reinterpret_cast<uintptr_t>(a->num_valid_tokens) & 3u) || (reinterpret_cast<uintptr_t>(a->dropout_rng) & 7u))
    return fail(MXFP8_ERR_INVALID_ARG, "%s: num_valid_tokens must be 4-byte and dropout_rng 8-byte aligned", me);
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u))
    return fail(MXFP8_ERR_INVALID_ARG, "%s: workspace must be non-null and 256-byte aligned", me);
  FwdLayout L;
  fwd_layout(a, &L);
  if (ws_bytes < L.total) return fail(MXFP8_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", me, ws_bytes, L.total);

  const int64_t T = a->T, H = a->H, I = a->I, E = a->E, N = a->N, B = a->block_size;
  uint8_t* w = static_cast<uint8_t*>(ws);
  auto at = [&](size_t off) { return w + off; };
  auto ints = [&](size_t off) { return reinterpret_cast<int32_t*>(w + off); };
  hipStream_t st = static_cast<hipStream_t>(stream);
  hipError_t e;
  const bool f16 = mx::fwd_down_fits(I);
  float* slot_aff = reinterpret_cast<float*>(at(L.slot_aff));

  mx::MoeFwdArgs g{};
  g.T = T; g.H = H; g.I = I; g.E = E; g.N = N; g.B = B;
  g.Hp = up128(H); g.Ip = up128(I);
  g.x_codes = at(L.x_codes); g.x_scales = at(L.x_scales);
  g.x_by_slot = mx::fwd_x_by_slot(H, I, N, B);
  g.w_codes = a->gate_up_codes; g.w_scales = at(L.wgu_pairs);
  g.b1 = a->gate_up_proj_bias;
  g.slot_tok = ints(L.slot_tok); g.slot_aff = slot_aff; g.b2e = a->block_to_expert; g.flag = ints(L.flag);
  g.tile_start = ints(L.tiles1);
  g.inter_codes = at(L.inter_codes); g.inter_scales = at(L.inter_scales);
  g.ckpt = a->gate_up_proj_act_checkpoint_T;
  g.ck8_codes = a->gate_up_checkpoint_codes; g.ck8_scales = a->gate_up_checkpoint_scales; g.ck8_fmt = a->fmt_checkpoint;
  g.dead = g.ckpt || g.ck8_codes ? ints(L.dead) : nullptr;
  g.geglu = a->activation == MXFP8_ACT_GEGLU; g.on_i = a->affinity_on;
  g.rr_tiles = 2 * I * H >= kRoundRobinWeightBytes;
  // the down projection: rows in scaled fp16, or Phase 3's product with a contraction of I
  mx::MoeFwdDownArgs d{};
  d.H = H; d.I = I; d.Ip = g.Ip; d.N = N; d.B = B;
  d.inter_codes = g.inter_codes; d.inter_scales = g.inter_scales;
  d.w_codes = a->down_codes; d.w_scales = at(L.wd_pairs);
  d.b2e = a->block_to_expert; d.flag = g.flag; d.tile_start = ints(L.tiles2);
  d.rows = reinterpret_cast<uint16_t*>(at(L.rows)); d.row_scale = reinterpret_cast<float*>(at(L.row_scale));
  d.rr_tiles = H * I >= kRoundRobinWeightBytes;
  mx::Phase3Args d3{};
  d3.dgu_row_codes = g.inter_codes; d3.dgu_row_scales = g.inter_scales;
  d3.wgu_codes = a->down_codes; d3.wgu_scales = d.w_scales;
  d3.slot_tok = g.slot_tok; d3.b2e = a->block_to_expert; d3.flag = g.flag; d3.tile_start = d.tile_start;
  d3.H = H; d3.I = I / 2; d3.N = N; d3.B = B; d3.dx_slot = reinterpret_cast<float*>(at(L.rows));
  d3.conc = device_cus(st);
  d3.parts = !f16 && mx::phase3_parts_bytes(d3) > 0 ? at(L.parts) : nullptr;
  d3.rr_tiles = d.rr_tiles;
  d3.ranges_done = 1;
#define STEP(call, what) \
  if ((e = (call)) != hipSuccess) return hip_status(e, what);
  const mx::MoeFwdPrep prep{a->hidden_states, T, H, g.Hp, I, g.Ip, E, N, B, at(L.x_codes), at(L.x_scales),
                            a->gate_up_scales, at(L.wgu_pairs), a->down_scales, at(L.wd_pairs), a->token_position_to_id,
                            a->block_to_expert, a->expert_affinities_masked, a->num_valid_tokens, ints(L.slot_tok), slot_aff,
                            ints(L.slot_of), ints(L.flag), reinterpret_cast<unsigned*>(at(L.done)), g.x_by_slot,
                            {mx::fwd_gate_up_ranges(g), f16 ? mx::fwd_down_ranges(d) : mx::phase3_ranges(d3)}};
  STEP(mx::launch_fwd_prep(prep, st), "X, weight scales and slots");
  STEP(mx::launch_fwd_gate_up(g, st), "gate/up projections and activation");
  if (f16) {
    STEP(mx::launch_fwd_down(d, st), "down projection");
  } else {
    STEP(mx::launch_phase3(d3, MXFP8_E4M3, MXFP8_E4M3, st), "down projection");
  }
  const mx::MoeCombineArgs c{f16 ? nullptr : d3.dx_slot, f16 ? d.rows : nullptr, f16 ? d.row_scale : nullptr, ints(L.slot_of),
                             a->affinity_on == 0 ? slot_aff : nullptr, a->down_proj_bias, a->residual,
                             a->output_hidden_states, T, E, H, drop};
  STEP(mx::launch_fwd_combine(c, st), "sum of the tokens' slots");
#undef STEP
  return ok();
}

/* ---- MoE forward of few tokens ------------------------------------------- */

namespace {
struct TokLayout {
  size_t x_codes, x_scales, units, list, done, s_codes, s_scales, rows, total;
};
}  // namespace

static int tokens_check_shapes(const moe_tokens_fwd_mxfp8_args* a) {
  const char* me = "moe_tokens_fwd_mxfp8";
  if (!a) return fail(MXFP8_ERR_INVALID_ARG, "%s: null args", me);
  const int64_t T = a->T, H = a->H, I = a->I, E = a->E, K = a->K;
  if (T < 0 || H <= 0 || I <= 0 || E <= 0 || K <= 0) return fail(MXFP8_ERR_INVALID_ARG, "%s: sizes must be positive", me);
  if (H % 32 || I % 32)
    return fail(MXFP8_ERR_INVALID_ARG, "%s: H and I must be multiples of 32 (got %lld, %lld)", me, (long long)H,
                (long long)I);
  if (K > MXFP8_ROUTER_MAX_K) return fail(MXFP8_ERR_INVALID_ARG, "%s: K above %d", me, MXFP8_ROUTER_MAX_K);
  if (T > MOE_TOKENS_FWD_MAX_TOKENS)
    return fail(MXFP8_ERR_UNSUPPORTED, "%s: more than %d tokens (moe_fwd_mxfp8 takes any number, over block lists)", me,
                MOE_TOKENS_FWD_MAX_TOKENS);
  // an expert's weight rows are read through one buffer, at 32-bit offsets
  if (I > INT32_MAX / 2 / H || H > (int64_t(1) << 22) || I > (int64_t(1) << 22) || E > MXFP8_ROUTER_MAX_EXPERTS ||
      T * K * I > INT32_MAX)
    return fail(MXFP8_ERR_UNSUPPORTED, "%s: more than %d experts, or sizes beyond 32-bit indexing", me,
                MXFP8_ROUTER_MAX_EXPERTS);
  return MXFP8_OK;
}

static void tokens_layout(const moe_tokens_fwd_mxfp8_args* a, TokLayout* L) {
  const int64_t T = a->T, H = a->H, I = a->I, M = T * a->K;
  size_t o = 0;
  auto put = [&](size_t& field, int64_t bytes) {
    field = o;
    o = up256(o + size_t(bytes));
  };
  const bool few = mx::tokens_few(T);
  put(L->x_codes, few ? 0 : T * H);
  put(L->x_scales, few ? 0 : T * H / 32);
  put(L->units, few ? 0 : (1 + 3 * mx::tokens_units(T, a->E, a->K)) * 4);
  put(L->list, few ? 0 : M * 4);
  put(L->done, few ? (H + 63) / 64 * 4 : 0);
  put(L->s_codes, M * I);
  put(L->s_scales, M * I / 32);
  put(L->rows, (M ? mx::tokens_splits(T, H, I, a->E, a->K) : 0) * M * H * 4);
  L->total = o;
}

size_t moe_tokens_fwd_mxfp8_workspace_size(const moe_tokens_fwd_mxfp8_args* a) {
  if (tokens_check_shapes(a)) return 0;
  TokLayout L;
  tokens_layout(a, &L);
  return L.total;
}

int moe_tokens_fwd_mxfp8(const moe_tokens_fwd_mxfp8_args* a, void* ws, size_t ws_bytes, void* stream) {
  const char* me = "moe_tokens_fwd_mxfp8";
  int rc = tokens_check_shapes(a);
  if (rc) return rc;
  if (a->affinity_on != 0 && a->affinity_on != 1)
    return fail(MXFP8_ERR_INVALID_ARG, "%s: affinity_on must be 0 (H) or 1 (I)", me);
  if (a->activation != MXFP8_ACT_SWIGLU && a->activation != MXFP8_ACT_GEGLU)
    return fail(MXFP8_ERR_INVALID_ARG, "%s: activation must be 0 (SwiGLU) or 1 (GeGLU)", me);
  if (a->affinity_on == 1 && (a->gate_up_proj_bias || a->down_proj_bias))
    return fail(MXFP8_ERR_UNSUPPORTED, "%s: a bias with the affinity on I is not supported", me);
  if (a->T == 0) return ok();
  const void* req[] = {a->hidden_states, a->topk_idx, a->topk_scores, a->gate_up_codes, a->gate_up_scales,
                       a->down_codes, a->down_scales, a->output_hidden_states};
  const void* opt[] = {a->gate_up_proj_bias, a->down_proj_bias, a->residual};
  for (const void* q : req)
    if (!q) return fail(MXFP8_ERR_INVALID_ARG, "%s: a required pointer is null", me);
  for (const void* q : req)
    if (!aligned16(q)) return fail(MXFP8_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", me);
  for (const void* q : opt)
    if (!aligned16(q)) return fail(MXFP8_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", me);
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u))
    return fail(MXFP8_ERR_INVALID_ARG, "%s: workspace must be non-null and 256-byte aligned", me);
  TokLayout L;
  tokens_layout(a, &L);
  if (ws_bytes < L.total) return fail(MXFP8_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", me, ws_bytes, L.total);
  uint8_t* w = static_cast<uint8_t*>(ws);
  mx::MoeTokensArgs p{};
  p.T = a->T; p.H = a->H; p.I = a->I; p.E = a->E; p.K = a->K;
  p.idx = a->topk_idx; p.scores = a->topk_scores;
  p.x = a->hidden_states;
  p.x_codes = w + L.x_codes; p.x_scales = w + L.x_scales;
  p.units = reinterpret_cast<int32_t*>(w + L.units); p.list = reinterpret_cast<int32_t*>(w + L.list);
  p.done = reinterpret_cast<unsigned*>(w + L.done);
  p.w_codes = a->gate_up_codes; p.w_scales = a->gate_up_scales;
  p.wd_codes = a->down_codes; p.wd_scales = a->down_scales;
  p.b1 = a->gate_up_proj_bias; p.b2 = a->down_proj_bias;
  p.s_codes = w + L.s_codes; p.s_scales = w + L.s_scales;
  p.rows = reinterpret_cast<float*>(w + L.rows);
  p.residual = a->residual; p.out = a->output_hidden_states;
  p.geglu = a->activation == MXFP8_ACT_GEGLU; p.on_i = a->affinity_on;
  p.splits = int(mx::tokens_splits(a->T, a->H, a->I, a->E, a->K));
  return hip_status(mx::launch_moe_tokens(p, static_cast<hipStream_t>(stream)), me);
}

}  // extern "C"
