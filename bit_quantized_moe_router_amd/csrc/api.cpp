// C ABI entry points: argument validation, workspace layout, dispatch.
// Every check below happens before anything is enqueued on the stream.
#include <cmath>
#include <cstdint>
#include <cstring>

#include "moe_internal.h"

namespace bqmoe {

static size_t al256(size_t x) { return (x + 255) & ~size_t(255); }

static bool layer_ok(const moe_layer* L) {
  if (!L) return false;
  if (L->d <= 0 || L->inter <= 0 || L->d % 128 || L->inter % 128 || L->d > MOE_MAX_DIM ||
      L->inter > MOE_MAX_DIM)
    return false;
  if (L->n_experts < 1 || L->n_experts > MOE_MAX_EXPERTS) return false;
  if (L->top_k < 1 || L->top_k > MOE_MAX_TOPK || L->top_k > L->n_experts) return false;
  if (L->n_shared < 0 || L->n_shared > 1) return false;
  if (!qtype_levels(L->q_gate) || !qtype_levels(L->q_up) || !qtype_levels(L->q_down)) return false;
  return true;
}

DecodeWs decode_ws_layout(const moe_layer* L, int T) {
  DecodeWs w{};
  const int k = L->top_k, d = L->d, I = L->inter, S = L->n_shared;
  w.max_slots = (T * k < L->n_experts ? T * k : L->n_experts) + S;
  w.rows = T * k + T * S;
  size_t o = 0;
  w.slots = o;
  o = al256(o + sizeof(int32_t) * kSlotRec * (1 + (size_t)w.max_slots));
  w.xs = o;
  o = al256(o + 2 * (size_t)T * d);
  w.xsum = o;
  o = al256(o + 16 * (size_t)T * (d / 32));
  w.hs = o;
  o = al256(o + 2 * (size_t)w.rows * I);
  w.hsum = o;
  o = al256(o + 16 * (size_t)w.rows * (I / 32));
  w.y = o;
  o = al256(o + 2 * (size_t)w.rows * d);
  w.total = o;
  return w;
}

PrefillWs prefill_ws_layout(const moe_layer* L, int T) {
  PrefillWs p{};
  const int k = L->top_k, d = L->d, I = L->inter, S = L->n_shared, E = L->n_experts;
  p.nblk = (T + kHistTokensPerBlock - 1) / kHistTokensPerBlock;
  const size_t rows_routed = (size_t)T * k;
  p.rows = (int)(rows_routed + (size_t)T * S);
  const size_t tm = (size_t)prefill_tile_rows(L);
  p.max_tiles = (int)(rows_routed / tm + (size_t)E + (S ? ((size_t)T + tm - 1) / tm : 0));
  size_t o = 0;
  p.ctrl = o;
  o = al256(o + 64);
  p.hist = o;
  o = al256(o + sizeof(int32_t) * (size_t)p.nblk * E);
  p.lrank = o;
  o = al256(o + sizeof(int32_t) * rows_routed);
  p.tiles = o;
  o = al256(o + sizeof(int32_t) * 4 * (size_t)p.max_tiles);
  p.xs = o;
  o = al256(o + 2 * (size_t)T * d);
  p.xsum = o;
  o = al256(o + 16 * (size_t)T * (d / 32));
  p.h = o;
  o = al256(o + 2 * (size_t)p.rows * I);
  p.hsum = o;
  o = al256(o + 16 * (size_t)p.rows * (I / 32));
  p.y = o;
  o = al256(o + 2 * (size_t)p.rows * d);
  p.x6 = o;
  o = al256(o + (size_t)T * d);
  p.h6 = o;
  o = al256(o + (size_t)p.rows * I);
  p.total = o;
  return p;
}

// The routing by scores keeps the tile list where PrefillWs has it and its own
// scratch behind it, in regions that the layer fills after routing.
static size_t scored_ws_need(const moe_layer* L, int T) {
  return prefill_ws_layout(L, T).xs + scored_ws_bytes(L, T);
}

// what moe_route_topk and the forward calls need
static size_t base_ws_need(const moe_layer* L, int T) {
  size_t b = prefill_ws_layout(L, T).total;
  if (T <= MOE_MAX_DECODE_TOKENS) {
    const size_t dcd = decode_ws_layout(L, T).total;
    if (dcd > b) b = dcd;
  }
  return b;
}

static bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + nb && y < x + na;
}

static bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// shared checks for the calls that take routing buffers
// (ws_need: the workspace bytes the call requires; 0 = base_ws_need(L, T))
static moe_status check_common(const moe_layer* L, const uint16_t* x, int32_t T, uint32_t flags,
                               const moe_routing* R, const void* ws, size_t ws_bytes,
                               bool need_experts, size_t ws_need = 0) {
  if (!layer_ok(L)) {
    if (!L) return MOE_ERR_INVALID_ARG;
    // distinguish plain invalid values from unsupported-but-meaningful shapes
    if (L->d <= 0 || L->inter <= 0 || L->n_experts <= 0 || L->top_k <= 0 ||
        L->top_k > L->n_experts || L->n_shared < 0 || L->n_shared > 1)
      return MOE_ERR_INVALID_ARG;
    return MOE_ERR_UNSUPPORTED;
  }
  if (T < 0) return MOE_ERR_INVALID_ARG;
  if (flags & ~(uint32_t)(MOE_LOGITS_GIVEN | MOE_ADD_RESIDUAL)) return MOE_ERR_INVALID_ARG;
  if ((int64_t)T * L->top_k > (int64_t)1 << 30) return MOE_ERR_UNSUPPORTED;
  if (!R || !R->logits || !R->topk_ids || !R->topk_w || !R->counts || !R->offsets ||
      !R->perm_tok || !R->inv_row)
    return MOE_ERR_INVALID_ARG;
  if (!(flags & MOE_LOGITS_GIVEN)) {
    if (!L->router_w || !x) return MOE_ERR_INVALID_ARG;
  }
  if (need_experts) {
    const size_t eb = moe_expert_bytes(L->q_gate, L->q_up, L->q_down, L->d, L->inter);
    if (!x || !L->experts || L->expert_stride < eb || L->expert_stride % 256 ||
        !aligned(L->experts, 256))
      return MOE_ERR_INVALID_ARG;
    if (L->n_shared && (!L->shared || !aligned(L->shared, 256))) return MOE_ERR_INVALID_ARG;
    if (!aligned(x, 16)) return MOE_ERR_INVALID_ARG;
    if (L->alt_experts) {  // the second copy of the routed experts
      const size_t ab =
          moe_expert_bytes(L->q_alt_gate, L->q_alt_up, L->q_alt_down, L->d, L->inter);
      if (!ab) return MOE_ERR_UNSUPPORTED;  // a code family outside the three
      if (!L->alt_select || L->alt_stride < ab || L->alt_stride % 256 ||
          !aligned(L->alt_experts, 256))
        return MOE_ERR_INVALID_ARG;
    }
  }
  if (!ws) return MOE_ERR_WORKSPACE;
  if (T > 0 && ws_bytes < (ws_need ? ws_need : base_ws_need(L, T))) return MOE_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

}  // namespace bqmoe

using namespace bqmoe;

extern "C" size_t moe_workspace_bytes(const moe_layer* L, int32_t T) {
  if (!layer_ok(L) || T < 0) return 0;
  if (T == 0) return 256;
  const size_t b = base_ws_need(L, T), s = scored_ws_need(L, T);
  return b > s ? b : s;
}

extern "C" moe_status moe_route_topk(const moe_layer* L, const uint16_t* x, int32_t T,
                                     uint32_t flags, moe_routing* R, void* ws, size_t ws_bytes,
                                     void* stream) {
  if (T == 0 && L && R) return MOE_OK;
  moe_status st = check_common(L, x, T, flags, R, ws, ws_bytes, false);
  if (st != MOE_OK) return st;
  const PrefillWs P = prefill_ws_layout(L, T);
  return launch_route_generic(L, x, T, flags, R, (uint8_t*)ws, P, stream) ? MOE_ERR_DEVICE
                                                                         : MOE_OK;
}

namespace bqmoe {
// decode_ws_only: the workspace need only hold the decode layout (the
// no-allocation entry point's fixed array), not moe_workspace_bytes
static moe_status check_decode(const moe_layer* L, const uint16_t* x, int32_t T, uint32_t flags,
                               const moe_routing* R, const void* ws, size_t ws_bytes,
                               const uint16_t* out, bool decode_ws_only) {
  if (T < 1 || T > MOE_MAX_DECODE_TOKENS) return MOE_ERR_INVALID_ARG;
  if (decode_ws_only && !layer_ok(L)) return L ? MOE_ERR_UNSUPPORTED : MOE_ERR_INVALID_ARG;
  const size_t need = decode_ws_only ? decode_ws_layout(L, T).total : 0;
  moe_status st = check_common(L, x, T, flags, R, ws, ws_bytes, true, need);
  if (st != MOE_OK) return st;
  if (T * L->top_k > kDecodeMaxRoutedRows || T * (L->top_k + L->n_shared) > kDecodeMaxRows ||
      L->d > kDecodeMaxDim || L->inter > kDecodeMaxDim || !decode_shape_ok(L, T))
    return MOE_ERR_UNSUPPORTED;
  if (!out || !aligned(out, 16)) return MOE_ERR_INVALID_ARG;
  const size_t bytes = (size_t)T * L->d * 2;
  if (overlaps(x, bytes, out, bytes)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status decode_call(const moe_layer* L, const uint16_t* x, int32_t T, uint32_t flags,
                       moe_routing* R, void* ws, size_t ws_bytes, uint16_t* out, uint32_t mask,
                       void* stream, bool decode_ws_only) {
  const moe_status st = check_decode(L, x, T, flags, R, ws, ws_bytes, out, decode_ws_only);
  if (st != MOE_OK) return st;
  const DecodeWs W = decode_ws_layout(L, T);
  return launch_decode(L, x, T, flags, R, (uint8_t*)ws, W, out, stream, mask) ? MOE_ERR_DEVICE
                                                                            : MOE_OK;
}

// ws_need as in check_common
static moe_status check_prefill(const moe_layer* L, const uint16_t* x, int32_t T, uint32_t flags,
                                const moe_routing* R, const void* ws, size_t ws_bytes,
                                const uint16_t* out, size_t ws_need) {
  moe_status st = check_common(L, x, T, flags, R, ws, ws_bytes, true, ws_need);
  if (st != MOE_OK) return st;
  if (L->alt_experts) return MOE_ERR_UNSUPPORTED;  // the second expert copy is read by decode
  if (L->d % 256) return MOE_ERR_UNSUPPORTED;  // the down GEMMs cover 256 columns per block
  if (!out || !aligned(out, 16)) return MOE_ERR_INVALID_ARG;
  const size_t bytes = (size_t)T * L->d * 2;
  if (overlaps(x, bytes, out, bytes)) return MOE_ERR_INVALID_ARG;
  const PrefillWs P = prefill_ws_layout(L, T);
  // the 2-bit and ternary kernels address their activation rows with 32-bit byte offsets
  if ((prefill_x2(L) || prefill_exact16(L)) && (size_t)P.rows * (size_t)(L->d > L->inter ? L->d : L->inter) * 2 >
                           (size_t)UINT32_MAX)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
}  // namespace bqmoe

static moe_status decode_impl(const moe_layer* L, const uint16_t* x, int32_t T, uint32_t flags,
                              moe_routing* R, void* ws, size_t ws_bytes, uint16_t* out,
                              uint32_t mask, void* stream) {
  return decode_call(L, x, T, flags, R, ws, ws_bytes, out, mask, stream, false);
}

static moe_status prefill_impl(const moe_layer* L, const uint16_t* x, int32_t T, uint32_t flags,
                               moe_routing* R, void* ws, size_t ws_bytes, uint16_t* out,
                               uint32_t mask, void* stream) {
  if (T == 0 && L && R) return MOE_OK;
  const moe_status st = check_prefill(L, x, T, flags, R, ws, ws_bytes, out, 0);
  if (st != MOE_OK) return st;
  const PrefillWs P = prefill_ws_layout(L, T);
  return launch_prefill(L, x, T, flags, R, (uint8_t*)ws, P, out, stream, mask) ? MOE_ERR_DEVICE
                                                                             : MOE_OK;
}

extern "C" moe_status moe_forward_decode(const moe_layer* L, const uint16_t* x, int32_t T,
                                         uint32_t flags, moe_routing* R, void* ws,
                                         size_t ws_bytes, uint16_t* out, void* stream) {
  return decode_impl(L, x, T, flags, R, ws, ws_bytes, out, ~0u, stream);
}

extern "C" moe_status moe_forward_prefill(const moe_layer* L, const uint16_t* x, int32_t T,
                                          uint32_t flags, moe_routing* R, void* ws,
                                          size_t ws_bytes, uint16_t* out, void* stream) {
  return prefill_impl(L, x, T, flags, R, ws, ws_bytes, out, ~0u, stream);
}

extern "C" moe_status moe_forward_decode_stages(const moe_layer* L, const uint16_t* x, int32_t T,
                                                uint32_t flags, moe_routing* R, void* ws,
                                                size_t ws_bytes, uint16_t* out,
                                                uint32_t stage_mask, void* stream) {
  if (stage_mask == 0 || (stage_mask & ~(uint32_t)MOE_DECODE_STAGES_ALL)) return MOE_ERR_INVALID_ARG;
  return decode_impl(L, x, T, flags, R, ws, ws_bytes, out, stage_mask, stream);
}

extern "C" moe_status moe_forward_prefill_stages(const moe_layer* L, const uint16_t* x, int32_t T,
                                                 uint32_t flags, moe_routing* R, void* ws,
                                                 size_t ws_bytes, uint16_t* out,
                                                 uint32_t stage_mask, void* stream) {
  if (stage_mask == 0 || (stage_mask & ~(uint32_t)MOE_PREFILL_STAGES_ALL)) return MOE_ERR_INVALID_ARG;
  return prefill_impl(L, x, T, flags, R, ws, ws_bytes, out, stage_mask, stream);
}

// ------------------------------------------------------- routing by scores
namespace bqmoe {
static bool scoring_ok(const moe_layer* L, const moe_scoring* S) {
  if (!L || !S || L->n_experts < 1 || L->top_k < 1) return false;
  if (S->score != MOE_SCORE_SOFTMAX && S->score != MOE_SCORE_SIGMOID) return false;
  if (S->n_groups < 1 || S->n_groups > MOE_MAX_GROUPS || L->n_experts % S->n_groups) return false;
  const int gs = L->n_experts / S->n_groups;
  if (S->topk_groups < 1 || S->topk_groups > S->n_groups) return false;
  if (S->group_top < 1 || S->group_top > 2 || S->group_top > gs) return false;
  if ((int64_t)S->topk_groups * gs < L->top_k) return false;
  if (S->renorm != 0 && S->renorm != 1) return false;
  return std::isfinite(S->scale) && aligned(S->choice_bias, 4);
}

// the scored routing on logits that are in R already; tiles: the grouped GEMMs' list too
static int route_scored(const moe_layer* L, const moe_scoring* S, int T, moe_routing* R,
                        uint8_t* ws, bool tiles, void* stream) {
  const PrefillWs P = prefill_ws_layout(L, T);
  ScoreOut O{};
  O.n_shared = L->n_shared;
  if (tiles) {
    O.tiles = (int32_t*)(ws + P.tiles);
    O.ctrl = (int32_t*)(ws + P.ctrl);
    O.tm = prefill_tile_rows(L);
  }
  return launch_route_scored(L, S, T, R, ws + P.xs, O, stream);
}
}  // namespace bqmoe

extern "C" moe_status moe_route_scored(const moe_layer* L, const moe_scoring* S, const uint16_t* x,
                                       int32_t T, uint32_t flags, moe_routing* R, void* ws,
                                       size_t ws_bytes, void* stream) {
  if (!scoring_ok(L, S)) return MOE_ERR_INVALID_ARG;
  if (T == 0 && R) return MOE_OK;
  const size_t need = layer_ok(L) && T > 0 ? scored_ws_need(L, T) : 0;
  const moe_status st = check_common(L, x, T, flags, R, ws, ws_bytes, false, need);
  if (st != MOE_OK) return st;
  if (!(flags & MOE_LOGITS_GIVEN) && launch_router_logits(L, x, T, R, stream))
    return MOE_ERR_DEVICE;
  return route_scored(L, S, T, R, (uint8_t*)ws, false, stream) ? MOE_ERR_DEVICE : MOE_OK;
}

extern "C" moe_status moe_forward_decode_scored(const moe_layer* L, const moe_scoring* S,
                                                const uint16_t* x, int32_t T, uint32_t flags,
                                                moe_routing* R, void* ws, size_t ws_bytes,
                                                uint16_t* out, void* stream) {
  if (!scoring_ok(L, S)) return MOE_ERR_INVALID_ARG;
  const moe_status st = check_decode(L, x, T, flags, R, ws, ws_bytes, out, false);
  if (st != MOE_OK) return st;
  const DecodeWs W = decode_ws_layout(L, T);
  uint8_t* w = (uint8_t*)ws;
  if (launch_decode_route(L, x, T, flags, R, w, W, stream, MOE_DECODE_STAGE_ROUTE))
    return MOE_ERR_DEVICE;
  ScoreOut O{};
  O.n_shared = L->n_shared;
  O.slots = (int32_t*)(w + W.slots);
  O.max_slots = W.max_slots;
  O.alt_select = L->alt_experts ? L->alt_select : nullptr;
  if (launch_route_scored(L, S, T, R, nullptr, O, stream)) return MOE_ERR_DEVICE;
  return launch_decode(L, x, T, flags, R, w, W, out, stream,
                       MOE_DECODE_STAGE_GATEUP | MOE_DECODE_STAGE_DOWN, true)
             ? MOE_ERR_DEVICE
             : MOE_OK;
}

extern "C" moe_status moe_forward_prefill_scored(const moe_layer* L, const moe_scoring* S,
                                                 const uint16_t* x, int32_t T, uint32_t flags,
                                                 moe_routing* R, void* ws, size_t ws_bytes,
                                                 uint16_t* out, void* stream) {
  if (!scoring_ok(L, S)) return MOE_ERR_INVALID_ARG;
  if (T == 0 && R) return MOE_OK;
  const size_t need = layer_ok(L) && T > 0 ? moe_workspace_bytes(L, T) : 0;
  const moe_status st = check_prefill(L, x, T, flags, R, ws, ws_bytes, out, need);
  if (st != MOE_OK) return st;
  if (!(flags & MOE_LOGITS_GIVEN) && launch_router_logits(L, x, T, R, stream))
    return MOE_ERR_DEVICE;
  if (route_scored(L, S, T, R, (uint8_t*)ws, true, stream)) return MOE_ERR_DEVICE;
  return launch_prefill(L, x, T, flags, R, (uint8_t*)ws, prefill_ws_layout(L, T), out, stream,
                        MOE_PREFILL_STAGES_ALL & ~(uint32_t)MOE_PREFILL_STAGE_ROUTE)
             ? MOE_ERR_DEVICE
             : MOE_OK;
}

// ----------------------------------------------------------- dense product
namespace bqmoe {
static bool linear_ok(const moe_linear* P) {
  return P && P->K > 0 && P->N > 0 && P->act >= MOE_ACT_NONE && P->act <= MOE_ACT_SIGMOID;
}
static bool linear_supported(const moe_linear* P) {
  return P->K <= MOE_MAX_DIM && P->N <= MOE_MAX_DIM && format_shape_ok(P->qtype, P->K, P->N);
}
constexpr int64_t kLinMaxStride = MOE_MAX_LINEAR_STRIDE;
// a [T][width] operand of 16-byte aligned rows
static bool rows_ok(const void* p, int64_t ld, int64_t width) {
  return aligned(p, 16) && ld >= width && ld % 8 == 0;
}
static size_t rows_bytes(int32_t T, int64_t ld, int64_t width) {
  return ((size_t)(T - 1) * (size_t)ld + (size_t)width) * 2;
}
}  // namespace bqmoe

extern "C" size_t moe_linear_workspace_bytes(const moe_linear* P, int32_t T) {
  if (!linear_ok(P) || !linear_supported(P) || T < 0) return 0;
  return lin_ws_bytes(P->K, P->N, T);
}

extern "C" moe_status moe_linear_forward(const moe_linear* P, const uint16_t* x, int64_t x_stride,
                                         int32_t T, const uint16_t* mul, int64_t mul_stride,
                                         const uint16_t* residual, int64_t residual_stride,
                                         uint16_t* out, int64_t out_stride, void* ws,
                                         size_t ws_bytes, void* stream) {
  if (!linear_ok(P)) return MOE_ERR_INVALID_ARG;
  if (!linear_supported(P)) return MOE_ERR_UNSUPPORTED;
  if (T < 0) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (T > MOE_MAX_LINEAR_ROWS || x_stride > kLinMaxStride || out_stride > kLinMaxStride ||
      (mul && mul_stride > kLinMaxStride) || (residual && residual_stride > kLinMaxStride))
    return MOE_ERR_UNSUPPORTED;
  if (!P->w || !aligned(P->w, 256) || !aligned(P->bias, 4)) return MOE_ERR_INVALID_ARG;
  if (!x || !rows_ok(x, x_stride, P->K)) return MOE_ERR_INVALID_ARG;
  if (mul && !rows_ok(mul, mul_stride, P->N)) return MOE_ERR_INVALID_ARG;
  if (residual && !rows_ok(residual, residual_stride, P->N)) return MOE_ERR_INVALID_ARG;
  if (!out || !rows_ok(out, out_stride, P->N)) return MOE_ERR_INVALID_ARG;
  // out may be mul or residual itself (each value is read before it is
  // written, by the same thread), but not x, nor either of them shifted
  const size_t ob = rows_bytes(T, out_stride, P->N);
  if (overlaps(x, rows_bytes(T, x_stride, P->K), out, ob)) return MOE_ERR_INVALID_ARG;
  if (mul && !(mul == out && mul_stride == out_stride) &&
      overlaps(mul, rows_bytes(T, mul_stride, P->N), out, ob))
    return MOE_ERR_INVALID_ARG;
  if (residual && !(residual == out && residual_stride == out_stride) &&
      overlaps(residual, rows_bytes(T, residual_stride, P->N), out, ob))
    return MOE_ERR_INVALID_ARG;
  const size_t need = lin_ws_need(P->K, P->N, T);
  if (need && (!ws || ws_bytes < need)) return MOE_ERR_WORKSPACE;
  if (need && (!aligned(ws, 256) || overlaps(ws, need, out, ob) ||
               overlaps(ws, need, x, rows_bytes(T, x_stride, P->K)) ||
               (mul && overlaps(ws, need, mul, rows_bytes(T, mul_stride, P->N))) ||
               (residual && overlaps(ws, need, residual, rows_bytes(T, residual_stride, P->N)))))
    return MOE_ERR_INVALID_ARG;
  const PackedLayout pl = packed_layout(P->qtype, P->K, P->N);
  const LinArgs A = {(const uint8_t*)P->w, pl.plane1, pl.scales, P->bias,  x,
                     mul,                  residual,  out,       x_stride, mul_stride,
                     residual_stride,      out_stride, P->K,     P->N,     P->qtype,
                     P->act};
  return launch_linear(A, T, (uint8_t*)ws, stream) ? MOE_ERR_DEVICE : MOE_OK;
}

extern "C" const char* moe_status_string(moe_status s) {
  switch (s) {
    case MOE_OK: return "ok";
    case MOE_ERR_INVALID_ARG: return "invalid argument";
    case MOE_ERR_UNSUPPORTED: return "unsupported shape or type";
    case MOE_ERR_WORKSPACE: return "workspace too small";
    case MOE_ERR_BAD_CODES: return "level index outside its alphabet";
    case MOE_ERR_DEVICE: return "HIP launch or runtime error";
  }
  return "unknown status";
}

extern "C" int moe_abi_version(void) { return 3; }
