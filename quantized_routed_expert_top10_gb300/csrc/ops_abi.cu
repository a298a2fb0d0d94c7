// C ABI of the operators at the block's edges (declared in include/strata_moe_ops.h): argument checks
// and the launch of each call.
#include <cmath>

#include "ops_common.cuh"

using namespace strata;

namespace {

constexpr int64_t STRIDE_MAX = int64_t(1) << 40;  // elements: T * stride * 4 bytes stays far inside 64 bits

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline bool known_type(int32_t t) { return t == STRATA_F32 || t == STRATA_BF16 || t == STRATA_F16; }
inline int64_t type_bytes(int32_t t) { return t == STRATA_F32 ? 4 : 2; }
inline bool good_stride(int64_t s, int64_t least) { return s >= least && s <= STRIDE_MAX; }
inline bool good_T(int32_t T) { return T >= 0 && T <= TMAX; }
inline bool flag(int32_t v) { return v == 0 || v == 1; }

// An operand: `rows` rows of `bytes` bytes, `step` >= bytes apart.
struct Rows {
  const char* p;  // null: no operand
  int64_t rows, step, bytes;
  int32_t type;
};
Rows rows_of(const void* p, int64_t rows, int64_t stride, int64_t n, int32_t type) {
  if (!p) return Rows{};  // its stride is not looked at
  return Rows{(const char*)p, rows, stride * type_bytes(type), n * type_bytes(type), type};
}
// a / b rounded down, b > 0
int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0 ? 1 : 0); }

// Some row of a and some row of b share a byte.  (Rows of one may lie between those of the other, as column ranges of one
// buffer do.)
bool overlap(const Rows& a, const Rows& b) {
  if (!a.p || !b.p) return false;
  const int64_t d = (int64_t)((uintptr_t)b.p - (uintptr_t)a.p);
  if (d >= (a.rows - 1) * a.step + a.bytes || -d >= (b.rows - 1) * b.step + b.bytes) return false;
  // row j of b begins d + j b.step - i a.step behind row i of a; they meet if that is in (-b.bytes, a.bytes)
  if (a.step == b.step) {  // j - i alone counts, and of its values only the two around -d / step come near enough
    const int64_t k = floor_div(-d, a.step);
    for (int64_t c = k; c <= k + 1; ++c)
      if (c > -a.rows && c < b.rows && d + c * a.step > -b.bytes && d + c * a.step < a.bytes) return true;
    return false;
  }
  for (int64_t i = 0; i < a.rows; ++i) {
    const int64_t at = i * a.step - d;                       // row i of a, from b's start
    const int64_t j = floor_div(at - b.bytes, b.step) + 1;  // the first row of b that ends behind it
    const int64_t first = j > 0 ? j : 0;
    if (first < b.rows && first * b.step < at + a.bytes) return true;
  }
  return false;
}
// Overlapping, and not the same array: a call may write an array that it reads row by row.
bool partly(const Rows& a, const Rows& b) {
  return overlap(a, b) && !(a.p == b.p && a.step == b.step && a.type == b.type);
}

inline strata_status launched(cudaError_t e) { return e == cudaSuccess ? STRATA_OK : STRATA_E_CUDA; }

}  // namespace

extern "C" {

strata_status strata_moe_select(const strata_select_t* sel, const void* logits, int32_t T, const float* bias,
                                int32_t* ids, float* weights, void* stream) {
  if (!sel || !good_T(T) || !logits || !ids || !weights) return STRATA_E_INVAL;
  const int E = sel->n_expert, G = sel->n_group;
  if (E < 1 || E > EMAX || G < 1 || G > STRATA_SELECT_GROUP_MAX || E % G != 0) return STRATA_E_INVAL;
  if (sel->top_group < 1 || sel->top_group > G || (sel->group_sum != 1 && sel->group_sum != 2)) return STRATA_E_INVAL;
  if (sel->top_k < 1 || sel->top_k > STRATA_SELECT_K_MAX || sel->top_k > sel->top_group * (E / G)) return STRATA_E_INVAL;
  if (sel->score != STRATA_SCORE_SOFTMAX && sel->score != STRATA_SCORE_SIGMOID) return STRATA_E_INVAL;
  if (!flag(sel->renorm) || !std::isfinite(sel->scale) || !known_type(sel->logits_type) || sel->reserved != 0)
    return STRATA_E_INVAL;
  if (!good_stride(sel->logits_stride, E)) return STRATA_E_INVAL;
  if (!aligned(logits, type_bytes(sel->logits_type)) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
    return STRATA_E_ALIGN;
  if (T == 0) return STRATA_OK;
  const Rows sl = rows_of(logits, T, sel->logits_stride, E, sel->logits_type);
  const Rows si = rows_of(ids, T, sel->top_k, sel->top_k, STRATA_F32), sw = rows_of(weights, T, sel->top_k, sel->top_k, STRATA_F32);
  if (overlap(sl, si) || overlap(sl, sw) || overlap(si, sw)) return STRATA_E_INVAL;
  return launched(launch_select(*sel, logits, T, bias, ids, weights, (cudaStream_t)stream));
}

strata_status strata_moe_norm(const strata_norm_t* nd, const void* x, int32_t T, const float* gain, void* out,
                              void* stream) {
  if (!nd || !good_T(T) || !x || !out) return STRATA_E_INVAL;
  const int n = nd->n;
  if (n < 1 || n > STRATA_NORM_N_MAX || !std::isfinite(nd->eps) || nd->eps < 0.f) return STRATA_E_INVAL;
  if (!known_type(nd->x_type) || !known_type(nd->out_type)) return STRATA_E_INVAL;
  if (!good_stride(nd->x_stride, n) || !good_stride(nd->out_stride, n)) return STRATA_E_INVAL;
  if (!aligned(x, type_bytes(nd->x_type)) || !aligned(out, type_bytes(nd->out_type)) || !aligned(gain, 4))
    return STRATA_E_ALIGN;
  if (T == 0) return STRATA_OK;
  if (partly(rows_of(x, T, nd->x_stride, n, nd->x_type), rows_of(out, T, nd->out_stride, n, nd->out_type)))
    return STRATA_E_INVAL;
  return launched(launch_norm(*nd, x, T, gain, out, (cudaStream_t)stream));
}

strata_status strata_moe_combine_norm(const strata_combine_norm_t* cn, const void* parts, const float* part_weights,
                                      const void* x, int32_t T, const float* post_gain, const float* channel_gate,
                                      const float* token_gate, const float* pre_gain, void* out, void* next,
                                      void* stream) {
  if (!cn || !good_T(T) || !parts || (!out && !next)) return STRATA_E_INVAL;
  const int n = cn->n, P = cn->n_part;
  if (n < 1 || n > STRATA_NORM_N_MAX || P < 1 || P > STRATA_NORM_PART_MAX) return STRATA_E_INVAL;
  if (cn->flags & ~(STRATA_POST_NORM | STRATA_TOKEN_SIGMOID) || cn->reserved != 0) return STRATA_E_INVAL;
  if (!std::isfinite(cn->eps) || cn->eps < 0.f || !std::isfinite(cn->residual_scale) || !std::isfinite(cn->block_scale))
    return STRATA_E_INVAL;
  if (!known_type(cn->part_type) || !known_type(cn->x_type) || !known_type(cn->next_type)) return STRATA_E_INVAL;
  // a gain or a sigmoid that nothing would apply is a mistake of the caller's
  if ((post_gain && !(cn->flags & STRATA_POST_NORM)) || ((cn->flags & STRATA_TOKEN_SIGMOID) && !token_gate) ||
      (pre_gain && !next))
    return STRATA_E_INVAL;
  if (!good_stride(cn->part_stride, n) || cn->part_stride > STRIDE_MAX / STRATA_NORM_PART_MAX ||
      !good_stride(cn->token_stride, (P - 1) * cn->part_stride + n))
    return STRATA_E_INVAL;
  if ((x && !good_stride(cn->x_stride, n)) || (out && !good_stride(cn->out_stride, n)) ||
      (next && !good_stride(cn->next_stride, n)))
    return STRATA_E_INVAL;
  if (!aligned(parts, type_bytes(cn->part_type)) || !aligned(x, type_bytes(cn->x_type)) ||
      !aligned(out, type_bytes(cn->x_type)) || !aligned(next, type_bytes(cn->next_type)) || !aligned(part_weights, 4) ||
      !aligned(post_gain, 4) || !aligned(channel_gate, 4) || !aligned(token_gate, 4) || !aligned(pre_gain, 4))
    return STRATA_E_ALIGN;
  if (T == 0) return STRATA_OK;
  const Rows sx = rows_of(x, T, cn->x_stride, n, cn->x_type), so = rows_of(out, T, cn->out_stride, n, cn->x_type);
  const Rows sn = rows_of(next, T, cn->next_stride, n, cn->next_type);
  if (overlap(so, sn) || partly(sx, so) || partly(sx, sn)) return STRATA_E_INVAL;
  for (int k = 0; k < P; ++k) {
    const char* p = (const char*)parts + k * cn->part_stride * type_bytes(cn->part_type);
    const Rows sp = rows_of(p, T, cn->token_stride, n, cn->part_type);
    if (overlap(sp, so) || overlap(sp, sn)) return STRATA_E_INVAL;
  }
  return launched(launch_combine_norm(*cn, parts, part_weights, x, T, post_gain, channel_gate, token_gate, pre_gain, out,
                                      next, (cudaStream_t)stream));
}

strata_status strata_moe_adapters(const strata_adapters_t* ad, const int32_t* seg_off, const int32_t* seg_adapter,
                                  int32_t n_seg, const void* x, int32_t T, const void* base, void* y, void* ws,
                                  size_t ws_bytes, void* stream) {
  if (!ad || !good_T(T) || n_seg < 0 || n_seg > TMAX || !seg_off || !x || !y || !ws) return STRATA_E_INVAL;
  if (n_seg > 0 && !seg_adapter) return STRATA_E_INVAL;
  if (!ad->a || !ad->b || ad->n_adapter < 1 || ad->n_adapter > STRATA_ADAPTER_COUNT_MAX) return STRATA_E_INVAL;
  if (ad->rank < 8 || ad->rank > STRATA_ADAPTER_RANK_MAX || ad->rank % 8 != 0) return STRATA_E_INVAL;
  if (ad->d_in < 8 || ad->d_in > STRATA_ADAPTER_DIM_MAX || ad->d_in % 8 != 0) return STRATA_E_INVAL;
  if (ad->d_out < 8 || ad->d_out > STRATA_ADAPTER_DIM_MAX || ad->d_out % 8 != 0) return STRATA_E_INVAL;
  if (!known_type(ad->x_type) || !known_type(ad->y_type)) return STRATA_E_INVAL;
  const int64_t na = (int64_t)ad->rank * ad->d_in, nb = (int64_t)ad->rank * ad->d_out;
  if (!good_stride(ad->a_stride, na) || !good_stride(ad->b_stride, nb) || !good_stride(ad->x_stride, ad->d_in) ||
      (base && !good_stride(ad->base_stride, ad->d_out)) || !good_stride(ad->y_stride, ad->d_out))
    return STRATA_E_INVAL;
  if (ad->a_stride % 8 || ad->b_stride % 8 || ad->x_stride % 8 || (base && ad->base_stride % 8) || ad->y_stride % 8)
    return STRATA_E_ALIGN;
  if (!aligned(ad->a, 16) || !aligned(ad->b, 16) || !aligned(x, 16) || !aligned(base, 16) || !aligned(y, 16) ||
      !aligned(ad->scale, 4) || !aligned(seg_off, 4) || !aligned(seg_adapter, 4))
    return STRATA_E_ALIGN;
  if (!aligned(ws, 256)) return STRATA_E_ALIGN;
  const WsLayout L = ws_layout(T);
  if (ws_bytes < L.total) return STRATA_E_WORKSPACE;
  if (T == 0 || n_seg == 0) return STRATA_OK;
  const Rows sx = rows_of(x, T, ad->x_stride, ad->d_in, ad->x_type), sy = rows_of(y, T, ad->y_stride, ad->d_out, ad->y_type);
  const Rows sb = rows_of(base, T, ad->base_stride, ad->d_out, ad->y_type);
  if (overlap(sx, sy) || partly(sb, sy)) return STRATA_E_INVAL;
  char* w = (char*)ws;
  return launched(launch_adapters(*ad, seg_off, seg_adapter, n_seg, x, T, base, y, (uint16_t*)(w + L.logits),
                                  (int*)(w + L.status), (cudaStream_t)stream));
}

}  // extern "C"
