// C ABI of the gates other than the plain softmax (moe_select,
// moe_route_scored) and of the expert half of a layer in 8-bit integers
// (moe_experts); declared in include/moe.h.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/moe.h"
#include "int8_layout.hpp"
#include "moe_kernels.hpp"

namespace {
inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }
template <typename... A>
int fail(int code, const char* fmt, A... a) {
  return moe::set_error(code, fmt, a...);
}
int hip_fail(hipError_t e, const char* what) { return fail(MOE_EHIP, "%s: %s", what, hipGetErrorString(e)); }
}  // namespace

int moe::gate_args(const char* who, const moe_gate_t* g, int E, int k, GateArgs* out) {
  if (!g) return fail(MOE_EINVAL, "%s: null gate", who);
  if (g->score != MOE_SCORE_SOFTMAX && g->score != MOE_SCORE_SIGMOID)
    return fail(MOE_EINVAL, "%s: score %d is neither MOE_SCORE_SOFTMAX nor MOE_SCORE_SIGMOID", who, (int)g->score);
  if (g->n_group < 1 || g->n_group > 64 || E % g->n_group != 0)
    return fail(MOE_EINVAL, "%s: %d groups do not divide %d experts (at most 64 groups)", who, (int)g->n_group, E);
  if (g->topk_group < 1 || g->topk_group > g->n_group)
    return fail(MOE_EINVAL, "%s: %d groups of %d kept", who, (int)g->topk_group, (int)g->n_group);
  if (g->group_top != 1 && g->group_top != 2)
    return fail(MOE_EINVAL, "%s: group_top %d is neither 1 nor 2", who, (int)g->group_top);
  if ((long long)g->topk_group * (E / g->n_group) < k)
    return fail(MOE_EINVAL, "%s: %d experts of %d kept groups, fewer than k=%d", who, g->topk_group * (E / g->n_group),
                (int)g->topk_group, k);
  if (!std::isfinite(g->scale)) return fail(MOE_EINVAL, "%s: scale is not finite", who);
  *out = GateArgs{g->score, g->n_group, g->topk_group, g->group_top, g->renorm != 0, g->scale, g->balance};
  return MOE_OK;
}

int moe::check_experts_int8(const char* who, const void* x, int T, int H, int E, int k, int I, int n_slots,
                            const void* slot_base, size_t slot_stride, const void* out, const void* ws,
                            size_t ws_bytes, const void* y) {
  if (T < 0 || E < 1 || E > kTableItems || k < 1 || k > E || n_slots < 1 || (long long)T * k > (1ll << 30))
    return fail(MOE_EINVAL, "%s: bad sizes T=%d E=%d k=%d n_slots=%d", who, T, E, k, n_slots);
  if (!int8_shape_ok(H, I)) return fail(MOE_EINVAL, "%s: unsupported int8 expert shape %dx%d", who, H, I);
  if (!int8_rows_ok((size_t)T * k, T, H, I))
    return fail(MOE_EINVAL, "%s: codes of %d tokens pass 32-bit offsets", who, T);
  if (slot_stride < int8_layout(H, I).bytes)
    return fail(MOE_EINVAL, "%s: slot_stride %zu < blob size %zu", who, slot_stride, int8_layout(H, I).bytes);
  if (!x || !slot_base || !out || !ws || !y) return fail(MOE_EINVAL, "%s: null pointer argument", who);
  if (!aligned16(x, slot_base, out, ws, y) || slot_stride % 16 != 0)
    return fail(MOE_EINVAL, "%s: int8 experts need 16-byte aligned buffers and slots", who);
  if (ws_bytes < int8_ws((size_t)T * k, T, H, I).bytes)
    return fail(MOE_EINVAL, "%s: workspace too small for %d tokens", who, T);
  return MOE_OK;
}

extern "C" {

size_t moe_select_workspace_size(int T, int E, int k) {
  if (T < 0 || E < 1 || E > 1024 || k < 1) return 0;
  return moe::select_workspace_bytes(T, E);
}

int moe_select(const float* logits, const moe_gate_t* gate, int T, int E, int k, int32_t* topk_idx, float* topk_w,
               int32_t* counts, int32_t* offsets, int32_t* perm_src, int32_t* perm_pos, void* workspace,
               size_t ws_bytes, void* stream) {
  if (T < 0 || E < 1 || E > 1024 || k < 1 || k > 16 || k > E || (long long)T * k > (1ll << 30))
    return fail(MOE_EINVAL, "moe_select: unsupported sizes T=%d E=%d k=%d", T, E, k);
  moe::GateArgs g;
  const int rc = moe::gate_args("moe_select", gate, E, k, &g);
  if (rc != MOE_OK) return rc;
  if (!counts || !offsets || !workspace || (T > 0 && (!logits || !topk_idx || !topk_w || !perm_src || !perm_pos)))
    return fail(MOE_EINVAL, "moe_select: null pointer argument");
  if (ws_bytes < moe::select_workspace_bytes(T, E) || (reinterpret_cast<uintptr_t>(workspace) & 15))
    return fail(MOE_EINVAL, "moe_select: workspace too small (%zu < %zu) or not 16-byte aligned", ws_bytes,
                moe::select_workspace_bytes(T, E));
  hipError_t e = moe::launch_select(logits, 1, nullptr, nullptr, g, T, E, k, topk_idx, topk_w, counts, offsets,
                                    perm_src, perm_pos, workspace, as_stream(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_select launch");
}

int moe_route_scored(const void* x, int dtype, const void* Wr, const float* bias, const moe_gate_t* gate, int T, int H,
                     int E, int k, int32_t* topk_idx, float* topk_w, float* logits, int32_t* counts, int32_t* offsets,
                     int32_t* perm_src, int32_t* perm_pos, void* workspace, size_t ws_bytes, void* stream) {
  if (T < 0 || H <= 0 || E <= 0 || E > 1024 || k < 1 || k > 16 || k > E || (H % 8) != 0)
    return fail(MOE_EINVAL, "moe_route_scored: unsupported sizes T=%d H=%d E=%d k=%d", T, H, E, k);
  if (dtype != MOE_DT_F32 && dtype != MOE_DT_BF16) return fail(MOE_EINVAL, "moe_route_scored: bad dtype %d", dtype);
  moe::GateArgs g;
  const int rc = moe::gate_args("moe_route_scored", gate, E, k, &g);
  if (rc != MOE_OK) return rc;
  if (!counts || !offsets || !workspace || (T > 0 && (!x || !Wr || !topk_idx || !topk_w || !perm_src || !perm_pos)))
    return fail(MOE_EINVAL, "moe_route_scored: null pointer argument");
  if (ws_bytes < moe::route_workspace_bytes(T, H, E, k))
    return fail(MOE_EINVAL, "moe_route_scored: workspace too small (%zu < %zu)", ws_bytes,
                moe::route_workspace_bytes(T, H, E, k));
  hipError_t e = moe::launch_route(x, dtype == MOE_DT_BF16, Wr, bias, T, H, E, k, topk_idx, topk_w, logits, counts,
                                   offsets, perm_src, perm_pos, workspace, as_stream(stream), nullptr, 0, nullptr,
                                   nullptr, &g);
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_route_scored launch");
}

size_t moe_experts_workspace_size(int T, int k, int E, int H, int I, int wfmt) {
  if (T < 0 || k < 1 || E < 1 || wfmt != MOE_W_INT8 || !moe::int8_shape_ok(H, I)) return 0;
  return moe::align_up(moe::int8_ws((size_t)T * k, T, H, I).bytes, 256) + (size_t)T * k * H * 4 + 256;
}

int moe_experts(const void* x, int dtype, const int32_t* topk_idx, const float* topk_w, const int32_t* perm_src,
                const int32_t* perm_pos, const int32_t* counts, const int32_t* offsets, const int32_t* slot_of, int T,
                int k, int E, int n_slots, const void* slot_base, size_t slot_stride, int wfmt, int H, int I,
                void* out, int out_dtype, void* workspace, size_t ws_bytes, void* stream) {
  if (wfmt != MOE_W_INT8)
    return fail(MOE_EINVAL, "moe_experts: needs int8 experts (format %d); moe_ffn and moe_ffn_grouped take the others",
                wfmt);
  if (dtype != MOE_DT_BF16) return fail(MOE_EINVAL, "moe_experts: activations must be bf16");
  if (out_dtype != MOE_DT_F32 && out_dtype != MOE_DT_BF16) return fail(MOE_EINVAL, "moe_experts: bad out dtype");
  if (T == 0) return MOE_OK;
  const size_t need = moe_experts_workspace_size(T, k, E, H, I, wfmt);
  if (need != 0 && ws_bytes < need)
    return fail(MOE_EINVAL, "moe_experts: workspace too small (%zu < %zu)", ws_bytes, need);
  char* ws = static_cast<char*>(workspace);
  void* y = ws && need ? ws + moe::align_up(moe::int8_ws((size_t)T * k, T, H, I).bytes, 256) : nullptr;
  const int rc = moe::check_experts_int8("moe_experts", x, T, H, E, k, I, n_slots, slot_base, slot_stride, out, ws,
                                         ws_bytes, y);
  if (rc != MOE_OK) return rc;
  if (!topk_idx || !topk_w || !perm_src || !perm_pos || !counts || !offsets)
    return fail(MOE_EINVAL, "moe_experts: null pointer argument");
  if (!slot_of && n_slots < E)
    return fail(MOE_EINVAL, "moe_experts: %d slots for %d experts need a slot table", n_slots, E);
  hipError_t e = moe::launch_experts_int8(x, T, k, E, topk_idx, topk_w, perm_src, perm_pos, counts, offsets, slot_of,
                                          n_slots, static_cast<const char*>(slot_base), slot_stride, H, I, out,
                                          out_dtype == MOE_DT_BF16, ws, static_cast<float*>(y), as_stream(stream));
  return e == hipSuccess ? MOE_OK : hip_fail(e, "moe_experts launch");
}

}  // extern "C"
