// C ABI of the operators that train through the layer: the grouping of given
// choices, rows out and back with their gradient, SwiGLU kept in 8 bits, the
// experts' products and their gradients; declared in include/moe.h.
#include <hip/hip_runtime.h>

#include "../../include/moe.h"
#include "moe_kernels.hpp"

namespace {
inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }
template <typename... A>
int fail(int code, const char* fmt, A... a) {
  return moe::set_error(code, fmt, a...);
}
int done(hipError_t e, const char* who) {
  return e == hipSuccess ? MOE_OK : fail(MOE_EHIP, "%s launch: %s", who, hipGetErrorString(e));
}
bool is_act(int dtype) { return dtype == MOE_DT_F32 || dtype == MOE_DT_BF16; }
bool off(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }
size_t elem(int dtype) { return dtype == MOE_DT_BF16 ? 2 : 4; }

constexpr int kMaxLen = 1 << 20;  // longest row

int check_rows(const char* who, int T, int k, int H, int rows_max, const int32_t* perm_pos) {
  // a block to a token at most: 2^24 of 256 threads is the longest launch
  if (T < 0 || T >= (1 << 24) || k < 1 || k > 16 || H < 1 || H > kMaxLen || rows_max < 0)
    return fail(MOE_EINVAL, "%s: unsupported sizes T=%d k=%d H=%d rows_max=%d", who, T, k, H, rows_max);
  if (T > 0 && !perm_pos) return fail(MOE_EINVAL, "%s: null pointer argument", who);
  if (off(perm_pos, 4)) return fail(MOE_EINVAL, "%s: a buffer is not aligned to its elements", who);
  return MOE_OK;
}

int check_matmul(const char* who, const void* a, const void* b, const int32_t* counts, const int32_t* offsets, int E,
                 int rows_max, int K, int N, const void* c, int out_dtype, bool rows) {
  if (E < 1 || E > 1024 || rows_max < 0 || rows_max > (1 << 30) || K < 8 || N < 8 || K % 8 != 0 || N % 8 != 0 ||
      K > (1 << 16) || N > (1 << 16) || (long long)K * N > (1ll << 30))
    return fail(MOE_EINVAL, "%s: unsupported sizes E=%d rows_max=%d K=%d N=%d", who, E, rows_max, K, N);
  if (!is_act(out_dtype)) return fail(MOE_EINVAL, "%s: bad out dtype %d", who, out_dtype);
  if (!counts || !offsets || (rows_max > 0 && (!a || !b)) || !(c || (rows && rows_max == 0)))
    return fail(MOE_EINVAL, "%s: null pointer argument", who);
  if (off(a, 16) || off(b, 16) || off(c, 16) || off(counts, 4) || off(offsets, 4))
    return fail(MOE_EINVAL, "%s: buffers must be 16-byte aligned", who);
  return MOE_OK;
}
}  // namespace

extern "C" {

size_t moe_group_workspace_size(int T, int k, int E) {
  if (T < 0 || k < 1 || k > 16 || E < 1 || E > 1024 || (long long)T * k > (1ll << 30)) return 0;
  return moe::group_workspace_bytes(T, k, E);
}

int moe_group(const int32_t* topk_idx, int T, int k, int E, int32_t* counts, int32_t* offsets, int32_t* perm_src,
              int32_t* perm_pos, void* workspace, size_t ws_bytes, void* stream) {
  if (T < 0 || k < 1 || k > 16 || E < 1 || E > 1024 || (long long)T * k > (1ll << 30))
    return fail(MOE_EINVAL, "moe_group: unsupported sizes T=%d E=%d k=%d", T, E, k);
  if (!counts || !offsets || (T > 0 && (!topk_idx || !perm_src || !perm_pos)))
    return fail(MOE_EINVAL, "moe_group: null pointer argument");
  if (off(topk_idx, 4) || off(counts, 4) || off(offsets, 4) || off(perm_src, 4) || off(perm_pos, 4))
    return fail(MOE_EINVAL, "moe_group: a buffer is not aligned to its elements");
  const size_t need = moe::group_workspace_bytes(T, k, E);
  if (need > 0 && (!workspace || ws_bytes < need || off(workspace, 4)))
    return fail(MOE_EINVAL, "moe_group: workspace too small (%zu < %zu) or not aligned", ws_bytes, need);
  return done(moe::launch_group(topk_idx, T, k, E, counts, offsets, perm_src, perm_pos, workspace, as_stream(stream)),
              "moe_group");
}

int moe_dispatch(const void* x, int dtype, const int32_t* perm_pos, int T, int k, int H, int rows_max, void* x_perm,
                 void* stream) {
  if (!is_act(dtype)) return fail(MOE_EINVAL, "moe_dispatch: bad dtype %d", dtype);
  const int rc = check_rows("moe_dispatch", T, k, H, rows_max, perm_pos);
  if (rc != MOE_OK) return rc;
  if (T == 0 || rows_max == 0) return MOE_OK;
  if (!x || !x_perm) return fail(MOE_EINVAL, "moe_dispatch: null pointer argument");
  if (off(x, elem(dtype)) || off(x_perm, elem(dtype)))
    return fail(MOE_EINVAL, "moe_dispatch: a buffer is not aligned to its elements");
  return done(moe::launch_dispatch(x, dtype == MOE_DT_BF16, perm_pos, T, k, H, rows_max, x_perm, as_stream(stream)),
              "moe_dispatch");
}

int moe_collect(const void* rows, int dtype, const int32_t* perm_pos, const float* topk_w, int T, int k, int H,
                int rows_max, void* out, int out_dtype, void* stream) {
  if (!is_act(dtype) || !is_act(out_dtype))
    return fail(MOE_EINVAL, "moe_collect: bad dtype %d or out dtype %d", dtype, out_dtype);
  const int rc = check_rows("moe_collect", T, k, H, rows_max, perm_pos);
  if (rc != MOE_OK) return rc;
  if (T == 0) return MOE_OK;
  if (!out || (!rows && rows_max > 0)) return fail(MOE_EINVAL, "moe_collect: null pointer argument");
  if (off(rows, elem(dtype)) || off(topk_w, 4) || off(out, elem(out_dtype)))
    return fail(MOE_EINVAL, "moe_collect: a buffer is not aligned to its elements");
  return done(moe::launch_collect(rows, dtype == MOE_DT_BF16, perm_pos, topk_w, T, k, H, rows_max, out,
                                  out_dtype == MOE_DT_BF16, as_stream(stream)),
              "moe_collect");
}

int moe_collect_backward(const void* dout, int out_dtype, const void* rows, int dtype, const int32_t* perm_pos,
                         const float* topk_w, int T, int k, int H, int rows_max, void* drows, float* dw,
                         void* stream) {
  if (!is_act(dtype) || !is_act(out_dtype))
    return fail(MOE_EINVAL, "moe_collect_backward: bad dtype %d or out dtype %d", dtype, out_dtype);
  const int rc = check_rows("moe_collect_backward", T, k, H, rows_max, perm_pos);
  if (rc != MOE_OK) return rc;
  if (!drows && !dw && rows_max > 0) return fail(MOE_EINVAL, "moe_collect_backward: neither drows nor dw");
  if (T == 0 || (!drows && !dw)) return MOE_OK;
  if (!dout || (dw && !rows && rows_max > 0)) return fail(MOE_EINVAL, "moe_collect_backward: null pointer argument");
  if (off(dout, elem(out_dtype)) || off(rows, elem(dtype)) || off(topk_w, 4) || off(drows, elem(dtype)) || off(dw, 4))
    return fail(MOE_EINVAL, "moe_collect_backward: a buffer is not aligned to its elements");
  return done(moe::launch_collect_backward(dout, out_dtype == MOE_DT_BF16, rows, dtype == MOE_DT_BF16, perm_pos, topk_w,
                                           T, k, H, rows_max, drows, dw, as_stream(stream)),
              "moe_collect_backward");
}

int moe_swiglu_save(const void* gu, int dtype, int rows, const int32_t* n_rows, int I, void* h, int8_t* codes,
                    float* scales, void* stream) {
  if (!is_act(dtype)) return fail(MOE_EINVAL, "moe_swiglu_save: bad dtype %d", dtype);
  if (rows < 0 || I < 1 || I > kMaxLen || (long long)rows * ((I + 127) / 128) > (1ll << 26))
    return fail(MOE_EINVAL, "moe_swiglu_save: unsupported sizes rows=%d I=%d", rows, I);
  if (rows == 0) return MOE_OK;
  if (!gu || !h || !codes || !scales) return fail(MOE_EINVAL, "moe_swiglu_save: null pointer argument");
  if (off(gu, elem(dtype)) || off(h, elem(dtype)) || off(scales, 4) || off(n_rows, 4))
    return fail(MOE_EINVAL, "moe_swiglu_save: a buffer is not aligned to its elements");
  return done(moe::launch_swiglu_save(gu, dtype == MOE_DT_BF16, rows, n_rows, I, h, codes, scales, as_stream(stream)),
              "moe_swiglu_save");
}

int moe_swiglu_backward(const int8_t* codes, const float* scales, const void* dh, int dtype, int rows,
                        const int32_t* n_rows, int I, void* dgu, void* h, void* stream) {
  if (!is_act(dtype)) return fail(MOE_EINVAL, "moe_swiglu_backward: bad dtype %d", dtype);
  if (rows < 0 || I < 1 || I > kMaxLen || (long long)rows * ((I + 127) / 128) > (1ll << 26))
    return fail(MOE_EINVAL, "moe_swiglu_backward: unsupported sizes rows=%d I=%d", rows, I);
  if (rows == 0) return MOE_OK;
  if (!codes || !scales || !dh || !dgu) return fail(MOE_EINVAL, "moe_swiglu_backward: null pointer argument");
  if (off(dh, elem(dtype)) || off(dgu, elem(dtype)) || off(h, elem(dtype)) || off(scales, 4) || off(n_rows, 4))
    return fail(MOE_EINVAL, "moe_swiglu_backward: a buffer is not aligned to its elements");
  return done(moe::launch_swiglu_backward(codes, scales, dh, dtype == MOE_DT_BF16, rows, n_rows, I, dgu, h,
                                          as_stream(stream)),
              "moe_swiglu_backward");
}

int moe_matmul_grouped(const void* a, const void* w, const int32_t* counts, const int32_t* offsets, int E,
                       int rows_max, int K, int N, int transposed, void* c, int out_dtype, void* stream) {
  const int rc = check_matmul("moe_matmul_grouped", a, w, counts, offsets, E, rows_max, K, N, c, out_dtype, true);
  if (rc != MOE_OK || rows_max == 0) return rc;
  return done(moe::launch_matmul_grouped(a, w, counts, offsets, E, rows_max, K, N, transposed != 0, c,
                                         out_dtype == MOE_DT_BF16, as_stream(stream)),
              "moe_matmul_grouped");
}

int moe_matmul_grouped_dw(const void* a, const void* dc, const int32_t* counts, const int32_t* offsets, int E,
                          int rows_max, int K, int N, void* dw, int out_dtype, void* stream) {
  const int rc = check_matmul("moe_matmul_grouped_dw", a, dc, counts, offsets, E, rows_max, K, N, dw, out_dtype, false);
  if (rc != MOE_OK) return rc;
  return done(moe::launch_matmul_grouped_dw(a, dc, counts, offsets, E, rows_max, K, N, dw, out_dtype == MOE_DT_BF16,
                                            as_stream(stream)),
              "moe_matmul_grouped_dw");
}

}  // extern "C"
