// Experts in 8-bit integers (MOE_W_INT8): blob and workspace layouts, launchers.
#pragma once
#include <hip/hip_runtime.h>

#include "../../include/moe.h"
#include "moe_kernels.hpp"

namespace moe {

// Blob: P1 and P2 with the row order of the bf16 blob. A row tile (16 rows) is
// K/64 fragments of 1 KiB; fragment byte 16 l + b is row (l % 16) of the tile,
// column 64 c + 16 (l / 16) + b of K for P1. P2's K is taken in the order that
// the gate/up product leaves its columns in (int8_k2_source): lane group q
// holds, of every 8 columns, the two that the accumulator lanes of group q
// hold. fp32 scales: P1's in row order (gate and up interleaved), P2's by
// column, and a reserved word behind them, which the size of a blob counts and
// nothing reads. Sections [P1 codes][P1 scales][P2 codes][P2 scales, word],
// 256-B aligned.
struct Int8Layout {
  size_t p1, p1s, p2, p2s, bytes;
};
inline Int8Layout int8_layout(int H, int I) {
  Int8Layout l{};
  const size_t HI = (size_t)H * I;
  l.p1 = 0;
  l.p1s = align_up(2 * HI, 256);
  l.p2 = align_up(l.p1s + (size_t)2 * I * 4, 256);
  l.p2s = align_up(l.p2 + HI, 256);
  l.bytes = align_up(l.p2s + (size_t)H * 4 + 4, 256);
  return l;
}
// H, I multiples of 64. The decode kernels hold 16 rows of I codes in LDS, and
// offsets inside one expert's matrix are 32 bits.
constexpr int kInt8MaxI = 8192, kInt8MaxH = 16384;
inline bool int8_shape_ok(int H, int I) {
  return H > 0 && I > 0 && H % 64 == 0 && I % 64 == 0 && H <= kInt8MaxH && I <= kInt8MaxI;
}
// Whether `rows` rows over `groups` experts run the tiled GEMM: from 4 rows an expert on. The decode kernels read a
// weight once for every 16 rows of its expert too, but with fewer rows in flight and each block forming h's codes for
// itself. Measured, decode against GEMM, us: 64 experts of 4096 x 2048, 2.3 rows each 222 / 252, 6 rows 285 / 267; 16 of
// 2048 x 768, 4 rows 30.2 / 28.8, 16 rows 49 / 30; 8 of 3968 x 1920, 4 rows 46.7 / 47.3, 32 rows 123 / 50; 96 of
// 1024 x 512, 2 rows 39.5 / 36.2, 3.3 rows 51 / 37.7; 48 of 2048 x 1024, 2 rows 51 / 59, 3.3 rows 63 / 61.
inline bool int8_gemm_pays(long long rows, long long groups) { return rows >= 4 * groups; }
inline bool int8_gemm_supported(int H, int I) { return int8_shape_ok(H, I) && H % 128 == 0 && I % 128 == 0; }

// Offsets inside the code buffers are 32 bits: codes of `tokens` rows of H and `rows` rows of I.
inline bool int8_rows_ok(size_t rows, size_t tokens, int H, int I) {
  return tokens * H <= 0xFFFFFFFFull && (rows + 16) * I <= 0xFFFFFFFFull;
}
template <typename... P>
inline bool aligned16(const P*... p) {
  return ((reinterpret_cast<uintptr_t>(p) | ...) & 15) == 0;
}

// K index of byte j of lane group q in P2's 64-wide chunk c.
__host__ __device__ inline int int8_k2_source(int c, int q, int j) { return 64 * c + 8 * (j >> 1) + 2 * q + (j & 1); }

// Workspace of the products: token codes and scales, h (fp32), its codes and
// scales, the plan (a count, then an entry for each group or 128-row tile).
struct Int8Ws {
  size_t xq, sx, h, hq, sh, plan, done, bytes;
  int entries;  // that the plan holds behind its count
};
inline Int8Ws int8_ws(size_t rows, size_t tokens, int H, int I) {
  Int8Ws w{};
  const size_t padded = (rows + 15) / 16 * 16;
  w.xq = 0;
  w.sx = align_up(tokens * H, 256);
  w.h = align_up(w.sx + tokens * 4, 256);
  w.hq = align_up(w.h + padded * I * 4, 256);
  w.sh = align_up(w.hq + padded * I, 256);
  w.plan = align_up(w.sh + padded * 4, 256);
  w.entries = (int)(rows / 128) + kTableItems + 1;
  w.done = w.plan + 256 + align_up((size_t)w.entries * 16, 256);  // counts by group of output columns
  w.bytes = w.done + align_up((size_t)H / 8, 256);
  return w;
}
hipError_t launch_pack_int8(int H, int I, const void* Q1, const void* Q3, const void* Q2, const void* S1,
                            const void* S3, const void* S2, void* blob, hipStream_t s);
// Listed items {slot, row_begin, rows > 0, expert} (host); x bf16 through perm_src; `gemm`: the tiled kernels.
hipError_t launch_ffn_int8_list(const void* x, const int32_t* perm_src, const int4* items, int n, int rows_total,
                                bool gemm, const char* slot_base, size_t slot_stride, int H, int I, float* y, void* ws,
                                hipStream_t s);
// The decode kernels over a work list in device memory (at most max_items); x bf16 [T, H].
hipError_t launch_ffn_int8_dev(const void* x, int T, const int32_t* perm_src, const int32_t* n_items,
                               const int4* items, int max_items, int rows_total, const char* slot_base,
                               size_t slot_stride, int H, int I, float* y, void* ws, hipStream_t s);
// A layer's expert half from a routing on the device to `out` [T, H]. ws: int8_ws(T k, T); y: T k rows of H fp32.
hipError_t launch_experts_int8(const void* x, int T, int k, int E, const int32_t* topk_idx, const float* topk_w,
                               const int32_t* perm_src, const int32_t* perm_pos, const int32_t* counts,
                               const int32_t* offsets, const int32_t* slot_of, int n_slots, const char* slot_base,
                               size_t slot_stride, int H, int I, void* out, bool out_bf16, void* ws, float* y, hipStream_t s);

// The checks of arguments shared by the entry points (`who` names the caller in the message).
int gate_args(const char* who, const moe_gate_t* gate, int E, int k, GateArgs* out);
int check_experts_int8(const char* who, const void* x, int T, int H, int E, int k, int I, int n_slots,
                       const void* slot_base, size_t slot_stride, const void* out, const void* ws, size_t ws_bytes,
                       const void* y);

}  // namespace moe
