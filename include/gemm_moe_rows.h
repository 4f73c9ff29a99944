/*
 * gemm_moe_rows.h -- tokens sorted by expert and back, on MI355X: what stands
 * before and behind the grouped products (gemm_*_grouped) of a
 * mixture-of-experts layer, with the gradients.  Same library, return codes
 * (enum gemm_status), stream and workspace rules as gemm_f16.h; formats of enum
 * gemm_mx4_format.
 *
 * A pair is a token t and its choice j of top_k, number t*top_k + j; there are
 * P = T*top_k of them.  Sorted by expert and, within an expert, by number, each
 * pair whose expert is in 0 .. E-1 has a slot; other pairs (a padded token's,
 * say with expert -1) have none.
 *     offsets [E+1]       expert e's slots are offsets[e] .. offsets[e+1]-1 (the
 *                         row groups of a grouped product)
 *     rows    [P]         number of the pair in a slot; -1 from offsets[E] on
 *     slots   [T, top_k]  slot of a pair; -1 without one
 * All three int64, on the device.  The calls below that take them read no slot
 * outside 0 .. P-1 (such a pair counts as one without).  In tables that no
 * gemm_moe_sort made, slots that two pairs share, or from offsets[E] on, leave in the
 * rows written there any of what is written to them, or parts of each.
 *
 * T below 2^23, P below 2^31, H at most 2^24, and T times the parts of a row of X or Y
 * (2048 bytes in gather, 1024 elements in combine) below 2^25; else GEMM_ERR_SHAPE.
 *
 * Results are deterministic; sums over rows are float32, in a fixed order.
 */
#ifndef GEMM_MOE_ROWS_H
#define GEMM_MOE_ROWS_H

#include "gemm_mx4.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The three tables of experts[t*ld + j], int32 (id_bytes 4) or int64 (8).  The
 * same expert may be chosen twice.  E at most 1024.
 * Needs gemm_moe_sort_workspace_bytes(T, top_k, E) bytes of workspace (may be 0),
 * 256-byte aligned; with workspace == NULL they are allocated in stream order.
 */
typedef struct gemm_moe_sort_args {
  const void* experts;
  int64_t ld, T;
  int64_t* offsets;
  int64_t* rows;
  int64_t* slots;
  int32_t id_bytes, top_k, E;
} gemm_moe_sort_args;

int gemm_moe_sort(const gemm_moe_sort_args* args, void* stream, void* workspace, size_t workspace_bytes);
size_t gemm_moe_sort_workspace_bytes(int64_t T, int32_t top_k, int32_t E);

/*
 * Y[slots[t,j]] := X[t] for all pairs with a slot; Y's rows from offsets[E] on
 * are zeros.  X [T, H], Y [P, H] of elements of elem_bytes (1, 2 or 4), unit
 * stride along H, row strides in elements.
 */
typedef struct gemm_moe_gather_args {
  const void* X;
  int64_t ldx;
  const int64_t* offsets;
  const int64_t* slots;
  void* Y;
  int64_t ldy, T, H;
  int32_t elem_bytes, E, top_k;
} gemm_moe_gather_args;

int gemm_moe_gather(const gemm_moe_gather_args* args, void* stream);

/*
 * Y[t] := sum over j with a slot of weights[t*ldw + j] X[slots[t,j]], X [P, H] and
 * Y [T, H] of format fmt, weights of fmt_w (GEMM_FMT_F32 or fmt), or 1 with
 * weights == NULL (which is gather's gradient).
 */
typedef struct gemm_moe_combine_args {
  const void* X;
  int64_t ldx;
  const int64_t* slots;
  const void* weights;
  int64_t ldw;
  void* Y;
  int64_t ldy, T, H;
  int32_t fmt, fmt_w, top_k;
} gemm_moe_combine_args;

int gemm_moe_combine(const gemm_moe_combine_args* args, void* stream);

/*
 * Gradients of gemm_moe_combine's X and weights, given those of its Y (DY [T, H]):
 *     DX[slots[t,j]] := weights[t,j] DY[t]; its rows from offsets[E] on are zeros
 *     DW[t*lddw + j] := sum_h DY[t,h] X[slots[t,j],h], 0 without a slot (of fmt_w)
 */
typedef struct gemm_moe_combine_backward_args {
  const void* DY;
  int64_t lddy;
  const void* X;
  int64_t ldx;
  const int64_t* offsets;
  const int64_t* slots;
  const void* weights;
  int64_t ldw;
  void* DX;
  int64_t lddx;
  void* DW;
  int64_t lddw, T, H;
  int32_t fmt, fmt_w, E, top_k;
} gemm_moe_combine_backward_args;

int gemm_moe_combine_backward(const gemm_moe_combine_backward_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_MOE_ROWS_H */
