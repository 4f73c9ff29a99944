// Host side of include/gemm_moe_rows.h: argument validation and launches of the
// sort by expert and of the kernels that move rows.  Everything is checked
// before the first HIP call, so on any error nothing is enqueued.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/gemm_moe_rows.h"
#include "host_launch.hpp"
#include "moe_rows_kernel.hpp"

using namespace gemmf16;

namespace {

constexpr int64_t kMaxPairs = INT64_C(1) << 31, kMaxTokens = INT64_C(1) << 23, kMaxRow = INT64_C(1) << 24;

// Chunks of the sort: one while a workgroup's passes over it cost less than a
// second launch.
void sort_chunks(int64_t P, int64_t* chunk, int64_t* chunks) {
  *chunk = P <= 16 * kSortThreads ? cdiv(P, kSortThreads) * kSortThreads : 2 * kSortThreads;
  while (cdiv(P, *chunk) > 256) *chunk *= 2;
  *chunks = cdiv(P, *chunk);
}

bool pairs_ok(int64_t T, int32_t top_k, int64_t* P) {
  return T > 0 && top_k > 0 && T < kMaxTokens && !__builtin_mul_overflow(T, (int64_t)top_k, P) && *P < kMaxPairs;
}

// Whether the experts' rows go past the caches.  us without | with it, of one run, in
// graphs over two sets of bfloat16 rows in turn (T x top_k x H): gather and the combine
// that reads its rows 4096 x 8 x 7168 (504 MiB) 232 | 189, 16384 x 8 x 7168 840 | 792;
// gather alone 107 | 96 and 410 | 410 (over and over on one set 425 | 362), combine 106 |
// 96 and 408 | 406 (424 | 375), its gradients 211 | 198 and 789 | 779.  Below the bound the pair gains and loses by turns: 384 MiB 166 |
// 158, 288 120 | 110, 219 97 | 108, 160 63 | 57, 72 27 | 29.
bool once(int64_t T, int64_t P, int64_t row_bytes) { return (double)(T + P) * (double)row_bytes > kOnceBytes; }
#define GEMM_ONCE(KERNEL, FMT, o) ((o) ? (const void*)KERNEL<FMT, true> : (const void*)KERNEL<FMT, false>)

int64_t elem_size(int32_t fmt) { return fmt == GEMM_FMT_F32 ? 4 : 2; }

}  // namespace

extern "C" {

size_t gemm_moe_sort_workspace_bytes(int64_t T, int32_t top_k, int32_t E) {
  int64_t P, chunk, chunks;
  if (!pairs_ok(T, top_k, &P) || E < 1 || E > kSortExperts) return 0;
  sort_chunks(P, &chunk, &chunks);
  return chunks > 1 ? (size_t)(chunks * E * 4) : 0;
}

int gemm_moe_sort(const gemm_moe_sort_args* args, void* stream, void* workspace, size_t workspace_bytes) {
  if (!args) return GEMM_ERR_NULL;
  const auto [experts, ld, T, offsets, rows, slots, id_bytes, top_k, E] = *args;
  if (!experts || !offsets || !rows || !slots) return GEMM_ERR_NULL;
  int64_t P;
  if (!pairs_ok(T, top_k, &P) || E < 1 || E > kSortExperts) return GEMM_ERR_SHAPE;
  if (id_bytes != 4 && id_bytes != 8) return GEMM_ERR_OPTS;
  if (ld <= 0) return GEMM_ERR_STRIDE;
  Range ri, ro, rr, rs;
  if (!byte_view(experts, T, top_k, ld, 1, id_bytes, &ri) || !byte_rows(offsets, 1, 1, 8 * (E + 1), &ro) ||
      !byte_rows(rows, 1, 1, 8 * P, &rr) || !byte_rows(slots, 1, 1, 8 * P, &rs))
    return GEMM_ERR_SHAPE;
  if ((uintptr_t)experts % id_bytes || ((uintptr_t)offsets & 7u) || ((uintptr_t)rows & 7u) || ((uintptr_t)slots & 7u))
    return GEMM_ERR_LAYOUT;
  if (overlap(ri, ro) || overlap(ri, rr) || overlap(ri, rs) || overlap(ro, rr) || overlap(ro, rs) || overlap(rr, rs))
    return GEMM_ERR_ALIAS;
  const size_t need = gemm_moe_sort_workspace_bytes(T, top_k, E);
  if (workspace && need) {
    const Range rw{(uintptr_t)workspace, (uintptr_t)workspace + need};
    if (overlap(rw, ri) || overlap(rw, ro) || overlap(rw, rr) || overlap(rw, rs)) return GEMM_ERR_ALIAS;
  }
  hipStream_t s = (hipStream_t)stream;
  Workspace ws;
  int rc = ws.take(workspace, workspace_bytes, need, s);
  if (rc) return rc;
  SortArgs a{experts, ld, top_k, id_bytes == 8, E, 0, P, 0, 0, (int32_t*)ws.get(), offsets, rows, slots};
  while ((1 << a.bits) < E) ++a.bits;
  sort_chunks(P, &a.chunk, &a.chunks);
  if (a.chunks > 1) rc = run((const void*)moe_count_kernel, dim3((unsigned)a.chunks), kSortThreads, &a, s);
  if (rc == GEMM_OK) rc = run((const void*)moe_place_kernel, dim3((unsigned)a.chunks), kSortThreads, &a, s);
  return ws.done(rc);
}

int gemm_moe_gather(const gemm_moe_gather_args* args, void* stream) {
  if (!args) return GEMM_ERR_NULL;
  const auto [X, ldx, offsets, slots, Y, ldy, T, H, elem_bytes, E, top_k] = *args;
  if (!X || !offsets || !slots || !Y) return GEMM_ERR_NULL;
  int64_t P;
  if (!pairs_ok(T, top_k, &P) || E < 1 || H <= 0 || H > kMaxRow) return GEMM_ERR_SHAPE;
  if (elem_bytes != 1 && elem_bytes != 2 && elem_bytes != 4) return GEMM_ERR_OPTS;
  if (ldx <= 0) return GEMM_ERR_STRIDE;
  if (ldy < H) return GEMM_ERR_LDC;
  Range rx, ro, rs, ry;
  if (!byte_view(X, T, H, ldx, 1, elem_bytes, &rx) || !byte_rows(offsets, 1, 1, 8 * ((int64_t)E + 1), &ro) ||
      !byte_rows(slots, 1, 1, 8 * P, &rs) || !byte_view(Y, P, H, ldy, 1, elem_bytes, &ry))
    return GEMM_ERR_SHAPE;
  if (overlap(ry, rx) || overlap(ry, ro) || overlap(ry, rs)) return GEMM_ERR_ALIAS;
  RowsArgs a{};
  a.in = X;
  a.ldi = ldx * elem_bytes;
  a.out = Y;
  a.ldo = ldy * elem_bytes;
  a.slots = slots;
  a.ld_slots = top_k;
  a.placed = offsets + E;
  a.T = T;
  a.P = P;
  a.H = H * elem_bytes;
  a.top_k = top_k;
  const int64_t chunks = cdiv(a.H, 16);
  a.parts = (int32_t)cdiv(chunks, kRowThreads);
  if (!fits_x(T * a.parts, kRowThreads)) return GEMM_ERR_SHAPE;
  const void* fn = once(T, P, a.H) ? (const void*)moe_gather_kernel<true> : (const void*)moe_gather_kernel<false>;
  return run(fn, dim3((unsigned)(T * a.parts)), kRowThreads, &a, (hipStream_t)stream);
}

int gemm_moe_combine(const gemm_moe_combine_args* args, void* stream) {
  if (!args) return GEMM_ERR_NULL;
  const auto [X, ldx, slots, weights, ldw, Y, ldy, T, H, fmt, fmt_w, top_k] = *args;
  if (!X || !slots || !Y) return GEMM_ERR_NULL;
  int64_t P;
  if (!pairs_ok(T, top_k, &P) || H <= 0 || H > kMaxRow) return GEMM_ERR_SHAPE;
  if (fmt < GEMM_FMT_F16 || fmt > GEMM_FMT_F32 || (weights && fmt_w != fmt && fmt_w != GEMM_FMT_F32)) return GEMM_ERR_OPTS;
  if (ldx <= 0 || (weights && ldw <= 0)) return GEMM_ERR_STRIDE;
  if (ldy < H) return GEMM_ERR_LDC;
  const int64_t es = elem_size(fmt);
  Range rx, rs, rw{}, ry;
  if (!byte_view(X, P, H, ldx, 1, es, &rx) || !byte_rows(slots, 1, 1, 8 * P, &rs) || !byte_view(Y, T, H, ldy, 1, es, &ry) ||
      (weights && !byte_view(weights, T, top_k, ldw, 1, elem_size(fmt_w), &rw)))
    return GEMM_ERR_SHAPE;
  if (overlap(ry, rx) || overlap(ry, rs) || (weights && overlap(ry, rw))) return GEMM_ERR_ALIAS;
  RowsArgs a{};
  a.in = X;
  a.ldi = ldx * es;
  a.out = Y;
  a.ldo = ldy * es;
  a.slots = slots;
  a.ld_slots = top_k;
  a.weights = weights;
  a.ldw = ldw;
  a.w32 = fmt_w == GEMM_FMT_F32;
  a.T = T;
  a.P = P;
  a.H = H;
  a.top_k = top_k;
  a.parts = (int32_t)cdiv(cdiv(H, 8), kRowThreads);
  if (!fits_x(T * a.parts, kRowThreads)) return GEMM_ERR_SHAPE;
  const bool o = once(T, P, H * es);
  const void* fn = fmt == GEMM_FMT_F16    ? GEMM_ONCE(moe_combine_kernel, MX_F16, o)
                   : fmt == GEMM_FMT_BF16 ? GEMM_ONCE(moe_combine_kernel, MX_BF16, o)
                                          : GEMM_ONCE(moe_combine_kernel, MX_F32, o);
  return run(fn, dim3((unsigned)(T * a.parts)), kRowThreads, &a, (hipStream_t)stream);
}

int gemm_moe_combine_backward(const gemm_moe_combine_backward_args* args, void* stream) {
  if (!args) return GEMM_ERR_NULL;
  const auto [DY, lddy, X, ldx, offsets, slots, weights, ldw, DX, lddx, DW, lddw, T, H, fmt, fmt_w, E, top_k] = *args;
  if (!DY || !X || !offsets || !slots || !weights || !DX || !DW) return GEMM_ERR_NULL;
  int64_t P;
  if (!pairs_ok(T, top_k, &P) || E < 1 || H <= 0 || H > kMaxRow) return GEMM_ERR_SHAPE;
  if (fmt < GEMM_FMT_F16 || fmt > GEMM_FMT_F32 || (fmt_w != fmt && fmt_w != GEMM_FMT_F32)) return GEMM_ERR_OPTS;
  if (lddy <= 0 || ldx <= 0 || ldw <= 0) return GEMM_ERR_STRIDE;
  if (lddx < H || lddw < top_k) return GEMM_ERR_LDC;
  const int64_t es = elem_size(fmt), ew = elem_size(fmt_w);
  Range rg, rx, ro, rs, rw, rd, rdw;
  if (!byte_view(DY, T, H, lddy, 1, es, &rg) || !byte_view(X, P, H, ldx, 1, es, &rx) ||
      !byte_rows(offsets, 1, 1, 8 * ((int64_t)E + 1), &ro) || !byte_rows(slots, 1, 1, 8 * P, &rs) ||
      !byte_view(weights, T, top_k, ldw, 1, ew, &rw) || !byte_view(DX, P, H, lddx, 1, es, &rd) ||
      !byte_view(DW, T, top_k, lddw, 1, ew, &rdw))
    return GEMM_ERR_SHAPE;
  for (const Range& in : {rg, rx, ro, rs, rw})
    if (overlap(rd, in) || overlap(rdw, in)) return GEMM_ERR_ALIAS;
  if (overlap(rd, rdw)) return GEMM_ERR_ALIAS;
  RowsArgs a{};
  a.in = X;
  a.ldi = ldx * es;
  a.dy = DY;
  a.ldy = lddy * es;
  a.out = DX;
  a.ldo = lddx * es;
  a.slots = slots;
  a.ld_slots = top_k;
  a.placed = offsets + E;
  a.weights = weights;
  a.ldw = ldw;
  a.dweights = DW;
  a.lddw = lddw;
  a.w32 = fmt_w == GEMM_FMT_F32;
  a.T = T;
  a.P = P;
  a.H = H;
  a.top_k = top_k;
  const bool o = once(T, 2 * P, H * es);
  const void* fn = fmt == GEMM_FMT_F16    ? GEMM_ONCE(moe_combine_back_kernel, MX_F16, o)
                   : fmt == GEMM_FMT_BF16 ? GEMM_ONCE(moe_combine_back_kernel, MX_BF16, o)
                                          : GEMM_ONCE(moe_combine_back_kernel, MX_F32, o);
  return run(fn, dim3((unsigned)T), 256, &a, (hipStream_t)stream);
}

}  // extern "C"
