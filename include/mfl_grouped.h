/*
 * mfl_grouped.h — C ABI of products whose weights are chosen per row: the
 * rows of each group (expert, adapter) from a list of choices, the product of
 * every group's rows with its own matrix, its gradients, and the sum of a
 * token's results.
 *
 *   group_rows        places: the choices in the order of their groups
 *   gemm_tn_grouped   D(i, n) = sum_k A(r_i, k) B(g, n, k)   for every place i of group g
 *   combine_rows      out(t, c) = sum_j w(t, j) X(slot(t, j), c)
 *   gemm_tn_adapters  D(r, n) = sum_k x(r, k) W(n, k) + the low-rank term of the
 *                     group that row r's place belongs to
 *
 * Places.  offsets holds groups + 1 numbers in device memory, the first of
 * them 0, growing: group g owns the places offsets[g] .. offsets[g + 1] - 1;
 * groups without places are allowed.  r_i is rows[i] (device memory), or i
 * where rows is NULL.  The kernels hold offsets inside [0, places] whatever
 * they are (of those that then do not grow the results are undefined); a row
 * number outside A counts as a row of zeros.  Places behind the last group belong
 * to none.
 *
 * Types.  A, B and their gradients' inputs are all MFL_F16 or all MFL_BF16;
 * D and dB are of that type or MFL_F32.  Products are summed in fp32 and
 * rounded once (to nearest even) at the end.
 *
 * Addressing (elements): A(r, k) = A[r lda + k], B(g, n, k) = B[g b_group +
 * n ldb + k], D(i, n) = D[i ldd + n].  n, k and every stride are multiples of
 * 8 and every matrix is 16-byte aligned (else MFL_E_MISALIGNED); strides reach
 * past a row (MFL_E_LEADING_DIM); n, k and the rank are at least 8 (0 is
 * MFL_E_UNSUPPORTED), they and the strides between rows at most 2^21, and
 * where rows are gathered A (x) spans less than 2 GiB (MFL_E_TOO_LARGE).  At
 * most 4096 groups.
 *
 * Values of one group's rows and of its matrix never reach another group's
 * results, whatever they are.
 *
 * Ownership and execution are gemm_tn's (mfl_gemm.h): nothing is allocated,
 * kept or synchronised; work runs on `stream`.  A workspace belongs to one
 * call until that call's work is done; its size comes from the *_plan
 * function, which makes the same checks without touching the GPU.  Outputs
 * must not overlap inputs, each other or the workspace.  Results are the same
 * bits for the same arguments: no sum depends on the order workgroups run in.
 */
#ifndef MFL_GROUPED_H
#define MFL_GROUPED_H

#include <stdint.h>

#include "mfl_attention.h"    /* MFL_BF16, MFL_E_WORKSPACE */

#ifdef __cplusplus
extern "C" {
#endif

#define MFL_I32 4
#define MFL_I64 5

/* ids: `count` numbers of type MFL_I32 or MFL_I64, `top` of each token in
 * turn (count a multiple of top); those outside [0, groups) are of no group.
 * The places are the choices sorted by group, in their own order within one,
 * those of no group behind:
 *   rows[i]    (count)       the token of place i
 *   offsets[g] (groups + 1)  the first place of group g
 *   slots[c]   (count)       the place of choice c, -1 for no group
 * The workspace is 4 (groups + 1) bytes for every 4096 choices (1024 with more
 * than 256 groups), at most 256 times that; none up to 8192 (1024). */
typedef struct {
  int32_t ids_type;
  int64_t count, top, groups;
} mfl_group_rows_t;

int group_rows(const mfl_group_rows_t* a, const void* ids, int32_t* rows, int32_t* offsets,
               int32_t* slots, void* workspace, int64_t workspace_bytes, void* stream);
int group_rows_plan(const mfl_group_rows_t* a, const void* ids, const int32_t* rows,
                    const int32_t* offsets, const int32_t* slots, int64_t* workspace_bytes);

/* Kernel: FEW for groups of few rows (16, 32 or 64 places per workgroup, the
 * weights straight from memory), TILE_128 and TILE_256 square tiles staged
 * through LDS.  The lengths are on the device, so AUTO goes by their mean. */
#define MFL_GROUPED_AUTO 0
#define MFL_GROUPED_FEW 1
#define MFL_GROUPED_TILE_128 2
#define MFL_GROUPED_TILE_256 3

typedef struct {
  int32_t dtype;               /* MFL_F16 or MFL_BF16 */
  int32_t out;                 /* type of D (of dB in the backward function) */
  int32_t algo;                /* MFL_GROUPED_* */
  int64_t groups;
  int64_t places;              /* rows of D */
  int64_t a_rows;              /* rows of A; at least places if rows is NULL */
  int64_t n, k;
  int64_t lda, ldb, b_group, ldd;
} mfl_grouped_t;

/* Rows of D of no group stay as they were. */
int gemm_tn_grouped(const mfl_grouped_t* a, const void* A, const void* B, const int32_t* offsets,
                    const int32_t* rows, void* D, void* stream);
/* the same checks; on success the kernel AUTO takes */
int gemm_tn_grouped_plan(const mfl_grouped_t* a, const void* A, const void* B,
                         const int32_t* offsets, const int32_t* rows, const void* D,
                         int32_t* algo);

/* Gradients of sum(D dD):
 *   dA(i, k)    = sum_n dD(i, n) B(g, n, k)      a row per place, in A's type;
 *                                                0 for places of no group
 *   dB(g, n, k) = sum_i dD(i, n) A(r_i, k)       of type f.out; 0 for groups
 *                                                without places
 * Either may be NULL.  A row that several places share has a row of dA for
 * each of them; combine_rows adds them by token.  f.ldd is dD's stride; f.algo
 * is AUTO (else MFL_E_ALGO_CASE). */
typedef struct {
  mfl_grouped_t f;
  int64_t ldda, lddb, db_group;
} mfl_grouped_grad_t;

int gemm_tn_grouped_backward(const mfl_grouped_grad_t* a, const void* dD, const void* A,
                             const void* B, const int32_t* offsets, const int32_t* rows, void* dA,
                             void* dB, void* stream);
int gemm_tn_grouped_backward_plan(const mfl_grouped_grad_t* a, const void* dD, const void* A,
                                  const void* B, const int32_t* offsets, const int32_t* rows,
                                  const void* dA, const void* dB);

/* out(t, c) = sum over j < top of w(t, j) X(slots[t top + j], c), tokens x n;
 * a slot outside [0, x_rows) adds nothing.  weights fp32, or NULL for 1.  X
 * and out: MFL_F16 or MFL_BF16, out also MFL_F32; n and the strides multiples
 * of 8, top at most 64.  Sums in fp32 in the order of j. */
typedef struct {
  int32_t dtype, out;
  int64_t tokens, top, n;
  int64_t x_rows, ldx, ldo;
} mfl_combine_t;

int combine_rows(const mfl_combine_t* a, const void* X, const int32_t* slots,
                 const float* weights, void* out, void* stream);

/* Gradients of sum(out dout), for slots and rows as group_rows gives them
 * (rows[slots[t top + j]] = t, x_rows entries):
 *   dX(i, c) = sum over the j with slots[t top + j] = i of w(t, j) dout(t, c),
 *              t = rows[i]; 0 where there is none
 *   dw(t, j) = sum_c dout(t, c) X(slots[t top + j], c); 0 for a slot outside,
 *              or one whose row is another token
 * dw may be NULL, as it must be without weights.  a->ldo is dout's stride,
 * a->out its type, which is X's. */
int combine_rows_backward(const mfl_combine_t* a, int64_t lddx, const void* dout, const void* X,
                          const int32_t* slots, const int32_t* rows, const float* weights,
                          void* dX, float* dw, void* stream);

/* A shared projection with low-rank adapters, every place i of group g:
 *   D(r_i, n) = sum_k x(r_i, k) W(n, k) + s_g sum_j h(i, j) B(g, n, j)
 *   h(i, j)   = sum_k x(r_i, k) A(g, j, k),  j < rank
 * and for places of no group the first sum alone.  scale holds s (fp32, one
 * per group), NULL for 1.  x, W, A and B are all MFL_F16 or all MFL_BF16, D
 * also MFL_F32.  rank is a multiple of 8.
 *
 * rows holds each row of x and D at most once, NULL: places are rows; rows of
 * D that no place leads to stay as they were.  s_g h is held in fp32 (as a
 * matrix operand in three numbers of the operands' type that add up to it, with
 * fp16 to 2^-38 of the largest beside it), sums are fp32, D is rounded once.  The
 * values of an adapter reach its own rows alone, whatever they are.
 *
 * Kernels as above: FEW adds the low-rank terms row by row, the TILEs by runs
 * of one group.  Small problems of a rank up to 64 are one launch by FEW and need
 * no workspace (0 bytes, NULL will do).  For others: 4 bytes per place, 4 bytes
 * for each of places x rank numbers (6 are asked for by TILE with an fp32 D, which
 * leaves 2 of them unused), up to 32 for alignment, and with FEW
 * places x n numbers of 4 bytes for each of its parts of k, which are at most
 * one for 256 of k and about 256 / (tiles of 64 columns). */
typedef struct {
  int32_t dtype, out, algo;
  int64_t groups, places;
  int64_t x_rows;              /* rows of x and D; at least places if rows is NULL */
  int64_t n, k, rank;
  int64_t ldx, ldw, lda, a_group, ldb, b_group, ldd;
} mfl_adapters_t;

int gemm_tn_adapters(const mfl_adapters_t* a, const void* x, const void* W, const void* A,
                     const void* B, const int32_t* offsets, const int32_t* rows,
                     const float* scale, void* D, void* workspace, int64_t workspace_bytes,
                     void* stream);
int gemm_tn_adapters_plan(const mfl_adapters_t* a, const void* x, const void* W, const void* A,
                          const void* B, const int32_t* offsets, const int32_t* rows,
                          const float* scale, const void* D, int32_t* algo,
                          int64_t* workspace_bytes);

#ifdef __cplusplus
}
#endif
#endif /* MFL_GROUPED_H */
