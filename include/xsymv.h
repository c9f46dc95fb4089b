/*
 * xsymv.h -- C ABI of the MI355X (gfx950) symmetric / Hermitian matrix-vector
 * product library (libxsymv.so).
 *
 *   y := alpha*S*x + beta*y
 *
 * S is an n x n symmetric matrix (xsymv_s, xsymv_d, xsymv_w) or Hermitian
 * matrix (xhemv_c, xhemv_z) of which only one triangle is stored and read.
 * The operation is eq.(1) of the CUDA-xSYMV report (Imamura, Mukunoki,
 * Yamada, Machida; IPSJ SIG Technical Report 2014-HPC-146 No.14, §1), and the
 * argument list is the BLAS one the report gives for its API (§2.2 Fig. 5),
 * with the HIP stream appended.  Element types: §2.2 (interleaved complex
 * pairs for [CZ]HEMV, double-double pairs for WSYMV).
 *
 * Arguments (all calls):
 *   uplo   'U'/'u': the upper triangle of A is stored; 'L'/'l': the lower.
 *          The other strict triangle is never read (it may hold anything).
 *   n      order of S, n >= 0.
 *   alpha, beta  host scalars, by value.
 *   A      DEVICE pointer, column-major, element (i, j) at A[i + j*lda];
 *          read only.  For the Hermitian calls the imaginary word of a
 *          diagonal element is never read (it is taken as zero).
 *   lda    leading dimension, lda >= max(1, n).
 *   x      DEVICE pointer, n elements with stride incx (incx != 0; a
 *          negative stride walks the vector backwards, as in BLAS); read only.
 *   y      DEVICE pointer, n elements with stride incy (incy != 0); updated
 *          in place.  With beta == 0 the old y is not read (may hold NaN).
 *   stream a hipStream_t (NULL = the default stream).
 *
 * Ownership: A, x and y belong to the caller and must stay valid until the
 * work enqueued on `stream` has finished.  The library keeps a device
 * workspace per (device, stream), allocated on first use and grown as needed
 * (hipMalloc), never exposed in results, unless the caller installs one with
 * xsymv_set_workspace.  Calls on one stream are ordered; calls on different
 * streams use different workspaces.
 *
 * Behaviour: every call is asynchronous on `stream` (it enqueues kernels and
 * returns).  Results are bitwise identical from run to run for the same
 * inputs, n, uplo and tile configuration: no floating-point atomics are used
 * and partial sums are combined in a fixed order.  n == 0, or alpha == 0 with
 * beta == 1, returns without touching y.  alpha == 0 scales y by beta only
 * (A and x are not read).
 *
 * HIP graphs: the first call of a shape (precision, uplo, n, configuration)
 * builds its work split and uploads it with a synchronising copy, and the
 * first call on a stream may allocate that stream's workspace; neither is
 * allowed while a stream is being captured.  A later call of the same shape
 * on a stream that has already run one enqueues only kernels and can be
 * recorded into a graph and replayed (with timing off).
 *
 * Return codes (checked before any device work; numbering follows the
 * argument positions, as BLAS xerbla does):
 *    0  success
 *   -1  uplo is not one of U, u, L, l
 *   -2  n < 0
 *   -4  A is NULL and n > 0
 *   -5  lda < max(1, n)
 *   -6  x is NULL and n > 0
 *   -7  incx == 0
 *   -9  y is NULL and n > 0
 *  -10  incy == 0
 *  1000 + e  the HIP runtime returned error e (hipError_t) on allocation,
 *            copy or launch.
 *  2000      the workspace the caller installed for this stream
 *            (xsymv_set_workspace) is smaller than the call needs; nothing
 *            was enqueued.
 */
#ifndef XSYMV_H
#define XSYMV_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct { float re, im; } xcomplex64;   /* layout of float2 */
typedef struct { double re, im; } xcomplex128; /* layout of double2 */
typedef struct { double hi, lo; } xdd;         /* value = hi + lo */

/* Precision codes for the helper calls below. */
enum { XSYMV_S = 0, XSYMV_D = 1, XSYMV_C = 2, XSYMV_Z = 3, XSYMV_W = 4 };

/* SSYMV, DSYMV: real symmetric, float / double (report §2.2 Fig. 5). */
int xsymv_s(char uplo, int n, float alpha, const float *A, int lda,
            const float *x, int incx, float beta, float *y, int incy,
            void *stream);
int xsymv_d(char uplo, int n, double alpha, const double *A, int lda,
            const double *x, int incx, double beta, double *y, int incy,
            void *stream);

/* CHEMV, ZHEMV: complex Hermitian (report §2.2 Fig. 5).  The mirrored
 * element is the conjugate: S(j,i) = conj(A(i,j)). */
int xhemv_c(char uplo, int n, xcomplex64 alpha, const xcomplex64 *A, int lda,
            const xcomplex64 *x, int incx, xcomplex64 beta, xcomplex64 *y,
            int incy, void *stream);
int xhemv_z(char uplo, int n, xcomplex128 alpha, const xcomplex128 *A, int lda,
            const xcomplex128 *x, int incx, xcomplex128 beta, xcomplex128 *y,
            int incy, void *stream);

/* WSYMV: double-double symmetric (report §2.2 Fig. 4 and Fig. 5).  Inputs
 * need not be normalised; outputs are (hi, lo) with hi = RN(hi + lo).  The
 * accumulations use double-double multiply-adds with one TwoSum of the high
 * words (the cheaper addition of the double-double library the report
 * builds on), merges and reductions the accurate addition; every result is
 * within 4*n*2^-104*(|alpha|*(|S||x|)_i + |beta|*|y_i|) of the exact value. */
int xsymv_w(char uplo, int n, xdd alpha, const xdd *A, int lda,
            const xdd *x, int incx, xdd beta, xdd *y, int incy,
            void *stream);

/* xGEMV, the general product the report sets SYMV against (a general matrix
 * is read whole and each element used once; the symmetric product reads one
 * triangle and uses each element twice, so it moves half the bytes -- report
 * §1, §2.1):
 *
 *   y := alpha*op(A)*x + beta*y,  op(A) = A (trans 'N'/'n'), A^T ('T'/'t')
 *                                or A^H ('C'/'c'; the same as 'T' for the
 *                                real and double-double types)
 *
 * BLAS xGEMV arguments: A is m x n, column-major, DEVICE pointer, element
 * (i, j) at A[i + j*lda], rows m..lda-1 never read; x has n elements for 'N'
 * and m otherwise, y the other length (DEVICE pointers, strides incx/incy as
 * for the symmetric calls).  Same ownership, asynchrony, determinism,
 * workspace (per device and stream, or installed with xsymv_set_workspace)
 * and beta == 0 / alpha == 0 rules as the symmetric calls.  m == 0, n == 0,
 * or alpha == 0 with beta == 1 return without touching y.
 *
 * Return codes (BLAS xerbla positions, checked before any device work):
 *   -1 trans not N/T/C (either case), -2 m < 0, -3 n < 0, -5 A NULL with
 *   m, n > 0, -6 lda < max(1, m), -7 x NULL, -8 incx == 0, -10 y NULL,
 *   -11 incy == 0; 1000 + hipError_t; 2000 installed workspace too small. */
int xgemv_s(char trans, int m, int n, float alpha, const float *A, int lda,
            const float *x, int incx, float beta, float *y, int incy, void *stream);
int xgemv_d(char trans, int m, int n, double alpha, const double *A, int lda,
            const double *x, int incx, double beta, double *y, int incy, void *stream);
int xgemv_c(char trans, int m, int n, xcomplex64 alpha, const xcomplex64 *A, int lda,
            const xcomplex64 *x, int incx, xcomplex64 beta, xcomplex64 *y, int incy,
            void *stream);
int xgemv_z(char trans, int m, int n, xcomplex128 alpha, const xcomplex128 *A, int lda,
            const xcomplex128 *x, int incx, xcomplex128 beta, xcomplex128 *y, int incy,
            void *stream);
int xgemv_w(char trans, int m, int n, xdd alpha, const xdd *A, int lda, const xdd *x,
            int incx, xdd beta, xdd *y, int incy, void *stream);

/* xGEMV configurations: each precision has a compiled list; info gives
 * waves per workgroup, stripes per wave, columns per group, non-temporal
 * loads (0/1) and rows per strip (outputs may be NULL; returns 0 or -1 for
 * a bad index).  Built in: one configuration per (precision, 'N' or a
 * transposition, size class of m*n: below 12288^2, below 20000^2, larger),
 * the fastest measured on MI355X at one order in each class.  select forces
 * entry idx for every later call of that precision; idx = -1 restores the
 * built-in choice (0 or -1 for a bad code or index).  current: the
 * configuration a call (prec, trans, m, n) runs (-1 for a bad code, trans,
 * m or n).  workspace_bytes: device workspace of one call on the current
 * device with that configuration (-1 cast to size_t on a bad code or when
 * the device cannot be queried).  xgemv_plan: the work split for m x n, strips of R
 * rows and G workgroups (host computation; blocks4 as for xsymv_strip_plan,
 * seg_base[NS+1]); returns the number of workgroups, -1 or -2. */
int xgemv_num_configs(int prec);
int xgemv_config_info(int prec, int idx, int *waves, int *stripes_per_wave,
                      int *cols_per_group, int *nontemporal, int *rows_per_strip);
int xgemv_select_config(int prec, int idx);
int xgemv_current_config(int prec, char trans, int m, int n);
size_t xgemv_workspace_bytes(int prec, char trans, int m, int n);
int xgemv_plan(int m, int n, int R, int G, int *blocks4, int max_blocks, int *seg_base,
               int max_strips);

/* Symmetric / Hermitian rank-2 update on the stored triangle (the report's
 * §5 carries the approach to other Level-2 BLAS; this is SYMV's partner in
 * reductions to tridiagonal form), BLAS xSYR2 / xHER2:
 *
 *   xsyr2_s/d/w:  A := alpha*x*y^T + alpha*y*x^T + A
 *   xher2_c/z:    A := alpha*x*y^H + conj(alpha)*y*x^H + A  (the diagonal
 *                 stays real: its imaginary word is written as zero)
 *
 * uplo as for the symmetric product; only the stored triangle of A (DEVICE
 * pointer, column-major, lda >= max(1, n)) is read and written -- the other
 * triangle and rows n..lda-1 are never touched.  x, y: DEVICE pointers, n
 * elements with strides incx, incy (!= 0; negative walks backwards).
 * Every stored element is updated by one lane in the BLAS reference order
 * (per column j: t1 = alpha*conj(y_j), t2 = conj(alpha*x_j),
 * a := (a + x_i*t1) + y_i*t2; Hermitian diagonal: Re(a) + Re(x_j*t1 +
 * y_j*t2)), without fused multiply-adds, so the results do not depend on the
 * work split.  n == 0 or alpha == 0: nothing is done.  Asynchronous on
 * `stream`; a workspace (2n elements) is used only for non-unit strides.
 * Return codes (BLAS xerbla positions): -1 uplo, -2 n < 0, -4 x NULL,
 * -5 incx == 0, -6 y NULL, -7 incy == 0, -8 A NULL, -9 lda < max(1, n);
 * 1000 + hipError_t; 2000 installed workspace too small. */
int xsyr2_s(char uplo, int n, float alpha, const float *x, int incx, const float *y,
            int incy, float *A, int lda, void *stream);
int xsyr2_d(char uplo, int n, double alpha, const double *x, int incx, const double *y,
            int incy, double *A, int lda, void *stream);
int xher2_c(char uplo, int n, xcomplex64 alpha, const xcomplex64 *x, int incx,
            const xcomplex64 *y, int incy, xcomplex64 *A, int lda, void *stream);
int xher2_z(char uplo, int n, xcomplex128 alpha, const xcomplex128 *x, int incx,
            const xcomplex128 *y, int incy, xcomplex128 *A, int lda, void *stream);
int xsyr2_w(char uplo, int n, xdd alpha, const xdd *x, int incx, const xdd *y, int incy,
            xdd *A, int lda, void *stream);

/* Rank-2 update configurations: waves per workgroup, stripes per wave,
 * columns per group, non-temporal access (0/1), work split (the cost models
 * of xsymv_strip_plan: 0 strip height, doubled in the diagonal triangle; 1
 * stored rows plus strip height; 2 strip height alone) and rows per strip.
 * Built in: one configuration per (precision, triangle, size class of n:
 * below 12288, below 20000, larger), the fastest measured on MI355X at one
 * order in each class.  select forces entry idx for every later call of
 * that precision; idx = -1 restores the built-in choice (0 or -1 for a bad
 * code or index).  current: the configuration a call (prec, uplo, n) runs
 * (-1 for a bad code, uplo or n). */
int xsyr2_num_configs(int prec);
int xsyr2_config_info(int prec, int idx, int *waves, int *stripes_per_wave,
                      int *cols_per_group, int *nontemporal, int *split,
                      int *rows_per_strip);
int xsyr2_select_config(int prec, int idx);
int xsyr2_current_config(int prec, char uplo, int n);

/* One GPU's share of the product, for the path sharded over several GPUs
 * (the report's §5 points to multi-GPU SYMV, its ref. [7]); on one GPU the
 * shards run one after another.  The columns are cut into panels of `panel`
 * consecutive columns (the last may be short), dealt to `nshards` shards
 * round by round: in even rounds shard g takes the round's g-th panel, in
 * odd rounds its (nshards-1-g)-th, which keeps the shards' triangle areas
 * close.  xsymv_shard_columns writes the global columns of `shard`
 * (ascending; cols may be NULL) and returns their count (-1: bad argument);
 * a host computation.
 *
 *   x[sd]symv_shard_X / xhemv_shard_[cz]:  p := the shard's share of S*x --
 *   every stored element A(i,j) of an owned column j taken in both roles
 *   (p_i += A(i,j) x_j, and p_j += conj(A(i,j)) x_i for i != j), the
 *   diagonal once (Hermitian: its real word) -- so that the shards' partials
 *   add up to S*x.
 *
 * Aloc: DEVICE pointer to the shard's local matrix, its columns in ascending
 * global order, each a full column of A (rows 0..n-1 at stride lda >=
 * max(1, n); only the uplo triangle is read).  x: DEVICE, n elements, stride
 * incx != 0.  p: DEVICE, n contiguous elements, overwritten (zeros when the
 * shard owns no column).  Deterministic: fixed-order partial sums, no
 * atomics.  Asynchronous on `stream`; uses the per-stream workspace
 * (xsymv_shard_workspace_bytes).  Codes: -1 uplo, -2 n < 0, -3 panel <= 0,
 * -4 nshards <= 0, -5 shard outside [0, nshards), -6 Aloc NULL while the
 * shard owns columns, -7 lda < max(1, n), -8 x NULL, -9 incx == 0,
 * -10 p NULL; 1000 + hipError_t; 2000 installed workspace too small.
 *
 *   xsymv_combine_X / xhemv_combine_[cz]:  y := beta*y + alpha*(P[0] + P[1]
 *   + ... + P[nshards-1]), partial g at P + g*ldp (DEVICE, n elements each),
 *   summed in rank order -- the fixed order that keeps the result the same
 *   from run to run, whatever the exchange did.  BLAS rules: beta == 0 does
 *   not read y, alpha == 0 does not read P, n == 0 or (alpha == 0 and
 *   beta == 1) returns at once.  y: DEVICE, stride incy != 0.  Codes: -1 n,
 *   -2 nshards <= 0, -4 P NULL, -5 ldp < max(1, n), -7 y NULL, -8 incy == 0;
 *   1000 + hipError_t. */
int xsymv_shard_columns(int n, int panel, int nshards, int shard, int *cols);
/* The work split of one shard's product (host computation, as
 * xsymv_strip_plan, over the shard's local columns): blocks4, strip_base and
 * seg_base as there, col0 (NS entries) the first local column of each
 * strip's sequence.  A strip without any of the shard's columns has an empty
 * sequence and (unless a workgroup's range steps through it) no segment.
 * Returns the number of workgroups (0 when the shard owns no column), -1 for
 * bad arguments, -2 if an output is too small. */
int xsymv_shard_plan(char uplo, int n, int R, int G, int split, int panel, int nshards,
                     int shard, int *blocks4, int max_blocks, int *strip_base, int *seg_base,
                     int *col0, int max_strips);
size_t xsymv_shard_workspace_bytes(int prec, char uplo, int n, int panel, int nshards,
                                   int shard);
int xsymv_shard_s(char uplo, int n, int panel, int nshards, int shard, const float *Aloc,
                  int lda, const float *x, int incx, float *p, void *stream);
int xsymv_shard_d(char uplo, int n, int panel, int nshards, int shard, const double *Aloc,
                  int lda, const double *x, int incx, double *p, void *stream);
int xhemv_shard_c(char uplo, int n, int panel, int nshards, int shard,
                  const xcomplex64 *Aloc, int lda, const xcomplex64 *x, int incx,
                  xcomplex64 *p, void *stream);
int xhemv_shard_z(char uplo, int n, int panel, int nshards, int shard,
                  const xcomplex128 *Aloc, int lda, const xcomplex128 *x, int incx,
                  xcomplex128 *p, void *stream);
int xsymv_shard_w(char uplo, int n, int panel, int nshards, int shard, const xdd *Aloc,
                  int lda, const xdd *x, int incx, xdd *p, void *stream);
int xsymv_combine_s(int n, int nshards, float alpha, const float *P, int ldp, float beta,
                    float *y, int incy, void *stream);
int xsymv_combine_d(int n, int nshards, double alpha, const double *P, int ldp, double beta,
                    double *y, int incy, void *stream);
int xhemv_combine_c(int n, int nshards, xcomplex64 alpha, const xcomplex64 *P, int ldp,
                    xcomplex64 beta, xcomplex64 *y, int incy, void *stream);
int xhemv_combine_z(int n, int nshards, xcomplex128 alpha, const xcomplex128 *P, int ldp,
                    xcomplex128 beta, xcomplex128 *y, int incy, void *stream);
int xsymv_combine_w(int n, int nshards, xdd alpha, const xdd *P, int ldp, xdd beta, xdd *y,
                    int incy, void *stream);

/* Triangular matrix-vector product (another of the Level-2 BLAS the report's
 * §5 carries the approach to), BLAS xTRMV:
 *
 *   x := op(T)*x,   op(T) = T ('N'), T^T ('T') or T^H ('C'; = 'T' for the
 *                   real types s, d, w)
 *
 * T is the uplo triangle of A (DEVICE pointer, column-major, lda >=
 * max(1, n)); diag 'N' takes the diagonal from A, 'U' takes ones and never
 * reads it.  The other triangle and rows n..lda-1 are never read.  x: DEVICE
 * pointer, n elements with stride incx (!= 0; negative walks backwards),
 * overwritten in place; gaps between strided elements are left alone.  Each
 * output is a fixed-order sum of partial sums (no atomics), so repeated calls
 * give identical bits.  The library reads all of x before it writes any of
 * it.  n == 0: nothing is done.  Asynchronous on `stream`; uses the
 * per-stream workspace (xtrmv_workspace_bytes).  Return codes (BLAS xerbla
 * positions): -1 uplo, -2 trans, -3 diag, -4 n < 0, -5 A NULL,
 * -6 lda < max(1, n), -7 x NULL, -8 incx == 0; 1000 + hipError_t; 2000
 * installed workspace too small. */
int xtrmv_s(char uplo, char trans, char diag, int n, const float *A, int lda, float *x,
            int incx, void *stream);
int xtrmv_d(char uplo, char trans, char diag, int n, const double *A, int lda, double *x,
            int incx, void *stream);
int xtrmv_c(char uplo, char trans, char diag, int n, const xcomplex64 *A, int lda,
            xcomplex64 *x, int incx, void *stream);
int xtrmv_z(char uplo, char trans, char diag, int n, const xcomplex128 *A, int lda,
            xcomplex128 *x, int incx, void *stream);
int xtrmv_w(char uplo, char trans, char diag, int n, const xdd *A, int lda, xdd *x,
            int incx, void *stream);

/* Triangular product configurations, same fields as the rank-2 update's.
 * Built in: one configuration per (precision, triangle, 'N' or a
 * transposition, size class of n: below 12288, below 20000, larger), the
 * fastest measured on MI355X at one order in each class.
 * xtrmv_select_config(prec, idx) forces configuration idx for every call of
 * that precision; idx = -1 restores the built-in choice (0, or -1 for a bad
 * code or index).  xtrmv_current_config: the configuration a call (prec,
 * uplo, trans, n) would use now (-1 for a bad code, uplo, trans or n).  xtrmv_workspace_bytes:
 * device workspace bytes of one call (precision, uplo, trans, n) with that
 * configuration on the current device (0 for n <= 0; -1 cast to size_t on a
 * bad precision code or when the device cannot be queried). */
int xtrmv_num_configs(int prec);
int xtrmv_config_info(int prec, int idx, int *waves, int *stripes_per_wave,
                      int *cols_per_group, int *nontemporal, int *split,
                      int *rows_per_strip);
int xtrmv_select_config(int prec, int idx);
int xtrmv_current_config(int prec, char uplo, char trans, int n);
size_t xtrmv_workspace_bytes(int prec, char uplo, char trans, int n);

/* Operators on rows in 8 bits -- the integer side of a layer that serves a
 * language model: rows are made by a norm, a gated activation or a cache's
 * store, and read back or multiplied with rows of weights.  A row of n
 * numbers v_j is held as n signed codes and one 32-bit scale:
 *
 *   a = max(max_j |v_j|, 2^-100)
 *   code_j = round_half_even(v_j * (127 / a)),  scale = a / 127
 *   value_j = code_j * scale
 *
 * A row that holds an infinity or a NaN gets a scale that is not finite and
 * reads back as NaN throughout; other rows are not touched by it.
 *
 * Matrices are in ROW order, DEVICE pointers: element (i, j) at p[i*ld + j],
 * ld >= max(1, row length), any alignment.  The gap after a row is never
 * written; the product may read the gap between two rows (what it holds does
 * not matter), nothing reads past the last row's end.  The letter of a call is
 * the type of its rows: s float, h IEEE half, b bfloat16 (16-bit words);
 * arithmetic and scales are in 32 bits, the norm's sum of squares in 64.  Calls
 * are asynchronous on `stream`, can be captured into a graph, and give the same
 * bytes every time.  m == 0 or n == 0: nothing is done.  Codes are checked in
 * the order of the arguments before any device work; pointers are only needed
 * where there are rows.
 *
 *   xsymv_q8norm_*:  h = x + r (rounded to r's type), v = h / sqrt(mean(h^2)
 *   + eps) * w, stored as codes q and scales (one a row).  rtype, wtype: the
 *   letter of r and h, and of w (n elements): the call's own letter or 's'.
 *   r NULL: no residual, h = x.  h NULL: not kept.  h may be r itself (with
 *   ldh == ldr) or x itself (with ldh == ldx, and r of x's type); nothing else
 *   may overlap an output.  Codes: -1 m < 0, -2 n < 0, -3 x NULL, -4 ldx,
 *   -5 rtype, -7 ldr, -8 wtype, -9 w NULL, -10 eps < 0 or not finite, -12 ldh,
 *   -13 q NULL, -14 ldq, -15 scale NULL; then -11 h is x and of another type,
 *   -12 h is x at another stride.
 *
 *   xsymv_q8glu_*:  v = g / (1 + exp(-g)) * u, stored as codes q and scales.
 *   g and u may be the halves of one matrix's rows.  Codes: -1 m, -2 n,
 *   -3 g NULL, -4 ldg, -5 u NULL, -6 ldu, -7 q NULL, -8 ldq, -9 scale NULL.
 *
 *   xsymv_q8store_*:  row i of x is stored as row slot[i] of a cache of cap
 *   rows of codes q and scales; a slot outside [0, cap) leaves its row out
 *   (padding).  Slots that name a row twice leave it undefined.  slot NULL:
 *   row i is stored as row i (cap >= m), which makes codes of any rows.
 *   Codes: -1 m, -2 n, -3 x NULL, -4 ldx, -6 cap < 0 (or < m without slots),
 *   -7 q NULL, -8 ldq, -9 scale NULL.
 *
 *   xsymv_q8read_*:  out row i = the values of row slot[i] of the cache, zeros
 *   for a slot outside [0, cap); slot NULL: row i.  Codes: -1 m, -2 n,
 *   -3 q NULL, -4 ldq, -5 scale NULL, -7 cap < 0 (or < m without slots),
 *   -8 out NULL, -9 ldo.
 *
 *   xsymv_q8gemm_*:  C[i, j] = (sum_l A[i, l] * W[j, l]) * sa[i] * sw[j] +
 *   bias[j], A m x k and W n x k codes, sa (m) and sw (n) scales, bias n
 *   floats or NULL, C m x n of the call's type.  The sum is exact (32-bit
 *   integers, k <= 131071); it, its products with the scales and the sum with
 *   the bias round once each to 32 bits.  k == 0: C = bias or zeros.  Codes:
 *   -1 m, -2 n, -3 k < 0 or > 131071, -4 A NULL, -5 lda, -6 sa NULL, -7 W
 *   NULL, -8 ldw, -9 sw NULL, -11 C NULL, -12 ldc.
 *   2000 installed workspace too small.
 * All: 1000 + hipError_t.
 *
 *   Of these calls only the product uses the stream's workspace: for the sums
 *   of its shares of k, and where many rows lie at strides that are slow to
 *   read for a copy of them (up to 1 GiB).  xsymv_q8gemm_workspace_bytes is
 *   what a product of m x n x k takes at most, whatever the operands' alignment
 *   (0 where it takes none).  A call that outgrows the stream's workspace waits
 *   for the stream's earlier work while it is replaced.  Where it cannot grow,
 *   for want of device memory or because the stream is being captured, the
 *   product is made without: the same bytes, in up to several times the time.
 *   For a graph of the usual speed, run a product of the same size on the
 *   stream before, or install a workspace of that many bytes.  A graph keeps the
 *   workspace of the stream it was captured on (the library frees such a one in
 *   xsymv_release only), so its replays must not overlap with products on that
 *   stream, nor with those of another graph captured there. */
typedef unsigned short xhalf;     /* IEEE half, its 16 bits */
typedef unsigned short xbfloat16; /* bfloat16, its 16 bits */
size_t xsymv_q8gemm_workspace_bytes(int m, int n, int k);
int xsymv_q8norm_s(int m, int n, const float *x, int ldx, char rtype, const void *r,
                    int ldr, char wtype, const void *w, float eps, void *h, int ldh,
                    signed char *q, int ldq, float *scale, void *stream);
int xsymv_q8glu_s(int m, int n, const float *g, int ldg, const float *u, int ldu,
                   signed char *q, int ldq, float *scale, void *stream);
int xsymv_q8store_s(int m, int n, const float *x, int ldx, const int *slot, int cap,
                     signed char *q, int ldq, float *scale, void *stream);
int xsymv_q8read_s(int m, int n, const signed char *q, int ldq, const float *scale,
                    const int *slot, int cap, float *out, int ldo, void *stream);
int xsymv_q8gemm_s(int m, int n, int k, const signed char *a, int lda, const float *sa,
                    const signed char *w, int ldw, const float *sw, const float *bias,
                    float *c, int ldc, void *stream);
int xsymv_q8norm_h(int m, int n, const xhalf *x, int ldx, char rtype, const void *r,
                    int ldr, char wtype, const void *w, float eps, void *h, int ldh,
                    signed char *q, int ldq, float *scale, void *stream);
int xsymv_q8glu_h(int m, int n, const xhalf *g, int ldg, const xhalf *u, int ldu,
                   signed char *q, int ldq, float *scale, void *stream);
int xsymv_q8store_h(int m, int n, const xhalf *x, int ldx, const int *slot, int cap,
                     signed char *q, int ldq, float *scale, void *stream);
int xsymv_q8read_h(int m, int n, const signed char *q, int ldq, const float *scale,
                    const int *slot, int cap, xhalf *out, int ldo, void *stream);
int xsymv_q8gemm_h(int m, int n, int k, const signed char *a, int lda, const float *sa,
                    const signed char *w, int ldw, const float *sw, const float *bias,
                    xhalf *c, int ldc, void *stream);
int xsymv_q8norm_b(int m, int n, const xbfloat16 *x, int ldx, char rtype, const void *r,
                    int ldr, char wtype, const void *w, float eps, void *h, int ldh,
                    signed char *q, int ldq, float *scale, void *stream);
int xsymv_q8glu_b(int m, int n, const xbfloat16 *g, int ldg, const xbfloat16 *u, int ldu,
                   signed char *q, int ldq, float *scale, void *stream);
int xsymv_q8store_b(int m, int n, const xbfloat16 *x, int ldx, const int *slot, int cap,
                     signed char *q, int ldq, float *scale, void *stream);
int xsymv_q8read_b(int m, int n, const signed char *q, int ldq, const float *scale,
                    const int *slot, int cap, xbfloat16 *out, int ldo, void *stream);
int xsymv_q8gemm_b(int m, int n, int k, const signed char *a, int lda, const float *sa,
                    const signed char *w, int ldw, const float *sw, const float *bias,
                    xbfloat16 *c, int ldc, void *stream);

/* Several answers to one prompt -- attention, pages and log probabilities for
 * sequences that are served together from one cache of 8-bit rows.
 *
 * A cache of `pages` pages of `ps` tokens for `kvheads` heads is two matrices of
 * rows as above (codes and one scale a row), the keys and the values: token t of
 * a sequence lies in page p = table[t / ps] of the sequence's row of the table,
 * and its row for head h is
 *
 *   row = (p * kvheads + h) * ps + t % ps        (pages * kvheads * ps < 2^31)
 *
 * DEVICE arrays of int: table (seqs rows of ldt entries), len (tokens of each
 * sequence), refs (for each page the sequences that hold it; 0: a free page).  A
 * len below zero counts as zero, one above ldt * ps as that (in the attention, as
 * 2^31 - 256 at most).  Where a call takes
 * `start` (seqs + 1 ascending numbers), rows start[i] to start[i + 1] - 1 of its
 * matrices are the last tokens of sequence i, of which a sequence may have none;
 * start NULL: row i is the last token of sequence i.  Rows outside start[0] to
 * start[seqs] are left as they are.  All calls are asynchronous on `stream`, can
 * be captured into a graph (the arrays are read when it is replayed), and give
 * the same bytes every time.  Codes are checked in the order of the arguments
 * before any device work; what device arrays hold cannot be refused: numbers of
 * pages and sequences that do not exist are passed over as said below, and no
 * number in them makes a call read or write outside its arrays.  The matrices of
 * a call may not overlap where it does not say so.
 *
 *   xsymv_q8attn_*:  for each row r and head h < heads, with the keys k_t and
 *   values v_t of head h * kvheads / heads (kvheads divides heads),
 *
 *     out = sum_t e^(s_t - lse) v_t,  s_t = scale * (q . k_t),  lse = log sum_t e^(s_t)
 *
 *   over the tokens t <= len - (the sequence's rows) + (the row's place among
 *   them, from 0): a row sees the tokens up to its own.  Head h of row r is at
 *   q[r * ldq + h * hd] and out[r * ldo + h * hd], and at lse[r * heads + h] (lse
 *   NULL: not kept).  Tokens whose page is outside [0, pages) are passed over; a
 *   row that sees none gets zeros and -infinity.  Scales of tokens that a row does
 *   not see mean nothing to it, whatever they are; in vs 2^120 and more count as no
 *   numbers.  16 <= hd <= 256.
 *   Sequences first[g] to first[g + 1] - 1 (groups + 1 ascending numbers from 0
 *   to seqs) have their first shared[g] tokens in common: their rows of the table
 *   name the same pages there, as far as each one's len goes (one that has ended may
 *   stay in its group), and these are read once for all of them where that takes less
 *   time.  groups == 0: nothing is shared.  Products of 16 bits
 *   (letters h and b) or 22 (s), sums in 32.  Uses the stream's workspace, up to
 *   xsymv_q8attn_workspace_bytes; where it cannot be had (as for the product
 *   above) the call is made without, in up to many times the time.
 *   Codes: -1 rows < 0 (or rows * heads over 2^31 - 1), -2 heads < 1 or not a
 *   multiple of kvheads (or heads * hd over 2^31 - 1), -3 kvheads < 1, -4 hd < 16 or
 *   > 256, -5 q NULL, -6 ldq, -7 seqs < 0, > 65536, or not rows without start, -9 len
 *   NULL, -10 table NULL, -11 ldt < 0, -12 groups < 0 or > 65536 - seqs, -13 first
 *   NULL, -14 shared NULL, -15 k NULL, -16 ldk < hd, -17 ks NULL, -18 v NULL, -19
 *   ldv < hd, -20 vs NULL, -21 pages < 0 or too many rows, -22 ps < 1, -23 scale not
 *   finite, -24 out NULL, -25 ldo, 2000 installed workspace too small.
 *
 *   xsymv_q8pages_grow:  sequence seq[i] gets add[i] tokens more (n of them, in
 *   order; n <= 8192): free pages, the lowest first, are entered in its row of
 *   the table, their refs set to one, and its len raised; got[i] = add[i].
 *   A sequence that does not exist, that is listed before, whose tokens would not
 *   fit its row of the table, or for which not enough free pages are left behind
 *   those before it in the list, stays as it is: got[i] = 0 (entries of its row
 *   behind its pages may become -1).  While grow or fork runs, len of a sequence
 *   that it lists (fork: as a child) may hold another number.  Codes: -1 n < 0 or >
 *   8192, -2 seq NULL, -3 add NULL, -4 seqs < 0, -5 len NULL, -6 table NULL, -7
 *   ldt < 0, -8 pages < 0, -9 ps < 1, -10 refs NULL, -11 got NULL.
 *
 *   xsymv_q8pages_slots:  slot[r * kvheads + h] = the cache's row of row r's token
 *   and head h, for xsymv_q8store_*; -1 where there is none.  Codes: -1 rows < 0,
 *   -2 kvheads < 1, -4 seqs < 0, or not rows without start, -5 len NULL, -6 table
 *   NULL, -7 ldt < 0, -8 pages < 0 or too many rows, -9 ps < 1, -10 slot NULL.
 *
 *   xsymv_q8pages_fork:  sequence child[i], which is empty (len 0), becomes a copy
 *   of parent[i] as that was before the call (n <= 8192): it holds the parent's
 *   whole pages too (their refs are raised) and a page of its own, the lowest
 *   free one, for a last page that is not full: src[i] = the parent's, dst[i] =
 *   the new one, for xsymv_q8pages_copy; both -1 where the last page is full.
 *   Both -2, and nothing done, where one of them does not exist, the child is not
 *   empty or listed before, or no free page is left.  Codes: -1 n < 0 or > 8192,
 *   -2 parent NULL, -3 child NULL, -4 seqs < 0, -5 len NULL, -6 table NULL, -7
 *   ldt < 0, -8 pages < 0, -9 ps < 1, -10 refs NULL, -11 src NULL, -12 dst NULL.
 *
 *   xsymv_q8pages_free:  sequence seq[i] gives its pages back: their refs are
 *   lowered, its entries become -1 and its len 0.  Sequences that do not exist are
 *   passed over; one that is listed twice is freed once.  Codes: -1 n < 0, -2 seq
 *   NULL, -3 seqs < 0, -4 len NULL, -5 table NULL, -6 ldt < 0, -7 pages < 0, -8
 *   ps < 1, -9 refs NULL.
 *
 *   xsymv_q8pages_compact:  with live[0] = the number of pages whose refs are not
 *   0, the live pages from place live[0] on are to move to the free places before
 *   it, the k-th of them (ascending) to the k-th place: src and dst list them for
 *   xsymv_q8pages_copy (pages / 2 entries each, -1 behind the last), out and rout
 *   are the table and refs as they are then (they may be table, with ldo == ldt,
 *   and refs); entries that name no live page become -1.  Codes: -1 seqs < 0, -2
 *   table NULL, -3 ldt < 0, -4 out NULL, -5 ldo < ldt, or not ldt where out is
 *   table, -6 pages < 0, -7 refs NULL, -8 rout NULL, -9 src NULL, -10 dst NULL,
 *   -11 live NULL.
 *
 *   xsymv_q8pages_copy:  page src[i] is copied to page dst[i], `rows` rows (kvheads
 *   * ps) of hd codes and their scales, of the keys and of the values (v NULL: of
 *   k alone), in each of `layers` caches of which one lies `stride` rows behind the
 *   other in the same matrices.  Pairs with a number outside [0, pages) are passed
 *   over.  A page that is the dst of two pairs, or of one and the src of another,
 *   is left undefined.  Codes: -1 n < 0, -2 src NULL, -3 dst NULL, -4 pages < 0, or
 *   pages * rows over 2^31 - 1, -5 rows < 0, -6 hd < 0, -7 k NULL, -8 ldk < hd, -9
 *   ks NULL, -11 ldv < hd, -12 vs NULL, -13 layers < 0, -14 stride < pages * rows
 *   with more than one layer.
 *
 *   xsymv_logp_*:  of m rows of n logits, log probabilities with lse = log sum_j
 *   e^(x_j): logp[i] = x[token[i]] - lse (0 for a token outside [0, n)), entropy[i]
 *   = -sum_j p_j log p_j, lse[i]; and the `top` largest logits, the larger first
 *   and the lower index first of equal ones: index[i * ldt + r], value[i * ldt + r]
 *   = x - lse.  token (with logp), entropy, lse and value may be NULL; index only
 *   with top == 0.  Tokens of logit -infinity have no part in the entropy.  A row
 *   of these alone: lse, logp and value -infinity, entropy 0; one without tokens (n
 *   == 0): lse -infinity, logp and entropy 0.  A row that holds a NaN or +infinity:
 *   NaN, and indexes of which only is said that they differ.
 *   Uses the stream's workspace, up to xsymv_logp_workspace_bytes, as xsymv_q8attn_*
 *   does.  Codes: -1 m < 0, -2 n < 0 or > 2^31 - 4096, -3 x NULL, -4 ldx, -6 logp
 *   NULL with token, -9 top < 0, > n or > 128, -10 index NULL, -12 ldt < top, 2000.
 * All: 1000 + hipError_t. */
size_t xsymv_q8attn_workspace_bytes(int rows, int heads, int kvheads, int hd, int seqs, int groups);
size_t xsymv_logp_workspace_bytes(int m, int n, int top);
int xsymv_q8attn_s(int rows, int heads, int kvheads, int hd, const float *q, int ldq, int seqs,
                   const int *start, const int *len, const int *table, int ldt, int groups,
                   const int *first, const int *shared, const signed char *k, int ldk,
                   const float *ks, const signed char *v, int ldv, const float *vs, int pages,
                   int ps, float scale, float *out, int ldo, float *lse, void *stream);
int xsymv_logp_s(int m, int n, const float *x, int ldx, const int *token, float *logp, float *entropy,
                 float *lse, int top, int *index, float *value, int ldt, void *stream);
int xsymv_q8attn_h(int rows, int heads, int kvheads, int hd, const xhalf *q, int ldq, int seqs,
                   const int *start, const int *len, const int *table, int ldt, int groups,
                   const int *first, const int *shared, const signed char *k, int ldk,
                   const float *ks, const signed char *v, int ldv, const float *vs, int pages,
                   int ps, float scale, xhalf *out, int ldo, float *lse, void *stream);
int xsymv_logp_h(int m, int n, const xhalf *x, int ldx, const int *token, float *logp, float *entropy,
                 float *lse, int top, int *index, float *value, int ldt, void *stream);
int xsymv_q8attn_b(int rows, int heads, int kvheads, int hd, const xbfloat16 *q, int ldq, int seqs,
                   const int *start, const int *len, const int *table, int ldt, int groups,
                   const int *first, const int *shared, const signed char *k, int ldk,
                   const float *ks, const signed char *v, int ldv, const float *vs, int pages,
                   int ps, float scale, xbfloat16 *out, int ldo, float *lse, void *stream);
int xsymv_logp_b(int m, int n, const xbfloat16 *x, int ldx, const int *token, float *logp, float *entropy,
                 float *lse, int top, int *index, float *value, int ldt, void *stream);
int xsymv_q8pages_grow(int n, const int *seq, const int *add, int seqs, int *len, int *table, int ldt,
                       int pages, int ps, int *refs, int *got, void *stream);
int xsymv_q8pages_slots(int rows, int kvheads, const int *start, int seqs, const int *len,
                        const int *table, int ldt, int pages, int ps, int *slot, void *stream);
int xsymv_q8pages_fork(int n, const int *parent, const int *child, int seqs, int *len, int *table,
                       int ldt, int pages, int ps, int *refs, int *src, int *dst, void *stream);
int xsymv_q8pages_free(int n, const int *seq, int seqs, int *len, int *table, int ldt, int pages,
                       int ps, int *refs, void *stream);
int xsymv_q8pages_compact(int seqs, const int *table, int ldt, int *out, int ldo, int pages,
                          const int *refs, int *rout, int *src, int *dst, int *live, void *stream);
int xsymv_q8pages_copy(int n, const int *src, const int *dst, int pages, int rows, int hd,
                       signed char *k, int ldk, float *ks, signed char *v, int ldv, float *vs,
                       int layers, int stride, void *stream);

/* Bytes of device workspace one call of precision `prec` and order n uses
 * with the configuration selected for it now, on the current device (0 for
 * n == 0; -1 cast to size_t for a bad precision code, or when the device
 * cannot be queried: the row-strip family's split depends on how many of
 * its workgroups the device holds at once). */
size_t xsymv_workspace_bytes(int prec, char uplo, int n);

/* Install a caller-owned device buffer of `bytes` bytes as the workspace of
 * `stream` on the current device (the optional caller-owned workspace of the
 * boundary; size it with xsymv_workspace_bytes).  Calls on that stream then
 * use it and never allocate a workspace; a call that needs more than `bytes`
 * returns 2000.  The buffer must stay valid, and must not be used by anything
 * else, while calls on the stream may still run; the library never frees it.
 * dev_ptr = NULL (with bytes = 0) removes an installed buffer, so the
 * library owns the stream's workspace again.  Replacing or removing waits for
 * the work queued on `stream` and frees a library-owned buffer of it.
 * Returns 0, -2 (NULL with bytes > 0) or 1000 + hipError_t.  Cached plans
 * (a few KB per order and configuration) are still allocated by the library. */
int xsymv_set_workspace(void *dev_ptr, size_t bytes, void *stream);

/* SSYMV for callers that cannot allocate device memory -- code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc.  The
 * same product, arguments, return codes, configuration choice, kernels and
 * work split as xsymv_s, hence the same bytes; but no device memory is ever
 * allocated (no hipMalloc, hipFree or pinned host memory, and no timing
 * events: xsymv_timing_* does not see these calls).  The partial sums and the
 * work split live in one static device array of XSYMV_STATIC_SCRATCH_BYTES
 * per GPU, part of the library's code object (every GPU the library runs on
 * holds it until the process ends).
 *
 * The first call of a shape (uplo, n, configuration) on a GPU writes the work
 * split into the array with a copy from host memory and waits for `stream`
 * (so it cannot be captured); later calls of that shape enqueue kernels only.
 * Calls on one GPU share the array: calls on one stream are ordered, but calls
 * that overlap in time on one GPU (other streams, other threads) race on it
 * and must not be issued.  Extra return codes, checked before any device work:
 *   3000  the call needs more than XSYMV_STATIC_SCRATCH_BYTES (partials of
 *         the configuration chosen for n, plus x gathered when incx != 1);
 *   3001  the configuration selected for (uplo, n) by a caller rule is not a
 *         row-strip one (column_runs 4, 5 or 6) -- only those are supported;
 *   3002  the current device index is 64 or more. */
#define XSYMV_STATIC_SCRATCH_BYTES ((size_t)32 << 20)
int xsymv_s_noalloc(char uplo, int n, float alpha, const float *A, int lda,
                    const float *x, int incx, float beta, float *y, int incy,
                    void *stream);

/* Release every library-owned workspace and cached tile plan of the current
 * device and forget installed workspaces (synchronises the device first).
 * Returns 0 or 1000 + hipError_t. */
int xsymv_release(void);

/* Tile configurations (the autotuner's search space, report §3 Table 1
 * plays this role for the report's CUDA kernels).  Each precision has a
 * fixed list of compiled configurations; xsymv_config_info describes entry
 * `idx`: waves per workgroup, columns per wave (row-strip family: columns
 * per group), stripes per tile (row-strip: waves x stripes per wave), rows
 * per stripe, non-temporal loads of A (0/1), x rows staged in LDS (0/1), and
 * the kernel family: 0 tiles, whole tile unrolled; 1 tiles, each wave walks
 * its columns one contiguous run at a time; 2 the same with the next run
 * prefetched; 3 tiles, all waves of a workgroup on one column; 4 row strips,
 * work split by strip height, doubled in the diagonal triangle; 5 row strips,
 * work split by stored rows plus strip height; 6 row strips, work split by
 * strip height alone.  Any output pointer may be NULL.  Returns 0, or -1 for a bad
 * index. */
int xsymv_num_configs(int prec);
int xsymv_config_info(int prec, int idx, int *waves, int *cols_per_wave,
                      int *stripes, int *rows_per_stripe, int *nontemporal,
                      int *x_in_lds, int *column_runs);

/* Select the configuration used for precision `prec`, uplo and every n in
 * [n_lo, n_hi] (later selections take precedence).  idx = -1 restores the
 * built-in choice for that range.  Returns 0 or -1 for bad arguments.
 *
 * Built-in choice: per (precision, uplo, range of n, stride class of lda),
 * the configuration the on-device autotuner measured fastest on MI355X over
 * a grid of orders from 64 to 32768 (the counterpart of the report's
 * per-size rules, §3 Table 3).  Stride class 0: lda * element size is a
 * multiple of 64 bytes (measured with lda = n); class 1: any other lda
 * (measured with lda = n + 1; where it has no rule, class 0's applies).
 * Entry 0 where no rule applies.  Caller selections (this call, autotune,
 * load_config) take precedence over it, for every lda. */
int xsymv_select_config(int prec, char uplo, int n_lo, int n_hi, int idx);
/* Configuration index that a call (prec, uplo, n) with a class-0 leading
 * dimension would use now; the _lda form for a given lda (-1 for a bad
 * precision or lda < 1). */
int xsymv_current_config(int prec, char uplo, int n);
int xsymv_current_config_lda(int prec, char uplo, int n, int lda);

/* Autotuner (the report's §3 tunes its CUDA kernels offline per GPU; this
 * is the on-device counterpart).  On the current device and `stream`, time
 * every compiled configuration of `prec` for (uplo, n) on device-generated
 * data: two warm-up calls, then `reps` timed calls each (HIP events; caches
 * flushed before each call when the matrix is under 1 GiB).  The lowest
 * median wins (ties: the lower index) and is installed for every n in
 * [n_lo, n_hi], as xsymv_select_config does.  Allocates, uses and frees
 * n*n elements of matrix plus vectors (and a 1 GiB flush buffer for small
 * matrices); synchronises `stream`.  best_idx and ms (median per
 * configuration, at most max_cfg entries) may be NULL.  Returns 0, -1 for a
 * bad argument, or 1000 + hipError_t. */
int xsymv_autotune(int prec, char uplo, int n, int n_lo, int n_hi, int reps,
                   void *stream, int *best_idx, float *ms, int max_cfg);
/* The same search on a matrix of leading dimension lda (>= n; -1 otherwise):
 * xsymv_autotune is this call with lda = n.  The installed rule applies to
 * every leading dimension. */
int xsymv_autotune_lda(int prec, char uplo, int n, int lda, int n_lo, int n_hi,
                       int reps, void *stream, int *best_idx, float *ms, int max_cfg);

/* Selection rules as a JSON file: {"library": ..., "rules": [{"prec": "s",
 * "uplo": "L", "n_lo": .., "n_hi": .., "waves": .., "cols_per_wave": ..,
 * "stripes": .., "nontemporal": .., "x_in_lds": .., "column_runs": ..},
 * ...]}.  Rules are matched to compiled
 * configurations by shape.  save: 0 or -1 (cannot write).  load: number of
 * rules installed (appended after the current ones, so they take
 * precedence), -1 (cannot read) or -2 (malformed).  clear: drop every caller
 * rule (back to the built-in choice).  save writes the caller rules only. */
int xsymv_save_config(const char *path);
int xsymv_load_config(const char *path);
int xsymv_clear_config(void);

/* Kernel timing for measurement.  xsymv_timing_enable(mode): 0 off (the
 * default); 1 every call times its main (streaming) kernel and its merge
 * kernel; 2 every call times itself whole.  The HIP events are bound to the
 * launches (hipExtLaunchKernel's start and stop events), so they take the
 * kernels' own start and end times.  Mode 1: main_ms runs from the main
 * kernel's start to its end, merge_ms from there to the merge's end (the
 * launch gap included).  Mode 2: no event is bound between the two kernels
 * (binding one there delays the merge by a few microseconds); main_ms is the
 * call's span, from the main kernel's start to the merge's end, and merge_ms
 * is 0.  Calls of one kernel (the rank-2 update, the shard combination)
 * record that kernel as main_ms and 0 in either mode.  xsymv_timing_read
 * waits for the recorded events, writes up to `max` (main_ms, merge_ms)
 * pairs, clears the record and returns how many it wrote (or
 * 1000 + hipError_t on failure).  xsymv_timing_enable returns 0, or -1 for
 * a mode other than 0, 1, 2. */
int xsymv_timing_enable(int mode);
int xsymv_timing_read(float *main_ms, float *merge_ms, int max);

/* Workgroups a row-strip configuration (column_runs 4, 5 or 6) is launched with
 * on the current device: the number of its workgroups the device holds at
 * once.  0 for other families, -1 for a bad index, -(1000 + hipError_t) on a
 * runtime error. */
int xsymv_config_workgroups(int prec, int idx, char uplo);

/* The row-strip work split the library uses for order n, strips of R rows,
 * G workgroups and cost model `split` (0: every column of a strip costs the
 * strip's height, doubled in its diagonal triangle -- family 4; 1: a column
 * costs its stored rows plus the strip's height -- family 5; 2: every column
 * costs the strip's height -- family 6), a host
 * computation with no device work: writes per workgroup
 * {first, end} of its range in the strips' concatenated column sequence,
 * its first segment slot and the strip of `first` into blocks4 (4 ints per
 * workgroup), the sequence position where each strip starts (NS+1 entries)
 * into strip_base and each strip's first segment slot (NS+1 entries, the
 * last = total segments) into seg_base.  Returns the number of workgroups
 * used, -1 for bad arguments, -2 if an output is too small. */
int xsymv_strip_plan(char uplo, int n, int R, int G, int split, int *blocks4,
                     int max_blocks, int *strip_base, int *seg_base, int max_strips);

/* Measurement helper: the device's plain streaming-read bandwidth, the
 * reference for "% of a measured stream-read peak" (the report puts its
 * results against both the specification and a measured bandwidth, §4).
 * Allocates `bytes` (>= 64 MiB) of device memory, fills it, then, for each
 * of ten layouts, times `reps` launches (after one warm-up) on `stream`:
 * 2048, 8192 or 32768 workgroups of 256 lanes, each reading its own
 * contiguous chunk with 4 or 8 non-temporal 16-byte loads in flight per
 * lane; and 256 or 512 workgroups of 1024 lanes sweeping the buffer together
 * in tiles of 2 or 4 such loads per lane (tile t to workgroup t mod grid).
 * Frees the buffer and synchronises the stream.  Writes the best layout's
 * median rate and the best single launch in GB/s (either may be NULL).
 * Returns 0, -1 for bad arguments or 1000 + hipError_t. */
int xsymv_read_bandwidth(size_t bytes, int reps, void *stream, float *gbps,
                         float *best_gbps);

/* Measurement helper: the device's plain read + write bandwidth, the
 * reference for the rank-2 update, which reads the stored triangle and
 * writes it back (the report sets its results beside a measured copy rate as
 * well as the specification, §4).  Allocates 2 * `bytes` (bytes >= 64 MiB),
 * fills them, then for each of four layouts (2048 or 8192 workgroups of 256
 * lanes, each copying its own contiguous chunk from one buffer to the other
 * with 4 or 8 non-temporal 16-byte loads and stores in flight per lane) times
 * `reps` launches after one warm-up.  Rates count the bytes read plus the
 * bytes written.  Writes the best layout's median rate and the best single
 * launch in GB/s (either may be NULL); frees the buffer and synchronises the
 * stream.  Returns 0, -1 for bad arguments or 1000 + hipError_t. */
int xsymv_copy_bandwidth(size_t bytes, int reps, void *stream, float *gbps, float *best_gbps);

/* Library version string. */
const char *xsymv_version(void);

#ifdef __cplusplus
}
#endif
#endif
