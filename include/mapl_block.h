/*
 * mapl_block.h -- C ABI of the operators between a pipeline stage's boundary and
 * its loss: the block edge with an 8-bit output, attention over packed sequences and
 * the last stage's loss, the latter two with their backward passes.  Same library and
 * conventions as mapl.h and mapl_stage.h: device pointers owned by the caller, no
 * allocation, work enqueued on `stream` without synchronising, host validation before
 * anything is enqueued, status codes MAPL_OK / MAPL_ERR_*.  Pointers need the
 * alignment of their element type only, except workspaces (16 bytes).  `dt`
 * (MAPL_BF16 or MAPL_F32) is the storage type of every floating-point tensor
 * unless stated otherwise; sums, softmax statistics and norms are fp32, each output
 * is rounded once to its type, nearest even.
 */
#ifndef MAPL_BLOCK_H
#define MAPL_BLOCK_H

#include "mapl_stage.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * The edge of a block whose normed output leaves as the operand of the 8-bit
 * projections behind it: stage_norm (mapl_stage.h) with
 *
 *   pkH = the pack of H [N][d] as fp8_pack makes it with square = 0,
 *
 * from H before its rounding to bf16 (fp32: of H as it is stored).  The rows' roots
 * and the products with them are fp64; bf16 outputs, and codes beside them, are
 * rounded once from there.  X_out and H are stored where they are not NULL (a backward
 * pass needs X_out, and H for the transposed operand of the weight gradient); w_pre is
 * required.  pkH is 16-byte aligned (MAPL_ERR_ARG) and of fp8_pack_bytes(N, d)
 * (MAPL_ERR_WORKSPACE), sizes as for both.  The backward pass is that of stage_norm.
 * Other rules as for stage_norm.
 * ---------------------------------------------------------------------- */
int stage_norm_pack(const void* X, const void* Y, const void* w_post, const void* gate, const void* w_pre,
                    void* X_out, void* H, void* pkH, size_t pkH_bytes, float res_scale, float eps, double p,
                    uint64_t seed, uint64_t offset, int64_t N, int64_t d, int64_t gate_rows, mapl_dtype dt,
                    hipStream_t stream);

/* ------------------------------------------------------------------------
 * Causal attention over packed sequences, grouped heads.
 *
 * The rows 0 .. N - 1 hold S sequences one behind the other: sequence s has the
 * rows cu[s] .. cu[s + 1] - 1 (cu [S + 1], int32, on the device, ascending, within
 * [0, N]; a sequence may be empty).  Query head h reads key head h / (Hq / Hkv).
 * Row i sees the rows j of its own sequence up to itself, start(i) <= j <= i:
 *
 *   s_ij  = scale * q_i . k_j
 *   lse_i = log sum_j exp(s_ij)                              (natural)
 *   o_i   = sum_j exp(s_ij - lse_i) v_j
 *
 * Q, O are N rows of Hq heads of D values, K, V of Hkv heads; row n of a tensor
 * begins at n times its leading dimension (ldq >= Hq D, ... ; in elements), so that
 * the three may be columns of one fused projection.  lse [Hq][N], fp32.  Rows
 * outside the sequences are neither read into a result nor written.  What a row
 * does not see never reaches it, infinities and NaN included; among what it sees
 * they act as in the formula (a row that sees only scores of -inf is NaN).  Products
 * q_i . k_j and scores have to be finite in fp32; rows whose largest score is beyond
 * 2^27 in size are formed one by one, some 250 times as slowly as others.
 * bf16: the weights exp(s_ij - m), m near the row's largest score, are rounded to
 * bf16 for the product with V, their sum is not.
 *
 * 1 <= D <= 128, Hkv >= 1 divides Hq, S >= 0, 0 <= N <= 2^28, N Hq <= 2^30, leading
 * dimensions to 2^22 (MAPL_ERR_SHAPE); 2^-64 <= scale <= 2^64 (MAPL_ERR_ARG).
 * Outputs may not overlap inputs.
 * The edges are data on the device and are not checked; edges that break the rules
 * give wrong rows, and never an access outside the tensors' N rows.
 * ---------------------------------------------------------------------- */
int stage_attn(const void* Q, const void* K, const void* V, const int32_t* cu, void* O, float* lse, float scale,
               int64_t S, int64_t N, int64_t Hq, int64_t Hkv, int64_t D, int64_t ldq, int64_t ldk, int64_t ldv,
               int64_t ldo, mapl_dtype dt, hipStream_t stream);

/* Backward of stage_attn, from its inputs and its stored O and lse, given gO = dL/dO:
 *
 *   p_ij  = exp(s_ij - lse_i),  delta_i = gO_i . o_i
 *   ds_ij = p_ij (gO_i . v_j - delta_i)
 *   gQ_i  = scale sum_j ds_ij k_j
 *   gK_j  = scale sum_h sum_i ds_ij q_i,  gV_j = sum_h sum_i p_ij gO_i
 *
 * with h over the query heads that read the key head.  bf16: p_ij and ds_ij are
 * rounded to bf16 for the products; the sums over rows and heads are fp32 and each
 * gradient is rounded once.  lse is a number of 24 bits, so p_ij is off by up to
 * 2^-21 |lse_i| of itself: less than a rounding to bf16 up to scores of 2^12, worth
 * nothing (0, infinite or NaN) beyond 2^20.  Sums have a fixed order: results are bitwise
 * repeatable.  `ws` of stage_attn_bwd_workspace_bytes(), 16-byte aligned.  Other rules
 * as for stage_attn. */
size_t stage_attn_bwd_workspace_bytes(int64_t N, int64_t Hq, int64_t Hkv, int64_t D);
int stage_attn_bwd(const void* gO, const void* Q, const void* K, const void* V, const void* O, const float* lse,
                   const int32_t* cu, void* gQ, void* gK, void* gV, float scale, int64_t S, int64_t N, int64_t Hq,
                   int64_t Hkv, int64_t D, int64_t ldgo, int64_t ldq, int64_t ldk, int64_t ldv, int64_t ldo,
                   int64_t ldgq, int64_t ldgk, int64_t ldgv, mapl_dtype dt, void* ws, size_t ws_bytes,
                   hipStream_t stream);

/* ------------------------------------------------------------------------
 * The loss of a row of logits z (Z [N][V]) with its label and a teacher's K largest
 * logits, at temperature T:
 *
 *   lse   = log sum_v exp(z_v),  lse_T = log sum_v exp(z_v / T)
 *   q_k   = exp(t_k / T) / sum_k' exp(t_k' / T)             over the row's entries
 *   loss  = w_ce (lse - z_label)
 *         + w_kd sum_k q_k (log q_k - (z_{id_k} / T - lse_T))
 *
 * labels [N], t_ids [N][K] int32, t_logits [N][K] fp32.  A label outside [0, V)
 * (-1 by convention) is none: its term is 0.  A teacher's id outside [0, V), or a
 * t_logit of -inf, is no entry; a row without entries has no second term.  Entries of
 * one id count one by one.  labels NULL: no labels; K = 0: no teacher (t_ids,
 * t_logits may be NULL); a weight of 0 leaves its term out.  A logit of -inf has no
 * weight; other values that are not finite make what they enter NaN or infinite.
 * loss [N] and stats [N][2] = (lse, lse_T) are fp32; stats is for the backward pass.
 * Long rows of small batches are split, and their sums joined in a fixed order;
 * `ws` of stage_distill_workspace_bytes(), 16-byte aligned, may be NULL when that is
 * 0.  0 <= N <= 2^23, 1 <= V <= 2^27, N V <= 2^36, 0 <= K <= 1024 (MAPL_ERR_SHAPE);
 * T > 0, T, 1 / T and the weights finite (MAPL_ERR_ARG).
 * ---------------------------------------------------------------------- */
size_t stage_distill_workspace_bytes(int64_t N, int64_t V);
int stage_distill(const void* Z, const int32_t* labels, const int32_t* t_ids, const float* t_logits, float* loss,
                  float* stats, float temperature, float w_ce, float w_kd, int64_t N, int64_t V, int64_t K,
                  mapl_dtype dt, void* ws, size_t ws_bytes, hipStream_t stream);

/* Backward of stage_distill from its inputs and its stats, given gloss = dL/dloss
 * [N], fp32 (the mean over N rows: 1 / N in each):
 *
 *   gZ_v = gloss (w_ce (exp(z_v - lse) - 1[v = label])
 *               + w_kd / T (exp(z_v / T - lse_T) - sum_{k: id_k = v} q_k))
 *
 * with the absent terms left out; a row of neither label nor entries is 0 whatever
 * its logits.  lse and lse_T are numbers of 24 bits, so the softmaxes are off by up to
 * 2^-22 |lse| (2^-22 |lse_T|) of themselves: an offset that all of a row's logits share
 * does not count in the loss, but one of 2^16 leaves a gradient six bits.  Each element
 * is rounded once.  gZ may be Z.  Other rules as for stage_distill. */
int stage_distill_bwd(const float* gloss, const void* Z, const float* stats, const int32_t* labels,
                      const int32_t* t_ids, const float* t_logits, void* gZ, float temperature, float w_ce, float w_kd,
                      int64_t N, int64_t V, int64_t K, mapl_dtype dt, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MAPL_BLOCK_H */
