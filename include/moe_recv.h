/*
 * moe_recv.h -- the receiver side of the expert-parallel exchange: where
 * each source's segment lands in a rank's receive buffer, and the regroup of
 * the received rows into one contiguous run per expert, ready for the
 * experts, with its inverse for the return trip; and the experts' matrix
 * products over those runs, with their gradients.  Exported by the same
 * library as moe_route.h; conventions (device pointers, caller-owned,
 * asynchronous on `stream`, host-side validation, status codes) are those of
 * moe_route.h.
 *
 * The group has R ranks; every rank is a source and a receiver.  Rank r owns
 * the contiguous experts [r*E/R, (r+1)*E/R) (the EP=8 placement example of
 * the "communication wall" explainer on juhe.plus).  Source s's send buffer
 * is one flat block cut into R segments at the prefix sums of its per-rank
 * counts, and a receive buffer is laid out the same way, the segment from
 * source s following those from sources < s (NCCL EP article on
 * hotelren.com, s3.3).  The experts then run on the received rows (Perseus
 * write-up on itsolotime.com, s1.1), so the receiver gathers each expert's
 * rows into one run: expert ascending, then source ascending, then arrival
 * order.  When the sources are consecutive token shards of one batch, that
 * order is the batch's own (expert, token) order.
 *
 * Input shared by the calls: src_offsets [R][E+1] int32, the kept expert
 * offsets of every source's dispatch layout (moe_dispatch_layout's
 * expert_offsets, one row per source, e.g. moe_dispatch_layout_chunks with
 * one chunk per source), as the count exchange delivers them to every rank.
 * Source s's segment for rank r is its send rows [src_offsets[s][r*E/R],
 * src_offsets[s][(r+1)*E/R]).  Offsets must be non-decreasing in e, and the
 * total over all sources must be < 2^31.
 *
 * Flat numbering.  The receive buffers of all R ranks lie end to end in rank
 * order, and so do their grouped buffers, so every offset below is a row of
 * one flat buffer (this is how all ranks are run on one device).  A rank
 * holding only its own buffer subtracts recv_offsets[r][0] from its rows.
 */
#ifndef MOE_RECV_H
#define MOE_RECV_H

#include "moe_route.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * moe_recv_layout -- receive offsets, expert-major segment starts, and the
 * two row maps that drive the regroup (the receiver's counterpart of
 * moe_dispatch_layout's pos / row_src).  Two launches: one workgroup for the
 * offsets, one thread per row for the maps.
 *
 *   src_offsets    [R][E+1] int32, as above.                          (in)
 *   E, R           1 <= R, R divides E, E <= MOE_MAX_EXPERTS.
 *   max_rows       entries of each row map, >= N (the total kept rows of
 *                  all sources), < 2^31.  The sum of all sources' slot
 *                  counts is always enough.
 *   recv_offsets   [R][R+1] int32: recv_offsets[r][s] is the first row of
 *                  source s's segment in rank r's region;
 *                  recv_offsets[r][R] ends the region (= the next rank's
 *                  [0]); recv_offsets[R-1][R] = N.                     (out)
 *   group_offsets  [E+1] int32: first grouped row of expert e; [E] = N.
 *                  Rank r's grouped rows start at group_offsets[r*E/R] =
 *                  recv_offsets[r][0].                                 (out)
 *   group_seg      [E][R] int32: first grouped row of source s's rows of
 *                  expert e.                                          (out)
 *   group_pos      [max_rows] int32: grouped row of receive row q for
 *                  q < N, -1 for q >= N.                               (out)
 *   group_src      [max_rows] int32: receive row held by grouped row p for
 *                  p < N (the inverse permutation), -1 for p >= N.     (out)
 *
 * Errors: MOE_ERR_NULL, MOE_ERR_SHAPE (E or R out of range, max_rows < 0 or
 * >= 2^31), MOE_ERR_ALIGN (arrays not 4-byte aligned).  With max_rows ==
 * 0 the maps may be NULL and only the offsets are written.  N > max_rows
 * leaves the maps incomplete (never written out of bounds).
 */
int moe_recv_layout(const int32_t *src_offsets, int E, int R, int64_t max_rows,
                    int32_t *recv_offsets, int32_t *group_offsets,
                    int32_t *group_seg, int32_t *group_pos, int32_t *group_src,
                    hipStream_t stream);

/*
 * moe_recv_regroup -- receive buffer -> grouped buffer:
 *     grouped[p] = recv[group_src[p]]   for every p < max_rows with
 *                                       0 <= group_src[p] < max_rows
 * and, for a quantised format, grouped_scales[p] = recv_scales[group_src[p]].
 * One workgroup per grouped row, one 16-byte vector per thread.  Rows (bf16
 * rows or quantised codes, moe_route.h) are moved unchanged; rows with a -1
 * map entry are not written.
 *
 *   recv            [max_rows rows, moe_row_bytes(H, quant)], 16-byte
 *                   aligned.                                          (in)
 *   recv_scales     [max_rows] fp32 (quantised formats; ignored, may be
 *                   NULL, for bf16).                                  (in)
 *   group_src       [max_rows] int32 from moe_recv_layout.            (in)
 *   grouped         [max_rows rows, same stride], 16-byte aligned, not
 *                   overlapping recv.                                 (out)
 *   grouped_scales  [max_rows] fp32, as recv_scales, not overlapping
 *                   it.                                               (out)
 *
 * Errors: MOE_ERR_NULL, MOE_ERR_SHAPE (H, quant as for moe_dispatch_pack;
 * max_rows < 0 or >= 2^31), MOE_ERR_ALIGN.  max_rows == 0: MOE_OK, nothing
 * launched.
 */
int moe_recv_regroup(const void *recv, const float *recv_scales, int64_t max_rows, int H,
                     int quant, const int32_t *group_src, void *grouped, float *grouped_scales,
                     hipStream_t stream);

/*
 * moe_recv_ungroup -- the inverse, after the experts: grouped buffer (the
 * experts' output rows, in grouped order) -> receive order, ready for the
 * return exchange:
 *     recv[q] = grouped[group_pos[q]]   (and the scales alike)
 * Arguments and errors as moe_recv_regroup with the buffers' roles swapped.
 */
int moe_recv_ungroup(const void *grouped, const float *grouped_scales, int64_t max_rows, int H,
                     int quant, const int32_t *group_pos, void *recv, float *recv_scales,
                     hipStream_t stream);

/* Activations of the experts' products. */
#define MOE_ACT_NONE 0   /* z                                                */
#define MOE_ACT_RELU 1   /* 0 where z <= 0 (slope 0), else z: NaN stays NaN  */
#define MOE_ACT_SILU 2   /* z / (1 + exp(-z))                                */
#define MOE_ACT_GELU 3   /* z (1 + erf(z / sqrt 2)) / 2                      */
#define MOE_ACT_SWIGLU 4 /* silu(z_gate) * z_up: two columns of z per output */

/*
 * moe_expert_matmul -- every expert's product with its own run of rows:
 *     z[p, :]   = x[p, :] W_e^T + bias_e
 *     out[p, :] = bf16_rne( act(z[p, :]) + residual[p, :] )
 * for the rows p of expert e, offsets[e] <= p + offsets[0] < offsets[e+1]:
 * row 0 of the buffers is row offsets[0] of the flat numbering, so a rank
 * holding only its own grouped buffer passes group_offsets + r*E/R and its
 * E/R experts, and the flat buffer of all ranks passes group_offsets and E.
 * E = 1 is a plain product.  bf16 inputs, fp32 sums (matrix cores); bias,
 * activation and residual are applied to the fp32 sum, which is rounded once.
 *
 *   x          [max_rows, K] bf16 bits.                               (in)
 *   offsets    [E+1] int32, device, non-decreasing: group_offsets.  (in)
 *   w          [E, N, K] bf16 bits; MOE_ACT_SWIGLU: [E, 2N, K], an expert's
 *              N gate rows, then its N up rows.                       (in)
 *   bias       [E, N] fp32 (MOE_ACT_SWIGLU: [E, 2N]), or NULL.        (in)
 *   act        MOE_ACT_*.
 *   residual   [max_rows, N] bf16 bits, or NULL; may be out itself.   (in)
 *   E, max_rows, K, N   1 <= E <= MOE_MAX_EXPERTS; 0 <= max_rows <= 2^31 -
 *              256, at least the rows of all runs (a run is cut at max_rows:
 *              nothing is read or written past it); K and N multiples of 16 in [16,
 *              MOE_MAX_HIDDEN].  A call whose outputs make 2^30 tiles of 256 x
 *              128 or more returns MOE_ERR_SHAPE.
 *   out        [max_rows, N] bf16 bits; rows of no run are not written. (out)
 *   preact     [max_rows, N] (MOE_ACT_SWIGLU: [max_rows, 2N]) bf16 bits of z
 *              rounded once, for the gradient; or NULL.               (out)
 *   workspace  NULL, or device scratch of *workspace_bytes bytes, 256-byte
 *              aligned, for calls of few outputs and a long sum, which share the
 *              sum out (up to 8 times faster; the sums' order is then another,
 *              and fixed too).  Calls that may run at once need one each.
 *   workspace_bytes  NULL, or a host pointer; with workspace NULL the size
 *              needed (0: none) is written and nothing launched.  It depends on
 *              E, max_rows, K, N and whether act is MOE_ACT_SWIGLU.
 *
 * Every array 16-byte aligned (offsets 4).  out and preact must not overlap
 * each other or the inputs (but for out == residual).
 * Errors: MOE_ERR_NULL; MOE_ERR_SHAPE; MOE_ERR_ALIGN; MOE_ERR_ALIAS (out or
 * preact starts where x or w does, or both at one place, or preact where
 * residual does); MOE_ERR_WORKSPACE when the workspace is too small or comes
 * without a size.  max_rows == 0: MOE_OK, nothing launched.
 */
int moe_expert_matmul(const void *x, const int32_t *offsets, const void *w, const float *bias,
                      int act, const void *residual, int E, int64_t max_rows, int K, int N,
                      void *out, void *preact, void *workspace, size_t *workspace_bytes,
                      hipStream_t stream);

/*
 * moe_expert_matmul_dx -- gradient of a product's input rows, carried through
 * the activation that produced them.  For z = x W_e^T and the gradient dy of
 * z:
 *     g[p, :]  = dy[p, :] W_e
 *     dx[p, :] = bf16_rne( g )                          (act MOE_ACT_NONE)
 *              = bf16_rne( act'(preact[p, :]) * g )     (x = act(preact))
 * MOE_ACT_SWIGLU: dx has 2K columns, the gate's gradient g * z_up *
 * silu'(z_gate), then the up projection's g * silu(z_gate).  preact is what
 * the forward call of the product before kept, so an expert of two products
 * takes two calls and rounds twice.  (A residual's gradient is dy itself.)
 *
 *   dy      [max_rows, N] bf16 bits.                                  (in)
 *   offsets, E, max_rows   as moe_expert_matmul.                      (in)
 *   w       [E, N, K] bf16 bits, the forward product's weights (for a
 *           product with MOE_ACT_SWIGLU, N here counts both halves).  (in)
 *   act     activation between the two products.
 *   preact  [max_rows, K] (MOE_ACT_SWIGLU: [max_rows, 2K]) bf16 bits; not
 *           used for MOE_ACT_NONE.                                    (in)
 *   dx      as preact; may be preact itself; rows of no run are not
 *           written.                                                  (out)
 *   K, N    multiples of 16 in [16, 2 * MOE_MAX_HIDDEN] (N) and [16,
 *           MOE_MAX_HIDDEN] (K).
 *   workspace, workspace_bytes   as moe_expert_matmul.
 *
 * Every array 16-byte aligned (offsets 4).  Errors: as moe_expert_matmul;
 * MOE_ERR_ALIAS when dx starts where dy or w does.
 */
int moe_expert_matmul_dx(const void *dy, const int32_t *offsets, const void *w, int act,
                         const void *preact, int E, int64_t max_rows, int K, int N, void *dx,
                         void *workspace, size_t *workspace_bytes, hipStream_t stream);

/* Flags of moe_expert_matmul_dw. */
#define MOE_GRAD_FP32 0           /* dw and dbias fp32                       */
#define MOE_GRAD_BF16 1           /* dw bf16 bits (dbias stays fp32)         */
#define MOE_GRAD_ACCUMULATE 0x100 /* add to dw and dbias (fp32 dw only)      */

/*
 * moe_expert_matmul_dw -- gradient of every expert's weights and bias:
 *     dw[e]    = sum over its rows p of dy[p, :]^T x[p, :]      [N, K]
 *     dbias[e] = sum over its rows p of dy[p, :]                [N]
 * in fp32, in a fixed order.  An expert without rows gets zeros (with
 * MOE_GRAD_ACCUMULATE: keeps what is there).
 *
 *   dy, x    [max_rows, N], [max_rows, K] bf16 bits.                  (in)
 *   offsets, E, max_rows, K, N   as moe_expert_matmul_dx.
 *   flags    MOE_GRAD_FP32 or MOE_GRAD_BF16; MOE_GRAD_FP32 |
 *            MOE_GRAD_ACCUMULATE.
 *   dw       [E, N, K] fp32 or bf16 bits.                             (out)
 *   dbias    [E, N] fp32, or NULL.                                    (out)
 *   workspace, workspace_bytes   as moe_expert_matmul.
 *
 * Every array 16-byte aligned (offsets 4).  Errors: MOE_ERR_NULL (dy and x
 * may be NULL when max_rows == 0), MOE_ERR_SHAPE (also unknown flags),
 * MOE_ERR_ALIGN, MOE_ERR_ALIAS when dw starts where dy or x does,
 * MOE_ERR_WORKSPACE.
 */
int moe_expert_matmul_dw(const void *dy, const void *x, const int32_t *offsets, int E,
                         int64_t max_rows, int K, int N, int flags, void *dw, float *dbias,
                         void *workspace, size_t *workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_RECV_H */
