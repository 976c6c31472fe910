/*
 * gdn_ffn.h -- C ABI of the gated feed-forward block of a layer, forward and
 * backward, on MI355X (gfx950).
 *
 *   g = x Wg^T,  u = x Wu^T,  h = act(g) u,  y = h Wd^T          (per token)
 *   dh = dy Wd,  du = dh act(g),  dg = dh u act'(g)
 *   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x,  dWd = dy^T h
 *
 * Sums are fp32 whatever the type (products of 16-bit operands on the matrix
 * units, of fp32 ones in fp32).  g and u stay in fp32; h, dg and du are operands
 * of the next product and are rounded to the type first (in fp16 they are infinite
 * beyond 65504); each output is rounded once.  Sums over the tokens are formed in
 * pieces of at most 131072 tokens (fp32: 16384) and joined in their order.
 *
 * Conventions: as in gdn_layer.h (caller-owned, contiguous, row-major device
 * pointers; asynchronous on `stream`, which must belong to the current device;
 * checks on the host before anything is launched; workspace of the caller, 16-byte
 * aligned, one call at a time; no output on an input or another output; equal
 * inputs give equal bits).  Where D and F are multiples of 8 (of 4 for fp32), x, dy
 * and the weights must be 16-byte aligned; otherwise to their element, and the call
 * first copies those that are not, or whose rows are not, into rows of such a length.
 */
#ifndef GDN_FFN_H_
#define GDN_FFN_H_

#include "gdr.h"

#ifdef __cplusplus
extern "C" {
#endif

/* x sigmoid(x); sigmoid(x); x Phi(x) with the normal distribution's Phi (no approximation) */
typedef enum { GDN_FFN_SILU = 0, GDN_FFN_SIGMOID = 1, GDN_FFN_GELU = 2 } gdn_ffn_act;

typedef struct ffn_problem {
    int64_t T;       /* tokens, 0 <= T <= 2^24 */
    int D, F;        /* width of x and y, of the hidden row; 1 <= D, F <= 65536, T * (D + 2 F) < 2^36 */
    gdr_dtype dtype; /* type of x, the weights, y, dy and of every gradient */
    gdn_ffn_act act;
} ffn_problem;

/* Bytes of workspace gated_ffn_fwd (bwd = 0) or gated_ffn_bwd (bwd != 0) needs; 0 if the problem is invalid. */
size_t ffn_workspace_size(const ffn_problem *p, int bwd);

/* Floats that a token takes in `saved`: g and u in fp32 and h in the type, F rounded up to a multiple of 8 (of 4
 * for fp32); -1 if invalid. */
int64_t ffn_saved_width(const ffn_problem *p);

/*
 * gated_ffn_fwd -- y = (act(x Wg^T) (x Wu^T)) Wd^T.
 *   x [T, D]   w_gate, w_up [F, D] (two halves of one [2F, D] tensor, say)   w_down [D, F]
 *   y [T, D]
 *   saved [T, ffn_saved_width(p)] fp32, 16-byte aligned, or NULL   what gated_ffn_bwd needs:
 *       g and u of every token, behind them h
 */
int gated_ffn_fwd(const ffn_problem *p, const void *x, const void *w_gate, const void *w_up, const void *w_down,
                  void *y, float *saved, void *ws, size_t ws_bytes, hipStream_t stream);

/*
 * gated_ffn_bwd -- the gradients of sum(dy * y).
 *   x and the weights as for gated_ffn_fwd, saved from it; dy [T, D]
 * Outputs, each NULL to skip it:
 *   dx [T, D]   dw_gate, dw_up [F, D] (both or neither)   dw_down [D, F]
 */
int gated_ffn_bwd(const ffn_problem *p, const void *x, const void *w_gate, const void *w_up, const void *w_down,
                  const float *saved, const void *dy, void *dx, void *dw_gate, void *dw_up, void *dw_down, void *ws,
                  size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_FFN_H_ */
