/*
 * gdn_layer.h -- C ABI of the operators that stand around the gated delta rule
 * in a layer, on MI355X (gfx950): the gated RMSNorm after the mixer, the
 * residual add with the RMSNorm before the next block, the per-channel gated
 * linear recurrence, and the single-token steps of serving.
 *
 * Formulas (fp32 arithmetic whatever the tensors' type, each output rounded once):
 *   gated norm   y = x r w act(z),  r = (sum_D x^2 / D + eps)^(-1/2) per row,
 *                act(z) = z sigmoid(z), sigmoid(z), or 1 where z is absent
 *   add norm     res' = res + s x,  y = res' r w,  r of the unrounded res'
 *   dropout      y = m x,  m = 1/(1-p) or 0 per element, from a counter-based generator;
 *                in the add norm m x stands for x
 *   recurrence   h_t = exp(g_t) h_{t-1} + x_t   per channel, h_{-1} = h0
 *   rule's step  S <- exp(g) S;  S <- S + beta k (v - S^T k)^T;  o = scale S^T q
 *                (one token of the recurrence in gdr.h)
 *
 * Conventions: as in gdr.h.  Tensors are caller-owned, contiguous, row-major
 * DEVICE pointers aligned to their element; calls are asynchronous on `stream`,
 * which must belong to the current device; validation happens on the host
 * before anything is launched, and on error nothing is launched and no output
 * is written; status codes of gdr.h.  The library allocates nothing; scratch
 * comes from the caller's workspace (16-byte aligned), which one call at a time
 * may use (calls on one stream may share one; two that can overlap may not).
 * An output may be the very buffer of an input where a call says so; other
 * overlaps of an output with an input or another output are refused.
 * Results do not depend on timing: equal inputs give equal bits.
 */
#ifndef GDN_LAYER_H_
#define GDN_LAYER_H_

#include "gdr.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { GDN_ACT_SILU = 0, GDN_ACT_SIGMOID = 1 } gdn_act;

/* Sizes of the two norms.  rows >= 0, 1 <= D <= 8192, eps >= 0 and finite. */
typedef struct norm_problem {
    int64_t rows;        /* rows (tokens, or tokens x heads) */
    int D;               /* elements in a row */
    float eps;
    gdr_dtype dtype;     /* type of x, z, y and of their gradients */
    gdr_dtype res_dtype; /* add norm: type of the residual stream and its gradient,
                            dtype itself or GDR_F32; not read by the gated norm */
    gdn_act act;         /* gated norm: the gate's function; not read by the add norm */
} norm_problem;

/* Bytes of workspace gated_norm_bwd and add_norm_bwd need; 0 if the problem is invalid or so small that they
 * need none. */
size_t norm_workspace_size(const norm_problem *p);

/*
 * gated_norm_fwd -- y = x r w act(z) per row.
 *   x, z [rows, D] dtype   z NULL: no gate (a plain RMSNorm)
 *   w [D] fp32
 *   y [rows, D] dtype      may be x or z
 */
int gated_norm_fwd(const norm_problem *p, const void *x, const void *z, const float *w, void *y, hipStream_t stream);

/*
 * gated_norm_bwd -- the gradients of sum(dy * y), with r recomputed from x.
 *   x, z, w as for gated_norm_fwd; dy [rows, D] dtype
 *   dx, dz [rows, D] dtype   dz NULL exactly where z is; dx may be x or dy, dz may be z or dy
 *   dw [D] fp32              summed over the rows in a fixed order
 * ws/ws_bytes: workspace (>= norm_workspace_size(p)).
 */
int gated_norm_bwd(const norm_problem *p, const void *x, const void *z, const float *w, const void *dy, void *dx,
                   void *dz, float *dw, void *ws, size_t ws_bytes, hipStream_t stream);

/*
 * add_norm_fwd -- res' = res + s x and y = RMSNorm(res') w.
 *   x [rows, D] dtype   res [rows, D] res_dtype
 *   w [D] fp32          scale s [D] fp32, NULL = 1
 *   y [rows, D] dtype   may be x;   res_out [rows, D] res_dtype   may be res
 */
int add_norm_fwd(const norm_problem *p, const void *x, const void *res, const float *w, const float *scale, void *y,
                 void *res_out, hipStream_t stream);

/*
 * add_norm_bwd -- the gradients of sum(dy * y) + sum(dres * res') at the stored res'.
 *   dy [rows, D] dtype       dres [rows, D] res_dtype, NULL = zero
 *   res [rows, D] res_dtype  the forward's res_out
 *   w [D] fp32               scale [D] fp32, NULL = 1
 *   x [rows, D] dtype        read for dscale: required with scale, else NULL
 * Outputs:
 *   dres_out [rows, D] res_dtype   gradient of res;  may be dres or res
 *   dx [rows, D] dtype             gradient of x;  may be dy or x.  NULL without scale
 *                                  (it is then dres_out, in dres_out's type)
 *   dw [D] fp32; dscale [D] fp32, NULL exactly where scale is
 * Without scale and with res_dtype != dtype, dx is written too where it is not NULL.
 * ws/ws_bytes: workspace (>= norm_workspace_size(p)).
 */
int add_norm_bwd(const norm_problem *p, const void *dy, const void *dres, const void *res, const float *w,
                 const void *x, const float *scale, void *dx, void *dres_out, float *dw, float *dscale, void *ws,
                 size_t ws_bytes, hipStream_t stream);

/*
 * Dropout.  The mask is a function of (seed, offset, row, column) alone and is computed
 * wherever it is needed, never stored: a forward and its backward give the same
 * gdn_dropout, calls that shall differ another offset (or seed).
 * Element `column` of row `row` has 16 bits b: with G = ceil(D / 8), group
 * n = row G + column / 8 and e = column % 8, Philox 4x32-10 (Salmon et al. 2011) with
 * key (seed low, seed high) and counter (n low, n high, offset low, offset high) gives
 * four words, and b is half e % 2 (low half first) of word e / 2.  The element is
 * dropped where b < t, t = floor(65536 p + 1/2), and multiplied by 65536 / (65536 - t)
 * otherwise: the probability is p to the nearest 2^-16, and the factor is its own.
 * A dropped element is 0 whatever x is.  t = 65536 drops all of them.
 */
typedef struct gdn_dropout {
    double p;                /* 0 <= p <= 1 */
    uint64_t seed, offset;
    const uint64_t *rng;     /* device {seed, offset}, 8-byte aligned, read by the kernels instead of the
                                two above (a captured graph then takes what it holds at each replay), or NULL */
} gdn_dropout;

/*
 * gdn_dropout_fwd -- y = m x; the gradient is the same call on dy.
 *   x, y [rows, D] dtype   y may be x
 * rows >= 0, D >= 1, rows * D <= 2^40.
 */
int gdn_dropout_fwd(int64_t rows, int64_t D, gdr_dtype dtype, const gdn_dropout *d, const void *x, void *y,
                    hipStream_t stream);

/*
 * dropout_add_norm_fwd -- res' = res + s m x and y = RMSNorm(res') w: add_norm_fwd of m x.
 */
int dropout_add_norm_fwd(const norm_problem *p, const gdn_dropout *d, const void *x, const void *res, const float *w,
                         const float *scale, void *y, void *res_out, hipStream_t stream);

/*
 * dropout_add_norm_bwd -- its gradients, as add_norm_bwd's: dx = s m dres_out, dscale = sum over the rows
 * of dres_out m x.  dx [rows, D] dtype is always written, and is dres_out's buffer in no case.
 */
int dropout_add_norm_bwd(const norm_problem *p, const gdn_dropout *d, const void *dy, const void *dres,
                         const void *res, const float *w, const void *x, const float *scale, void *dx, void *dres_out,
                         float *dw, float *dscale, void *ws, size_t ws_bytes, hipStream_t stream);

/* Sizes of the gated linear recurrence.  The token axis is flattened over the
 * batch, as in gdr.h: dense B sequences of T tokens, or (cu_seqlens != NULL,
 * B = 1) N sequences of T tokens in all, empty ones allowed. */
typedef struct glr_problem {
    int B, T;                       /* B >= 1, T >= 0; B*T, rounded up to a multiple of 384, times
                                       ceil(D / 128) < 2^30; without tokens N*D < 2^31 */
    int D;                          /* channels, 1 <= D <= 2^20 */
    int N;                          /* number of sequences when varlen; ignored when cu_seqlens == NULL */
    const int32_t *cu_seqlens;      /* device [N+1] or NULL (dense) */
    const int32_t *cu_seqlens_host; /* host mirror of cu_seqlens [N+1]; required iff cu_seqlens != NULL.
                                       It must hold the same values; it is read during the call only. */
    gdr_dtype dtype;                /* type of x, h, dh, dx */
    int polls;                      /* how often a workgroup looks for the results of earlier ones before it
                                       computes them itself; <= 0 selects the default.  Results are the same
                                       for every value. */
} glr_problem;

/* Rows of `states`: one for every GLR_TILE tokens of the flattened axis; -1 if invalid. */
#define GLR_TILE 16
int64_t glr_num_states(const glr_problem *p);

/* Bytes of workspace glr_fwd and glr_bwd need; 0 if the problem is invalid or needs none. */
size_t glr_workspace_size(const glr_problem *p);

/*
 * glr_fwd -- h_t = exp(g_t) h_{t-1} + x_t in each sequence, channel by channel.
 *   x [B*T, D] dtype
 *   g [B*T, D] fp32     the log-gate, as a rule <= 0 (-inf: the state is dropped).  Values above 0 are
 *                       taken, but the sum of g over consecutive tokens of a sequence must stay
 *                       below 80: products of gates are formed over up to 12288 tokens in fp32
 *   h0 [N, D] fp32      states before the first tokens, NULL = zero
 * Outputs:
 *   h [B*T, D] dtype
 *   ht [N, D] fp32 or NULL                       states after the last tokens (h0 for an empty sequence)
 *   states [glr_num_states(p), D] fp32 or NULL   for glr_bwd: row i is the state that token
 *                                                GLR_TILE*i meets (h0 where it begins a sequence)
 * The states are carried in fp32.  ws/ws_bytes: workspace (>= glr_workspace_size(p)).
 */
int glr_fwd(const glr_problem *p, const void *x, const float *g, const float *h0, void *h, float *ht, float *states,
            void *ws, size_t ws_bytes, hipStream_t stream);

/*
 * glr_bwd -- the gradients of sum(dh * h) + sum(dht * ht).
 *   x, g, h0 as for glr_fwd, states from it (h_{t-1} is recomputed from them in fp32)
 *   dh [B*T, D] dtype   dht [N, D] fp32, NULL = zero
 * Outputs:
 *   dx [B*T, D] dtype   dg [B*T, D] fp32
 *   dh0 [N, D] fp32 or NULL (skip)
 */
int glr_bwd(const glr_problem *p, const void *x, const float *g, const float *h0, const float *states, const void *dh,
            const float *dht, void *dx, float *dg, float *dh0, void *ws, size_t ws_bytes, hipStream_t stream);

/*
 * glr_step -- one token for each of N rows, on states kept in a pool.
 *   x [N, D] dtype   g [N, D] fp32
 *   slots [N] int32 or NULL   row n's place in the pool; NULL: row n has slot n (N <= nslots).
 *       A row whose slot is outside [0, nslots) is padding: its h is written as zero and no state is touched.
 *       Rows with the same slot are successive tokens of that state, in the order of the rows.
 *   state [nslots, D] fp32    read and updated in place
 *   h [N, D] dtype            may be x
 * 0 <= N <= 65536, 1 <= D <= 2^20, N * ceil(D / 512) < 2^25.
 * With slots each row looks through those of all others (64 at a time): little up to a thousand
 * rows, most of the call beyond (D = 2048 bf16, us with slots and without: 1024 rows 11 and 9,
 * 4096 rows 88 and 21, 16384 rows 1070 and 86).
 */
int glr_step(int N, int D, int64_t nslots, gdr_dtype dtype, const void *x, const float *g, const int32_t *slots,
             float *state, void *h, hipStream_t stream);

/*
 * gdr_step -- one token of the gated delta rule for each of N rows, on states kept in a pool.
 *   q, k [N, HK, K]   v [N, HV, V]   beta [N, HV]   dtype
 *   g [N, HV] fp32              raw log-gate of the token
 *   slots [N] int32 or NULL     as for glr_step
 *   state [nslots, HV, K, V] fp32   read and updated in place (gdr_chunk_fwd's ht_out, sequence by sequence)
 *   o [N, HV, V] dtype          may be v
 * scale <= 0 selects 1/sqrt(K).  0 <= N <= 65536; K = V in {64, 128}; HV % HK == 0, HV <= 1024,
 * N * HV < 2^24.  Many rows with slots as for glr_step (HV = 32, K = 128: 1024 rows 805 and 768 us,
 * 4096 rows 4790 and 3170).
 */
int gdr_step(int N, int HK, int HV, int K, int V, int64_t nslots, float scale, gdr_dtype dtype, const void *q,
             const void *k, const void *v, const float *g, const void *beta, const int32_t *slots, float *state,
             void *o, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_LAYER_H_ */
