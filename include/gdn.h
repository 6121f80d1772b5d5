/*
 * gdn.h -- C ABI of the GB300 (sm_103a) chunked Gated DeltaNet training path.
 *
 * The operation (one value head h, one document, state reset to zero at the
 * document start, q/k head j = h / (HV/H)):
 *
 *     S_t = a_t S_{t-1} + beta_t k^_t (v_t - a_t S_{t-1}^T k^_t)^T,   a_t = exp(g_t)
 *     o_t = scale * S_t^T q^_t
 *
 * with q^, k^ the L2-normalised q, k (x / sqrt(x.x + 1e-6)) when l2norm != 0,
 * else q, k as given; S is a dk x dv matrix kept in FP32.  This is the gated
 * delta rule that the flashinfer Cake GDN training pages run: "packed GDN
 * layers" over variable-length documents with head dim 128, BF16 q/k/v and
 * output gradient, FP32 g and beta, grouped heads (H query/key heads, HV value
 * heads), optional in-kernel q/k L2 norm, chunk states every 64 tokens
 * ("feat(cake_gdn_kcp): ... Cake GDN chunked autograd backend - #8172" page,
 * its #8181 section; "#8542" page, the opening description and the save-set
 * table).  The backward returns the gradients of sum(o * dO) with respect to
 * q, k, v, g and beta.
 *
 * Conventions (all entry points):
 *   - Sizes: dk = dv = 128, HV % H == 0, T = cu_seqlens[N], chunk = 64.
 *   - Layouts, all contiguous and token-major:
 *       q, k, dq, dk      [T][H][128]   BF16
 *       v, dO, o, dv      [T][HV][128]  BF16
 *       g, beta, dg, dbeta [T][HV]      FP32
 *       cu_seqlens        [N+1]         int32, 0 = cu[0] <= cu[1] <= ... <= cu[N] = T
 *     Device pointers must be 16-byte aligned.
 *   - cu_seqlens is passed twice: the host copy drives planning (chunk counts,
 *     segment plan, buffer sizes) and the device copy drives the kernels.  The
 *     two must hold the same values.
 *   - Ownership: the caller allocates and owns every buffer (inputs, outputs,
 *     `saved`, `workspace`).  The library allocates no device memory at run
 *     time and launches everything asynchronously on `stream` in stream order;
 *     it never synchronises the host except in gdn_device_status().  Calls on
 *     different streams must use different workspaces.  The library keeps no
 *     per-call state outside the caller's buffers, except two process-wide
 *     items: the optional launch counters and timing events of
 *     gdn_profile_enable() / gdn_profile_read(), and the fixed device array of
 *     gdn_fwd_noalloc(), which every GPU that loads the library reserves
 *     (GDN_FWD_NOALLOC_SCRATCH_BYTES) whether or not that entry point is
 *     called.
 *   - Errors are returned, never thrown.  Host-side checks (null pointers,
 *     sizes, cu_seqlens, alignment, buffer sizes) return before any launch.
 *     Conditions only the device can see (a saved buffer whose header does
 *     not match the call, a bounded wait that ran out) are written to an
 *     error word in the workspace; later kernels of the same call then skip
 *     their work, and gdn_device_status() reports the word.
 *   - Results are bitwise reproducible run to run for a fixed problem and plan
 *     (every reduction has a fixed order).
 */
#ifndef GDN_H_
#define GDN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st; /* cudaStream_t */

typedef struct {
    int64_t T;        /* total packed tokens (= cu_seqlens[N]) */
    int32_t N;        /* number of documents (>= 1; empty documents allowed) */
    int32_t H;        /* query/key heads */
    int32_t HV;       /* value heads, a multiple of H */
    int32_t dk;       /* must be 128 */
    int32_t dv;       /* must be 128 */
    float scale;      /* output scale (typically dk^-0.5) */
    int32_t l2norm;   /* non-zero: L2-normalise q and k inside the kernels */
    int32_t segments; /* 0: the planner chooses the segment split;
                         > 0: split the longest document into `segments`
                         segments (see gdn_plan_segment_chunks()) */
    int32_t saved_form; /* what the forward keeps for the backward:
                           GDN_SAVED_FULL (0): the state tape plus the per-chunk
                             UT blocks and V_new (the backward recomputes nothing);
                           GDN_SAVED_REPLAY (1): the state tape only; the backward
                             runs the UT / WY preparation again and recomputes
                             V_new = U - W S from the saved states (the pages'
                             replay form, "#8542" page, save-set table).
                           Both give the same bits; see gdn_saved_bytes(). */
} gdn_problem;

#define GDN_SAVED_FULL 0
#define GDN_SAVED_REPLAY 1

typedef enum {
    GDN_OK = 0,
    GDN_ERR_INVALID_ARG = 1,        /* null pointer, bad size, bad cu_seqlens, misalignment */
    GDN_ERR_UNSUPPORTED = 2,        /* dk or dv != 128, HV % H != 0 */
    GDN_ERR_WORKSPACE_TOO_SMALL = 3,/* ws_bytes below the gdn_saved_bytes() figure */
    GDN_ERR_SAVED_MISMATCH = 4,     /* device-side: `saved` was not written by a forward of this problem */
    GDN_ERR_CUDA = 5,               /* a CUDA runtime call or launch failed */
    GDN_ERR_TIMEOUT = 6,            /* device-side: a bounded wait ran out */
    GDN_ERR_DEVICE = 7,             /* device-side: any other kernel-detected fault */
    GDN_ERR_GATE_RANGE = 8          /* device-side (KDA entry points): a key channel's decay within one
                                       16-token block is steeper than 2^-96 (see gdn_kda_fwd) */
} gdn_status;

/*
 * Byte sizes of the caller-owned buffers for this problem.
 *   saved_bytes      the set gdn_fwd() writes for gdn_bwd(): a 4 KiB header,
 *                    the BF16 state entering every 64-token chunk of every
 *                    value head (32 KiB per chunk and value head; the pages'
 *                    "h tape" of states every 64 tokens), and, where a
 *                    document is split into P > 1 segments, the FP32 segment
 *                    transfer plane M_seg ((P-1) x HV x 64 KiB per document)
 *                    that the backward's merges read ("#8542" page: the full
 *                    saved set keeps M_seg at P > 1).  In the full form
 *                    (prob->saved_form == GDN_SAVED_FULL) it also keeps the
 *                    per-chunk UT blocks (T = (I + A)^-1 with its scaled forms
 *                    and the gated Aqk rows, 33 KiB per chunk and value head)
 *                    and the BF16 V_new^T = (U - W S)^T of every chunk (16 KiB
 *                    per chunk and value head; the pages' v_new rows); the
 *                    replay form (GDN_SAVED_REPLAY) keeps neither and the
 *                    backward recomputes them.
 *   workspace_bytes  scratch for one gdn_fwd / gdn_bwd / gdn_ckpt_fwd_bwd call
 *                    (in the replay form it also holds the recomputed blocks).
 * Returns GDN_ERR_INVALID_ARG / GDN_ERR_UNSUPPORTED on a bad problem.
 */
gdn_status gdn_saved_bytes(const gdn_problem *prob, const int32_t *cu_seqlens_host,
                           size_t *saved_bytes, size_t *workspace_bytes);

/*
 * Forward.  Writes o.  If `saved` is non-null it also writes the saved set
 * (header + state tape [+ M_seg]) that gdn_bwd() consumes; with saved == NULL
 * no state is stored (the forward of a checkpointed step).
 */
gdn_status gdn_fwd(const gdn_problem *prob, const void *q, const void *k, const void *v,
                   const float *g, const float *beta, const int32_t *cu_seqlens_dev,
                   const int32_t *cu_seqlens_host, void *o, void *saved, void *workspace,
                   size_t ws_bytes, struct CUstream_st *stream);

/*
 * Backward.  Given dO and the saved set of a gdn_fwd() of the same problem and
 * inputs, writes dq, dk, dv (BF16) and dg, dbeta (FP32).  Every output element
 * is written (no accumulation into the caller's buffers).  A saved set whose
 * header does not match the problem sets GDN_ERR_SAVED_MISMATCH on the device
 * (see gdn_device_status) and leaves the gradients unwritten.
 */
gdn_status gdn_bwd(const gdn_problem *prob, const void *q, const void *k, const void *v,
                   const float *g, const float *beta, const int32_t *cu_seqlens_dev,
                   const int32_t *cu_seqlens_host, const void *dO, const void *saved,
                   void *dq, void *dk, void *dv, float *dg, float *dbeta, void *workspace,
                   size_t ws_bytes, struct CUstream_st *stream);

/*
 * Activation-checkpointed step: a forward that keeps no states and writes o,
 * then a forward that writes the saved set into `saved_scratch` (saved_bytes
 * large), then the backward.  This is the pages' "ckpt" operation, two
 * forwards plus one backward.  With o == NULL the first forward, which would
 * produce nothing, is skipped.
 */
gdn_status gdn_ckpt_fwd_bwd(const gdn_problem *prob, const void *q, const void *k,
                            const void *v, const float *g, const float *beta,
                            const int32_t *cu_seqlens_dev, const int32_t *cu_seqlens_host,
                            const void *dO, void *o, void *dq, void *dk, void *dv, float *dg,
                            float *dbeta, void *saved_scratch, void *workspace,
                            size_t ws_bytes, struct CUstream_st *stream);

/*
 * Per-document boundary states.  These are gdn_fwd / gdn_bwd for documents
 * that do not start from a zero state or whose last state is wanted: the
 * state passed between the pieces of a document split across calls (or
 * across devices): the pages' incoming boundary states S_in, kept in FP32
 * ("#8542" page, the save-set table's S_in row).
 * Every state is FP32 S in [N][HV][dk][dv] layout (document, value head,
 * k index, v index), 16-byte aligned, caller-owned.
 *
 * gdn_fwd_states: as gdn_fwd, with
 *   s_in   the state each document starts from (NULL: zero);
 *   s_out  written with the state after each document's last token (NULL:
 *          not written).  An empty document passes s_in through.
 *   o, saved and s_out may each be NULL, but not all three.
 * A saved set written here already holds the effect of s_in (the state
 * entering every chunk), so the backward needs no s_in.
 *
 * gdn_bwd_states: as gdn_bwd, with
 *   ds_out the gradient of the loss with respect to s_out (NULL: zero);
 *   ds_in  written with the gradient with respect to s_in (NULL: not
 *          written).  An empty document passes ds_out through.
 * The gradients dq, dk, dv, dg, dbeta then include the terms of ds_out.
 */
gdn_status gdn_fwd_states(const gdn_problem *prob, const void *q, const void *k, const void *v,
                          const float *g, const float *beta, const int32_t *cu_seqlens_dev,
                          const int32_t *cu_seqlens_host, const float *s_in, void *o, float *s_out,
                          void *saved, void *workspace, size_t ws_bytes, struct CUstream_st *stream);
gdn_status gdn_bwd_states(const gdn_problem *prob, const void *q, const void *k, const void *v,
                          const float *g, const float *beta, const int32_t *cu_seqlens_dev,
                          const int32_t *cu_seqlens_host, const void *dO, const float *ds_out,
                          const void *saved, void *dq, void *dk, void *dv, float *dg, float *dbeta,
                          float *ds_in, void *workspace, size_t ws_bytes, struct CUstream_st *stream);

/*
 * The short causal convolution + SiLU in front of the GDN layer, over the
 * packed q/k/v channels (C = (2 H + HV) x 128 = 10,240 at (16, 48)), restarting
 * at every document ("#8542" page: the B23 shape description and the family's
 * conv1d + SiLU training backend; its save-set table keeps at most three
 * history rows, a four-tap kernel).  Per channel c, with W taps:
 *     z[t, c] = b[c] + sum_{i<W} w[c, i] x[t - (W-1) + i, c]   (x = 0 before t's document)
 *     y[t, c] = z / (1 + exp(-z))
 * Layouts: x, y, dy, dx [T][C] BF16 (token-major, contiguous); w, dw [C][W]
 * FP32; b, db [C] FP32 (b may be NULL: no bias; db may be NULL: not
 * written).  C must be a multiple of 8, 1 <= W <= 4 (else
 * GDN_ERR_INVALID_ARG / GDN_ERR_UNSUPPORTED).  Pointers 16-byte aligned.
 * Accumulation is FP32 in a fixed order; dw and db are sums of per-range
 * partials added in range order (bitwise reproducible).  The caller owns
 * every buffer; the backward needs `workspace` of gdn_conv1d_workspace_bytes,
 * which opens with the device status word that gdn_device_status reads (a
 * bounded wait on a row copy that never completes sets GDN_ERR_TIMEOUT there).
 */
typedef struct {
    int64_t T;   /* total packed tokens (= cu_seqlens[N]) */
    int32_t N;   /* documents */
    int32_t C;   /* channels */
    int32_t W;   /* taps */
} gdn_conv_problem;
gdn_status gdn_conv1d_workspace_bytes(const gdn_conv_problem *prob, const int32_t *cu_seqlens_host,
                                      size_t *workspace_bytes);
gdn_status gdn_conv1d_fwd(const gdn_conv_problem *prob, const void *x, const float *w, const float *b,
                          const int32_t *cu_seqlens_dev, const int32_t *cu_seqlens_host, void *y,
                          struct CUstream_st *stream);
gdn_status gdn_conv1d_bwd(const gdn_conv_problem *prob, const void *x, const float *w, const float *b,
                          const int32_t *cu_seqlens_dev, const int32_t *cu_seqlens_host, const void *dy,
                          void *dx, float *dw, float *db, void *workspace, size_t ws_bytes,
                          struct CUstream_st *stream);

/*
 * The per-channel-decay form (KDA): the same recurrence with one decay per key channel,
 *
 *     S_t = Diag(a_t) S_{t-1} + beta_t k^_t (v_t - (Diag(a_t) S_{t-1})^T k^_t)^T,   a_t = exp(g_t) in R^dk
 *     o_t = scale * S_t^T q^_t
 *
 * ("perf(cake_kda) ... #7097" page: the packed KDA training family beside the GDN one; the pages
 * print no formula, and this is the GDN rule above with its scalar decay replaced by a per-channel
 * one).  Conventions as for the GDN entry points, except:
 *   - g and dg are [T][HV][128] FP32: the log decay of each key channel (g <= 0 for a decay);
 *   - the saved set holds the header, the BF16 state entering every chunk (32 KiB per chunk and
 *     value head), M_seg where a document is split, and the BF16 V_new^T of every chunk (16 KiB
 *     per chunk and value head).  With prob->saved_form == GDN_SAVED_FULL (the default) it also
 *     keeps the forward's per-chunk blocks of decay products and UT tiles (82,944 B per chunk and
 *     value head: Kd, -W^T, T'', T, Aqk, M^T, Q~, the scalars), which the backward reads; with
 *     GDN_SAVED_REPLAY the backward recomputes them (the pages' replay of w, u and the A
 *     matrices).  Both give the same gradients, bit for bit;
 *   - a chunk in which some key channel decays by more than 2^-96 within one 16-token block (a
 *     log decay below -66.5 over 16 tokens) is refused on the device: the error word is set to
 *     GDN_ERR_GATE_RANGE and the outputs are left unwritten.  Below that bound every chunk is
 *     computed (the kernels factor the decays per 16-token block, and the factors must stay in
 *     BF16's exponent range).
 * gdn_kda_saved_bytes: the sizes of `saved` and of the workspace (forward and backward).
 * gdn_kda_fwd: writes o (required) and, if `saved` is non-null, the saved set.
 * gdn_kda_bwd: given dO and the saved set of a gdn_kda_fwd of the same problem and inputs, writes
 *   dq, dk, dv (BF16), dg [T][HV][128] and dbeta [T][HV] (FP32).
 */
gdn_status gdn_kda_saved_bytes(const gdn_problem *prob, const int32_t *cu_seqlens_host,
                               size_t *saved_bytes, size_t *workspace_bytes);
gdn_status gdn_kda_fwd(const gdn_problem *prob, const void *q, const void *k, const void *v,
                       const float *g, const float *beta, const int32_t *cu_seqlens_dev,
                       const int32_t *cu_seqlens_host, void *o, void *saved, void *workspace,
                       size_t ws_bytes, struct CUstream_st *stream);
gdn_status gdn_kda_bwd(const gdn_problem *prob, const void *q, const void *k, const void *v,
                       const float *g, const float *beta, const int32_t *cu_seqlens_dev,
                       const int32_t *cu_seqlens_host, const void *dO, const void *saved, void *dq,
                       void *dk, void *dv, float *dg, float *dbeta, void *workspace, size_t ws_bytes,
                       struct CUstream_st *stream);

/*
 * Element types of the entry points below (those above are BF16).
 */
#define GDN_BF16 0
#define GDN_FP16 1
#define GDN_FP32 2

/*
 * The recurrent form, for generation: N sequences take their next tokens on a pool of states.
 * The operation is gdn_fwd's (gdn_step: one decay per value head, g [T][HV]) or gdn_kda_fwd's
 * (gdn_kda_step: one per key channel, g [T][HV][128], of any steepness), token by token.
 *   states     [slots][HV][128][128] FP32 (the layout of gdn_fwd_states' s_out: a prefill can write
 *              into the pool), updated in place.
 *   cu_seqlens_dev [N+1] int32: sequence n has the tokens cu[n] .. cu[n+1]-1, none or any number.
 *              NULL: one token each (T == N).  There is no host copy: lengths may change between
 *              replays of a captured graph.
 *   slot_in    [N] int32: the slot each sequence starts from; -1: from the zero state.
 *              NULL: sequence n's slot is n (slots >= N).
 *   slot_out   [T] int32: the slot the state after each token goes to; -1: nowhere.  To verify
 *              drafted tokens, give every token a slot and go on from the last accepted one's.
 *              NULL: the state after a sequence's last token goes back to the slot it came from
 *              (nowhere if that is -1).
 *              A sequence reads its slot before it writes any, so its own slots may repeat; a slot
 *              that one sequence writes must not be read or written by another in the same call.
 *   q, k, v    token-major rows of 128 values per head (H, H, HV heads), heads contiguous, with
 *              q_stride, k_stride, v_stride elements from token to token (0: contiguous), so that
 *              they may be views of one packed row; o [T][HV][128] contiguous.  All four of type
 *              `dtype`; strides and pointers in whole 16 bytes.
 *   dev_err    a device int, zero at first; nonzero afterwards (gdn_device_status(dev_err) reads it):
 *              GDN_ERR_DEVICE for a slot outside the pool or bad cu_seqlens.  A sequence with a bad
 *              slot_in or bad bounds is skipped (its o rows keep what they held); a bad slot_out
 *              is not written to.  The call never clears the word.
 *   (The tables and dev_err may start at any element: a view of a longer one.)
 * The states are read once and written once per slot_out, whatever the number of tokens; sums and
 * states are FP32.  Tokens outside cu_seqlens' range are no sequence's: their o rows keep what they held.
 * Long prompts belong to gdn_fwd_states, whose chunks are faster from about 250 tokens a sequence on for one sequence
 * of 4 or 16 value heads (256 tokens: 52 us, here 60), 130 for one of 48 (128 tokens: 46 us both), 64 for four of 48
 * (50 us, here 58) and 32 for sixteen or more of 48 (sixteen: 97 us, here 96; of 64 tokens 97 and 162).  The
 * per-channel rule has no chunked form that takes and gives states.
 * T below 2^30 (else GDN_ERR_UNSUPPORTED, as for the two operators below).
 *
 * The kernels of gdn_step, gdn_kda_step, gdn_conv1d_step and gdn_qk_norm_rope_* are launched with programmatic stream
 * serialization: they may be placed while the kernel before them in the stream ends, and wait for it before they touch
 * memory; to the caller the stream is in order as always.
 */
typedef struct {
    int64_t T;        /* tokens in all; 0 does nothing */
    int32_t N;        /* sequences */
    int32_t H;        /* query/key heads */
    int32_t HV;       /* value heads, a multiple of H */
    int32_t dk;       /* must be 128 */
    int32_t dv;       /* must be 128 */
    int32_t slots;    /* states in the pool */
    float scale;      /* output scale */
    int32_t l2norm;   /* non-zero: L2-normalise q and k inside the kernel */
    int32_t dtype;    /* of q, k, v, o */
    int64_t q_stride, k_stride, v_stride;
} gdn_step_problem;
gdn_status gdn_step(const gdn_step_problem *prob, const void *q, const void *k, const void *v,
                    const float *g, const float *beta, const int32_t *cu_seqlens_dev,
                    const int32_t *slot_in, const int32_t *slot_out, float *states, void *o,
                    int32_t *dev_err, struct CUstream_st *stream);
gdn_status gdn_kda_step(const gdn_step_problem *prob, const void *q, const void *k, const void *v,
                        const float *g, const float *beta, const int32_t *cu_seqlens_dev,
                        const int32_t *slot_in, const int32_t *slot_out, float *states, void *o,
                        int32_t *dev_err, struct CUstream_st *stream);

/*
 * gdn_conv1d_fwd for generation: the convolution + SiLU over the next tokens of N sequences, with
 * the last W-1 rows of each kept in a pool of windows.
 *   x, y       T rows of C channels, x_stride and y_stride elements apart (0: contiguous); y must
 *              not overlap x;
 *   w, b       [C][W] and [C] FP32, b may be NULL;
 *   window     [slots][W-1][C], oldest row first, updated in place (not read with W = 1, may then
 *              be NULL); the rows of a prompt's end, or zero rows where there are fewer;
 *   dtype      of x, y and window; strides and pointers in whole 16 bytes.
 * cu_seqlens_dev, slot_in (-1: zero rows), slot_out and dev_err are gdn_step's; a sequence with a
 * bad slot_in or bad bounds is skipped (where cu_seqlens goes back, sequences after that may be, too).
 * 1 <= W <= 4, C a multiple of 8.
 */
typedef struct {
    int64_t T;
    int32_t N;
    int32_t C;
    int32_t W;
    int32_t slots;
    int32_t dtype;
    int64_t x_stride, y_stride;
} gdn_conv_step_problem;
gdn_status gdn_conv1d_step(const gdn_conv_step_problem *prob, const void *x, const float *w, const float *b,
                           const int32_t *cu_seqlens_dev, const int32_t *slot_in, const int32_t *slot_out,
                           void *window, void *y, int32_t *dev_err, struct CUstream_st *stream);

/*
 * The norm of q and k per head with the position rotation in the same pass, for layers that put them
 * between the convolution and the rule, and its gradients.  The rule needs keys of about unit length: with GDN_NORM_L2 and
 * weights near one its own l2norm may then be 0.  GDN_NORM_RMS leaves keys of length near sqrt(D), and GDN_NORM_NONE those
 * that come in, with which the state would grow without bound: keep the rule's l2norm there.
 * For each token at position p and each head's row x of D values:
 *     x^ = x r,  r = 1 / sqrt(x.x / D + eps)  (GDN_NORM_RMS),  1 / sqrt(x.x + eps)  (GDN_NORM_L2),
 *          1  (GDN_NORM_NONE)
 *     z  = w x^                        (w [D] FP32, one for q and one for k; NULL: ones)
 *     pair i < rot / 2 of z's first rot values, (a, b):
 *     y  = m (a cos(p f_i) - b sin(p f_i),  b cos(p f_i) + a sin(p f_i));  the rest of z unchanged
 * with pairs (z[i], z[i + rot/2]) (GDN_ROPE_HALF) or (z[2i], z[2i+1]) (GDN_ROPE_PAIRS).
 *   freq       [rot/2] FP64 on the device: f in radians per position (gdn_rope_frequencies).  The
 *              angle is reduced in 64-bit fixed point, so it is as exact at position 10^9 as at 1.
 *   positions  [T] int32, p of each token; NULL: p counts from 0 in each of the N packed documents
 *              of cu_seqlens_dev [N+1], or, where that is NULL too, p is the token's index.
 *              Tokens outside cu_seqlens' range take the position from the nearest document.
 *   strides    elements from token to token and from head to head (0: contiguous): q and k may be
 *              views of a packed row.  q_* and k_* describe q, k and (backward) dq, dk; qo_* and ko_*
 *              the outputs and (backward) dqo, dko.  The D values of a row are contiguous.
 *   HQ, HK     heads, either may be 0 (its pointers are then unused).
 * Forward: qo, ko; each may be its input (same strides).  Backward: dq, dk (each may be dqo, dko, same
 * strides), and the weights' gradients dwq, dwk [D] FP32 (each NULL: not wanted; not NULL with its w NULL is allowed), summed
 * over all tokens and heads in a fixed order.  x must be what the forward read.
 * Any even rot <= D, any D <= 512, HQ + HK <= 65536 (beyond: GDN_ERR_UNSUPPORTED), any alignment of at least the
 * element's; sums in FP32.  The fast kernels take
 * strides and pointers in whole 16 bytes, D a multiple of 8 up to 256 and, in the half layout, rot a multiple of 4; the
 * others are several times slower.
 * gdn_qk_workspace_bytes: the backward's scratch (16-byte aligned), for the partial sums of dwq and dwk.
 */
#define GDN_ROPE_HALF 0
#define GDN_ROPE_PAIRS 1
#define GDN_NORM_NONE 0
#define GDN_NORM_RMS 1
#define GDN_NORM_L2 2
typedef struct {
    int64_t T;        /* tokens; 0 writes only zero dwq, dwk */
    int32_t N;        /* documents of cu_seqlens_dev */
    int32_t HQ, HK;   /* heads of q and k */
    int32_t D;        /* values per head */
    int32_t rot;      /* of them rotated: even, 0 .. D */
    int32_t layout;   /* GDN_ROPE_* */
    int32_t norm;     /* GDN_NORM_* */
    int32_t dtype;    /* of q, k, the outputs and their gradients */
    float eps;
    float mscale;     /* m */
    int64_t q_token, q_head, k_token, k_head;
    int64_t qo_token, qo_head, ko_token, ko_head;
} gdn_qk_problem;
gdn_status gdn_qk_workspace_bytes(const gdn_qk_problem *prob, size_t *workspace_bytes);
gdn_status gdn_qk_norm_rope_fwd(const gdn_qk_problem *prob, const void *q, const void *k, const float *wq,
                                const float *wk, const double *freq, const int32_t *positions,
                                const int32_t *cu_seqlens_dev, void *qo, void *ko, struct CUstream_st *stream);
gdn_status gdn_qk_norm_rope_bwd(const gdn_qk_problem *prob, const void *q, const void *k, const float *wq,
                                const float *wk, const double *freq, const int32_t *positions,
                                const int32_t *cu_seqlens_dev, const void *dqo, const void *dko, void *dq,
                                void *dk, float *dwq, float *dwk, void *workspace, size_t ws_bytes,
                                struct CUstream_st *stream);

/*
 * The rotation's frequencies, on the host: f_i = base^(-2i/rot), i < rot/2, changed for contexts `factor`
 * times longer than the trained `original` positions:
 *   GDN_ROPE_PLAIN   as they are;
 *   GDN_ROPE_LINEAR  f_i / factor (position interpolation, arXiv:2306.15595);
 *   GDN_ROPE_BASE    with base factor^(rot/(rot-2)) times larger (the lowest frequency is divided by
 *                    factor, the highest is kept; rot > 2);
 *   GDN_ROPE_PARTS   by parts (YaRN, arXiv:2309.00071): pairs that turn more than `fast` times within
 *                    `original` are kept, fewer than `slow` times divided by factor, a linear ramp over the pair
 *                    index between; *mscale = 0.1 ln(factor) + 1 (1 otherwise).
 * freq receives rot/2 values.
 */
#define GDN_ROPE_PLAIN 0
#define GDN_ROPE_LINEAR 1
#define GDN_ROPE_BASE 2
#define GDN_ROPE_PARTS 3
gdn_status gdn_rope_frequencies(int32_t rot, double base, int32_t scaling, double factor, double original,
                                double fast, double slow, double *freq, float *mscale);

/*
 * Linear attention with a fixed decay per value head (retention): the rule without its delta term,
 *
 *     S_t = a S_{t-1} + k_t v_t^T,   o_t = scale * S_t^T q_t,   a = exp(decay[h])
 *
 * over packed documents, forward, backward and, for generation, token by token on a pool of states (arXiv:2307.08621 gives
 * the three forms).  q and k enter as they are: norms, rotations and feature maps are the caller's (gdn_qk_norm_rope_fwd).
 *   q, k, v    rows of 128 values per head (H, H, HV heads; q/k head h / (HV/H) belongs to value head h), BF16, heads
 *              contiguous, q_stride, k_stride, v_stride elements from token to token (0: contiguous), multiples of 8;
 *              dq, dk, dv lie as q, k, v.  o, dO [T][HV][128] contiguous.
 *   decay      [HV] FP32 log decays, <= 0 (-inf: nothing is kept); constants of the layer, without a gradient.
 *   s_in       [N][HV][128][128] FP32 (S[dk][dv], the layout of gdn_fwd_states' and of the pools): the state each document
 *              starts from; NULL: zero.
 *   s_out      the state after each document's last token; NULL: not wanted.  An empty document passes s_in through.
 *              It may be s_in.
 *   ds_out, ds_in   the gradients of s_out (NULL: zero) and s_in (NULL: not wanted; may be ds_out).
 *   dev_err    a device int, zero at first (gdn_device_status(dev_err) reads it, the call never clears it):
 *              GDN_ERR_INVALID_ARG where the device copy of cu_seqlens is not the host's (documents then go by the device's
 *              bounds or are left out, and nothing but the outputs and the workspace is written), GDN_ERR_TIMEOUT for a
 *              bounded wait that ran out.
 * The forward needs nothing saved for the backward but its inputs: the backward walks the documents again.  Sums and
 * states are FP32; the state keeps FP32's exactness, and is rounded to BF16 once, where it meets the rows.
 * Heads with decays down to -0.7 are held up to 2^65 times larger or smaller on the way: in them, products (q . k) v and states
 * above 1e16 can overflow, and those below 1e-18 lose bits.
 * Inside a chunk of 128 tokens of a document, a value that is not finite also reaches the tokens before it; those of other
 * documents, and rows outside cu_seqlens' range, reach none.
 * Results are the same bits from run to run; dq and dk are sums over the value heads of a group in order.
 * Outputs do not overlap inputs, but for the states as said.  T below 2^30 (else GDN_ERR_UNSUPPORTED).
 * The kernels of gdn_la_*, gdn_add_norm_* and gdn_step_tables are launched as gdn_step's are: to the caller the stream is in order.
 * Every CTA looks for its document in the device's table: past a thousand documents of a few tokens that is most of the time.
 * gdn_la_workspace_bytes: what the forward and the backward need (16-byte aligned; 0: nothing).
 *     The backward of groups (HV > H) takes 128 KiB to each begun chunk of 128 tokens of a document and q/k head; documents
 *     that are cut, 64 KiB (the backward 128) to a segment and value head.
 */
typedef struct {
    int64_t T;        /* total packed tokens (= cu_seqlens[N]) */
    int32_t N;        /* documents (>= 1; empty ones allowed) */
    int32_t H;        /* query/key heads */
    int32_t HV;       /* value heads, a multiple of H */
    int32_t dk;       /* must be 128 */
    int32_t dv;       /* must be 128 */
    float scale;      /* output scale */
    int32_t segment;  /* 0: the planner decides where documents are cut into segments that run side by side;
                         > 0: segments of so many chunks of 128 tokens */
    int64_t q_stride, k_stride, v_stride;
} gdn_la_problem;
gdn_status gdn_la_workspace_bytes(const gdn_la_problem *prob, const int32_t *cu_seqlens_host, size_t *fwd_bytes,
                                  size_t *bwd_bytes);
gdn_status gdn_la_fwd(const gdn_la_problem *prob, const void *q, const void *k, const void *v, const float *decay,
                      const int32_t *cu_seqlens_dev, const int32_t *cu_seqlens_host, const float *s_in, void *o,
                      float *s_out, int32_t *dev_err, void *workspace, size_t ws_bytes, struct CUstream_st *stream);
gdn_status gdn_la_bwd(const gdn_la_problem *prob, const void *q, const void *k, const void *v, const float *decay,
                      const int32_t *cu_seqlens_dev, const int32_t *cu_seqlens_host, const float *s_in, const void *dO,
                      const float *ds_out, void *dq, void *dk, void *dv, float *ds_in, int32_t *dev_err,
                      void *workspace, size_t ws_bytes, struct CUstream_st *stream);
/*
 * The recurrent form: gdn_step's arguments and conventions, with decay [HV] in place of g and beta, and l2norm 0 (else
 * GDN_ERR_UNSUPPORTED).  Types BF16, FP16, FP32.
 */
gdn_status gdn_la_step(const gdn_step_problem *prob, const void *q, const void *k, const void *v, const float *decay,
                       const int32_t *cu_seqlens_dev, const int32_t *slot_in, const int32_t *slot_out, float *states,
                       void *o, int32_t *dev_err, struct CUstream_st *stream);

/*
 * The root-mean-square norm in front of a layer, with the residual's addition, and its gradients.  For each of T rows of C:
 *     h = x + r, rounded to the type (r NULL: h = x);   z = w h / sqrt(mean h^2 + eps)
 *     y = z rounded to the type;   y8 = z / s in E4M3,   s = max |z| / 448 (at least 2^-100)
 * with one s to `group` neighbouring values (32, 64 or 128, of which C is a multiple) or, with group 0, to a row.
 *   x, r, h, y   `dtype`, x_stride, r_stride, h_stride, y_stride elements from row to row (0: C).  h may be x or r (same
 *                stride), and NULL where r is; y, or y8 with scales, may be NULL.
 *   y8           [T][C] bytes, contiguous, C apart;  scales [T][C / group] FP32 ([T] with group 0);  w [C] FP32.
 * Backward, of y (what reads y8 takes its gradient to be z's): with h as the forward left it (h_stride), dy (y_stride) and
 * dres (r_stride), the gradient that reaches h along the stream (NULL: none), dx (x_stride) is the gradient of x and of r, and
 * dw [C] FP32 (NULL: not wanted) the weights', summed over the rows in a fixed order.  dx may be dy or dres (same stride).
 * Sums in FP32: rows whose squares add up to more than its range (4,096 values of 3 10^17) come out as zeros.  Any C up to 2^20
 * (else GDN_ERR_UNSUPPORTED), any alignment of at least the element's; the fast kernels take C a multiple of 8 up to 16384 with
 * strides and pointers in whole 16 bytes, the others are several times slower.
 * gdn_add_norm_workspace_bytes: the backward's scratch (16-byte aligned; not needed without dw).
 */
typedef struct {
    int64_t T;        /* rows; 0 writes only a zero dw */
    int32_t C;        /* values of a row */
    int32_t dtype;    /* GDN_BF16, GDN_FP16, GDN_FP32 */
    int32_t group;    /* values to a scale of y8; 0: a row */
    float eps;
    int64_t x_stride, r_stride, h_stride, y_stride;
} gdn_norm_problem;
gdn_status gdn_add_norm_workspace_bytes(const gdn_norm_problem *prob, size_t *workspace_bytes);
gdn_status gdn_add_norm_fwd(const gdn_norm_problem *prob, const void *x, const void *r, const float *w, void *h, void *y,
                            void *y8, float *scales, struct CUstream_st *stream);
gdn_status gdn_add_norm_bwd(const gdn_norm_problem *prob, const void *h, const float *w, const void *dy, const void *dres,
                            void *dx, float *dw, void *workspace, size_t ws_bytes, struct CUstream_st *stream);

/*
 * The tables of a generation step (cu_seqlens, positions, slot_in, slot_out of the entry points above) from the requests'
 * lengths, with the blocks of the states' pools handed out on the way; all on the GPU, so that a captured step goes on by
 * itself.  A request keeps a state to every `block` tokens: block j's slot holds the state after the last token taken of
 * j block .. (j+1) block - 1, so earlier blocks are what others with the same beginning can start from.  With `block` as long
 * as the longest context a request has one slot.
 * A slot stands in one request's row, and goes back with it.  A request that begins as another did takes a slot from the end of
 * the free list for itself, between two steps, copies the state of the other's block there, and has it in its own row.
 *   lengths      [N] tokens that each request takes now; -1: it has ended, its blocks go back
 *   context      [N] tokens it has taken before;  context_out [N]: after this step (0 where it has ended)
 *   block_table  [N][max_blocks] slots of its blocks: ceil(context / block) are read, the new ones written behind them
 *   free_list    [slots], free_count, free_count_out [1]: the slots that are free, taken from the end.  Blocks that go back
 *                are put there first, in the order of requests and blocks, then new ones are taken, in that order.
 *   cu_seqlens   [N+1];  positions [T] (NULL: not wanted), of each token, 0 past the last
 *   slot_in      [N] slot of the state before the first token, -1: none yet
 *   slot_out     [T] where the state after each token goes: its block's slot for the last token of a block and of this
 *                step, else -1
 * Where the tokens are more than T, or the blocks more than are free, the first request that does not fit and all after it
 * take no tokens in this step: their entries of cu_seqlens repeat and their context stays.
 * context_out may be context, free_count_out free_count (the call then works on the books in place).
 * dev_err: GDN_ERR_DEVICE for a length below -1, a context or length past max_blocks * block (the request takes nothing and
 * gives nothing back), a free_count outside the pool or more blocks given back than there are.
 * N up to 16384 and max_blocks * block below 2^30 (else GDN_ERR_UNSUPPORTED).  The pointers may start at any element.
 */
typedef struct {
    int32_t N;           /* requests */
    int32_t T;           /* entries of positions and slot_out */
    int32_t block;       /* tokens of a block */
    int32_t max_blocks;  /* entries of a row of block_table */
    int32_t slots;       /* states in the pool */
} gdn_tables_problem;
gdn_status gdn_step_tables(const gdn_tables_problem *prob, const int32_t *lengths, const int32_t *context,
                           int32_t *context_out, int32_t *block_table, int32_t *free_list, const int32_t *free_count,
                           int32_t *free_count_out, int32_t *cu_seqlens, int32_t *positions, int32_t *slot_in,
                           int32_t *slot_out, int32_t *dev_err, struct CUstream_st *stream);

/* Static description of a status code. */
const char *gdn_status_string(gdn_status s);

/*
 * Synchronises `stream`, then returns the device-side error word of the last
 * call that used `workspace` (GDN_OK if none), or GDN_ERR_CUDA if the stream
 * reports a CUDA error.
 */
gdn_status gdn_device_status(void *workspace, struct CUstream_st *stream);

/*
 * Introspection for tests and tools: byte offsets, into the workspace, of the
 * chunk tables every call builds from cu_seqlens (int32 arrays:
 * offsets[0] -> chunk_offsets[N+1], the index of each document's first chunk;
 * offsets[1] -> chunk_doc[NC]; offsets[2] -> chunk_tok0[NC], first token of
 * each chunk; offsets[3] -> chunk_len[NC], 1..64 tokens), and NC.
 */
gdn_status gdn_chunk_table_offsets(const gdn_problem *prob, const int32_t *cu_seqlens_host,
                                   size_t offsets[4], int32_t *num_chunks);

/*
 * Introspection for tests and tools: byte offsets, into the workspace, of the
 * intermediate tapes a gdn_bwd() call leaves there (each [NC][HV] blocks):
 *   offsets[0] UT blocks, 33,792 B each (T' at 0, T'' at 8 KiB, Aqk at 16 KiB,
 *              T at 24 KiB: BF16 64 x 64 tiles in the kernels' swizzled tile
 *              layout; then 1 KiB of per-token scalars)      (replay form; else 0)
 *   offsets[1] V_new^T tiles, 16 KiB each (BF16 128 x 64)   (replay form; else 0)
 *   offsets[2] dS' tiles, 32 KiB each (BF16 128 x 128 dS'^T: the gradient of
 *              the state leaving each chunk)
 *   offsets[3] dV_new^T tiles, 16 KiB each (BF16 128 x 64)
 */
gdn_status gdn_backward_tape_offsets(const gdn_problem *prob, const int32_t *cu_seqlens_host,
                                     size_t offsets[4]);

/*
 * Forward for callers that cannot allocate device memory.  The pages have no
 * counterpart to this entry point; it exists for hosts that give a library
 * only its inputs and outputs (plugin-style runtimes without a workspace
 * query, or latency-bound paths that may not call cudaMalloc because it
 * synchronises the device).
 *
 * It computes exactly what gdn_fwd(prob, ..., o, saved = NULL, ...) computes,
 * with the workspace taken from a fixed array of GDN_FWD_NOALLOC_SCRATCH_BYTES
 * (64 MiB) that the library keeps in device memory on every GPU where it is
 * loaded, until the process exits.  Inputs and `o` are the caller's, as for
 * gdn_fwd; no saved set is written (use gdn_fwd for training).
 *   - A problem whose forward workspace exceeds 64 MiB is refused with
 *     GDN_ERR_WORKSPACE_TOO_SMALL before any launch (at HV = 48 that is about
 *     40 chunks of 64 tokens; see gdn_saved_bytes for the general size).
 *   - The first call on a device, with that device current, looks up the
 *     array's device address (cudaGetSymbolAddress); make that first call
 *     before any stream capture.
 *   - Every call shares the one array and the array keeps the last call's
 *     contents; the forward rewrites everything it reads.  Calls that overlap
 *     on the GPU (different streams, or different host threads) race on the
 *     array and must be serialised by the caller.
 *   - Device-side conditions (a device copy of cu_seqlens that disagrees with
 *     the host copy, a bounded wait that ran out) are recorded in the array,
 *     which the caller cannot address, so this entry point reports only
 *     host-side statuses; after such a condition the kernels skip their work
 *     and `o` is left undefined (whatever it held before the call).  A caller
 *     that needs the device-side status uses gdn_fwd with its own workspace
 *     and gdn_device_status.
 * No cudaMalloc, cudaFree or allocating library routine is called.
 */
#define GDN_FWD_NOALLOC_SCRATCH_BYTES (64u << 20)
gdn_status gdn_fwd_noalloc(const gdn_problem *prob, const void *q, const void *k, const void *v,
                           const float *g, const float *beta, const int32_t *cu_seqlens_dev,
                           const int32_t *cu_seqlens_host, void *o, struct CUstream_st *stream);

/*
 * Optional per-kernel timing, for benchmarks and tools.  The library counts
 * every kernel it launches; while profiling is enabled it also records a CUDA
 * event pair on the launching stream around each launch.  gdn_profile_read()
 * synchronises on the recorded events, fills up to max_entries records (one
 * per kernel that launched since the last read: its name, the number of
 * launches, how many of them were timed, and their summed device time in ms),
 * resets the counters and returns the number of kernels with launches.  The
 * bookkeeping is process-wide and thread-safe.
 */
typedef struct {
    const char *name;
    long long launches;
    long long timed_launches;
    double total_ms;
} gdn_kernel_stat;
void gdn_profile_enable(int on);
int gdn_profile_read(gdn_kernel_stat *out, int max_entries);

/*
 * The segment length (in 64-token chunks) the planner uses for this problem:
 * documents longer than this are split into ceil(chunks / seg) segments whose
 * transfer operators are composed by a merge kernel (the intra-GPU segment
 * split).  With prob->segments > 0 the answer is ceil(max_doc_chunks /
 * prob->segments), i.e. the longest document gets `segments` segments.
 * Returns 0 on an invalid problem.
 */
int32_t gdn_plan_segment_chunks(const gdn_problem *prob, const int32_t *cu_seqlens_host);

/*
 * Tensor-pipe probe, for the roofline's own BF16 peak: the benchmark reports
 * tensor-core fractions against the vendor's dense figure and against the rate
 * this probe measures with the library's own tcgen05 code.  Launches one CTA per SM of
 * the current device on `stream`; each issues iters x 4 BF16 tcgen05 products
 * of M = 128, N = 256, K = 16 (FP32 accumulation in TMEM) on operand tiles
 * that stay in shared memory, so no memory traffic competes with the tensor
 * cores.  *flops receives the products' FLOP count (2 M N K each); the caller
 * times the launch with events on `stream` and reads *dev_err (a device int,
 * zero on entry) afterwards: nonzero means a bounded wait ran out.
 * iters: 1 .. 2^20.  Returns GDN_ERR_INVALID_ARG outside that range or for a
 * null pointer, GDN_ERR_CUDA if the launch fails; nothing is allocated.
 */
gdn_status gdn_tensor_probe(int32_t iters, int32_t *dev_err, double *flops, struct CUstream_st *stream);

#ifdef __cplusplus
}
#endif
#endif /* GDN_H_ */
