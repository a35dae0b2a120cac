/*
 * dspark_tokens.h -- C ABI of what the tokens of a round bring with them: their
 * positions, which rotate queries and keys, and their histories, which edit the
 * logits that the round verifies.
 *
 *   dspark_rotary, dspark_rotary_backward
 *                          rotary positions of queries and keys, and their gradient
 *   dspark_cache_append    the rotation on the way into the paged cache: what
 *                          dspark_cache_attend reads then
 *   dspark_edit_logits, dspark_edit_logits_backward
 *                          penalties for repeated tokens, biases and grammar masks
 *                          on the logits of verified rows, and their gradient
 *   dspark_history_append  the emitted tokens (or prompts) join the histories
 *
 * One round: dspark_draft -> dspark_schedule -> dspark_cache_reserve -> the target's
 * layers, each dspark_cache_append and dspark_cache_attend (its k_new and v_new NULL)
 * -> dspark_edit_logits on the target's rows, each with the drafts before it ->
 * dspark_verify -> dspark_cache_commit -> dspark_history_append.
 *
 * The conventions of dspark.h and dspark_serving.h hold: device pointers, 16-byte
 * aligned unless stated (int32 arrays and the fp32 parameters of requests: their
 * element's alignment); caller-owned buffers; host-side validation first; asynchronous
 * on `stream`; data errors OR a DSPARK_DEVERR_* bit into the first word of the
 * workspace, which is 256 bytes for every operation here.  Nothing is allocated and
 * every call may be captured into a graph.  Calls that share a workspace must be
 * ordered on one stream only where the error word is read or cleared between them.
 */
#ifndef DSPARK_TOKENS_H
#define DSPARK_TOKENS_H

#include "dspark_serving.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ----------------------------------------------------------------- rotary --
 * Of every head the first `rot` elements are rot / 2 pairs, and pair i of a row at
 * position t turns by the angle t f_i:
 *   (a, b) -> magnitude (a cos t f_i - b sin t f_i, b cos t f_i + a sin t f_i)
 * The elements from rot on stay as they are. */
typedef enum {
  DSPARK_ROTARY_HALF = 0,        /* pair i: elements i and i + rot / 2 */
  DSPARK_ROTARY_INTERLEAVED = 1  /* pair i: elements 2 i and 2 i + 1   */
} dspark_rotary_layout;

typedef enum {
  DSPARK_ROTARY_PLAIN = 0,   /* f_i = base^(-2 i / rot)                                       */
  DSPARK_ROTARY_LINEAR = 1,  /* f_i / factor                                                  */
  DSPARK_ROTARY_BASE = 2,    /* base factor^(rot / (rot - 2)) for base: the fastest pair stays,
                                the slowest is stretched by `factor`                          */
  DSPARK_ROTARY_BY_TURNS = 3 /* by the turns c_i = context f_i / (2 pi) of a pair over the
                                original context: f_i (w_i + (1 - w_i) / factor),
                                w_i = (c_i - slow) / (fast - slow) within [0, 1]              */
} dspark_rotary_scaling;

/* Frequencies f_i, i < rot / 2, radians a token, in 64 bits.  Host memory; no GPU is
 * touched.  rot even, 2 <= rot <= 256 (BASE: 4 at least); base > 1; factor >= 1, context > 0 and
 * 0 < slow < fast where the scaling reads them. */
dspark_status dspark_rotary_frequencies(int rot, double base, dspark_rotary_scaling scaling,
                                        double factor, double context, double slow, double fast,
                                        double *freqs);
/* The form in which the kernels take frequencies: turns a token, f / (2 pi), as
 * 64-bit fractions of one turn, rounded once.  position * turns then drops the whole
 * turns exactly, and the angle is off by 2^-65 turns for each token of the position: less
 * than 2^-33 turns however far the position.  Host memory; 1 <= n <= 128; finite
 * frequencies of any sign below 2^20 in magnitude. */
dspark_status dspark_rotary_turns(int n, const double *freqs, uint64_t *turns);

/* Positions of the rows, any int32 (negative ones turn back):
 *   positions [n_rows] int32, or NULL:
 *   row_offset [R + 1] int32: row row_offset[rho] + j of the n that request rho has is
 *     at kv_len[rho] - n + j (the last n of its kv_len tokens), or with kv_len NULL at
 *     j (packed sequences); rows that belong to no request are left as they were;
 *   row_offset NULL (R is not read): row i at kv_len[i] - 1, or with kv_len NULL at i
 *     (one sequence).
 * With positions and row_offset both given, row_offset only says which rows there are.
 * A row_offset that is negative, decreases or passes n_rows sets DSPARK_DEVERR_LENGTH,
 * and which of its rows are then left as they were is unspecified.
 * Inputs
 *   q [n_rows][Hq][D], q_stride elements from row to row; k [n_rows][Hkv][D] likewise,
 *     NULL with Hkv = 0: q alone
 *   turns [rot / 2] (8-byte aligned) from dspark_rotary_turns, on the device; magnitude
 *     finite and not 0
 *   D a multiple of 8 up to 256, 2 <= rot <= D even; 1 <= Hq <= 1024, 0 <= Hkv <= 1024;
 *     1 <= n_rows <= 4194304; 1 <= R <= 4194304; strides multiples of 16 bytes
 * Outputs: q_out, k_out [n_rows][H][D] (dt) with strides of their own; each may be its
 *   input (in place: the same stride then), and overlaps nothing else: rows of one stride may
 *   stand side by side (heads of one buffer), with two different strides neither array may
 *   reach into the other's first to last byte (DSPARK_ERR_VALUE).  cos, sin and the
 *   rotation are fp32; the result is rounded once. */
dspark_status dspark_rotary(int n_rows, int Hq, int Hkv, int D, int rot, dspark_rotary_layout layout,
                            dspark_dtype dt, float magnitude, const uint64_t *turns,
                            const int32_t *positions, int R, const int32_t *row_offset,
                            const int32_t *kv_len, const void *q, int64_t q_stride, const void *k,
                            int64_t k_stride, void *q_out, int64_t q_out_stride, void *k_out,
                            int64_t k_out_stride, void *ws, size_t ws_bytes, hipStream_t stream);

/* The gradient: from those of the rotated queries and keys to those of the unrotated
 * ones, (a, b) -> magnitude (a cos + b sin, b cos - a sin).  Arguments as above. */
dspark_status dspark_rotary_backward(int n_rows, int Hq, int Hkv, int D, int rot,
                                     dspark_rotary_layout layout, dspark_dtype dt, float magnitude,
                                     const uint64_t *turns, const int32_t *positions, int R,
                                     const int32_t *row_offset, const int32_t *kv_len,
                                     const void *g_q, int64_t q_stride, const void *g_k,
                                     int64_t k_stride, void *q_out, int64_t q_out_stride,
                                     void *k_out, int64_t k_out_stride, void *ws, size_t ws_bytes,
                                     hipStream_t stream);

/* ----------------------------------------------------------- cache_append --
 * Before the attention of a layer: the new rows' keys are rotated and, with the values,
 * written into their slots of the pages; their queries are rotated for
 * dspark_cache_attend, which then takes k_new = v_new = NULL.  Rows, cache and error
 * bits as there: request rho's row j of n is token kv_len[rho] - n + j.
 *   rot 0: no rotation (turns NULL); else as dspark_rotary, with magnitude on queries
 *     and keys both
 *   positions [rows_capacity] int32: positions for the rotation that are not the
 *     tokens' places in the cache; NULL: those
 *   q, q_out: NULL both with keys and values alone (Hq is then not read); q_out may be q,
 *     and overlaps neither part of it nor k_new and v_new (as for dspark_rotary)
 *   k_new, v_new [rows_capacity][Hkv][D], kv_stride elements from row to row
 *   row_offset [R + 1], or NULL: one row each (rows_capacity = R)
 * Rows that no request has (from row_offset[R] on) are neither read nor written.  Rows
 * before token 0 and kv_len outside [0, page * max_pages] (taken as 0) set
 * DSPARK_DEVERR_LENGTH and reach no page; a page number outside [0, n_pages) sets
 * DSPARK_DEVERR_PAGE, and its tokens are not written.  A row_offset that is negative,
 * decreases or passes rows_capacity sets DSPARK_DEVERR_LENGTH, and which of the rows are
 * then written is unspecified (never a slot outside the pages). */
dspark_status dspark_cache_append(int R, int rows_capacity, int Hq, int Hkv, int D, int page,
                                  int max_pages, int n_pages, dspark_dtype dt, int rot,
                                  dspark_rotary_layout layout, float magnitude,
                                  const uint64_t *turns, const int32_t *positions, const void *q,
                                  int64_t q_stride, void *q_out, int64_t q_out_stride,
                                  const void *k_new, const void *v_new, int64_t kv_stride,
                                  void *k_pages, void *v_pages, int64_t k_page_stride,
                                  int64_t v_page_stride, const int32_t *table,
                                  const int32_t *row_offset, const int32_t *kv_len, void *ws,
                                  size_t ws_bytes, hipStream_t stream);

/* ------------------------------------------------------------ edit_logits --
 * For row j of request rho (rows [row_offset[rho], row_offset[rho + 1]) of X) let
 *   n_v  the times that v was generated: among history[rho][prompt_len .. hist_len)
 *        and drafts[rho][0 .. j) (the drafts that the row stands behind),
 *   s_v  whether v was seen: n_v > 0 or v among history[rho][0 .. prompt_len).
 * Then, in fp32 and in this order, rounded once at the end:
 *   x = s_v ? (x > 0 ? x / repetition : x * repetition) : x
 *   x = x - frequency n_v
 *   x = x - (n_v > 0 ? presence : 0)
 *   x = x + bias_v
 *   x = v allowed ? x : -infinity    (whatever x was, NaN included)
 * A row whose mask allows nothing is all -infinity (dspark_verify and dspark_logprobs
 * report such a row).
 * Inputs
 *   X [n_rows][row_stride] logits (dt), V of each row; row_stride >= V, a multiple of 16
 *     bytes; 1 <= V <= 262144, any V; 1 <= n_rows <= 4194304
 *   row_offset [R + 1], or NULL: one row each (R = n_rows); 1 <= R <= n_rows
 *   history [R][hist_stride] int32 with hist_len [R], prompt_len [R] (NULL: all of it was
 *     generated); history NULL: none.  1 <= hist_stride <= 1048575.  -1: no token.
 *   drafts [R][gamma] int32, the x of dspark_draft; NULL with gamma = 0: none.  A row
 *     behind the last draft counts all of them.  gamma <= 1048575.  -1: no token.
 *   repetition, frequency, presence [R] fp32, each NULL for none; repetition within
 *     [0.001, 1000], the others finite
 *   bias_ids [R][n_bias] int32 (-1: none) and bias [R][n_bias] fp32, 0 <= n_bias <= 1023;
 *     an id that stands again in its request counts the first time only
 *   mask [n_masks][mask_stride] uint32, mask_stride >= ceil(V / 32): bit v % 32 of word
 *     v / 32 is 1 where v is allowed; mask_index [n_rows] int32, the row's mask or -1 for
 *     none (NULL: row i has mask i, n_masks >= n_rows).  mask NULL: none.
 * Output: out [n_rows][out_stride] (dt); it may be X itself (out_stride = row_stride: then
 *   only the lines of a row, 128 bytes from its start on, in which something changes are
 *   read and written), and otherwise overlaps nothing of X (as for dspark_rotary:
 *   DSPARK_ERR_VALUE).  Columns from V on and rows that no request has stay as they were.
 * A token or bias id outside [0, V) and not -1 sets DSPARK_DEVERR_TOKEN and is skipped; a
 * slice of row_offset that decreases or passes n_rows, a hist_len outside
 * [0, hist_stride] or prompt_len outside [0, hist_len] sets DSPARK_DEVERR_LENGTH and
 * counts as empty, 0 and 0 (rows that two of the other slices share, as only offsets out of
 * order make them, are unspecified); a mask_index outside [-1, n_masks) sets it and counts as -1;
 * a parameter out of its range sets DSPARK_DEVERR_NONFINITE and counts as none.
 * Workspace: 256 bytes (the error word). */
dspark_status dspark_edit_logits(int n_rows, int V, int64_t row_stride, dspark_dtype dt,
                                 const void *X, int R, const int32_t *row_offset,
                                 const int32_t *history, int hist_stride, const int32_t *hist_len,
                                 const int32_t *prompt_len, const int32_t *drafts, int gamma,
                                 const float *repetition, const float *frequency,
                                 const float *presence, int n_bias, const int32_t *bias_ids,
                                 const float *bias, int n_masks, const uint32_t *mask,
                                 int64_t mask_stride, const int32_t *mask_index, void *out,
                                 int64_t out_stride, void *ws, size_t ws_bytes,
                                 hipStream_t stream);

/* Gradient with respect to the raw logits X, from that of the edited ones:
 *   dX = v allowed ? (s_v ? (x > 0 ? G / repetition : G repetition) : G) : 0
 * (the counts are constants; biases and the other penalties only add).  X is read only
 * where repetition is given.  G [n_rows][g_stride]; dX [n_rows][dx_stride] may be G
 * itself, but not a part of it or X.  Everything else as above. */
dspark_status dspark_edit_logits_backward(int n_rows, int V, int64_t row_stride, dspark_dtype dt,
                                          const void *X, const void *G, int64_t g_stride, int R,
                                          const int32_t *row_offset, const int32_t *history,
                                          int hist_stride, const int32_t *hist_len,
                                          const int32_t *prompt_len, const int32_t *drafts,
                                          int gamma, const float *repetition, int n_masks,
                                          const uint32_t *mask, int64_t mask_stride,
                                          const int32_t *mask_index, void *dX, int64_t dx_stride,
                                          void *ws, size_t ws_bytes, hipStream_t stream);

/* --------------------------------------------------------- history_append --
 * The histories that dspark_edit_logits reads grow: request rho's new tokens go to
 * history[rho][hist_len[rho] ..] and its length to hist_len_out (which may be hist_len, not a
 * part of it).
 *   tokens [R][width]: the first n_acc[rho] + 1 (the y of dspark_verify; -1: none), or
 *     with n_acc and row_offset NULL all of them;
 *   tokens [n_tokens] with row_offset [R + 1] alone: request rho's are those in
 *     [row_offset[rho], row_offset[rho + 1]), a prompt's (tokens may be NULL with
 *     n_tokens = 0: no request has any);
 *   with n_acc and row_offset both, tokens [R][width], and row_offset is what
 *     dspark_cache_reserve left in its workspace: as in dspark_cache_commit, n_acc[rho] + 1
 *     has to be within the request's rows, so that a round which found no pages (and
 *     has no rows there) leaves the histories as they were
 *   prompt_len [R] or NULL: set to the new length where a request got tokens
 * A request whose tokens do not fit, or with n_acc outside [-1, width) or past its rows,
 * a bad slice or a hist_len outside [0, hist_stride], sets DSPARK_DEVERR_LENGTH and
 * stays as it is.
 * 1 <= R <= 1048576; 1 <= hist_stride <= 1048575; 1 <= width <= 1048575. */
dspark_status dspark_history_append(int R, int width, int n_tokens, const int32_t *tokens,
                                    const int32_t *n_acc, const int32_t *row_offset,
                                    int hist_stride, int32_t *history, const int32_t *hist_len,
                                    int32_t *hist_len_out, int32_t *prompt_len, void *ws,
                                    size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* DSPARK_TOKENS_H */
