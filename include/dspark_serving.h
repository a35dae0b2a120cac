/*
 * dspark_serving.h -- C ABI of what stands on either side of dspark_verify in
 * a server: the paged key-value cache that the verified rows read, and the log
 * probabilities that go out with the emitted tokens (or back as gradients).
 *
 *   dspark_logprobs, dspark_logprobs_backward
 *                          log probabilities of given tokens with entropy and
 *                          the top alternatives, and their gradient
 *   dspark_cache_attend    attention of the new rows of every request over its
 *                          pages, which the rows' own keys and values join
 *   dspark_cache_fork, _reserve, _commit, _release, _compact
 *                          the pages: shared, taken, copied, given back, moved
 *
 * One round of a server with a paged target (Blog, "Variable-length
 * verification without wasting kernels"): dspark_draft -> dspark_schedule ->
 * dspark_cache_reserve(row_offset) -> the target's layers, each with one
 * dspark_cache_attend over the reserved rows -> dspark_verify ->
 * dspark_cache_commit(reserved rows, n_acc) -> dspark_logprobs(P, y).  The reserved
 * rows are row_offset again for a host that has read `missing` and found 0; one that
 * does not wait for it (a captured round) passes the copy that reserve leaves in its
 * workspace, and a round that found no room then changes nothing.
 *
 * The conventions of dspark.h hold: device pointers, 16-byte aligned unless
 * stated; caller-owned buffers; host-side validation first; asynchronous on
 * `stream`; data errors OR a DSPARK_DEVERR_* bit into the first word of the
 * workspace.  Nothing is allocated and every call may be captured into a graph.
 * Calls that share a workspace, and calls that change a cache's arrays, must be
 * ordered on one stream.
 */
#ifndef DSPARK_SERVING_H
#define DSPARK_SERVING_H

#include "dspark.h"

#ifdef __cplusplus
extern "C" {
#endif

/* More bits of the sticky device error word. */
#define DSPARK_DEVERR_PAGE 32    /* a page number outside [0, n_pages) in a table       */
#define DSPARK_DEVERR_NO_PAGES 64 /* dspark_cache_reserve found too few free pages      */

/* --------------------------------------------------------------- logprobs --
 * For every logit row i with z = X[i] / temp, m = max z, S = sum_v exp(z_v - m):
 *   logp[i]     = z_t - m - log S, t the row's token
 *   entropy[i]  = -sum_v p_v log p_v = log S - sum_v exp(z_v - m)(z_v - m) / S
 *   top_ids[i][j], top_logp[i][j], j < k: the k largest logits in descending
 *                 order, equal ones by ascending index, and their log
 *                 probabilities
 *   stats[i]    = (m, S), as dspark_tv_overlap takes them (S belongs to the
 *                 rounded m: with temp != 1 and |m| > 2^31 it may overflow, and
 *                 dspark_logprobs_backward then takes the row as without stats)
 * A masked logit (-infinity) has probability 0, adds nothing to the entropy and
 * counts as an alternative (log probability -infinity) only behind every other.
 * Inputs
 *   X [n_rows][row_stride] logits (dt), V of each row used; row_stride >= V and
 *     a multiple of 16 bytes; 1 <= V <= 262144, any V; 1 <= n_rows <= 4194304
 *   tokens  [n_rows] int32, or with row_offset [R][tok_stride]: row
 *     row_offset[rho] + j takes tokens[rho * tok_stride + j] (the layout of
 *     dspark_verify's y, tok_stride = gamma + 1).  -1, and a j past tok_stride:
 *     no token, logp = 0.  Another value outside [0, V) sets DSPARK_DEVERR_TOKEN
 *     and gives NaN.  NULL (with logp NULL): no tokens at all.
 *   row_offset [R + 1] int32 as written by dspark_schedule, or NULL; rows from
 *     row_offset[R] on are not read and their outputs stay as they were.  An
 *     end past n_rows sets DSPARK_DEVERR_LENGTH and is taken as n_rows.
 *     1 <= R <= n_rows: n_rows is the rows' capacity, as dspark_verify's
 *     rows_capacity, so a batch whose requests have fewer rows than there are
 *     requests still comes in a buffer of R rows.
 *   0 <= k <= 64, k <= V
 * Outputs (fp32; top_ids int32): logp, entropy, stats, top_ids, top_logp; each
 *   of logp, entropy, stats may be NULL; top_ids and top_logp are given iff k > 0.
 * A row whose maximum or S is not finite (all masked, a NaN, +infinity) sets
 * DSPARK_DEVERR_NONFINITE; its outputs are NaN and its top_ids -1.
 * Workspace: dspark_logprobs_workspace(n_rows, V, k, dt) bytes. */
size_t dspark_logprobs_workspace(int n_rows, int V, int k, dspark_dtype dt);
dspark_status dspark_logprobs(int n_rows, int V, int64_t row_stride, dspark_dtype dt, float temp,
                              const void *X, const int32_t *tokens, int tok_stride, int R,
                              const int32_t *row_offset, int k, float *logp, float *entropy,
                              float *stats, int32_t *top_ids, float *top_logp, void *ws,
                              size_t ws_bytes, hipStream_t stream);

/* Gradient of L with respect to the logits, from the gradients of dspark_logprobs'
 * outputs (p from stats, all sums as in dspark_logprobs):
 *   dX[i][v] = (1/temp) [ g_logp[i] (1[v = t] - p_v)
 *                         + sum_j g_top[i][j] (1[v = top_ids[i][j]] - p_v)
 *                         - g_entropy[i] p_v (log p_v + entropy[i]) ]
 * Inputs: X, tokens, tok_stride, R, row_offset as above; stats [n_rows][2] and
 *   entropy [n_rows] as written by dspark_logprobs; g_logp, g_entropy [n_rows],
 *   g_top [n_rows][k] fp32, each of them NULL for zeros (entropy may be NULL
 *   when g_entropy is; top_ids and g_top are given iff k > 0).  A row without
 *   a token takes g_logp as 0.  An index outside [0, V) in top_ids sets
 *   DSPARK_DEVERR_TOKEN and its g_top counts as 0, as does a token's g_logp.
 * Output: dX [n_rows][dx_stride] (dt), rounded once; it may be X itself (with
 *   dx_stride = row_stride).  Columns from V on and rows from row_offset[R] on
 *   stay as they were.  A row whose stats are not finite gets zeros and sets
 *   DSPARK_DEVERR_NONFINITE.
 * Workspace: 256 bytes (the error word). */
dspark_status dspark_logprobs_backward(int n_rows, int V, int64_t row_stride, dspark_dtype dt,
                                       float temp, const void *X, const int32_t *tokens,
                                       int tok_stride, int R, const int32_t *row_offset,
                                       const float *stats, const float *entropy,
                                       const float *g_logp, const float *g_entropy, int k,
                                       const int32_t *top_ids, const float *g_top, void *dX,
                                       int64_t dx_stride, void *ws, size_t ws_bytes,
                                       hipStream_t stream);

/* ----------------------------------------------------------- cache layout --
 * A cache holds the keys and values of R requests in n_pages pages of `page`
 * tokens (page a power of two, 16 <= page <= 256).  For one layer:
 *   k_pages [n_pages][Hkv][page][D]   token t of a request: page table[t / page],
 *   v_pages [n_pages][Hkv][D][page]   slot t % page (values lie along the tokens,
 *                                     the order in which the product reads them)
 * with page_stride elements from one page to the next, so the layers of a model
 * may lie side by side within a page: [n_pages][layers][Hkv][page][D].
 * State of the requests (int32, shared by all layers):
 *   lens  [R]            tokens held
 *   table [R][max_pages] page numbers; entries from ceil(lens / page) on are -1
 *   refs  [n_pages]      table entries that hold the page; 0: free
 * The page operations read lens, table, refs and write lens_out, table_out,
 * refs_out: either all three the same arrays (in place) or three that overlap
 * none of them.  1 <= R <= 8192; 1 <= n_pages <= 4194304; 1 <= max_pages with
 * R * max_pages <= 2^28 and page * max_pages <= 2^30.
 * A page number outside [0, n_pages) that an operation comes upon within a
 * request's length sets DSPARK_DEVERR_PAGE; such an entry is never followed.  A
 * length outside [0, page * max_pages] sets DSPARK_DEVERR_LENGTH and is read as
 * 0 by fork and release; commit and compact leave that request as it is, and
 * reserve the whole state.
 * Workspace of every page operation: dspark_cache_workspace(R, n_pages) bytes. */
size_t dspark_cache_workspace(int R, int n_pages);

/* Requests dst[i], i < n, become copies of src[i] as they were before the call,
 * sharing their pages (a best-of-n reply, a branch of a conversation).  The
 * same src may stand several times.  A number outside [0, R), a dst that
 * already holds tokens or stands again sets DSPARK_DEVERR_LENGTH and that pair
 * is skipped (of a dst that stands twice, the first pair counts). 1 <= n <= R. */
dspark_status dspark_cache_fork(int R, int page, int max_pages, int n_pages, int n,
                                const int32_t *src, const int32_t *dst, const int32_t *lens,
                                const int32_t *table, const int32_t *refs, int32_t *lens_out,
                                int32_t *table_out, int32_t *refs_out, void *ws, size_t ws_bytes,
                                hipStream_t stream);

/* Room for the new rows of a round: request rho grows by row_offset[rho + 1] -
 * row_offset[rho] tokens (0: it stays).  New pages are the lowest free ones, in
 * the order of the requests.  A partly filled last page that others hold too is
 * first copied to a new page (whole, in both pools), because the new tokens
 * will be written into it; where every holder writes it in this call, the
 * first of them keeps it.  All or nothing: with too few free pages (sets
 * DSPARK_DEVERR_NO_PAGES), a length outside [0, page * max_pages] before or
 * after, or a decreasing row_offset (DSPARK_DEVERR_LENGTH) the state stays as
 * it was.
 *   k_pages, v_pages: the whole pools, page p at byte p * page_bytes of each
 *     (16-byte multiples); NULL both: no pages are copied (state only)
 *   missing [1] int32: 0 when done, the pages short, or -1 on a bad length
 * The reserved rows: R + 1 int32 at byte 256 of the workspace, row_offset where the
 * call is done and zeros where it changed nothing.  They stay until the next reserve
 * over the workspace (and a call over it with another R).  Given as row_offset,
 * dspark_cache_attend has no rows after a reserve that changed nothing, so it writes
 * neither pages nor outputs, and dspark_cache_commit leaves every request as it is
 * (and sets DSPARK_DEVERR_LENGTH where n_acc >= 0).  With the caller's own row_offset
 * they would take the last tokens held for the round's. */
dspark_status dspark_cache_reserve(int R, int page, int max_pages, int n_pages,
                                   const int32_t *row_offset, const int32_t *lens,
                                   const int32_t *table, const int32_t *refs, int32_t *lens_out,
                                   int32_t *table_out, int32_t *refs_out, void *k_pages,
                                   void *v_pages, size_t page_bytes, int32_t *missing, void *ws,
                                   size_t ws_bytes, hipStream_t stream);

/* After the verification: of the n = row_offset[rho + 1] - row_offset[rho] rows
 * that request rho reserved, the first n_acc[rho] + 1 stay (the anchor and the
 * accepted drafts; n_acc as dspark_verify wrote it, -1: none).  The rest leave
 * its length, and pages wholly behind it are given back.  n_acc + 1 outside
 * [0, n] or n outside [0, lens] sets DSPARK_DEVERR_LENGTH and the request
 * stays as it is. */
dspark_status dspark_cache_commit(int R, int page, int max_pages, int n_pages,
                                  const int32_t *row_offset, const int32_t *n_acc,
                                  const int32_t *lens, const int32_t *table, const int32_t *refs,
                                  int32_t *lens_out, int32_t *table_out, int32_t *refs_out,
                                  void *ws, size_t ws_bytes, hipStream_t stream);

/* Requests which[i], i < n, leave: their pages are given back (freed when no
 * other request holds them) and their length is 0.  Twice the same: once.  A
 * number outside [0, R) sets DSPARK_DEVERR_LENGTH and is skipped.  1 <= n <= R. */
dspark_status dspark_cache_release(int R, int page, int max_pages, int n_pages, int n,
                                   const int32_t *which, const int32_t *lens,
                                   const int32_t *table, const int32_t *refs, int32_t *lens_out,
                                   int32_t *table_out, int32_t *refs_out, void *ws,
                                   size_t ws_bytes, hipStream_t stream);

/* Moves the pages in use to the numbers [0, n_live): the i-th used page from
 * n_live on goes to the i-th free one below, in both pools (NULL both: numbers
 * only).  n_live [1] int32; the pool's end is then free, so a caller may shrink
 * it or hand it on.  A table entry that names a free page from n_live on sets
 * DSPARK_DEVERR_PAGE too and stays as it is. */
dspark_status dspark_cache_compact(int R, int page, int max_pages, int n_pages,
                                   const int32_t *lens, const int32_t *table, const int32_t *refs,
                                   int32_t *lens_out, int32_t *table_out, int32_t *refs_out,
                                   void *k_pages, void *v_pages, size_t page_bytes,
                                   int32_t *n_live, void *ws, size_t ws_bytes,
                                   hipStream_t stream);

/* ----------------------------------------------------------- cache_attend --
 * Attention of every request's new rows over its pages.  Request rho has the
 * rows [row_offset[rho], row_offset[rho + 1]), n of them (1 + ell in a verified
 * round, 1 in plain decoding, a prompt's length when it enters), the last n of
 * its kv_len[rho] tokens.  Row j = 0..n-1 is token kv_len - n + j and sees the
 * tokens 0..kv_len - n + j, the last `window` of them if window > 0:
 *   s_t = scale q . k_t,  out = sum_t softmax(s)_t v_t,  lse = log sum_t exp(s_t)
 * Query head h reads key-value head h / (Hq / Hkv).  A row that sees nothing
 * (kv_len too small) gives zeros and lse = -infinity.  What lies in slots that
 * a row does not see never reaches it, NaN and infinity included.
 * Inputs
 *   dt BF16 or F32 for q, the new rows, the pages and out; statistics and sums
 *     are fp32 (BF16: the probabilities enter the product as a bf16 and a bf16
 *     remainder, 16 bits together)
 *   Hq a multiple of Hkv, Hq <= 1024; D one of 64, 96, 128, 256;
 *     1 <= rows_capacity <= 1048576
 *   q [rows_capacity][Hq][D], q_stride elements from row to row
 *   k_new, v_new [rows_capacity][Hkv][D], kv_stride elements from row to row:
 *     written into their slots of k_pages and v_pages first; or NULL both when
 *     the pages already hold them
 *   strides in elements, multiples of 16 bytes
 *   row_offset [R + 1], or NULL: one row each (rows_capacity = R)
 *   kv_len [R]: lens_out of dspark_cache_reserve; table, n_pages as above
 *   1e-30 <= scale <= 1e30; window >= 0 (0: none)
 * Outputs: out [rows_capacity][Hq][D] (dt); lse [rows_capacity][Hq] fp32 or
 *   NULL.  Rows from row_offset[R] on stay as they were.
 * A slice of row_offset that decreases or passes rows_capacity, or a kv_len
 * outside [0, page * max_pages] sets DSPARK_DEVERR_LENGTH: the slice counts as
 * empty, the length as 0.  New rows that would lie before token 0 set it too
 * and are not written.  A bad page number sets DSPARK_DEVERR_PAGE: its tokens
 * count as masked.
 * Workspace: dspark_cache_attend_workspace(R, rows_capacity, Hq, Hkv, D, dt). */
size_t dspark_cache_attend_workspace(int R, int rows_capacity, int Hq, int Hkv, int D,
                                     dspark_dtype dt);
dspark_status dspark_cache_attend(int R, int rows_capacity, int Hq, int Hkv, int D, int page,
                                  int max_pages, int n_pages, dspark_dtype dt, float scale,
                                  int window, const void *q, int64_t q_stride, const void *k_new,
                                  const void *v_new, int64_t kv_stride, void *k_pages,
                                  void *v_pages, int64_t k_page_stride, int64_t v_page_stride,
                                  const int32_t *table, const int32_t *row_offset,
                                  const int32_t *kv_len, void *out, float *lse, void *ws,
                                  size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* DSPARK_SERVING_H */
