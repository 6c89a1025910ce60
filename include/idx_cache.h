/*
 * idx_cache.h -- the paged 8-bit KV cache whose pages the indexer (idx.h)
 * selects: page lists and slot maps from request lengths, the quantising write
 * of new keys and values, and attention over all or over the selected pages.
 * The conventions of idx.h hold (device pointers, caller-owned memory, host
 * validation before any launch, status codes, void* stream), with two
 * additions:
 *   - Workspaces here are plain scratch: they need no zero fill, and hold
 *     nothing from one call to the next. Calls that may overlap need distinct
 *     ones.
 *   - Integer arrays that live on the device are never trusted: a page, slot,
 *     request or id outside its range is skipped as described per call, and no
 *     access leaves the arrays whose sizes the call was given.
 *
 * A page holds page_size (16, 32 or 64) consecutive tokens of one request, for
 * all Hkv heads. D == IDX_HEAD_DIM. Codes are 8-bit floating point (e4m3, no
 * infinities, largest 448, pattern 0x7F / 0xFF NaN), with one fp32 scale for
 * each page and head: value = code * scale.
 *   k_cache [n_pages, Hkv, page_size, D]   a token's key is a row
 *   v_cache [n_pages, Hkv, D, page_size]   a token's value is a column
 *   k_scale, v_scale [n_pages, Hkv] float32, finite, at least 2^IDX_CACHE_MIN_EXP
 * n_pages * Hkv <= 2^31 - 1; the caches themselves may be larger than 4 GiB.
 */
#ifndef IDX_CACHE_H
#define IDX_CACHE_H

#include "idx.h"

#ifdef __cplusplus
extern "C" {
#endif

#define IDX_MAX_GROUP 64         /* Hq / Hkv of the attention calls               */
#define IDX_MIN_SOFTCAP 0x1p-20f /* smallest and largest cap of scores: a capped score is off */
#define IDX_MAX_SOFTCAP 0x1p16f  /* by up to 2^-20 of a cap up to 64, 2^-19 of itself above  */
#define IDX_CACHE_MIN_EXP (-120) /* idx_cache_write: least scale, 2^-120          */

/*
 * idx_page_tables -- one step of the page allocator, and the lists the other
 * calls read. Request b holds seq_len[b] tokens in the pages
 * table[b, 0 .. ceil(seq_len[b] / page_size)) and changes by n_new[b] tokens: a
 * positive count adds tokens, a negative one takes the last tokens back
 * (rejected drafts; -seq_len[b] ends the request), never below zero.
 *   Free pages wait in a ring: entry (head + i) % n_pages, i < count, with
 *   cursor = {head, count}. Requests take new pages from the front in request
 *   order, pages given back join at the end in request order and serve the
 *   NEXT call (never this one).
 *   A request that adds tokens is refused, and keeps its length and pages, if
 *   it would pass max_pages, if its token rows would pass n_tokens, or if the
 *   pages needed by the requests up to and including it (refused ones for
 *   those two reasons left out) exceed the free count. One that needs no new
 *   page is not refused for the last reason.
 * Inputs
 *   seq_len [B], n_new [B]   (seq_len is clamped to [0, max_pages * page_size])
 *   cursor  [2] {head, count}; taken modulo n_pages / clamped to [0, n_pages]
 * Updated in place
 *   table     [B, max_pages]: the new pages' entries; all others keep their
 *             values (also those of pages given back)
 *   free_ring [n_pages]: the given back pages' entries
 * Outputs
 *   seq_out    [B] lengths after the step        cursor_out [3] {head, count,
 *              requests refused}
 *   kv_indptr  [B+1], kv_indices [n_indices]: the requests' pages, packed as
 *              idx_select_paged takes them (entries past n_indices are dropped,
 *              those past kv_indptr[B] keep their values)
 *   tok_indptr [B+1]: the packed rows of the new tokens, max(n_new, 0) each, for
 *              refused requests too (clamped to n_tokens)
 *   slots      [n_tokens] page * page_size + offset of each new token; -1 for a
 *              refused request's tokens and for rows past tok_indptr[B]
 *   tok_req    [n_tokens] the row's request; -1 past tok_indptr[B]
 *   tok_len    [n_tokens] position + 1 (the tokens the row sees); 0 where slots
 *              is -1
 * No output may alias an input: with cursor and seq_len left as they are, a
 * repeated call gives the same result.
 * B >= 1 and B <= IDX_MAX_REQUESTS, max_pages, n_pages >= 1, n_tokens >= 0,
 * B * max_pages, max_pages * page_size and n_pages * page_size <= 2^31 - 1,
 * page_size >= 1. slots, tok_req and tok_len may be NULL when n_tokens is 0.
 */
int idx_page_tables(const int32_t* seq_len, const int32_t* n_new, const int32_t* cursor,
                    int32_t* table, int32_t* free_ring, int32_t* seq_out, int32_t* cursor_out,
                    int32_t* kv_indptr, int32_t* kv_indices, int32_t* tok_indptr, int32_t* slots,
                    int32_t* tok_req, int32_t* tok_len, int B, int max_pages, int page_size,
                    int n_pages, int64_t n_indices, int n_tokens, void* stream);

/*
 * idx_cache_write -- quantises the keys and values of n_tok tokens into their
 * slots. For each page and head that receives tokens:
 *   s = the smallest power of two, at least 2^IDX_CACHE_MIN_EXP, with
 *       amax <= 448 s, amax over the call's finite values for that page and head;
 *   a page whose first written offset is above 0 keeps its earlier tokens: the
 *   scale becomes max(s, old scale) and, where it grew, the earlier codes become
 *   e4m3(code * (old / new)) (exact unless they fall below the normal range, when
 *   the old scale is a power of two);
 *   new codes are e4m3(x / scale), rounded to nearest even; an infinite x is
 *   stored as +-448, NaN as NaN.
 * Powers of two: e4m3 keeps its relative precision under them, and a growing
 * scale leaves the codes exact instead of rounding them once more.
 * Offsets past the tokens written keep their codes.
 *   k, v   [n_tok, Hkv, D] dtype dt, 16-byte aligned, token rows k_stride /
 *          v_stride elements apart (multiples of 8, at least Hkv * D)
 *   slots  [n_tok] page * page_size + offset (idx_page_tables); a negative slot
 *          or one past the last page is skipped. A call's slots are distinct,
 *          and the tokens of one page lie in consecutive rows, in order of
 *          their offsets and without gaps; otherwise that page's contents are
 *          unspecified.
 * n_tok >= 0 (0: nothing is enqueued) and n_tok * ceil(Hkv / 2) below 2^28 (the launch; larger
 * calls are refused, IDX_ERR_INVALID_ARG), dt IDX_F32 or IDX_BF16, page_size 16, 32 or 64.
 */
int idx_cache_write(const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                    const int32_t* slots, uint8_t* k_cache, uint8_t* v_cache, float* k_scale,
                    float* v_scale, int n_tok, int Hkv, int D, int n_pages, int page_size,
                    idx_dtype dt, void* stream);

/*
 * idx_attend -- attention of single tokens (decode steps, or prompt tokens that
 * each bring their own selection). Row r, query head hq, with the KV head
 * h = hq / (Hq / Hkv) and request b = row_req[r]:
 *   x_j   = scale * q[r,hq,:] . key(j,h)           for the visible tokens j
 *   x_j   = softcap * tanh(x_j / softcap)          if softcap > 0
 *   x_j  -= slopes[hq] * (kv_len[r] - 1 - j)       if slopes is given
 *   out[r,hq,:] = sum_j softmax(x)_j * value(j,h,:)
 * Visible are the tokens j < kv_len[r] of the pages in request b's list
 * kv_indices[kv_indptr[b] .. kv_indptr[b+1]) (clamped to max_pages pages); with
 * ids, those of the listed page slots ids[r, 0..K) alone (as idx_select_paged
 * and idx_select_prefill write them; -1 and slots past the list are skipped, a
 * slot listed twice counts twice). A list position outside [0, n_indices) or a
 * page outside [0, n_pages) holds no tokens. A row that sees nothing, or whose
 * request is outside [0, B), gets zeros. Codes of tokens a row does not see do
 * not reach it, whatever they are.
 *   q   [R, Hq, D] bf16, 16-byte aligned, rows q_stride elements apart (a
 *       multiple of 8, at least Hq * D)
 *   out [R, Hq, D] bf16, dense, 16-byte aligned
 *   kv_len [R]; row_req [R] or NULL (row r is request r; then R <= B): for rows as
 *       idx_page_tables packs them, tok_len and tok_req
 *   ids [R, K] or NULL (then K is 0); slopes [Hq] float32 or NULL
 * A prefix mask (tokens of a prefix see all of it) needs no argument: give each
 * row of the prefix the prefix's length as kv_len.
 * Scores, softmax statistics and sums are fp32; keys and queries meet as exact
 * bf16 products; a probability is rounded to 11 bits (fp16) before it meets its
 * value, whose e4m3 code is exact there. That holds while the value scales of the tokens that
 * a row sees lie within 2^20 of each other, and none above 2^70 (a row's sums are kept in
 * units of the largest it sees). No bit of a row depends on the codes of tokens that it does
 * not see, nor on the scales of pages that it sees nothing of.
 * scale finite, its product with any key scale 0 or at least 2^-126 in size; |q| at most
 * 2^104 (products of queries and codes are summed before the key scale meets them) and the
 * scores finite in fp32; softcap 0 (none) or from IDX_MIN_SOFTCAP to IDX_MAX_SOFTCAP.
 * R >= 0 (0: nothing is enqueued), B >= 1,
 * 1 <= Hq / Hkv <= IDX_MAX_GROUP, Hq a multiple of Hkv, page_size 16, 32 or 64.
 * Calls whose launch would pass 2^32 - 1 threads are refused (IDX_ERR_INVALID_ARG): R * Hkv
 * from 2^24 on, from 2^23 on for groups above 32 heads.
 * max_pages may be any bound of the lists' lengths; how rows are cut for the chip goes
 * by it, so that work spreads best when it is near the longest list.
 * ws: at least idx_attend_workspace_bytes(...) bytes (256-byte aligned; may be
 * NULL when that is 0): partial results of rows split over several workgroups.
 */
size_t idx_attend_workspace_bytes(int R, int Hq, int Hkv, int max_pages, int K, int page_size);
int idx_attend(const void* q, int64_t q_stride, const uint8_t* k_cache, const uint8_t* v_cache,
               const float* k_scale, const float* v_scale, const int32_t* kv_indptr,
               const int32_t* kv_indices, const int32_t* kv_len, const int32_t* row_req,
               const int32_t* ids, const float* slopes, void* out, int R, int B, int Hq, int Hkv,
               int D, int n_pages, int64_t n_indices, int max_pages, int page_size, int K,
               float scale, float softcap, idx_dtype dt, void* ws, size_t ws_bytes, void* stream);

/*
 * idx_attend_prefill -- idx_attend for packed prompt tokens: request b's token
 * rows are tok_indptr[b] .. tok_indptr[b+1] (as idx_page_tables writes them), so
 * that rows of one request share the keys and values they read. Row t sees the
 * tokens j < kv_len[t] of its request's pages (tok_len of idx_page_tables gives
 * the causal mask; any lengths are allowed). Rows outside the requests' ranges
 * (past tok_indptr[B]) keep their output. tok_indptr is ascending within
 * [0, n_tok]; entries outside that range are clamped to it.
 *   q, out [n_tok, Hq, D]; kv_len [n_tok]; the other arguments, the limits and
 *   the arithmetic are those of idx_attend. B <= IDX_MAX_REQUESTS. The launch is taken at 512
 *   threads for each KV head and tile of 256 rows (token, head of the group), of 16 rows in
 *   calls of few rows a request: refused where n_tok * Hq + 256 * B * Hkv reaches 2^31, or a
 *   sixteenth of that.
 * Calls of few rows a request (n_tok * Hq / Hkv / B up to 64: drafted tokens) share out
 * the keys among waves, longer prompts the rows; a batch of both does best as two calls. B
 * counts requests without rows too: a prompt among many idle requests runs best in a call
 * whose lists name the requests that have rows.
 */
size_t idx_attend_prefill_workspace_bytes(int n_tok, int B, int Hq, int Hkv, int max_pages,
                                          int page_size);
int idx_attend_prefill(const void* q, int64_t q_stride, const uint8_t* k_cache,
                       const uint8_t* v_cache, const float* k_scale, const float* v_scale,
                       const int32_t* kv_indptr, const int32_t* kv_indices,
                       const int32_t* tok_indptr, const int32_t* kv_len, const float* slopes,
                       void* out, int n_tok, int B, int Hq, int Hkv, int D, int n_pages,
                       int64_t n_indices, int max_pages, int page_size, float scale,
                       float softcap, idx_dtype dt, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* IDX_CACHE_H */
