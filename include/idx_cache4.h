/*
 * idx_cache4.h -- the paged KV cache in 4 bits: the quantising write, reading back,
 * and attention over all or over the selected pages. Pages, page lists, slots and the
 * rows' lengths are those of idx_cache.h (idx_page_tables serves both caches), and so
 * are its conventions: workspaces are plain scratch, integer arrays on the device are
 * never trusted.
 *
 * A page holds page_size (16, 32 or 64) consecutive tokens of one request, for all Hkv
 * heads. D == IDX_HEAD_DIM. Codes are 4-bit floating point (e2m1: 0, 0.5, 1, 1.5, 2, 3,
 * 4, 6 and their negatives); each 32 dims of a token and head share a scale of 8 bits,
 * a power of two (e8m0: 2^(byte - 127), byte 255 NaN): value = code * scale.
 *   k_cache [n_pages, Hkv, page_size, D/2]  a token's key is a row; byte j holds the dims
 *                                           2 j (low four bits) and 2 j + 1
 *   v_cache [n_pages, Hkv, D, page_size/2]  a token's value is a column; byte j of a dim
 *                                           holds the tokens 2 j (low four bits), 2 j + 1
 *   k_scale [n_pages, Hkv, page_size, D/32], v_scale [n_pages, Hkv, D/32, page_size]
 * all 16-byte aligned. n_pages * Hkv <= 2^31 - 1; the caches may be larger than 4 GiB.
 */
#ifndef IDX_CACHE4_H
#define IDX_CACHE4_H

#include "idx.h"
#include "idx_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

#define IDX_CACHE4_BLOCK 32       /* dims of one scale                              */
#define IDX_CACHE4_MIN_EXP (-60)  /* idx_cache4_write: least scale, 2^-60           */
#define IDX_CACHE4_MAX_EXP 60     /*   and largest, 2^60                            */

/*
 * idx_cache4_write -- quantises the keys and values of n_tok tokens into their slots.
 * For each token, head and 32 dims:
 *   s = the smallest power of two with amax = max |x| <= 6 s, but at least
 *       2^IDX_CACHE4_MIN_EXP and at most 2^IDX_CACHE4_MAX_EXP;
 *   codes are e2m1(x / s), rounded to nearest even; what is larger, infinities too, is
 *   stored as +-6 s. A NaN makes the block's scale NaN.
 * A token's codes depend on the token alone: neighbours in its page keep theirs.
 *   k, v   [n_tok, Hkv, D] dtype dt, 16-byte aligned, token rows k_stride / v_stride
 *          elements apart (multiples of 8, at least Hkv * D)
 *   slots  [n_tok] page * page_size + offset (idx_page_tables); a negative slot or one
 *          past the last page is skipped. A call's slots are distinct (what a slot given
 *          twice holds is unspecified), in any order; rows of consecutive slots share their
 *          stores.
 * n_tok >= 0 (0: nothing is enqueued) and n_tok * ceil(Hkv / 2) below 2^28 (the launch;
 * larger calls are refused, IDX_ERR_INVALID_ARG), dt IDX_F32 or IDX_BF16.
 */
int idx_cache4_write(const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                     const int32_t* slots, uint8_t* k_cache, uint8_t* v_cache, uint8_t* k_scale,
                     uint8_t* v_scale, int n_tok, int Hkv, int D, int n_pages, int page_size,
                     idx_dtype dt, void* stream);

/*
 * idx_cache4_read -- the keys and values of given slots: code * scale, exact in both
 * dtypes for scales from 2^-125 on (and up to 2^125).
 *   slots  [n_tok], in any order, any number of times; a negative slot or one past the
 *          last page gives zeros. Rows of consecutive slots share what they read.
 *   k, v   [n_tok, Hkv, D] dtype dt, 16-byte aligned, token rows k_stride / v_stride
 *          elements apart (multiples of 8, at least Hkv * D); either may be NULL
 * n_tok and the launch as idx_cache4_write.
 */
int idx_cache4_read(const int32_t* slots, const uint8_t* k_cache, const uint8_t* v_cache,
                    const uint8_t* k_scale, const uint8_t* v_scale, void* k, void* v,
                    int64_t k_stride, int64_t v_stride, int n_tok, int Hkv, int D, int n_pages,
                    int page_size, idx_dtype dt, void* stream);

/*
 * idx_attend4, idx_attend4_prefill -- idx_attend and idx_attend_prefill (idx_cache.h) over
 * the 4-bit cache: the same rows, lists, selections, masks, caps, biases, outputs, limits
 * of sizes and workspaces, with these differences:
 *   - a key meets its query as exact bf16 products with its scales in the key (no limit
 *     of their ratios): x is scale times their fp32 sum. Key scales are NaN or from 2^-125
 *     to 2^125, and |q| times the largest that a row sees is at most 2^117 (in place of
 *     idx_cache.h's limit of |q|; a sum reaches 768 times that);
 *   - a probability is rounded to 11 bits (fp16); it, or its value's code, which is exact,
 *     takes the value's scale, relative to the largest that the row sees among its unit (16
 *     tokens from a multiple of 16 on; one 2^25 or more below that counts as zero); a product
 *     of weight and scale is off by up to 2^-33 of the row's largest product of a weight and
 *     its unit's largest scale;
 *   - value scales are NaN or from 2^IDX_CACHE4_MIN_EXP to 2^IDX_CACHE4_MAX_EXP, as the
 *     write gives them (others: the outputs of the rows that see them are unspecified).
 * A NaN scale makes NaN of what it reaches: of a key, the rows that see the token; of a
 * value, its 32 dims of those rows. Bytes of tokens that a row does not see do not reach it,
 * whatever they are. The visible lengths of other rows of a prompt decide whether weight or
 * code takes the scale: a row's bits may differ with them, within the bounds above.
 */
size_t idx_attend4_workspace_bytes(int R, int Hq, int Hkv, int max_pages, int K, int page_size);
int idx_attend4(const void* q, int64_t q_stride, const uint8_t* k_cache, const uint8_t* v_cache,
                const uint8_t* k_scale, const uint8_t* v_scale, const int32_t* kv_indptr,
                const int32_t* kv_indices, const int32_t* kv_len, const int32_t* row_req,
                const int32_t* ids, const float* slopes, void* out, int R, int B, int Hq, int Hkv,
                int D, int n_pages, int64_t n_indices, int max_pages, int page_size, int K,
                float scale, float softcap, idx_dtype dt, void* ws, size_t ws_bytes, void* stream);

size_t idx_attend4_prefill_workspace_bytes(int n_tok, int B, int Hq, int Hkv, int max_pages,
                                           int page_size);
int idx_attend4_prefill(const void* q, int64_t q_stride, const uint8_t* k_cache,
                        const uint8_t* v_cache, const uint8_t* k_scale, const uint8_t* v_scale,
                        const int32_t* kv_indptr, const int32_t* kv_indices,
                        const int32_t* tok_indptr, const int32_t* kv_len, const float* slopes,
                        void* out, int n_tok, int B, int Hq, int Hkv, int D, int n_pages,
                        int64_t n_indices, int max_pages, int page_size, float scale,
                        float softcap, idx_dtype dt, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* IDX_CACHE4_H */
