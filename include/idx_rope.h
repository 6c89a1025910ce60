/*
 * idx_rope.h -- rotary positions of queries and keys (before idx_score and
 * idx_select see them, and before a cache write), and of their gradients, back.
 * The conventions of idx.h hold (device pointers, caller-owned memory, host
 * validation before any launch, status codes, void* stream); the table functions
 * run on the host alone.
 *
 * Of each row of D = IDX_HEAD_DIM dims, the dims first .. first + rot are taken as
 * rot / 2 pairs; pair i of a token at position p turns by the angle p * f_i:
 *   a' = factor * (a cos - b sin),  b' = factor * (b cos + a sin)
 * The pairs are (i, rot / 2 + i) of the part (halves), or (2 i, 2 i + 1) with
 * IDX_ROPE_ADJACENT. The other dims pass unchanged.
 */
#ifndef IDX_ROPE_H
#define IDX_ROPE_H

#include "idx.h"

#ifdef __cplusplus
extern "C" {
#endif

#define IDX_ROPE_ADJACENT 0x1u /* pairs of neighbouring dims                         */
#define IDX_ROPE_INVERSE 0x2u  /* turns back: the gradient of the call without it     */

/* How idx_rope_table stretches frequencies for contexts of `stretch` times the
 * length `original`; n_i = original * f_i / (2 pi) are the turns of pair i over it. */
#define IDX_ROPE_PLAIN 0    /* f_i = base^(-2 i / rot)                                   */
#define IDX_ROPE_LINEAR 1   /* f_i / stretch                                             */
#define IDX_ROPE_BASE 2     /* a larger base: base * stretch^(rot / (rot - 2)), rot > 2  */
#define IDX_ROPE_BY_TURNS 3 /* f_i * (w + (1 - w) / stretch), w rising from 0 to 1 with  */
                            /* n_i between lo and hi turns                               */
#define IDX_ROPE_BY_INDEX 4 /* the same with w falling with i, from 1 at the pair with hi */
                            /* turns (rounded down) to 0 at the one with lo (rounded up)  */

/*
 * idx_rope_turns -- the table of idx_rope from frequencies in radians a token:
 * turns[i] = f_i / (2 pi) in units of 2^-64 of a turn, rounded (off by less than a unit;
 * negative frequencies modulo 2^64). A token's angle is then one 64-bit product, exact
 * modulo a turn: positions cost no bits, however far. 1 <= pairs <= D / 2; each f_i
 * finite and at most 4 in size. Host memory; upload the table once.
 */
int idx_rope_turns(const double* inv_freq, int pairs, uint64_t* turns);

/*
 * idx_rope_table -- the same from a base and one of the kinds above.
 * rot even, 2 <= rot <= D; base > 1, finite; stretch >= 1, original > 0 and
 * 0 < lo < hi where the kind uses them (ignored elsewhere), all finite.
 */
int idx_rope_table(double base, int rot, int kind, double stretch, double original, double lo,
                   double hi, uint64_t* turns);

/*
 * idx_rope -- turns the rows of n_tok tokens.
 *   q, q_out [n_tok, Hq, D], k, k_out [n_tok, Hkv, D], dtype dt, 16-byte aligned, heads
 *       dense, token rows their strides apart (in elements: multiples of 8, at least the
 *       heads times D). An output is its input (same pointer and stride) or does not
 *       overlap it. k, k_out may be NULL with Hkv = 0
 *   tok_len [n_tok] position + 1 (idx_page_tables); a row whose tok_len is 0 or less is
 *       no token: its outputs stay as they are
 *   turns [rot / 2] on the device
 * Angles come from the table's whole numbers without rounding, sine, cosine and sums are
 * fp32: off by at most 2^-21 * |factor| * (|a| + |b|), then rounded once to dt.
 * rot a multiple of 16, 16 <= rot <= D; first a multiple of 8, first + rot <= D; factor
 * finite; n_tok >= 0 (0: nothing is enqueued) and below 2^24 (the launch), Hq >= 1, Hkv >= 0;
 * dt IDX_F32 or IDX_BF16.
 */
int idx_rope(const void* q, const void* k, int64_t q_stride, int64_t k_stride,
             const int32_t* tok_len, const uint64_t* turns, void* q_out, void* k_out,
             int64_t q_out_stride, int64_t k_out_stride, int n_tok, int Hq, int Hkv, int D,
             int first, int rot, float factor, uint32_t flags, idx_dtype dt, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* IDX_ROPE_H */
