/*
 * libsdm: choosing slots, and banks held in 8 or 4 bits, on an AMD Instinct
 * MI355X (gfx950). Part of libsdm, with the conventions of sdm.h: every pointer
 * of a compute call is a device pointer to a contiguous, row-major array that
 * the caller owns, the library allocates nothing and keeps no state, work is
 * only enqueued on `hip_stream` (so calls may be captured in a HIP graph, and
 * calls on several streams may run at once), the cheap argument checks run on
 * the host before any HIP call, and a failing call enqueues nothing and returns
 * a status code of sdm.h with a message for sdm_last_error().
 *
 *   sdm_route                scores -> slots and weights, as sdm_gather and the
 *                            decode take them
 *   sdm_route_backward       gradient of the weights -> gradient of the scores
 *   sdm_bank_pack            rows -> rows of a packed bank (8 or 4 bits)
 *   sdm_gather_packed        sdm_gather (without a stash) from a packed bank
 *   sdm_gather_weight_grad   gradient of a gather's weights, from any bank
 */
#ifndef SDM_MEMORY_H
#define SDM_MEMORY_H

#include <stdint.h>

#include "sdm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SDM_MAX_KEYS 65536  /* most keys of a route */
#define SDM_MAX_ROUTE_TOKENS (1LL << 21) /* most tokens of a route: 1024 threads each of a grid */
#define SDM_MAX_GROUPS 256  /* most groups of a route */
#define SDM_PACK_BLOCK 32   /* columns of a packed row that share a scale */

/*
 * Packed element types. A packed bank is two arrays:
 *   codes   [num_slots, row_bytes]        the elements' codes, row_bytes =
 *           sdm_packed_row_bytes(): the code bytes of a row rounded up to 16
 *   scales  [num_slots, scale_row_bytes]  a byte for each block of 32 columns,
 *           scale_row_bytes = sdm_packed_scale_bytes(): rounded up to 4
 * Both 16-byte and 4-byte aligned. Scale byte b < 255 stands for 2^(b - 127),
 * 255 for not-a-number. Column c of a row has the value code * scale[c / 32]:
 *   SDM_MX8  code byte c: sign, 4 bits of exponent (bias 7), 3 of fraction; the
 *            largest value is 448; 0x7f and 0xff are not a number.
 *   SDM_MX4  half of byte c / 2 (the low half for even c): sign, 2 bits of
 *            exponent (bias 1), 1 of fraction: 0, 0.5, 1, 1.5, 2, 3, 4, 6.
 * A float32 holds every such value exactly, but those of a caller's own bytes that are
 * past its range (scales above 2^119), which read as infinite.
 */
enum {
    SDM_MX8 = 4,
    SDM_MX4 = 5
};

/* Score functions of a route. */
enum {
    SDM_SOFTMAX = 0, /* over the keys of a row */
    SDM_SIGMOID = 1
};

/* Bytes of one row of `codes` and of `scales`; 0 for another dtype, or a
 * head_dim outside 1..SDM_MAX_ROW_BYTES. */
int64_t sdm_packed_row_bytes(int packed_dtype, int64_t head_dim);
int64_t sdm_packed_scale_bytes(int packed_dtype, int64_t head_dim);

/*
 * sdm_route: for each token, the k best keys and their weights.
 *
 * With x a row of logits (NaN counts as -inf, +inf as the largest float32):
 *     s = softmax(x), or 1 / (1 + exp(-x))
 *     c = s + bias          (bias only steers the choice)
 * A key is eligible when x > -inf and its bias is neither -inf nor NaN; the
 * others rank below every eligible key and have weight 0.
 * With groups > 1 the keys are `groups` equal consecutive runs: a group's value
 * is the sum of its group_top largest eligible c (-inf if none is eligible),
 * only the kept_groups best groups' keys can be chosen.
 * The k keys of largest c are chosen, in descending order. Values are compared
 * as computed in float64 (keys without a bias: by x, which has the same order;
 * groups always by their values, so that groups of saturated scores are equal),
 * and every tie goes to the lowest key or group, so the choice is a function of
 * the inputs alone.
 *     u_j = s of chosen key j (0 if not eligible)
 *     w_j = scale * u_j / (normalise ? sum_j u_j : 1)     (0 where that sum is 0)
 *     idx_j = (t mod streams) * stream_slots + key
 * The slots of one token are distinct, and with stream_slots >= keys the slots
 * of different streams are too, as the decode needs them.
 *
 * Arguments:
 *   logits      [tokens, keys] of logit_dtype (SDM_F32 or SDM_BF16).
 *   tokens      0..SDM_MAX_ROUTE_TOKENS; 0 enqueues nothing. keys 1..SDM_MAX_KEYS.
 *   k           1..SDM_MAX_WIDTH, at most kept_groups * keys / groups.
 *   score       SDM_SOFTMAX or SDM_SIGMOID.
 *   bias        NULL, or [keys] float32.
 *   groups      1..SDM_MAX_GROUPS, a divisor of keys; kept_groups in 1..groups;
 *               group_top 1 or 2.
 *   scale       finite.
 *   streams     >= 1; stream_slots >= 0 (0: all streams share the keys' slots).
 *   idx         [tokens, k] SDM_I32 or SDM_I64 (idx_dtype), written; every slot
 *               must fit the type (SDM_E_RANGE).
 *   w           [tokens, k] SDM_F32 or SDM_BF16 (w_dtype), written.
 * Weights are computed in float64 for the chosen keys (a softmax's sum over all
 * keys in float32), rounded to float32 and then to w_dtype.
 * Errors: SDM_E_DTYPE, SDM_E_SHAPE, SDM_E_RANGE, SDM_E_NULL, SDM_E_ALIGN,
 * SDM_E_OVERLAP, SDM_E_HIP.
 */
int sdm_route(const void* logits, int logit_dtype, int64_t tokens, int64_t keys, int32_t k, int score,
              const float* bias, int32_t groups, int32_t kept_groups, int32_t group_top, int32_t normalise,
              float scale, int64_t streams, int64_t stream_slots, void* idx, int idx_dtype, void* w, int w_dtype,
              void* hip_stream);

/*
 * sdm_route_backward: gradient of sdm_route's weights with respect to its logits.
 *
 * With idx as sdm_route gave it (the choice itself has no gradient) and dw the
 * gradient of w:
 *     normalise:  du_j = scale * (dw_j - sum_m dw_m u_m / U) / U,   U = sum_m u_m
 *     otherwise:  du_j = scale * dw_j
 *     softmax:    dlogits_i = s_i (du_i - sum_j du_j s_j)     (du_i = 0 if i is not chosen)
 *     sigmoid:    dlogits_i = s_i (1 - s_i) du_i
 * du_j is 0 for a chosen key that is not eligible, and all of a row's where U is 0;
 * dlogits is 0 for a key at -inf, also where other gradients are not finite. A key that
 * its bias alone excludes is in a softmax's sum all the same, and has that part.
 * A renormalised softmax's gradient is 0 outside the chosen keys.
 * The part of the chosen keys is computed in float64, with a full softmax's sum over
 * all keys taken from float32 exponentials relative to the row's largest logit, whose
 * own is exactly 1, and added in float64: 1 - s of a key far above the rest is as
 * precise as the others' terms. A full softmax's other keys are computed in float32,
 * where a score below 2^-126 may count as 0. Each value is rounded to float32 and then
 * to the logits' type.
 *
 * Arguments: as sdm_route (bias only tells which keys are eligible), with
 *   dw       [tokens, k] of w_dtype.
 *   dlogits  [tokens, keys] of logit_dtype, written whole; must not overlap an input.
 * A slot of idx that is not one of its token's `keys` slots adds nothing; a slot
 * given more than once gets the sum of its terms (in no fixed order; the route
 * gives distinct slots).
 * Errors: as sdm_route.
 */
int sdm_route_backward(const void* logits, int logit_dtype, int64_t tokens, int64_t keys, int32_t k, int score,
                       const float* bias, int32_t normalise, float scale, int64_t streams, int64_t stream_slots,
                       const void* idx, int idx_dtype, const void* dw, int w_dtype, void* dlogits,
                       void* hip_stream);

/*
 * sdm_bank_pack: quantise rows as they are written to a packed bank.
 *
 * For i < n, row (row_idx ? row_idx[i] : i) of `rows` goes to slot (slots ?
 * slots[i] : i) of the packed bank. In each block of 32 columns, with a the
 * largest finite magnitude and M = 448 (SDM_MX8) or 6 (SDM_MX4):
 *     scale = 2^e,  e the least integer in [-127, 127] with a <= M 2^e
 *     code  = x / 2^e rounded to the nearest code, ties to the even code
 * All of it is exact arithmetic: the bits depend on nothing but the row. The
 * sign of a zero is kept. An element that is not finite is not-a-number in
 * SDM_MX8 (code 0x7f) and makes its block not-a-number in SDM_MX4 (scale 255,
 * codes 0). Bytes between a row's codes or scales and the next row's are set
 * to 0. Slots that no i names keep their contents, and an i whose slot or row is
 * negative, or past its array, stores nothing.
 *
 * Arguments:
 *   codes, scales  the packed bank of packed_dtype: num_slots, head_dim >= 1.
 *   rows           [num_rows, head_dim] of row_dtype (SDM_F32 or SDM_BF16).
 *   n              >= 0; 0 enqueues nothing. n <= num_rows without row_idx,
 *                  n <= num_slots without slots.
 *   row_idx, slots NULL, or [n] of idx_dtype (SDM_I32 or SDM_I64).
 * Precondition (checked under SDM_DEBUG_VALIDATE): one slot is given twice only
 * with the same row (after a decode, say, with row_idx = slots = the slots
 * written, to bring a packed copy up to date).
 * Errors: SDM_E_DTYPE, SDM_E_SHAPE, SDM_E_RANGE, SDM_E_NULL, SDM_E_ALIGN,
 * SDM_E_OVERLAP (rows, codes and scales), SDM_E_HIP.
 */
int sdm_bank_pack(void* codes, void* scales, int packed_dtype, int64_t num_slots, int64_t head_dim,
                  const void* rows, int row_dtype, int64_t num_rows, int64_t n, const void* row_idx,
                  const void* slots, int idx_dtype, void* hip_stream);

/*
 * sdm_gather_packed: per-token weighted sums of a packed bank's rows.
 *
 * Operation, order of summation, padding and preconditions: sdm_gather's without
 * a stash. out_o[t] = sum_n w_o[t,n] value(idx_o[t,n]) with one fused
 * multiply-add chain over n ascending from +0 per element: bit for bit what
 * sdm_gather gives on the float32 bank of the packed rows' values (NaN aside: a
 * NaN is a NaN in both, its payload is not fixed). A width of 1 with weight 1
 * reads rows back as float32.
 * Arguments: as sdm_gather, with codes, scales, packed_dtype for the bank.
 * Errors: as sdm_gather.
 */
int sdm_gather_packed(const void* codes, const void* scales, int packed_dtype, int64_t num_slots, int64_t head_dim,
                      int64_t tokens, int64_t chunk, int64_t valid, const int32_t* chunk_valid, int idx_dtype,
                      int w_dtype, const void* idx0, const void* w0, int32_t width0, float* out0, const void* idx1,
                      const void* w1, int32_t width1, float* out1, void* hip_stream);

/*
 * sdm_gather_weight_grad: gradient of a gather's weights.
 *
 *     dw_o[t,n] = sum_d dout_o[t,d] bank[idx_o[t,n], d]
 * for the gather of the same bank and slots; 0 for a padding token, whose slots
 * and dout are not read. Sums are float32 in an order fixed by the call's
 * sizes, types and alignments, rounded once to w_dtype.
 *
 * Arguments: as sdm_gather (no stash), with
 *   bank        [num_slots, head_dim] of bank_dtype SDM_F32 or SDM_BF16, scales
 *               NULL; or the codes of a packed bank of bank_dtype SDM_MX8 or
 *               SDM_MX4 and its scales.
 *   dout0, dout1  [tokens, head_dim] float32.
 *   dw0, dw1      [tokens, width] of w_dtype, written; must not overlap an input
 *                 or one another.
 * Errors: as sdm_gather.
 */
int sdm_gather_weight_grad(const void* bank, const void* scales, int bank_dtype, int64_t num_slots,
                           int64_t head_dim, int64_t tokens, int64_t chunk, int64_t valid,
                           const int32_t* chunk_valid, int idx_dtype, int w_dtype, const void* idx0,
                           const float* dout0, int32_t width0, void* dw0, const void* idx1, const float* dout1,
                           int32_t width1, void* dw1, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* SDM_MEMORY_H */
