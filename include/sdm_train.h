/*
 * libsdm: training a router and a bank on an AMD Instinct MI355X (gfx950). Part of
 * libsdm, with the conventions of sdm.h and sdm_memory.h: every pointer of a compute
 * call is a device pointer to a contiguous, row-major array that the caller owns, the
 * library allocates nothing and keeps no state, work is only enqueued on `hip_stream`
 * (so calls may be captured in a HIP graph, and calls on several streams may run at
 * once), the cheap argument checks run on the host before any HIP call, and a failing
 * call enqueues nothing and returns a status code of sdm.h with a message for
 * sdm_last_error().
 *
 *   sdm_route_balance            how often a route chose each key, and the loss that
 *                                keeps the choice even
 *   sdm_route_balance_backward   that loss's gradient -> gradient of the scores
 *   sdm_lookup                   scaled rows of a bank (an embedding), with dropout
 *   sdm_lookup_grad              gradient of a lookup -> gradient of the bank
 *   sdm_gather_bank_grad         gradient of a gather's sums -> gradient of the bank
 *
 * Workspaces. Three of the calls take scratch memory of the caller: `workspace`,
 * 16-byte aligned, of at least the bytes that the call's size function gives. What it
 * holds before does not matter, and nothing in it is meant to be read afterwards. It is
 * in use until the call's work is done: calls (and replays of captured calls) that may
 * run at once need one each.
 */
#ifndef SDM_TRAIN_H
#define SDM_TRAIN_H

#include <stdint.h>

#include "sdm_memory.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SDM_MAX_GRAD_ENTRIES 0x7fffffffLL /* most entries, and most slots, of a gradient to a bank */
#define SDM_MAX_LOOKUP_ROWS 0x7fffffffLL  /* most rows of a lookup */
/* Lookups and gradients to a bank take rows of at most 65535 * 256 columns. */

/* What a gradient to a bank does with dbank. */
enum {
    SDM_GRAD_WRITE = 0, /* dbank is written whole, rows of slots that no entry names with 0 */
    SDM_GRAD_ADD = 1    /* rows of slots that some entry names are added to, others not touched */
};

/*
 * sdm_route_balance: how evenly a route uses its keys.
 *
 * Tokens, their keys and scores as in sdm_route; token t is live when t mod chunk <
 * valid (chunk_valid given: < chunk_valid[t / chunk]), as in sdm_gather. The tokens
 * form sequences: each chunk is one (per_chunk), or all tokens together are. With n_g
 * the live tokens of sequence g, G the number of sequences that have any, s_t the
 * scores of token t (softmax, or sigmoid; NaN and -inf logits have score 0, +inf counts
 * as the largest float32) and
 *     p_ti = s_ti / sum_i s_ti         (0 in a row whose logits are all NaN or -inf)
 * (a score below 2^-126 may count as 0; where a row's largest logit is at most -64, its
 * sigmoid scores are taken relative to the largest, so that this goes by their quotient)
 * the results are
 *     counts_gi = number of (t, j), t live in g, with idx_tj key i of token t
 *     mean_gi   = sum_{t live in g} p_ti / n_g                       (0 where n_g = 0)
 *     coef_g    = scale keys / (k n_g^2 G)                           (0 where n_g = 0)
 *     loss      = sum_g coef_g sum_i counts_gi sum_{t live in g} p_ti
 * so that the loss is `scale` where every key is chosen equally often, and coef_g
 * counts_gi is its derivative by p_ti (the counts have none).
 *
 * Arguments: logits, tokens, keys, k, score, streams, stream_slots and idx as
 * sdm_route's (idx [tokens, k]; a slot that is not one of its token's keys is not
 * counted), and
 *   chunk       >= 1, a divisor of tokens; valid 0..chunk, or chunk_valid NULL or
 *               [tokens / chunk] int32 (counted as if clamped to 0..chunk).
 *   scale       finite.
 *   counts      [sequences, keys] int32; mean [sequences, keys], coef [sequences] and
 *               loss [1] float32; all written. sequences = per_chunk ? tokens / chunk
 *               : 1; without tokens there is nothing to write but loss = 0 and, of the
 *               one sequence of a call without per_chunk, zeros.
 *   workspace   of sdm_route_balance_workspace() bytes.
 * p is float32, its row's sum of float32 terms; sums over up to 255 tokens are float32,
 * those over all tokens and keys float64; every sum is taken in an order fixed by the
 * call's sizes.
 * Errors: SDM_E_DTYPE, SDM_E_SHAPE, SDM_E_RANGE, SDM_E_NULL, SDM_E_ALIGN,
 * SDM_E_OVERLAP, SDM_E_HIP.
 */
int sdm_route_balance(const void* logits, int logit_dtype, int64_t tokens, int64_t keys, int32_t k, int score,
                      int64_t chunk, int64_t valid, const int32_t* chunk_valid, int32_t per_chunk, float scale,
                      int64_t streams, int64_t stream_slots, const void* idx, int idx_dtype, int32_t* counts,
                      float* mean, float* coef, float* loss, void* workspace, int64_t workspace_bytes,
                      void* hip_stream);

/* Bytes of sdm_route_balance's workspace; 0 for sizes that the call refuses. */
int64_t sdm_route_balance_workspace(int64_t tokens, int64_t keys, int64_t chunk, int32_t per_chunk);

/*
 * sdm_route_balance_backward: gradient of sdm_route_balance's loss with respect to
 * its logits.
 *
 * With counts and coef as sdm_route_balance gave them, f_i = dloss coef_g counts_gi and
 *     softmax:  d_ti = p_ti (f_i - sum_j f_j p_tj)
 *     sigmoid:  d_ti = p_ti (1 - s_ti) (f_i - sum_j f_j p_tj)
 * for a live token t of sequence g; 0 for the others, and for keys whose score is 0.
 *     dlogits = d,  or dlogits + d (accumulate)
 * Counts are taken relative to their mean, or in a row where one key has more than 4/5 of
 * the share to that key's count (p sums to 1, so that a constant changes nothing): there
 * nothing cancels, however far that key is above the rest. A row's gradient depends on no
 * other row. A count's difference to the mean is rounded to float32, exact below 2^24, and a
 * difference to a key's count is that of two of those; the rest is float32, and the sum is
 * rounded once to the logits' type.
 *
 * Arguments: as sdm_route_balance, with
 *   counts, coef  [sequences, keys] and [sequences].
 *   dloss         NULL (1), or [1] float32.
 *   dlogits       [tokens, keys] of logit_dtype: written whole, or (accumulate) rows of
 *                 live tokens added to and the others not touched. Must not overlap an
 *                 input.
 * Errors: as sdm_route_balance.
 */
int sdm_route_balance_backward(const void* logits, int logit_dtype, int64_t tokens, int64_t keys, int score,
                               int64_t chunk, int64_t valid, const int32_t* chunk_valid, int32_t per_chunk,
                               const int32_t* counts, const float* coef, const float* dloss, int32_t accumulate,
                               void* dlogits, void* hip_stream);

/*
 * sdm_lookup: scaled rows of a bank, with dropout.
 *
 * With T = dropout * 2^16 rounded to the nearest whole number (ties to even) and
 * a = scale * 2^16 / (2^16 - T), rounded to float32:
 *     out_ic = a * value(idx_i, c)   where column c of row i stays, else 0
 * rounded to float32 and then to out_dtype. A row whose idx lies outside the bank is 0.
 * Without dropout (T = 0) all columns stay; otherwise column c stays when its 16 random
 * bits, as a number, are at least T. Those bits are half c mod 2 (0: the low one) of
 * word (c mod 8) / 2 of Philox4x32-10 (Salmon, Moraes, Dror, Shaw: Parallel random
 * numbers: as easy as 1, 2, 3; 2011) with
 *     key      seed mod 2^32, seed / 2^32
 *     counter  c / 8, i, offset mod 2^32, offset / 2^32
 * of seed = rng[0] and offset = rng[1]: the mask is a function of these and of (i, c)
 * alone, and is not stored. Another step, layer or device takes another offset.
 *
 * Arguments:
 *   bank        [num_slots, head_dim] of bank_dtype SDM_F32 or SDM_BF16, scales NULL;
 *               or the codes of a packed bank of bank_dtype SDM_MX8 or SDM_MX4 and its
 *               scales (sdm_memory.h).
 *   n           0..SDM_MAX_LOOKUP_ROWS, and at most 2^28 * max(1, 256 / ceil(head_dim / 8)), the
 *               quotient rounded down; 0 enqueues nothing.
 *   idx         [n] of idx_dtype SDM_I32 or SDM_I64: any values.
 *   scale       finite, and so that a is finite. dropout in [0, 1 - 2^-16].
 *   rng         [2] uint64 in device memory (so that a captured call can be replayed
 *               with others); may be NULL where T = 0.
 *   out         [n, head_dim] of out_dtype SDM_F32 or SDM_BF16, written.
 * Errors: as sdm_route_balance.
 */
int sdm_lookup(const void* bank, const void* scales, int bank_dtype, int64_t num_slots, int64_t head_dim, int64_t n,
               const void* idx, int idx_dtype, float scale, float dropout, const uint64_t* rng, void* out, int out_dtype,
               void* hip_stream);

/*
 * sdm_lookup_grad: gradient of a lookup with respect to its bank.
 *
 *     dbank_s = a sum_{i : idx_i = s} m_i dout_i      (or dbank_s + that: SDM_GRAD_ADD)
 * with a, and m the mask of columns that stay, as in sdm_lookup of the same idx, scale,
 * dropout and rng. Rows whose idx lies outside the bank add nothing, and their dout is not
 * read; neither is a dropped column's dout ever counted, whatever it holds. Sums are
 * float32, over at most 48 rows of a slot in ascending order. Where a slot has more, such sums
 * are added in float32 in their order, of which there are at most 17 then, or, always where
 * there are more, in float64 and rounded to float32. All of this is fixed by the call's sizes
 * and idx: the same inputs give the same bits. The result is rounded once to bank_dtype.
 *
 * Arguments: as sdm_lookup, with
 *   n           0..SDM_MAX_GRAD_ENTRIES (0: dbank is zeroed, or left).
 *   num_slots   1..SDM_MAX_GRAD_ENTRIES.
 *   dout        [n, head_dim] of dout_dtype SDM_F32 or SDM_BF16.
 *   dbank       [num_slots, head_dim] of bank_dtype SDM_F32 or SDM_BF16; mode one of
 *               SDM_GRAD_*. Must not overlap an input.
 *               (SDM_GRAD_WRITE into more than 2^38 - 2^17 bytes may be refused.)
 *   workspace   of sdm_bank_grad_workspace(n, num_slots, head_dim) bytes.
 * Errors: as sdm_route_balance.
 */
int sdm_lookup_grad(int64_t n, const void* idx, int idx_dtype, const void* dout, int dout_dtype, float scale,
                    float dropout, const uint64_t* rng, void* dbank, int bank_dtype, int64_t num_slots,
                    int64_t head_dim, int mode, void* workspace, int64_t workspace_bytes, void* hip_stream);

/*
 * sdm_gather_bank_grad: gradient of a gather's outputs with respect to its bank.
 *
 *     dbank_s = sum_{(o, t, n) : idx_o[t,n] = s} w_o[t,n] dout_o[t]    (or dbank_s + that)
 * over the live tokens t of sdm_gather (or sdm_gather_packed's values) with the same slots
 * and weights; padding tokens' slots and weights may hold anything, their dout is not read. Sums are float32,
 * fused multiply-adds over the entries of a slot in ascending order (o, t, n), put together
 * as in sdm_lookup_grad; the result is rounded once to bank_dtype.
 *
 * Arguments: tokens, chunk, valid, chunk_valid, idx and w as sdm_gather's (a slot outside
 * the bank adds nothing), with tokens * (width0 + width1) <= SDM_MAX_GRAD_ENTRIES and
 *   dout0, dout1  [tokens, head_dim] float32.
 *   dbank, num_slots, head_dim, mode  as sdm_lookup_grad's.
 *   workspace     of sdm_bank_grad_workspace(tokens * (width0 + width1), num_slots,
 *                 head_dim) bytes.
 * Errors: as sdm_route_balance.
 */
int sdm_gather_bank_grad(int64_t tokens, int64_t chunk, int64_t valid, const int32_t* chunk_valid, int idx_dtype,
                         int w_dtype, const void* idx0, const void* w0, const float* dout0, int32_t width0,
                         const void* idx1, const void* w1, const float* dout1, int32_t width1, void* dbank,
                         int bank_dtype, int64_t num_slots, int64_t head_dim, int mode, void* workspace,
                         int64_t workspace_bytes, void* hip_stream);

/*
 * Bytes of the workspace of a gradient to a bank: at most 27 an entry, and 1 GiB or 16 an
 * entry, whichever is more, for sums of runs, and a MiB. 0 where one of the three is outside
 * its range.
 */
int64_t sdm_bank_grad_workspace(int64_t entries, int64_t num_slots, int64_t head_dim);

#ifdef __cplusplus
}
#endif

#endif /* SDM_TRAIN_H */
