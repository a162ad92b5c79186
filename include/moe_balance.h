/* Balance loss of the router with per-expert counts, and the gradient of the
 * router's logits, for MI355X (gfx950).
 *
 * Definitions (t token, e expert, j pick, b sequence; s as in moe_route_sort.h):
 *   s[t,e]     = sigmoid(logits[t,e]),  p[t,e] = s[t,e] / sum_e s[t,e]
 *                (p[t] = 0 where every logit of the row is -infinity)
 *   sequences  tokens [seq_offsets[b], seq_offsets[b+1]) for b < B, or one
 *              sequence of all M tokens (seq_offsets NULL, B = 1)
 *   mask       a token with mask[t] == 0 is padding: its logits, ids and
 *              gradients are never used and its gradient is zero
 *   tokens[b]  = unmasked tokens of b (n_b);  tokens[B] = sequences with n_b > 0 (B')
 *   counts[b,e] = routes ids[t,j] == e of b's unmasked tokens; an id outside
 *              [0, E) is a dropped route and counts nowhere
 *   shares[b,e] = (1 / n_b) * sum of p[t,e] over b's unmasked tokens (0 if n_b == 0)
 *   loss       = coef / B' * sum_b E / (k n_b) * sum_e counts[b,e] * shares[b,e]
 *              over the sequences with n_b > 0 (0 if there is none)
 * A row whose scores all underflow is normalised from logits shifted by their
 * maximum, so p sums to 1 for every row with a logit above -infinity.  A NaN in
 * an unmasked row reaches the shares and the loss, and that row's gradient.
 */
#ifndef MOE_BALANCE_H_
#define MOE_BALANCE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Workspace bytes of moe_balance_loss; (size_t)-1 for invalid sizes. */
size_t moe_balance_workspace_bytes(int M, int E, int k, int B);

/*
 * moe_balance_loss
 *   logits       [M, E] row-major FP32 or BF16 (MRS_DTYPE_F32 / MRS_DTYPE_BF16)
 *   ids          [M, k] int32
 *   seq_offsets  NULL (B must be 1), or int32[B + 1] on the device,
 *                nondecreasing from 0 to M (read on the device; other values
 *                are clamped to [0, M] and give unspecified results)
 *   mask         NULL (every token counts) or uint8[M]
 *   0 <= M <= 2^30, 1 <= E <= 4096, 1 <= k <= 64, M k < 2^31, 1 <= B <= 65535
 *                (MRS_ERR_OVERFLOW for more tokens or routes)
 *   loss float[1], counts int32[B, E], tokens int32[B + 1], shares float[B, E] (written)
 *   workspace    device scratch of moe_balance_workspace_bytes() bytes, 16-byte
 *                aligned; never cleared between calls; calls that may overlap in
 *                time need distinct workspaces
 * The sums run in a fixed order: equal inputs give equal bits.  Asynchronous on
 * `stream`; one to three launches; allocates nothing.  Returns MRS_OK or a negative
 * MRS_ERR_* code before any launch.
 */
int moe_balance_loss(const void* logits, int logits_dtype, const int32_t* ids, const int32_t* seq_offsets,
                     const uint8_t* mask, int M, int E, int k, int B, float coef, float* loss, int32_t* counts,
                     int32_t* tokens, float* shares, void* workspace, size_t workspace_bytes, void* stream);

/*
 * moe_route_far_weights -- the routing weights of tokens so far off that FP32
 * scores cannot hold them, in place of those of moe_route_sort.
 *
 * For each token t whose kept picks' logits (ids[t,j] in [0, E)) all lie below
 * -87, where the scores are subnormal or zero and their FP32 quotient is coarse,
 * infinite or NaN:
 *     weights[t,j] = exp(x_j - max_i x_i) / sum_i exp(x_i - max_i x_i),
 *                    x_j = logits[t, ids[t,j]]
 * which is the limit that moe_router_backward differentiates: 0 for a dropped
 * pick, 0 for all where every pick is -infinity, NaN for all where one is NaN (a
 * NaN does not count as a logit of -87 or more).  Other tokens' weights are not
 * written.
 *   logits, logits_dtype, ids, M, E, k   as for moe_balance_loss
 *   weights      float[M, k], as moe_route_sort wrote them
 * Asynchronous on `stream`; one launch (none for M == 0); allocates nothing.
 */
int moe_route_far_weights(const void* logits, int logits_dtype, const int32_t* ids, int M, int E, int k,
                          float* weights, void* stream);

/*
 * moe_router_backward -- grad_logits = d(total) / d(logits), where total has
 *   grad_loss as its derivative by the balance loss (counts are constants), and
 *   grad_w[t, j] as its derivative by the routing weights
 *     w[t, j] = s[t, ids[t,j]] / sum_i s[t, ids[t,i]]   (dropped routes left out)
 *
 *   grad_w       NULL (no such term) or float[M, k]
 *   counts       NULL (no balance term) or int32[B, E], with tokens int32[B + 1],
 *                both as written by moe_balance_loss for the same arguments
 *   grad_loss    NULL (taken as 1) or one float on the device
 *   grad_logits  [M, E] of the logits' type (written, every row), computed in
 *                FP32 and rounded once
 *   other arguments as for moe_balance_loss; coef is that of the loss
 * Asynchronous on `stream`; one launch; needs no workspace and allocates nothing.
 */
int moe_router_backward(const void* logits, int logits_dtype, const int32_t* ids, const float* grad_w,
                        const int32_t* counts, const int32_t* tokens, const float* grad_loss,
                        const int32_t* seq_offsets, const uint8_t* mask, int M, int E, int k, int B, float coef,
                        void* grad_logits, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BALANCE_H_ */
