/*
 * moe_topk.h -- C ABI of the top-k mixture-of-experts block for B200 (sm_100a):
 * the router that chooses K experts per token with weights, its gradient, the
 * experts' weighted product and its gradients, and the layer norm in front of
 * them, both directions. It stands beside the top-1 gate of moe_top1.h, in the
 * same library, and shares its status codes, its routing struct and its rules:
 *
 * Pointers.  Every tensor pointer is a DEVICE pointer owned by the caller; the
 *   library never allocates, frees, copies to the host or synchronises. All work
 *   is enqueued in order on `stream` (a cudaStream_t; NULL = legacy default
 *   stream) of the current device, so the calls can be captured in a CUDA graph.
 * Workspace.  Caller-owned device memory, 256-byte aligned, cleared once with
 *   moe_top1_workspace_init; its first 256 bytes hold the flag word that
 *   moe_top1_device_flags reads. Calls that share a workspace must be ordered on
 *   one stream (two graphs that may run at once need a workspace each).
 * Errors.  Arguments are checked on the host before anything is launched; a bad
 *   argument returns a status and enqueues nothing. Device values are trusted:
 *   a routing must be what moe_topk_route wrote for the same tokens.
 * Determinism.  For the same inputs, sizes, alignments and device every output is the
 *   same from run to run, bit for bit: fixed-order sums, no floating-point atomics. The
 *   order itself goes by sizes and alignments, so a token's last bits may differ between
 *   calls of different T, or with arrays that start elsewhere.
 */
#ifndef MOE_TOPK_H
#define MOE_TOPK_H

#include "moe_top1.h"

#ifdef __cplusplus
extern "C" {
#endif

/* 1: layer norm, the router and the experts' weighted product, both directions. */
#define MOE_TOPK_ABI_VERSION 1

/* Element types. */
typedef enum {
    MOE_DTYPE_F32 = 0,
    MOE_DTYPE_BF16 = 1,
    MOE_DTYPE_F16 = 2
} moe_dtype_t;

/* MOE_TOPK_ABI_VERSION of the built library. */
int32_t moe_topk_abi_version(void);

/* How logits become scores. */
typedef enum {
    MOE_SCORE_SOFTMAX = 0, /* softmax over the E experts */
    MOE_SCORE_SIGMOID = 1  /* the logistic function of each logit */
} moe_score_t;

#define MOE_TOPK_RENORM 0x1u /* the K weights of a token are divided by their sum */

/* The rule that chooses experts. */
typedef struct {
    int32_t E;          /* experts, 1 .. 256 */
    int32_t K;          /* experts per token, 1 .. 16, at most E */
    moe_score_t score;
    uint32_t flags;     /* MOE_TOPK_RENORM or 0 */
    float scale;        /* factor of every weight, finite */
    int32_t groups;     /* 1 .. 32, a divisor of E: groups of E / groups neighbouring experts */
    int32_t top_groups; /* groups a token may choose from; top_groups * (E / groups) >= K */
    int32_t group_best; /* 1 or 2, at most E / groups: a group's score is the sum of its best ones */
} moe_topk_rule_t;

/* Bytes of workspace for T tokens, E experts, K experts per token and H channels:
 * enough for moe_topk_route, and with H > 0 for the experts' calls too. 0 for sizes
 * that no call accepts. */
size_t moe_topk_workspace_bytes(int64_t T, int32_t E, int32_t K, int32_t H);

/*
 * Router. For every token t, from logits[t, 0..E) (elements of `dtype`, rows ld >= E
 * elements apart):
 *   s[e] = softmax or logistic function of the logits,   v[e] = s[e] + bias[e]
 *   an expert whose logit is -inf or NaN is masked: v[e] = -inf, behind all others; so is
 *     one whose v is NaN where v is what is compared (with a bias, or sums of a group's two
 *     best), as every softmax score of a row with a NaN or +inf is
 *   with groups: a group's score is the sum of its group_best largest v; the
 *     top_groups groups with the largest scores stay (ties: the lower group)
 *   the K experts with the largest v among those that stay are chosen, largest
 *     first (ties: the lower index)
 *   weights[t, k] = scale * s[e_k], or with MOE_TOPK_RENORM
 *     scale * s[e_k] / sum_j s[e_j]
 * bias [E] (float, finite; NULL: none) takes part in the choice only. Choices are
 * those of exact arithmetic on the given logits and bias, as far as fp64 tells two
 * values apart; without a bias the experts' order is that of the logits themselves.
 * Renormalised weights are ratios of exponentials and do not depend on the scores
 * being representable. Where a token has fewer than K unmasked experts to choose
 * from, masked ones fill up, with the weight of their score (-inf: 0); a row of
 * nothing but -inf gives experts by index with weights 0.
 *
 * out: expert_idx [T * K] (pair p = t * K + k), counts [E] and offsets [E + 1] over
 * pairs, and perm [T * K], the pairs grouped by expert, ascending inside a group.
 * weights [T * K] float. T = 0 zeroes counts and offsets. 0 <= T, T * K < 2^31 - 256.
 * Outputs overlap neither each other nor an input. Needs the workspace.
 */
moe_status_t moe_topk_route(const void* logits, moe_dtype_t dtype, int64_t T, int64_t ld,
                            const moe_topk_rule_t* rule, const float* bias, const moe_routing_t* out,
                            float* weights, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradient of the logits through the weights, the choice held fixed: with
 * g[k] = scale * d_weights[t, k] on the chosen experts,
 *   softmax:               d[e]   = s[e] (g[e] - sum_k s[e_k] g[k]),  g[e] = 0 if e is not chosen
 *   sigmoid:               d[e_k] = g[k] s (1 - s)
 *   renormalised softmax:  d[e_k] = r[k] (g[k] - sum_j r[j] g[j]),   r = s / sum of the chosen s
 *   renormalised sigmoid:  d[e_k] = r[k] (g[k] - sum_j r[j] g[j]) (1 - s[e_k])
 * and 0 for all other experts. d_logits [T, E] is dense, of the logits' type;
 * accumulate = 1 adds to it (a balance loss's gradient, say), 0 overwrites it. The
 * balance bias has no gradient. Experts outside [0, E) in expert_idx are left out.
 * d_logits overlaps no input. No workspace.
 */
moe_status_t moe_topk_route_bwd(const void* logits, moe_dtype_t dtype, int64_t T, int64_t ld,
                                const moe_topk_rule_t* rule, const int32_t* expert_idx,
                                const float* d_weights, void* d_logits, int32_t accumulate, void* stream);

/*
 * The experts' weighted product. With e = expert_idx[t * K + k] and w = weights[t, k],
 *   y[t, o] = sum_k w (sum_i W[e, o, i] x[t, i] + bias[e, o])
 * x, y [T, H], W [E, H, H] (W[e][o][i], y = W x) and bias [E, H] (NULL: none) have
 * elements of `dtype`, MOE_DTYPE_BF16 or MOE_DTYPE_F16, and are dense and 16-byte
 * aligned; weights [T * K] float. routing is what moe_topk_route wrote, all of it from one
 * call: for K = 2 and many tokens expert_idx is read in place of offsets and perm wherever
 * it is given, bias or not (tokens are then grouped by their two experts), else offsets and
 * perm are, and with a bias and K > 1 expert_idx too. It may be NULL where there is no bias
 * or K = 1. Products and sums over i are fp32 on the tensor cores, the K rows of a token are
 * added in fp32, in the order of k (grouped: the lower expert first), and the result is
 * rounded once.
 * 1 <= E <= 256, 1 <= K <= min(16, E), H a multiple of 64 with 64 <= H <= 4096,
 * 0 <= T * K < 2^31 - 256. y overlaps no input. Needs the workspace.
 */
moe_status_t moe_topk_fwd(const void* x, const void* W, const void* bias, moe_dtype_t dtype,
                          const moe_routing_t* routing, const float* weights, int64_t T, int32_t E,
                          int32_t K, int32_t H, void* y, void* workspace, size_t workspace_bytes,
                          void* stream);

/*
 * Its gradients, from the output's gradient d_out [T, H]:
 *   d_x[t, i]       = sum_k w sum_o W[e, o, i] d_out[t, o]
 *   dW[e, o, i]     = sum of w d_out[t, o] x[t, i] over the pairs (t, k) of expert e
 *   db[e, o]        = sum of w d_out[t, o] over them
 *   d_weights[t, k] = sum_o d_out[t, o] (sum_i W[e, o, i] x[t, i] + bias[e, o])
 * d_x, dW and db have elements of `dtype`, d_weights [T * K] is float. Any of them may
 * be NULL to skip it; an expert without pairs gets zeros in dW and db. d_weights comes
 * from fp32 sums throughout; d_x rounds as y does above; for dW every w d_out enters the
 * tensor cores as two numbers of `dtype` that add up to it (its upper 16 bits for bf16, 22
 * for fp16, whatever its size; fp32 sums, one rounding at the end), for db it is fp32.
 * Sums over tokens have a fixed order. bias is read for d_weights only; routing as above,
 * and expert_idx may be NULL unless d_weights and a bias are given.
 * Outputs overlap neither each other nor an input. Needs the workspace.
 */
moe_status_t moe_topk_bwd(const void* x, const void* W, const void* bias, moe_dtype_t dtype,
                          const void* d_out, const moe_routing_t* routing, const float* weights,
                          int64_t T, int32_t E, int32_t K, int32_t H, void* d_x, void* dW, void* db,
                          float* d_weights, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Layer norm over the last axis of x [T, H]:
 *   mean[t] = (1/H) sum_h x[t, h]
 *   rstd[t] = 1 / sqrt((1/H) sum_h (x[t, h] - mean[t])^2 + eps)
 *   y[t, h] = (x[t, h] - mean[t]) * rstd[t] * gamma[h] + beta[h]
 * x has elements of `dtype`, rows ldx >= H elements apart; y [T, H] has the same
 * type and is dense. gamma and beta [H] have elements of `param_dtype`, which is
 * `dtype` or MOE_DTYPE_F32; NULL stands for ones and zeros. mean and rstd [T]
 * (float) are kept for the backward; both may be NULL. Sums and statistics are
 * fp32, the squared deviations are taken from the mean already known; y is
 * rounded once. y may be x itself (dense) and must not overlap anything else.
 * 0 <= T < 2^31 - 256, 1 <= H <= 8192, eps finite and >= 0. A row of equal values
 * with eps = 0 has rstd = inf and y = NaN, as the formula says.
 */
moe_status_t moe_layer_norm_fwd(const void* x, moe_dtype_t dtype, int64_t T, int32_t H, int64_t ldx,
                                const void* gamma, const void* beta, moe_dtype_t param_dtype, float eps,
                                void* y, float* mean, float* rstd, void* stream);

/* Bytes of workspace moe_layer_norm_bwd needs. */
size_t moe_layer_norm_workspace_bytes(int64_t T, int32_t H);

/*
 * Its gradients, from x, the output's gradient dy [T, H] and the forward's mean
 * and rstd. With n = (x - mean) * rstd and u = dy * gamma:
 *   dx[t, h]  = rstd[t] * (u[t, h] - (1/H) sum_j u[t, j] - n[t, h] * (1/H) sum_j u[t, j] n[t, j])
 *   dgamma[h] = sum_t dy[t, h] n[t, h],     dbeta[h] = sum_t dy[t, h]
 * dy and dx are dense, of x's type; dgamma and dbeta [H] have gamma's type
 * (`param_dtype`); gamma may be NULL (ones). Any of dx, dgamma, dbeta may be NULL
 * to skip it. The sums over tokens are fp32 in a fixed order, rounded once.
 * Outputs are overwritten; T = 0 writes zeros to dgamma and dbeta. dx may be dy
 * itself; otherwise outputs overlap neither each other nor an input. The
 * workspace is needed for dgamma and dbeta only.
 */
moe_status_t moe_layer_norm_bwd(const void* x, const void* dy, moe_dtype_t dtype, int64_t T, int32_t H,
                                int64_t ldx, const void* gamma, moe_dtype_t param_dtype, const float* mean,
                                const float* rstd, void* dx, void* dgamma, void* dbeta, void* workspace,
                                size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_TOPK_H */
