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
 * Determinism.  For the same inputs and device every output is the same from run
 *   to run, bit for bit: fixed-order sums, no floating-point atomics.
 */
#ifndef MOE_TOPK_H
#define MOE_TOPK_H

#include "moe_top1.h"

#ifdef __cplusplus
extern "C" {
#endif

/* 1: layer norm, both directions. */
#define MOE_TOPK_ABI_VERSION 1

/* Element types. */
typedef enum {
    MOE_DTYPE_F32 = 0,
    MOE_DTYPE_BF16 = 1,
    MOE_DTYPE_F16 = 2
} moe_dtype_t;

/* MOE_TOPK_ABI_VERSION of the built library. */
int32_t moe_topk_abi_version(void);

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
