// topk.h -- host-side declarations shared by the files of the top-k block.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "moe_topk.h"

namespace moe {

inline bool dtype_ok(moe_dtype_t d) { return d == MOE_DTYPE_F32 || d == MOE_DTYPE_BF16 || d == MOE_DTYPE_F16; }
inline size_t dtype_bytes(moe_dtype_t d) { return d == MOE_DTYPE_F32 ? 4 : 2; }

// SMs of the current device.
cudaError_t device_sms(int* out);

// The dynamic shared-memory limit of a kernel, set once per device: `done` is a bit per
// device, a static of the caller's.
cudaError_t set_smem_once(const void* kernel, int bytes, std::atomic<uint64_t>& done);

// Workspace of the router: the reserved head, then per-block counts and bases.
size_t topk_route_ws_bytes(int64_t T, int E);
// The same with the experts' areas behind it, for sizes the experts' calls accept.
size_t topk_experts_ws_bytes(int64_t T, int E, int K, int H);
bool topk_experts_sizes_ok(int64_t T, int E, int K, int H);

}  // namespace moe
