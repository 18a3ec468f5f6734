// topk_api.cu -- what the files of the top-k block (include/moe_topk.h) share: the
// ABI version and the facts about the current device.
#include <mutex>

#include "checks.h"
#include "topk.h"

namespace moe {
namespace {

constexpr int kMaxDevices = 64;
int g_sms[kMaxDevices];
std::mutex g_mu;

}  // namespace

cudaError_t device_sms(int* out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(g_mu);
    if (g_sms[dev] == 0) {
        e = cudaDeviceGetAttribute(&g_sms[dev], cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
    }
    *out = g_sms[dev];
    return cudaSuccess;
}

cudaError_t set_smem_once(const void* kernel, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    const uint64_t bit = uint64_t{1} << dev;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

}  // namespace moe

extern "C" int32_t moe_topk_abi_version(void) { return MOE_TOPK_ABI_VERSION; }

extern "C" size_t moe_topk_workspace_bytes(int64_t T, int32_t E, int32_t K, int32_t H) {
    using namespace moe;
    if (T < 0 || E < 1 || E > 256 || K < 1 || K > 16 || K > E || T >= kMaxT / K || H < 0) return 0;
    if (H == 0) return topk_route_ws_bytes(T, E);
    return topk_experts_sizes_ok(T, E, K, H) ? topk_experts_ws_bytes(T, E, K, H) : 0;
}
