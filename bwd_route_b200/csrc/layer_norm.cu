// layer_norm.cu -- layer norm over the last axis, forward and backward.
//
//   y  = (x - mean) rstd gamma + beta,   rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//   dx = rstd (u - mean(u) - n mean(u n)),   u = dy gamma,  n = (x - mean) rstd
//   dgamma = sum_t dy n,   dbeta = sum_t dy
//
// Bound: HBM. Both directions are one pass: a row is read once into registers, its
// sums are taken from there, and the result is written from there. A row belongs to 4 to
// 512 threads (values_per_thread); the block's other threads have rows of their own, and
// the block walks over the rows with the next row's loads in flight, so gamma, beta and
// (backward) the thread's column sums stay in registers. Loads are 16 bytes wide where every
// row starts on 16, else two values, else one. 1,048,576 x 256 fp32 forward: 335 to 368 us,
// 5.8 to 6.4 TB/s (a copy: 6.55). 262,144 x 256 fp32 backward: 120 to 132 us, 6.1 TB/s or more, and 3 to 4 us for the
// second kernel. One row of 1024 bf16: 2.9 us on the device. 524,288 x 16 fp16 forward, a
// row for every four threads: 17 us (a warp for a row: 111).
//
// dgamma and dbeta: a thread always sees the same columns, so it adds up its rows in
// registers; every kFlush rows it adds that to its shared-memory sums (so an fp32 chain grows
// by one addition per 64 rows of a team, a few hundred for as many rows as memory holds), the
// block's row teams are added in order, and a second kernel adds the blocks in order. No atomics: the same bits from run to run.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "checks.h"
#include "common.cuh"
#include "elem.cuh"
#include "internal.h"
#include "moe_topk.h"
#include "topk.h"

namespace moe {
namespace {

constexpr int kMaxH = 8192;
constexpr int kPerThread = 16;    // values of a row a thread holds at most
constexpr int kFlush = 64;        // rows between two flushes of the column sums
constexpr int kMaxBlocks = 1024;  // partial-sum rows the workspace holds

// Sum over the tpr threads of a row; every thread of the block calls it.
template <int V>
__device__ __forceinline__ void team_sum(float (&v)[V], float (*red)[16], int tpr) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        if (off >= tpr) continue;
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
    }
    if (tpr <= 32) return;
    const int warp = threadIdx.x >> 5, wpr = tpr >> 5;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < V; ++i) red[i][warp] = v[i];
    __syncthreads();
    const int w0 = warp & ~(wpr - 1);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float s = 0.0f;
        for (int w = 0; w < wpr; ++w) s += red[i][w0 + w];
        v[i] = s;
    }
}

// The N * VEC parameters of this thread's columns (1 or 0 where there is no array).
template <typename P, int VEC, int N>
__device__ __forceinline__ void load_params(const P* p, float none, int tpr, int r, int H, float (&out)[N * VEC]) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int c = (j * tpr + r) * VEC;
        Chunk<P, VEC> v;
        const bool on = p && c < H;
        if (on) v = *reinterpret_cast<const Chunk<P, VEC>*>(p + c);
#pragma unroll
        for (int i = 0; i < VEC; ++i) out[j * VEC + i] = on ? to_f(v.v[i]) : none;
    }
}

template <typename T, int VEC, int N>
__device__ __forceinline__ void load_row(const T* row, int tpr, int r, int H, bool valid, Chunk<T, VEC> (&v)[N]) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int c = (j * tpr + r) * VEC;
        if (valid && c < H) v[j] = *reinterpret_cast<const Chunk<T, VEC>*>(row + c);
    }
}

template <typename T, typename P, int VEC, int N, int BLOCK>
__global__ void __launch_bounds__(BLOCK)
norm_fwd_kernel(const T* x, int64_t ldx, const P* __restrict__ gamma, const P* __restrict__ beta, float eps, T* y,
                float* __restrict__ mean, float* __restrict__ rstd, int64_t T_, int H, int tpr_) {
    griddep_wait();  // every global access below comes after the previous grid
    __shared__ float s_red[2][1][16];
    const int tpr = BLOCK == 512 ? 512 : tpr_;
    const int team = threadIdx.x / tpr, r = threadIdx.x % tpr, teams = BLOCK / tpr;
    const float h = static_cast<float>(H);
    float g[N * VEC], b[N * VEC];
    load_params<P, VEC, N>(gamma, 1.0f, tpr, r, H, g);
    load_params<P, VEC, N>(beta, 0.0f, tpr, r, H, b);
    const int64_t step = static_cast<int64_t>(gridDim.x) * teams;
    int64_t row = static_cast<int64_t>(blockIdx.x) * teams + team;
    Chunk<T, VEC> next[N];
    load_row<T, VEC, N>(x + row * ldx, tpr, r, H, row < T_, next);
    for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * teams; row0 < T_; row0 += step, row += step) {
        const bool valid = row < T_;
        float v[N * VEC];
        float s[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const bool on = valid && (j * tpr + r) * VEC < H;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                v[j * VEC + i] = on ? to_f(next[j].v[i]) : 0.0f;
                s[0] += v[j * VEC + i];
            }
        }
        load_row<T, VEC, N>(x + (row + step) * ldx, tpr, r, H, row + step < T_, next);
        team_sum(s, s_red[0], tpr);
        const float mu = s[0] / h;
        s[0] = 0.0f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const bool on = (j * tpr + r) * VEC < H;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                v[j * VEC + i] -= mu;
                if (on) s[0] += v[j * VEC + i] * v[j * VEC + i];
            }
        }
        team_sum(s, s_red[1], tpr);
        const float rs = rsqrtf(s[0] / h + eps);
        if (!valid) continue;
        T* out = y + row * H;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int c = (j * tpr + r) * VEC;
            Chunk<T, VEC> o;
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                o.v[i] = from_f<T>(v[j * VEC + i] * rs * g[j * VEC + i] + b[j * VEC + i]);
            if (c < H) *reinterpret_cast<Chunk<T, VEC>*>(out + c) = o;
        }
        if (r == 0) {
            if (mean) mean[row] = mu;
            if (rstd) rstd[row] = rs;
        }
    }
}

// part: [gridDim.x][2][H] column sums of the block's rows (dgamma, dbeta), or NULL.
// One row team's chain (loads, two sums over the team, stores) is long where H is odd and
// values come one by one; two or four rows a team at once were slower: fewer teams run.
template <typename T, typename P, int VEC, int N, int BLOCK>
__global__ void __launch_bounds__(BLOCK)
norm_bwd_kernel(const T* __restrict__ x, const T* dy, int64_t ldx, const P* __restrict__ gamma,
                const float* __restrict__ mean, const float* __restrict__ rstd, T* dx, float* __restrict__ part,
                int64_t T_, int H, int tpr_) {
    griddep_wait();  // every global access below comes after the previous grid
    extern __shared__ float s_sum[];  // [2][N * VEC][BLOCK], each thread its own
    __shared__ float s_red[2][2][16];
    const int tpr = BLOCK == 512 ? 512 : tpr_;
    const int team = threadIdx.x / tpr, r = threadIdx.x % tpr, teams = BLOCK / tpr;
    const float inv_h = 1.0f / static_cast<float>(H);
    constexpr int EPT = N * VEC;
    float g[EPT], ag[EPT], ab[EPT];
    load_params<P, VEC, N>(gamma, 1.0f, tpr, r, H, g);
#pragma unroll
    for (int k = 0; k < EPT; ++k) ag[k] = ab[k] = 0.0f;
    if (part)
#pragma unroll
        for (int k = 0; k < 2 * EPT; ++k) s_sum[k * BLOCK + threadIdx.x] = 0.0f;
    const int64_t step = static_cast<int64_t>(gridDim.x) * teams;
    int64_t row = static_cast<int64_t>(blockIdx.x) * teams + team;
    Chunk<T, VEC> nx[N], ny[N];
    float nmu = 0.0f, nrs = 0.0f;
    auto fetch = [&](int64_t rw) {
        const bool on = rw < T_;
        load_row<T, VEC, N>(x + rw * ldx, tpr, r, H, on, nx);
        load_row<T, VEC, N>(dy + rw * H, tpr, r, H, on, ny);
        nmu = on ? mean[rw] : 0.0f;
        nrs = on ? rstd[rw] : 0.0f;
    };
    fetch(row);
    int since = 0, phase = 0;
    for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * teams; row0 < T_; row0 += step, row += step) {
        const bool valid = row < T_;
        float n[EPT], u[EPT];
        float s[2] = {0.0f, 0.0f};
        const float mu = nmu, rs = nrs;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const bool on = valid && (j * tpr + r) * VEC < H;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int k = j * VEC + i;
                const float d = on ? to_f(ny[j].v[i]) : 0.0f;
                n[k] = on ? (to_f(nx[j].v[i]) - mu) * rs : 0.0f;
                ag[k] += d * n[k];
                ab[k] += d;
                u[k] = d * g[k];
                s[0] += u[k];
                s[1] += u[k] * n[k];
            }
        }
        fetch(row + step);
        if (dx) {
            team_sum(s, s_red[phase], tpr);
            phase ^= 1;
            const float c1 = s[0] * inv_h, c2 = s[1] * inv_h;
            if (valid) {
                T* out = dx + row * H;
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const int c = (j * tpr + r) * VEC;
                    Chunk<T, VEC> o;
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const int k = j * VEC + i;
                        o.v[i] = from_f<T>(rs * (u[k] - c1 - n[k] * c2));
                    }
                    if (c < H) *reinterpret_cast<Chunk<T, VEC>*>(out + c) = o;
                }
            }
        }
        if (part && ++since == kFlush) {
            since = 0;
#pragma unroll
            for (int k = 0; k < EPT; ++k) {
                s_sum[k * BLOCK + threadIdx.x] += ag[k];
                s_sum[(EPT + k) * BLOCK + threadIdx.x] += ab[k];
                ag[k] = ab[k] = 0.0f;
            }
        }
    }
    if (!part) return;
#pragma unroll
    for (int k = 0; k < EPT; ++k) {
        s_sum[k * BLOCK + threadIdx.x] += ag[k];
        s_sum[(EPT + k) * BLOCK + threadIdx.x] += ab[k];
    }
    __syncthreads();
    // the row teams in order; column of (k, r): chunk k / VEC, element k % VEC
    for (int i = threadIdx.x; i < EPT * tpr; i += BLOCK) {
        const int k = i / tpr, rr = i % tpr;
        const int c = ((k / VEC) * tpr + rr) * VEC + k % VEC;
        if (c >= H) continue;
        float a = 0.0f, b = 0.0f;
        for (int t = 0; t < teams; ++t) {
            a += s_sum[k * BLOCK + t * tpr + rr];
            b += s_sum[(EPT + k) * BLOCK + t * tpr + rr];
        }
        part[(static_cast<int64_t>(blockIdx.x) * 2) * H + c] = a;
        part[(static_cast<int64_t>(blockIdx.x) * 2 + 1) * H + c] = b;
    }
}

// Adds the blocks' column sums: 32 columns a block, 32 runs of blocks each, then the
// runs in order. blockIdx.y: 0 dgamma, 1 dbeta.
template <typename P>
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float* __restrict__ part, int nblk, int H,
                                                           P* __restrict__ dgamma, P* __restrict__ dbeta) {
    griddep_wait();  // every global access below comes after the previous grid
    __shared__ float s[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x, q = threadIdx.y;
    P* out = blockIdx.y ? dbeta : dgamma;
    if (!out) return;
    float a = 0.0f;
    if (c < H) {
#pragma unroll 8
        for (int b = q; b < nblk; b += 32) a += part[(static_cast<int64_t>(b) * 2 + blockIdx.y) * H + c];
    }
    s[q][threadIdx.x] = a;
    __syncthreads();
    if (q == 0 && c < H) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) sum += s[i][threadIdx.x];
        out[c] = from_f<P>(sum);
    }
}

// Threads per row: the fewest powers of two that hold H at `per` values a thread.
int threads_per_row(int H, int per) {
    int t = 4;
    while (t * per < H) t *= 2;
    return t;
}

// Values of a row a thread holds, for chunks of `width` (V: 16 bytes). More of them make fewer
// threads of a row and shorter sums, fewer a lighter loop. Backward, 8 / 16 a thread: 64,035 x 131
// fp16 39 / 57 us, 32,513 x 258 41 / 50, 8,371 x 1002 27 / 37; forward 30 / 38, 27 / 23, 16 / 18.
// Whole 16-byte chunks of 16-bit values (65,536 x 128): 15 / 14, forward 10 / 9; fp32 20 / 21,
// 10 / 10, and 22 / 21, 13 / 10 at 16,384 x 512, where 8 a thread leave the warp.
int values_per_thread(int H, int width, int V) {
    if (H > 2048 && width != V) return kPerThread;
    return width == V && (V == 8 || H > 256) ? kPerThread : 8;
}

// Blocks: enough for every row team to have a row, at most what runs at once
// (asked once per kernel and device; it also sets the kernel's shared-memory limit).
struct Resident {
    std::atomic<int> blocks[64];
};

template <typename K>
cudaError_t persistent_grid(K kernel, Resident& known, int block, size_t smem, int64_t want, int* grid) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    int cap = known.blocks[dev].load(std::memory_order_relaxed);
    if (cap == 0) {
        int per_sm = 0, sms = 0;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e == cudaSuccess) e = device_sms(&sms);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, block, smem);
        if (e != cudaSuccess) return e;
        cap = sms * (per_sm < 1 ? 1 : per_sm);
        if (cap > kMaxBlocks) cap = kMaxBlocks;
        known.blocks[dev].store(cap, std::memory_order_relaxed);
    }
    *grid = static_cast<int>(want < cap ? want : cap);
    return cudaSuccess;
}

struct FwdArgs {
    const void* x;
    int64_t ldx;
    const void* gamma;
    const void* beta;
    float eps;
    void* y;
    float* mean;
    float* rstd;
    int64_t T;
    int H;
};

struct BwdArgs {
    const void* x;
    const void* dy;
    int64_t ldx;
    const void* gamma;
    const float* mean;
    const float* rstd;
    void* dx;
    void* dgamma;
    void* dbeta;
    float* part;
    int64_t T;
    int H;
};

template <typename T, typename P, int VEC, int N, int BLOCK>
cudaError_t fwd_launch(const FwdArgs& a, int tpr, cudaStream_t s) {
    auto kernel = norm_fwd_kernel<T, P, VEC, N, BLOCK>;
    const int teams = BLOCK / tpr;
    static Resident known;
    int grid = 0;
    cudaError_t e = persistent_grid(kernel, known, BLOCK, 0, (a.T + teams - 1) / teams, &grid);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(grid), dim3(BLOCK), 0, s, static_cast<const T*>(a.x), a.ldx,
                      static_cast<const P*>(a.gamma), static_cast<const P*>(a.beta), a.eps, static_cast<T*>(a.y), a.mean,
                      a.rstd, a.T, a.H, tpr);
}

template <typename T, typename P, int VEC, int N, int BLOCK>
cudaError_t bwd_launch(const BwdArgs& a, int tpr, cudaStream_t s) {
    auto kernel = norm_bwd_kernel<T, P, VEC, N, BLOCK>;
    const int teams = BLOCK / tpr;
    const size_t smem = sizeof(float) * 2 * N * VEC * BLOCK;
    static Resident known;
    int grid = 0;
    // a block writes 2 H partial sums: beyond two blocks an SM it gets 16 turns of rows at
    // least (4099 x 1001: the second kernel takes 2.9 us instead of 4.4)
    int sms = 0;
    cudaError_t e = device_sms(&sms);
    if (e != cudaSuccess) return e;
    const int64_t turns = (a.T + teams - 1) / teams;
    const int64_t want = a.part && turns > 2 * sms ? std::max<int64_t>(2 * sms, (turns + 15) / 16) : turns;
    e = persistent_grid(kernel, known, BLOCK, smem, want, &grid);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kernel, dim3(grid), dim3(BLOCK), smem, s, static_cast<const T*>(a.x), static_cast<const T*>(a.dy),
                   a.ldx, static_cast<const P*>(a.gamma), a.mean, a.rstd, static_cast<T*>(a.dx), a.part, a.T, a.H, tpr);
    if (e != cudaSuccess || !a.part) return e;
    return launch_pdl(norm_reduce_kernel<P>, dim3((a.H + 31) / 32, 2), dim3(32, 32), 0, s,
                      static_cast<const float*>(a.part), grid, a.H, static_cast<P*>(a.dgamma), static_cast<P*>(a.dbeta));
}

// Chunk count per thread by row length; above 4096 values a row takes 512 threads.
template <bool FWD, typename T, typename P, typename A>
cudaError_t norm_dispatch(const A& a, int width, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    const int tpr = threads_per_row(a.H, values_per_thread(a.H, width, V));
    const int chunks = (a.H + width * tpr - 1) / (width * tpr);  // of a thread
#define MOE_NORM(VEC, N, BLOCK)                                       \
    do {                                                              \
        if constexpr (FWD) return fwd_launch<T, P, VEC, N, BLOCK>(a, tpr, s); \
        else return bwd_launch<T, P, VEC, N, BLOCK>(a, tpr, s);       \
    } while (0)
    if (width == V) {
        if (tpr > 256) MOE_NORM(V, kPerThread / V, 512);
        if (chunks == 1) MOE_NORM(V, 1, 256);
        if constexpr (V == 4) {
            if (chunks == 2) MOE_NORM(V, 2, 256);
        }
        MOE_NORM(V, kPerThread / V, 256);
    }
    if (width == 2) {
        if (tpr > 256) MOE_NORM(2, kPerThread / 2, 512);
        if (chunks <= 2) MOE_NORM(2, 2, 256);
        if (chunks <= 4) MOE_NORM(2, 4, 256);
        MOE_NORM(2, kPerThread / 2, 256);
    }
    if (tpr > 256) MOE_NORM(1, kPerThread, 512);
    if (chunks <= 4) MOE_NORM(1, 4, 256);
    if (chunks <= 8) MOE_NORM(1, 8, 256);
    MOE_NORM(1, kPerThread, 256);
#undef MOE_NORM
}

template <bool FWD, typename A>
cudaError_t norm_types(const A& a, moe_dtype_t dtype, moe_dtype_t param, int width, cudaStream_t s) {
    if (dtype == MOE_DTYPE_F32) return norm_dispatch<FWD, float, float>(a, width, s);
    if (dtype == MOE_DTYPE_BF16)
        return param == MOE_DTYPE_F32 ? norm_dispatch<FWD, __nv_bfloat16, float>(a, width, s)
                                      : norm_dispatch<FWD, __nv_bfloat16, __nv_bfloat16>(a, width, s);
    return param == MOE_DTYPE_F32 ? norm_dispatch<FWD, __half, float>(a, width, s)
                                  : norm_dispatch<FWD, __half, __half>(a, width, s);
}

// Values that are loaded at once: 16 bytes of them where every row and parameter array
// starts on 16 bytes (a float parameter array's chunk then starts on 16 bytes too), two
// where they start on two values, else one.
int chunk_width(moe_dtype_t dtype, int H, int64_t ldx, const void* const* ptrs, int n, moe_dtype_t param,
                const void* const* params, int np) {
    for (const int v : {static_cast<int>(16 / dtype_bytes(dtype)), 2}) {
        bool ok = H % v == 0 && ldx % v == 0;
        for (int i = 0; i < n; ++i) ok = ok && aligned(ptrs[i], v * dtype_bytes(dtype));
        const size_t pb = v * dtype_bytes(param);
        for (int i = 0; i < np; ++i) ok = ok && aligned(params[i], pb < 16 ? pb : 16);
        if (ok) return v;
    }
    return 1;
}

moe_status_t norm_shape(moe_dtype_t dtype, moe_dtype_t param, int64_t T, int32_t H, int64_t ldx) {
    if (T < 0 || H < 1 || ldx < H) return MOE_ERR_INVALID_ARG;
    if (!dtype_ok(dtype) || !dtype_ok(param) || (param != dtype && param != MOE_DTYPE_F32)) return MOE_ERR_INVALID_ARG;
    if (T >= kMaxT || H > kMaxH || ldx > (int64_t{1} << 31)) return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

size_t rows_bytes(int64_t T, int32_t H, int64_t ld, size_t b) { return T > 0 ? (static_cast<size_t>(T - 1) * ld + H) * b : 0; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_layer_norm_fwd(const void* x, moe_dtype_t dtype, int64_t T, int32_t H, int64_t ldx,
                                const void* gamma, const void* beta, moe_dtype_t param_dtype, float eps, void* y,
                                float* mean, float* rstd, void* stream) {
    moe_status_t st = norm_shape(dtype, param_dtype, T, H, ldx);
    if (st != MOE_OK) return st;
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!x || !y)) return MOE_ERR_INVALID_ARG;
    const size_t b = dtype_bytes(dtype), pb = dtype_bytes(param_dtype);
    if (!aligned(x, b) || !aligned(y, b) || !aligned(gamma, pb) || !aligned(beta, pb) || !aligned(mean, 4) ||
        !aligned(rstd, 4))
        return MOE_ERR_MISALIGNED;
    const bool in_place = y == x && ldx == H;
    const Range outs[3] = {{y, static_cast<size_t>(T) * H * b}, {mean, sizeof(float) * T}, {rstd, sizeof(float) * T}};
    const Range ins[2] = {{gamma, H * pb}, {beta, H * pb}};
    const Range xr = {x, rows_bytes(T, H, ldx, b)};
    if (any_alias(outs, 3, ins, 2) || any_alias(outs + (in_place ? 1 : 0), in_place ? 2 : 3, &xr, 1)) return MOE_ERR_ALIAS;
    if (T == 0) return MOE_OK;
    const void *ptrs[2] = {x, y}, *params[2] = {gamma, beta};
    const FwdArgs a{x, ldx, gamma, beta, eps, y, mean, rstd, T, H};
    return cuda_status(norm_types<true>(a, dtype, param_dtype, chunk_width(dtype, H, ldx, ptrs, 2, param_dtype, params, 2),
                                        static_cast<cudaStream_t>(stream)));
}

size_t moe_layer_norm_workspace_bytes(int64_t T, int32_t H) {
    if (T < 0 || T >= kMaxT || H < 1 || H > kMaxH) return 0;
    const size_t rows = static_cast<size_t>(T < kMaxBlocks ? T : kMaxBlocks);
    return 256 + align_up(rows * 2 * H * sizeof(float), 256);
}

moe_status_t moe_layer_norm_bwd(const void* x, const void* dy, moe_dtype_t dtype, int64_t T, int32_t H, int64_t ldx,
                                const void* gamma, moe_dtype_t param_dtype, const float* mean, const float* rstd,
                                void* dx, void* dgamma, void* dbeta, void* workspace, size_t workspace_bytes,
                                void* stream) {
    moe_status_t st = norm_shape(dtype, param_dtype, T, H, ldx);
    if (st != MOE_OK) return st;
    if (!dx && !dgamma && !dbeta) return MOE_OK;
    if (T > 0 && (!x || !dy || !mean || !rstd)) return MOE_ERR_INVALID_ARG;
    const size_t b = dtype_bytes(dtype), pb = dtype_bytes(param_dtype);
    if (!aligned(x, b) || !aligned(dy, b) || !aligned(dx, b) || !aligned(gamma, pb) || !aligned(dgamma, pb) ||
        !aligned(dbeta, pb) || !aligned(mean, 4) || !aligned(rstd, 4))
        return MOE_ERR_MISALIGNED;
    const size_t row_bytes = static_cast<size_t>(T) * H * b;
    const Range outs[4] = {{dx, row_bytes},
                           {dgamma, H * pb},
                           {dbeta, H * pb},
                           {workspace, (dgamma || dbeta) && workspace ? workspace_bytes : 0}};
    const Range ins[5] = {{x, rows_bytes(T, H, ldx, b)},
                          {gamma, H * pb},
                          {mean, sizeof(float) * T},
                          {rstd, sizeof(float) * T},
                          {dx == dy ? nullptr : dy, row_bytes}};
    if (any_alias(outs, 4, ins, 5)) return MOE_ERR_ALIAS;
    if (dx == dy) {  // dy is then an output too
        const Range d[1] = {{dy, row_bytes}};
        if (any_alias(outs + 1, 3, d, 1)) return MOE_ERR_ALIAS;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        cudaError_t e = cudaSuccess;
        if (dgamma) e = cudaMemsetAsync(dgamma, 0, H * pb, s);
        if (e == cudaSuccess && dbeta) e = cudaMemsetAsync(dbeta, 0, H * pb, s);
        return cuda_status(e);
    }
    float* part = nullptr;
    if (dgamma || dbeta) {
        if (!workspace) return MOE_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return MOE_ERR_MISALIGNED;
        if (workspace_bytes < moe_layer_norm_workspace_bytes(T, H)) return MOE_ERR_WORKSPACE;
        part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + 256);
    }
    const void* ptrs[3] = {x, dy, dx};
    const BwdArgs a{x, dy, ldx, gamma, mean, rstd, dx, dgamma, dbeta, part, T, H};
    return cuda_status(
        norm_types<false>(a, dtype, param_dtype, chunk_width(dtype, H, ldx, ptrs, 3, param_dtype, &gamma, 1), s));
}

}  // extern "C"
