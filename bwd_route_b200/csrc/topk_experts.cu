// topk_experts.cu -- the experts' weighted product of the top-k block and its gradients,
// on tcgen05 (bf16 or fp16 operands, fp32 accumulators in tensor memory).
//
//   y_t    = sum_k w_tk (W_e x_t + b_e),  e = e_tk
//   d_x_t  = sum_k w_tk W_e^T g_t
//   d_w_tk = g_t . (W_e x_t + b_e) = x_t . (W_e^T g_t) + g_t . b_e
//   dW_e   = sum over the pairs of e of w g x^T,   db_e = sum of w g
//
// The pairs (t, k) of an expert are contiguous in the routing's perm, so every expert is
// a dense product over rows gathered on the fly.
//
//   pair_kernel   : rows of y and d_x. Persistent, one block per SM; a tile is 128 pairs
//     of one expert x BN outputs. Four warps gather the rows by cp.async into a swizzled
//     ring, one warp streams the expert's weights by TMA (K-major for y, MN-major for
//     d_x), one thread issues the MMAs into one of two tensor-memory accumulators, eight
//     warps drain the other. With K = 1 a pair's row is the result; else it goes to the
//     workspace in fp32, so that a token's sum over k is fp32 from end to end and y and d_x
//     are rounded once. The backward's epilogue also takes x . (W_e^T g) from the fp32
//     accumulators, with its warps' rows of x brought in by cp.async beside them.
//     Bound by shared memory: a chunk of 64 channels moves 96 KB (rows in, weights in, both
//     read by the MMA) at 128 bytes a cycle, 768 cycles against the MMA's 512, and an epilogue
//     that moves 8 bytes a value through it. 16,384 tokens, E 16, K 2, H 1024, d_x: 78 us,
//     0.88 PFLOP/s (54 % of a library product's); 16-bit rows with a power of two per 32
//     columns took 69, but carried a rounding of 11 bits for each of the K.
//   duo_kernel    : y and d_x for K = 2 and many tokens: see there. 262,144 tokens, E 8,
//     H 256, y: 81 us and 13 for the grouping, 0.85 PFLOP/s and 3.3 TB/s (floor 42 us by
//     either); bound by the epilogue's chain (tensor memory, two weights, rounding,
//     transpose, store), the tensor pipe runs 40 % of the time.
//   join_kernel   : adds the K rows of a token (and w b_e) in the order of k in fp32, one
//     rounding; in the backward also d_w from the column parts and g . b_e. 16,384 tokens,
//     K 2, H 1024, backward: 47 us for 201 MB (4.3 TB/s, in part from L2).
//   wgrad_kernel  : dW and db. The pairs are the contraction index: both operands are
//     MN-major. Four warps gather rows of g and x by cp.async, eight multiply the staged rows
//     of g by w (the weight depends on the pair, the contraction index, so it has to be in one
//     operand), leave the products as two 16-bit numbers each for the MMAs (fp16 with a power of
//     two per expert from wgrad_peak_kernel) and add them up for db; a unit is a
//     256 x 256 tile of dW[e] over a piece of e's pairs (topk_plan.h). 16,384 tokens, E 16,
//     K 2, H 1024: 123 us, 0.56 PFLOP/s of dW alone; a stage of 32 pairs moves 176 KB through
//     shared memory (rows in, two parts out, read by the MMAs), 1375 cycles. One part, rounded,
//     takes 85 us at that size and leaves dW's relative error at 2.3e-3 in bf16 where the rounding
//     of the result alone gives 1.7e-3, as two parts do. A third group of four scaling warps was
//     slower (141 us for the call instead of 130), as their registers then are fewer.
//   wgrad_sum_kernel: adds the pieces of cut experts in order; zeros for experts without
//     pairs. 7 us at that size.
//
// The tensor cores cut what they add to an fp32 accumulator towards zero, so a sum of 1024
// terms in steps of 16 comes out up to 64 * 2^-24 smaller: d_weights, which is not rounded
// to 16 bits afterwards, shows it (relative error 1.0e-6 at H = 1024, 2e-7 at H = 128).
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "checks.h"
#include "common.cuh"
#include "elem.cuh"
#include "internal.h"
#include "moe_topk.h"
#include "topk.h"
#include "topk_plan.h"

namespace moe {
namespace {

constexpr int kMaxE = 256, kMaxK = 16, kMaxH = 4096;
constexpr unsigned kFull = 0xffffffffu;

// One lane of a converged warp.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t x;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(x));
    return x;
}
// A wait of a whole warp whose outcome is the same in every lane for the compiler too.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* flags) {
    return __all_sync(kFull, mbar_wait(bar, parity, abort, flags));
}
// Two of them, asked for together: where both are there already, one latency.
__device__ __forceinline__ bool warp_wait_both(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb, volatile int* abort,
                                               uint32_t* flags) {
    const bool ra = mbar_try_wait(smem_u32(a), pa), rb = mbar_try_wait(smem_u32(b), pb);
    if (__all_sync(kFull, ra && rb)) return true;
    return warp_wait(a, pa, abort, flags) && warp_wait(b, pb, abort, flags);
}
// D[tmem] (+)= A[smem] * B[smem]^T, kind::f16 (both operands fp16 or both bf16), fp32 sums.
// The whole warp comes here with the same operands, which then sit in uniform registers as
// the instruction wants them, and the elected lane issues. The descriptors come as words:
// the upper ones are constants, the lower ones a constant plus the operand's address / 16.
__device__ __forceinline__ void mma_f16(uint32_t leader, uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo,
                                        uint32_t b_hi, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "setp.ne.b32 q, %7, 0;\n\t"
        "mov.b64 da, {%1, %2};\n\t"
        "mov.b64 db, {%3, %4};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void commit_f16(uint32_t leader, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)), "r"(leader)
        : "memory");
}

// The elected lane expects `bytes` on the barrier; loads one box.
__device__ __forceinline__ void expect_f16(uint32_t leader, uint64_t* bar, uint32_t bytes) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
        "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(smem_u32(bar)), "r"(bytes), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void load_box(uint32_t leader, uint32_t dst, const CUtensorMap* map, int32_t c0, int32_t c1,
                                         uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar)), "r"(leader)
        : "memory");
}

template <typename T>
struct MmaFormat;
template <>
struct MmaFormat<__half> {
    static constexpr uint32_t value = 0;
};
template <>
struct MmaFormat<__nv_bfloat16> {
    static constexpr uint32_t value = 1;
};

// Instruction descriptor of kind::f16 with fp32 accumulation; mn: the operand is MN-major.
template <typename T>
__device__ __forceinline__ uint32_t idesc_f16(int M, int N, int a_mn, int b_mn) {
    return (1u << 4) | (MmaFormat<T>::value << 7) | (MmaFormat<T>::value << 10) | (static_cast<uint32_t>(a_mn) << 15) |
           (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}

// Descriptor words of 16-bit operands in the 128-byte swizzle, 8-row groups 1024 bytes
// apart. K-major: rows of 64 elements along K; 16 of them are 32 bytes on. MN-major: rows
// along K of 64 elements of M or N, groups of 64 along M or N lbo bytes apart; 16 rows are
// 2048 bytes on. (The layout of sw128_desc.)
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kKStep = 32 >> 4, kMnStep = 2048 >> 4;
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo_bytes) { return (addr >> 4) | ((lbo_bytes >> 4) << 16); }

template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&s)[8]) {
    uint4 v;
    T* e = reinterpret_cast<T*>(&v);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = from_f<T>(s[i]);
    return v;
}

// Division of pair numbers (below 2^31) by K: q = (p * mul) >> shift, exact for
// shift = 31 + ceil(log2 K), mul = floor(2^shift / K) + 1.
struct DivK {
    uint32_t mul;
    int shift;
    __device__ __forceinline__ int operator()(int p) const {
        return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(p)) * mul) >> shift);
    }
};
inline DivK div_by(int K) {
    int s = 0;
    while ((1 << s) < K) ++s;
    return {static_cast<uint32_t>((uint64_t{1} << (31 + s)) / static_cast<uint32_t>(K) + 1), 31 + s};
}

__device__ __forceinline__ void st_shared_u4(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Largest i with start[i] <= v (start ascending, start[0] = 0 <= v < start[n]; empty spans skipped).
__device__ __forceinline__ int span_of(const int* start, int n, int v) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= v) lo = mid;
        else hi = mid;
    }
    return lo;
}

// start[i] = exclusive sum of count(0 .. i), start[n] = total; one warp, any n.
template <typename F>
__device__ __forceinline__ void warp_starts(int* start, int n, F count) {
    const int lane = threadIdx.x & 31;
    int carry = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + lane;
        const int c = i < n ? count(i) : 0;
        int incl = c;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int u = __shfl_up_sync(kFull, incl, off);
            if (lane >= off) incl += u;
        }
        if (i < n) start[i] = carry + incl - c;
        carry += __shfl_sync(kFull, incl, 31);
    }
    if (lane == 0) start[n] = carry;
}

// ---------------------------------------------------------------- y and d_x
// Warps 0-7 epilogue (tensor-memory quadrant w % 4, column half w / 4), 8-11 row gather,
// 12 MMA issuer and tensor-memory owner, 13 weight loader.
constexpr int kPairThreads = 448;
constexpr int kPEpiWarps = 8, kPProducer0 = 256, kPMmaWarp = 12, kPLoadWarp = 13;
constexpr int kMaxStages = 8;

struct __align__(8) PairCtl {
    uint64_t afull[kMaxStages], aempty[kMaxStages], bfull[kMaxStages], bempty[kMaxStages];
    uint64_t tfull[2], tempty[2];
    uint32_t tmem_base;
    int abort;
    int off[kMaxE + 1];
    int tstart[kMaxE + 1];
};

template <int BN, bool DX>
struct PairCfg {
    static constexpr int BM = 128;
    static constexpr int A_BYTES = BM * 128;
    static constexpr int B_BYTES = BN * 128;
    static constexpr int A_STAGES = BN == 256 ? 5 : 6;
    static constexpr int B_STAGES = BN == 256 ? 3 : 5;
    static constexpr int RING_BYTES = A_STAGES * A_BYTES + B_STAGES * B_BYTES;
    static constexpr int HALVES = BN == 64 ? 1 : 2;        // column parts the epilogue warps share out
    static constexpr int HALF = BN / HALVES;
    static constexpr int STEP_BYTES = 32 * 64;             // 32 rows x 32 columns of one warp
    static constexpr int STG_BYTES = kPEpiWarps * STEP_BYTES * (DX ? 2 : 1);  // d_x: two steps of rows of x
    static constexpr int TMEM_COLS = 2 * BN;
    static constexpr int SMEM_BYTES = 1024 + RING_BYTES + STG_BYTES + static_cast<int>(sizeof(PairCtl));
    static_assert(A_STAGES <= kMaxStages && B_STAGES <= kMaxStages, "stages");
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
};

struct DuoWs {
    int32_t* count;  // [E * E] counts, [E * E] places taken, [E * E + 1] starts
    int32_t* list;   // [T]
};

struct PairArgs {
    const void* src;       // rows of tokens: x (y) or d_out (d_x)
    const void* other;     // d_x: x, for the weights' gradient (may be NULL)
    const void* bias;      // y: may be NULL
    const float* weights;  // [P]
    const int32_t* offsets;
    const int32_t* perm;
    int E, K, H;
    DivK by_k;
    int64_t P;
    void* out;             // [T][H]; d_x: may be NULL (only the weights' gradient)
    float* rows;           // [P][H], K > 1
    float* dw_part;        // [parts][P], d_x with `other`
    DuoWs duo;             // K = 2: see duo_kernel
    uint32_t* flags;
};

// DX = false: B_e[n][k] = W[e][n][k], K-major. DX = true: B_e[n][k] = W[e][k][n], MN-major
// straight from W.
// ONE: K = 1, a pair's row is the result.
template <typename T, int BN, bool DX, bool ONE>
__global__ void __launch_bounds__(kPairThreads, 1)
pair_kernel(const __grid_constant__ CUtensorMap tm_w, const PairArgs A) {
    using C = PairCfg<BN, DX>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* aring = smem;
    uint8_t* bring = smem + C::A_STAGES * C::A_BYTES;
    uint8_t* stg = smem + C::RING_BYTES;
    PairCtl* ctl = reinterpret_cast<PairCtl*>(smem + C::RING_BYTES + C::STG_BYTES);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int H = A.H;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::A_STAGES; ++s) {
            mbar_init(&ctl->afull[s], 128);  // 128 gather threads
            mbar_init(&ctl->aempty[s], 1);   // tcgen05.commit
        }
        for (int s = 0; s < C::B_STAGES; ++s) {
            mbar_init(&ctl->bfull[s], 1);    // arrive.expect_tx + TMA bytes
            mbar_init(&ctl->bempty[s], 1);   // tcgen05.commit
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ctl->tfull[b], 1);
            mbar_init(&ctl->tempty[b], kPEpiWarps);
        }
        ctl->abort = 0;
        fence_mbar_init();
    }
    if (warp == kPLoadWarp && lane == 0) tma_prefetch_desc(&tm_w);
    if (warp == kPMmaWarp) {
        tmem_alloc(&ctl->tmem_base, C::TMEM_COLS);
        tmem_relinquish();
    }
    griddep_wait();  // the prologue above overlaps the previous kernel; global memory from here on
    for (int e = threadIdx.x; e <= A.E; e += kPairThreads) ctl->off[e] = A.offsets[e];
    __syncthreads();
    if (warp == 0)
        warp_starts(ctl->tstart, A.E, [&](int e) { return (ctl->off[e + 1] - ctl->off[e] + C::BM - 1) / C::BM; });
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    const int NT = (H + BN - 1) / BN, KCH = H / 64;
    const int ntiles = ctl->tstart[A.E] * NT;  // below 2^31: checked by the caller
    volatile int* abort = &ctl->abort;
    auto tile_rows = [&](int tile, int& e, int& row0, int& nrows) {
        const int mt = tile / NT;
        e = span_of(ctl->tstart, A.E, mt);
        row0 = ctl->off[e] + (mt - ctl->tstart[e]) * C::BM;
        nrows = min(C::BM, ctl->off[e + 1] - row0);
    };

    if (warp >= kPProducer0 / 32 && warp < kPProducer0 / 32 + 4) {
        // ---------------- row gather: 16 bytes per lane, 8 lanes per 128-byte row segment
        const T* src = static_cast<const T*>(A.src);
        const int ptid = threadIdx.x - kPProducer0;
        const int prow = ptid >> 3, pg = ptid & 7;
        int nxt[8];
        const T* row[8];  // this lane's 16 bytes of the first chunk of its rows
        unsigned there = 0;
        // the pairs of a tile's rows; their tokens are worked out a tile later, when the loads are there
        auto load_pairs = [&](int tile, int (&t)[8]) {
            int e, row0, nrows;
            tile_rows(tile, e, row0, nrows);
#pragma unroll
            for (int it = 0; it < 8; ++it) {
                const int r = it * 16 + prow;
                t[it] = r < nrows ? A.perm[row0 + r] : -1;
            }
        };
        auto to_tokens = [&](const int (&pair)[8]) {
            there = 0;
#pragma unroll
            for (int it = 0; it < 8; ++it) {
                row[it] = src + static_cast<int64_t>(pair[it] < 0 ? 0 : A.by_k(pair[it])) * H + pg * 8;
                there |= pair[it] < 0 ? 0u : 1u << it;
            }
        };
        if (static_cast<int>(blockIdx.x) < ntiles) {
            load_pairs(blockIdx.x, nxt);
            to_tokens(nxt);
        }
        const uint32_t to = smem_u32(aring) + prow * 128 + ((pg ^ (prow & 7)) << 4);  // rows 16 apart swizzle alike
        int sa = 0;
        uint32_t pa = 0;
        bool ok = true;
        for (int tile = blockIdx.x; tile < ntiles && ok; tile += gridDim.x) {
            if (tile + static_cast<int>(gridDim.x) < ntiles) load_pairs(tile + gridDim.x, nxt);
            for (int kc = 0; kc < KCH; ++kc) {
                if (!(ok = mbar_wait(&ctl->aempty[sa], pa ^ 1, abort, A.flags))) break;
                const uint32_t a_u32 = to + sa * C::A_BYTES;
#pragma unroll
                for (int it = 0; it < 8; ++it)
                    cp_async_16_l2_256(a_u32 + it * 16 * 128, row[it] + kc * 64, (there >> it) & 1u ? 16u : 0u);
                cp_async_arrive_noinc(&ctl->afull[sa]);
                if (++sa == C::A_STAGES) {
                    sa = 0;
                    pa ^= 1;
                }
            }
            to_tokens(nxt);
        }
    } else if (warp == kPLoadWarp) {
        // ---------------- weight loader. Boxes may reach past the expert's last row or column block
        // (H not a multiple of BN): those columns of the accumulator are not used.
        {
            const uint32_t leader = elect_one(), ring = smem_u32(bring);
            int sb = 0;
            uint32_t pb = 0;
            bool ok = true;
            for (int tile = blockIdx.x; tile < ntiles && ok; tile += gridDim.x) {
                int e, row0, nrows;
                tile_rows(tile, e, row0, nrows);
                const int n0 = (tile % NT) * BN;
                const int ng = DX ? min(BN, H - n0) / 64 : 0;
                for (int kc = 0; kc < KCH; ++kc) {
                    if (!(ok = warp_wait(&ctl->bempty[sb], pb ^ 1, abort, A.flags))) break;
                    if (DX) {
                        expect_f16(leader, &ctl->bfull[sb], ng * 64 * 128);
                        for (int g = 0; g < ng; ++g)
                            load_box(leader, ring + sb * C::B_BYTES + g * 64 * 128, &tm_w, n0 + g * 64, e * H + kc * 64,
                                        &ctl->bfull[sb]);
                    } else {
                        expect_f16(leader, &ctl->bfull[sb], C::B_BYTES);
                        load_box(leader, ring + sb * C::B_BYTES, &tm_w, kc * 64, e * H + n0, &ctl->bfull[sb]);
                    }
                    if (++sb == C::B_STAGES) {
                        sb = 0;
                        pb ^= 1;
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == kPMmaWarp) {
        // ---------------- MMA issuer (the warp stays together, one lane issues)
        {
            const uint32_t leader = elect_one();
            const uint32_t a0 = desc_lo(smem_u32(aring), 16), b0 = desc_lo(smem_u32(bring), DX ? 64 * 128 : 16);
            int sa = 0, sb = 0;
            uint32_t pa = 0, pb = 0;
            int acc = 0;
            uint32_t acc_phase = 0;
            bool ok = true;
            for (int tile = blockIdx.x; tile < ntiles && ok; tile += gridDim.x) {
                if (!(ok = warp_wait(&ctl->tempty[acc], acc_phase ^ 1, abort, A.flags))) break;
                tc_fence_after();
                const uint32_t idesc = idesc_f16<T>(128, min(BN, H - (tile % NT) * BN), 0, DX ? 1 : 0);
                const uint32_t d = tmem + static_cast<uint32_t>(acc * BN);
                for (int kc = 0; kc < KCH; ++kc) {
                    if (!(ok = warp_wait_both(&ctl->afull[sa], pa, &ctl->bfull[sb], pb, abort, A.flags))) break;
                    fence_proxy_async_smem();
                    tc_fence_after();
                    const uint32_t a = a0 + sa * (C::A_BYTES >> 4), b = b0 + sb * (C::B_BYTES >> 4);
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_f16(leader, d, a + ks * kKStep, kDescHi, b + ks * (DX ? kMnStep : kKStep), kDescHi, idesc, ks != 0 ? 1u : kc != 0);
                    commit_f16(leader, &ctl->aempty[sa]);
                    commit_f16(leader, &ctl->bempty[sb]);
                    if (++sa == C::A_STAGES) {
                        sa = 0;
                        pa ^= 1;
                    }
                    if (++sb == C::B_STAGES) {
                        sb = 0;
                        pb ^= 1;
                    }
                }
                if (!ok) break;
                commit_f16(leader, &ctl->tfull[acc]);
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1;
            }
        }
        __syncwarp();
    } else if (warp < kPEpiWarps) {
        // ---------------- epilogue: this lane's row is 32 (w % 4) + lane; columns of half w / 4,
        // 32 a step
        constexpr int HALF = C::HALF;
        const int q = warp & 3, half = warp >> 2;
        const uint32_t my = smem_u32(stg + warp * C::STEP_BYTES * (DX ? 2 : 1));
        const int myrow = 32 * q + lane;
        const int R4 = lane >> 2, j4 = lane & 3;  // row and 16-byte granule of a lane where a warp moves 8 rows
        const uint32_t swz = (lane >> 1) & 3;     // granule g of row r sits at g ^ ((r >> 1) & 3)
        T* out = static_cast<T*>(A.out);
        auto tile_pair = [&](int tile) -> int {
            int e, row0, nrows;
            tile_rows(tile, e, row0, nrows);
            return myrow < nrows ? A.perm[row0 + myrow] : -1;
        };
        auto tile_cols = [&](int tile) { return half < C::HALVES ? min(HALF, H - (tile % NT) * BN - half * HALF) : 0; };
        // d_x: this warp's 32 rows of x, 32 columns from col, into one of its two buffers
        auto fetch_x = [&](int pair, int col, int buf) {
            const T* xs = static_cast<const T*>(A.other);
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const int R = it * 8 + R4;
                const int pr = __shfl_sync(kFull, pair, R);
                cp_async_16(my + buf * C::STEP_BYTES + R * 64 + ((j4 ^ ((R >> 1) & 3)) << 4),
                            xs + static_cast<int64_t>(pr < 0 ? 0 : A.by_k(pr)) * H + col + j4 * 8, pr < 0 ? 0u : 16u);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        int tile = blockIdx.x;
        int p_next = tile < ntiles ? tile_pair(tile) : -1;
        int buf = 0;
        if (DX && A.other && tile < ntiles && tile_cols(tile) > 0) fetch_x(p_next, (tile % NT) * BN + half * HALF, 0);
        int acc = 0;
        uint32_t acc_phase = 0;
        for (; tile < ntiles; tile += gridDim.x) {
            const int p = p_next, next_tile = tile + gridDim.x;
            const float w = p >= 0 ? A.weights[p] : 0.0f;
            if (next_tile < ntiles) p_next = tile_pair(next_tile);
            const int nt = tile % NT, col0 = nt * BN + half * HALF, ncols = tile_cols(tile);
            const int e = ONE && !DX ? span_of(ctl->tstart, A.E, tile / NT) : 0;  // for the bias
            if (!mbar_wait(&ctl->tfull[acc], acc_phase, abort, A.flags)) break;
            __syncwarp();
            tc_fence_after();
            const uint32_t tbase = tmem + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(acc * BN + half * HALF);
            // where the lane's share of rows 8 it + R4 goes: the output, or rows of the workspace
            uint8_t* dst[4];
            unsigned there = 0;
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const int pr = __shfl_sync(kFull, p, it * 8 + R4);
                there |= pr >= 0 ? 1u << it : 0u;
                const int64_t at = static_cast<int64_t>(pr < 0 ? 0 : pr) * H + col0;
                dst[it] = ONE ? reinterpret_cast<uint8_t*>(out + at + j4 * 8) : reinterpret_cast<uint8_t*>(A.rows + at + j4 * 4);
            }
            float dot = 0.0f;
            uint32_t tm[2][32];
            if (ncols > 0) {
                tmem_ld_32x32b_x32_async(tbase, tm[0]);
                tmem_ld_wait_tied(tm[0]);
            }
#pragma unroll
            for (int i = 0; i < HALF / 32; ++i) {
                const int c = 32 * i;
                if (c >= ncols) break;
                const bool more = c + 32 < ncols;
                // the next step's sums on the way; after the last the next tile may have the accumulator
                if (more) {
                    tmem_ld_32x32b_x32_async(tbase + static_cast<uint32_t>(c + 32), tm[(i + 1) & 1]);
                } else {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl->tempty[acc]);
                }
                float v[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(tm[i & 1][j]);
                const int col = col0 + c;
                const uint32_t stage = my + (DX ? buf * C::STEP_BYTES : 0);
                bool store = true;
                if (DX) {
                    if (A.other) {
                        // the next step's rows of x (of this tile or the next) on the way, this one's here
                        if (more) fetch_x(p, col + 32, buf ^ 1);
                        else if (next_tile < ntiles && tile_cols(next_tile) > 0)
                            fetch_x(p_next, (next_tile % NT) * BN + half * HALF, buf ^ 1);
                        else asm volatile("cp.async.commit_group;" ::: "memory");
                        asm volatile("cp.async.wait_group 1;" ::: "memory");
                        __syncwarp();
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            const uint4 raw = ld_shared_u4(stage + lane * 64 + ((g ^ swz) << 4));
                            const T* xv = reinterpret_cast<const T*>(&raw);
#pragma unroll
                            for (int j = 0; j < 8; ++j) dot += v[8 * g + j] * to_f(xv[j]);
                        }
                    }
                    buf ^= 1;
                    store = out != nullptr;
                } else if (ONE && A.bias) {
                    const T* br = static_cast<const T*>(A.bias) + static_cast<int64_t>(e) * H + col;
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const Chunk<T, 8> bv = *reinterpret_cast<const Chunk<T, 8>*>(br + 8 * g);
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[8 * g + j] += to_f(bv.v[j]);
                    }
                }
                if (store && ONE) {
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        float s[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) s[j] = v[8 * g + j] * w;
                        st_shared_u4(stage + lane * 64 + ((g ^ swz) << 4), pack8<T>(s));
                    }
                    __syncwarp();
#pragma unroll
                    for (int it = 0; it < 4; ++it) {
                        const int R = it * 8 + R4;
                        const uint4 val = ld_shared_u4(stage + R * 64 + ((j4 ^ ((R >> 1) & 3)) << 4));
                        if ((there >> it) & 1u) *reinterpret_cast<uint4*>(dst[it] + 2 * c) = val;
                    }
                } else if (store) {
                    // fp32: 16 columns at a time
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (h) __syncwarp();
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            const int j = 16 * h + 4 * g;
                            st_shared_v4(stage + lane * 64 + ((g ^ swz) << 4), v[j] * w, v[j + 1] * w, v[j + 2] * w, v[j + 3] * w);
                        }
                        __syncwarp();
#pragma unroll
                        for (int it = 0; it < 4; ++it) {
                            const int R = it * 8 + R4;
                            const float4 val = ld_shared_v4(stage + R * 64 + ((j4 ^ ((R >> 1) & 3)) << 4));
                            if ((there >> it) & 1u) *reinterpret_cast<float4*>(dst[it] + 4 * (c + 16 * h)) = val;
                        }
                    }
                }
                __syncwarp();
                if (more) tmem_ld_wait_tied(tm[(i + 1) & 1]);
            }
            if (ncols <= 0) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->tempty[acc]);
                if (DX && A.other && next_tile < ntiles && tile_cols(next_tile) > 0)
                    fetch_x(p_next, (next_tile % NT) * BN + half * HALF, buf);
            }
            if (DX && A.other && p >= 0 && half < C::HALVES)
                A.dw_part[static_cast<int64_t>(nt * C::HALVES + half) * A.P + p] = dot;
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1;
        }
        if (DX) asm volatile("cp.async.wait_all;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kPMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// ---------------------------------------------------------------- two experts per token
// K = 2 with many tokens per pair of experts: the tokens are grouped by their two experts
// (lo <= hi), so that a tile of 128 tokens has both products in tensor memory at once and
// writes the sum itself: x is read once, no row waits for another, one rounding.
constexpr int kDuoMaxE = 32, kDuoMaxH = 256;
constexpr int kDuoTokens = 2048;  // tokens of a block of the two grouping kernels

// Counts of the classes lo * E + hi over a block's tokens, added to count [E * E] (zeroed).
__global__ void __launch_bounds__(256) duo_count_kernel(const int32_t* __restrict__ expert_idx, int64_t T_, int E,
                                                        int32_t* __restrict__ count) {
    griddep_wait();  // every global access below comes after the previous grid
    __shared__ int hist[kDuoMaxE * kDuoMaxE];
    const int n = E * E;
    for (int i = threadIdx.x; i < n; i += 256) hist[i] = 0;
    __syncthreads();
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kDuoTokens;
#pragma unroll
    for (int j = 0; j < kDuoTokens / 256; ++j) {
        const int64_t t = t0 + j * 256 + threadIdx.x;
        if (t < T_) {
            const int2 e = *reinterpret_cast<const int2*>(expert_idx + 2 * t);
            atomicAdd(&hist[min(e.x, e.y) * E + max(e.x, e.y)], 1);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += 256)
        if (hist[i]) atomicAdd(&count[i], hist[i]);
}

// list: the tokens by class, as 2 t + (the slot of the lower expert); start [E * E + 1]: where
// each class begins. The order inside a class varies from run to run and changes no result:
// a token's numbers do not depend on its row. taken [E * E] (zeroed): places given out.
__global__ void __launch_bounds__(256)
duo_group_kernel(const int32_t* __restrict__ expert_idx, int64_t T_, int E, const int32_t* __restrict__ count,
                 int32_t* __restrict__ taken, int32_t* __restrict__ start, int32_t* __restrict__ list) {
    griddep_wait();  // every global access below comes after the previous grid
    __shared__ int hist[kDuoMaxE * kDuoMaxE], base[kDuoMaxE * kDuoMaxE];
    __shared__ int s_warp[8];
    const int n = E * E;
    for (int i = threadIdx.x; i < n; i += 256) hist[i] = 0;
    __syncthreads();
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kDuoTokens;
    constexpr int N = kDuoTokens / 256;
    int bin[N], rank[N], code[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int64_t t = t0 + j * 256 + threadIdx.x;
        bin[j] = -1;
        if (t < T_) {
            const int2 e = *reinterpret_cast<const int2*>(expert_idx + 2 * t);
            bin[j] = min(e.x, e.y) * E + max(e.x, e.y);
            code[j] = static_cast<int>(2 * t) + (e.x <= e.y ? 0 : 1);
            rank[j] = atomicAdd(&hist[bin[j]], 1);
        }
    }
    // exclusive sums of the counts: four neighbouring classes a thread
    int c[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int b = threadIdx.x * 4 + i;
        c[i] = b < n ? count[b] : 0;
        sum += c[i];
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int u = __shfl_up_sync(kFull, incl, off);
        if (lane >= off) incl += u;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int at = incl - sum;
    for (int w = 0; w < warp; ++w) at += s_warp[w];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int b = threadIdx.x * 4 + i;
        if (b < n) {
            base[b] = at + (hist[b] ? atomicAdd(&taken[b], hist[b]) : 0);
            if (blockIdx.x == 0) start[b] = at;
        }
        at += c[i];
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) start[n] = static_cast<int32_t>(T_);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (bin[j] >= 0) list[base[bin[j]] + rank[j]] = code[j];
}

// Warps as in pair_kernel. A tile's rows (all of H, at most 4 chunks of 64 columns) stay in
// shared memory while both experts' weights pass by, 128 output columns at a time: 128
// rows of either expert's W are one operand of 256, so one MMA does both, and its 256
// accumulator columns are one half of tensor memory. (Where fewer than 128 columns are
// left, the rest of either half is computed from what lies there and not used.)
template <bool DX>
struct DuoCfg {
    static constexpr int A_BYTES = 128 * 128, B_BYTES = 256 * 128;
    static constexpr int A_STAGES = DX ? 5 : 6;  // a tile of 256 columns and a part of the next
    static constexpr int B_STAGES = 3;
    static constexpr int RING_BYTES = A_STAGES * A_BYTES + B_STAGES * B_BYTES;
    static constexpr int STEP_BYTES = 32 * 64;
    static constexpr int STG_BYTES = kPEpiWarps * STEP_BYTES * (DX ? 2 : 1);
    static constexpr int TMEM_COLS = 512;
};

struct __align__(8) DuoCtl {
    uint64_t afull[8], aempty[8], bfull[4], bempty[4];
    uint64_t tfull[2], tempty[2];
    uint32_t tmem_base;
    int abort;
    int start[kDuoMaxE * kDuoMaxE + 1];
    int tstart[kDuoMaxE * kDuoMaxE + 1];
};
// y: behind it, for every epilogue warp, the biases of a tile's two experts in its columns, [2][128] fp32.
constexpr int kDuoBias = 2 * 128 * 4;
template <bool DX>
constexpr int duo_smem() {
    return 1024 + DuoCfg<DX>::RING_BYTES + DuoCfg<DX>::STG_BYTES + static_cast<int>(sizeof(DuoCtl)) + 16 +
           (DX ? 0 : kPEpiWarps * kDuoBias);
}
static_assert(duo_smem<false>() <= 227 * 1024 && duo_smem<true>() <= 227 * 1024, "shared memory");

struct DuoArgs {
    const void* src;       // rows of tokens: x (y) or d_out (d_x)
    const void* other;     // d_x: x, for the weights' gradient (may be NULL)
    const void* bias;      // y: may be NULL
    const float* weights;  // [T][2]
    const int32_t* start;  // [E * E + 1]
    const int32_t* list;   // [T]
    int E, H;
    int64_t P;
    void* out;             // [T][H]; d_x: may be NULL
    float* dw_part;        // [2][P], d_x with `other`
    uint32_t* flags;
};

template <typename T, bool DX>
__global__ void __launch_bounds__(kPairThreads, 1)
duo_kernel(const __grid_constant__ CUtensorMap tm_w, const DuoArgs A) {
    using C = DuoCfg<DX>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* aring = smem;
    uint8_t* bring = smem + C::A_STAGES * C::A_BYTES;
    uint8_t* stg = smem + C::RING_BYTES;
    DuoCtl* ctl = reinterpret_cast<DuoCtl*>(smem + C::RING_BYTES + C::STG_BYTES);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int H = A.H, KCH = H / 64, NS = (H + 127) / 128, n = A.E * A.E;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::A_STAGES; ++s) {
            mbar_init(&ctl->afull[s], 128);  // 128 gather threads
            mbar_init(&ctl->aempty[s], 1);   // tcgen05.commit
        }
        for (int s = 0; s < C::B_STAGES; ++s) {
            mbar_init(&ctl->bfull[s], 1);    // arrive.expect_tx + TMA bytes
            mbar_init(&ctl->bempty[s], 1);   // tcgen05.commit
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ctl->tfull[b], 1);
            mbar_init(&ctl->tempty[b], kPEpiWarps);
        }
        ctl->abort = 0;
        fence_mbar_init();
    }
    if (warp == kPLoadWarp && lane == 0) tma_prefetch_desc(&tm_w);
    if (warp == kPMmaWarp) {
        tmem_alloc(&ctl->tmem_base, C::TMEM_COLS);
        tmem_relinquish();
    }
    griddep_wait();  // the prologue above overlaps the previous kernel; global memory from here on
    for (int i = threadIdx.x; i <= n; i += kPairThreads) ctl->start[i] = A.start[i];
    __syncthreads();
    if (warp == 0) warp_starts(ctl->tstart, n, [&](int i) { return (ctl->start[i + 1] - ctl->start[i] + 127) / 128; });
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    const int ntiles = ctl->tstart[n];
    volatile int* abort = &ctl->abort;
    auto tile_rows = [&](int tile, int& cls, int& row0, int& nrows) {
        cls = span_of(ctl->tstart, n, tile);
        row0 = ctl->start[cls] + (tile - ctl->tstart[cls]) * 128;
        nrows = min(128, ctl->start[cls + 1] - row0);
    };

    if (warp >= kPProducer0 / 32 && warp < kPProducer0 / 32 + 4) {
        // ---------------- row gather
        const T* src = static_cast<const T*>(A.src);
        const int ptid = threadIdx.x - kPProducer0;
        const int prow = ptid >> 3, pg = ptid & 7;
        int nxt[8];
        const T* row[8];
        unsigned there = 0;
        auto load_codes = [&](int tile, int (&c)[8]) {
            int cls, row0, nrows;
            tile_rows(tile, cls, row0, nrows);
#pragma unroll
            for (int it = 0; it < 8; ++it) c[it] = it * 16 + prow < nrows ? A.list[row0 + it * 16 + prow] : -1;
        };
        auto to_rows = [&](const int (&c)[8]) {
            there = 0;
#pragma unroll
            for (int it = 0; it < 8; ++it) {
                row[it] = src + static_cast<int64_t>(c[it] < 0 ? 0 : c[it] >> 1) * H + pg * 8;
                there |= c[it] < 0 ? 0u : 1u << it;
            }
        };
        if (static_cast<int>(blockIdx.x) < ntiles) {
            load_codes(blockIdx.x, nxt);
            to_rows(nxt);
        }
        const uint32_t to = smem_u32(aring) + prow * 128 + ((pg ^ (prow & 7)) << 4);  // rows 16 apart swizzle alike
        int sa = 0;
        uint32_t pa = 0;
        bool ok = true;
        for (int tile = blockIdx.x; tile < ntiles && ok; tile += gridDim.x) {
            if (tile + static_cast<int>(gridDim.x) < ntiles) load_codes(tile + gridDim.x, nxt);
            for (int kc = 0; kc < KCH; ++kc) {
                if (!(ok = mbar_wait(&ctl->aempty[sa], pa ^ 1, abort, A.flags))) break;
                const uint32_t a_u32 = to + sa * C::A_BYTES;
#pragma unroll
                for (int it = 0; it < 8; ++it)
                    cp_async_16_l2_256(a_u32 + it * 16 * 128, row[it] + kc * 64, (there >> it) & 1u ? 16u : 0u);
                cp_async_arrive_noinc(&ctl->afull[sa]);
                if (++sa == C::A_STAGES) {
                    sa = 0;
                    pa ^= 1;
                }
            }
            to_rows(nxt);
        }
    } else if (warp == kPLoadWarp) {
        // ---------------- weight loader: columns, experts, chunks in the MMAs' order
        {
            const uint32_t leader = elect_one(), ring = smem_u32(bring);
            int sb = 0;
            uint32_t pb = 0;
            bool ok = true;
            for (int tile = blockIdx.x; tile < ntiles && ok; tile += gridDim.x) {
                int cls, row0, nrows;
                tile_rows(tile, cls, row0, nrows);
                const int lo = cls / A.E * H, hi = cls % A.E * H;  // the experts' first rows
                for (int n0 = 0; n0 < H && ok; n0 += 128) {
                    const int ng = min(128, H - n0) / 64;
                    for (int kc = 0; kc < KCH; ++kc) {
                        if (!(ok = warp_wait(&ctl->bempty[sb], pb ^ 1, abort, A.flags))) break;
                        const uint32_t b = ring + sb * C::B_BYTES;
                        if (DX) {
                            expect_f16(leader, &ctl->bfull[sb], 2 * ng * 64 * 128);
                            for (int g = 0; g < ng; ++g) {
                                load_box(leader, b + g * 64 * 128, &tm_w, n0 + g * 64, lo + kc * 64, &ctl->bfull[sb]);
                                load_box(leader, b + (g + 2) * 64 * 128, &tm_w, n0 + g * 64, hi + kc * 64, &ctl->bfull[sb]);
                            }
                        } else {
                            expect_f16(leader, &ctl->bfull[sb], C::B_BYTES);
                            load_box(leader, b, &tm_w, kc * 64, lo + n0, &ctl->bfull[sb]);
                            load_box(leader, b + 128 * 128, &tm_w, kc * 64, hi + n0, &ctl->bfull[sb]);
                        }
                        if (++sb == C::B_STAGES) {
                            sb = 0;
                            pb ^= 1;
                        }
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == kPMmaWarp) {
        // ---------------- MMA issuer: sums of 128 columns of the lower expert at 256 buf, of the higher
        // 128 columns on
        {
            const uint32_t leader = elect_one();
            const uint32_t a0 = desc_lo(smem_u32(aring), 16), b0 = desc_lo(smem_u32(bring), DX ? 64 * 128 : 16);
            int sa = 0, sb = 0;
            uint32_t pa = 0, pb = 0;
            int buf = 0;
            uint32_t buf_phase = 0;
            const uint32_t idesc = idesc_f16<T>(128, 256, 0, DX ? 1 : 0);
            bool ok = true;
            for (int tile = blockIdx.x; tile < ntiles && ok; tile += gridDim.x) {
                for (int ns = 0; ns < NS && ok; ++ns) {
                    if (!(ok = warp_wait(&ctl->tempty[buf], buf_phase ^ 1, abort, A.flags))) break;
                    tc_fence_after();
                    const uint32_t d = tmem + static_cast<uint32_t>(buf * 256);
                    for (int kc = 0; kc < KCH; ++kc) {
                        const int a = sa + kc >= C::A_STAGES ? sa + kc - C::A_STAGES : sa + kc;
                        const uint32_t ph = pa ^ (sa + kc >= C::A_STAGES ? 1u : 0u);
                        ok = ns == 0 ? warp_wait_both(&ctl->afull[a], ph, &ctl->bfull[sb], pb, abort, A.flags)
                                     : warp_wait(&ctl->bfull[sb], pb, abort, A.flags);
                        if (!ok) break;
                        fence_proxy_async_smem();
                        tc_fence_after();
                        const uint32_t al = a0 + a * (C::A_BYTES >> 4), bl = b0 + sb * (C::B_BYTES >> 4);
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            mma_f16(leader, d, al + ks * kKStep, kDescHi, bl + ks * (DX ? kMnStep : kKStep), kDescHi, idesc, ks != 0 ? 1u : kc != 0);
                        commit_f16(leader, &ctl->bempty[sb]);
                        if (ns == NS - 1) commit_f16(leader, &ctl->aempty[a]);
                        if (++sb == C::B_STAGES) {
                            sb = 0;
                            pb ^= 1;
                        }
                    }
                    if (!ok) break;
                    commit_f16(leader, &ctl->tfull[buf]);
                    buf ^= 1;
                    if (buf == 0) buf_phase ^= 1;
                }
                sa += KCH;
                if (sa >= C::A_STAGES) {
                    sa -= C::A_STAGES;
                    pa ^= 1;
                }
            }
        }
        __syncwarp();
    } else if (warp < kPEpiWarps) {
        // ---------------- epilogue: this lane's row is 32 (w % 4) + lane; columns of half w / 4 of
        // every 128, 32 a step
        const int q = warp & 3, half = warp >> 2;
        const uint32_t my = smem_u32(stg + warp * C::STEP_BYTES * (DX ? 2 : 1));
        const int myrow = 32 * q + lane;
        const int R4 = lane >> 2, j4 = lane & 3;
        const uint32_t swz = (lane >> 1) & 3;
        T* out = static_cast<T*>(A.out);
        auto tile_code = [&](int tile) -> int {
            int cls, row0, nrows;
            tile_rows(tile, cls, row0, nrows);
            return myrow < nrows ? A.list[row0 + myrow] : -1;
        };
        auto fetch_x = [&](int code, int col, int b) {  // as in pair_kernel
            const T* xs = static_cast<const T*>(A.other);
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const int R = it * 8 + R4;
                const int c = __shfl_sync(kFull, code, R);
                cp_async_16(my + b * C::STEP_BYTES + R * 64 + ((j4 ^ ((R >> 1) & 3)) << 4),
                            xs + static_cast<int64_t>(c < 0 ? 0 : c >> 1) * H + col + j4 * 8, c < 0 ? 0u : 16u);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // the warp's steps of a tile: columns 128 ns + 64 half + 32 i below H
        const int first_col = half * 64;
        const uint32_t sbias = ((smem_u32(ctl) + static_cast<uint32_t>(sizeof(DuoCtl)) + 15) & ~15u) + warp * kDuoBias;
        int tile = blockIdx.x;
        int next = tile < ntiles ? tile_code(tile) : -1;
        int xb = 0;
        if (DX && A.other && tile < ntiles && first_col < H) fetch_x(next, first_col, 0);
        int buf = 0;
        uint32_t buf_phase = 0;
        bool ok = true;
        for (; tile < ntiles && ok; tile += gridDim.x) {
            const int code = next, next_tile = tile + gridDim.x;
            // weight of the lower expert, of the higher
            const float wl = code >= 0 ? A.weights[code] : 0.0f, wh = code >= 0 ? A.weights[code ^ 1] : 0.0f;
            if (next_tile < ntiles) next = tile_code(next_tile);
            if (!DX && A.bias) {
                // eight columns a lane: expert lane / 16, columns 128 ns + 64 half + 8 (lane % 8)
                const int cls = span_of(ctl->tstart, n, tile);
                const int e = lane < 16 ? cls / A.E : cls % A.E, c = 128 * ((lane >> 3) & 1) + 64 * half + 8 * (lane & 7);
                Chunk<T, 8> b{};
                if (c < H) b = *reinterpret_cast<const Chunk<T, 8>*>(static_cast<const T*>(A.bias) + static_cast<int64_t>(e) * H + c);
                const uint32_t to = sbias + (lane >> 3) * 256 + 32 * (lane & 7);
                st_shared_v4(to, to_f(b.v[0]), to_f(b.v[1]), to_f(b.v[2]), to_f(b.v[3]));
                st_shared_v4(to + 16, to_f(b.v[4]), to_f(b.v[5]), to_f(b.v[6]), to_f(b.v[7]));
                __syncwarp();
            }
            uint8_t* dst[4];
            unsigned there = 0;
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const int c = __shfl_sync(kFull, code, it * 8 + R4);
                there |= c >= 0 ? 1u << it : 0u;
                dst[it] = reinterpret_cast<uint8_t*>(out) + (static_cast<int64_t>(c < 0 ? 0 : c >> 1) * H + j4 * 8) * 2;
            }
            float dl = 0.0f, dh = 0.0f;
            for (int ns = 0; ns < NS && ok; ++ns) {
                if (!(ok = mbar_wait(&ctl->tfull[buf], buf_phase, abort, A.flags))) break;
                __syncwarp();
                tc_fence_after();
                const uint32_t tb = tmem + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(buf * 256 + half * 64);
                const int steps = min(2, (H - ns * 128 - half * 64) / 32);  // 0 or 2: H is a multiple of 64
                for (int i = 0; i < steps; ++i) {
                    const int col = ns * 128 + half * 64 + 32 * i;
                    uint32_t ta[32], th[32];
                    tmem_ld_32x32b_x32_async(tb + 32 * i, ta);
                    tmem_ld_32x32b_x32_async(tb + 128 + 32 * i, th);
                    const uint32_t stage = my + (DX ? xb * C::STEP_BYTES : 0);
                    if (DX && A.other) {
                        // the next step's rows of x: of this tile, or the first of the next
                        const int ncol = i == 0 ? col + 32 : col + 96;
                        if (ncol < H) fetch_x(code, ncol, xb ^ 1);
                        else if (next_tile < ntiles) fetch_x(next, first_col, xb ^ 1);
                        else asm volatile("cp.async.commit_group;" ::: "memory");
                    }
                    tmem_ld_wait_tied(ta);
                    tmem_ld_wait_tied(th);
                    if (i == 1) {  // the columns are read: the next ones may have the accumulators
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&ctl->tempty[buf]);
                    }
                    if (DX) {
                        if (A.other) {
                            asm volatile("cp.async.wait_group 1;" ::: "memory");
                            __syncwarp();
#pragma unroll
                            for (int g = 0; g < 4; ++g) {
                                const uint4 raw = ld_shared_u4(stage + lane * 64 + ((g ^ swz) << 4));
                                const T* xv = reinterpret_cast<const T*>(&raw);
#pragma unroll
                                for (int j = 0; j < 8; ++j) {
                                    const float xf = to_f(xv[j]);
                                    dl += __uint_as_float(ta[8 * g + j]) * xf;
                                    dh += __uint_as_float(th[8 * g + j]) * xf;
                                }
                            }
                        }
                        xb ^= 1;
                        if (!out) {
                            __syncwarp();
                            continue;
                        }
                    }
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        float s[8];
                        if (!DX && A.bias) {
                            // the same words for every lane; the higher expert's 512 bytes on
                            const uint32_t from = sbias + ns * 256 + (32 * i + 8 * g) * 4;
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const float4 bl = ld_shared_v4(from + 16 * h), bh = ld_shared_v4(from + 512 + 16 * h);
                                const int j = 8 * g + 4 * h;
                                s[4 * h] = wl * (__uint_as_float(ta[j]) + bl.x) + wh * (__uint_as_float(th[j]) + bh.x);
                                s[4 * h + 1] = wl * (__uint_as_float(ta[j + 1]) + bl.y) + wh * (__uint_as_float(th[j + 1]) + bh.y);
                                s[4 * h + 2] = wl * (__uint_as_float(ta[j + 2]) + bl.z) + wh * (__uint_as_float(th[j + 2]) + bh.z);
                                s[4 * h + 3] = wl * (__uint_as_float(ta[j + 3]) + bl.w) + wh * (__uint_as_float(th[j + 3]) + bh.w);
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                s[j] = wl * __uint_as_float(ta[8 * g + j]) + wh * __uint_as_float(th[8 * g + j]);
                        }
                        st_shared_u4(stage + lane * 64 + ((g ^ swz) << 4), pack8<T>(s));
                    }
                    __syncwarp();
#pragma unroll
                    for (int it = 0; it < 4; ++it) {
                        const int R = it * 8 + R4;
                        const uint4 val = ld_shared_u4(stage + R * 64 + ((j4 ^ ((R >> 1) & 3)) << 4));
                        if ((there >> it) & 1u) *reinterpret_cast<uint4*>(dst[it] + 2 * col) = val;
                    }
                    __syncwarp();
                }
                if (steps == 0) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl->tempty[buf]);
                }
                buf ^= 1;
                if (buf == 0) buf_phase ^= 1;
            }
            if (DX && A.other && ok && code >= 0) {
                A.dw_part[static_cast<int64_t>(half) * A.P + code] = dl;
                A.dw_part[static_cast<int64_t>(half) * A.P + (code ^ 1)] = dh;
            }
        }
        if (DX) asm volatile("cp.async.wait_all;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kPMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// ---------------------------------------------------------------- join
struct JoinArgs {
    const float* rows;     // [P][H]
    void* out;             // [T][H], or NULL
    const float* dw_part;  // [parts][P]; d_weights only
    int parts;
    const void* g;         // [T][H]: d_weights, with bias
    const void* bias;      // [E][H] or NULL: added to the forward's rows, part of d_weights
    const int32_t* expert_idx;
    const float* weights;  // [P]: forward, with bias
    float* d_weights;      // [P] or NULL (the forward)
    int64_t T;
    int K, H;
};

// LPT lanes per token, four columns each at a time; U tokens per turn, so that enough loads
// are on the way; KM: an upper bound of K. DW: the backward (d_weights may be NULL).
template <typename T, int KM, int U, bool DW>
__global__ void __launch_bounds__(256, KM <= 4 ? 4 : 2) join_kernel(const JoinArgs A, int LPT) {
    griddep_wait();  // every global access below comes after the previous grid
    const int lane = threadIdx.x & 31, sub = lane % LPT, K = A.K, H = A.H, per_warp = 32 / LPT;
    const int64_t P = A.T * K;
    const bool with_bias = A.bias != nullptr, rows = A.out != nullptr;
    const int64_t step = static_cast<int64_t>(gridDim.x) * 8 * per_warp * U;
    // a warp's tokens run in step: lanes past the last token only take part in the shuffles
    for (int64_t base = (static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * per_warp * U; base < A.T; base += step) {
        int64_t t[U];
        const T* br[U][KM];
        float wk[U][KM], dot[U][KM];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            t[u] = base + u * per_warp + lane / LPT;
#pragma unroll
            for (int k = 0; k < KM; ++k) {
                const bool on = with_bias && t[u] < A.T && k < K;
                br[u][k] = static_cast<const T*>(A.bias) + (on ? static_cast<int64_t>(A.expert_idx[t[u] * K + k]) * H : 0);
                wk[u][k] = !DW && on ? A.weights[t[u] * K + k] : 0.0f;
                dot[u][k] = 0.0f;
            }
        }
        for (int c = sub * 4; c < H; c += LPT * 4) {
            Chunk<float, 4> r[U][KM];
            Chunk<T, 4> gv[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (t[u] >= A.T) continue;
                if (rows)
#pragma unroll
                    for (int k = 0; k < KM; ++k)
                        if (k < K) r[u][k] = *reinterpret_cast<const Chunk<float, 4>*>(A.rows + (t[u] * K + k) * H + c);
                if (DW && with_bias) gv[u] = *reinterpret_cast<const Chunk<T, 4>*>(static_cast<const T*>(A.g) + t[u] * H + c);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (t[u] >= A.T) continue;
                float s[4] = {0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < KM; ++k) {
                    if (k >= K) continue;
                    if (rows)
#pragma unroll
                        for (int i = 0; i < 4; ++i) s[i] += r[u][k].v[i];
                    if (with_bias) {
                        const Chunk<T, 4> bv = *reinterpret_cast<const Chunk<T, 4>*>(br[u][k] + c);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (DW) dot[u][k] += to_f(gv[u].v[i]) * to_f(bv.v[i]);
                            else s[i] = fmaf(to_f(bv.v[i]), wk[u][k], s[i]);
                        }
                    }
                }
                if (rows) {
                    Chunk<T, 4> o;
#pragma unroll
                    for (int i = 0; i < 4; ++i) o.v[i] = from_f<T>(s[i]);
                    *reinterpret_cast<Chunk<T, 4>*>(static_cast<T*>(A.out) + t[u] * H + c) = o;
                }
            }
        }
        if (DW && A.d_weights) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int k = 0; k < KM; ++k) {
                    if (k >= K) continue;
                    float d = dot[u][k];
                    if (t[u] < A.T)
                        for (int i = sub; i < A.parts; i += LPT) d += A.dw_part[i * P + t[u] * K + k];
                    for (int off = LPT / 2; off >= 1; off >>= 1) d += __shfl_xor_sync(kFull, d, off);
                    if (t[u] < A.T && sub == 0) A.d_weights[t[u] * K + k] = d;
                }
        }
    }
}

// ---------------------------------------------------------------- dW and db
// Warps 0-7 scale the rows of g and drain the sums, 8-11 gather, 12 issues the MMAs, 13
// looks pairs up.
constexpr int kWThreads = 448;
constexpr int kWGather0 = 8, kWMmaWarp = 12, kWLookWarp = 13;
constexpr int kMaxPieces = kMaxE + kWUnits;

struct WCfg {
    static constexpr int KT = 32;              // pairs per stage
    static constexpr int RW = KT / 4;          // rows of a stage a warp gathers, or scales
    static constexpr int GROUP = KT * 128;     // 64 columns of a stage's rows
    static constexpr int OP = 4 * GROUP;       // 256 columns
    static constexpr int STAGE = 3 * OP;       // w g's upper part (before: g), x, w g's lower part: 48 KiB
    static constexpr int STAGES = 4;
    static constexpr int STG = 8 * 32 * 64;    // staging: 32 rows x 64 bytes a warp
    static constexpr int LOOK = 128;           // pairs looked up at a time
    static constexpr int LOOKS = 3;            // blocks of them on the way
    static constexpr int STEPS = LOOK / KT;    // stages of a block
};

struct __align__(16) WCtl {
    int64_t row[WCfg::LOOKS][WCfg::LOOK];  // first element of the pair's token
    float weight[WCfg::LOOKS][WCfg::LOOK];
    uint64_t raw[WCfg::STAGES], full[WCfg::STAGES], empty[WCfg::STAGES];
    uint64_t lfull[WCfg::LOOKS], lempty[WCfg::LOOKS];
    uint64_t tfull, tempty;
    uint32_t tmem_base;
    int abort;
    int off[kMaxE + 1];
    int pstart[kMaxE + 1];  // first piece of each expert
    int sstart[kMaxE + 1];  // first slot of each expert (experts of two pieces or more)
    uint16_t order[kMaxPieces + 4];  // pieces, most pairs first
    float db[8][32][8];
};
constexpr int kWSmem = 1024 + WCfg::STAGES * WCfg::STAGE + WCfg::STG + static_cast<int>(sizeof(WCtl));
static_assert(kWSmem <= 227 * 1024, "shared memory");

struct WgradArgs {
    const void* x;
    const void* g;
    const float* weights;
    const int32_t* offsets;
    const int32_t* perm;
    int E, K, H, extra;
    DivK by_k;
    int64_t P;
    void* dW;       // may be NULL (db only)
    void* db;       // may be NULL
    float* part;    // [slots][H][H]
    float* part_db; // [slots][H]
    int32_t* starts;  // [E + 1]: first slot of each expert, for wgrad_sum_kernel
    uint32_t* peak;   // [E], fp16 with dW: see wgrad_peak_kernel
    uint32_t* flags;
};

// fp16: w g is staged times a power of two per expert that brings the expert's largest finite
// |w g| to [2^14, 2^15), and the sums are divided by it. Unscaled, a term above 65,504 would
// be infinite and one below 6e-5 would lose its bits, though dW itself is in range. `peak`: the
// bits of that largest value; below 2^-112 the factor stays at 2^126, the largest that has an inverse.
__device__ __forceinline__ int peak_exponent(uint32_t peak) { return max(static_cast<int>(peak >> 23), 15); }
__device__ __forceinline__ float peak_factor(uint32_t peak) {
    return __uint_as_float(static_cast<uint32_t>(268 - peak_exponent(peak)) << 23);
}
__device__ __forceinline__ float peak_inverse(uint32_t peak) {
    return __uint_as_float(static_cast<uint32_t>(peak_exponent(peak) - 14) << 23);
}

// peak[e] (zeroed): bits of the largest finite |w g| over the pairs of expert e. A warp takes
// eight slots of perm, a lane each, reads their rows of g and leaves one maximum per expert.
// Bound by L2: K reads of g. fp16 only; 16,384 tokens, K 2, H 1024: 16 us.
constexpr int kPeakSlots = 8;  // of a warp at a time: 32 of them leave most of the GPU idle (38 us)
__global__ void __launch_bounds__(256) wgrad_peak_kernel(const WgradArgs A) {
    griddep_wait();  // every global access below comes after the previous grid
    __shared__ int off[kMaxE + 1];
    for (int e = threadIdx.x; e <= A.E; e += 256) off[e] = A.offsets[e];
    __syncthreads();
    const int lane = threadIdx.x & 31;
    const int64_t step = static_cast<int64_t>(gridDim.x) * 8 * kPeakSlots;
    for (int64_t base = (static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * kPeakSlots; base < A.P; base += step) {
        const bool valid = lane < kPeakSlots && base + lane < A.P;
        const int pair = valid ? A.perm[base + lane] : 0;
        const float w = valid ? fabsf(A.weights[pair]) : 0.0f;
        const int e = valid ? span_of(off, A.E, static_cast<int>(base) + lane) : -1;
        const int n = static_cast<int>(A.P - base < kPeakSlots ? A.P - base : kPeakSlots), token = A.by_k(pair);
        uint32_t mine = 0;  // the largest finite |g| of this lane's row, as fp16
        for (int i = 0; i < n; ++i) {
            const int t = __shfl_sync(kFull, token, i);
            const uint4* row = reinterpret_cast<const uint4*>(static_cast<const __half*>(A.g) + static_cast<int64_t>(t) * A.H);
            uint32_t m = 0;
            for (int c = lane; c < A.H / 8; c += 32) {
                const uint4 v = __ldg(row + c);
                const uint32_t word[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t a = word[j] & 0x7fff7fffu;
                    m = __vmaxu2(m, a & __vcmpltu2(a, 0x7c007c00u));
                }
            }
            m = __reduce_max_sync(kFull, max(m & 0xffffu, m >> 16));
            if (lane == i) mine = m;
        }
        float peak = w < INFINITY ? w * __half2float(__ushort_as_half(static_cast<unsigned short>(mine))) : 0.0f;
        if (peak == INFINITY) peak = 3e38f;
        const unsigned same = __match_any_sync(kFull, e);
        const uint32_t most = __reduce_max_sync(same, __float_as_uint(peak));
        if (e >= 0 && most != 0 && lane == __ffs(same) - 1) atomicMax(&A.peak[e], most);
    }
}

// Pieces and slots of every expert, from the offsets in shared memory (warp 0).
template <typename CtlT>
__device__ __forceinline__ void piece_starts(CtlT* ctl, int E, int64_t P, int extra) {
    warp_starts(ctl->pstart, E, [&](int e) { return wgrad_pieces(ctl->off[e + 1] - ctl->off[e], P, extra); });
    warp_starts(ctl->sstart, E, [&](int e) {
        const int n = wgrad_pieces(ctl->off[e + 1] - ctl->off[e], P, extra);
        return n > 1 ? n : 0;
    });
}

struct Unit {
    int e, piece, pieces, lo, hi, o0, i0;
};

// Two 16-bit numbers that add up to s: the upper one is s cut off, always of a smaller
// magnitude, the lower one the rest, rounded (16 bits of s for bf16; 22 for fp16, down to its
// last step, 2^-39 of the expert's largest). So both have the sign of s, and an infinite x times
// either is the same infinity; an infinite s is infinite in both. Masks rather than conversions back and forth: 127 us instead of 141 for
// dW alone at the size above, 110 without any of this arithmetic.
template <typename T>
__device__ __forceinline__ void split8(const float (&s)[8], uint4& hi, uint4& lo) {
    constexpr uint32_t kKeep = std::is_same<T, __half>::value ? 0xffffe000u : 0xffff0000u;
    float h[8], l[8], most = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        h[i] = __uint_as_float(__float_as_uint(s[i] * (1.0f - 0x1p-24f)) & kKeep);
        l[i] = s[i] - h[i];
        most = fmaxf(most, fabsf(s[i]));
    }
    if (most == INFINITY) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (fabsf(s[i]) == INFINITY) l[i] = s[i];
    }
    hi = pack8<T>(h);
    lo = pack8<T>(l);
}

template <typename T>
__global__ void __launch_bounds__(kWThreads, 1) wgrad_kernel(const WgradArgs A) {
    using C = WCfg;
    constexpr bool kScaled = std::is_same<T, __half>::value;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* stg = smem + C::STAGES * C::STAGE;
    WCtl* ctl = reinterpret_cast<WCtl*>(smem + C::STAGES * C::STAGE + C::STG);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int H = A.H;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&ctl->raw[s], 128);  // the gather threads' copies
            mbar_init(&ctl->full[s], 4);   // the four warps that scale it
            mbar_init(&ctl->empty[s], 1);  // tcgen05.commit
        }
        for (int s = 0; s < C::LOOKS; ++s) {
            mbar_init(&ctl->lfull[s], 32);      // the looking lanes
            mbar_init(&ctl->lempty[s], 8 + 4);  // scaling and gather warps
        }
        mbar_init(&ctl->tfull, 1);
        mbar_init(&ctl->tempty, 8);
        ctl->abort = 0;
        fence_mbar_init();
    }
    if (warp == kWMmaWarp) {
        tmem_alloc(&ctl->tmem_base, 512);
        tmem_relinquish();
    }
    griddep_wait();  // the prologue above overlaps the previous kernel; global memory from here on
    for (int e = threadIdx.x; e <= A.E; e += kWThreads) ctl->off[e] = A.offsets[e];
    __syncthreads();
    if (warp == 0) piece_starts(ctl, A.E, A.P, A.extra);
    __syncthreads();
    const int npieces = ctl->pstart[A.E];  // at most E + extra
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e <= A.E; e += kWThreads) A.starts[e] = ctl->sstart[e];
    // The pieces by size, largest first: the blocks take units in turns that run back and forth, so
    // that a large unit is followed by a small one. The stages hold the sizes meanwhile.
    int* sizes = reinterpret_cast<int*>(smem);
    for (int i = threadIdx.x; i < npieces; i += kWThreads) {
        const int e = span_of(ctl->pstart, A.E, i), n = ctl->off[e + 1] - ctl->off[e], q = ctl->pstart[e + 1] - ctl->pstart[e];
        sizes[i] = (n + q - 1) / q;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < npieces; i += kWThreads) {
        const int mine = sizes[i];
        int rank = 0;
        for (int o = 0; o < npieces; ++o) rank += (sizes[o] > mine || (sizes[o] == mine && o < i)) ? 1 : 0;
        ctl->order[rank] = static_cast<uint16_t>(i);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    volatile int* abort = &ctl->abort;
    const int nt = (H + kWTile - 1) / kWTile, tiles = nt * nt;
    const int nunits = npieces * tiles;
    // the block's unit of a turn, -1 after the last
    auto unit_number = [&](int turn) {
        const int g = static_cast<int>(gridDim.x), b = static_cast<int>(blockIdx.x);
        const int64_t u = static_cast<int64_t>(turn) * g + ((turn & 1) ? g - 1 - b : b);
        return u < nunits ? static_cast<int>(u) : -1;
    };
    auto unit_of = [&](int u) {
        Unit r;
        const int piece = ctl->order[u / tiles], tile = u % tiles;
        r.e = span_of(ctl->pstart, A.E, piece);
        r.pieces = ctl->pstart[r.e + 1] - ctl->pstart[r.e];
        r.piece = piece - ctl->pstart[r.e];
        const int64_t n = ctl->off[r.e + 1] - ctl->off[r.e];
        r.lo = ctl->off[r.e] + static_cast<int>(n * r.piece / r.pieces);
        r.hi = ctl->off[r.e] + static_cast<int>(n * (r.piece + 1) / r.pieces);
        r.o0 = (tile / nt) * kWTile;
        r.i0 = (tile % nt) * kWTile;
        return r;
    };

    if (warp == kWLookWarp) {
        // ---------------- lookup: tokens and weights of the pairs, up to three blocks ahead of the rows;
        // a block's pairs are read two blocks ahead of its tokens' entry, its weights one
        constexpr int N = C::LOOK / 32;
        int slot = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int turn = 0, u; ok && (u = unit_number(turn)) >= 0; ++turn) {
            const Unit r = unit_of(u);
            int p0[N], p1[N];
            float w0[N];
            auto pairs = [&](int at, int (&p)[N]) {
#pragma unroll
                for (int i = 0; i < N; ++i) p[i] = at + 32 * i + lane < r.hi ? A.perm[at + 32 * i + lane] : -1;
            };
            auto weights = [&](const int (&p)[N], float (&w)[N]) {
#pragma unroll
                for (int i = 0; i < N; ++i) w[i] = p[i] >= 0 ? A.weights[p[i]] : 0.0f;
            };
            const float f = kScaled && A.peak ? peak_factor(A.peak[r.e]) : 1.0f;
            auto scaled = [&](float w) {  // a finite weight stays finite (of a row of zeros, else f w is below 2^39)
                return !kScaled ? w : fabsf(w) < INFINITY ? fminf(fmaxf(w * f, -3e38f), 3e38f) : w;
            };
            pairs(r.lo, p0);
            pairs(r.lo + C::LOOK, p1);
            weights(p0, w0);
            for (int at = r.lo; at < r.hi; at += C::LOOK) {
                int p2[N];
                float w1[N];
                pairs(at + 2 * C::LOOK, p2);
                weights(p1, w1);
                if (!(ok = mbar_wait(&ctl->lempty[slot], phase ^ 1, abort, A.flags))) break;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    ctl->row[slot][32 * i + lane] = p0[i] < 0 ? 0 : static_cast<int64_t>(A.by_k(p0[i])) * H;
                    ctl->weight[slot][32 * i + lane] = scaled(w0[i]);
                    p0[i] = p1[i];
                    p1[i] = p2[i];
                    w0[i] = w1[i];
                }
                mbar_arrive(&ctl->lfull[slot]);
                if (++slot == C::LOOKS) {
                    slot = 0;
                    phase ^= 1;
                }
            }
        }
    } else if (warp >= kWGather0 && warp < kWGather0 + 4) {
        // ---------------- gather: rows of g and x as they are, MN-major; a warp moves a row of 256
        // columns at a time; rows past the piece's end are zeros
        const T* g = static_cast<const T*>(A.g);
        const T* x = static_cast<const T*>(A.x);
        const int w4 = warp - kWGather0;
        int stage = 0, slot = 0;
        uint32_t phase = 0, lphase = 0;
        bool ok = true;
        // a warp has rows RW w4 .. of a stage: row i of them swizzles by i % 8
        uint32_t to[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            to[i] = smem_u32(smem) + (lane >> 3) * C::GROUP + (C::RW * w4 + i) * 128 + (((lane & 7) ^ i) << 4);
        for (int turn = 0, u; ok && (u = unit_number(turn)) >= 0; ++turn) {
            const Unit r = unit_of(u);
            const bool on_g = lane * 8 < min(kWTile, H - r.o0), on_x = lane * 8 < min(kWTile, H - r.i0);
            const T* gl = g + r.o0 + (on_g ? lane * 8 : 0);
            const T* xl = x + r.i0 + (on_x ? lane * 8 : 0);
            for (int at = r.lo; ok && at < r.hi; at += C::LOOK) {
                if (!(ok = mbar_wait(&ctl->lfull[slot], lphase, abort, A.flags))) break;
                const int steps = min(C::STEPS, (r.hi - at + C::KT - 1) / C::KT);
                for (int st = 0; st < steps; ++st) {
                    longlong2 rows[C::RW / 2];
#pragma unroll
                    for (int i = 0; i < C::RW / 2; ++i)
                        rows[i] = *reinterpret_cast<const longlong2*>(&ctl->row[slot][st * C::KT + C::RW * w4 + 2 * i]);
                    const int left = r.hi - at - st * C::KT - C::RW * w4;  // rows of the warp that are pairs
                    if (!(ok = mbar_wait(&ctl->empty[stage], phase ^ 1, abort, A.flags))) break;
                    const uint32_t base = stage * C::STAGE;
#pragma unroll
                    for (int i = 0; i < C::RW; ++i) {
                        const int64_t row = (i & 1) ? rows[i / 2].y : rows[i / 2].x;
                        const uint32_t bytes = i < left ? 16u : 0u, at_i = to[i & 7] + (i >> 3) * 1024 + base;
                        if (on_g) cp_async_16(at_i, gl + row, bytes);
                        if (on_x) cp_async_16(at_i + C::OP, xl + row, bytes);
                    }
                    cp_async_arrive_noinc(&ctl->raw[stage]);
                    if (++stage == C::STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->lempty[slot]);
                if (++slot == C::LOOKS) {
                    slot = 0;
                    lphase ^= 1;
                }
            }
        }
    } else if (warp == kWMmaWarp) {
        // ---------------- MMA issuer: two halves of 128 rows of dW, the tile's columns
        {
            const uint32_t leader = elect_one();
            const uint32_t g0 = desc_lo(smem_u32(smem), C::GROUP);
            int stage = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            for (int turn = 0, u; ok && (u = unit_number(turn)) >= 0; ++turn) {
                const Unit r = unit_of(u);
                const int halves = (min(kWTile, H - r.o0) + 127) / 128;
                const uint32_t idesc = idesc_f16<T>(128, min(kWTile, H - r.i0), 1, 1);
                if (!(ok = warp_wait(&ctl->tempty, acc_phase ^ 1, abort, A.flags))) break;
                tc_fence_after();
                for (int p0 = r.lo; p0 < r.hi; p0 += C::KT) {
                    if (!(ok = warp_wait(&ctl->full[stage], phase, abort, A.flags))) break;
                    fence_proxy_async_smem();
                    tc_fence_after();
                    const uint32_t gl = g0 + stage * (C::STAGE >> 4), xl = gl + (C::OP >> 4);
#pragma unroll
                    for (int ks = 0; ks < C::KT / 16; ++ks) {
                        const uint32_t on = ks != 0 ? 1u : p0 != r.lo;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (h >= halves) break;
                            const uint32_t a = gl + (2 * h * C::GROUP >> 4) + ks * kMnStep;
                            mma_f16(leader, tmem + 256 * h, a, kDescHi, xl + ks * kMnStep, kDescHi, idesc, on);
                            mma_f16(leader, tmem + 256 * h, a + (2 * C::OP >> 4), kDescHi, xl + ks * kMnStep, kDescHi, idesc, 1u);
                        }
                    }
                    commit_f16(leader, &ctl->empty[stage]);
                    if (++stage == C::STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
                commit_f16(leader, &ctl->tfull);
                acc_phase ^= 1;
            }
        }
        __syncwarp();
    } else if (warp < 8) {
        // ---------------- scale the staged rows of g in place (db on the way), then drain dW: rows
        // 32 (w % 4) + lane of each half, columns of half w / 4
        const int q = warp & 3, ch = warp >> 2;
        const uint32_t my = smem_u32(stg + warp * 32 * 64);
        int stage = 0, slot = 0;
        uint32_t phase = 0, lphase = 0, acc_phase = 0;
        bool ok = true;
        T* dW = static_cast<T*>(A.dW);
        // warps 0-3 and 4-7 scale stages in turn, so that one stage's latency hides behind the other's;
        // rows RW q .., row i of them swizzled by i % 8
        int turns = 0;
        uint32_t to[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            to[i] = smem_u32(smem) + (lane >> 3) * C::GROUP + (C::RW * q + i) * 128 + (((lane & 7) ^ i) << 4);
        for (int turn = 0, u; (u = unit_number(turn)) >= 0; ++turn) {
            const Unit r = unit_of(u);
            const int rows = min(kWTile, H - r.o0), cols = min(kWTile, H - r.i0);
            const bool on = lane * 8 < rows;
            const bool add = A.db && r.i0 == 0;
            const float inv = kScaled && A.peak ? peak_inverse(A.peak[r.e]) : 1.0f;
            float db[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            for (int at = r.lo; ok && at < r.hi; at += C::LOOK) {
                if (!(ok = mbar_wait(&ctl->lfull[slot], lphase, abort, A.flags))) break;
                const int steps = min(C::STEPS, (r.hi - at + C::KT - 1) / C::KT);
                for (int st = 0; st < steps; ++st) {
                    if ((turns++ & 1) == ch) {
                        if (!(ok = mbar_wait(&ctl->raw[stage], phase, abort, A.flags))) break;
#pragma unroll
                        for (int h = 0; h < C::RW / 8; ++h) {
                            float wr[8];
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const float4 w4 = *reinterpret_cast<const float4*>(&ctl->weight[slot][st * C::KT + C::RW * q + 8 * h + 4 * i]);
                                wr[4 * i] = w4.x;
                                wr[4 * i + 1] = w4.y;
                                wr[4 * i + 2] = w4.z;
                                wr[4 * i + 3] = w4.w;
                            }
                            const uint32_t base = stage * C::STAGE + h * 1024;
                            if (on) {
                                uint4 raw[8];
#pragma unroll
                                for (int i = 0; i < 8; ++i) raw[i] = ld_shared_u4(to[i] + base);
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    const T* v = reinterpret_cast<const T*>(&raw[i]);
                                    float s[8];
#pragma unroll
                                    for (int j = 0; j < 8; ++j) s[j] = wr[i] * to_f(v[j]);
                                    if (add)
#pragma unroll
                                        for (int j = 0; j < 8; ++j) db[j] += s[j];
                                    uint4 upper, lower;
                                    split8<T>(s, upper, lower);
                                    st_shared_u4(to[i] + base, upper);
                                    st_shared_u4(to[i] + base + 2 * C::OP, lower);
                                }
                            }
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&ctl->full[stage]);
                    }
                    if (++stage == C::STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->lempty[slot]);
                if (++slot == C::LOOKS) {
                    slot = 0;
                    lphase ^= 1;
                }
            }
            if (add) {
                // the eight warps' sums, in order (warps that gave up come here too: the barrier counts them)
                asm volatile("bar.sync 1, 256;" ::: "memory");
#pragma unroll
                for (int j = 0; j < 8; ++j) ctl->db[warp][lane][j] = db[j];
                asm volatile("bar.sync 1, 256;" ::: "memory");
                if (warp == 0 && on) {
                    for (int k = 1; k < 8; ++k)
#pragma unroll
                        for (int j = 0; j < 8; ++j) db[j] += ctl->db[k][lane][j];
                    if (kScaled)
#pragma unroll
                        for (int j = 0; j < 8; ++j) db[j] *= inv;
                    const int o = r.o0 + lane * 8;
                    if (r.pieces == 1) {
                        *reinterpret_cast<uint4*>(static_cast<T*>(A.db) + static_cast<int64_t>(r.e) * H + o) = pack8<T>(db);
                    } else {
                        float* d = A.part_db + (static_cast<int64_t>(ctl->sstart[r.e]) + r.piece) * H + o;
#pragma unroll
                        for (int j = 0; j < 8; ++j) d[j] = db[j];
                    }
                }
            }
            if (!ok || !(ok = mbar_wait(&ctl->tfull, acc_phase, abort, A.flags))) continue;
            __syncwarp();
            tc_fence_after();
            for (int mh = 0; mh < (rows + 127) / 128 && dW; ++mh) {
                const int o_first = mh * 128 + 32 * q;
                if (o_first >= rows) break;  // rows is a multiple of 64, so a warp's 32 are in or out together
                for (int c = ch * 128; c < min(cols, ch * 128 + 128); c += 32) {
                    float v[32];
                    tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(mh * 256 + c), v);
                    if (kScaled)
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] *= inv;
                    if (r.pieces == 1) {
                        // 32 rows x 64 bytes through shared memory: 4 lanes a row, 8 rows an instruction
#pragma unroll
                        for (int gg = 0; gg < 4; ++gg) {
                            float s[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) s[i] = v[8 * gg + i];
                            st_shared_u4(my + lane * 64 + ((gg ^ ((lane >> 1) & 3)) << 4), pack8<T>(s));
                        }
                        __syncwarp();
#pragma unroll
                        for (int it = 0; it < 4; ++it) {
                            const int R = it * 8 + (lane >> 2), j = lane & 3;
                            const uint4 val = ld_shared_u4(my + R * 64 + ((j ^ ((R >> 1) & 3)) << 4));
                            const int64_t o = r.o0 + o_first + R;
                            *reinterpret_cast<uint4*>(dW + (static_cast<int64_t>(r.e) * H + o) * H + r.i0 + c + j * 8) = val;
                        }
                        __syncwarp();
                    } else {
                        // fp32 sums of this piece, two steps of 16 columns
                        const int64_t slot = static_cast<int64_t>(ctl->sstart[r.e]) + r.piece;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
#pragma unroll
                            for (int gg = 0; gg < 4; ++gg)
                                st_shared_v4(my + lane * 64 + ((gg ^ ((lane >> 1) & 3)) << 4), v[16 * h + 4 * gg],
                                             v[16 * h + 4 * gg + 1], v[16 * h + 4 * gg + 2], v[16 * h + 4 * gg + 3]);
                            __syncwarp();
#pragma unroll
                            for (int it = 0; it < 4; ++it) {
                                const int R = it * 8 + (lane >> 2), j = lane & 3;
                                const float4 val = ld_shared_v4(my + R * 64 + ((j ^ ((R >> 1) & 3)) << 4));
                                const int64_t o = r.o0 + o_first + R;
                                *reinterpret_cast<float4*>(A.part + (slot * H + o) * H + r.i0 + c + 16 * h + j * 4) = val;
                            }
                            __syncwarp();
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->tempty);
            acc_phase ^= 1;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kWMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Expert blockIdx.y: zeros if it has no pairs, the sum of its pieces in order if it was
// cut; whole pieces were written by wgrad_kernel.
template <typename T>
__global__ void __launch_bounds__(256) wgrad_sum_kernel(const WgradArgs A) {
    griddep_wait();  // every global access below comes after the previous grid
    __shared__ float4 sums[256];
    const int e = blockIdx.y, H = A.H;
    const int64_t slot = A.starts[e];
    const int pieces = A.starts[e + 1] - static_cast<int>(slot);
    if (pieces == 0 && A.offsets[e + 1] > A.offsets[e]) return;
    const int64_t nW = static_cast<int64_t>(H) * H;
    // G threads share four elements: each adds pieces g, g + G, ... in order, then the G sums in order
    int G = 1;
    while (G < 8 && pieces > 4 && G < pieces) G *= 2;
    const int per = 256 / G, g = threadIdx.x / per, at = threadIdx.x % per;
    auto add = [&](const float* part, int64_t stride, T* out, int64_t count) {
        if (pieces <= 4) {  // a thread adds its elements' pieces alone, two of four elements at a time
            const int64_t step = static_cast<int64_t>(gridDim.x) * 256 * 4;
            for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4; i < count; i += 2 * step) {
                float4 v[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[h][j] = j < pieces && i + h * step < count
                                      ? __ldcg(reinterpret_cast<const float4*>(part + (slot + j) * stride + i + h * step))
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (i + h * step >= count) continue;
                    Chunk<T, 4> o;
                    o.v[0] = from_f<T>(v[h][0].x + v[h][1].x + v[h][2].x + v[h][3].x);
                    o.v[1] = from_f<T>(v[h][0].y + v[h][1].y + v[h][2].y + v[h][3].y);
                    o.v[2] = from_f<T>(v[h][0].z + v[h][1].z + v[h][2].z + v[h][3].z);
                    o.v[3] = from_f<T>(v[h][0].w + v[h][1].w + v[h][2].w + v[h][3].w);
                    *reinterpret_cast<Chunk<T, 4>*>(out + i + h * step) = o;
                }
            }
            return;
        }
        for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * per * 4; i0 < count; i0 += static_cast<int64_t>(gridDim.x) * per * 4) {
            const int64_t i = i0 + at * 4;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < count) {
#pragma unroll 4
                for (int j = g; j < pieces; j += G) {
                    const float4 v = __ldcg(reinterpret_cast<const float4*>(part + (slot + j) * stride + i));
                    a.x += v.x;
                    a.y += v.y;
                    a.z += v.z;
                    a.w += v.w;
                }
            }
            sums[threadIdx.x] = a;
            __syncthreads();
            if (g == 0 && i < count) {
                for (int k = 1; k < G; ++k) {
                    const float4 v = sums[k * per + at];
                    a.x += v.x;
                    a.y += v.y;
                    a.z += v.z;
                    a.w += v.w;
                }
                Chunk<T, 4> o;
                o.v[0] = from_f<T>(a.x);
                o.v[1] = from_f<T>(a.y);
                o.v[2] = from_f<T>(a.z);
                o.v[3] = from_f<T>(a.w);
                *reinterpret_cast<Chunk<T, 4>*>(out + i) = o;
            }
            __syncthreads();
        }
    };
    if (A.dW) add(A.part, nW, static_cast<T*>(A.dW) + e * nW, nW);
    if (A.db) add(A.part_db, H, static_cast<T*>(A.db) + static_cast<int64_t>(e) * H, H);
}

// ---------------------------------------------------------------- launches
bool weight_map(CUtensorMap* map, const void* W, moe_dtype_t dtype, uint64_t rows, uint64_t cols, uint32_t box_rows) {
    EncodeTiledFn enc = get_encode_tiled();
    if (!enc) return false;
    const cuuint64_t dims[2] = {cols, rows};
    const cuuint64_t strides[1] = {cols * 2};
    const cuuint32_t box[2] = {64, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, dtype == MOE_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
               const_cast<void*>(W), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int BN, bool DX>
cudaError_t pair_launch(const void* W, moe_dtype_t dtype, const PairArgs& a, int sms, cudaStream_t s, int* parts) {
    using C = PairCfg<BN, DX>;
    CUtensorMap map;
    if (!weight_map(&map, W, dtype, static_cast<uint64_t>(a.E) * a.H, a.H, DX ? 64 : BN)) return cudaErrorInvalidValue;
    auto kernel = a.K == 1 ? pair_kernel<T, BN, DX, true> : pair_kernel<T, BN, DX, false>;
    static std::atomic<uint64_t> ready[2];
    cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kernel), C::SMEM_BYTES, ready[a.K == 1 ? 1 : 0]);
    if (e != cudaSuccess) return e;
    const int nt = (a.H + BN - 1) / BN;
    *parts = nt * C::HALVES;
    const int64_t tiles = (a.P / 128 + (a.P < a.E ? a.P : a.E)) * nt;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(tiles < sms ? tiles : sms)), dim3(kPairThreads), C::SMEM_BYTES, s, map, a);
}

// Columns per tile: the width whose tiles take the SMs the least time. A tile of 64, 128 or
// 256 columns takes about 10, 11 or 18 (the two halves of the wider ones drain at once, the
// gather is the same), and the tiles go around in whole turns. Forward and backward, K = 2:
// 5003 tokens, E 4, H 128: 64 columns 37.7 us, 128: 35.4; 4,000, E 8, H 256: 50.8 / 48.5,
// 256: 53.0; 2,500, E 16, H 1024: 115.6 / 105.8 / 111.9; 30,000, E 8, H 256: 142.9 / 129.9 / 133.0.
int tile_columns(int64_t P, int E, int H, int sms) {
    const int64_t hit = P < E ? P : E, some = P / 128 + hit / 2, rows = some > hit ? some : hit;  // of 128 pairs, about
    auto time = [&](int bn, int each) { return (rows * ((H + bn - 1) / bn) + sms - 1) / sms * each; };
    int best = 64;
    int64_t least = time(64, 10);
    if (H > 64 && time(128, 11) < least) least = time(128, 11), best = 128;
    if (H > 128 && time(256, 18) < least) best = 256;
    return best;
}

template <typename T, bool DX>
cudaError_t pair_width(const void* W, moe_dtype_t dtype, const PairArgs& a, int sms, cudaStream_t s, int* parts) {
    const int bn = tile_columns(a.P, a.E, a.H, sms);
    if (bn == 256) return pair_launch<T, 256, DX>(W, dtype, a, sms, s, parts);
    if (bn == 128) return pair_launch<T, 128, DX>(W, dtype, a, sms, s, parts);
    return pair_launch<T, 64, DX>(W, dtype, a, sms, s, parts);
}

template <typename T, bool DW>
cudaError_t join_launch(const JoinArgs& a, int sms, cudaStream_t s) {
    // the most lanes a token that work seven eighths of the time at two turns each. Product and join,
    // forward / backward, 8, 16 and 32 lanes: H 192, K 3, 224,532 tokens: 262 / 356 us, 259 / 373,
    // 282 / 429; H 128, K 4, 98,489: 96 / 126, 96 / 130, 99 / 149; H 1024, K 2, 16,384: 124 / 128,
    // 105 / 127, 105 / 123
    int lpt = 32;
    while (lpt > 8 && 8 * a.H < 7 * (lpt * 8) * ((a.H + lpt * 8 - 1) / (lpt * 8))) lpt /= 2;
    auto go = [&](auto kernel, int u) {
        const int64_t tokens = 8 * (32 / lpt) * u, want = (a.T + tokens - 1) / tokens, cap = static_cast<int64_t>(sms) * 8;
        return launch_pdl(kernel, dim3(static_cast<unsigned>(want < cap ? want : cap)), dim3(256), 0, s, a, lpt);
    };
    if (a.K <= 2) return go(join_kernel<T, 2, DW ? 1 : 2, DW>, DW ? 1 : 2);
    if (a.K <= 4) return go(join_kernel<T, 4, 1, DW>, 1);
    if (a.K <= 8) return go(join_kernel<T, 8, 1, DW>, 1);
    return go(join_kernel<T, 16, 1, DW>, 1);
}

// Whether the tokens are grouped by their two experts. Grouping takes about 13 us, which the
// waiting rows' traffic has to outweigh, and the tiles of the E (E + 1) / 2 classes must not be
// mostly empty. Rows joined / grouped, forward + backward for d_x and d_weights: E 8, H 256:
// 20,000 tokens 64 / 64 us, 24,576: 70 / 64, 73,728: 193 / 119; E 4, H 64: 65,536: 54 / 60, 98,304:
// 82 / 74; E 24, H 64: 65,536: 56 / 69, 150,000: 132 / 108; E 16, H 128: 32,768: 52 / 64, 49,152:
// 78 / 74; E 24, H 256: 30,000 (100 a class) 91 / 78; E 32, H 256: 50,000 (95 a class) 141 / 113.
bool takes_duo(const int32_t* expert_idx, int64_t T_, int E, int K, int H) {
    return K == 2 && expert_idx && aligned(expert_idx, 8) && H <= kDuoMaxH && E <= kDuoMaxE && T_ * H >= (6 << 20) &&
           T_ >= 96 * static_cast<int64_t>(E * (E + 1) / 2);
}

template <typename T, bool DX>
cudaError_t duo_launch(const void* W, moe_dtype_t dtype, DuoArgs a, const DuoWs& ws, const int32_t* expert_idx, int64_t T_,
                       int sms, cudaStream_t s) {
    CUtensorMap map;
    if (!weight_map(&map, W, dtype, static_cast<uint64_t>(a.E) * a.H, a.H, DX ? 64 : 128)) return cudaErrorInvalidValue;
    auto kernel = duo_kernel<T, DX>;
    static std::atomic<uint64_t> ready;
    cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kernel), duo_smem<DX>(), ready);
    const int n = a.E * a.E;
    if (e == cudaSuccess) e = cudaMemsetAsync(ws.count, 0, sizeof(int32_t) * 2 * n, s);
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>((T_ + kDuoTokens - 1) / kDuoTokens));
    e = launch_pdl(duo_count_kernel, grid, dim3(256), 0, s, expert_idx, T_, a.E, ws.count);
    if (e != cudaSuccess) return e;
    e = launch_pdl(duo_group_kernel, grid, dim3(256), 0, s, expert_idx, T_, a.E, ws.count, ws.count + n, ws.count + 2 * n, ws.list);
    if (e != cudaSuccess) return e;
    a.start = ws.count + 2 * n;
    a.list = ws.list;
    const int64_t tiles = T_ / 128 + n;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(tiles < sms ? tiles : sms)), dim3(kPairThreads), duo_smem<DX>(), s, map, a);
}

DuoArgs duo_args(const PairArgs& a) {
    DuoArgs d{};
    d.src = a.src;
    d.other = a.other;
    d.bias = a.bias;
    d.weights = a.weights;
    d.E = a.E;
    d.H = a.H;
    d.P = a.P;
    d.out = a.out;
    d.dw_part = a.dw_part;
    d.flags = a.flags;
    return d;
}

template <typename T>
cudaError_t fwd_type(const void* W, moe_dtype_t dtype, const PairArgs& a, int64_t T_, const int32_t* expert_idx, int sms,
                     cudaStream_t s) {
    if (takes_duo(expert_idx, T_, a.E, a.K, a.H))
        return duo_launch<T, false>(W, dtype, duo_args(a), a.duo, expert_idx, T_, sms, s);
    int parts = 0;
    cudaError_t e = pair_width<T, false>(W, dtype, a, sms, s, &parts);
    if (e != cudaSuccess || a.K == 1) return e;
    JoinArgs j{};
    j.rows = a.rows;
    j.out = a.out;
    j.bias = a.bias;
    j.expert_idx = expert_idx;
    j.weights = a.weights;
    j.T = T_;
    j.K = a.K;
    j.H = a.H;
    return join_launch<T, false>(j, sms, s);
}

template <typename T>
cudaError_t wgrad_launch(WgradArgs a, int sms, cudaStream_t s) {
    static std::atomic<uint64_t> ready;
    cudaError_t e = set_smem_once(reinterpret_cast<const void*>(wgrad_kernel<T>), kWSmem, ready);
    if (e != cudaSuccess) return e;
    if (std::is_same<T, __half>::value && a.dW) {
        e = cudaMemsetAsync(a.peak, 0, sizeof(uint32_t) * a.E, s);
        if (e != cudaSuccess) return e;
        const int64_t want = (a.P + 8 * kPeakSlots - 1) / (8 * kPeakSlots), cap = static_cast<int64_t>(sms) * 8;
        e = launch_pdl(wgrad_peak_kernel, dim3(static_cast<unsigned>(want < cap ? want : cap)), dim3(256), 0, s, a);
        if (e != cudaSuccess) return e;
    } else {
        a.peak = nullptr;
    }
    const int64_t hit = a.P < a.E ? a.P : a.E;
    const int64_t units = (hit + a.extra) * wgrad_tiles(a.H);
    e = launch_pdl(wgrad_kernel<T>, dim3(static_cast<unsigned>(units < sms ? units : sms)), dim3(kWThreads), kWSmem, s, a);
    if (e != cudaSuccess) return e;
    // 32 blocks an SM for the experts that are cut, each at least 128 elements (of eight pieces)
    const int cut = a.E < a.extra ? a.E : a.extra, most = a.H * a.H / 128 < 256 ? a.H * a.H / 128 : 256;
    int x = cut > 0 ? (32 * sms + cut - 1) / cut : most;
    if (x > most) x = most;
    return launch_pdl(wgrad_sum_kernel<T>, dim3(x, a.E), dim3(256), 0, s, a);
}

moe_status_t check_sizes(moe_dtype_t dtype, int64_t T, int E, int K, int H) {
    if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16) return MOE_ERR_INVALID_ARG;
    if (T < 0) return MOE_ERR_INVALID_ARG;
    if (E < 1 || E > kMaxE || K < 1 || K > kMaxK || K > E) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (H < 64 || H > kMaxH || H % 64 != 0 || T >= kMaxT / K) return MOE_ERR_UNSUPPORTED_SHAPE;
    // tile numbers stay in 32 bits
    if ((T * K / 128 + E + 1) * (H / 64) >= kMaxT) return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

template <typename T>
cudaError_t bwd_type(const void* W, const void* bias, moe_dtype_t dtype, PairArgs a, const WgradArgs& wg, int64_t T_,
                     const int32_t* expert_idx, float* d_weights, int sms, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    if (a.out || d_weights) {
        const bool duo = takes_duo(expert_idx, T_, a.E, a.K, a.H);
        int parts = 2;
        e = duo ? duo_launch<T, true>(W, dtype, duo_args(a), a.duo, expert_idx, T_, sms, s)
                : pair_width<T, true>(W, dtype, a, sms, s, &parts);
        if (e == cudaSuccess && (d_weights || (a.K > 1 && !duo))) {
            JoinArgs j{};
            j.rows = a.rows;
            j.out = a.K > 1 && !duo ? a.out : nullptr;
            j.dw_part = a.dw_part;
            j.parts = parts;
            j.g = a.src;
            j.bias = d_weights ? bias : nullptr;  // part of d_weights only, and expert_idx with it
            j.expert_idx = expert_idx;
            j.d_weights = d_weights;
            j.T = T_;
            j.K = a.K;
            j.H = a.H;
            e = join_launch<T, true>(j, sms, s);
        }
    }
    if (e == cudaSuccess && (wg.dW || wg.db)) e = wgrad_launch<T>(wg, sms, s);
    return e;
}

}  // namespace

size_t topk_experts_ws_bytes(int64_t T, int E, int K, int H) {
    return experts_ws(T, E, K, H, topk_route_ws_bytes(T, E)).total;
}
bool topk_experts_sizes_ok(int64_t T, int E, int K, int H) { return check_sizes(MOE_DTYPE_BF16, T, E, K, H) == MOE_OK; }

}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_topk_fwd(const void* x, const void* W, const void* bias, moe_dtype_t dtype,
                          const moe_routing_t* routing, const float* weights, int64_t T, int32_t E, int32_t K,
                          int32_t H, void* y, void* workspace, size_t workspace_bytes, void* stream) {
    moe_status_t st = check_sizes(dtype, T, E, K, H);
    if (st != MOE_OK) return st;
    if (!routing || !W) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!x || !y || !weights || !routing->offsets || !routing->perm)) return MOE_ERR_INVALID_ARG;
    if (T > 0 && K > 1 && bias && !routing->expert_idx) return MOE_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(W, 16) || !aligned(bias, 16) || !aligned(y, 16) || !aligned(weights, 4) ||
        !aligned(routing->offsets, 4) || !aligned(routing->perm, 4) || !aligned(routing->expert_idx, 4))
        return MOE_ERR_MISALIGNED;
    const size_t P = static_cast<size_t>(T) * K, act = 2 * static_cast<size_t>(T) * H;
    const Range outs[2] = {{y, act}, {workspace, workspace ? workspace_bytes : 0}};
    const Range ins[7] = {{x, act}, {W, 2 * static_cast<size_t>(E) * H * H}, {bias, 2 * static_cast<size_t>(E) * H},
                          {weights, 4 * P}, {routing->offsets, sizeof(int32_t) * (E + 1)}, {routing->perm, 4 * P},
                          {routing->expert_idx, 4 * P}};
    if (any_alias(outs, 2, ins, 7)) return MOE_ERR_ALIAS;
    if (T == 0) return MOE_OK;
    const ExpertsWs L = experts_ws(T, E, K, H, topk_route_ws_bytes(T, E));
    if (!workspace) return MOE_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return MOE_ERR_MISALIGNED;
    if (workspace_bytes < L.total) return MOE_ERR_WORKSPACE;
    int sms = 0;
    if (device_sms(&sms) != cudaSuccess) return MOE_ERR_CUDA;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    PairArgs a{};
    a.src = x;
    a.bias = bias;
    a.weights = weights;
    a.offsets = routing->offsets;
    a.perm = routing->perm;
    a.E = E;
    a.K = K;
    a.by_k = div_by(K);
    a.H = H;
    a.P = static_cast<int64_t>(P);
    a.out = y;
    a.rows = reinterpret_cast<float*>(ws + L.rows);
    a.duo = {reinterpret_cast<int32_t*>(ws + L.duo), reinterpret_cast<int32_t*>(ws + L.list)};
    a.flags = reinterpret_cast<uint32_t*>(ws);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(dtype == MOE_DTYPE_BF16 ? fwd_type<__nv_bfloat16>(W, dtype, a, T, routing->expert_idx, sms, s)
                                               : fwd_type<__half>(W, dtype, a, T, routing->expert_idx, sms, s));
}

moe_status_t moe_topk_bwd(const void* x, const void* W, const void* bias, moe_dtype_t dtype, const void* d_out,
                          const moe_routing_t* routing, const float* weights, int64_t T, int32_t E, int32_t K,
                          int32_t H, void* d_x, void* dW, void* db, float* d_weights, void* workspace,
                          size_t workspace_bytes, void* stream) {
    moe_status_t st = check_sizes(dtype, T, E, K, H);
    if (st != MOE_OK) return st;
    if (!routing) return MOE_ERR_INVALID_ARG;
    if (!d_x && !dW && !db && !d_weights) return MOE_OK;
    if ((d_x || d_weights) && !W) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!d_out || !weights || !routing->offsets || !routing->perm)) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (dW || db || d_weights) && !x) return MOE_ERR_INVALID_ARG;
    if (T > 0 && d_weights && bias && !routing->expert_idx) return MOE_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(W, 16) || !aligned(bias, 16) || !aligned(d_out, 16) || !aligned(d_x, 16) ||
        !aligned(dW, 16) || !aligned(db, 16) || !aligned(d_weights, 4) || !aligned(weights, 4) ||
        !aligned(routing->offsets, 4) || !aligned(routing->perm, 4) || !aligned(routing->expert_idx, 4))
        return MOE_ERR_MISALIGNED;
    const size_t P = static_cast<size_t>(T) * K, act = 2 * static_cast<size_t>(T) * H;
    const size_t wb = 2 * static_cast<size_t>(E) * H * H, bb = 2 * static_cast<size_t>(E) * H;
    const Range outs[5] = {{d_x, act}, {dW, wb}, {db, bb}, {d_weights, 4 * P}, {workspace, workspace ? workspace_bytes : 0}};
    const Range ins[8] = {{x, act}, {W, wb}, {bias, bb}, {d_out, act}, {weights, 4 * P},
                          {routing->offsets, sizeof(int32_t) * (E + 1)}, {routing->perm, 4 * P},
                          {routing->expert_idx, 4 * P}};
    if (any_alias(outs, 5, ins, 8)) return MOE_ERR_ALIAS;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        cudaError_t e = cudaSuccess;
        if (dW) e = cudaMemsetAsync(dW, 0, wb, s);
        if (e == cudaSuccess && db) e = cudaMemsetAsync(db, 0, bb, s);
        return cuda_status(e);
    }
    const ExpertsWs L = experts_ws(T, E, K, H, topk_route_ws_bytes(T, E));
    if (!workspace) return MOE_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return MOE_ERR_MISALIGNED;
    if (workspace_bytes < L.total) return MOE_ERR_WORKSPACE;
    int sms = 0;
    if (device_sms(&sms) != cudaSuccess) return MOE_ERR_CUDA;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    PairArgs a{};
    a.src = d_out;
    a.other = d_weights ? x : nullptr;
    a.weights = weights;
    a.offsets = routing->offsets;
    a.perm = routing->perm;
    a.E = E;
    a.K = K;
    a.by_k = div_by(K);
    a.H = H;
    a.P = static_cast<int64_t>(P);
    a.out = d_x;
    a.rows = reinterpret_cast<float*>(ws + L.rows);
    a.duo = {reinterpret_cast<int32_t*>(ws + L.duo), reinterpret_cast<int32_t*>(ws + L.list)};
    a.dw_part = reinterpret_cast<float*>(ws + L.dw_part);
    a.flags = reinterpret_cast<uint32_t*>(ws);
    WgradArgs g{};
    g.x = x;
    g.g = d_out;
    g.weights = weights;
    g.offsets = routing->offsets;
    g.perm = routing->perm;
    g.E = E;
    g.K = K;
    g.by_k = a.by_k;
    g.H = H;
    g.P = static_cast<int64_t>(P);
    g.extra = wgrad_extra(g.P, E, H);
    g.dW = dW;
    g.db = db;
    g.part = reinterpret_cast<float*>(ws + L.part);
    g.part_db = reinterpret_cast<float*>(ws + L.part_db);
    g.starts = reinterpret_cast<int32_t*>(ws + L.starts);
    g.peak = reinterpret_cast<uint32_t*>(ws + L.peak);
    g.flags = a.flags;
    return cuda_status(dtype == MOE_DTYPE_BF16
                           ? bwd_type<__nv_bfloat16>(W, bias, dtype, a, g, T, routing->expert_idx, d_weights, sms, s)
                           : bwd_type<__half>(W, bias, dtype, a, g, T, routing->expert_idx, d_weights, sms, s));
}

}  // extern "C"
