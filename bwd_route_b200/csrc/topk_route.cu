// topk_route.cu -- the router of the top-k block: K experts per token with their
// weights, the lists that group the T * K pairs by expert, and the gradient of the
// logits.
//
//   s = softmax(l) or sigmoid(l);  v = s + bias;  masked (l = -inf or NaN): v = -inf
//   groups: the top_groups groups with the largest sum of their `best` largest v stay
//   the K largest v that stay, largest first, equal ones by index;  w = scale * s
//   (renormalised: scale * s / sum of the chosen s, taken as a ratio of exponentials,
//   so that it is finite where every s underflows)
//
// Choices are exact. Without a bias the order of v is that of the logits, which are
// compared as they are. With a bias (or sums of scores per group) v is computed in
// fp32, and where two neighbours among the chosen, or the last of them and any other
// expert, lie within the error of that computation and are no true tie the token is
// chosen again in fp64; about one in a thousand is.
//
// A token belongs to LPT lanes with VPL consecutive experts each. Up to 64 experts a
// warp works on 32 / LPT tokens at once: K rounds of a local maximum, a shuffle maximum
// over the lanes and a ballot, whose lowest lane holds the lowest index. Above, a warp
// takes one token and finds the K largest through a threshold (choose_by_threshold). The
// block counts its pairs per expert in shared memory; a second kernel turns the blocks'
// counts into each block's base positions, a third writes the lists (stable, as in
// route.cu). Few tokens take one launch of one block that does all three.
//
// What bounds it: the issue of instructions, about 650 a token of 256 experts with a bias
// and groups (59 % of the issue slots used, 13 % of the DRAM bandwidth). 65,536 x 256 fp32,
// 4 of 8 groups stay, K = 8: choice 67 us, scan 5.3, lists 10.0; rounds of a warp
// maximum instead of the threshold took 130 us, fp64 for every open token on the spot 112.
// 8 tokens x 64 experts: 6.9 us on the device, one chain of dependent steps. 262,144 x 8, K = 2:
// 19 us by logits, 24 with a bias; 262,144 x 64, K = 6, with a bias: 132 us.
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "checks.h"
#include "common.cuh"
#include "elem.cuh"
#include "internal.h"
#include "moe_topk.h"
#include "topk.h"

namespace moe {
namespace {

constexpr int kMaxE = 256, kMaxK = 16, kMaxGroups = 32;
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kSmallThreads = 1024;
constexpr int kMaxBlocks = 1024;      // rows of per-block counts the workspace holds
constexpr int kSmallPairs = 8192;     // pairs the one-block kernel keeps in shared memory
constexpr unsigned kFull = 0xffffffffu;

// What the choice compares: logits, or scores (a bias, or group sums, make the difference).
enum Mode : int { kLogits = 0, kSigmoid = 1, kSoftmax = 2 };

struct Rule {
    int E, K, G, S, top_groups, best;  // S: experts per group
    int sigmoid, renorm;
    float scale;
};

// ---------------------------------------------------------------- keys
// Unsigned integers in the order of the values (-0 counts as +0). 0: not a candidate;
// 1: a masked expert; both below the key of every number.
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ uint64_t key_of(double v) {
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
    return (b >> 63) ? ~b : (b | (1ull << 63));
}
__device__ __forceinline__ float value_of(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
template <typename V>
struct KeyOf;
template <>
struct KeyOf<float> {
    using type = uint32_t;
};
template <>
struct KeyOf<double> {
    using type = uint64_t;
};

__device__ __forceinline__ float exp_v(float x) { return expf(x); }
__device__ __forceinline__ double exp_v(double x) { return exp(x); }
// Only compared (fp32): an absolute error of 7 * 2^-24 is inside the border test. The
// exponent l log2 e is rounded once (|l| 2^-23 relative in the power, at most 1.3 * 2^-24
// after the factor s (1 - s)), ex2 and rcp are off by 2 units in the last place at most
// each, the sums by one.
__device__ __forceinline__ float sigmoid_v(float l) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(l * -1.44269504f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}
__device__ __forceinline__ double sigmoid_v(double l) { return 1.0 / (1.0 + exp(-l)); }

template <int LPT, typename V>
__device__ __forceinline__ V lanes_max(V v) {
#pragma unroll
    for (int off = LPT / 2; off >= 1; off >>= 1) {
        const V o = __shfl_xor_sync(kFull, v, off);
        v = o > v ? o : v;
    }
    return v;
}
template <int LPT, typename V>
__device__ __forceinline__ V lanes_sum(V v) {
#pragma unroll
    for (int off = LPT / 2; off >= 1; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
    return v;
}

// ---------------------------------------------------------------- one token's row
template <typename T, int VPL>
__device__ __forceinline__ void load_logits(const T* row, int e0, int E, bool vec, bool valid, float (&l)[VPL]) {
    constexpr int C = VPL * sizeof(T) < 16 ? VPL : 16 / sizeof(T);
    static_assert(VPL % C == 0, "whole chunks");
    if (vec) {
#pragma unroll
        for (int j = 0; j < VPL; j += C) {
            Chunk<T, C> c;
            const bool on = valid && e0 + j < E;
            if (on) c = *reinterpret_cast<const Chunk<T, C>*>(row + e0 + j);
#pragma unroll
            for (int i = 0; i < C; ++i) l[j + i] = on ? to_f(c.v[i]) : 0.0f;
        }
    } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j) l[j] = (valid && e0 + j < E) ? to_f(row[e0 + j]) : 0.0f;
    }
}

// The bias of a lane's experts, NaN past the last one: what is no expert is then NaN in
// every value that is compared. A NaN of the caller's masks its expert like a NaN logit.
template <int VPL>
__device__ __forceinline__ void load_bias(const float* bias, int e0, int E, float (&b)[VPL]) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        b[j] = e0 + j < E && bias ? bias[e0 + j] : 0.0f;
        if (b[j] != b[j]) b[j] = -INFINITY;
        if (e0 + j >= E) b[j] = __int_as_float(0x7fffffff);
    }
}

__device__ __forceinline__ bool is_masked(float l) { return !(l > -INFINITY); }

// Maximum and sum of exponentials of a softmax row over its lanes (fp32 or fp64). A row
// of nothing but -inf gives m = 0, z = 1 (every score is then exp(-inf) = 0).
template <typename V, int LPT, int VPL>
__device__ __forceinline__ void softmax_stats(const float (&l)[VPL], int e0, int E, V& m, V& z) {
    float mx = -INFINITY;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
        if (e0 + j < E && l[j] > mx) mx = l[j];
    mx = lanes_max<LPT>(mx);
    if (mx == -INFINITY) mx = 0.0f;
    V s = 0;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
        if (e0 + j < E) s += exp_v(static_cast<V>(l[j]) - static_cast<V>(mx));
    s = lanes_sum<LPT>(s);
    m = mx;
    z = s == V(0) ? V(1) : s;
}

// Shared memory of one warp: per token of the warp its K chosen experts and their keys'
// values, and with groups the values and the group scores.
template <typename V>
struct WarpSmem {
    int* slot;    // [32 / LPT][K]
    float* slot_v;
    V* val;       // [32 / LPT][E padded], group selection only
    V* gscore;    // [32 / LPT][G]
};

__device__ __forceinline__ int pad_e(int e) { return e + (e >> 5); }
__host__ __device__ constexpr int padded(int ep) { return ep + ep / 32 + 1; }

// The groups that stay, through shared memory: bit g of kept. Returns whether fp32 leaves
// that open.
template <typename V, int LPT, int VPL, int MODE>
__device__ __forceinline__ bool group_kept(const V (&v)[VPL], int e0, int tok, const Rule& R, V* vals, V* gscores, float tol,
                                           unsigned& kept) {
    constexpr unsigned kMine = LPT == 32 ? kFull : (1u << (LPT & 31)) - 1u;
    const int sub = (threadIdx.x & 31) % LPT;
    V* val = vals + tok * padded(LPT * VPL);
    V* gs = gscores + tok * R.G;
    bool unsure = false;
#pragma unroll
    for (int j = 0; j < VPL; ++j) val[pad_e(e0 + j)] = v[j];
    __syncwarp();
    for (int g = sub; g < R.G; g += LPT) {
        V a = -INFINITY, b = -INFINITY;
        for (int i = 0; i < R.S; ++i) {
            const V x = val[pad_e(g * R.S + i)];
            if (x > a) {
                b = a;
                a = x;
            } else if (x > b) {
                b = x;
            }
        }
        gs[g] = R.best == 2 ? a + b : a;
    }
    __syncwarp();
    kept = 0;
    for (int i = 0; i < R.G; i += LPT) {
        const int g = i + sub;
        bool keep = false;
        if (g < R.G) {
            const V mine = gs[g];
            int rank = 0;
            for (int o = 0; o < R.G; ++o) {
                const V x = gs[o];
                rank += (x > mine || (x == mine && o < g)) ? 1 : 0;
            }
            keep = rank < R.top_groups;
            if (sizeof(V) == 4 && MODE != kLogits) {
                // sums of two are off by up to twice as much; unsure: a kept group that could fall
                // out, or a dropped one that could come in
                const float t2 = 2.0f * tol * (1.0f + fabsf(static_cast<float>(mine)));
                int above = 0, near = 0;
                for (int o = 0; o < R.G; ++o) {
                    const float d = static_cast<float>(gs[o]) - static_cast<float>(mine);
                    above += d > t2 ? 1 : 0;
                    near += (o != g && fabsf(d) <= t2) ? 1 : 0;
                }
                unsure |= near > 0 && above < R.top_groups && above + near >= R.top_groups;
            }
        }
        const unsigned b = __ballot_sync(kFull, keep);
        kept |= ((b >> (tok * LPT)) & kMine) << i;
    }
    return unsure;
}

// Bit j: the lane's expert e0 + j is in a group that stays.
template <int VPL>
__device__ __forceinline__ unsigned group_alive(unsigned kept, int e0, const Rule& R) {
    unsigned alive = 0;
    for (int g = e0 / R.S; g < R.G && g * R.S < e0 + VPL; ++g) {
        if (!((kept >> g) & 1u)) continue;
        const int lo = max(g * R.S - e0, 0), hi = min((g + 1) * R.S - e0, VPL);
        alive |= ((1u << hi) - 1u) & ~((1u << lo) - 1u);
    }
    return alive;
}

// Chooses the experts of the warp's tokens: slot[k] of each. V = float: returns whether a
// choice lies too near a border to be certain (true for some lane of the token).
template <typename V, typename T, int LPT, int VPL, int MODE>
__device__ __forceinline__ bool choose(const float (&l)[VPL], const T* row, const float* __restrict__ bias,
                                       const Rule& R, const WarpSmem<V>& sm) {
    using Key = typename KeyOf<V>::type;
    constexpr bool kFast = sizeof(V) == 4;
    const int lane = threadIdx.x & 31, sub = lane % LPT, tok = lane / LPT, g0 = tok * LPT, e0 = sub * VPL;
    constexpr unsigned kMine = LPT == 32 ? kFull : (1u << (LPT & 31)) - 1u;
    V m = 0, z = 1;
    if (MODE == kSoftmax) softmax_stats<V, LPT, VPL>(l, e0, R.E, m, z);
    const V inv_z = V(1) / z;
    auto score = [&](float x) -> V {
        return MODE == kSigmoid ? sigmoid_v(static_cast<V>(x)) : exp_v(static_cast<V>(x) - m) * inv_z;
    };
    Key key[VPL];
    V v[VPL];  // what groups are scored by
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        const int e = e0 + j;
        V order;
        if (MODE != kLogits) {
            v[j] = score(l[j]);
            if (bias && e < R.E) v[j] += static_cast<V>(bias[e]);
            order = bias ? v[j] : static_cast<V>(l[j]);
        } else {
            v[j] = order = static_cast<V>(l[j]);
        }
        const bool off = is_masked(l[j]) || order != order;
        if (off) v[j] = -INFINITY;
        key[j] = e >= R.E ? Key(0) : off ? Key(1) : key_of(order);
    }
    bool unsure = false;
    // border of two values in fp32; see sigmoid_v. The softmax adds the error of its sum:
    // 17 + 21 units for 256 terms.
    const float tol = MODE == kSigmoid ? 0x1p-20f : 0x1p-17f;
    if (R.G > 1) {
        unsigned kept;
        unsure = group_kept<V, LPT, VPL, MODE>(v, e0, tok, R, sm.val, sm.gscore, tol, kept);
        const unsigned alive = group_alive<VPL>(kept, e0, R);
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (!((alive >> j) & 1u)) key[j] = 0;
    }
    constexpr bool kCheck = kFast && MODE != kLogits;
    int* slot = sm.slot + tok * R.K;
    float* slot_v = sm.slot_v + tok * R.K;
    for (int k = 0; k < R.K; ++k) {
        Key best = 0;
        int at = 0;
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (key[j] > best) {
                best = key[j];
                at = j;
            }
        const Key top = lanes_max<LPT>(best);
        const unsigned b = (__ballot_sync(kFull, best == top && top != 0) >> g0) & kMine;
        const bool win = b != 0 && sub == __ffs(b) - 1;
        if (win) {
            slot[k] = e0 + at;
            if constexpr (kCheck) slot_v[k] = top == 1 ? -INFINITY : value_of(static_cast<uint32_t>(top));
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (j == at) key[j] = 0;
        } else if (b == 0 && sub == 0) {
            slot[k] = -1;
        }
    }
    __syncwarp();
    if constexpr (kCheck) {
        if (bias) {
            // equal logits and equal biases are a true tie, in index order already
            for (int k = sub; k + 1 < R.K; k += LPT) {
                const int ea = slot[k], eb = slot[k + 1];
                const float a = slot_v[k], b = slot_v[k + 1];
                if (a - b <= tol * (1.0f + fabsf(a)) && !(to_f(row[ea]) == to_f(row[eb]) && bias[ea] == bias[eb])) unsure = true;
            }
            // Any expert left that comes near the last one chosen, not the next alone: that one may be a
            // true tie with another, larger one behind it.
            const float last = slot_v[R.K - 1], low = last - tol * (1.0f + fabsf(last));
            if (last > -INFINITY) {
                const int el = slot[R.K - 1];
#pragma unroll
                for (int j = 0; j < VPL; ++j)
                    if (key[j] > 1 && value_of(static_cast<uint32_t>(key[j])) >= low &&
                        !(l[j] == to_f(row[el]) && bias[e0 + j] == bias[el]))
                        unsure = true;
            }
        }
    }
    return unsure;
}

// A whole warp on one token (fp32). A threshold that at least K values reach gives a few
// candidates, a lane each, which are ranked by counting. The threshold is the last token's,
// where that leaves between K and 32 candidates, else the largest of the lanes' maxima that
// enough lanes reach. Returns false where the
// fp32 values leave the choice open, or more than 32 reach the threshold (equal values).
// Dropped experts are NaN, which no comparison lets through; masked ones -inf.
template <typename T, int VPL, int MODE>
__device__ __forceinline__ bool choose_by_threshold(const float (&l)[VPL], const float (&b)[VPL], const T* row,
                                                    const float* __restrict__ bias, const Rule& R, int* slot,
                                                    float* slot_v, uint2* cand, int* found, float* groups, float2& stats,
                                                    float& guess) {
    const int lane = threadIdx.x & 31, e0 = lane * VPL;
    const float nan = __int_as_float(0x7fffffff);
    constexpr float tol = MODE == kSigmoid ? 0x1p-20f : 0x1p-17f;  // as in choose()
    bool unsure = false;
    float order[VPL];
    if (MODE == kSoftmax || (!R.sigmoid && !R.renorm)) softmax_stats<float, 32, VPL>(l, e0, R.E, stats.x, stats.y);
    if (MODE == kLogits) {
#pragma unroll
        for (int j = 0; j < VPL; ++j) order[j] = is_masked(l[j]) ? -INFINITY : l[j] + b[j];
    } else {
        const float inv_z = MODE == kSoftmax ? 1.0f / stats.y : 1.0f;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const float s = MODE == kSigmoid ? sigmoid_v(l[j]) : expf(l[j] - stats.x) * inv_z;
            order[j] = l[j] > -INFINITY && (MODE == kSigmoid || s == s) ? s + b[j] : -INFINITY;
        }
    }
    bool keep = true;
    if (R.G > 1) {
        const int L = R.S / VPL;  // lanes a group spans
        if (R.S % VPL == 0 && (L & (L - 1)) == 0) {
            float a = -INFINITY, c = -INFINITY;
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                c = fmaxf(c, fminf(a, order[j]));
                a = fmaxf(a, order[j]);
            }
            for (int off = 1; off < L; off <<= 1) {
                const float oa = __shfl_xor_sync(kFull, a, off), oc = __shfl_xor_sync(kFull, c, off);
                c = fmaxf(fminf(a, oa), fmaxf(c, oc));
                a = fmaxf(a, oa);
            }
            const float mine = R.best == 2 ? a + c : a;
            const int g = lane >> (31 - __clz(L));
            // the group's lanes compare it with the others in turn: counts of groups above, and (scores)
            // of groups too near to tell, itself among them. Sums of two are off by up to twice as much.
            const float t2 = MODE == kLogits || !(mine > -INFINITY) ? 0.0f : 2.0f * tol * (1.0f + fabsf(mine));
            int count = 0;
            for (int o0 = 0; o0 < R.G; o0 += L) {  // every lane takes the same number of turns
                const int o = o0 + (lane & (L - 1));
                const float x = __shfl_sync(kFull, mine, (o * L) & 31);
                if (o < R.G) {
                    if (MODE == kLogits) {
                        count += (x > mine || (x == mine && o < g)) ? 1 : 0;
                    } else {
                        const float d = x - mine;
                        count += d > t2 ? 1 : !(fabsf(d) > t2) ? 256 : 0;  // -inf - -inf counts as near
                    }
                }
            }
            for (int off = 1; off < L; off <<= 1) count += __shfl_xor_sync(kFull, count, off);
            const int above = count & 255;
            keep = g < R.G && above < R.top_groups;
            if (MODE != kLogits) unsure = keep && above + (count >> 8) > R.top_groups;
        } else {
            unsigned kept;
            unsure = group_kept<float, 32, VPL, MODE>(order, e0, 0, R, groups, groups + padded(32 * VPL), tol, kept);
            const unsigned alive = group_alive<VPL>(kept, e0, R);
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (!((alive >> j) & 1u)) order[j] = nan;
            keep = alive != 0;
        }
    }
    const bool check = MODE != kLogits && bias;
    if (MODE != kLogits && !bias) {  // groups were chosen by scores, experts are by logits
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (order[j] == order[j]) order[j] = is_masked(l[j]) ? -INFINITY : l[j];
    }
    const int need = R.K;
    int n = 0;
#pragma unroll
    for (int j = 0; j < VPL; ++j) n += order[j] >= guess ? 1 : 0;
    if (!keep) n = 0;
    float tau = guess;
    int total = __reduce_add_sync(kFull, n);
    if (total < need || total > 32) {
        float top = nan;
#pragma unroll
        for (int j = 0; j < VPL; ++j) top = fmaxf(top, order[j]);
        uint32_t cur = !keep || top != top ? 0u : key_of(top);
        tau = -INFINITY;
        for (int reached = 0;;) {
            const uint32_t mx = __reduce_max_sync(kFull, cur);
            if (mx == 0) break;
            const bool at_top = cur == mx;
            reached += __popc(__ballot_sync(kFull, at_top));
            if (reached >= need) {
                tau = value_of(mx);
                break;
            }
            if (at_top) cur = 0;
        }
        n = 0;
#pragma unroll
        for (int j = 0; j < VPL; ++j) n += order[j] >= tau ? 1 : 0;
        if (!keep) n = 0;
        total = __reduce_add_sync(kFull, n);
        if (total > 32) return false;
    }
    // the list's order does not matter: its entries are ranked by value and index, as one
    // 64-bit number each
    if (n) {
        int at = atomicAdd(found, n);
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (order[j] >= tau) cand[at++] = make_uint2(static_cast<uint32_t>(~(e0 + j)), __float_as_uint(order[j]));
    }
    __syncwarp();
    if (lane == 0) *found = 0;
    const uint2 mine = lane < total ? cand[lane] : make_uint2(0u, 0u);
    const float my_v = __uint_as_float(mine.y);
    const uint64_t my_key = (static_cast<uint64_t>(key_of(my_v)) << 32) | mine.x;
    if (lane < total) reinterpret_cast<uint64_t*>(cand)[lane] = my_key;
    __syncwarp();
    int rank = 0;
#pragma unroll 4
    for (int o = 0; o < total; ++o) rank += reinterpret_cast<const uint64_t*>(cand)[o] > my_key ? 1 : 0;
    if (lane < total && rank < need) {
        slot[rank] = static_cast<int>(~mine.x);
        slot_v[rank] = my_v;
    }
    // the next token's guess follows the value a few places behind the last one needed
    const unsigned b_guess = __ballot_sync(kFull, lane < total && rank == min(total - 1, need + 4));
    const float at_guess = __shfl_sync(kFull, my_v, __ffs(b_guess) - 1);
    guess = guess == guess && fabsf(guess) < INFINITY ? guess + 0.25f * (at_guess - guess) : at_guess;
    if (check) {
        __syncwarp();
        if (lane + 1 < R.K) {
            const float x = slot_v[lane], y = slot_v[lane + 1];
            if (x - y <= tol * (1.0f + fabsf(x))) {
                // equal logits and equal biases are a true tie, in index order already
                const int ea = slot[lane], eb = slot[lane + 1];
                if (!(to_f(row[ea]) == to_f(row[eb]) && bias[ea] == bias[eb])) unsure = true;
            }
        }
        // any expert left that comes near the last one chosen, as in choose()
        const float last = slot_v[R.K - 1], low = last - tol * (1.0f + fabsf(last));
        int near = 0;
#pragma unroll
        for (int j = 0; j < VPL; ++j) near += order[j] >= low ? 1 : 0;
        if (!keep) near = 0;
        if (__reduce_add_sync(kFull, near) > R.K && last > -INFINITY) {
            const int el = slot[R.K - 1];
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                const int e = e0 + j;
                const bool left = keep && order[j] >= low && (order[j] < last || (order[j] == last && e > el));
                if (left && !(to_f(row[e]) == to_f(row[el]) && bias[e] == bias[el])) unsure = true;
            }
        }
    }
    return !__any_sync(kFull, unsure);
}

// Weight of a chosen expert with logit x. Each of `lanes` neighbouring lanes has one (on)
// or none; stats: maximum and sum of the softmax row, where that is what divides.
template <int LANES>
__device__ __forceinline__ float weight_of(float x, bool on, float2 stats, const Rule& R) {
    float m = 0.0f, z = 1.0f;
    const float low = R.sigmoid ? (x >= 0.0f ? 0.0f : x) : x;  // keeps a NaN
    if (R.renorm) {  // ratios: the largest chosen exponent is 0
        m = on ? low : -INFINITY;
#pragma unroll
        for (int off = LANES / 2; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
        if (m == -INFINITY) m = 0.0f;
    } else if (!R.sigmoid) {
        m = stats.x;
        z = stats.y;
    }
    float p = expf(low - m);
    if (R.sigmoid) p = p / (1.0f + expf(-fabsf(x)));
    if (R.renorm) {
        z = on ? p : 0.0f;
#pragma unroll
        for (int off = LANES / 2; off >= 1; off >>= 1) z += __shfl_xor_sync(kFull, z, off);
        if (z == 0.0f) z = 1.0f;
    }
    return R.scale * (p / z);
}

// One token that the fp32 pass left open, by a whole warp: the choice by rounds (in fp64
// where scores decide), weights and counts. Out of line: it is rare.
template <typename T, int VPL, int MODE>
__device__ __noinline__ void route_again(const T* row, int64_t t, bool vec, const float* __restrict__ bias, const Rule& R,
                                         int* slot, float* slot_v, double* groups, int* hist,
                                         int32_t* __restrict__ expert_idx, float* __restrict__ weights, int* s_idx) {
    using V = typename std::conditional<MODE == kLogits, float, double>::type;
    const int lane = threadIdx.x & 31, e0 = lane * VPL;
    float l[VPL];
    load_logits<T, VPL>(row, e0, R.E, vec, true, l);
    V* val = reinterpret_cast<V*>(groups);
    WarpSmem<V> sm{slot, slot_v, val, val + padded(32 * VPL)};
    choose<V, T, 32, VPL, MODE>(l, row, bias, R, sm);
    float2 stats = make_float2(0.0f, 1.0f);
    if (!R.sigmoid && !R.renorm) softmax_stats<float, 32, VPL>(l, e0, R.E, stats.x, stats.y);
    const bool on = lane < R.K;
    const int e = on ? slot[lane] : 0;
    const float w = weight_of<32>(on ? to_f(row[e]) : 0.0f, on, stats, R);
    if (on) {
        expert_idx[t * R.K + lane] = e;
        weights[t * R.K + lane] = w;
        atomicAdd(&hist[e], 1);
        if (s_idx) s_idx[t * R.K + lane] = e;
    }
    __syncwarp();
}

// Shared memory of one warp: slots of its tokens (K experts and values each), softmax
// statistics, candidates and their number, and with groups (8-byte elements, enough for
// route_again) values and group scores.
struct WarpArea {
    int* slot;
    float* slot_v;
    float2* stats;
    uint2* cand;
    int* found;  // zero between tokens
    double* groups;
};
// Tokens whose slots a warp keeps: those it works on at once, or (a token per warp) those
// whose weights it computes together, a lane per chosen expert.
__host__ __device__ inline int slot_tokens(int lpt, int K) { return lpt < 32 ? 32 / lpt : K <= 4 ? 8 : K <= 8 ? 4 : 2; }
__host__ __device__ inline int warp_bytes(const Rule& R, int lpt, int vpl) {
    const int n = slot_tokens(lpt, R.K), tpw = 32 / lpt;
    int b = n * R.K * 8 + n * 8 + 256 + 8;
    if (R.G > 1) {
        const int again = padded(lpt < 32 ? 64 : 32 * vpl) + R.G, now = (tpw * (padded(lpt * vpl) + R.G) + 1) / 2;
        b += 8 * (again > now ? again : now);
    }
    return b;
}
__device__ __forceinline__ WarpArea warp_area(uint8_t* p, int lpt, int K) {
    const int n = slot_tokens(lpt, K);
    WarpArea a;
    a.slot = reinterpret_cast<int*>(p);
    a.slot_v = reinterpret_cast<float*>(p + n * K * 4);
    a.stats = reinterpret_cast<float2*>(p + n * K * 8);
    a.cand = reinterpret_cast<uint2*>(a.stats + n);
    a.found = reinterpret_cast<int*>(a.cand + 32);
    a.groups = reinterpret_cast<double*>(a.found + 2);
    return a;
}

// Routes tokens t0, t0 + step, ... below t1 (a token per group of LPT lanes: t0 is the
// group's first): writes expert_idx and weights, adds to the block's histogram. s_idx:
// the pairs' experts kept for the one-block kernel, or NULL.
template <typename T, int LPT, int VPL, int MODE>
__device__ __forceinline__ void route_tokens(const T* logits, int64_t ld, int64_t t0, int64_t t1, int64_t step, bool vec,
                                             const float* __restrict__ bias, const Rule& R, const WarpArea& A, int* hist,
                                             int32_t* __restrict__ expert_idx, float* __restrict__ weights, int* s_idx) {
    const int lane = threadIdx.x & 31, sub = lane % LPT, tok = lane / LPT, e0 = sub * VPL, K = R.K;
    const int64_t first = t0 - tok;  // the warp's first token
    float next[VPL];
    load_logits<T, VPL>(logits + (t0 < t1 ? t0 : 0) * ld, e0, R.E, vec, t0 < t1, next);
    if constexpr (LPT == 32) {
        const int batch = slot_tokens(32, K), lanes = 32 / batch;
        float b[VPL];
        load_bias<VPL>(bias, e0, R.E, b);
        float guess = __int_as_float(0x7fffffff);
        if (lane == 0) *A.found = 0;
        __syncwarp();
        for (int64_t tb = t0; tb < t1; tb += batch * step) {
            unsigned open = 0;  // tokens of the batch left open
            for (int i = 0; i < batch; ++i) {
                const int64_t t = tb + i * step;
                if (t >= t1) break;
                float l[VPL];
#pragma unroll
                for (int j = 0; j < VPL; ++j) l[j] = next[j];
                const int64_t tn = t + step;
                load_logits<T, VPL>(logits + (tn < t1 ? tn : 0) * ld, e0, R.E, vec, tn < t1, next);
                float2 stats = make_float2(0.0f, 1.0f);
                if (!choose_by_threshold<T, VPL, MODE>(l, b, logits + t * ld, bias, R, A.slot + i * K,
                                                       A.slot_v + i * K, A.cand, A.found,
                                                       reinterpret_cast<float*>(A.groups), stats, guess))
                    open |= 1u << i;
                if (lane == 0) A.stats[i] = stats;
            }
            __syncwarp();
            // weights of the batch: lane (i, k)
            const int i = lane / lanes, k = lane % lanes;
            const int64_t t = tb + i * step;
            const bool done = t < t1 && !((open >> i) & 1u), on = done && k < K;
            const int e = on ? A.slot[i * K + k] : 0;
            const float x = on ? to_f(logits[t * ld + e]) : 0.0f;
            const float w = lanes == 4 ? weight_of<4>(x, on, A.stats[i], R)
                            : lanes == 8 ? weight_of<8>(x, on, A.stats[i], R) : weight_of<16>(x, on, A.stats[i], R);
            if (on) {
                expert_idx[t * K + k] = e;
                weights[t * K + k] = w;
                atomicAdd(&hist[e], 1);
                if (s_idx) s_idx[t * K + k] = e;
            } else if (t < t1 && k == 0) {
                expert_idx[t * K] = -1;  // left open: below
            }
            __syncwarp();
        }
    } else {
        WarpSmem<float> sm{A.slot, A.slot_v, reinterpret_cast<float*>(A.groups),
                           reinterpret_cast<float*>(A.groups) + 32 / LPT * padded(LPT * VPL)};
        for (int64_t t = t0; t - tok < t1; t += step) {
            const bool valid = t < t1;
            float l[VPL];
#pragma unroll
            for (int j = 0; j < VPL; ++j) l[j] = next[j];
            const int64_t tn = t + step;
            load_logits<T, VPL>(logits + (tn < t1 ? tn : 0) * ld, e0, R.E, vec, tn < t1, next);
            const T* row = logits + (valid ? t : 0) * ld;
            const bool unsure = choose<float, T, LPT, VPL, MODE>(l, row, bias, R, sm);
            constexpr unsigned kMine = (1u << LPT) - 1u;
            const bool open = (__ballot_sync(kFull, unsure) >> (tok * LPT)) & kMine;
            float2 stats = make_float2(0.0f, 1.0f);
            if (!R.sigmoid && !R.renorm) softmax_stats<float, LPT, VPL>(l, e0, R.E, stats.x, stats.y);
            // K experts over LPT lanes, so the sums of a renormalised token take K / LPT turns
            const int* slot = A.slot + tok * K;
            float m = stats.x, z = stats.y;
            if (R.renorm) {
                m = -INFINITY;
                for (int k = sub; k < K; k += LPT) {
                    const float x = to_f(row[slot[k]]);
                    m = fmaxf(m, R.sigmoid && x >= 0.0f ? 0.0f : x);
                }
                m = lanes_max<LPT>(m);
                if (m == -INFINITY) m = 0.0f;
                z = 0.0f;
                for (int k = sub; k < K; k += LPT) {
                    const float x = to_f(row[slot[k]]);
                    const float p = expf((R.sigmoid && x >= 0.0f ? 0.0f : x) - m);
                    z += R.sigmoid ? p / (1.0f + expf(-fabsf(x))) : p;
                }
                z = lanes_sum<LPT>(z);
                if (z == 0.0f) z = 1.0f;
            }
            if (valid && !open) {
                for (int k = sub; k < K; k += LPT) {
                    const int e = slot[k];
                    const float x = to_f(row[e]);
                    float p = expf((R.sigmoid && x >= 0.0f ? 0.0f : x) - m);
                    if (R.sigmoid) p = p / (1.0f + expf(-fabsf(x)));
                    expert_idx[t * K + k] = e;
                    weights[t * K + k] = R.scale * (p / z);
                    atomicAdd(&hist[e], 1);
                    if (s_idx) s_idx[t * K + k] = e;
                }
            } else if (valid && sub == 0) {
                expert_idx[t * K] = -1;
            }
            __syncwarp();
        }
    }
    // the tokens left open, one after the other; a lane looks at one of the warp's tokens
    constexpr int TPW = 32 / LPT;
    const int64_t per_step = TPW, turns = t1 > first ? (t1 - first + step - 1) / step : 0;
    for (int64_t i0 = 0; i0 < turns * per_step; i0 += 32) {
        const int64_t i = i0 + lane, t = first + i / per_step * step + i % per_step;
        const bool mine = i < turns * per_step && t < t1 && expert_idx[t * K] < 0;
        for (unsigned todo = __ballot_sync(kFull, mine); todo; todo &= todo - 1) {
            const int64_t tt = __shfl_sync(kFull, t, __ffs(todo) - 1);
            route_again<T, (LPT == 32 ? VPL : 2), MODE>(logits + tt * ld, tt, vec, bias, R, A.slot, A.slot_v, A.groups, hist,
                                                        expert_idx, weights, s_idx);
        }
    }
}

// Exclusive sums of n <= 256 values (one per thread of the first 256; others pass 0).
__device__ __forceinline__ int exclusive_scan_256(int v, int* s_warp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int u = __shfl_up_sync(kFull, incl, off);
        if (lane >= off) incl += u;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp && w < 8; ++w) before += s_warp[w];
    __syncthreads();
    return before + incl - v;
}

// Writes perm for the n pairs idx[0..n) whose first pair has number p0: the next position
// of expert e is s_base[e], which the whole block fills in bases() once its pairs are
// counted. s_pos: [warps][E]. Pairs of one expert stay in order: a warp has a run of
// consecutive pairs, lanes of one expert are ranked by __match_any_sync.
template <int WARPS, typename F>
__device__ __forceinline__ void scatter_pairs(const int* idx, int n, int32_t p0, int E, const int* s_base, int* s_pos,
                                              int32_t* __restrict__ perm, F bases) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int run = ((n + WARPS - 1) / WARPS + 31) & ~31;
    const int lo = min(n, warp * run), hi = min(n, lo + run);
    int* pos = s_pos + warp * E;
    const unsigned below = (1u << lane) - 1u;
    // four steps' indices are read at once
    constexpr int N = 4;
    int e[N];
    auto read = [&](int i) {
#pragma unroll
        for (int j = 0; j < N; ++j) e[j] = i + 32 * j + lane < hi ? idx[i + 32 * j + lane] : -1;
    };
    read(lo);
    for (int i = lane; i < E; i += 32) pos[i] = 0;
    __syncwarp();
    for (int i = lo; i < hi; i += 32 * N) {
        if (i != lo) read(i);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const unsigned same = __match_any_sync(kFull, e[j]);
            if (e[j] >= 0 && (same & below) == 0) pos[e[j]] += __popc(same);
            __syncwarp();
        }
    }
    bases();
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += WARPS * 32) {
        int at = s_base[e];
        for (int w = 0; w < WARPS; ++w) {
            const int c = s_pos[w * E + e];
            s_pos[w * E + e] = at;
            at += c;
        }
    }
    __syncthreads();
    for (int i = lo; i < hi; i += 32 * N) {
        if (hi - lo > 32 * N) read(i);  // else they are still here
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const unsigned same = __match_any_sync(kFull, e[j]);
            const int at = e[j] >= 0 ? pos[e[j]] : 0;
            if (e[j] >= 0) perm[at + __popc(same & below)] = p0 + i + 32 * j + lane;
            __syncwarp();
            if (e[j] >= 0 && (same & below) == 0) pos[e[j]] = at + __popc(same);
            __syncwarp();
        }
    }
}

// ---------------------------------------------------------------- kernels
// Tokens [b * tpb, (b + 1) * tpb) of block b; blk_counts [gridDim.x][E].
template <typename T, int LPT, int VPL, int MODE>
__global__ void __launch_bounds__(kThreads, 4)
topk_route_kernel(const T* __restrict__ logits, int64_t ld, int64_t T_, int tpb, bool vec,
                  const float* __restrict__ bias, Rule R, int32_t* __restrict__ expert_idx,
                  float* __restrict__ weights, int32_t* __restrict__ blk_counts) {
    griddep_wait();  // every global access below comes after the previous grid
    extern __shared__ __align__(16) uint8_t smem[];
    int* hist = reinterpret_cast<int*>(smem);
    const int warp = threadIdx.x >> 5, tok = (threadIdx.x & 31) / LPT;
    const WarpArea A = warp_area(smem + kMaxE * 4 + warp * warp_bytes(R, LPT, VPL), LPT, R.K);
    constexpr int TPW = 32 / LPT;
    for (int e = threadIdx.x; e < R.E; e += kThreads) hist[e] = 0;
    __syncthreads();
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tpb;
    const int64_t t1 = t0 + tpb < T_ ? t0 + tpb : T_;
    route_tokens<T, LPT, VPL, MODE>(logits, ld, t0 + warp * TPW + tok, t1, kWarps * TPW, vec, bias, R, A, hist, expert_idx,
                                    weights, nullptr);
    __syncthreads();
    for (int e = threadIdx.x; e < R.E; e += kThreads) blk_counts[static_cast<int64_t>(blockIdx.x) * R.E + e] = hist[e];
}

// One block: routes every token, then counts, offsets and perm.
template <typename T, int LPT, int VPL, int MODE>
__global__ void __launch_bounds__(kSmallThreads)
topk_route_small_kernel(const T* __restrict__ logits, int64_t ld, int T_, bool vec, const float* __restrict__ bias,
                        Rule R, int32_t* __restrict__ expert_idx, float* __restrict__ weights,
                        int32_t* __restrict__ counts, int32_t* __restrict__ offsets, int32_t* __restrict__ perm) {
    griddep_wait();  // every global access below comes after the previous grid
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int s_warp[32];
    __shared__ int s_base[kMaxE];
    constexpr int TPW = 32 / LPT, WARPS = kSmallThreads / 32;
    int* hist = reinterpret_cast<int*>(smem);
    int* s_idx = hist + kMaxE;                                       // [T * K]
    uint8_t* areas = reinterpret_cast<uint8_t*>(s_idx + (T_ * R.K + 3) / 4 * 4);  // slots, then scatter positions
    const int warp = threadIdx.x >> 5, tok = (threadIdx.x & 31) / LPT;
    const WarpArea A = warp_area(areas + warp * warp_bytes(R, LPT, VPL), LPT, R.K);
    for (int e = threadIdx.x; e < R.E; e += kSmallThreads) hist[e] = 0;
    __syncthreads();
    route_tokens<T, LPT, VPL, MODE>(logits, ld, warp * TPW + tok, T_, WARPS * TPW, vec, bias, R, A, hist, expert_idx, weights,
                                    s_idx);
    __syncthreads();
    const int e = threadIdx.x;
    const int c = e < R.E ? hist[e] : 0;
    const int off = exclusive_scan_256(c, s_warp);
    if (e < R.E) {
        counts[e] = c;
        offsets[e] = off;
        s_base[e] = off;
    }
    if (e == 0) offsets[R.E] = T_ * R.K;
    __syncthreads();
    scatter_pairs<WARPS>(s_idx, T_ * R.K, 0, R.E, s_base, reinterpret_cast<int*>(areas), perm, [] {});
}

// 32 experts a block (a lane each), the routing blocks in 32 runs (a warp each): sums of
// the runs, then every block's base inside its expert and the expert's count.
__global__ void __launch_bounds__(1024) topk_scan_kernel(const int32_t* __restrict__ blk_counts, int nblk, int E,
                                                         int32_t* __restrict__ blk_base, int32_t* __restrict__ counts) {
    griddep_wait();  // every global access below comes after the previous grid
    __shared__ int s_run[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
    const int run = (nblk + 31) / 32, lo = warp * run, hi = min(nblk, lo + run);
    constexpr int N = kMaxBlocks / 32;  // blocks of a run at most; their counts stay in registers
    int c[N], sum = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        c[i] = lo + i < hi && e < E ? blk_counts[static_cast<int64_t>(lo + i) * E + e] : 0;
        sum += c[i];
    }
    s_run[warp][lane] = sum;
    __syncthreads();
    int at = 0;
    for (int w = 0; w < warp; ++w) at += s_run[w][lane];
    if (e < E) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (lo + i < hi) blk_base[static_cast<int64_t>(lo + i) * E + e] = at;
            at += c[i];
        }
        if (warp == 31) counts[e] = at;
    }
}

__global__ void __launch_bounds__(kThreads)
topk_scatter_kernel(const int32_t* __restrict__ expert_idx, int64_t pairs, int ppb, int E,
                    const int32_t* __restrict__ blk_base, const int32_t* __restrict__ counts,
                    int32_t* __restrict__ offsets, int32_t* __restrict__ perm) {
    griddep_wait();  // every global access below comes after the previous grid
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int s_warp[32];
    __shared__ int s_base[kMaxE];
    const int e = threadIdx.x;
    // on the way while the pairs are counted
    const int count = e < E ? counts[e] : 0;
    const int before = e < E ? blk_base[static_cast<int64_t>(blockIdx.x) * E + e] : 0;
    if (blockIdx.x == 0 && e == 0) offsets[E] = static_cast<int32_t>(pairs);
    const int64_t p0 = static_cast<int64_t>(blockIdx.x) * ppb;
    const int n = static_cast<int>(pairs - p0 < ppb ? pairs - p0 : ppb);
    scatter_pairs<kWarps>(expert_idx + p0, n, static_cast<int32_t>(p0), E, s_base, reinterpret_cast<int*>(smem), perm, [&] {
        const int off = exclusive_scan_256(count, s_warp);
        if (e < E) {
            s_base[e] = off + before;
            if (blockIdx.x == 0) offsets[e] = off;
        }
    });
}

// Gradient of the logits: a token per LPT lanes, its row of gradients built in shared
// memory (zeros and the K chosen entries) and written as a whole. 262,144 x 8 fp32, K = 2,
// softmax: 5.8 us for 21 MB (3.6 TB/s, from L2 as a step finds it); 20,479 x 60 bf16, K = 4:
// 5.8 us, a chain of three dependent loads.
//   renormalised: d l_k = w_k (g_k - sum_j w_j g_j) for the chosen, w summing to 1, times
//   (1 - s_k) for the sigmoid; softmax: d l_e = s_e (g_e - sum_j s_j g_j), g = 0 for the
//   others; sigmoid: g_k s_k (1 - s_k).  g: the weight's gradient times scale.
// A lane has chunks of C experts, LPT chunks apart: 16 bytes of them where the rows allow it,
// two, or one (204,600 x 82 fp16, K 7, softmax: 45 us with two, 70 with a lane's 16 in a row).
template <typename T, int LPT, int VPL, int C>
__global__ void __launch_bounds__(kThreads)
topk_route_bwd_kernel(const T* __restrict__ logits, int64_t ld, int64_t T_, Rule R, const int32_t* __restrict__ expert_idx,
                      const float* __restrict__ d_weights, T* d_logits, int accumulate) {
    griddep_wait();  // every global access below comes after the previous grid
    __shared__ __align__(16) float s_row[kWarps][32 * VPL];
    constexpr int TPW = 32 / LPT;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % LPT, tok = lane / LPT;
    float* row_d = s_row[warp] + tok * LPT * VPL;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps * TPW;
    for (int64_t base = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * TPW; base < T_; base += step) {
        const int64_t t = base + tok;
        const bool valid = t < T_;
        const T* row = logits + (valid ? t : 0) * ld;
#pragma unroll
        for (int j = 0; j < VPL; ++j) row_d[j * LPT + sub] = 0.0f;
        __syncwarp();
        auto pair = [&](int k, int& e, float& g) {  // an index outside the row is left out
            e = valid ? expert_idx[t * R.K + k] : -1;
            if (static_cast<unsigned>(e) >= static_cast<unsigned>(R.E)) e = -1;
            g = valid ? R.scale * d_weights[t * R.K + k] : 0.0f;
        };
        int e;
        float g;
        if (R.renorm) {
            float m = -INFINITY, z = 0.0f, dot = 0.0f;
            auto unnormalised = [&](float x) {
                const float p = expf((R.sigmoid && x >= 0.0f ? 0.0f : x) - m);
                return R.sigmoid ? p / (1.0f + expf(-fabsf(x))) : p;
            };
            for (int k = sub; k < R.K; k += LPT) {
                pair(k, e, g);
                if (e >= 0) {
                    const float x = to_f(row[e]);
                    m = fmaxf(m, R.sigmoid ? fminf(x, 0.0f) : x);
                }
            }
            m = lanes_max<LPT>(m);
            if (m == -INFINITY) m = 0.0f;
            for (int k = sub; k < R.K; k += LPT) {
                pair(k, e, g);
                if (e >= 0) z += unnormalised(to_f(row[e]));
            }
            z = lanes_sum<LPT>(z);
            if (z == 0.0f) z = 1.0f;
            // the weights are quotients: a weight of 1 is exactly 1, and its gradient exactly 0
            for (int k = sub; k < R.K; k += LPT) {
                pair(k, e, g);
                if (e >= 0) dot += unnormalised(to_f(row[e])) / z * g;
            }
            dot = lanes_sum<LPT>(dot);
            for (int k = sub; k < R.K; k += LPT) {
                pair(k, e, g);
                if (e >= 0) {
                    const float x = to_f(row[e]);
                    float d = unnormalised(x) / z * (g - dot);
                    if (R.sigmoid) d /= 1.0f + expf(x);
                    row_d[e] = d;
                }
            }
        } else if (R.sigmoid) {
            for (int k = sub; k < R.K; k += LPT) {
                pair(k, e, g);
                if (e >= 0) {
                    const float x = to_f(row[e]), q = expf(-fabsf(x));
                    row_d[e] = g * (q / ((1.0f + q) * (1.0f + q)));  // s (1 - s), the same for x and -x
                }
            }
        } else {
            for (int k = sub; k < R.K; k += LPT) {
                pair(k, e, g);
                if (e >= 0) row_d[e] = g;
            }
            __syncwarp();
            float l[VPL], mx = -INFINITY, z = 0.0f, dot = 0.0f;
#pragma unroll
            for (int j = 0; j < VPL; j += C) {
                const int c = j * LPT + sub * C;
                Chunk<T, C> x;
                const bool on = valid && c < R.E;
                if (on) x = *reinterpret_cast<const Chunk<T, C>*>(row + c);
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    l[j + i] = on ? to_f(x.v[i]) : -INFINITY;
                    if (l[j + i] > mx) mx = l[j + i];
                }
            }
            mx = lanes_max<LPT>(mx);
            if (mx == -INFINITY) mx = 0.0f;
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                l[j] = expf(l[j] - mx);
                z += l[j];
            }
            z = lanes_sum<LPT>(z);
            const float inv = z == 0.0f ? 1.0f : 1.0f / z;
#pragma unroll
            for (int j = 0; j < VPL; j += C)
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    l[j + i] *= inv;
                    dot += l[j + i] * row_d[j * LPT + sub * C + i];
                }
            dot = lanes_sum<LPT>(dot);
#pragma unroll
            for (int j = 0; j < VPL; j += C)
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    float& d = row_d[j * LPT + sub * C + i];
                    d = l[j + i] * (d - dot);
                }
        }
        __syncwarp();
        if (valid) {
            T* out = d_logits + t * R.E;
#pragma unroll
            for (int j = 0; j < VPL; j += C) {
                const int c = j * LPT + sub * C;
                if (c >= R.E) continue;
                Chunk<T, C> o;
                if (accumulate) o = *reinterpret_cast<const Chunk<T, C>*>(out + c);
#pragma unroll
                for (int i = 0; i < C; ++i) o.v[i] = from_f<T>((accumulate ? to_f(o.v[i]) : 0.0f) + row_d[c + i]);
                *reinterpret_cast<Chunk<T, C>*>(out + c) = o;
            }
        }
        __syncwarp();
    }
}

// ---------------------------------------------------------------- launches
struct RouteArgs {
    const void* logits;
    int64_t ld, T;
    bool vec;
    const float* bias;
    Rule R;
    moe_routing_t out;
    float* weights;
    int32_t* blk_counts;
    int32_t* blk_base;
};

// Shared memory of the one-block kernel, 0 where there are too many tokens for it: at most
// four a warp.
int small_smem(const RouteArgs& a, int warp_area) {
    if (a.T > 4 * (kSmallThreads / 32) || a.T * a.R.K > kSmallPairs) return 0;
    const int per_warp = warp_area > a.R.E * 4 ? warp_area : a.R.E * 4;
    const int smem = kMaxE * 4 + (static_cast<int>(a.T) * a.R.K + 3) / 4 * 16 + kSmallThreads / 32 * per_warp;
    return smem <= 200 * 1024 ? smem : 0;
}

template <typename T, int VPL, int MODE>
cudaError_t route_small(const RouteArgs& a, int smem, cudaStream_t s) {
    auto kernel = topk_route_small_kernel<T, 32, VPL, MODE>;
    static std::atomic<uint64_t> ready;
    cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kernel), 200 * 1024, ready);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(1), dim3(kSmallThreads), smem, s, static_cast<const T*>(a.logits), a.ld,
                      static_cast<int>(a.T), a.vec, a.bias, a.R, a.out.expert_idx, a.weights, a.out.counts, a.out.offsets,
                      a.out.perm);
}

template <typename T, int LPT, int VPL, int MODE>
cudaError_t route_launch(const RouteArgs& a, cudaStream_t s) {
    const Rule& R = a.R;
    const int wb = warp_bytes(R, LPT, VPL);
    int sms = 0;
    cudaError_t e = device_sms(&sms);
    if (e != cudaSuccess) return e;
    // tokens per block: whole steps of the block's warps, four blocks an SM where there are enough
    constexpr int step = kWarps * (32 / LPT);
    const int64_t steps = (a.T + step - 1) / step;
    int64_t want = static_cast<int64_t>(sms) * 4;
    if (want > kMaxBlocks) want = kMaxBlocks;
    const int64_t per = (steps + want - 1) / want;
    const int tpb = static_cast<int>(per) * step;
    const int nblk = static_cast<int>((a.T + tpb - 1) / tpb);
    const int smem = kMaxE * 4 + kWarps * wb;
    auto kernel = topk_route_kernel<T, LPT, VPL, MODE>;
    static std::atomic<uint64_t> ready;
    e = set_smem_once(reinterpret_cast<const void*>(kernel), 128 * 1024, ready);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kernel, dim3(nblk), dim3(kThreads), smem, s, static_cast<const T*>(a.logits), a.ld, a.T, tpb, a.vec,
                   a.bias, R, a.out.expert_idx, a.weights, a.blk_counts);
    if (e != cudaSuccess) return e;
    e = launch_pdl(topk_scan_kernel, dim3((R.E + 31) / 32), dim3(1024), 0, s, a.blk_counts, nblk, R.E, a.blk_base,
                   a.out.counts);
    if (e != cudaSuccess) return e;
    return launch_pdl(topk_scatter_kernel, dim3(nblk), dim3(kThreads), kWarps * R.E * 4, s, a.out.expert_idx,
                      a.T * R.K, tpb * R.K, R.E, a.blk_base, a.out.counts, a.out.offsets, a.out.perm);
}

// Few tokens: one block, a warp per token (the shortest chain). Many: a token per 1 to 8
// lanes up to 64 experts, where a warp's rounds serve several tokens, a warp per token above.
template <typename T, int MODE>
cudaError_t route_width(const RouteArgs& a, cudaStream_t s) {
    const int E = a.R.E, vpl = E <= 64 ? 2 : E <= 128 ? 4 : 8;
    if (const int smem = small_smem(a, warp_bytes(a.R, 32, vpl))) {
        if (vpl == 2) return route_small<T, 2, MODE>(a, smem, s);
        if (vpl == 4) return route_small<T, 4, MODE>(a, smem, s);
        return route_small<T, 8, MODE>(a, smem, s);
    }
    if (E <= 8) return route_launch<T, 1, 8, MODE>(a, s);
    if (E <= 16) return route_launch<T, 2, 8, MODE>(a, s);
    if (E <= 32) return route_launch<T, 4, 8, MODE>(a, s);
    if (E <= 64) return route_launch<T, 8, 8, MODE>(a, s);
    if (E <= 128) return route_launch<T, 32, 4, MODE>(a, s);
    return route_launch<T, 32, 8, MODE>(a, s);
}

template <typename T>
cudaError_t route_type(const RouteArgs& a, cudaStream_t s) {
    const bool scores = a.bias || (a.R.G > 1 && a.R.best == 2);
    return !scores ? route_width<T, kLogits>(a, s) : a.R.sigmoid ? route_width<T, kSigmoid>(a, s) : route_width<T, kSoftmax>(a, s);
}

template <typename T, int C>
cudaError_t route_bwd_width(const void* logits, int64_t ld, int64_t T_, const Rule& R, const int32_t* idx, const float* dw,
                            void* out, int acc, cudaStream_t s) {
    int sms = 0;
    cudaError_t e = device_sms(&sms);
    if (e != cudaSuccess) return e;
    auto go = [&](auto kernel, int lpt) {
        const int64_t tokens = kWarps * (32 / lpt), want = (T_ + tokens - 1) / tokens, cap = static_cast<int64_t>(sms) * 8;
        return launch_pdl(kernel, dim3(static_cast<unsigned>(want < cap ? want : cap)), dim3(kThreads), 0, s,
                          static_cast<const T*>(logits), ld, T_, R, idx, dw, static_cast<T*>(out), acc);
    };
    if (R.E <= 8) return go(topk_route_bwd_kernel<T, 1, 8, C>, 1);
    if (R.E <= 16) return go(topk_route_bwd_kernel<T, 1, 16, C>, 1);
    if (R.E <= 32) return go(topk_route_bwd_kernel<T, 2, 16, C>, 2);
    if (R.E <= 64) return go(topk_route_bwd_kernel<T, 4, 16, C>, 4);
    if (R.E <= 128) return go(topk_route_bwd_kernel<T, 8, 16, C>, 8);
    return go(topk_route_bwd_kernel<T, 16, 16, C>, 16);
}

template <typename T>
cudaError_t route_bwd_type(const void* logits, int64_t ld, int64_t T_, const Rule& R, const int32_t* idx, const float* dw,
                           void* out, int acc, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    auto fits = [&](int c) {  // every row of either array starts on c values
        return R.E % c == 0 && ld % c == 0 && aligned(logits, c * sizeof(T)) && aligned(out, c * sizeof(T));
    };
    if (fits(V)) return route_bwd_width<T, V>(logits, ld, T_, R, idx, dw, out, acc, s);
    if (fits(2)) return route_bwd_width<T, 2>(logits, ld, T_, R, idx, dw, out, acc, s);
    return route_bwd_width<T, 1>(logits, ld, T_, R, idx, dw, out, acc, s);
}

moe_status_t check_rule(const moe_topk_rule_t* r, Rule* out) {
    if (!r) return MOE_ERR_INVALID_ARG;
    if (r->score != MOE_SCORE_SOFTMAX && r->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
    if (r->flags & ~MOE_TOPK_RENORM) return MOE_ERR_INVALID_ARG;
    if (!std::isfinite(r->scale)) return MOE_ERR_INVALID_ARG;
    if (r->E < 1 || r->E > kMaxE || r->K < 1 || r->K > kMaxK || r->K > r->E) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (r->groups < 1 || r->groups > kMaxGroups || r->E % r->groups != 0) return MOE_ERR_UNSUPPORTED_SHAPE;
    const int S = r->E / r->groups;
    if (r->top_groups < 1 || r->top_groups > r->groups || r->top_groups * S < r->K) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (r->group_best < 1 || r->group_best > 2 || r->group_best > S) return MOE_ERR_UNSUPPORTED_SHAPE;
    *out = Rule{r->E, r->K, r->groups, S, r->top_groups, r->group_best, r->score == MOE_SCORE_SIGMOID ? 1 : 0,
                (r->flags & MOE_TOPK_RENORM) ? 1 : 0, r->scale};
    if (r->top_groups == r->groups) out->G = 1, out->S = r->E, out->top_groups = 1;  // every group stays
    return MOE_OK;
}

moe_status_t check_tokens(int64_t T, int64_t ld, int E, int K, moe_dtype_t dtype) {
    if (T < 0 || ld < E || !dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
    if (T >= kMaxT / K || ld > (int64_t{1} << 31)) return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

bool rows_vec(const void* p, int E, int64_t ld, size_t b) {
    const int c = static_cast<int>(16 / b);
    return E % c == 0 && ld % c == 0 && aligned(p, 16);
}

size_t strided_bytes(int64_t T, int64_t n, int64_t ld, size_t b) {
    return T > 0 ? (static_cast<size_t>(T - 1) * ld + n) * b : 0;
}

}  // namespace

size_t topk_route_ws_bytes(int64_t T, int E) {
    const int64_t blocks = T < kMaxBlocks ? T : kMaxBlocks;
    return 256 + 2 * align_up(static_cast<size_t>(blocks) * E * sizeof(int32_t), 256);
}

}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_topk_route(const void* logits, moe_dtype_t dtype, int64_t T, int64_t ld, const moe_topk_rule_t* rule,
                            const float* bias, const moe_routing_t* out, float* weights, void* workspace,
                            size_t workspace_bytes, void* stream) {
    RouteArgs a{};
    moe_status_t st = check_rule(rule, &a.R);
    if (st == MOE_OK) st = check_tokens(T, ld, a.R.E, a.R.K, dtype);
    if (st != MOE_OK) return st;
    const int E = a.R.E, K = a.R.K;
    if (!out || !out->counts || !out->offsets) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!logits || !weights || !out->expert_idx || !out->perm)) return MOE_ERR_INVALID_ARG;
    const size_t b = dtype_bytes(dtype);
    if (!aligned(logits, b) || !aligned(bias, 4) || !aligned(weights, 4) || !aligned(out->expert_idx, 4) ||
        !aligned(out->counts, 4) || !aligned(out->offsets, 4) || !aligned(out->perm, 4))
        return MOE_ERR_MISALIGNED;
    const size_t pairs = static_cast<size_t>(T) * K;
    const Range outs[6] = {{out->expert_idx, 4 * pairs}, {out->counts, sizeof(int32_t) * E},
                           {out->offsets, sizeof(int32_t) * (E + 1)}, {out->perm, 4 * pairs},
                           {weights, 4 * pairs},       {workspace, workspace ? workspace_bytes : 0}};
    const Range ins[2] = {{logits, strided_bytes(T, E, ld, b)}, {bias, sizeof(float) * E}};
    if (any_alias(outs, 6, ins, 2)) return MOE_ERR_ALIAS;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        cudaError_t e = cudaMemsetAsync(out->counts, 0, sizeof(int32_t) * E, s);
        if (e == cudaSuccess) e = cudaMemsetAsync(out->offsets, 0, sizeof(int32_t) * (E + 1), s);
        return cuda_status(e);
    }
    if (!workspace) return MOE_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return MOE_ERR_MISALIGNED;
    const size_t need = topk_route_ws_bytes(T, E);
    if (workspace_bytes < need) return MOE_ERR_WORKSPACE;
    a.logits = logits;
    a.ld = ld;
    a.T = T;
    a.vec = rows_vec(logits, E, ld, b);
    a.bias = bias;
    a.out = *out;
    a.weights = weights;
    a.blk_counts = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + 256);
    a.blk_base = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + 256 + (need - 256) / 2);
    if (dtype == MOE_DTYPE_F32) return cuda_status(route_type<float>(a, s));
    if (dtype == MOE_DTYPE_BF16) return cuda_status(route_type<__nv_bfloat16>(a, s));
    return cuda_status(route_type<__half>(a, s));
}

moe_status_t moe_topk_route_bwd(const void* logits, moe_dtype_t dtype, int64_t T, int64_t ld,
                                const moe_topk_rule_t* rule, const int32_t* expert_idx, const float* d_weights,
                                void* d_logits, int32_t accumulate, void* stream) {
    Rule R;
    moe_status_t st = check_rule(rule, &R);
    if (st == MOE_OK) st = check_tokens(T, ld, R.E, R.K, dtype);
    if (st != MOE_OK) return st;
    if (T > 0 && (!logits || !expert_idx || !d_weights || !d_logits)) return MOE_ERR_INVALID_ARG;
    const size_t b = dtype_bytes(dtype), pairs = static_cast<size_t>(T) * R.K;
    if (!aligned(logits, b) || !aligned(d_logits, b) || !aligned(expert_idx, 4) || !aligned(d_weights, 4))
        return MOE_ERR_MISALIGNED;
    const Range outs[1] = {{d_logits, static_cast<size_t>(T) * R.E * b}};
    const Range ins[3] = {{logits, strided_bytes(T, R.E, ld, b)}, {expert_idx, 4 * pairs}, {d_weights, 4 * pairs}};
    if (any_alias(outs, 1, ins, 3)) return MOE_ERR_ALIAS;
    if (T == 0) return MOE_OK;
    const int acc = accumulate ? 1 : 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == MOE_DTYPE_F32)
        return cuda_status(route_bwd_type<float>(logits, ld, T, R, expert_idx, d_weights, d_logits, acc, s));
    if (dtype == MOE_DTYPE_BF16)
        return cuda_status(route_bwd_type<__nv_bfloat16>(logits, ld, T, R, expert_idx, d_weights, d_logits, acc, s));
    return cuda_status(route_bwd_type<__half>(logits, ld, T, R, expert_idx, d_weights, d_logits, acc, s));
}

}  // extern "C"
