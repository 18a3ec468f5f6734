// topk_plan.h -- how the experts' kernels of the top-k block cut their work, and the
// workspace that goes with it.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "internal.h"
#include "moe_topk.h"

namespace moe {

// Weight gradient: dW[e] is cut into kWTile x kWTile tiles, and the pairs of an expert
// into pieces (see wgrad_pieces); a piece's tile is one unit of work.
constexpr int kWTile = 256;
constexpr int kWMinPiece = 128;  // pairs a piece of a cut expert has at least
constexpr int kWUnits = 148;     // units that fill the GPU

inline int wgrad_tiles(int H) {
    const int n = (H + kWTile - 1) / kWTile;
    return n * n;
}
// Pieces beyond one per expert that the experts share in proportion to their pairs. With few
// tiles, as many as fill the GPU once; with several tiles an expert, half as many experts as fill
// it or more, and pairs enough, as many as fill it twice, since experts of uneven sizes would
// leave the one turn to the largest; where the experts alone fill it, one is cut where its tiles
// would take a block longer than an even share of all the work. dW, filled once / twice, uneven
// experts: 25,780 tokens, K 1, E 13, H 640: 206 / 86 us; 12,000, K 2, E 30, H 512 (648 pairs a
// piece): 72 / 62; 2,000, K 2, E 8, H 1024 (444): 37 / 45; 4,500, K 1, E 13, H 640 (281): 40 / 46.
// Even experts lose by it (25,780 tokens: 64 / 86).
inline int wgrad_extra(int64_t P, int E, int H) {
    const int tiles = wgrad_tiles(H), fill = kWUnits / tiles;
    if (E >= fill) return fill;
    const bool twice = tiles > 1 && 2 * E > fill && P >= 512 * static_cast<int64_t>(fill);
    return (twice ? 2 : 1) * fill - E;
}
// Pieces of an expert with n of the P pairs: at most E + extra in all.
__host__ __device__ inline int wgrad_pieces(int n, int64_t P, int extra) {
    if (n <= 0) return 0;
    int q = 1 + static_cast<int>(static_cast<int64_t>(n) * extra / P);
    const int most = n / kWMinPiece;
    if (q > most) q = most < 1 ? 1 : most;
    return q;
}

struct ExpertsWs {
    size_t rows = 0;     // float [T * K][H]: the pairs' rows, K > 1
    size_t dw_part = 0;  // float [ceil(H / 64) + 1][T * K]: column parts of the weights' gradient
    size_t duo = 0;      // int32 [3 * E * E + 1], K = 2: classes of tokens
    size_t list = 0;     // int32 [T], K = 2: tokens by class
    size_t part = 0;     // float [2 * extra][H][H]
    size_t part_db = 0;  // float [2 * extra][H]
    size_t starts = 0;   // int32 [E + 1]: first slot of each expert
    size_t peak = 0;     // uint32 [E]: bits of each expert's largest |w g|, fp16
    size_t total = 0;
};

inline ExpertsWs experts_ws(int64_t T, int E, int K, int H, size_t begin) {
    ExpertsWs L;
    const size_t P = static_cast<size_t>(T) * K, nb = static_cast<size_t>((H + 63) / 64 + 1);
    const size_t slots = 2 * static_cast<size_t>(wgrad_extra(T * K, E, H));
    size_t off = align_up(begin, 256);
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align_up(off + bytes, 256);
        return at;
    };
    L.rows = take(K > 1 ? sizeof(float) * P * H : 0);
    L.dw_part = take(sizeof(float) * nb * P);
    L.duo = take(K == 2 ? sizeof(int32_t) * (3 * static_cast<size_t>(E) * E + 1) : 0);
    L.list = take(K == 2 ? sizeof(int32_t) * T : 0);
    L.part = take(sizeof(float) * slots * H * H);
    L.part_db = take(sizeof(float) * slots * H);
    L.starts = take(sizeof(int32_t) * (static_cast<size_t>(E) + 1));
    L.peak = take(sizeof(uint32_t) * static_cast<size_t>(E));
    L.total = off;
    return L;
}

}  // namespace moe
