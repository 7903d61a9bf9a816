// The adapters' first product, t[m][j] = sum_k x[m][k] A[a][j][k]: what the kernel in front of the fused path and the
// weight-streaming kernel share of it, and the latter's tasks, which its drain warps do beside the stream.
#pragma once

#include "ql_common.cuh"

namespace ql {
namespace lora {

constexpr int kTile = 16;              // rows of one tile (MMA M)
constexpr int kMaxRank = 128;

// D (16 x 8, fp32) += A (16 x 16, bf16) . B (16 x 8, bf16)
__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 rows x 8 ranks over 32 columns: lane (g, c) holds 16 bytes, columns 8c .. 8c+7, of rows g and g + 8 and of rank
// g.  The MMA's k order is whatever the lanes hold, the same for both operands, so a dot product keeps its terms.
__device__ __forceinline__ void dot_block(float (&d)[4], const uint4 x0, const uint4 x1, const uint4 a) {
    mma_bf16_16816(d, x0.x, x1.x, x0.y, x1.y, a.x, a.y);
    mma_bf16_16816(d, x0.z, x1.z, x0.w, x1.w, a.z, a.w);
}

// The adapter of row m, -1 for none; an id outside [-1, L) is recorded and counts as none.
__device__ __forceinline__ int adapter_of(const int* ids, int m, int L) {
    const int a = ids[m];
    if (a >= -1 && a < L) return a;
    record_status(QL_ERR_INVALID_ARG);
    return -1;
}

// The weight-streaming path's first product (M <= 64), as tasks of one warp each: (member of a gate/up pair, row tile,
// n-th distinct adapter of the tile, 16 ranks, K slice).  The slices' partial sums are added in order by the kernel that
// uses them.
struct DotTasks {
    const __nv_bfloat16* x;      // [M][K]
    const __nv_bfloat16* a[2];   // [L][r][K] of each member
    const int* ids;              // [M]
    float* tp;                   // [slices][pairs][M][r]
    int M, K, r, L, pairs;
    int per_tile;                // tasks are laid out for this many distinct adapters in a tile
    int chunks;                  // ceil(r / 16)
    int slices;
};

__device__ __forceinline__ void run_dot_tasks(const DotTasks& p, int worker, int workers) {
    const int lane = static_cast<int>(threadIdx.x & 31), g = lane >> 2, c = lane & 3;
    const int tiles = (p.M + kTile - 1) / kTile;
    const int kb_all = p.K / 32;
    for (int task = worker; task < p.pairs * tiles * p.per_tile * p.chunks * p.slices; task += workers) {
        const int z = task % p.slices;
        int rest = task / p.slices;
        const int j0 = (rest % p.chunks) * 16;
        rest /= p.chunks;
        const int nth = rest % p.per_tile;
        rest /= p.per_tile;
        const int m0 = (rest % tiles) * kTile, pair = rest / tiles;
        const int mine = lane < kTile && m0 + lane < p.M ? adapter_of(p.ids, m0 + lane, p.L) : -1;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, mine);
        uint32_t leaders = __ballot_sync(0xFFFFFFFFu, mine >= 0 && (__ffs(same) - 1) == lane);
        for (int n = 0; n < nth; ++n) leaders &= leaders - 1;
        if (leaders == 0) continue;
        const int adapter = __shfl_sync(0xFFFFFFFFu, mine, __ffs(leaders) - 1);
        const int id0 = __shfl_sync(0xFFFFFFFFu, mine, g), id1 = __shfl_sync(0xFFFFFFFFu, mine, g + 8);
        const int kb1 = static_cast<int>(static_cast<int64_t>(kb_all) * (z + 1) / p.slices);
        int kb = static_cast<int>(static_cast<int64_t>(kb_all) * z / p.slices);
        // rows past M repeat the last one, ranks past r the first; neither is written
        const uint4* x0 = reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(min(m0 + g, p.M - 1)) * p.K) + c;
        const uint4* x1 = reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(min(m0 + g + 8, p.M - 1)) * p.K) + c;
        const bool second = j0 + 8 < p.r;
        const uint4* a0 = reinterpret_cast<const uint4*>((pair == 0 ? p.a[0] : p.a[1]) + (static_cast<int64_t>(adapter) * p.r + j0 + g) * p.K) + c;
        const uint4* a1 = second ? a0 + static_cast<int64_t>(p.K) : a0;          // 8 rows of K bf16 further
        float d0[4] = {0.0f, 0.0f, 0.0f, 0.0f}, d1[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        constexpr int U = 3;                       // column blocks in flight
        for (; kb + U <= kb1; kb += U) {
            uint4 vx0[U], vx1[U], va0[U], va1[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                vx0[u] = __ldg(x0 + 4 * (kb + u));
                vx1[u] = __ldg(x1 + 4 * (kb + u));
                va0[u] = __ldg(a0 + 4 * (kb + u));
                va1[u] = __ldg(a1 + 4 * (kb + u));
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                dot_block(d0, vx0[u], vx1[u], va0[u]);
                dot_block(d1, vx0[u], vx1[u], va1[u]);
            }
        }
        for (; kb < kb1; ++kb) {
            const uint4 vx0 = __ldg(x0 + 4 * kb), vx1 = __ldg(x1 + 4 * kb);
            dot_block(d0, vx0, vx1, __ldg(a0 + 4 * kb));
            dot_block(d1, vx0, vx1, __ldg(a1 + 4 * kb));
        }
        const int64_t at = ((static_cast<int64_t>(z) * p.pairs + pair) * p.M + m0) * p.r + j0 + 2 * c;
        if (!in_bounds(at, static_cast<int64_t>(p.slices) * p.pairs * p.M * p.r)) continue;
        float* out = p.tp + at;
        if (id0 == adapter) {
            *reinterpret_cast<float2*>(out + g * p.r) = make_float2(d0[0], d0[1]);
            if (second) *reinterpret_cast<float2*>(out + g * p.r + 8) = make_float2(d1[0], d1[1]);
        }
        if (id1 == adapter) {
            *reinterpret_cast<float2*>(out + (g + 8) * p.r) = make_float2(d0[2], d0[3]);
            if (second) *reinterpret_cast<float2*>(out + (g + 8) * p.r + 8) = make_float2(d1[2], d1[3]);
        }
    }
}

}  // namespace lora
}  // namespace ql
